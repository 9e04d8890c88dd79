// avey_quant.cuh -- the 8-bit rounding shared by avey_quantize_rows and the
// products that quantise their own input.
#pragma once

#include "avey_common.cuh"
#include "avey_internal.h"

namespace avey {

// Whether every row of x (both planes of a pair) is whole groups of 8 values on
// 16-byte boundaries.
inline bool quant_rows_fast(const void *x, int dt, long long rows, int cols, long long ld) {
  const long long es = dt == AVEY_F32 ? 4 : 2;
  return cols % 8 == 0 && aligned16(x) && (ld * es) % 16 == 0 && (dt != AVEY_BF16X2 || (rows * ld * es) % 16 == 0);
}

// Eight consecutive values of a row as they lie in memory.
template <int DT>
struct QuantRaw {
  uint4 w[DT == AVEY_BF16 ? 1 : 2];  // fp32: two words; pair: hi and lo

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (auto &x : w) x = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (DT == AVEY_F32) {
      const uint32_t a[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a[i]);
    } else {
      const uint32_t a[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
      }
      if constexpr (DT == AVEY_BF16X2) {
        const uint32_t b[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 t = fadd2(make_float2(v[2 * i], v[2 * i + 1]),
                                 make_float2(__uint_as_float(b[i] << 16), __uint_as_float(b[i] & 0xffff0000u)));
          v[2 * i] = t.x;
          v[2 * i + 1] = t.y;
        }
      }
    }
  }
};

// One row of x, in groups of 8 consecutive values; values past the row's end
// are 0.  FAST: rows of whole groups on 16-byte boundaries.
template <int DT, bool FAST>
struct QuantSource {
  const float *f = nullptr;
  const bf16 *h = nullptr, *l = nullptr;
  int cols;

  __device__ __forceinline__ QuantSource(const void *x, long long row, long long rows, int cols_, long long ld)
      : cols(cols_) {
    if constexpr (DT == AVEY_F32) {
      f = static_cast<const float *>(x) + row * ld;
    } else {
      h = static_cast<const bf16 *>(x) + row * ld;
      if constexpr (DT == AVEY_BF16X2) l = h + rows * ld;
    }
  }

  __device__ __forceinline__ void load(int g, QuantRaw<DT> &r) const {
    const int c = g * 8;
    if constexpr (FAST) {
      if (c >= cols) {
        r.clear();
      } else if constexpr (DT == AVEY_F32) {
        r.w[0] = *reinterpret_cast<const uint4 *>(f + c);
        r.w[1] = *reinterpret_cast<const uint4 *>(f + c + 4);
      } else {
        r.w[0] = *reinterpret_cast<const uint4 *>(h + c);
        if constexpr (DT == AVEY_BF16X2) r.w[1] = *reinterpret_cast<const uint4 *>(l + c);
      }
    } else {
      uint32_t b[8] = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c + i >= cols) continue;
        if constexpr (DT == AVEY_F32) {
          b[i] = __float_as_uint(f[c + i]);
        } else {
          b[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(h[c + i])) << (16 * (i & 1));
          if constexpr (DT == AVEY_BF16X2)
            b[4 + i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(l[c + i])) << (16 * (i & 1));
        }
      }
      r.w[0] = make_uint4(b[0], b[1], b[2], b[3]);
      if constexpr (DT != AVEY_BF16) r.w[1] = make_uint4(b[4], b[5], b[6], b[7]);
    }
  }
};

// Running maximum of |x| and what tells whether any value is not finite; with
// SQ the sum of squares.
template <int DT, bool SQ>
struct QuantScan {
  float mx = 0.f;               // bf16: unused
  float2 chk = {0.f, 0.f};      // NaN once a value was not finite; bf16: unused
  uint32_t m2 = 0;              // bf16: maxima of the two halves' bits, which order NaN above infinity
  float2 ss = {0.f, 0.f};

  __device__ __forceinline__ void add(const QuantRaw<DT> &r) {
    float v[8];
    if (DT != AVEY_BF16 || SQ) r.values(v);
    if constexpr (DT == AVEY_BF16) {
      const uint32_t a[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, a[i] & 0x7fff7fffu);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        mx = fmaxf(fmaxf(mx, fabsf(v[i])), fabsf(v[i + 1]));
        chk = ffma2(make_float2(v[i], v[i + 1]), make_float2(0.f, 0.f), chk);
      }
    }
    if constexpr (SQ) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) ss = ffma2(make_float2(v[i], v[i + 1]), make_float2(v[i], v[i + 1]), ss);
    }
  }
  // Bits of the largest |x|, at least those of infinity if one is not finite.
  __device__ __forceinline__ uint32_t bits() const {
    if constexpr (DT == AVEY_BF16) {
      const uint32_t m = max(m2 & 0xffffu, m2 >> 16) << 16;
      return m;
    } else {
      return chk.x == 0.f && chk.y == 0.f ? __float_as_uint(mx) : 0x7f800000u;
    }
  }
  __device__ __forceinline__ float squares() const { return ss.x + ss.y; }
};

// Squares of finite values may leave fp32 (from |x| = 1.8e19 on), which would leave
// the scale s / sqrt(mean(x^2)) at 0.
__device__ __forceinline__ bool squares_overflow(float ss, uint32_t max_bits) {
  return ss == INFINITY && max_bits < 0x7f800000u;
}
// The normalised scale of such a row, by L lanes of one warp, of which this is number
// `me`: the squares are those of the values times 2^-96, where none overflows, what is
// lost below is nothing to their sum, and 1e-6 is far below an ulp of the mean.  A
// function apart that reads the row again, so that the rows that do not need it pay
// no registers for it.
template <int DT, int L>
__device__ __noinline__ float shrunk_scale(const void *x, long long row, long long rows, int cols, long long ld,
                                           int me) {
  constexpr float kShrink = 0x1p-96f;
  const QuantSource<DT, false> src(x, row, rows, cols, ld);
  float ss = 0.f, mx = 0.f;
#pragma unroll 1
  for (int g = me; g < (cols + 7) / 8; g += L) {
    QuantRaw<DT> r;
    float v[8];
    src.load(g, r);
    r.values(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mx = fmaxf(mx, fabsf(v[i]));
      ss = fmaf(v[i] * kShrink, v[i] * kShrink, ss);
    }
  }
  const uint32_t lanes = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << ((threadIdx.x & 31) - me);
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) {
    ss += __shfl_xor_sync(lanes, ss, off);
    mx = fmaxf(mx, __shfl_xor_sync(lanes, mx, off));
  }
  return __fmul_rn(mx, 1.0f / 127.0f) * kShrink * (1.0f / sqrtf(ss / static_cast<float>(cols)));
}

// The scale of a row from the bits of its largest magnitude, and the rounding.
struct RowScale {
  float scale;  // s; NaN for a row that is not finite
  float s, inv;
  bool zero, slow;
  static constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number

  // short_values: x has so few bits that half the largest value, 63.5 steps to
  // within rounding, is met often.  inv is then moved by an ulp or two until the
  // fast rounding of that value is right.
  __device__ __forceinline__ RowScale(uint32_t max_bits, bool short_values) {
    const bool bad = max_bits >= 0x7f800000u;
    s = __fmul_rn(__uint_as_float(max_bits), 1.0f / 127.0f);
    scale = bad ? __uint_as_float(0x7fc00000u) : s;
    zero = bad || s == 0.0f;
    slow = s < 1e-30f;  // 1 / s may overflow
    inv = 1.0f / s;
    if (short_values && !zero && !slow) {
      const float h = 0.5f * __uint_as_float(max_bits), r = fmaf(-63.0f, s, h);
      const bool up = 2.0f * r >= s;  // 64 is even: it takes the tie
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const bool got = fmaf(h, inv, kMagic) - kMagic == 64.0f;
        if (got != up) inv = __uint_as_float(__float_as_uint(inv) + (up ? 1u : ~0u));
      }
    }
  }

  // RNE of the exact x / s, tie to even.  The remainder r = x - q s is exact in
  // fp32 (a multiple of half an ulp of s, at most about s / 2), so 2 |r| against
  // s tells whether q, off by at most one, is right.
  __device__ __forceinline__ int exact(float x) const {
    float q = rintf(__fdiv_rn(x, s));
    const float r = fmaf(-q, s, x), r2 = fabsf(r) * 2.0f;
    if (r2 >= s) {
      const float o = q + copysignf(1.0f, r);
      if (r2 > s || (static_cast<int>(q) & 1)) q = o;
    }
    return static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
  }

  // Eight values.  The low byte of x * inv + 1.5 * 2^23 is q; inv is off by a
  // few ulp, so q may be off by one next to a half, where 2 |r| reaches s, and is
  // put right there.  Scales whose inverse overflows take the division.
  template <int DT>
  __device__ __forceinline__ uint2 quantize8(const QuantRaw<DT> &raw) const {
    float v[8];
    raw.values(v);
    if (zero) return make_uint2(0u, 0u);
    uint32_t b[8];
    float far = 0.f;
    const float2 inv2 = make_float2(inv, inv), m2 = make_float2(kMagic, kMagic);
    const float2 minus_m = make_float2(-kMagic, -kMagic), minus_s = make_float2(-s, -s);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 x = make_float2(v[j], v[j + 1]);
      const float2 t = ffma2(x, inv2, m2);
      const float2 r = ffma2(fadd2(t, minus_m), minus_s, x);
      b[j] = __float_as_uint(t.x);
      b[j + 1] = __float_as_uint(t.y);
      far = fmaxf(fmaxf(far, fabsf(r.x)), fabsf(r.y));
    }
    if (far * 2.0f >= s || slow) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = __uint_as_float(b[j]);
        const float r = fmaf(kMagic - t, s, v[j]), r2 = fabsf(r) * 2.0f;
        if (r2 > s || (r2 == s && (b[j] & 1u))) b[j] = __float_as_uint(t + copysignf(1.0f, r));
      }
      if (slow) {
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
          float x = v[0];
#pragma unroll
          for (int q = 1; q < 8; ++q) x = q == j ? v[q] : x;
          const uint32_t e = static_cast<uint32_t>(exact(x));
#pragma unroll
          for (int q = 0; q < 8; ++q) b[q] = q == j ? e : b[q];
        }
      }
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                         __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
    return make_uint2(w[0], w[1]);
  }
};

}  // namespace avey
