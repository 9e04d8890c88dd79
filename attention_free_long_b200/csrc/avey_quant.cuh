// avey_quant.cuh -- the 8-bit rounding shared by avey_quantize_rows and the
// products that quantise their own input.
#pragma once

#include "avey_common.cuh"
#include "avey_internal.h"

namespace avey {

// Whether every row of x (both planes of a pair) starts on a 16-byte boundary.
inline bool quant_rows_aligned(const void *x, int dt, long long rows, long long ld) {
  const long long es = dt == AVEY_F32 ? 4 : 2;
  return aligned16(x) && (ld * es) % 16 == 0 && (dt != AVEY_BF16X2 || (rows * ld * es) % 16 == 0);
}

// One row of x, in groups of 8 consecutive values; values past the row's end
// are 0.
template <int DT>
struct QuantSource {
  const float *f = nullptr;
  const bf16 *h = nullptr, *l = nullptr;
  int cols;
  bool aligned;

  __device__ __forceinline__ QuantSource(const void *x, long long row, long long rows, int cols_,
                                         long long ld, int aligned_)
      : cols(cols_), aligned(aligned_ != 0) {
    if constexpr (DT == AVEY_F32) {
      f = static_cast<const float *>(x) + row * ld;
    } else {
      h = static_cast<const bf16 *>(x) + row * ld;
      if constexpr (DT == AVEY_BF16X2) l = h + rows * ld;
    }
  }

  __device__ __forceinline__ void load(int g, float (&v)[8]) const {
    const int c = g * 8;
    if (aligned && c + 8 <= cols) {
      if constexpr (DT == AVEY_F32) {
        const float4 a = *reinterpret_cast<const float4 *>(f + c);
        const float4 b = *reinterpret_cast<const float4 *>(f + c + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(h + c);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = unpack_bf16(aw[i]);
          v[2 * i] = p.x;
          v[2 * i + 1] = p.y;
        }
        if constexpr (DT == AVEY_BF16X2) {
          const uint4 b = *reinterpret_cast<const uint4 *>(l + c);
          const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 p = unpack_bf16(bw[i]);
            v[2 * i] += p.x;
            v[2 * i + 1] += p.y;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = 0.f;
        if (c + i < cols) {
          if constexpr (DT == AVEY_F32) {
            v[i] = f[c + i];
          } else {
            v[i] = __bfloat162float(h[c + i]);
            if constexpr (DT == AVEY_BF16X2) v[i] += __bfloat162float(l[c + i]);
          }
        }
      }
    }
  }
};

// Running maximum of |x| as its bit pattern (which orders NaN above infinity
// above every finite value) and sum of squares.
__device__ __forceinline__ void quant_scan(const float (&v)[8], uint32_t &mx, float &ss) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    mx = max(mx, __float_as_uint(v[j]) & 0x7fffffffu);
    ss = fmaf(v[j], v[j], ss);
  }
}

// The scale of a row from the bits of its largest magnitude, and the rounding.
struct RowScale {
  float scale;  // s; NaN for a row that is not finite
  float s, inv;
  bool zero, slow;

  __device__ __forceinline__ explicit RowScale(uint32_t max_bits) {
    const bool bad = max_bits >= 0x7f800000u;
    s = __fmul_rn(__uint_as_float(max_bits), 1.0f / 127.0f);
    scale = bad ? __uint_as_float(0x7fc00000u) : s;
    zero = bad || s == 0.0f;
    slow = s < 1e-30f;  // 1 / s may overflow
    inv = 1.0f / s;
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

  // Eight values.  x * inv + 1.5 * 2^23 rounds to a whole number whose low byte
  // is q; inv is off by a few ulp, so q may be wrong next to a half, where
  // 2 |r| reaches s: then (and for scales whose inverse overflows) all eight
  // take the exact form.
  __device__ __forceinline__ uint2 quantize8(const float (&v)[8]) const {
    if (zero) return make_uint2(0u, 0u);
    constexpr float kMagic = 12582912.0f;
    uint32_t b[8];
    float far = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = fmaf(v[j], inv, kMagic);
      b[j] = __float_as_uint(t);
      far = fmaxf(far, fabsf(fmaf(kMagic - t, s, v[j])));
    }
    if (slow || far * 2.0f >= s) {
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
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                         __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
    return make_uint2(w[0], w[1]);
  }
};

}  // namespace avey
