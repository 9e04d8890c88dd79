// avey_linear_few.cu -- the 8-bit product for up to 16 rows (single tokens of a
// decoder or a head): bound by one read of the weights, and by latency.
//
// A warp owns 16 output channels and walks K in steps of 64: mma.sync m16n8k32
// with the weights as A straight from global memory and eight tokens as B from
// shared memory.  A sum does not care about the order of its terms, so both
// operands use the order that suits the loads: lane 4 g + q takes the 16 bytes
// k = 16 q .. 16 q + 15 of its channels (g and g + 8) and of token g, and two
// MMAs eat them as "columns" 4 q .. and 16 + 4 q ..  A warp's loads cover whole
// 64-byte pieces of 16 rows; rows are prefetched into L2 before the block
// prepares its tokens.  Rows that come unrounded are quantised by every block for
// itself (a few KB from L2), which saves the launch of the rounding kernel.
// 12 rows against 50368 x 768 weights take 13.1 us here; rounded apart and with
// channels as the rows of a tile 13.5, two launches.  More rows or longer ones mean
// more to prepare per block: from 9 rows on only up to K = 768 (12 rows against
// 65536 x 1024: 19.4 and 17.4 us; 40000 x 2048: 27.5 and 21.7), and none from 17.
// Up to 8 rows fit up to K = 12160, 96 KB of tokens.
// Scored (1 x 768 -> 50368: 12.7 us, with the logits in memory 14.9) a block leaves the
// softmax statistics of its channels, and a block per token joins them.
#include <algorithm>

#include "avey_common.cuh"
#include "avey_internal.h"
#include "avey_quant.cuh"
#include "avey_score.cuh"

namespace avey {
namespace {

struct FewArgs {
  const void *x;
  long long ld_x;
  int x_fast, prenorm;
  const float *x_scale;
  int rows, N, K, stride;  // stride: bytes of a token in shared memory
  const int8_t *Wq;
  long long ld_w;
  const float *w_scale, *bias, *residual;
  long long ld_res;
  int relu2;
  void *out;
  long long ld_out;
  // scores: (max, sum, weighted sum) of token t over block b's words at
  // partial[t * blocks + b], and the logits of the given tokens
  const int32_t *ids;
  float4 *partial;
  float *given;
};

// What the products become besides AVEY_F32, AVEY_BF16 and AVEY_BF16X2.
constexpr int kScore = -1;

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One row of x as 8-bit integers into shared memory (zeros behind K), by a warp.
template <int DT, bool FAST>
__device__ __forceinline__ void quantize_row_to(const FewArgs &a, int row, int8_t *dst, float *scale, int lane) {
  const QuantSource<DT, FAST> src(a.x, row, a.rows, a.K, a.ld_x);
  constexpr int kHold = 4;
  const int groups = a.stride / 8;
  QuantRaw<DT> v[kHold];
  QuantScan<DT, true> scan;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    if (lane + 32 * i < groups)
      src.load(lane + 32 * i, v[i]);
    else
      v[i].clear();
  }
#pragma unroll
  for (int i = 0; i < kHold; ++i) scan.add(v[i]);
  for (int g = lane + 32 * kHold; g < groups; g += 32) {
    QuantRaw<DT> t;
    src.load(g, t);
    scan.add(t);
  }
  const uint32_t mx = __reduce_max_sync(0xffffffffu, scan.bits());
  float ss = scan.squares();
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const RowScale rs(mx, false);
  const bool again = a.prenorm && squares_overflow(ss, mx);
  if (lane == 0)
    *scale = a.prenorm ? rs.scale * (1.0f / sqrtf(ss / static_cast<float>(a.K) + 1e-6f)) : rs.scale;
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (lane + 32 * i < groups) *reinterpret_cast<uint2 *>(dst + (lane + 32 * i) * 8) = rs.quantize8(v[i]);
  for (int g = lane + 32 * kHold; g < groups; g += 32) {
    QuantRaw<DT> t;
    src.load(g, t);
    *reinterpret_cast<uint2 *>(dst + g * 8) = rs.quantize8(t);
  }
  if (again) {
    const float sc = shrunk_scale<DT, 32>(a.x, row, a.rows, a.K, a.ld_x, lane);
    if (lane == 0) *scale = sc;
  }
}

// The statistics of this block's words for every token, from its warps' sums.
template <int NB, int WARPS>
__device__ __forceinline__ void score_block(const FewArgs &a, const int (&acc)[NB][4], const float *xs, int n0,
                                            int warp, int lane) {
  __shared__ float4 parts[WARPS][NB * 8];
  const int g = lane >> 2, q = lane & 3;
  float y[2][NB * 2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = n0 + g + 8 * h;
    const bool in = n < a.N;
    const float w = in ? __ldg(a.w_scale + n) : 0.f, bias = in && a.bias ? __ldg(a.bias + n) * kLog2e : 0.f;
    const float low = in ? max_nan(bias, kMaskedWord) : kMaskedWord;
#pragma unroll
    for (int c = 0; c < NB * 2; ++c) {
      const int t = (c >> 1) * 8 + 2 * q + (c & 1);
      const float p = static_cast<float>(acc[c >> 1][2 * h + (c & 1)]) * (xs[t] * kLog2e);
      if (in && t < a.rows && a.ids && a.ids[t] == n) a.given[t] = fmaf(p, w, bias);
      y[h][c] = fmaf(p, w, low);
    }
  }
#pragma unroll
  for (int c = 0; c < NB * 2; ++c) {
    float m = fmaxf(fmaxf(y[0][c], y[1][c]), kLowest);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float d0 = y[0][c] - m, d1 = y[1][c] - m, e0 = ex2(d0), e1 = ex2(d1);
    float s = e0 + e1, t = fmaf(e0, d0, e1 * d1);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, off);
      t += __shfl_xor_sync(0xffffffffu, t, off);
    }
    if (g == 0) parts[warp][(c >> 1) * 8 + 2 * q + (c & 1)] = make_float4(m, s, t, 0.f);
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < a.rows) {
    Stat2 st{kLowest, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < WARPS; ++i) join2(st, Stat2{parts[i][t].x, parts[i][t].y, parts[i][t].z});
    a.partial[static_cast<long long>(t) * gridDim.x + blockIdx.x] = make_float4(st.m, st.s, st.t, 0.f);
  }
  grid_release();
}

constexpr int kJoinThreads = 256;

// One block per token: joins its blocks' statistics.
__global__ void __launch_bounds__(kJoinThreads)
    score_few_join(int N, int blocks, const int32_t *ids, const float4 *partial,
                   const float *given, float *logprob, float *stats, float *entropy, int *status) {
  __shared__ float4 parts[kJoinThreads / 32];
  const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait();
  Stat2 st{kLowest, 0.f, 0.f};
  for (int i = threadIdx.x; i < blocks; i += kJoinThreads) {
    const float4 v = partial[static_cast<long long>(row) * blocks + i];
    join2(st, Stat2{v.x, v.y, v.z});
  }
  rebase2(st, warp_max(st.m));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    st.s += __shfl_xor_sync(0xffffffffu, st.s, off);
    st.t += __shfl_xor_sync(0xffffffffu, st.t, off);
  }
  if (lane == 0) parts[warp] = make_float4(st.m, st.s, st.t, 0.f);
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int i = 1; i < kJoinThreads / 32; ++i) join2(st, Stat2{parts[i].x, parts[i].y, parts[i].z});
  int id = ids ? ids[row] : -1;
  if (id >= N) {
    record_status(status, AVEY_ERR_DEVICE_BOUNDS);
    id = -1;
  }
  write_scores(st, row, id >= 0, id >= 0 ? given[row] : 0.f, logprob, stats, entropy);
}

// NB blocks of eight tokens, WARPS x 16 channels a block, DT the type of x.
// Four thread blocks an SM, or from 56832 channels on some wait and prepare the
// tokens after the others (12 x 768 -> 65536: 19.9 us with three an SM, 15.7 with
// four; 50368: 12.9 and 13.4; 1 x 1024 -> 65536: 20.2 and 15.8).
template <int NB, int WARPS, int DT, int OUT>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 4 : 0) linear_i8_few(const FewArgs a) {
  extern __shared__ __align__(16) int8_t xs_q[];
  __shared__ float xs[NB * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int n0 = (blockIdx.x * WARPS + warp) * 16;
  const int k16 = (a.K + 15) / 16 * 16;  // bytes of a weight row that may be read
  {
    const int lines = (k16 + 127) / 128;
    for (int i = lane; i < 16 * lines; i += 32) {
      const int n = n0 + i / lines;
      if (n < a.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.Wq + n * a.ld_w + (i % lines) * 128));
    }
  }
  for (int t = warp; t < NB * 8; t += WARPS) {
    int8_t *dst = xs_q + t * a.stride;
    if (t >= a.rows) {
      for (int i = lane * 8; i < a.stride; i += 256) *reinterpret_cast<uint2 *>(dst + i) = make_uint2(0, 0);
      if (lane == 0) xs[t] = 0.f;
    } else if constexpr (DT == AVEY_I8) {
      const int8_t *src = static_cast<const int8_t *>(a.x) + t * a.ld_x;
      for (int i = lane * 16; i < a.stride; i += 512) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (i < k16) w = *reinterpret_cast<const uint4 *>(src + i);
        if (i < a.K && i + 16 > a.K) {  // bytes behind K are not ours
          uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int keep = a.K - i - 4 * j;
            v[j] = keep >= 4 ? v[j] : keep <= 0 ? 0u : v[j] & (0xffffffffu >> (32 - 8 * keep));
          }
          w = make_uint4(v[0], v[1], v[2], v[3]);
        }
        *reinterpret_cast<uint4 *>(dst + i) = w;
      }
      if (lane == 0) xs[t] = a.x_scale[t];
    } else {
      if (a.x_fast)
        quantize_row_to<DT, true>(a, t, dst, xs + t, lane);
      else
        quantize_row_to<DT, false>(a, t, dst, xs + t, lane);
    }
  }
  __syncthreads();
  if (OUT != kScore && n0 >= a.N) return;

  int acc[NB][4] = {};
  const int8_t *w0 = a.Wq + static_cast<long long>(min(n0 + g, a.N - 1)) * a.ld_w + q * 16;
  const int8_t *w1 = a.Wq + static_cast<long long>(min(n0 + g + 8, a.N - 1)) * a.ld_w + q * 16;
  const int8_t *xrow = xs_q + g * a.stride + q * 16;
  constexpr int UN = 4;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = 0; k0 < k16; k0 += 64 * UN) {
    uint4 u[UN], v[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int k = k0 + 64 * i;
      const bool in = k + q * 16 < k16;
      u[i] = in ? __ldg(reinterpret_cast<const uint4 *>(w0 + k)) : zero;
      v[i] = in ? __ldg(reinterpret_cast<const uint4 *>(w1 + k)) : zero;
    }
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int k = k0 + 64 * i;
      if (k >= k16) break;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 x = *reinterpret_cast<const uint4 *>(xrow + b * 8 * a.stride + k);
        mma_s8(acc[b], u[i].x, v[i].x, u[i].y, v[i].y, x.x, x.y);
        mma_s8(acc[b], u[i].z, v[i].z, u[i].w, v[i].w, x.z, x.w);
      }
    }
  }
  if constexpr (OUT == kScore) {
    score_block<NB, WARPS>(a, acc, xs, n0, warp, lane);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = n0 + g + 8 * h;
    if (n >= a.N) continue;
    const float w = __ldg(a.w_scale + n), bias = a.bias ? __ldg(a.bias + n) : 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = b * 8 + 2 * q + e;
        if (t >= a.rows) continue;
        float y = fmaf(static_cast<float>(acc[b][2 * h + e]) * xs[t], w, bias);
        if (a.relu2) {
          y = y < 0.f ? 0.f : y;  // NaN stays NaN
          y *= y;
        }
        const long long at = t * a.ld_out + n;
        if constexpr (OUT == AVEY_F32) {
          if (a.residual) y += a.residual[t * a.ld_res + n];
          static_cast<float *>(a.out)[at] = y;
        } else {
          bf16 *hi = static_cast<bf16 *>(a.out) + at;
          *hi = __float2bfloat16_rn(y);
          if constexpr (OUT == AVEY_BF16X2) {
            float vh, vl;
            split_bf16(y, vh, vl);
            hi[a.rows * a.ld_out] = __float2bfloat16_rn(vl);
          }
        }
      }
    }
  }
}

// Four warps a block while that leaves SMs without one; eight share the
// preparation of the tokens among more channels.
inline int few_warps(int N) { return N <= 64 * sm_count() ? 4 : 8; }
inline int few_grid(int N) {
  const int channels = 16 * few_warps(N);
  return (N + channels - 1) / channels;
}

constexpr int kFewShared = 96 * 1024;  // at most two blocks' worth of an SM

template <int NB, int WARPS, int DT, int OUT>
avey_status run_few(const FewArgs &a, cudaStream_t s) {
  auto kern = linear_i8_few<NB, WARPS, DT, OUT>;
  const int bytes = NB * 8 * a.stride;
  // static arrays (the scales, the scores' parts) count toward the 48 KB that need no request
  constexpr int kStatic = NB * 8 * 4 + (OUT == kScore ? WARPS * NB * 8 * static_cast<int>(sizeof(float4)) : 0);
  if (bytes + kStatic > 48 * 1024) {
    // the limit is the kernel's, whichever thread calls it: always the largest, so that no
    // call lowers another's before its launch
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewShared);
    if (e != cudaSuccess) {
      cudaGetLastError();
      set_detail("linear_i8_few: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
      return AVEY_ERR_CUDA;
    }
  }
  kern<<<few_grid(a.N), WARPS * 32, bytes, s>>>(a);
  AVEY_CHECK_LAUNCH("linear_i8_few", s);
  return AVEY_OK;
}

template <int NB, int DT, int OUT>
avey_status run_few_warps(const FewArgs &a, cudaStream_t s) {
  if (few_warps(a.N) == 4) return run_few<NB, 4, DT, OUT>(a, s);
  return run_few<NB, 8, DT, OUT>(a, s);
}

template <int NB, int DT>
avey_status run_few_out(const FewArgs &a, int out_dt, cudaStream_t s) {
  if (out_dt == kScore) return run_few_warps<NB, DT, kScore>(a, s);
  if (out_dt == AVEY_F32) return run_few_warps<NB, DT, AVEY_F32>(a, s);
  if (out_dt == AVEY_BF16) return run_few_warps<NB, DT, AVEY_BF16>(a, s);
  return run_few_warps<NB, DT, AVEY_BF16X2>(a, s);
}

inline int few_stride(int K) { return (K + 127) / 128 * 128 + 64; }  // odd multiples of 64: no bank conflicts
inline int few_blocks(int rows) { return rows <= 8 ? 1 : 2; }

}  // namespace

bool linear_few_fits(int rows, int K) {
  return rows <= kFewRows && (few_blocks(rows) == 1 || K <= 768) && K <= kFewShared && 8 * few_stride(K) <= kFewShared;
}

bool linear_few_quantizes(avey_dtype x_dt, int rows, int K) {
  return x_dt != AVEY_I8 && linear_few_fits(rows, K);
}

namespace {

FewArgs few_args(const avey_linear_i8_params *p, const void *x, avey_dtype x_dt, int64_t ld_x,
                 const float *x_scale, int prenorm, int rows) {
  FewArgs a{};
  a.x = x;
  a.ld_x = ld_x;
  a.x_fast = x_dt != AVEY_I8 && quant_rows_fast(x, x_dt, rows, p->K, ld_x);
  a.prenorm = prenorm;
  a.x_scale = x_scale;
  a.rows = rows;
  a.N = p->N;
  a.K = p->K;
  a.stride = few_stride(p->K);
  a.Wq = p->Wq;
  a.ld_w = p->ld_w;
  a.w_scale = p->w_scale;
  a.bias = p->bias;
  a.relu2 = p->act == AVEY_ACT_RELU2;
  return a;
}

avey_status run_few_any(const FewArgs &a, avey_dtype x_dt, int out_dt, cudaStream_t s) {
  const bool one = few_blocks(a.rows) == 1;
#define AVEY_FEW(DT) return one ? run_few_out<1, DT>(a, out_dt, s) : run_few_out<2, DT>(a, out_dt, s)
  switch (x_dt) {
    case AVEY_F32: AVEY_FEW(AVEY_F32);
    case AVEY_BF16: AVEY_FEW(AVEY_BF16);
    case AVEY_BF16X2: AVEY_FEW(AVEY_BF16X2);
    default: AVEY_FEW(AVEY_I8);
  }
#undef AVEY_FEW
}

}  // namespace

avey_status launch_linear_few(const avey_linear_i8_params *p, const void *x, avey_dtype x_dt, int64_t ld_x,
                              const float *x_scale, int prenorm, int rows, const float *residual,
                              int64_t ld_res, void *out, avey_dtype out_dt, int64_t ld_out,
                              cudaStream_t s) {
  FewArgs a = few_args(p, x, x_dt, ld_x, x_scale, prenorm, rows);
  a.residual = residual;
  a.ld_res = ld_res;
  a.out = out;
  a.ld_out = ld_out;
  return run_few_any(a, x_dt, out_dt, s);
}

size_t score_few_bytes(int rows, int N) {
  return static_cast<size_t>(rows) * few_grid(N) * sizeof(float4) + static_cast<size_t>(rows) * sizeof(float);
}

avey_status launch_score_few(const avey_linear_i8_params *p, const void *x, avey_dtype x_dt, int64_t ld_x,
                             const float *x_scale, int prenorm, int rows, const int32_t *ids, float *logprob,
                             float *stats, float *entropy, void *ws, cudaStream_t s) {
  FewArgs a = few_args(p, x, x_dt, ld_x, x_scale, prenorm, rows);
  const int blocks = few_grid(p->N);
  a.ids = ids;
  a.partial = static_cast<float4 *>(ws);
  a.given = reinterpret_cast<float *>(a.partial + static_cast<size_t>(rows) * blocks);
  const avey_status st = run_few_any(a, x_dt, kScore, s);
  if (st != AVEY_OK) return st;
  const cudaError_t e = launch_after(score_few_join, static_cast<unsigned>(rows), kJoinThreads, 0, s, p->N, blocks,
                                     ids, a.partial, a.given, logprob, stats, entropy, device_status_word());
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_detail("score_few_join launch failed: %s", cudaGetErrorString(e));
    return AVEY_ERR_CUDA;
  }
  AVEY_CHECK_LAUNCH("score_few_join", s);
  return AVEY_OK;
}

}  // namespace avey
