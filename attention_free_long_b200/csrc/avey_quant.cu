// avey_quant.cu -- rows of activations (or weight channels) as 8-bit integers
// with one fp32 scale per row:
//   s = fl32(max |x| * fl32(1 / 127)),  q = RNE(x / s) clamped to [-127, 127]
//   scale = s, or s / sqrt(mean(x^2) + 1e-6) with prenorm
// One read of x and one write of q: HBM-bound (5 bytes a value from fp32, 3
// from bf16).  A row stays in registers between the maximum and the rounding
// (32 values a thread); only rows longer than 1024 values a warp, or 8192 a
// block, are read again.
#include <algorithm>

#include "avey_common.cuh"
#include "avey_internal.h"
#include "avey_quant.cuh"

namespace avey {
namespace {

constexpr int kGroups = 4;  // groups of 8 values a thread keeps in registers

// WPR warps per row: one when rows are short and many, eight otherwise.
template <int DT, int WPR>
__global__ void __launch_bounds__(256) quantize_rows(const void *__restrict__ x, int rows, int cols,
                                                     long long ld_x, int aligned, int prenorm,
                                                     int8_t *__restrict__ q, long long ld_q,
                                                     float *__restrict__ scale) {
  constexpr int RPB = 8 / WPR;  // rows per block
  __shared__ uint32_t s_max[8];
  __shared__ float s_sum[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * RPB + warp / WPR;
  const bool live = row < rows;
  const int step = 32 * WPR, me = (warp % WPR) * 32 + lane;
  const int groups = live ? ((cols + 15) / 16) * 2 : 0;  // up to roundup16(cols)
  const QuantSource<DT> src(x, live ? row : 0, rows, cols, ld_x, aligned);

  float v[kGroups][8];
  uint32_t mx = 0;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int g = me + i * step;
    if (g < groups) {
      src.load(g, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i) quant_scan(v[i], mx, ss);
  for (int g = me + kGroups * step; g < groups; g += step) {
    float t[8];
    src.load(g, t);
    quant_scan(t, mx, ss);
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  if constexpr (WPR > 1) {
    if (lane == 0) {
      s_max[warp] = mx;
      s_sum[warp] = ss;
    }
    __syncthreads();
    mx = 0;
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      mx = max(mx, s_max[(warp / WPR) * WPR + w]);
      ss += s_sum[(warp / WPR) * WPR + w];
    }
  }
  if (!live) return;
  const RowScale rs(mx);
  if (me == 0)
    scale[row] = prenorm ? rs.scale * (1.0f / sqrtf(ss / static_cast<float>(cols) + 1e-6f)) : rs.scale;
  int8_t *qr = q + row * ld_q;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int g = me + i * step;
    if (g < groups) *reinterpret_cast<uint2 *>(qr + g * 8ll) = rs.quantize8(v[i]);
  }
  for (int g = me + kGroups * step; g < groups; g += step) {
    float t[8];
    src.load(g, t);
    *reinterpret_cast<uint2 *>(qr + g * 8ll) = rs.quantize8(t);
  }
}

template <int DT>
avey_status run_quantize(const void *x, int rows, int cols, long long ld_x, int prenorm, int8_t *q,
                         long long ld_q, float *scale, cudaStream_t s) {
  const int al = quant_rows_aligned(x, DT, rows, ld_x) ? 1 : 0;
  // as few warps a row as hold it (1024 values each); with fewer rows than SMs
  // eight, which spreads the loads of a row
  constexpr int kHold = kGroups * 256;
  if (cols > 4 * kHold || rows <= sm_count())
    quantize_rows<DT, 8><<<rows, 256, 0, s>>>(x, rows, cols, ld_x, al, prenorm, q, ld_q, scale);
  else if (cols > 2 * kHold)
    quantize_rows<DT, 4><<<(rows + 1) / 2, 256, 0, s>>>(x, rows, cols, ld_x, al, prenorm, q, ld_q, scale);
  else if (cols > kHold)
    quantize_rows<DT, 2><<<(rows + 3) / 4, 256, 0, s>>>(x, rows, cols, ld_x, al, prenorm, q, ld_q, scale);
  else
    quantize_rows<DT, 1><<<(rows + 7) / 8, 256, 0, s>>>(x, rows, cols, ld_x, al, prenorm, q, ld_q, scale);
  AVEY_CHECK_LAUNCH("quantize_rows", s);
  return AVEY_OK;
}

}  // namespace

avey_status check_quant_source(const char *fn, const void *x, avey_dtype dt, int cols, int64_t ld_x) {
  AVEY_REQUIRE(dt == AVEY_F32 || dt == AVEY_BF16 || dt == AVEY_BF16X2, AVEY_ERR_UNSUPPORTED,
               "%s: dtype %d unsupported (F32, BF16 or BF16X2)", fn, int(dt));
  AVEY_REQUIRE(ld_x >= cols, AVEY_ERR_INVALID_ARG, "%s: ld_x=%lld < %d columns", fn,
               static_cast<long long>(ld_x), cols);
  AVEY_REQUIRE((reinterpret_cast<uintptr_t>(x) & (dt == AVEY_F32 ? 3 : 1)) == 0, AVEY_ERR_INVALID_ARG,
               "%s: x is not aligned to its element", fn);
  return AVEY_OK;
}

avey_status launch_quantize_rows(const void *x, avey_dtype dt, int rows, int cols, int64_t ld_x,
                                 int prenorm, int8_t *q, int64_t ld_q, float *scale, cudaStream_t s) {
  if (rows == 0) return AVEY_OK;
  switch (dt) {
    case AVEY_F32: return run_quantize<AVEY_F32>(x, rows, cols, ld_x, prenorm, q, ld_q, scale, s);
    case AVEY_BF16: return run_quantize<AVEY_BF16>(x, rows, cols, ld_x, prenorm, q, ld_q, scale, s);
    default: return run_quantize<AVEY_BF16X2>(x, rows, cols, ld_x, prenorm, q, ld_q, scale, s);
  }
}

}  // namespace avey

using namespace avey;

extern "C" avey_status avey_quantize_rows(const void *x, avey_dtype dt, int rows, int cols,
                                          int64_t ld_x, int prenorm, int8_t *q, int64_t ld_q,
                                          float *scale, avey_stream_t stream) {
  AVEY_REQUIRE(rows >= 0 && cols >= 1, AVEY_ERR_INVALID_ARG,
               "avey_quantize_rows: need rows >= 0 and cols >= 1 (rows=%d cols=%d)", rows, cols);
  const avey_status st = check_quant_source("avey_quantize_rows", x, dt, cols, ld_x);
  if (st != AVEY_OK) return st;
  AVEY_REQUIRE(cols <= (1 << 30), AVEY_ERR_UNSUPPORTED, "avey_quantize_rows: cols=%d > 2^30", cols);
  AVEY_REQUIRE(ld_q >= cols && ld_q % 16 == 0, AVEY_ERR_INVALID_ARG,
               "avey_quantize_rows: ld_q=%lld must be a multiple of 16, >= %d",
               static_cast<long long>(ld_q), cols);
  if (rows == 0) return AVEY_OK;
  AVEY_REQUIRE(x && q && scale, AVEY_ERR_INVALID_ARG, "avey_quantize_rows: null pointer");
  AVEY_REQUIRE(aligned16(q) && (reinterpret_cast<uintptr_t>(scale) & 3) == 0, AVEY_ERR_INVALID_ARG,
               "avey_quantize_rows: q 16-byte and scale 4-byte aligned");
  return launch_quantize_rows(x, dt, rows, cols, ld_x, prenorm ? 1 : 0, q, ld_q, scale,
                              reinterpret_cast<cudaStream_t>(stream));
}
