// avey_quant.cu -- rows of activations (or weight channels) as 8-bit integers
// with one fp32 scale per row:
//   s = fl32(max |x| * fl32(1 / 127)),  q = RNE(x / s) clamped to [-127, 127]
//   scale = s, or s / sqrt(mean(x^2) + 1e-6) with prenorm
// One read of x and one write of q: HBM-bound (5 bytes a value from fp32, 3
// from bf16).  A row stays in registers between the maximum and the rounding
// (32 values a thread); only rows longer than 8192 values are read again.
#include <algorithm>

#include "avey_common.cuh"
#include "avey_internal.h"
#include "avey_quant.cuh"

namespace avey {
namespace {

constexpr int kGroups = 4;  // groups of 8 values a thread keeps in registers

// LPR threads per row: as few as hold it.  The normalised forms are held to 64
// registers: the call behind the rounding would raise them to 72, three blocks an SM.
template <int DT, int LPR, bool PRENORM, bool FAST>
__global__ void __launch_bounds__(256, PRENORM ? 4 : 0) quantize_rows(const void *__restrict__ x, int rows, int cols,
                                                     long long ld_x, int8_t *__restrict__ q,
                                                     long long ld_q, float *__restrict__ scale) {
  constexpr int RPB = 256 / LPR, WPR = LPR / 32;  // rows per block, warps per row
  __shared__ uint32_t s_max[8];
  __shared__ float s_sum[8];
  grid_release();  // the product that follows may prepare itself
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int me = threadIdx.x % LPR;
  const long long row = static_cast<long long>(blockIdx.x) * RPB + threadIdx.x / LPR;
  const bool live = row < rows;
  const int groups = live ? ((cols + 15) / 16) * 2 : 0;  // up to roundup16(cols)
  const QuantSource<DT, FAST> src(x, live ? row : 0, rows, cols, ld_x);

  QuantRaw<DT> v[kGroups];
  QuantScan<DT, PRENORM> scan;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int g = me + i * LPR;
    if (g < groups)
      src.load(g, v[i]);
    else
      v[i].clear();
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i) scan.add(v[i]);
  for (int g = me + kGroups * LPR; g < groups; g += LPR) {
    QuantRaw<DT> t;
    src.load(g, t);
    scan.add(t);
  }
  uint32_t mx = scan.bits();
  float ss = scan.squares();
#pragma unroll
  for (int off = (LPR < 32 ? LPR : 32) / 2; off > 0; off >>= 1) {
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (PRENORM) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  }
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
  const RowScale rs(mx, DT == AVEY_BF16);
  if (me == 0)
    scale[row] = PRENORM ? rs.scale * (1.0f / sqrtf(ss / static_cast<float>(cols) + 1e-6f)) : rs.scale;
  constexpr int L = LPR < 32 ? LPR : 32;
  const bool again = PRENORM && me < L && squares_overflow(ss, mx);
  int8_t *qr = q + row * ld_q;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int g = me + i * LPR;
    if (g < groups) *reinterpret_cast<uint2 *>(qr + g * 8ll) = rs.quantize8(v[i]);
  }
  for (int g = me + kGroups * LPR; g < groups; g += LPR) {
    QuantRaw<DT> t;
    src.load(g, t);
    *reinterpret_cast<uint2 *>(qr + g * 8ll) = rs.quantize8(t);
  }
  if (again) {
    const int lane0 = threadIdx.x % LPR;
    const long long r = static_cast<long long>(blockIdx.x) * RPB + threadIdx.x / LPR;
    const float sc = shrunk_scale<DT, L>(x, r, rows, cols, ld_x, lane0);
    if (lane0 == 0) scale[r] = sc;
  }
}

template <int DT, bool PRENORM, bool FAST>
avey_status run_quantize(const void *x, int rows, int cols, long long ld_x, int8_t *q, long long ld_q,
                         float *scale, cudaStream_t s) {
#define AVEY_QUANTIZE(LPR) \
  quantize_rows<DT, LPR, PRENORM, FAST><<<(rows - 1) / (256 / LPR) + 1, 256, 0, s>>>(x, rows, cols, ld_x, q, ld_q, scale)
  // a thread holds 32 values; with fewer rows than SMs a block per row spreads
  // the loads of a row
  if (cols > 128 * 32 || (rows <= sm_count() && cols > 256))
    AVEY_QUANTIZE(256);
  else if (cols > 64 * 32)
    AVEY_QUANTIZE(128);
  else if (cols > 32 * 32)
    AVEY_QUANTIZE(64);
  else if (cols > 16 * 32)
    AVEY_QUANTIZE(32);
  else if (cols > 8 * 32)
    AVEY_QUANTIZE(16);
  else
    AVEY_QUANTIZE(8);
#undef AVEY_QUANTIZE
  AVEY_CHECK_LAUNCH("quantize_rows", s);
  return AVEY_OK;
}

template <int DT>
avey_status run_quantize(const void *x, int rows, int cols, long long ld_x, int prenorm, int8_t *q,
                         long long ld_q, float *scale, cudaStream_t s) {
  if (quant_rows_fast(x, DT, rows, cols, ld_x))
    return prenorm ? run_quantize<DT, true, true>(x, rows, cols, ld_x, q, ld_q, scale, s)
                   : run_quantize<DT, false, true>(x, rows, cols, ld_x, q, ld_q, scale, s);
  return prenorm ? run_quantize<DT, true, false>(x, rows, cols, ld_x, q, ld_q, scale, s)
                 : run_quantize<DT, false, false>(x, rows, cols, ld_x, q, ld_q, scale, s);
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
  {
    const uint64_t n = rows, es = dt == AVEY_F32 ? 4 : 2;
    const ByteRows xr{reinterpret_cast<uintptr_t>(x), dt == AVEY_BF16X2 ? 2 * n : n, cols * es, ld_x * es};
    // with the zeros behind the columns
    const ByteRows qr{reinterpret_cast<uintptr_t>(q), n, (cols + 15ull) / 16 * 16, static_cast<uint64_t>(ld_q)};
    AVEY_REQUIRE(!rows_overlap(xr, qr), AVEY_ERR_INVALID_ARG, "avey_quantize_rows: q overlaps x");
  }
  return launch_quantize_rows(x, dt, rows, cols, ld_x, prenorm ? 1 : 0, q, ld_q, scale,
                              reinterpret_cast<cudaStream_t>(stream));
}
