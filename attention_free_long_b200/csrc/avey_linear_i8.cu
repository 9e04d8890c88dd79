// avey_linear_i8.cu -- y = act(s_t w_n sum_k q_tk Wq_nk + b_n) + r_tn on tcgen05
// (kind::i8, int32 accumulators in TMEM).
//
// CTA pairs (cta_group::2) own 256 x BN output tiles; roles and barriers are
// those of the layer GEMMs (avey_tc.cu): a TMA producer warp, one thread of
// CTA 0 issuing the MMAs, four epilogue warps per CTA, two accumulators so
// that the epilogue of a tile overlaps the MMAs of the next.  A K step is 128
// bytes = 128 values, four MMAs of K = 32.
#include <algorithm>

#include "avey_common.cuh"
#include "avey_internal.h"

namespace avey {
namespace {

constexpr int kBK = 128;
constexpr int kLinEpi = 4, kLinThreads = 64 + 32 * kLinEpi;

template <int BN>
struct LinLayout {
  static constexpr int PM = 256;
  static constexpr uint32_t A_BYTES = 128 * kBK;        // this CTA's rows
  static constexpr uint32_t B_BYTES = (BN / 2) * kBK;   // this CTA's half of the channels
  static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 6 : 8;
  static constexpr uint32_t TILES_BYTES = STAGES * STAGE_BYTES;
  static constexpr uint32_t CTRL_BYTES = 1024;
  static constexpr uint32_t STAGING_BYTES = kLinEpi * 8192;
  static constexpr uint32_t SMEM_BYTES = TILES_BYTES + CTRL_BYTES + STAGING_BYTES + 1024;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(STAGES <= 8, "the control block holds at most 8 stages");
};

struct LinArgs {
  int rows, N, K;
  int tiles_m, tiles_n;
  long long num_tiles;
  const float *x_scale, *w_scale, *bias;
  int relu2;
  const float *residual;
  // TMA stores write whole 16-byte pieces: they cover the columns < N_tma, and
  // plain stores through out the rest of a row
  int N_tma;
  void *out;
  long long ld_out;
  int *status;
};

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
  }
}

__device__ __forceinline__ uint32_t lin_sw128(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }
__device__ __forceinline__ uint32_t lin_sw64(int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) << 4); }
__device__ __forceinline__ void lin_st4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Four consecutive fp32 of a row of n, zeros past its end; p + i 16-byte aligned.
__device__ __forceinline__ float4 load4(const float *p, int i, int n) {
  if (i + 4 <= n) return __ldg(reinterpret_cast<const float4 *>(p + i));
  return make_float4(i < n ? p[i] : 0.f, i + 1 < n ? p[i + 1] : 0.f, i + 2 < n ? p[i + 2] : 0.f, 0.f);
}
// The same without the read-only path, for a residual that the call overwrites.
__device__ __forceinline__ float4 load4_rw(const float *p, int i, int n) {
  if (i + 4 <= n) return *reinterpret_cast<const float4 *>(p + i);
  return make_float4(i < n ? p[i] : 0.f, i + 1 < n ? p[i + 1] : 0.f, i + 2 < n ? p[i + 2] : 0.f, 0.f);
}

// The columns from N_tma of a row's 32-column chunk.
template <int OUT>
__device__ __forceinline__ void store_rest(const LinArgs &a, int row, int col0, const float (&v)[32]) {
  const long long at = static_cast<long long>(row) * a.ld_out;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int c = col0 + j;
    if (c < a.N_tma || c >= a.N) continue;
    if constexpr (OUT == AVEY_F32) {
      static_cast<float *>(a.out)[at + c] = v[j];
    } else {
      bf16 *hi = static_cast<bf16 *>(a.out) + at + c;
      *hi = __float2bfloat16_rn(v[j]);
      if constexpr (OUT == AVEY_BF16X2) {
        float h, l;
        split_bf16(v[j], h, l);
        hi[static_cast<long long>(a.rows) * a.ld_out] = __float2bfloat16_rn(l);
      }
    }
  }
}

template <int BN, int OUT, bool RES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLinThreads, 1)
    linear_i8_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmO0, const __grid_constant__ CUtensorMap tmO1,
                   const LinArgs a) {
  using P = LinLayout<BN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t *ctrl = smem_raw + pad + P::TILES_BYTES;
  const uint32_t sbase = raw_s + pad;
  const uint32_t cbase = sbase + P::TILES_BYTES;
  // control block: full[8] @0, empty[8] @64, tfull[2] @128, tempty[2] @144,
  // drain @160, tmem base @168, abort flag @172
  auto full_bar = [&](int s) { return cbase + 8u * s; };
  auto empty_bar = [&](int s) { return cbase + 64u + 8u * s; };
  auto tfull_bar = [&](int i) { return cbase + 128u + 8u * i; };
  auto tempty_bar = [&](int i) { return cbase + 144u + 8u * i; };
  const uint32_t drain_bar = cbase + 160u;
  volatile uint32_t *tmem_holder = reinterpret_cast<volatile uint32_t *>(ctrl + 168);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(ctrl + 172);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull_bar(i), 1);
      mbar_init(tempty_bar(i), 2 * kLinEpi);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmO0);
    if (OUT == AVEY_BF16X2) prefetch_tmap(&tmO1);
  }
  cluster_sync_all();
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(ctrl + 168), P::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int kchunks = (a.K + kBK - 1) / kBK;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      for (long long tile = pair; ok && tile < a.num_tiles; tile += npairs) {
        const int mt = static_cast<int>(tile / a.tiles_n), nt = static_cast<int>(tile % a.tiles_n);
        const int arow = mt * P::PM + static_cast<int>(rank) * 128;
        const int brow = nt * BN + static_cast<int>(rank) * (BN / 2);
        for (int kc = 0; kc < kchunks; ++kc) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * P::STAGE_BYTES);
          const uint32_t full0 = mapa_shared(full_bar(stage), 0);
          const uint32_t st = sbase + stage * P::STAGE_BYTES;
          tma_load_3d_pair(st, &tmA, full0, kc * kBK, arow, 0);
          tma_load_3d_pair(st + P::A_BYTES, &tmB, full0, kc * kBK, brow, 0);
          ++issued;
          if (++stage == P::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        record_status(a.status, AVEY_ERR_DEVICE_TIMEOUT);
      }
      // Drain: a stage's last use is over once the pair's MMA has released it.
      for (int s = 0; s < P::STAGES; ++s) {
        if (issued > s) {
          const long long last = ((issued - 1 - s) / P::STAGES) * P::STAGES + s;
          drain_wait(empty_bar(s), static_cast<uint32_t>((last / P::STAGES) & 1));
        }
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------- MMA issue (CTA 0)
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_s8_s32(P::PM, BN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (long long tile = pair; ok && tile < a.num_tiles; tile += npairs) {
        if (!mbar_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kc = 0; kc < kchunks; ++kc) {
          if (!mbar_wait(full_bar(stage), phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = sbase + stage * P::STAGE_BYTES;
          const uint64_t da = sdesc_k_sw128(st), db = sdesc_k_sw128(st + P::A_BYTES);
          const int steps = min(kBK / 32, (a.K - kc * kBK + 31) / 32);  // the rest is zeros
          for (int kk = 0; kk < steps; ++kk)
            tc_mma_i8_pair(d_tmem, da + 2u * kk, db + 2u * kk, idesc, (kc | kk) != 0);
          tc_commit_pair_both(empty_bar(stage));
          if (++stage == P::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair_both(tfull_bar(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) {
        *abort_flag = 1;
        record_status(a.status, AVEY_ERR_DEVICE_TIMEOUT);
      }
      tc_commit_pair_both(drain_bar);
      drain_wait(drain_bar, 0);
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int quarter = warp & 3;  // TMEM lanes 32*quarter .. +31
    const uint32_t stg = cbase + P::CTRL_BYTES + static_cast<uint32_t>(warp - 2) * 8192u;
    const uint32_t tempty_r0 = mapa_shared(tempty_bar(0), 0), tempty_r1 = mapa_shared(tempty_bar(1), 0);
    int acc = 0, it = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (long long tile = pair; tile < a.num_tiles; tile += npairs) {
      const int mt = static_cast<int>(tile / a.tiles_n), nt = static_cast<int>(tile % a.tiles_n);
      const int row0 = mt * P::PM + static_cast<int>(rank) * 128 + quarter * 32;
      const int row = row0 + lane;
      const bool valid = row < a.rows;
      const float xs = valid ? a.x_scale[row] : 0.f;
      if (!mbar_wait(tfull_bar(acc), acc_phase, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t taddr =
          tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int ch = 0; ch < BN / 32; ++ch) {
        const int col0 = nt * BN + ch * 32;
        if (col0 >= a.N || row0 >= a.rows) break;  // warp-uniform
        float v[32];
        tmem_ld32(taddr + ch * 32, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c = col0 + 4 * q;
          const float4 w = load4(a.w_scale, c, a.N);
          const float4 b = a.bias ? load4(a.bias, c, a.N) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float ww[4] = {w.x, w.y, w.z, w.w}, bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float y = fmaf(static_cast<float>(__float_as_int(v[4 * q + j])) * xs, ww[j], bb[j]);
            if (a.relu2) {
              // written so that NaN stays NaN
              y = y < 0.f ? 0.f : y;
              y *= y;
            }
            v[4 * q + j] = y;
          }
        }
        if constexpr (RES) {
          const float *rr = a.residual + static_cast<long long>(row) * a.ld_out;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 x = valid ? load4_rw(rr, col0 + 4 * q, a.N) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[4 * q] += x.x;
            v[4 * q + 1] += x.y;
            v[4 * q + 2] += x.z;
            v[4 * q + 3] += x.w;
          }
        }
        if (col0 + 32 > a.N_tma && valid) store_rest<OUT>(a, row, col0, v);
        if (col0 >= a.N_tma) continue;  // warp-uniform
        const uint32_t buf = stg + (it & 1) * 4096;
        if (it >= 2) {  // the store issued from this buffer two chunks ago must have read it
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
        }
        if constexpr (OUT == AVEY_F32) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            lin_st4(buf + lin_sw128(lane, c), __float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                    __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
        } else if constexpr (OUT == AVEY_BF16) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            lin_st4(buf + lin_sw64(lane, c), pack_bf16(v[8 * c], v[8 * c + 1]),
                    pack_bf16(v[8 * c + 2], v[8 * c + 3]), pack_bf16(v[8 * c + 4], v[8 * c + 5]),
                    pack_bf16(v[8 * c + 6], v[8 * c + 7]));
        } else {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) split_pack(v[2 * j], v[2 * j + 1], hi[j], lo[j]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            lin_st4(buf + lin_sw64(lane, c), hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
            lin_st4(buf + 2048 + lin_sw64(lane, c), lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&tmO0, buf, col0, row0, 0);
          if constexpr (OUT == AVEY_BF16X2) tma_store_3d(&tmO1, buf + 2048, col0, row0, 0);
          bulk_commit();
        }
        ++it;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc ? tempty_r1 : tempty_r0);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (!ok) {
      *abort_flag = 1;
      record_status(a.status, AVEY_ERR_DEVICE_TIMEOUT);
    }
    if (lane == 0) bulk_wait_all();  // outputs written
  }

  tc_fence_before();
  __syncthreads();
  // Both CTAs past their loops: the pair's MMAs have drained and no remote
  // arrival is still on its way.
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, P::TMEM_COLS);
  }
  cluster_sync_all();
}

template <int BN, int OUT, bool RES>
avey_status run_linear_pair(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &o0,
                            const CUtensorMap &o1, const LinArgs &a, cudaStream_t st) {
  using P = LinLayout<BN>;
  auto kern = linear_i8_pair<BN, OUT, RES>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(P::SMEM_BYTES));
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_detail("linear_i8: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    return AVEY_ERR_CUDA;
  }
  const int cap = std::max(1, sm_count() / 2);
  const int pairs = static_cast<int>(std::min<long long>(a.num_tiles, cap));
  kern<<<2 * pairs, kLinThreads, P::SMEM_BYTES, st>>>(ma, mb, o0, o1, a);
  AVEY_CHECK_LAUNCH("linear_i8", st);
  return AVEY_OK;
}

template <int BN>
avey_status run_linear_bn(const avey_linear_i8_params *p, const int8_t *xq, int64_t ld_xq, LinArgs a,
                          void *out, avey_dtype out_dt, cudaStream_t s) {
  CUtensorMap ma, mb, o0, o1;
  a.tiles_m = (a.rows + 255) / 256;
  a.tiles_n = (a.N + BN - 1) / BN;
  a.num_tiles = static_cast<long long>(a.tiles_m) * a.tiles_n;
  if (!encode_i8_map(&ma, xq, a.K, a.rows, ld_xq, 128)) return AVEY_ERR_CUDA;
  if (!encode_i8_map(&mb, p->Wq, a.K, a.N, p->ld_w, BN / 2)) return AVEY_ERR_CUDA;
  const bool f32 = out_dt == AVEY_F32;
  const uint64_t rs = static_cast<uint64_t>(a.ld_out) * (f32 ? 4 : 2);
  a.N_tma = a.N - a.N % (f32 ? 4 : 8);
  a.out = out;
  const int inner = std::max(a.N_tma, 1);
  if (!encode_map(&o0, f32, out, inner, a.rows, 1, rs, rs * a.rows, 32, 32, f32 ? 128 : 64))
    return AVEY_ERR_CUDA;
  o1 = o0;
  if (out_dt == AVEY_BF16X2 &&
      !encode_map(&o1, false, static_cast<bf16 *>(out) + static_cast<long long>(a.rows) * a.ld_out, inner,
                  a.rows, 1, rs, rs * a.rows, 32, 32, 64))
    return AVEY_ERR_CUDA;
  if (out_dt == AVEY_BF16) return run_linear_pair<BN, AVEY_BF16, false>(ma, mb, o0, o1, a, s);
  if (out_dt == AVEY_BF16X2) return run_linear_pair<BN, AVEY_BF16X2, false>(ma, mb, o0, o1, a, s);
  if (a.residual) return run_linear_pair<BN, AVEY_F32, true>(ma, mb, o0, o1, a, s);
  return run_linear_pair<BN, AVEY_F32, false>(ma, mb, o0, o1, a, s);
}

inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

}  // namespace

avey_status launch_linear_i8(const avey_linear_i8_params *p, const int8_t *xq, int64_t ld_xq,
                             const float *x_scale, int rows, const float *residual, void *out,
                             avey_dtype out_dt, int64_t ld_out, cudaStream_t s) {
  if (rows == 0) return AVEY_OK;
  LinArgs a{};
  a.rows = rows;
  a.N = p->N;
  a.K = p->K;
  a.x_scale = x_scale;
  a.w_scale = p->w_scale;
  a.bias = p->bias;
  a.relu2 = p->act == AVEY_ACT_RELU2;
  a.residual = residual;
  a.ld_out = ld_out;
  a.status = device_status_word();
  // the widest tile that still gives every pair of SMs one
  const long long tm = (rows + 255) / 256, pairs = sm_count() / 2;
  if (tm * ((p->N + 255) / 256) >= pairs) return run_linear_bn<256>(p, xq, ld_xq, a, out, out_dt, s);
  if (tm * ((p->N + 127) / 128) >= pairs) return run_linear_bn<128>(p, xq, ld_xq, a, out, out_dt, s);
  return run_linear_bn<64>(p, xq, ld_xq, a, out, out_dt, s);
}

avey_status check_linear_i8(const char *fn, const avey_linear_i8_params *p, const void *x,
                            avey_dtype x_dt, int64_t ld_x, const float *x_scale, int prenorm, int rows) {
  AVEY_REQUIRE(p != nullptr, AVEY_ERR_INVALID_ARG, "%s: null params", fn);
  AVEY_REQUIRE(rows >= 0 && p->K >= 1 && p->N >= 1, AVEY_ERR_INVALID_ARG,
               "%s: need rows >= 0, K >= 1 and N >= 1 (rows=%d K=%d N=%d)", fn, rows, p->K, p->N);
  AVEY_REQUIRE(p->K <= 131071, AVEY_ERR_UNSUPPORTED, "%s: K=%d > 131071 overflows the int32 sum", fn, p->K);
  AVEY_REQUIRE(rows <= (1 << 30) && p->N <= (1 << 30), AVEY_ERR_UNSUPPORTED,
               "%s: problem too large (rows=%d N=%d)", fn, rows, p->N);
  AVEY_REQUIRE(p->act == AVEY_ACT_NONE || p->act == AVEY_ACT_RELU2, AVEY_ERR_INVALID_ARG, "%s: bad act %d",
               fn, p->act);
  AVEY_REQUIRE(p->ld_w >= p->K && p->ld_w % 16 == 0, AVEY_ERR_INVALID_ARG,
               "%s: ld_w=%lld must be a multiple of 16, >= K=%d", fn, static_cast<long long>(p->ld_w), p->K);
  if (x_dt == AVEY_I8) {
    AVEY_REQUIRE(ld_x >= p->K && ld_x % 16 == 0, AVEY_ERR_INVALID_ARG,
                 "%s: ld_x=%lld of 8-bit rows must be a multiple of 16, >= K=%d", fn,
                 static_cast<long long>(ld_x), p->K);
    AVEY_REQUIRE(!prenorm, AVEY_ERR_INVALID_ARG, "%s: 8-bit rows carry their own scale, prenorm included", fn);
    AVEY_REQUIRE(rows == 0 || x_scale, AVEY_ERR_INVALID_ARG, "%s: 8-bit rows need x_scale", fn);
    AVEY_REQUIRE(aligned16(x) && (reinterpret_cast<uintptr_t>(x_scale) & 3) == 0, AVEY_ERR_INVALID_ARG,
                 "%s: 8-bit x 16-byte and x_scale 4-byte aligned", fn);
  } else {
    const avey_status st = check_quant_source(fn, x, x_dt, p->K, ld_x);
    if (st != AVEY_OK) return st;
    AVEY_REQUIRE(!x_scale, AVEY_ERR_INVALID_ARG, "%s: x_scale goes with 8-bit x only", fn);
  }
  AVEY_REQUIRE(rows == 0 || (x && p->Wq && p->w_scale), AVEY_ERR_INVALID_ARG, "%s: null pointer", fn);
  AVEY_REQUIRE(aligned16(p->Wq) && aligned16(p->w_scale) && aligned16(p->bias), AVEY_ERR_INVALID_ARG,
               "%s: Wq, w_scale and bias must be 16-byte aligned", fn);
  return AVEY_OK;
}

}  // namespace avey

using namespace avey;

extern "C" size_t avey_linear_i8_workspace_bytes(avey_dtype x_dt, int rows, int K) {
  if (x_dt == AVEY_I8 || rows <= 0 || K <= 0) return 0;
  return align256(static_cast<size_t>(rows) * round16(K)) + align256(static_cast<size_t>(rows) * 4);
}

extern "C" avey_status avey_linear_i8(const avey_linear_i8_params *p, const void *x, avey_dtype x_dt,
                                      int64_t ld_x, const float *x_scale, int prenorm, int rows,
                                      const float *residual, void *out, avey_dtype out_dt,
                                      int64_t ld_out, void *ws, size_t ws_bytes, avey_stream_t stream) {
  const char *fn = "avey_linear_i8";
  avey_status st = check_linear_i8(fn, p, x, x_dt, ld_x, x_scale, prenorm, rows);
  if (st != AVEY_OK) return st;
  AVEY_REQUIRE(out_dt == AVEY_F32 || out_dt == AVEY_BF16 || out_dt == AVEY_BF16X2, AVEY_ERR_UNSUPPORTED,
               "%s: output dtype %d unsupported (F32, BF16 or BF16X2)", fn, int(out_dt));
  AVEY_REQUIRE(ld_out >= p->N && ld_out % 8 == 0, AVEY_ERR_INVALID_ARG,
               "%s: ld_out=%lld must be a multiple of 8, >= N=%d", fn, static_cast<long long>(ld_out), p->N);
  AVEY_REQUIRE(!residual || out_dt == AVEY_F32, AVEY_ERR_UNSUPPORTED, "%s: a residual needs an F32 output", fn);
  AVEY_REQUIRE(!residual || p->act == AVEY_ACT_NONE, AVEY_ERR_UNSUPPORTED,
               "%s: a residual goes with AVEY_ACT_NONE", fn);
  if (rows == 0) return AVEY_OK;
  AVEY_REQUIRE(out, AVEY_ERR_INVALID_ARG, "%s: null output", fn);
  AVEY_REQUIRE(aligned16(out) && aligned16(residual), AVEY_ERR_INVALID_ARG,
               "%s: out and residual must be 16-byte aligned", fn);
  const size_t need = avey_linear_i8_workspace_bytes(x_dt, rows, p->K);
  AVEY_REQUIRE(need == 0 || (ws && (reinterpret_cast<uintptr_t>(ws) & 255) == 0), AVEY_ERR_INVALID_ARG,
               "%s: workspace must be 256-byte aligned", fn);
  AVEY_REQUIRE(ws_bytes >= need, AVEY_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu required", fn, ws_bytes,
               need);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int8_t *xq = static_cast<const int8_t *>(x);
  const float *xs = x_scale;
  int64_t ld_xq = ld_x;
  if (x_dt != AVEY_I8) {
    ld_xq = round16(p->K);
    int8_t *q = static_cast<int8_t *>(ws);
    float *sc = reinterpret_cast<float *>(q + align256(static_cast<size_t>(rows) * ld_xq));
    st = launch_quantize_rows(x, x_dt, rows, p->K, ld_x, prenorm ? 1 : 0, q, ld_xq, sc, s);
    if (st != AVEY_OK) return st;
    xq = q;
    xs = sc;
  }
  return launch_linear_i8(p, xq, ld_xq, xs, rows, residual, out, out_dt, ld_out, s);
}

// ------------------------------------------------------------- scoring ------

// Logits of the simple form live in the workspace, in chunks of rows.
static inline int64_t score_ld(int N) { return (static_cast<int64_t>(N) + 7) / 8 * 8; }
static inline int score_chunk(int rows, int N) {
  const int64_t fit = (256ll << 20) / (score_ld(N) * 4);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows, std::max<int64_t>(256, fit / 256 * 256))));
}

extern "C" size_t avey_score_tokens_i8_workspace_bytes(int rows, int K, int N) {
  if (rows <= 0 || K <= 0 || N <= 0) return 0;
  return avey_linear_i8_workspace_bytes(AVEY_F32, rows, K) +
         align256(static_cast<size_t>(score_chunk(rows, N)) * score_ld(N) * 4);
}

extern "C" avey_status avey_score_tokens_i8(const avey_linear_i8_params *p, const void *x, avey_dtype x_dt,
                                            int64_t ld_x, const float *x_scale, int prenorm, int rows,
                                            const int32_t *ids, float *logprob, float *stats,
                                            float *entropy, void *ws, size_t ws_bytes,
                                            avey_stream_t stream) {
  const char *fn = "avey_score_tokens_i8";
  avey_status st = check_linear_i8(fn, p, x, x_dt, ld_x, x_scale, prenorm, rows);
  if (st != AVEY_OK) return st;
  AVEY_REQUIRE(p->act == AVEY_ACT_NONE, AVEY_ERR_UNSUPPORTED, "%s: act must be AVEY_ACT_NONE", fn);
  AVEY_REQUIRE((ids != nullptr) == (logprob != nullptr), AVEY_ERR_INVALID_ARG,
               "%s: ids and logprob go together", fn);
  if (rows == 0) return AVEY_OK;
  AVEY_REQUIRE(logprob || stats || entropy, AVEY_ERR_INVALID_ARG, "%s: no output", fn);
  AVEY_REQUIRE(((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(logprob) |
                 reinterpret_cast<uintptr_t>(entropy)) & 3) == 0 &&
                   (reinterpret_cast<uintptr_t>(stats) & 7) == 0,
               AVEY_ERR_INVALID_ARG, "%s: stats 8-byte, other rows 4-byte aligned", fn);
  const size_t need = avey_score_tokens_i8_workspace_bytes(rows, p->K, p->N);
  AVEY_REQUIRE(ws && (reinterpret_cast<uintptr_t>(ws) & 255) == 0, AVEY_ERR_INVALID_ARG,
               "%s: workspace must be 256-byte aligned", fn);
  AVEY_REQUIRE(ws_bytes >= need, AVEY_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu required", fn, ws_bytes,
               need);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int8_t *xq = static_cast<const int8_t *>(x);
  const float *xs = x_scale;
  int64_t ld_xq = ld_x;
  if (x_dt != AVEY_I8) {
    ld_xq = round16(p->K);
    int8_t *q = static_cast<int8_t *>(ws);
    float *sc = reinterpret_cast<float *>(q + align256(static_cast<size_t>(rows) * ld_xq));
    st = launch_quantize_rows(x, x_dt, rows, p->K, ld_x, prenorm ? 1 : 0, q, ld_xq, sc, s);
    if (st != AVEY_OK) return st;
    xq = q;
    xs = sc;
  }
  float *logits = reinterpret_cast<float *>(static_cast<char *>(ws) +
                                            avey_linear_i8_workspace_bytes(AVEY_F32, rows, p->K));
  const int64_t ld = score_ld(p->N);
  const int chunk = score_chunk(rows, p->N);
  for (int r0 = 0; r0 < rows; r0 += chunk) {
    const int n = std::min(chunk, rows - r0);
    st = launch_linear_i8(p, xq + r0 * ld_xq, ld_xq, xs + r0, n, nullptr, logits, AVEY_F32, ld, s);
    if (st != AVEY_OK) return st;
    st = launch_token_logprobs(logits, AVEY_F32, n, p->N, ld, ids ? ids + r0 : nullptr, 0,
                               logprob ? logprob + r0 : nullptr, stats ? stats + 2ll * r0 : nullptr,
                               entropy ? entropy + r0 : nullptr, nullptr, nullptr, s);
    if (st != AVEY_OK) return st;
  }
  return AVEY_OK;
}
