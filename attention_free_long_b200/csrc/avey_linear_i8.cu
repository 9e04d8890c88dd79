// avey_linear_i8.cu -- y = act(s_t w_n sum_k q_tk Wq_nk + b_n) + r_tn on tcgen05
// (kind::i8, int32 accumulators in TMEM).
//
// CTA pairs (cta_group::2) own 256 x BN output tiles; roles and barriers are
// those of the layer GEMMs (avey_tc.cu): a TMA producer warp, a warp of CTA 0
// issuing the MMAs, epilogue warps, two accumulators so that the epilogue of a
// tile overlaps the MMAs of the next.  A K step is 128 bytes = 128 values, four
// MMAs of K = 32.
//
// What bounds it: long contractions the tensor pipe (8192^3 to bf16 runs at 3.0
// POP/s, 0.97 of what the pipe does at the 1.33 GHz that the power cap leaves it);
// short ones the epilogue, which has about 3100 tensor cycles a tile of K = 768 to get
// 32768 sums out of TMEM and takes about 5000.  Up to K = 1024 a pair keeps its
// 256 rows of x in shared memory and walks the channels (ARES): half the bytes
// from L2 and into shared memory, 44 instead of 48 us for 8192 x 768 x 8192 to
// bf16.
// Up to 64 tokens against many channels swap the operands: bound by one read of the
// weights (32 x 768 -> 50368 to fp32: 13.0 us, 39 MB).
#include <algorithm>
#include <utility>

#include "avey_common.cuh"
#include "avey_internal.h"
#include "avey_score.cuh"

namespace avey {
namespace {

constexpr int kBK = 128;
// K steps of x that fit beside a ring of three stages at least
constexpr int kResidentSteps = 8;

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// mbar_wait for a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait_suspend(bar, parity))) return true;
    if ((it & 127u) == 0 &&
        __any_sync(0xffffffffu, *abort != 0 || globaltimer_ns() - t0 > kWaitLimitNs))
      return false;
  }
}

// What the epilogue does with the products besides AVEY_F32, AVEY_BF16 and
// AVEY_BF16X2 (stores): running softmax statistics of each row.
constexpr int kScore = -1;

template <int BN, int OUT, bool RES, bool ARES, bool SWAP = false>
struct LinLayout {
  static constexpr int PM = 256;
  // epilogue warps: sixteen, but for fp32 outputs (8192 x 768 x 8192: 63 us with
  // eight, 69 with sixteen; 32768 x 768 x 1536 to pairs: 62 and 55) and for the two
  // chunks of a quarter's rows that swapped tiles have
  static constexpr int EPI = OUT == AVEY_F32 || SWAP ? 8 : 16;
  static constexpr int GROUPS = EPI / 4;                // warps that share a quarter's chunks
  static constexpr int THREADS = 64 + 32 * EPI;
  static constexpr uint32_t A_BYTES = 128 * kBK;        // this CTA's rows, one K step
  static constexpr uint32_t B_BYTES = (BN / 2) * kBK;   // this CTA's half of the channels
  static constexpr uint32_t STAGE_BYTES = ARES ? B_BYTES : A_BYTES + B_BYTES;
  // staging of stores (and of the residual, fetched a chunk ahead): a 32 x 32
  // chunk a buffer
  static constexpr uint32_t BUF = OUT == kScore || SWAP ? 0 : OUT == AVEY_BF16 ? 2048 : 4096;
  static constexpr int BUFS = RES ? 3 : 1;
  static constexpr uint32_t STAGING_BYTES = EPI * BUFS * BUF;
  static constexpr uint32_t CTRL_BYTES = 1024;
  // each warp's scales and biases: of a chunk, for the scores of all its chunks of a tile
  static constexpr int CHUNKS = OUT == kScore ? BN / 32 / GROUPS : 1;
  static constexpr uint32_t COLS_BYTES = EPI * CHUNKS * 64 * 4;
  static constexpr uint32_t REST_BYTES = STAGING_BYTES + CTRL_BYTES + COLS_BYTES + 1024;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  // stages and shared memory for this many K steps
  static constexpr int stages(int ksteps) {
    const uint32_t room = 232448 - REST_BYTES - (ARES ? ksteps * A_BYTES : 0);
    const int n = static_cast<int>(room / STAGE_BYTES);
    return n < 8 ? n : 8;
  }
  static constexpr uint32_t tiles_bytes(int ksteps) {
    return (ARES ? ksteps * A_BYTES : 0) + stages(ksteps) * STAGE_BYTES;
  }
  // the most that any number of K steps takes
  static constexpr uint32_t max_bytes() {
    uint32_t most = 0;
    for (int k = 1; k <= kResidentSteps; ++k) most = tiles_bytes(k) > most ? tiles_bytes(k) : most;
    return most + REST_BYTES;
  }
  static_assert(stages(ARES ? kResidentSteps : 1) >= 3, "shared memory budget");
};

struct LinArgs {
  int rows, N, K;
  int stages;            // of the ring
  uint32_t tiles_bytes;  // resident rows and ring
  int tiles_m, tiles_n;
  long long num_tiles;
  const float *x_scale, *w_scale, *bias;
  int relu2;
  const float *residual;
  long long ld_res;
  int res_tma;  // the residual's rows lie on 16-byte boundaries
  // TMA stores write whole 16-byte pieces: they cover the columns < N_tma, and
  // plain stores through out the rest of a row
  int N_tma;
  void *out;
  long long ld_out;
  float4 *partial;  // kScore: (max, sum, weighted sum) of a row's share of the words
  int *status;
};

// The tiles first, first + step, .. below end as (row block, column block).
struct TileWalk {
  long long tile, end;
  int mt, nt, step_m, step_n, tiles_n, step;
  __device__ __forceinline__ TileWalk(const LinArgs &a, long long first, long long end_, long long step_)
      : tile(first), end(end_), tiles_n(a.tiles_n), step(static_cast<int>(step_)) {
    mt = static_cast<int>(first / a.tiles_n);
    nt = static_cast<int>(first - static_cast<long long>(mt) * a.tiles_n);
    step_m = step / a.tiles_n;
    step_n = step - step_m * a.tiles_n;
  }
  __device__ __forceinline__ bool more() const { return tile < end; }
  __device__ __forceinline__ void next() {
    tile += step;
    mt += step_m;
    nt += step_n;
    if (nt >= tiles_n) {
      nt -= tiles_n;
      ++mt;
    }
  }
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

__device__ __forceinline__ void ld_shared4(uint32_t addr, float (&r)[4]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
               : "r"(addr)
               : "memory");
}

// First tile of pair p's share: shares are contiguous in the order (row block,
// column block).
__host__ __device__ __forceinline__ long long share_start(long long p, long long tiles, int npairs) {
  return p * tiles / npairs;
}

// The columns from N_tma of a row's 32-column chunk, residual included.
template <int OUT, bool RES>
__device__ __forceinline__ void store_rest(const LinArgs &a, int row, int col0, const float (&v)[32]) {
  const long long at = static_cast<long long>(row) * a.ld_out;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int c = col0 + j;
    if (c < a.N_tma || c >= a.N) continue;
    if constexpr (OUT == AVEY_F32) {
      static_cast<float *>(a.out)[at + c] = RES && a.res_tma ? v[j] + a.residual[row * a.ld_res + c] : v[j];
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

// Scale, bias and activation of a 32-column chunk of int32 sums; w and b are
// the chunk's columns in shared memory.
__device__ __forceinline__ void lin_values(float (&v)[32], float xs, const float *w, const float *b,
                                           int relu2) {
  const float2 x2 = make_float2(xs, xs);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 w4 = *reinterpret_cast<const float4 *>(w + 4 * q);
    const float4 b4 = *reinterpret_cast<const float4 *>(b + 4 * q);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 f = make_float2(static_cast<float>(__float_as_int(v[4 * q + 2 * h])),
                                   static_cast<float>(__float_as_int(v[4 * q + 2 * h + 1])));
      const float2 y = ffma2(fmul2(f, x2), h ? make_float2(w4.z, w4.w) : make_float2(w4.x, w4.y),
                             h ? make_float2(b4.z, b4.w) : make_float2(b4.x, b4.y));
      v[4 * q + 2 * h] = y.x;
      v[4 * q + 2 * h + 1] = y.y;
    }
  }
  if (relu2) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 y = make_float2(max_nan(v[j], 0.f), max_nan(v[j + 1], 0.f));  // NaN stays NaN
      const float2 z = fmul2(y, y);
      v[j] = z.x;
      v[j + 1] = z.y;
    }
  }
}

// The same with channels as rows (this lane's scale ws and bias bs) and tokens as
// columns, whose scales are w.
__device__ __forceinline__ void lin_values_swapped(float (&v)[32], float ws, float bs, const float *x, int relu2) {
  const float2 w2 = make_float2(ws, ws), b2 = make_float2(bs, bs);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 x4 = *reinterpret_cast<const float4 *>(x + 4 * q);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 f = make_float2(static_cast<float>(__float_as_int(v[4 * q + 2 * h])),
                                   static_cast<float>(__float_as_int(v[4 * q + 2 * h + 1])));
      float2 y = ffma2(fmul2(f, h ? make_float2(x4.z, x4.w) : make_float2(x4.x, x4.y)), w2, b2);
      if (relu2) {
        y = make_float2(max_nan(y.x, 0.f), max_nan(y.y, 0.f));  // NaN stays NaN
        y = fmul2(y, y);
      }
      v[4 * q + 2 * h] = y.x;
      v[4 * q + 2 * h + 1] = y.y;
    }
  }
}

// A 32 x 32 chunk of channels x tokens: each token's 32 channels are one store.
template <int OUT>
__device__ __forceinline__ void store_swapped(const LinArgs &a, int channel, int token0, float (&v)[32]) {
  if (OUT == AVEY_F32 && a.residual) {  // all loads before the first store, which it might be
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (token0 + j < a.N) v[j] += a.residual[static_cast<long long>(token0 + j) * a.ld_res + channel];
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const long long t = token0 + j;
    if (t >= a.N) break;
    const float y = v[j];
    if constexpr (OUT == AVEY_F32) {
      static_cast<float *>(a.out)[t * a.ld_out + channel] = y;
    } else {
      bf16 *hi = static_cast<bf16 *>(a.out) + t * a.ld_out + channel;
      *hi = __float2bfloat16_rn(y);
      if constexpr (OUT == AVEY_BF16X2) {
        float h, l;
        split_bf16(y, h, l);
        hi[a.N * a.ld_out] = __float2bfloat16_rn(l);
      }
    }
  }
}

// A pair of sums of columns 2 j, 2 j + 1 as logits in units of log 2.
__device__ __forceinline__ float2 score_pair(uint32_t r0, uint32_t r1, float xs, const float *w, const float *b, int j) {
  const float2 f = make_float2(static_cast<float>(static_cast<int>(r0)), static_cast<float>(static_cast<int>(r1)));
  return ffma2(fmul2(f, make_float2(xs, xs)), *reinterpret_cast<const float2 *>(w + 2 * j),
               *reinterpret_cast<const float2 *>(b + 2 * j));
}

// A tile's columns of this warp into a row's running statistics, 16 at a time: the
// exponentials of one part are computed among the logits of the next, so that
// neither the exponential unit nor the others wait for a whole part.
template <int PARTS>
__device__ __forceinline__ void score_tile(uint32_t taddr, uint32_t step, float xs, const float *cols, Stat2 &st) {
  uint32_t raw[16];
  float2 y[8];
  tmem_ld16(taddr, raw);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = score_pair(raw[2 * j], raw[2 * j + 1], xs, cols, cols + 32, j);
#pragma unroll
  for (int h = 0; h < PARTS; ++h) {
    float m = st.m;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max3f(m, y[j].x, y[j].y);
    rebase2(st, m);
    const float2 minus = make_float2(-m, -m);
    float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, t[2] = {s[0], s[0]};
    if (h + 1 < PARTS) tmem_ld16(taddr + ((h + 1) >> 1) * step + ((h + 1) & 1) * 16, raw);
    const float *w = cols + ((h + 1) >> 1) * 64 + ((h + 1) & 1) * 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 d = fadd2(y[j], minus);
      const float2 e = make_float2(ex2(d.x), ex2(d.y));
      if (h + 1 < PARTS) y[j] = score_pair(raw[2 * j], raw[2 * j + 1], xs, w, w + 32, j);
      s[j & 1] = fadd2(s[j & 1], e);
      t[j & 1] = ffma2(e, d, t[j & 1]);
    }
    s[0] = fadd2(s[0], s[1]);
    t[0] = fadd2(t[0], t[1]);
    st.s += s[0].x + s[0].y;
    st.t += t[0].x + t[0].y;
  }
}

// SWAP: few tokens against many channels.  The channels are the rows (A), the
// tokens the columns, so that all lanes of TMEM and all epilogue warps have work;
// LinArgs' rows counts channels and N tokens, and outputs go straight to memory.
template <int BN, int OUT, bool RES, bool ARES, bool SWAP = false>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(LinLayout<BN, OUT, RES, ARES, SWAP>::THREADS, 1)
    linear_i8_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmO0, const __grid_constant__ CUtensorMap tmO1,
                   const __grid_constant__ CUtensorMap tmR, const LinArgs a) {
  using P = LinLayout<BN, OUT, RES, ARES, SWAP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  const int kchunks = (a.K + kBK - 1) / kBK;
  // shared memory: resident rows (ARES), ring, staging, control block, columns
  const uint32_t abase = raw_s + pad;
  const uint32_t sbase = abase + (ARES ? static_cast<uint32_t>(kchunks) * P::A_BYTES : 0u);
  const uint32_t gbase = abase + a.tiles_bytes;
  const uint32_t cbase = gbase + P::STAGING_BYTES;
  uint8_t *ctrl = smem_raw + pad + a.tiles_bytes + P::STAGING_BYTES;
  // control block: full[8] @0, empty[8] @64, tfull[2] @128, tempty[2] @144,
  // drain @160, tmem base @168, abort flag @172, afull[8] @192, aempty[8] @256,
  // residual[8 warps][3] @320
  auto full_bar = [&](int s) { return cbase + 8u * s; };
  auto empty_bar = [&](int s) { return cbase + 64u + 8u * s; };
  auto tfull_bar = [&](int i) { return cbase + 128u + 8u * i; };
  auto tempty_bar = [&](int i) { return cbase + 144u + 8u * i; };
  const uint32_t drain_bar = cbase + 160u;
  volatile uint32_t *tmem_holder = reinterpret_cast<volatile uint32_t *>(ctrl + 168);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(ctrl + 172);
  auto afull_bar = [&](int k) { return cbase + 192u + 8u * k; };
  auto aempty_bar = [&](int k) { return cbase + 256u + 8u * k; };
  auto res_bar = [&](int w, int i) { return cbase + 320u + 24u * w + 8u * i; };
  static_assert(320 + 24 * 8 <= P::CTRL_BYTES && kResidentSteps <= 8, "control block");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  // Tiles of this pair: dealt round robin, or a contiguous share, so that rows
  // stay in shared memory and a row's statistics in one thread's registers.
  constexpr bool SHARE = ARES || OUT == kScore;
  const long long t_first = SHARE ? share_start(pair, a.num_tiles, npairs) : pair;
  const long long t_end = SHARE ? share_start(pair + 1, a.num_tiles, npairs) : a.num_tiles;
  const long long t_step = SHARE ? 1 : npairs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull_bar(i), 1);
      mbar_init(tempty_bar(i), 2 * P::EPI);
    }
    mbar_init(drain_bar, 1);
    if (ARES) {
      for (int k = 0; k < kchunks; ++k) {
        mbar_init(afull_bar(k), 1);
        mbar_init(aempty_bar(k), 1);
      }
    }
    if (RES) {
      for (int w = 0; w < P::EPI; ++w)
        for (int i = 0; i < P::BUFS; ++i) mbar_init(res_bar(w, i), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    if (OUT != kScore && !SWAP) prefetch_tmap(&tmO0);
    if (OUT == AVEY_BF16X2 && !SWAP) prefetch_tmap(&tmO1);
    if (RES) prefetch_tmap(&tmR);
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
  grid_wait();  // the rows may still be on their way through the rounding kernel

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The whole warp walks the loop, so that addresses stay in uniform
    // registers; one lane issues.
    const bool one = elect_one();
    const uint32_t full0 = mapa_shared(full_bar(0), 0), afull0 = mapa_shared(afull_bar(0), 0);
    int stage = 0;
    uint32_t phase = 0, aphase = 0;
    long long issued = 0;
    bool ok = true, fresh = true;  // fresh: the pair's first tile of a row block
    for (TileWalk w(a, t_first, t_end, t_step); ok && w.more(); w.next()) {
      const int arow = w.mt * P::PM + static_cast<int>(rank) * 128;
      const int brow = w.nt * BN + static_cast<int>(rank) * (BN / 2);
      fresh = fresh || w.nt == 0;
      for (int kc = 0; kc < kchunks; ++kc) {
        if (ARES && fresh) {
          if (!warp_wait(aempty_bar(kc), aphase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (one) {
            if (rank == 0) mbar_arrive_expect_tx(afull_bar(kc), 2 * P::A_BYTES);
            tma_load_3d_pair(abase + kc * P::A_BYTES, &tmA, afull0 + 8u * kc, kc * kBK, arow, 0);
          }
        }
        if (!warp_wait(empty_bar(stage), phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t st = sbase + stage * P::STAGE_BYTES, bar = full0 + 8u * stage;
        if (one) {
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * P::STAGE_BYTES);
          if (!ARES) tma_load_3d_pair(st, &tmA, bar, kc * kBK, arow, 0);
          tma_load_3d_pair(ARES ? st : st + P::A_BYTES, &tmB, bar, kc * kBK, brow, 0);
        }
        ++issued;
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ARES && fresh) aphase ^= 1u;
      fresh = false;
    }
    if (one) {
      if (!ok) {
        *abort_flag = 1;
        record_status(a.status, AVEY_ERR_DEVICE_TIMEOUT);
      }
      // Drain: a stage's last use is over once the pair's MMA has released it
      // (and with it every earlier read of the resident rows).
      for (int s = 0; s < a.stages; ++s) {
        if (issued > s) {
          const long long last = ((issued - 1 - s) / a.stages) * a.stages + s;
          drain_wait(empty_bar(s), static_cast<uint32_t>((last / a.stages) & 1));
        }
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------- MMA issue (CTA 0)
    // Issued from one thread's own loop, a 128-byte K step took about 1000
    // cycles, twice the tensor time of its four MMAs; warp-uniform code keeps
    // descriptors in uniform registers.
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_s8_s32(P::PM, BN);
      const bool one = elect_one();
      const int last_steps = (a.K - (kchunks - 1) * kBK + 31) / 32;  // MMAs of the last K step; the rest is zeros
      const uint64_t desc_a = sdesc_k_sw128(abase), desc_s = sdesc_k_sw128(sbase);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0, aphase = 0;
      bool ok = true, fresh = true;
      for (TileWalk w(a, t_first, t_end, t_step); ok && w.more();) {
        if (!warp_wait(tempty_bar(acc), acc_phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        fresh = fresh || w.nt == 0;
        const bool leave = w.nt == a.tiles_n - 1;  // the row block's last tile
        w.next();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kc = 0; kc < kchunks; ++kc) {
          if (ARES && fresh && !warp_wait(afull_bar(kc), aphase, abort_flag)) {
            ok = false;
            break;
          }
          if (!warp_wait(full_bar(stage), phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ds = desc_s + static_cast<uint32_t>(stage) * (P::STAGE_BYTES >> 4);
          const uint64_t da = ARES ? desc_a + static_cast<uint32_t>(kc) * (P::A_BYTES >> 4) : ds;
          const uint64_t db = ARES ? ds : ds + (P::A_BYTES >> 4);
          const bool whole = kc + 1 < kchunks || last_steps == kBK / 32;
          if (one) {
            tc_mma_i8_pair(d_tmem, da, db, idesc, kc != 0);
            if (whole) {
#pragma unroll
              for (int kk = 1; kk < kBK / 32; ++kk) tc_mma_i8_pair(d_tmem, da + 2u * kk, db + 2u * kk, idesc, 1u);
            } else {
              for (int kk = 1; kk < last_steps; ++kk)
                tc_mma_i8_pair(d_tmem, da + 2u * kk, db + 2u * kk, idesc, 1u);
            }
            tc_commit_pair_both(empty_bar(stage));
            if (ARES && leave) tc_commit_pair_both(aempty_bar(kc));
            if (kc + 1 == kchunks) tc_commit_pair_both(tfull_bar(acc));
          }
          __syncwarp();
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ARES && fresh) aphase ^= 1u;
        fresh = false;
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (one) {
        if (!ok) {
          *abort_flag = 1;
          record_status(a.status, AVEY_ERR_DEVICE_TIMEOUT);
        }
        tc_commit_pair_both(drain_bar);
        drain_wait(drain_bar, 0);
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    // A warp has a quarter of the CTA's rows (TMEM lanes 32*quarter .. +31) and
    // every GROUPS-th 32-column chunk.
    const int ew = warp - 2, quarter = warp & 3, group = ew >> 2;
    const uint32_t stg = gbase + static_cast<uint32_t>(ew) * P::BUFS * P::BUF;
    const uint32_t tempty_r0 = mapa_shared(tempty_bar(0), 0), tempty_r1 = mapa_shared(tempty_bar(1), 0);
    float *cols = reinterpret_cast<float *>(ctrl + P::CTRL_BYTES) + ew * P::CHUNKS * 64;  // [chunk][scale, bias][32]
    auto row_of = [&](int mt) { return mt * P::PM + static_cast<int>(rank) * 128 + quarter * 32; };
    auto row_scale = [&](int mt) {
      const int row = row_of(mt) + lane;
      return row < a.rows ? __ldg((SWAP ? a.w_scale : a.x_scale) + row) * (OUT == kScore ? kLog2e : 1.f) : 0.f;
    };
    auto row_bias = [&](int mt) {
      const int row = row_of(mt) + lane;
      return SWAP && a.bias && row < a.rows ? __ldg(a.bias + row) : 0.f;
    };
    // Scale and bias of this lane's column of CHUNKS chunks from column block nt,
    // chunk ch: fetched a chunk (scores: a tile) ahead, and nothing is computed
    // from the loads before they are stored.  The scores work in units of log 2,
    // where words past the last have the value -1e30, as those with a bias below
    // it (-inf among them): finite, so that 0 * (y - m) stays 0.
    float cw[P::CHUNKS], cb[P::CHUNKS];
    auto fetch_columns = [&](int nt, int ch) {
#pragma unroll
      for (int i = 0; i < P::CHUNKS; ++i) {
        const int c = nt * BN + (ch + i * P::GROUPS) * 32 + lane;
        cw[i] = 0.f;
        cb[i] = OUT == kScore ? kMaskedWord : 0.f;
        if (c < a.N) {
          cw[i] = __ldg((SWAP ? a.x_scale : a.w_scale) + c);
          if (!SWAP && a.bias)
            cb[i] = __ldg(a.bias + c);
          else if (OUT == kScore)
            cb[i] = 0.f;
        }
      }
    };
    auto put_columns = [&]() {
#pragma unroll
      for (int i = 0; i < P::CHUNKS; ++i) {
        cols[i * 64 + lane] = cw[i];
        cols[i * 64 + 32 + lane] = OUT == kScore ? max_nan(cb[i] * kLog2e, kMaskedWord) : cb[i];
      }
      __syncwarp();
    };
    // The residual of a chunk into staging buffer `to`, a chunk ahead.
    uint32_t coming = 0;  // buffers with a copy in flight
    auto fetch_residual = [&](int row0, int col0, int to) {
      if (!a.res_tma) {
        // a row's 32 columns at a time, four bytes a lane
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
        const int n = min(32, a.rows - row0);
        const float *r = a.residual + row0 * a.ld_res + col0 + lane;
        const uint32_t at = stg + to * P::BUF + (lane & 3) * 4;
        if (col0 + lane < a.N) {
#pragma unroll 8
          for (int j = 0; j < n; ++j) cp_async4(at + lin_sw128(j, lane >> 2), r + j * a.ld_res);
        }
        cp_async_commit();
        return;
      }
      if (col0 >= a.N_tma) return;
      if (lane == 0) {
        bulk_wait_read<1>();  // the store from this buffer, three chunks ago at least, has read it
        mbar_arrive_expect_tx(res_bar(ew, to), P::BUF);
        tma_load_3d(stg + to * P::BUF, &tmR, res_bar(ew, to), col0, row0, 0);
      }
      coming |= 1u << to;
    };
    int acc = 0, buf = 0;
    uint32_t acc_phase = 0, res_phase = 0;  // res_phase: a bit for each buffer
    bool ok = true, have = false;           // have: this chunk's columns and residual have been fetched
    TileWalk walk(a, t_first, t_end, t_step);
    float xs_next = walk.more() ? row_scale(walk.mt) : 0.f, bs_next = walk.more() ? row_bias(walk.mt) : 0.f;
    if (OUT == kScore && walk.more()) fetch_columns(walk.nt, group);
    Stat2 st{kLowest, 0.f, 0.f};
    while (walk.more()) {
      const int mt = walk.mt, nt = walk.nt;
      walk.next();  // the tile after this one
      const int row0 = row_of(mt);
      const int row = row0 + lane;
      const bool valid = row < a.rows;
      const float xs = xs_next, bs = bs_next;
      if (walk.more() && walk.mt != mt) {
        xs_next = row_scale(walk.mt);
        bs_next = row_bias(walk.mt);
      }
      if constexpr (OUT == kScore) {
        __syncwarp();  // the last tile's columns have been read
        put_columns();
        if (walk.more()) fetch_columns(walk.nt, group);
      }
      if (!warp_wait(tfull_bar(acc), acc_phase, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t taddr =
          tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(quarter * 32) << 16);
      if constexpr (OUT == kScore) {
        // words past the last have their value
        if (row0 < a.rows) score_tile<2 * P::CHUNKS>(taddr + group * 32, P::GROUPS * 32, xs, cols, st);
      }
#pragma unroll 1
      for (int ch = OUT == kScore ? BN / 32 : group; ch < BN / 32; ch += P::GROUPS) {
        const int col0 = nt * BN + ch * 32;
        if (col0 >= a.N || row0 >= a.rows) break;  // warp-uniform
        const float *w_s = cols, *b_s = w_s + 32;
        const int this_buf = buf;
        if constexpr (P::BUFS > 1) buf = buf + 1 == P::BUFS ? 0 : buf + 1;
        if constexpr (OUT != kScore) {
          if (!have) {
            fetch_columns(nt, ch);
            if constexpr (RES) fetch_residual(row0, col0, this_buf);
          }
          put_columns();
          // the next chunk: of this tile, or the first of the next one
          const bool here = ch + P::GROUPS < BN / 32 && col0 + 32 * P::GROUPS < a.N;
          const int nrow = here ? row0 : row_of(walk.mt);
          const int nnt = here ? nt : walk.nt, nch = here ? ch + P::GROUPS : group;
          have = (here || walk.more()) && nrow < a.rows && nnt * BN + nch * 32 < a.N;
          if (have) {
            fetch_columns(nnt, nch);
            if constexpr (RES) fetch_residual(nrow, nnt * BN + nch * 32, buf);
          }
        }
        float v[32];
        tmem_ld32(taddr + ch * 32, v);
        if constexpr (SWAP) {
          lin_values_swapped(v, xs, bs, w_s, a.relu2);
          __syncwarp();
          if (valid) store_swapped<OUT>(a, row, col0, v);
        } else {
          lin_values(v, xs, w_s, b_s, a.relu2);
          __syncwarp();
          const uint32_t at = stg + this_buf * P::BUF;
          auto add_residual = [&]() {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float r[4];
              ld_shared4(at + lin_sw128(lane, c), r);
#pragma unroll
              for (int j = 0; j < 4; ++j) v[4 * c + j] += r[j];
            }
          };
          if (RES && !a.res_tma) {
            // all but the copies of the next chunk, which are under way if it has been fetched
            if (have)
              cp_async_wait<1>();
            else
              cp_async_wait<0>();
            __syncwarp();
            add_residual();
          }
          if (col0 + 32 > a.N_tma && valid) store_rest<OUT, RES>(a, row, col0, v);
          if (col0 < a.N_tma) {  // warp-uniform
            if (RES && a.res_tma) {
              if (!warp_wait(res_bar(ew, this_buf), res_phase >> this_buf & 1u, abort_flag)) {
                ok = false;
                break;
              }
              res_phase ^= 1u << this_buf;
              coming &= ~(1u << this_buf);
              add_residual();
            } else {
              // the last store issued from this buffer must have read it
              if (lane == 0) bulk_wait_read<P::BUFS - 1>();
              __syncwarp();
            }
            if constexpr (OUT == AVEY_F32) {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                lin_st4(at + lin_sw128(lane, c), __float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                        __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
            } else if constexpr (OUT == AVEY_BF16) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                lin_st4(at + lin_sw64(lane, c), pack_bf16(v[8 * c], v[8 * c + 1]),
                        pack_bf16(v[8 * c + 2], v[8 * c + 3]), pack_bf16(v[8 * c + 4], v[8 * c + 5]),
                        pack_bf16(v[8 * c + 6], v[8 * c + 7]));
            } else {
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) split_pack(v[2 * j], v[2 * j + 1], hi[j], lo[j]);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                lin_st4(at + lin_sw64(lane, c), hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
                lin_st4(at + 2048 + lin_sw64(lane, c), lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&tmO0, at, col0, row0, 0);
              if constexpr (OUT == AVEY_BF16X2) tma_store_3d(&tmO1, at + 2048, col0, row0, 0);
            }
          }
          if (lane == 0) bulk_commit();  // one group a chunk, an empty one too
        }
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc ? tempty_r1 : tempty_r0);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
      if constexpr (OUT == kScore) {
        // the row block or the share ends here: pair p meets row block mt in
        // slot p + mt alone, since both only grow along the tiles
        if (nt == a.tiles_n - 1 || !walk.more()) {
          const long long slot = static_cast<long long>(pair) + mt;
          a.partial[(slot * P::GROUPS + group) * 256 + static_cast<int>(rank) * 128 + quarter * 32 + lane] =
              make_float4(st.m, st.s, st.t, 0.f);
          st = Stat2{kLowest, 0.f, 0.f};
        }
      }
    }
    if (!ok) {
      *abort_flag = 1;
      record_status(a.status, AVEY_ERR_DEVICE_TIMEOUT);
      if constexpr (RES) {
        // residual copies in flight must land before the block leaves
        cp_async_wait<0>();
        if (lane == 0)
          for (int i = 0; i < P::BUFS; ++i)
            if (coming >> i & 1u) drain_wait(res_bar(ew, i), res_phase >> i & 1u);
      }
    }
    if (OUT != kScore && !SWAP && lane == 0) bulk_wait_all();  // outputs written
  }

  tc_fence_before();
  __syncthreads();
  if (OUT == kScore) grid_release();
  // Both CTAs past their loops: the pair's MMAs have drained and no remote
  // arrival is still on its way.
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, P::TMEM_COLS);
  }
  cluster_sync_all();
}

template <int BN, int OUT, bool RES, bool ARES, bool SWAP = false>
avey_status run_linear_pair(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &o0,
                            const CUtensorMap &o1, const CUtensorMap &r, LinArgs a, int pairs, bool after,
                            cudaStream_t st) {
  using P = LinLayout<BN, OUT, RES, ARES, SWAP>;
  auto kern = linear_i8_pair<BN, OUT, RES, ARES, SWAP>;
  const int ksteps = (a.K + kBK - 1) / kBK;
  a.stages = P::stages(ksteps);
  a.tiles_bytes = P::tiles_bytes(ksteps);
  const uint32_t bytes = a.tiles_bytes + P::REST_BYTES;
  // the limit is the kernel's, whichever thread calls it: always the largest, so that no
  // call lowers another's before its launch
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(P::max_bytes()));
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_detail("linear_i8: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    return AVEY_ERR_CUDA;
  }
  if (after) {
    e = launch_after(kern, 2 * pairs, P::THREADS, bytes, st, ma, mb, o0, o1, r, a);
    if (e != cudaSuccess) {
      cudaGetLastError();
      set_detail("linear_i8 launch failed: %s", cudaGetErrorString(e));
      return AVEY_ERR_CUDA;
    }
  } else {
    kern<<<2 * pairs, P::THREADS, bytes, st>>>(ma, mb, o0, o1, r, a);
  }
  AVEY_CHECK_LAUNCH(OUT == kScore ? "score_i8" : "linear_i8", st);
  return AVEY_OK;
}

inline int pairs_for(long long tiles) {
  return static_cast<int>(std::min<long long>(tiles, std::max(1, sm_count() / 2)));
}

template <int BN>
avey_status run_linear_bn(const avey_linear_i8_params *p, const int8_t *xq, int64_t ld_xq, LinArgs a,
                          void *out, avey_dtype out_dt, bool after, cudaStream_t s) {
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
  CUtensorMap mr = o0;
  const uint64_t res_rs = static_cast<uint64_t>(a.ld_res) * 4;
  a.res_tma = a.residual && aligned16(a.residual) && res_rs % 16 == 0;
  if (a.res_tma && !encode_map(&mr, true, a.residual, inner, a.rows, 1, res_rs, res_rs * a.rows, 32, 32, 128))
    return AVEY_ERR_CUDA;
  const int pairs = pairs_for(a.num_tiles);
#define AVEY_LINEAR(OUT, ARES) run_linear_pair<BN, OUT, false, ARES>(ma, mb, o0, o1, mr, a, pairs, after, s)
  if (a.residual) return run_linear_pair<BN, AVEY_F32, true, false>(ma, mb, o0, o1, mr, a, pairs, after, s);
  // fp32 outputs and pairs are bound by their stores (8192 x 768 x 8192 to fp32:
  // 61 us with x in the ring, 65 resident; to bf16: 48 and 44)
  if constexpr (BN == 256) {
    if (a.K <= kBK * kResidentSteps && out_dt == AVEY_BF16) return AVEY_LINEAR(AVEY_BF16, true);
  }
  if (out_dt == AVEY_BF16) return AVEY_LINEAR(AVEY_BF16, false);
  if (out_dt == AVEY_BF16X2) return AVEY_LINEAR(AVEY_BF16X2, false);
  return AVEY_LINEAR(AVEY_F32, false);
#undef AVEY_LINEAR
}

constexpr int kSwapRows = 64;
inline bool swap_pays(int rows, int N) { return rows <= kSwapRows && (N + 255ll) / 256 * 8 > sm_count(); }

// Up to kSwapRows tokens against all channels, channels as rows.
avey_status run_linear_swapped(const avey_linear_i8_params *p, const int8_t *xq, int64_t ld_xq, LinArgs a,
                               void *out, avey_dtype out_dt, bool after, cudaStream_t s) {
  CUtensorMap ma, mb;
  if (!encode_i8_map(&ma, p->Wq, a.K, a.N, p->ld_w, 128)) return AVEY_ERR_CUDA;
  if (!encode_i8_map(&mb, xq, a.K, a.rows, ld_xq, kSwapRows / 2)) return AVEY_ERR_CUDA;
  std::swap(a.rows, a.N);
  a.tiles_m = (a.rows + 255) / 256;
  a.tiles_n = 1;
  a.num_tiles = a.tiles_m;
  a.out = out;
  const int pairs = pairs_for(a.num_tiles);
#define AVEY_LINEAR(OUT) run_linear_pair<kSwapRows, OUT, false, false, true>(ma, mb, ma, ma, ma, a, pairs, after, s)
  if (out_dt == AVEY_BF16) return AVEY_LINEAR(AVEY_BF16);
  if (out_dt == AVEY_BF16X2) return AVEY_LINEAR(AVEY_BF16X2);
  return AVEY_LINEAR(AVEY_F32);
#undef AVEY_LINEAR
}

inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

}  // namespace

avey_status launch_linear_i8(const avey_linear_i8_params *p, const int8_t *xq, int64_t ld_xq,
                             const float *x_scale, int rows, const float *residual, int64_t ld_res,
                             void *out, avey_dtype out_dt, int64_t ld_out, bool after, cudaStream_t s) {
  if (rows == 0) return AVEY_OK;
  if (linear_few_fits(rows, p->K))
    return launch_linear_few(p, xq, AVEY_I8, ld_xq, x_scale, 0, rows, residual, ld_res, out, out_dt, ld_out, s);
  LinArgs a{};
  a.rows = rows;
  a.N = p->N;
  a.K = p->K;
  a.x_scale = x_scale;
  a.w_scale = p->w_scale;
  a.bias = p->bias;
  a.relu2 = p->act == AVEY_ACT_RELU2;
  a.residual = residual;
  a.ld_res = ld_res;
  a.ld_out = ld_out;
  a.status = device_status_word();
  // Up to 64 tokens against many channels: channels as rows (32 x 768 x 50368 to
  // fp32: 17.3 us as a tile of 256 tokens, of which two of eight warps' lanes hold
  // one, 13.0 so; 16384 channels 10.3 and 8.1, 4096 6.4 and 6.4, 1536 6.2 and 6.4;
  // 128 tokens to bf16 15.6 and 17.0).
  const long long tm = (rows + 255) / 256, pairs = sm_count() / 2;
  if (swap_pays(rows, p->N))
    return run_linear_swapped(p, xq, ld_xq, a, out, out_dt, after, s);
  // The widest tile that gives every pair of SMs one, 128 columns down to every
  // second pair (1003 x 1008 x 2048: 9.8 us with 64, 9.0 with 128, 11.2 with 256;
  // 256 x 256 x 256: 5.5, 6.4 and 8.2; 4096 x 768 x 1536: 16.4, 12.2 and 12.4;
  // 32768 x 768 x 1536: 64, 44 and 38).
  if (tm * ((p->N + 255) / 256) >= pairs) return run_linear_bn<256>(p, xq, ld_xq, a, out, out_dt, after, s);
  if (2 * tm * ((p->N + 127) / 128) >= pairs) return run_linear_bn<128>(p, xq, ld_xq, a, out, out_dt, after, s);
  return run_linear_bn<64>(p, xq, ld_xq, a, out, out_dt, after, s);
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

// x as 8-bit rows at the start of the workspace.
static size_t quantized_bytes(int rows, int K) {
  return align256(static_cast<size_t>(rows) * round16(K)) + align256(static_cast<size_t>(rows) * 4);
}
static avey_status quantize_to_ws(const avey_linear_i8_params *p, const void *x, avey_dtype x_dt, int64_t ld_x,
                                  int prenorm, int rows, void *ws, const int8_t **xq, int64_t *ld_xq,
                                  const float **xs, cudaStream_t s) {
  *ld_xq = round16(p->K);
  int8_t *q = static_cast<int8_t *>(ws);
  float *sc = reinterpret_cast<float *>(q + align256(static_cast<size_t>(rows) * *ld_xq));
  *xq = q;
  *xs = sc;
  return launch_quantize_rows(x, x_dt, rows, p->K, ld_x, prenorm ? 1 : 0, q, *ld_xq, sc, s);
}

extern "C" size_t avey_linear_i8_workspace_bytes(avey_dtype x_dt, int rows, int K) {
  if (x_dt == AVEY_I8 || rows <= 0 || K <= 0 || linear_few_quantizes(x_dt, rows, K)) return 0;
  return quantized_bytes(rows, K);
}

extern "C" avey_status avey_linear_i8(const avey_linear_i8_params *p, const void *x, avey_dtype x_dt,
                                      int64_t ld_x, const float *x_scale, int prenorm, int rows,
                                      const float *residual, int64_t ld_res, void *out,
                                      avey_dtype out_dt, int64_t ld_out, void *ws, size_t ws_bytes,
                                      avey_stream_t stream) {
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
  AVEY_REQUIRE(!residual || ld_res >= p->N, AVEY_ERR_INVALID_ARG, "%s: ld_res=%lld < N=%d", fn,
               static_cast<long long>(ld_res), p->N);
  if (rows == 0) return AVEY_OK;
  AVEY_REQUIRE(out, AVEY_ERR_INVALID_ARG, "%s: null output", fn);
  AVEY_REQUIRE(aligned16(out) && (reinterpret_cast<uintptr_t>(residual) & 3) == 0, AVEY_ERR_INVALID_ARG,
               "%s: out must be 16-byte and the residual 4-byte aligned", fn);
  {
    const uint64_t n = rows, N = p->N, K = p->K;
    const uint64_t oes = out_dt == AVEY_F32 ? 4 : 2, xes = x_dt == AVEY_I8 ? 1 : x_dt == AVEY_F32 ? 4 : 2;
    const ByteRows o{reinterpret_cast<uintptr_t>(out), out_dt == AVEY_BF16X2 ? 2 * n : n, N * oes, ld_out * oes};
    const ByteRows xr{reinterpret_cast<uintptr_t>(x), x_dt == AVEY_BF16X2 ? 2 * n : n, K * xes, ld_x * xes};
    const ByteRows r{reinterpret_cast<uintptr_t>(residual), n, N * 4, static_cast<uint64_t>(ld_res) * 4};
    AVEY_REQUIRE(!rows_overlap(o, xr), AVEY_ERR_INVALID_ARG, "%s: out overlaps x", fn);
    AVEY_REQUIRE(!residual || (r.at == o.at && (ld_res == ld_out || rows == 1)) || !rows_overlap(o, r),
                 AVEY_ERR_INVALID_ARG, "%s: out overlaps the residual without being it", fn);
  }
  const size_t need = avey_linear_i8_workspace_bytes(x_dt, rows, p->K);
  AVEY_REQUIRE(need == 0 || (ws && (reinterpret_cast<uintptr_t>(ws) & 255) == 0), AVEY_ERR_INVALID_ARG,
               "%s: workspace must be 256-byte aligned", fn);
  AVEY_REQUIRE(ws_bytes >= need, AVEY_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu required", fn, ws_bytes,
               need);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (linear_few_quantizes(x_dt, rows, p->K))
    return launch_linear_few(p, x, x_dt, ld_x, nullptr, prenorm ? 1 : 0, rows, residual, ld_res, out, out_dt, ld_out, s);
  const int8_t *xq = static_cast<const int8_t *>(x);
  const float *xs = x_scale;
  int64_t ld_xq = ld_x;
  if (x_dt != AVEY_I8) {
    st = quantize_to_ws(p, x, x_dt, ld_x, prenorm, rows, ws, &xq, &ld_xq, &xs, s);
    if (st != AVEY_OK) return st;
  }
  return launch_linear_i8(p, xq, ld_xq, xs, rows, residual, ld_res, out, out_dt, ld_out, x_dt != AVEY_I8, s);
}

// ------------------------------------------------------------- scoring ------

namespace avey {
namespace {

constexpr int kScoreGroups = LinLayout<256, kScore, false, true>::GROUPS;

// One warp per row: joins the row's partial statistics, and computes the given
// token's logit again from its K bytes of either operand.
__global__ void __launch_bounds__(256)
    score_join(const LinArgs a, int npairs, const int8_t *__restrict__ xq, long long ld_xq,
               const int8_t *__restrict__ Wq, long long ld_w, const int32_t *__restrict__ ids,
               float *__restrict__ logprob, float *__restrict__ stats, float *__restrict__ entropy) {
  const int row = blockIdx.x * 8 + static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  grid_wait();
  if (row >= a.rows) return;
  const int mt = row / 256;
  const long long first = static_cast<long long>(mt) * a.tiles_n, last = first + a.tiles_n - 1;
  // the pairs whose shares hold tiles first .. last
  long long p0 = first * npairs / a.num_tiles, p1 = last * npairs / a.num_tiles;
  while (share_start(p0 + 1, a.num_tiles, npairs) <= first) ++p0;
  while (share_start(p0, a.num_tiles, npairs) > first) --p0;
  while (share_start(p1 + 1, a.num_tiles, npairs) <= last) ++p1;
  while (share_start(p1, a.num_tiles, npairs) > last) --p1;
  Stat2 st{kLowest, 0.f, 0.f};
  constexpr int G = kScoreGroups;
  const int parts = G * static_cast<int>(p1 - p0 + 1);
  for (int i = lane; i < parts; i += 32) {
    const float4 v = a.partial[((p0 + i / G + mt) * G + i % G) * 256 + (row & 255)];
    join2(st, Stat2{v.x, v.y, v.z});
  }
  rebase2(st, warp_max(st.m));
  int id = ids ? ids[row] : -1;
  if (id >= a.N) {
    if (lane == 0) record_status(a.status, AVEY_ERR_DEVICE_BOUNDS);
    id = -1;
  }
  int acc = 0;
  if (id >= 0) {
    const int8_t *x = xq + row * ld_xq, *w = Wq + id * ld_w;
    const int whole = a.K / 4;
    for (int i = lane; i < whole; i += 32)
      acc = __dp4a(reinterpret_cast<const int *>(x)[i], reinterpret_cast<const int *>(w)[i], acc);
    const int k = whole * 4 + lane;
    if (k < a.K) acc += static_cast<int>(x[k]) * static_cast<int>(w[k]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    st.s += __shfl_xor_sync(0xffffffffu, st.s, off);
    st.t += __shfl_xor_sync(0xffffffffu, st.t, off);
    acc += __shfl_xor_sync(0xffffffffu, acc, off);
  }
  if (lane != 0) return;
  float y = 0.f;
  if (id >= 0)
    y = fmaf(static_cast<float>(acc) * (a.x_scale[row] * kLog2e), a.w_scale[id],
             a.bias ? a.bias[id] * kLog2e : 0.f);
  write_scores(st, row, id >= 0, y, logprob, stats, entropy);
}

inline int64_t score_ld(int N) { return (static_cast<int64_t>(N) + 7) / 8 * 8; }
inline size_t score_partial_bytes(int rows) {
  const size_t slots = static_cast<size_t>((rows + 255) / 256) + std::max(1, sm_count() / 2);
  return slots * kScoreGroups * 256 * sizeof(float4);
}

avey_status launch_score_i8(const avey_linear_i8_params *p, const int8_t *xq, int64_t ld_xq,
                            const float *x_scale, int rows, const int32_t *ids, float *logprob,
                            float *stats, float *entropy, float4 *partial, bool after, cudaStream_t s) {
  LinArgs a{};
  a.rows = rows;
  a.N = p->N;
  a.K = p->K;
  a.x_scale = x_scale;
  a.w_scale = p->w_scale;
  a.bias = p->bias;
  a.partial = partial;
  a.status = device_status_word();
  a.tiles_m = (rows + 255) / 256;
  a.tiles_n = (p->N + 255) / 256;
  a.num_tiles = static_cast<long long>(a.tiles_m) * a.tiles_n;
  const int pairs = pairs_for(a.num_tiles);
  CUtensorMap ma, mb;
  if (!encode_i8_map(&ma, xq, a.K, rows, ld_xq, 128)) return AVEY_ERR_CUDA;
  if (!encode_i8_map(&mb, p->Wq, a.K, a.N, p->ld_w, 128)) return AVEY_ERR_CUDA;
  const avey_status st = a.K <= kBK * kResidentSteps
                             ? run_linear_pair<256, kScore, false, true>(ma, mb, ma, ma, ma, a, pairs, after, s)
                             : run_linear_pair<256, kScore, false, false>(ma, mb, ma, ma, ma, a, pairs, after, s);
  if (st != AVEY_OK) return st;
  const cudaError_t e = launch_after(score_join, (rows + 7) / 8, 256, 0, s, a, pairs, xq, ld_xq, p->Wq, p->ld_w,
                                     ids, logprob, stats, entropy);
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_detail("score_join launch failed: %s", cudaGetErrorString(e));
    return AVEY_ERR_CUDA;
  }
  AVEY_CHECK_LAUNCH("score_join", s);
  return AVEY_OK;
}

}  // namespace
}  // namespace avey

// Scores take the few-row kernel where it fits (linear_few_fits).  Else up to 16 rows
// send their logits through the workspace, and up to this many where channels become
// the rows of a tile (swap_pays; 32 x 768 -> 50368: 19.3 us so, 21.2 with the
// statistics in the product; 17 x 256: 14.5 and 18.3).  All others keep the statistics
// in the product.
static constexpr int kLogitRows = 32;

extern "C" size_t avey_score_tokens_i8_workspace_bytes(int rows, int K, int N) {
  if (rows <= 0 || K <= 0 || N <= 0) return 0;
  return quantized_bytes(rows, K) +
         std::max(align256(static_cast<size_t>(std::min(rows, kLogitRows)) * score_ld(N) * 4),
                  std::max(score_partial_bytes(rows), score_few_bytes(std::min(rows, kFewRows), N)));
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
  char *rest = static_cast<char *>(ws) + quantized_bytes(rows, p->K);
  if (linear_few_fits(rows, p->K))
    return launch_score_few(p, x, x_dt, ld_x, x_scale, prenorm ? 1 : 0, rows, ids, logprob, stats, entropy, rest, s);
  float *logits = reinterpret_cast<float *>(rest);
  const int64_t ld = score_ld(p->N);
  const int8_t *xq = static_cast<const int8_t *>(x);
  const float *xs = x_scale;
  int64_t ld_xq = ld_x;
  if (x_dt != AVEY_I8) {
    st = quantize_to_ws(p, x, x_dt, ld_x, prenorm, rows, ws, &xq, &ld_xq, &xs, s);
    if (st != AVEY_OK) return st;
  }
  if (rows > (swap_pays(rows, p->N) ? kLogitRows : kFewRows))
    return launch_score_i8(p, xq, ld_xq, xs, rows, ids, logprob, stats, entropy,
                           reinterpret_cast<float4 *>(rest), x_dt != AVEY_I8, s);
  st = launch_linear_i8(p, xq, ld_xq, xs, rows, nullptr, 0, logits, AVEY_F32, ld, x_dt != AVEY_I8, s);
  if (st != AVEY_OK) return st;
  return launch_token_logprobs(logits, AVEY_F32, rows, p->N, ld, ids, 0, logprob, stats, entropy, nullptr,
                               nullptr, s);
}
