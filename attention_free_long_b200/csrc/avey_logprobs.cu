// avey_logprobs.cu -- scoring of logits rows and its gradient.
//
//   m = max_j x_j, z = log sum_j exp(x_j - m), logprob = x_id - m - z,
//   entropy = z - sum_j e_j (x_j - m) / sum_j e_j,  e_j = exp(x_j - m),
//   the `top` largest by (value desc, index asc).
//
// Forward: one pass over the row with a running maximum; each thread carries
// (m, s, t) = (max, sum e, sum e (x - m)) and rescales s and t once a batch
// when its maximum grows.  A row belongs to one block, or to a cluster of up to eight blocks when there are
// few rows, whose partial results meet in distributed shared memory.
// Alternatives: the `top`-th largest of the threads' maxima is a bar that `top`
// elements reach, so every alternative reaches it and lies with a thread whose
// maximum does: about `top` of them.  A thread knows which batch its maximum
// came from and the largest maximum of its other batches; mostly that one is
// below the bar, and eight vectors of the thread are read a second time, four
// threads' at once.  What reaches the bar goes through sorted lists, one a warp.
// Backward: dx_j = g (1[j = id] - p_j) - h p_j (log p_j + entropy), one read and
// one write of the row.
#include <algorithm>
#include <cmath>

#include "avey_common.cuh"
#include "avey_internal.h"

namespace avey {
namespace {

constexpr int kLpThreads = 256;       // threads of the gradient's blocks
constexpr int kBatch = 8;             // 16-byte vectors a thread takes at once
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;
// exp(d) is 0 in fp32 from here down; keeps 0 * (x - m) finite
constexpr float kFar = -200.0f;
// down to here x - m is finite for every m
constexpr float kLow = -1e30f;

__device__ __forceinline__ float fast_exp(float d) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d * kLog2e));
  return r;
}

// Unsigned integers in the order of the floats; -0 counts as +0.
__device__ __forceinline__ uint32_t ord_of(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float ord_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
// (value desc, index asc) as one descending key; 0 is "none".
__device__ __forceinline__ uint64_t key_of(float f, uint32_t index) {
  return (static_cast<uint64_t>(ord_of(f)) << 32) | (~index);
}

__device__ __forceinline__ float min3f(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &w, float *v) {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float *v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ float max(const uint4 &w) {
    return fmaxf(max3f(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z)), __uint_as_float(w.w));
  }
  static __device__ __forceinline__ float max_all(const uint4 *w) {
    float m = max(w[0]);
#pragma unroll
    for (int i = 1; i < kBatch; ++i) m = fmaxf(m, max(w[i]));
    return m;
  }
  static __device__ __forceinline__ float min_all(const uint4 *w) {
    float m = INFINITY;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      m = min3f(min3f(m, __uint_as_float(w[i].x), __uint_as_float(w[i].y)), __uint_as_float(w[i].z),
                __uint_as_float(w[i].w));
    return m;
  }
  static __device__ __forceinline__ void set(uint32_t *w, int i, float x) { w[i] = __float_as_uint(x); }
  static __device__ __forceinline__ float to_f(float x) { return x; }
  static __device__ __forceinline__ float from_f(float x) { return x; }
};
template <>
struct Vec<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &w, float *v) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float *v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                      pack_bf16(v[6], v[7]));
  }
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ __nv_bfloat162 b2(uint32_t w) {
    return *reinterpret_cast<const __nv_bfloat162 *>(&w);
  }
  static __device__ __forceinline__ float max(const uint4 &w) {
    const __nv_bfloat162 m = __hmax2(__hmax2(b2(w.x), b2(w.y)), __hmax2(b2(w.z), b2(w.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ float max_all(const uint4 *w) {
    __nv_bfloat162 m = b2(w[0].x);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      m = __hmax2(__hmax2(__hmax2(m, b2(w[i].x)), b2(w[i].y)), __hmax2(b2(w[i].z), b2(w[i].w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ float min_all(const uint4 *w) {
    __nv_bfloat162 m = b2(w[0].x);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      m = __hmin2(__hmin2(__hmin2(m, b2(w[i].x)), b2(w[i].y)), __hmin2(b2(w[i].z), b2(w[i].w)));
    return fminf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ void set(uint32_t *w, int i, bf16 x) {
    const uint32_t b = __bfloat16_as_ushort(x);
    w[i / 2] = (i & 1) ? (w[i / 2] & 0x0000ffffu) | (b << 16) : (w[i / 2] & 0xffff0000u) | b;
  }
  static __device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ bf16 from_f(float x) { return __float2bfloat16_rn(x); }
};

// A row as 16-byte vectors of aligned addresses: vector u holds elements
// u * N - shift .. , of which those outside [0, V) do not exist.
template <typename T>
struct Row {
  static constexpr int N = Vec<T>::N;
  const T *p;
  int V, shift, vecs;
  __device__ __forceinline__ Row(const T *base, int V_) : p(base), V(V_) {
    shift = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(T));
    vecs = static_cast<int>((static_cast<long long>(V) + shift + N - 1) / N);
  }
  __device__ __forceinline__ int first(int u) const { return u * N - shift; }
  __device__ __forceinline__ bool whole(int u) const {
    const int e = first(u);
    return e >= 0 && e <= V - N;
  }
  // Elements that do not exist are -inf.  Plain loads, as the gradient may
  // overwrite the row it reads.
  __device__ __forceinline__ uint4 load(int u) const {
    const int e = first(u);
    if (whole(u)) return *reinterpret_cast<const uint4 *>(p + e);
    uint32_t w[4] = {Vec<T>::kNegInf, Vec<T>::kNegInf, Vec<T>::kNegInf, Vec<T>::kNegInf};
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e + i >= 0 && e + i < V) Vec<T>::set(w, i, p[e + i]);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

struct Stat {
  float m, s, t;  // maximum (kLowest for none), sum e, sum e (x - m)
};
// s and t relative to M >= m
__device__ __forceinline__ void rebase(Stat &a, float M) {
  const float d = fmaxf(a.m - M, kFar), f = fast_exp(a.m - M);
  a.t = f * fmaf(a.s, d, a.t);
  a.s *= f;
  a.m = M;
}

// One vector's terms into two running pairs of sums.  CLAMP: some elements are
// so low that x - m may be infinite.
template <typename T, bool CLAMP>
__device__ __forceinline__ void add_terms(const uint4 &w, float m, float2 &s, float2 &t) {
  constexpr int N = Vec<T>::N;
  float v[N];
  Vec<T>::unpack(w, v);
  const float2 minus = make_float2(-m, -m), l2 = make_float2(kLog2e, kLog2e);
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    float2 d = fadd2(make_float2(v[j], v[j + 1]), minus);
    const float2 y = fmul2(d, l2);
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
    if (CLAMP) d = make_float2(fmaxf(d.x, kFar), fmaxf(d.y, kFar));
    s = fadd2(s, e);
    t = ffma2(e, d, t);
  }
}

// With TOP: a thread's largest value, the first vector of the batch it came from,
// and the largest value of the other batches.
struct Best {
  float first = -INFINITY, second = -INFINITY;
  int batch = 0;
};

// A batch of vectors u, u + stride, .. into a thread's statistics; s and t are
// the running sums.
template <typename T, bool TOP>
__device__ __forceinline__ void add_batch(const uint4 (&w)[kBatch], int u, Stat &st, float2 &s, float2 &t, Best &best) {
  const float top = Vec<T>::max_all(w);
  if constexpr (TOP) {
    best.second = fmaxf(best.second, fminf(best.first, top));
    best.batch = top > best.first ? u : best.batch;
    best.first = fmaxf(best.first, top);
  }
  if (top > st.m) {
    st.s = s.x + s.y;
    st.t = t.x + t.y;
    rebase(st, top);
    s = make_float2(st.s, 0.f);
    t = make_float2(st.t, 0.f);
  }
  if (Vec<T>::min_all(w) >= kLow) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) add_terms<T, false>(w[i], st.m, s, t);
  } else {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) add_terms<T, true>(w[i], st.m, s, t);
  }
}


// Descending sort of one value per lane.
__device__ __forceinline__ uint32_t warp_sort(uint32_t v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
      v = ((lane & j) == 0) == ((lane & k) == 0) ? max(v, o) : min(v, o);
    }
  }
  return v;
}

// The L largest of two descending lists of L lanes each, descending; o is the
// second list reversed.
template <int L, typename K>
__device__ __forceinline__ K merge_reversed(K v, K o, int lane) {
  v = max(v, o);
#pragma unroll
  for (int j = L / 2; j > 0; j >>= 1) {
    o = __shfl_xor_sync(0xffffffffu, v, j);
    v = (lane & j) == 0 ? max(v, o) : min(v, o);
  }
  return v;
}
// The L largest of W descending lists (list i at lists + 32 i), in every group
// of L lanes.  A warp takes them side by side, 32 / L lists to a register.
template <int L, int W, typename K>
__device__ __forceinline__ K merge_lists(const K *lists, int lane) {
  constexpr int R = L * W / 32;
  K r[R];
#pragma unroll
  for (int i = 0; i < R; ++i) r[i] = lists[(i * (32 / L) + lane / L) * 32 + (lane & (L - 1))];
#pragma unroll
  for (int n = R / 2; n > 0; n >>= 1) {
#pragma unroll
    for (int i = 0; i < n; ++i)
      r[i] = merge_reversed<L>(r[i], __shfl_xor_sync(0xffffffffu, r[i + n], L - 1), lane);
  }
#pragma unroll
  for (int g = L; g < 32; g <<= 1) r[0] = merge_reversed<L>(r[0], __shfl_xor_sync(0xffffffffu, r[0], 2 * g - 1), lane);
  return r[0];
}
template <int W, typename K>
__device__ __forceinline__ K merge_top(const K *lists, int top, int lane) {
  if (top <= 8) return merge_lists<8, W>(lists, lane);
  if (top <= 16) return merge_lists<16, W>(lists, lane);
  return merge_lists<32, W>(lists, lane);
}

struct LpArgs {
  const void *x;
  long long ld;
  int rows, V, blocks;  // blocks of a row (the cluster size)
  const int32_t *ids;
  int top;
  float *logprob, *stats, *entropy;
  int32_t *top_ids;
  float *top_lp;
  int *status;
};

// Statistics of the share of a row that W warps hold, given to all threads.
template <int W>
__device__ __forceinline__ Stat row_stats(Stat st, float (*sm)[W], int warp, int lane) {
  rebase(st, warp_max(st.m));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    st.s += __shfl_xor_sync(0xffffffffu, st.s, off);
    st.t += __shfl_xor_sync(0xffffffffu, st.t, off);
  }
  if constexpr (W == 1) return st;
  if (lane == 0) {
    sm[0][warp] = st.m;
    sm[1][warp] = st.s;
    sm[2][warp] = st.t;
  }
  __syncthreads();
  float M = sm[0][0];
#pragma unroll
  for (int i = 1; i < W; ++i) M = fmaxf(M, sm[0][i]);
  Stat all{M, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < W; ++i) {
    Stat o{sm[0][i], sm[1][i], sm[2][i]};
    rebase(o, M);
    all.s += o.s;
    all.t += o.t;
  }
  return all;
}

// What the statistics of a whole row say.
struct RowResult {
  float m, z, entropy;
  bool empty, bad;
  __device__ __forceinline__ explicit RowResult(const Stat &all) {
    const float nan = __uint_as_float(0x7fc00000u);
    empty = all.s == 0.f;
    // a finite row has 1 <= s <= V; +inf or NaN leave an infinite maximum or a NaN sum
    bad = !(all.s < INFINITY) || all.m == INFINITY;
    m = bad ? nan : empty ? -INFINITY : all.m;
    z = bad ? nan : empty ? 0.f : logf(all.s);
    entropy = bad ? nan : empty ? 0.f : z - all.t / all.s;
  }
  // log probability of a word with logit x
  __device__ __forceinline__ float logprob(float x) const { return empty ? -INFINITY : (x - m) - z; }
};

__device__ __forceinline__ void write_row(const LpArgs &a, long long row, const RowResult &res, int id, float x_id) {
  if (a.logprob) a.logprob[row] = id < 0 ? 0.f : res.logprob(x_id);
  if (a.stats) reinterpret_cast<float2 *>(a.stats)[row] = make_float2(res.m, res.z);
  if (a.entropy) a.entropy[row] = res.entropy;
}
__device__ __forceinline__ void write_top(const LpArgs &a, long long row, const RowResult &res, uint64_t key, int lane) {
  const bool has = !res.bad && key != 0;
  a.top_ids[row * a.top + lane] = has ? static_cast<int32_t>(~static_cast<uint32_t>(key)) : -1;
  a.top_lp[row * a.top + lane] =
      res.bad ? res.m : has ? res.logprob(ord_value(static_cast<uint32_t>(key >> 32))) : -INFINITY;
}

// The logit of a row's given token; an id past the vocabulary becomes none.
template <typename T>
__device__ __forceinline__ float given_logit(const LpArgs &a, const Row<T> &r, int &id) {
  if (id >= a.V) {
    record_status(a.status, AVEY_ERR_DEVICE_BOUNDS);
    id = -1;
  }
  return id >= 0 ? Vec<T>::to_f(r.p[id]) : 0.f;
}

// A vector's elements of at least `bar`, one vector per lane from element e0,
// into the warp's descending list of 32 keys over the lanes.
template <typename T>
__device__ __forceinline__ void insert_top(const uint4 &w, bool in, uint32_t e0, float bar, uint64_t &list, int lane) {
  constexpr int N = Vec<T>::N;
  uint32_t lanes = __ballot_sync(0xffffffffu, in && Vec<T>::max(w) >= bar);
  if (lanes == 0) return;
  float v[N];
  uint32_t want = 0;
  Vec<T>::unpack(w, v);
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (in && v[j] >= bar && v[j] > -INFINITY) want |= 1u << j;
  if (__popc(lanes) > 4) {
    // many equal values: only those that would still enter the list
    const uint64_t full = __shfl_sync(0xffffffffu, list, 31);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if ((want >> j & 1) && key_of(v[j], e0 + j) <= full) want &= ~(1u << j);
  }
  lanes = __ballot_sync(0xffffffffu, want != 0);
  while (lanes) {
    const int src = __ffs(lanes) - 1;
    uint64_t mine = 0;
    if (lane == src) {
      const int j = __ffs(want) - 1;
      float f = v[0];
#pragma unroll
      for (int q = 1; q < N; ++q) f = q == j ? v[q] : f;
      mine = key_of(f, e0 + j);
      want &= want - 1;
    }
    const uint64_t nk = __shfl_sync(0xffffffffu, mine, src);
    const int pos = __popc(__ballot_sync(0xffffffffu, list > nk));
    const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
    if (lane >= pos) list = lane == pos ? nk : up;
    lanes = __ballot_sync(0xffffffffu, want != 0);
  }
}

// The elements of at least `bar` of this warp's threads, as one descending list
// of 32 over the lanes.  first: the first vector of lane 0.
template <typename T>
__device__ __forceinline__ uint64_t select_top(const Row<T> &r, int first, int stride, const Best &best, float bar, int lane) {
  static_assert(kBatch == 8, "a batch of four threads to a warp");
  uint64_t list = 0;
  const bool mine = best.first >= bar && best.first > -INFINITY;
  uint32_t all = __ballot_sync(0xffffffffu, mine && best.second >= bar);
  uint32_t one = __ballot_sync(0xffffffffu, mine) & ~all;
  // threads of which one batch reaches the bar, four at a time
  while (one) {
    int owner = 32;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (lane >> 3 == i && one) owner = __ffs(one) - 1;
      one &= one - 1;
    }
    const int batch = __shfl_sync(0xffffffffu, best.batch, owner & 31);
    const long long u = batch + static_cast<long long>(lane & 7) * stride;
    const bool in = owner < 32 && u < r.vecs;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (in) w = r.load(static_cast<int>(u));
    insert_top<T>(w, in, static_cast<uint32_t>(r.first(static_cast<int>(u))), bar, list, lane);
  }
  // threads of which several do
  while (all) {
    const int owner = first + __ffs(all) - 1;
    all &= all - 1;
    for (long long u0 = owner; u0 < r.vecs; u0 += 32ll * stride) {
      const long long u = u0 + static_cast<long long>(lane) * stride;
      const bool in = u < r.vecs;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (in) w = r.load(static_cast<int>(u));
      insert_top<T>(w, in, static_cast<uint32_t>(r.first(static_cast<int>(u))), bar, list, lane);
    }
  }
  return list;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t a) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// W warps to a row: one (four rows a block), or all of a block's; or, with
// CLUSTER, a cluster of a.blocks blocks, block `rank` taking the vectors u with
// u / (32 W) % blocks == rank.
template <typename T, bool TOP, int W, bool CLUSTER>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W, W == 1 ? 8 : 32 / W) token_logprobs(const LpArgs a) {
  constexpr int N = Vec<T>::N;
  static_assert(!CLUSTER || W == 8, "clusters are made of blocks of eight warps");
  __shared__ float sm[3][W];
  __shared__ float s_out[3];
  __shared__ uint64_t lists[TOP && W > 1 ? W : 1][32];
  __shared__ uint32_t maxima[TOP && W > 1 ? W : 1][32];
  __shared__ uint32_t s_best[TOP ? 32 : 1];
  __shared__ uint64_t s_top[TOP && CLUSTER ? 32 : 1];
  const int warp = W == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = CLUSTER ? a.blocks : 1, rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
  const long long row = W == 1 ? blockIdx.x * 4ll + (threadIdx.x >> 5) : blockIdx.x / C;
  if (W == 1 && row >= a.rows) return;
  const int stride = C * 32 * W;
  const Row<T> r(static_cast<const T *>(a.x) + row * a.ld, a.V);
  const bool writer = rank == 0 && warp == 0 && lane == 0;
  int id = writer && a.ids ? a.ids[row] : -1;

  Stat st{kLowest, 0.f, 0.f};
  Best best;
  {
    float2 s2 = make_float2(0.f, 0.f), t2 = s2;
    const int whole_end = static_cast<int>((static_cast<long long>(a.V) + r.shift) / N);
    int u = rank * 32 * W + warp * 32 + lane;
    if (r.shift == 0 || u > 0) {
      const uint4 *src = reinterpret_cast<const uint4 *>(r.p - r.shift);  // vector 0, of which 0 .. shift - 1 is not ours
      for (; u + (kBatch - 1) * stride < whole_end; u += kBatch * stride) {
        uint4 w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) w[i] = __ldg(src + u + i * stride);
        add_batch<T, TOP>(w, u, st, s2, t2, best);
      }
    }
    for (; u < r.vecs; u += kBatch * stride) {
      uint4 w[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        w[i] = make_uint4(Vec<T>::kNegInf, Vec<T>::kNegInf, Vec<T>::kNegInf, Vec<T>::kNegInf);
        if (u + i * stride < r.vecs) w[i] = r.load(u + i * stride);
      }
      add_batch<T, TOP>(w, u, st, s2, t2, best);
    }
    st.s = s2.x + s2.y;
    st.t = t2.x + t2.y;
  }
  const float x_id = writer ? given_logit(a, r, id) : 0.f;  // not needed before the sums are joined
  uint32_t sorted = 0;
  if constexpr (TOP) {
    sorted = warp_sort(ord_of(best.first), lane);
    if (W > 1) maxima[warp][lane] = sorted;
  }
  Stat all = row_stats<W>(st, sm, warp, lane);
  float bar = -INFINITY;
  if constexpr (TOP && W > 1) {
    if (warp == 0) s_best[lane] = merge_top<W>(&maxima[0][0], a.top, lane);
  }
  if constexpr (CLUSTER) {
    if (threadIdx.x == 0) {
      s_out[0] = all.m;
      s_out[1] = all.s;
      s_out[2] = all.t;
    }
    __syncwarp();
    cluster_sync_all();
    const uint32_t addr = smem_u32(s_out);
    Stat part[8];
    float CM = kLowest;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      part[c] = Stat{kLowest, 0.f, 0.f};
      if (c < C) {
        const uint32_t at = mapa_shared(addr, c);
        part[c] = Stat{ld_cluster_f32(at), ld_cluster_f32(at + 4), ld_cluster_f32(at + 8)};
      }
      CM = fmaxf(CM, part[c].m);
    }
    all = Stat{CM, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      rebase(part[c], CM);
      all.s += part[c].s;
      all.t += part[c].t;
    }
    if constexpr (TOP) {
      // the lists of all blocks, in the place of the warps' lists
      if (warp < C) maxima[warp][lane] = ld_cluster_u32(mapa_shared(smem_u32(&s_best[lane]), warp));
      if (warp >= C) maxima[warp][lane] = 0;
      __syncthreads();
      bar = ord_value(__shfl_sync(0xffffffffu, merge_top<W>(&maxima[0][0], a.top, lane), a.top - 1));
    }
  } else if constexpr (TOP && W > 1) {
    __syncthreads();
    bar = ord_value(s_best[a.top - 1]);
  } else if constexpr (TOP) {
    bar = ord_value(__shfl_sync(0xffffffffu, sorted, a.top - 1));
  }
  const RowResult res(all);
  if (writer) write_row(a, row, res, id, x_id);
  if constexpr (TOP) {
    uint64_t key = select_top(r, rank * 32 * W + warp * 32, stride, best, bar, lane);
    if constexpr (W > 1) {
      lists[warp][lane] = key;
      __syncthreads();
      if (warp == 0) key = merge_top<W>(&lists[0][0], a.top, lane);
    }
    if constexpr (CLUSTER) {
      if (warp == 0) s_top[lane] = key;
      __syncwarp();
      cluster_sync_all();
      if (rank == 0) {
        if (warp < C)
          lists[warp][lane] = ld_cluster_u64(mapa_shared(smem_u32(&s_top[lane]), warp));
        else
          lists[warp][lane] = 0;
        __syncthreads();
        if (warp == 0) key = merge_top<W>(&lists[0][0], a.top, lane);
      }
    }
    if (rank == 0 && warp == 0 && lane < a.top) write_top(a, row, res, key, lane);
  }
  if constexpr (CLUSTER) {
    __syncwarp();
    cluster_sync_all();  // no block leaves while its memory is read
  }
}

template <typename T, bool TOP>
avey_status run_logprobs(LpArgs a, int rows, cudaStream_t s) {
  const int sms = sm_count();
  const long long vecs = (a.V + Vec<T>::N - 1) / Vec<T>::N;
  a.rows = rows;
  a.blocks = 1;
  // Few rows: several blocks a row, as long as a thread has four vectors and the
  // blocks find room at once (1 x 50368 fp32: 9.8 us with one, 6.8 with eight;
  // 300 rows: 14.8 with one, 20.6 with two).  Many rows: fewer warps to a row,
  // whose ends cost less (6554 x 50368 bf16: 115 us with eight, 107 with four;
  // 2000 x 2000: 10.4 with eight, 5.9 with four, 4.8 with one), unless a long
  // row would be left to one warp at the end.
  while (a.blocks < 8 && static_cast<long long>(rows) * a.blocks * 2 <= 2ll * sms && vecs >= 1024ll * a.blocks)
    a.blocks *= 2;
  const int C = a.blocks;
  const int W = rows >= 8 * sms && vecs <= 1024 ? 1 : rows > 4 * sms || vecs <= 256 ? 4 : 8;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  cfg.attrs = at;
  if (C > 1) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
  }
  cfg.gridDim = dim3(W == 1 && C == 1 ? (static_cast<unsigned>(rows) + 3) / 4 : static_cast<unsigned>(rows) * C);
  cfg.blockDim = dim3(C > 1 || W == 8 ? 256 : 128);
  const cudaError_t e = C > 1    ? cudaLaunchKernelEx(&cfg, token_logprobs<T, TOP, 8, true>, static_cast<const LpArgs>(a))
                        : W == 1 ? cudaLaunchKernelEx(&cfg, token_logprobs<T, TOP, 1, false>, static_cast<const LpArgs>(a))
                        : W == 4 ? cudaLaunchKernelEx(&cfg, token_logprobs<T, TOP, 4, false>, static_cast<const LpArgs>(a))
                                 : cudaLaunchKernelEx(&cfg, token_logprobs<T, TOP, 8, false>, static_cast<const LpArgs>(a));
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_detail("token_logprobs launch failed: %s", cudaGetErrorString(e));
    return AVEY_ERR_CUDA;
  }
  AVEY_CHECK_LAUNCH("token_logprobs", s);
  return AVEY_OK;
}

// ---- backward ---------------------------------------------------------------

struct LpGradArgs {
  const void *x;
  long long ld;
  int V, parts;  // blocks of a row
  const int32_t *ids;
  const float *stats, *entropy, *d_logprob, *d_entropy;
  void *dx;
  long long ld_d;
  int *status;
};

constexpr int kGradBatch = 4;  // vectors a thread loads at once
constexpr int kGradVecs = 8;   // and takes at most

template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_grad(const LpGradArgs a) {
  constexpr int N = Vec<T>::N;
  const long long row = blockIdx.x / a.parts;
  const int part = static_cast<int>(blockIdx.x - row * a.parts);
  const Row<T> r(static_cast<const T *>(a.x) + row * a.ld, a.V);
  T *out = static_cast<T *>(a.dx) + row * a.ld_d;
  // whole vectors of x are whole 16-byte words of the gradient too
  const bool same = ((reinterpret_cast<uintptr_t>(r.p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  int id = a.d_logprob ? a.ids[row] : -1;
  if (id >= a.V) {
    if (part == 0 && threadIdx.x == 0) record_status(a.status, AVEY_ERR_DEVICE_BOUNDS);
    id = -1;
  }
  const float g = id >= 0 ? a.d_logprob[row] : 0.f;
  const float h = a.d_entropy ? a.d_entropy[row] : 0.f;
  const float2 st = reinterpret_cast<const float2 *>(a.stats)[row];
  const float H = a.d_entropy ? a.entropy[row] : 0.f;
  const bool none = (g == 0.f && h == 0.f) || st.x == -INFINITY;
  const float2 m2 = make_float2(-st.x, -st.x), z2 = make_float2(-st.y, -st.y);
  const float2 h2 = make_float2(-h, -h), c2 = make_float2(-fmaf(h, H, g), -fmaf(h, H, g));
  const float2 l2 = make_float2(kLog2e, kLog2e);
  // The gradient of the words of one vector; element `hot` of it is the given one.
  auto gradient = [&](const uint4 &w, float (&v)[N], int hot) {
    Vec<T>::unpack(w, v);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      // log p, kept finite (NaN too stays) so that 0 * log p is 0
      float2 lp = fadd2(fadd2(make_float2(v[j], v[j + 1]), m2), z2);
      lp = make_float2(max_nan(lp.x, kFar), max_nan(lp.y, kFar));
      const float2 y = fmul2(lp, l2);
      float2 p;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(y.x));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(y.y));
      const float2 d = fmul2(p, ffma2(h2, lp, c2));
      v[j] = d.x;
      v[j + 1] = d.y;
    }
    if (static_cast<unsigned>(hot) < static_cast<unsigned>(N)) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (j == hot) v[j] += g;
    }
  };
  const int per = (r.vecs + a.parts - 1) / a.parts;
  const int begin = part * per, end = min(r.vecs, begin + per);
  const int hi = static_cast<int>((static_cast<long long>(a.V) + r.shift) / N);
  int u = begin + static_cast<int>(threadIdx.x);
  const int fast_end = same && !none ? min(end, hi) : 0;
  if (u > 0 || r.shift == 0) {
    const uint4 *src = reinterpret_cast<const uint4 *>(r.p - r.shift);
    uint4 *dst = reinterpret_cast<uint4 *>(out - r.shift);
    for (; u + (kGradBatch - 1) * kLpThreads < fast_end; u += kGradBatch * kLpThreads) {
      uint4 w[kGradBatch];
#pragma unroll
      for (int i = 0; i < kGradBatch; ++i) w[i] = src[u + i * kLpThreads];
#pragma unroll
      for (int i = 0; i < kGradBatch; ++i) {
        float v[N];
        gradient(w[i], v, id - r.first(u + i * kLpThreads));
        dst[u + i * kLpThreads] = Vec<T>::pack(v);
      }
    }
  }
  for (; u < end; u += kLpThreads) {
    const int e0 = r.first(u);
    float v[N];
    if (none) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = 0.f;
    } else {
      gradient(r.load(u), v, id >= 0 ? id - e0 : -1);
    }
    if (same && r.whole(u)) {
      *reinterpret_cast<uint4 *>(out + e0) = Vec<T>::pack(v);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (e0 + j >= 0 && e0 + j < a.V) out[e0 + j] = Vec<T>::from_f(v[j]);
    }
  }
}

template <typename T>
avey_status run_logprobs_grad(LpGradArgs a, int rows, cudaStream_t s) {
  const long long vecs = (static_cast<long long>(a.V) + 2 * Vec<T>::N - 2) / Vec<T>::N;
  long long parts = (vecs + kGradVecs * kLpThreads - 1) / (kGradVecs * kLpThreads);
  parts = std::max<long long>(1, std::min<long long>(parts, 0x7fffffffll / rows));
  a.parts = static_cast<int>(parts);
  token_logprobs_grad<T><<<static_cast<unsigned>(rows * parts), kLpThreads, 0, s>>>(a);
  AVEY_CHECK_LAUNCH("token_logprobs_grad", s);
  return AVEY_OK;
}

avey_status check_logits(const char *fn, avey_dtype dt, int rows, int V, int64_t ld, const void *x) {
  AVEY_REQUIRE(dt == AVEY_F32 || dt == AVEY_BF16, AVEY_ERR_UNSUPPORTED,
               "%s: dtype %d unsupported (F32 or BF16)", fn, int(dt));
  AVEY_REQUIRE(rows >= 0 && V >= 1, AVEY_ERR_INVALID_ARG, "%s: need rows >= 0 and V >= 1 (rows=%d V=%d)",
               fn, rows, V);
  AVEY_REQUIRE(ld >= V, AVEY_ERR_INVALID_ARG, "%s: leading dimension %lld < V=%d", fn,
               static_cast<long long>(ld), V);
  AVEY_REQUIRE(rows < (1 << 28) && V <= (1 << 30), AVEY_ERR_UNSUPPORTED,
               "%s: problem too large (rows=%d V=%d)", fn, rows, V);
  AVEY_REQUIRE((reinterpret_cast<uintptr_t>(x) & (dt == AVEY_F32 ? 3 : 1)) == 0, AVEY_ERR_INVALID_ARG,
               "%s: logits are not aligned to their element", fn);
  return AVEY_OK;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7) == 0; }

}  // namespace

avey_status launch_token_logprobs(const void *logits, avey_dtype dt, int rows, int V, int64_t ld,
                                  const int32_t *ids, int top, float *logprob, float *stats,
                                  float *entropy, int32_t *top_ids, float *top_lp, cudaStream_t s) {
  if (rows == 0) return AVEY_OK;
  LpArgs a{};
  a.x = logits;
  a.ld = ld;
  a.V = V;
  a.ids = ids;
  a.top = top;
  a.logprob = logprob;
  a.stats = stats;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_lp = top_lp;
  a.status = device_status_word();
  if (dt == AVEY_F32)
    return top > 0 ? run_logprobs<float, true>(a, rows, s) : run_logprobs<float, false>(a, rows, s);
  return top > 0 ? run_logprobs<bf16, true>(a, rows, s) : run_logprobs<bf16, false>(a, rows, s);
}

}  // namespace avey

using namespace avey;

extern "C" avey_status avey_token_logprobs(const void *logits, avey_dtype dt, int rows, int V,
                                           int64_t ld, const int32_t *ids, int top, float *logprob,
                                           float *stats, float *entropy, int32_t *top_ids,
                                           float *top_logprobs, avey_stream_t stream) {
  const avey_status st = check_logits("avey_token_logprobs", dt, rows, V, ld, logits);
  if (st != AVEY_OK) return st;
  AVEY_REQUIRE(top >= 0 && top <= 32, top < 0 ? AVEY_ERR_INVALID_ARG : AVEY_ERR_UNSUPPORTED,
               "avey_token_logprobs: top=%d outside [0, 32]", top);
  if (rows == 0) return AVEY_OK;
  AVEY_REQUIRE(logits, AVEY_ERR_INVALID_ARG, "avey_token_logprobs: null logits");
  AVEY_REQUIRE((ids != nullptr) == (logprob != nullptr), AVEY_ERR_INVALID_ARG,
               "avey_token_logprobs: ids and logprob go together");
  AVEY_REQUIRE((top > 0) == (top_ids != nullptr) && (top > 0) == (top_logprobs != nullptr),
               AVEY_ERR_INVALID_ARG, "avey_token_logprobs: top=%d and its outputs do not match", top);
  AVEY_REQUIRE(logprob || stats || entropy || top > 0, AVEY_ERR_INVALID_ARG,
               "avey_token_logprobs: no output");
  AVEY_REQUIRE(aligned4(ids) && aligned4(logprob) && aligned8(stats) && aligned4(entropy) &&
                   aligned4(top_ids) && aligned4(top_logprobs),
               AVEY_ERR_INVALID_ARG, "avey_token_logprobs: stats 8-byte, other rows 4-byte aligned");
  return launch_token_logprobs(logits, dt, rows, V, ld, ids, top, logprob, stats, entropy, top_ids,
                               top_logprobs, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" avey_status avey_token_logprobs_backward(const void *logits, avey_dtype dt, int rows, int V,
                                                    int64_t ld, const int32_t *ids, const float *stats,
                                                    const float *entropy, const float *d_logprob,
                                                    const float *d_entropy, void *dlogits,
                                                    int64_t ld_d, avey_stream_t stream) {
  const char *fn = "avey_token_logprobs_backward";
  const avey_status st = check_logits(fn, dt, rows, V, ld, logits);
  if (st != AVEY_OK) return st;
  AVEY_REQUIRE(ld_d >= V, AVEY_ERR_INVALID_ARG, "%s: leading dimension %lld < V=%d", fn,
               static_cast<long long>(ld_d), V);
  if (rows == 0) return AVEY_OK;
  AVEY_REQUIRE(logits && stats && dlogits, AVEY_ERR_INVALID_ARG, "%s: null pointer", fn);
  AVEY_REQUIRE(!d_logprob || ids, AVEY_ERR_INVALID_ARG, "%s: d_logprob needs ids", fn);
  AVEY_REQUIRE(!d_entropy || entropy, AVEY_ERR_INVALID_ARG, "%s: d_entropy needs entropy", fn);
  AVEY_REQUIRE((reinterpret_cast<uintptr_t>(dlogits) & (dt == AVEY_F32 ? 3 : 1)) == 0 && aligned4(ids) &&
                   aligned8(stats) && aligned4(entropy) && aligned4(d_logprob) && aligned4(d_entropy),
               AVEY_ERR_INVALID_ARG, "%s: dlogits aligned to its element, stats 8-byte, rows 4-byte", fn);
  {
    const uintptr_t es = dt == AVEY_F32 ? 4 : 2;
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(logits), d0 = reinterpret_cast<uintptr_t>(dlogits);
    const uintptr_t xn = x0 + (static_cast<uintptr_t>(rows - 1) * ld + V) * es;
    const uintptr_t dn = d0 + (static_cast<uintptr_t>(rows - 1) * ld_d + V) * es;
    AVEY_REQUIRE((x0 == d0 && ld == ld_d) || dn <= x0 || xn <= d0, AVEY_ERR_INVALID_ARG,
                 "%s: dlogits overlaps the logits without being them", fn);
  }
  LpGradArgs a{};
  a.x = logits;
  a.ld = ld;
  a.V = V;
  a.ids = ids;
  a.stats = stats;
  a.entropy = entropy;
  a.d_logprob = d_logprob;
  a.d_entropy = d_entropy;
  a.dx = dlogits;
  a.ld_d = ld_d;
  a.status = device_status_word();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == AVEY_F32 ? run_logprobs_grad<float>(a, rows, s) : run_logprobs_grad<bf16>(a, rows, s);
}
