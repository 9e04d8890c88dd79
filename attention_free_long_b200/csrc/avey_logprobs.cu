// avey_logprobs.cu -- scoring of logits rows and its gradient.
//
//   m = max_j x_j, z = log sum_j exp(x_j - m), logprob = x_id - m - z,
//   entropy = z - sum_j e_j (x_j - m) / sum_j e_j,  e_j = exp(x_j - m),
//   the `top` largest by (value desc, index asc).
//
// Forward: one pass over the row with a running maximum; each thread carries
// (m, s, t) = (max, sum e, sum e (x - m)) and rescales s and t once a batch
// when its maximum grows.  A row belongs to one warp, to one block, or, when there
// are few rows, to a cluster of up to eight blocks, whose partial results meet in
// distributed shared memory.
// Alternatives: the `top`-th largest of the threads' maxima is a bar that `top`
// elements reach, so every alternative reaches it and lies with a thread whose
// maximum does: about `top` of them.  A thread knows which batch its maximum
// came from and the largest maximum of its other batches; mostly that one is
// below the bar, and eight vectors of the thread are read a second time, four
// threads' at once.  What reaches the bar waits in a queue, one a warp, whose 32
// oldest entries are sorted and merged into the warp's list together; the list's
// `top`-th then raises the bar.
// Backward: dx_j = g (1[j = id] - p_j) - h p_j (log p_j + entropy), one read and
// one write of the row.
#include <algorithm>
#include <cmath>

#include "avey_common.cuh"
#include "avey_internal.h"

namespace avey {
namespace {

constexpr int kLpThreads = 256;       // threads of the gradient's blocks
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
  template <int B>
  static __device__ __forceinline__ float max_all(const uint4 (&w)[B]) {
    float m = max(w[0]);
#pragma unroll
    for (int i = 1; i < B; ++i) m = fmaxf(m, max(w[i]));
    return m;
  }
  template <int B>
  static __device__ __forceinline__ float min_all(const uint4 (&w)[B]) {
    float m = INFINITY;
#pragma unroll
    for (int i = 0; i < B; ++i)
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
  template <int B>
  static __device__ __forceinline__ float max_all(const uint4 (&w)[B]) {
    __nv_bfloat162 m = b2(w[0].x);
#pragma unroll
    for (int i = 0; i < B; ++i)
      m = __hmax2(__hmax2(__hmax2(m, b2(w[i].x)), b2(w[i].y)), __hmax2(b2(w[i].z), b2(w[i].w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  template <int B>
  static __device__ __forceinline__ float min_all(const uint4 (&w)[B]) {
    __nv_bfloat162 m = b2(w[0].x);
#pragma unroll
    for (int i = 0; i < B; ++i)
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
// the running sums.  PART: n of them, the others are -inf.
template <typename T, bool TOP, bool PART, int B>
__device__ __forceinline__ void add_batch(const uint4 (&w)[B], int u, int n, Stat &st, float2 &s, float2 &t,
                                          Best &best) {
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
  if constexpr (PART) {
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (i < n) add_terms<T, true>(w[i], st.m, s, t);
  } else if (Vec<T>::min_all(w) >= kLow) {
#pragma unroll
    for (int i = 0; i < B; ++i) add_terms<T, false>(w[i], st.m, s, t);
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) add_terms<T, true>(w[i], st.m, s, t);
  }
}

// Descending sort of the first n lanes' values; the other lanes hold 0.
template <typename K>
__device__ __forceinline__ K warp_sort(K v, int n, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
    if (k > 2 && n <= k / 2) break;
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const K o = __shfl_xor_sync(0xffffffffu, v, j);
      v = ((lane & j) == 0) == ((lane & k) == 0) ? max(v, o) : min(v, o);
    }
  }
  return v;
}
// The `top` largest of the lanes' values, descending over the lanes (then any).
__device__ __forceinline__ uint32_t warp_largest(uint32_t v, int top, int lane) {
  if (top > 4) return warp_sort(v, 32, lane);
  uint32_t r = 0;
  for (int i = 0; i < top; ++i) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, v);
    if (lane == i) r = m;
    if (lane == __ffs(__ballot_sync(0xffffffffu, v == m)) - 1) v = 0;
  }
  return r;
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

// A warp's candidates: the largest 32 sorted so far, and those still in line.
struct Select {
  uint64_t *queue;  // 64 keys of this warp
  uint64_t list;    // lane i: the i-th largest, 0 for none
  float bar;        // at least `top` elements of the row reach it
  int top, lane, waiting;
  bool none;  // the list is empty

  // The first 32 of the queue into the list.
  __device__ __forceinline__ void merge(int count) {
    __syncwarp();
    const uint64_t key = warp_sort(lane < count ? queue[lane] : 0ull, count, lane);
    // zeros behind it: reversed they meet the end of the list
    list = none ? key : merge_reversed<32>(list, __shfl_xor_sync(0xffffffffu, key, 31), lane);
    none = false;
  }
  // The elements of at least `bar` of one vector per lane, whose first element is e0.
  template <typename T>
  __device__ __forceinline__ void add(const uint4 &w, bool in, uint32_t e0) {
    constexpr int N = Vec<T>::N;
    if (!__any_sync(0xffffffffu, in && Vec<T>::max(w) >= bar)) return;
    float v[N];
    uint32_t want = 0;
    Vec<T>::unpack(w, v);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (in && v[j] >= bar && v[j] > -INFINITY) want |= 1u << j;
    uint32_t lanes = __ballot_sync(0xffffffffu, want != 0);
    while (lanes) {
      if (want) {
        const int j = __ffs(want) - 1;
        float f = v[0];
#pragma unroll
        for (int q = 1; q < N; ++q) f = q == j ? v[q] : f;
        queue[waiting + __popc(lanes & ((1u << lane) - 1u))] = key_of(f, e0 + j);
        want &= want - 1;
      }
      waiting += __popc(lanes);
      if (waiting >= 32) {
        merge(32);
        __syncwarp();
        const uint64_t rest = queue[32 + lane];
        __syncwarp();
        waiting -= 32;
        if (lane < waiting) queue[lane] = rest;
        // of equal values only those that still enter the list
        const uint64_t last = __shfl_sync(0xffffffffu, list, top - 1);
        if (last != 0) {
          bar = ord_value(static_cast<uint32_t>(last >> 32));
#pragma unroll
          for (int j = 0; j < N; ++j)
            if ((want >> j & 1) && key_of(v[j], e0 + j) < last) want &= ~(1u << j);
        }
      }
      lanes = __ballot_sync(0xffffffffu, want != 0);
    }
  }
  __device__ __forceinline__ uint64_t finish() {
    if (waiting) merge(waiting);
    return list;
  }
};

// The elements of at least `bar` of this warp's threads, as one descending list
// of 32 over the lanes, the first `top` of which are right.  first: the first
// vector of lane 0.
template <typename T, int B>
__device__ __forceinline__ uint64_t select_top(const Row<T> &r, int first, int stride, const Best &best, float bar,
                                               int top, uint64_t *queue, int lane) {
  constexpr int OWNERS = 32 / B;
  Select sel{queue, 0, bar, top, lane, 0, true};
  const bool mine = best.first >= bar && best.first > -INFINITY;
  uint32_t all = __ballot_sync(0xffffffffu, mine && best.second >= bar);
  uint32_t one = __ballot_sync(0xffffffffu, mine) & ~all;
  // threads of which one batch reaches the bar: each its own, where that takes
  // fewer steps (short rows), else OWNERS of them at a time
  const int steps = min(B, (r.vecs + stride - 1) / stride);
  if (steps * OWNERS < __popc(one) + OWNERS) {
    const bool in1 = one >> lane & 1u;
    one = 0;
    for (int i = 0; i < steps; ++i) {
      const long long u = best.batch + static_cast<long long>(i) * stride;
      const bool in = in1 && u < r.vecs;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (in) w = r.load(static_cast<int>(u));
      sel.add<T>(w, in, static_cast<uint32_t>(r.first(static_cast<int>(u))));
    }
  }
  while (one) {
    int owner = 32;
#pragma unroll
    for (int i = 0; i < OWNERS; ++i) {
      if (lane / B == i && one) owner = __ffs(one) - 1;
      one &= one - 1;
    }
    const int batch = __shfl_sync(0xffffffffu, best.batch, owner & 31);
    const long long u = batch + static_cast<long long>(lane % B) * stride;
    const bool in = owner < 32 && u < r.vecs;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (in) w = r.load(static_cast<int>(u));
    sel.add<T>(w, in, static_cast<uint32_t>(r.first(static_cast<int>(u))));
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
      sel.add<T>(w, in, static_cast<uint32_t>(r.first(static_cast<int>(u))));
    }
  }
  return sel.finish();
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

// B 16-byte vectors are loaded at once.  W warps to a row: one (four rows a block), or all of a block's; or, with
// CLUSTER, a cluster of a.blocks blocks, block `rank` taking the vectors u with
// u / (32 W) % blocks == rank.
template <typename T, bool TOP, int W, int B, bool CLUSTER>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W, W == 1 ? (B == 4 ? 10 : 8) : 32 / W)
    token_logprobs(const LpArgs a) {
  constexpr int N = Vec<T>::N;
  static_assert(!CLUSTER || W == 8, "clusters are made of blocks of eight warps");
  __shared__ float sm[3][W];
  __shared__ float s_out[3];
  __shared__ uint64_t lists[TOP && W > 1 ? W : 1][32];
  __shared__ uint32_t maxima[TOP && W > 1 ? W : 1][32];
  __shared__ uint32_t s_best[TOP ? 32 : 1];
  __shared__ uint64_t s_top[TOP && CLUSTER ? 32 : 1];
  __shared__ uint64_t queues[TOP ? (W == 1 ? 4 : W) : 1][64];
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
    const uint4 *src = reinterpret_cast<const uint4 *>(r.p - r.shift);  // vector 0, of which 0 .. shift - 1 is not ours
    // u0: vector of lane 0; the same branches for the whole warp
    for (int u0 = rank * 32 * W + warp * 32;;) {
      const int u = u0 + lane;
      uint4 w[B];
      if ((r.shift == 0 || u0 > 0) && u0 + 31 + (B - 1) * stride < whole_end) {
#pragma unroll
        for (int i = 0; i < B; ++i) w[i] = __ldg(src + u + i * stride);
        add_batch<T, TOP, false>(w, u, B, st, s2, t2, best);
      } else if (u0 < r.vecs) {
        const int n = min(B, (r.vecs - u0 + stride - 1) / stride);
#pragma unroll
        for (int i = 0; i < B; ++i) {
          w[i] = make_uint4(Vec<T>::kNegInf, Vec<T>::kNegInf, Vec<T>::kNegInf, Vec<T>::kNegInf);
          if (i < n && u + i * stride < r.vecs) w[i] = r.load(u + i * stride);
        }
        add_batch<T, TOP, true>(w, u, n, st, s2, t2, best);
      } else {
        break;
      }
      u0 += B * stride;
    }
    st.s = s2.x + s2.y;
    st.t = t2.x + t2.y;
  }
  const float x_id = writer ? given_logit(a, r, id) : 0.f;  // not needed before the sums are joined
  uint32_t sorted = 0;
  if constexpr (TOP) {
    sorted = warp_largest(ord_of(best.first), a.top, lane);
    if (a.top > 8 && r.vecs > B * stride) {
      // other elements than the first ones, so that many alternatives too have a bar
      // that few elements reach (14781 x 9171 bf16, 32 of them: 219 -> 136 us)
      const uint32_t second = warp_sort(ord_of(best.second), 32, lane);
      sorted = merge_reversed<32>(sorted, __shfl_xor_sync(0xffffffffu, second, 31), lane);
    }
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
    uint64_t key = select_top<T, B>(r, rank * 32 * W + warp * 32, stride, best, bar, a.top,
                                    queues[W == 1 ? threadIdx.x >> 5 : warp], lane);
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
  // blocks find room at once (1 x 50368 fp32: 6.2 us with one, 4.0 with eight;
  // 300 rows: 14.0 with one, 18.5 with two).  Many rows: fewer warps to a row,
  // whose ends cost less (6554 x 50368 bf16: 107 us with eight, 101 with four;
  // 2000 x 2000: 9.8 with eight, 5.9 with four, 4.2 with one), unless a long
  // row would be left to one warp at the end (5000 x 12000 fp32: 38 with four, 46
  // with one; 18000 x 16000 bf16, 8 alternatives: 147 and 128).
  while (a.blocks < 8 && static_cast<long long>(rows) * a.blocks * 2 <= 2ll * sms && vecs >= 1024ll * a.blocks)
    a.blocks *= 2;
  const int C = a.blocks;
  const bool narrow = rows >= 8 * sms && vecs <= (rows >= 48 * sms ? 2048 : 1024);
  const int W = narrow ? 1 : rows > 4 * sms || vecs <= 256 ? 4 : 8;
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
  // rows of at most four vectors a lane: batches of four, more warps an SM
  // (30000 x 250 bf16: 18.2 us with batches of eight, 14.9 with four)
  void (*const kern)(LpArgs) = C > 1                ? token_logprobs<T, TOP, 8, 8, true>
                               : W == 1 && vecs <= 128 ? token_logprobs<T, TOP, 1, 4, false>
                               : W == 1                ? token_logprobs<T, TOP, 1, 8, false>
                               : W == 4                ? token_logprobs<T, TOP, 4, 8, false>
                                                       : token_logprobs<T, TOP, 8, 8, false>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
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
  int rows, V, parts;  // blocks of a row
  const int32_t *ids;
  const float *stats, *entropy, *d_logprob, *d_entropy;
  void *dx;
  long long ld_d;
  int *status;
};

constexpr int kGradBatch = 4;  // vectors a thread loads at once
constexpr int kGradVecs = 8;   // and takes at most

// TPR threads to a row's part: a whole block, or a warp to a whole row.
template <typename T, int TPR>
__global__ void __launch_bounds__(kLpThreads, TPR == 32 ? 5 : 0) token_logprobs_grad(const LpGradArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr bool BLOCK = TPR == kLpThreads;
  const long long row =
      BLOCK ? blockIdx.x / a.parts : blockIdx.x * static_cast<long long>(kLpThreads / TPR) + threadIdx.x / TPR;
  if (!BLOCK && row >= a.rows) return;
  const int part = BLOCK ? static_cast<int>(blockIdx.x - row * a.parts) : 0;
  const int me = threadIdx.x % TPR;
  const Row<T> r(static_cast<const T *>(a.x) + row * a.ld, a.V);
  T *out = static_cast<T *>(a.dx) + row * a.ld_d;
  // whole vectors of x are whole 16-byte words of the gradient too
  const bool same = ((reinterpret_cast<uintptr_t>(r.p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  int id = a.d_logprob ? a.ids[row] : -1;
  if (id >= a.V) {
    if (part == 0 && me == 0) record_status(a.status, AVEY_ERR_DEVICE_BOUNDS);
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
  const int fast_end = same && !none ? min(end, hi) : 0;
  // Vector u, whose elements are w, some of which may not exist.
  auto put = [&](int u, const uint4 &w) {
    const int e0 = r.first(u);
    float v[N];
    if (none) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = 0.f;
    } else {
      gradient(w, v, id >= 0 ? id - e0 : -1);
    }
    if (same && r.whole(u)) {
      *reinterpret_cast<uint4 *>(out + e0) = Vec<T>::pack(v);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (e0 + j >= 0 && e0 + j < a.V) out[e0 + j] = Vec<T>::from_f(v[j]);
    }
  };
  const uint4 *src = reinterpret_cast<const uint4 *>(r.p - r.shift);
  uint4 *dst = reinterpret_cast<uint4 *>(out - r.shift);
  int u = begin + me;
  // The vector that begins before the row: a warp's lane goes on in step with the
  // others; in a block its thread takes its few vectors one by one.
  const bool apart = u == 0 && r.shift != 0;
  if (!BLOCK && apart) {
    put(0, r.load(0));
    u = TPR;
  }
  for (; (!BLOCK || !apart) && u + (kGradBatch - 1) * TPR < fast_end; u += kGradBatch * TPR) {
    uint4 w[kGradBatch];
#pragma unroll
    for (int i = 0; i < kGradBatch; ++i) w[i] = src[u + i * TPR];
#pragma unroll
    for (int i = 0; i < kGradBatch; ++i) {
      float v[N];
      gradient(w[i], v, id - r.first(u + i * TPR));
      dst[u + i * TPR] = Vec<T>::pack(v);
    }
  }
  if constexpr (BLOCK) {
    for (; u < end; u += TPR) put(u, none ? make_uint4(0, 0, 0, 0) : r.load(u));
  } else {
    for (; u < end; u += kGradBatch * TPR) {
      uint4 w[kGradBatch];
#pragma unroll
      for (int i = 0; i < kGradBatch; ++i)
        if (u + i * TPR < end) w[i] = r.load(u + i * TPR);
#pragma unroll
      for (int i = 0; i < kGradBatch; ++i)
        if (u + i * TPR < end) put(u + i * TPR, w[i]);
    }
  }
}

template <typename T>
avey_status run_logprobs_grad(LpGradArgs a, int rows, cudaStream_t s) {
  const long long vecs = (static_cast<long long>(a.V) + 2 * Vec<T>::N - 2) / Vec<T>::N;
  // Short rows: a warp to each (30000 x 1000 bf16: 63 us with a block, 28 so; 8000 x
  // 4096: 31 and 22; 3000 x 8192: 16.0 and 17.0).
  if (vecs <= 1024 && rows >= 8 * sm_count()) {
    a.parts = 1;
    token_logprobs_grad<T, 32><<<(static_cast<unsigned>(rows) + 7) / 8, kLpThreads, 0, s>>>(a);
    AVEY_CHECK_LAUNCH("token_logprobs_grad", s);
    return AVEY_OK;
  }
  long long parts = (vecs + kGradVecs * kLpThreads - 1) / (kGradVecs * kLpThreads);
  parts = std::max<long long>(1, std::min<long long>(parts, 0x7fffffffll / rows));
  a.parts = static_cast<int>(parts);
  token_logprobs_grad<T, kLpThreads><<<static_cast<unsigned>(rows * parts), kLpThreads, 0, s>>>(a);
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
    const uint64_t n = rows, es = dt == AVEY_F32 ? 4 : 2;
    const ByteRows x{reinterpret_cast<uintptr_t>(logits), n, V * es, ld * es};
    const ByteRows d{reinterpret_cast<uintptr_t>(dlogits), n, V * es, ld_d * es};
    AVEY_REQUIRE((x.at == d.at && ld == ld_d) || !rows_overlap(x, d), AVEY_ERR_INVALID_ARG,
                 "%s: dlogits overlaps the logits without being them", fn);
  }
  LpGradArgs a{};
  a.x = logits;
  a.ld = ld;
  a.rows = rows;
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
