// avey_score.cuh -- softmax statistics of scored rows, shared by the products that
// score their outputs.  They work on logits in units of log 2, y = logit * log2 e.
#pragma once

#include "avey_common.cuh"
#include "avey_internal.h"

namespace avey {

constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kFar2 = -200.0f;  // ex2 is 0 in fp32 from here down
// The value of words past the last and of those whose bias is lower (-inf among
// them): finite, so that 0 * (y - m) stays 0.
constexpr float kMaskedWord = -1e30f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// (max, sum 2^(y - max), sum 2^(y - max) (y - max))
struct Stat2 {
  float m, s, t;
};
__device__ __forceinline__ void rebase2(Stat2 &a, float M) {
  const float d = a.m - M, f = ex2(d);
  a.t = f * fmaf(a.s, fmaxf(d, kFar2), a.t);
  a.s *= f;
  a.m = M;
}
__device__ __forceinline__ void join2(Stat2 &a, Stat2 b) {
  const float M = fmaxf(a.m, b.m);
  rebase2(a, M);
  rebase2(b, M);
  a.s += b.s;
  a.t += b.t;
}

// A row's outputs from its statistics; given: it has a given token, of logit y.
__device__ __forceinline__ void write_scores(const Stat2 &st, long long row, bool given, float y, float *logprob,
                                             float *stats, float *entropy) {
  const bool empty = st.m <= 0.5f * kMaskedWord;
  const bool bad = !(st.s < INFINITY) || st.m == INFINITY;
  const float nan = __uint_as_float(0x7fc00000u);
  const float z = logf(st.s);
  if (logprob) logprob[row] = !given ? 0.f : bad ? nan : empty ? -INFINITY : fmaf(y - st.m, kLn2, -z);
  if (stats)
    reinterpret_cast<float2 *>(stats)[row] =
        bad ? make_float2(nan, nan) : empty ? make_float2(-INFINITY, 0.f) : make_float2(st.m * kLn2, z);
  if (entropy) entropy[row] = bad ? nan : empty ? 0.f : fmaf(-kLn2, st.t / st.s, z);
}

}  // namespace avey
