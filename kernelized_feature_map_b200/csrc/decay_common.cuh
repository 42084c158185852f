// decay_common.cuh -- device helpers of the operators on packed sequences and
// state pools: the sequence and segment a CTA works on, and the pool row an
// index names.
#pragma once

#include <stdint.h>

#include "kata_common.cuh"

namespace kata {

constexpr int kStatusInvalidArg = 1;  // KATA_ERR_INVALID_ARG

// One segment of one packed sequence: tokens [t0, t1) of [s0, s1).
struct Segment {
  int seq;     // sequence, -1: there is no segment of this number
  int s0, s1;  // the sequence's tokens
  int seg, n_seg;
  int t0, t1;  // the segment's tokens
  int rec;     // records of the split sequences before this one, in segments
};

// Token range of sequence n.  cu is used as its running maximum clamped to
// [0, T], so ranges never overlap or leave the tensors whatever it holds.
// All lanes of a warp take part; lane l looks at sequence n0 + l and carry is
// the end of sequence n0 - 1.  Returns false where the entries had to be
// mended.
__device__ __forceinline__ bool seq_range(const int* __restrict__ cu, int n0, int N, int T, int carry, int lane,
                                          int& s0, int& s1) {
  const int n = n0 + lane;
  const int c0 = cu ? (n < N ? cu[n] : T) : (n == 0 ? 0 : T);
  const int c1 = cu ? (n < N ? cu[n + 1] : T) : T;
  int e = n < N ? min(max(c1, 0), T) : 0;
  const int b = n < N ? min(max(c0, 0), T) : 0;
  // running maximum over the ends, the first sequence's start included
  e = max(e, b);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, e, o);
    if (lane >= o) e = max(e, x);
  }
  e = max(e, carry);
  int prev = __shfl_up_sync(0xffffffffu, e, 1);
  if (lane == 0) prev = carry;
  s0 = max(prev, b);
  s1 = max(e, s0);
  return n >= N || (c0 >= 0 && c1 <= T && c0 <= c1);
}

// What find_segment counts: segments (an empty sequence is one empty segment),
// only those of sequences that are cut into more than one, these sequences, or
// those that are not cut.
enum FindWhat { kSegments, kSplitSegments, kSplitSequences, kWholeSequences };

// The target-th segment, or the first segment of the target-th split
// sequence, when every sequence is cut into segments of L tokens.  Called by
// a whole warp; the result is the same in all lanes.  `valid` is false where
// cu's entries up to the target had to be mended.
__device__ __forceinline__ Segment find_segment(const int* __restrict__ cu, int N, int T, int L, FindWhat what,
                                                int target, int lane, bool& valid) {
  Segment r{-1, 0, 0, 0, 0, 0, 0, 0};
  int carry = 0, counted = 0, recs = 0;
  valid = true;
  for (int n0 = 0; n0 < N; n0 += 32) {
    int s0, s1;
    const bool ok = seq_range(cu, n0, N, T, carry, lane, s0, s1);
    valid = valid && __all_sync(0xffffffffu, ok);
    const int n = n0 + lane;
    const int segs = n < N ? max(1, (s1 - s0 + L - 1) / L) : 0;
    const int rec = segs > 1 ? segs : 0;
    const int mine = what == kSegments        ? segs
                     : what == kSplitSegments ? rec
                     : what == kWholeSequences ? (segs == 1 ? 1 : 0)
                                               : (rec > 0 ? 1 : 0);
    int pc = mine, pr = rec;  // inclusive prefix sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, pc, o), y = __shfl_up_sync(0xffffffffu, pr, o);
      if (lane >= o) {
        pc += x;
        pr += y;
      }
    }
    const bool here = target >= counted + pc - mine && target < counted + pc;
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
      const int src = __ffs(who) - 1;
      r.seq = n0 + src;
      r.s0 = __shfl_sync(0xffffffffu, s0, src);
      r.s1 = __shfl_sync(0xffffffffu, s1, src);
      r.n_seg = __shfl_sync(0xffffffffu, segs, src);
      r.seg = what == kSplitSequences || what == kWholeSequences ? 0 : target - (counted + __shfl_sync(0xffffffffu, pc - mine, src));
      r.rec = recs + __shfl_sync(0xffffffffu, pr - rec, src);
      r.t0 = r.s0 + r.seg * L;
      r.t1 = min(r.s1, r.t0 + L);
      return r;
    }
    counted += __shfl_sync(0xffffffffu, pc, 31);
    recs += __shfl_sync(0xffffffffu, pr, 31);
    carry = __shfl_sync(0xffffffffu, s1, 31);
  }
  return r;
}

// Sequences that are not cut into segments of L tokens.  Called by a whole warp.
__device__ __forceinline__ int count_whole(const int* __restrict__ cu, int N, int T, int L, int lane) {
  int carry = 0, count = 0;
  for (int n0 = 0; n0 < N; n0 += 32) {
    int s0, s1;
    seq_range(cu, n0, N, T, carry, lane, s0, s1);
    count += __popc(__ballot_sync(0xffffffffu, n0 + lane < N && s1 - s0 <= L));
    carry = __shfl_sync(0xffffffffu, s1, 31);
  }
  return count;
}

// Pool row named by index i of `idx` (null: i itself), or -1 where the index
// is negative, out of range, or (unique) already named by an earlier one; the
// latter two report.  Called by a whole warp, the same result in all lanes.
__device__ __forceinline__ int pool_row(const int* __restrict__ idx, int i, int rows, bool unique, int lane,
                                        int* status) {
  if (!idx) return i;
  const int s = idx[i], first = unique && lane < i ? idx[lane] : -1;  // both loads at once
  if (s < 0) return -1;
  bool bad = s >= rows || first == s;
  if (unique)
    for (int j = lane + 32; j < i; j += 32) bad = bad || idx[j] == s;
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) report_status(status, kStatusInvalidArg);
    return -1;
  }
  return s;
}

// The decay's logarithm as used: at most 0 (a larger one or NaN reports and
// counts as 0) and finite (-infinity becomes a number whose exponential is 0
// and whose product with 0 is 0).
__device__ __forceinline__ float used_log_decay(float g, int* status) {
  if (!(g <= 0.f)) {
    report_status(status, kStatusInvalidArg);
    return 0.f;
  }
  return fmaxf(g, -1e30f);
}

// exp(g), g <= 0, as hi + lo.  A single fp32 factor is off by up to 2^-25,
// and a recurrence that multiplies by it every token is off by that times the
// tokens walked: at a = 1 - 2^-12 more than 2^-13 over the state's reach.  Up
// to g = -0.5 (beyond, nothing reaches far) hi is 1 + expm1(g) rounded and lo
// what that rounding left out, exactly.
__device__ __forceinline__ void decay_factor(float g, float& hi, float& lo) {
  if (g > -0.5f) {
    const float e = expm1f(g);
    hi = 1.f + e;
    lo = e - (hi - 1.f);
  } else {
    hi = expf(g);
    lo = 0.f;
  }
}

}  // namespace kata
