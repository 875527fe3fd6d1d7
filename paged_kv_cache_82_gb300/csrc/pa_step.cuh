// pa_step.cuh -- device helpers of the kernels that take a step's metadata
// token by token (norm + rotation, bounds, selection, selected attention).
#pragma once

#include "pa_common.cuh"
#include "pa_step.h"

namespace pa {

// The request that token t belongs to: the largest r < num_seqs with qsl[r] <=
// t (called by a whole warp; qsl is non-decreasing and starts at 0).  A 32-ary
// search: one load per lane and round, two rounds up to 1024 requests.  The
// caller checks that t really lies in [qsl[r], qsl[r + 1]).
__device__ __forceinline__ int warp_find_request(const int32_t* __restrict__ qsl,
                                                 int num_seqs, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = num_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int64_t i = lo + (int64_t)lane * step;
    const unsigned below = __ballot_sync(~0u, i < hi && __ldg(qsl + i) <= t);
    if (below == 0) break;
    lo += (31 - __clz(below)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The same with the request's metadata; in: t is one of its tokens.  Where the
// requests have equally many tokens (a decode step), t's place among the tokens
// names the request: one round of loads instead of the search's two or three
// before the request's own.
struct TokenReq {
  int r;
  ReqMeta m;
  bool in;
};
__device__ __forceinline__ TokenReq warp_token_request(
    const int32_t* __restrict__ qsl, const int32_t* __restrict__ seq_lens, int num_seqs,
    int64_t t, int64_t num_tokens, int max_query_len, int max_seq_len,
    int max_blocks_per_seq) {
  TokenReq q;
  q.r = (int)(t * num_seqs / num_tokens);
  q.m = load_req(qsl, seq_lens, q.r, num_tokens, max_query_len, max_seq_len,
                 max_blocks_per_seq);
  q.in = t >= q.m.q0 && t < (int64_t)q.m.q0 + q.m.n;
  if (!q.in) {
    q.r = warp_find_request(qsl, num_seqs, t);
    q.m = load_req(qsl, seq_lens, q.r, num_tokens, max_query_len, max_seq_len,
                   max_blocks_per_seq);
    q.in = t >= q.m.q0 && t < (int64_t)q.m.q0 + q.m.n;
  }
  return q;
}

// Flags broken metadata of any request, of those no token points to as well (a
// negative length or count of tokens).  Every thread of the grid calls it, with its
// number and how many they are.
__device__ __forceinline__ void check_requests(const StepView& s, int64_t thread,
                                               int64_t threads) {
  for (int64_t r = thread; r < s.num_seqs; r += threads)
    if (!load_req(s.query_start_loc, s.seq_lens, (int)r, s.num_tokens, s.max_query_len,
                  s.max_seq_len, s.max_blocks_per_seq)
             .ok)
      flag_error(s.err, PA_DEV_ERR_METADATA);
}

// fl32(x / s) for many x and one s: from the correctly rounded 1 / s by two of
// Markstein's corrections (IBM J. Res. Dev. 34, 1990).  x * rcp is within 3/2
// of a step of x / s; the first correction leaves the quotient within one step,
// so that the second rounds it correctly.  A third of the instructions of a
// division.  easy: s and 1 / s are normal with room (the quotient of a 16-bit
// or narrower x does not vanish, the remainders stay exact where they decide
// anything); elsewhere, for quotients that overflow and for NaN, the plain
// operations.
struct Divisor {
  float s, rcp;
  bool easy;
  // used: false where no division follows (saves the reciprocal)
  __device__ __forceinline__ explicit Divisor(float d, bool used = true) : s(d) {
    easy = used && d >= 0x1p-100f && d <= 0x1p+16f;
    rcp = easy ? __frcp_rn(d) : 0.f;
  }
  __device__ __forceinline__ float corrected(float x) const {
    const float y0 = x * rcp;
    float y = fmaf(fmaf(-y0, s, x), rcp, y0);
    y = fmaf(fmaf(-y, s, x), rcp, y);
    // (a correction turns -0 into 0: the sign is x's)
    return fabsf(y0) <= 0x1p+100f ? copysignf(y, x) : y0;
  }
};

// y[i] = fl32(x[i] / d)
template <int kN>
__device__ __forceinline__ void divide(const float (&x)[kN], const Divisor& d,
                                       float (&y)[kN]) {
  if (d.easy) {
#pragma unroll
    for (int i = 0; i < kN; ++i) y[i] = d.corrected(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) y[i] = __fdiv_rn(x[i], d.s);
  }
}

}  // namespace pa
