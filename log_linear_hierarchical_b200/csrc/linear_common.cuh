// Linear attention with a decay for each head: what its kernels share.
//
// Per (batch, head), with l = exp(log_decay[h]) and a D x D state S (fp32):
//   S_t = l S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t.
// Backward, with G_t = dL/dS_t = l G_{t+1} + scale q_t dO_t^T and G after the last token the
// gradient of the final state:
//   dq_t = scale * S_t dO_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dL/dS_0 = l G_1.
// All four are one operation on three token streams (x, y, z) and a state M,
//   out_i = f1 sum_{j <= i} l^{i-j} (x_i . y_j) z_j + f2 l^{i+1} M^T x_i   (time order), or
//   out_i = f1 sum_{j >= i} l^{j-i} (x_i . y_j) z_j + f2 l^{n-1-i} M^T x_i (reversed),
//   o:  (q, k, v),   M = S            dv: (k, q, dO), M = G,   reversed
//   dq: (dO, v, k),  M = S^T          dk: (v, dO, q), M = G^T, reversed
// over a chunk of n tokens, after which M becomes l^n M + w sum_j l^{n-1-j} y_j z_j^T (time
// order) or l^n M + w sum_j l^{j+1} y_j z_j^T (reversed).  No exponent is ever negative, so
// nothing overflows however strong the decay.
//
// A long sequence is cut into segments that run in parallel: a first pass leaves each
// segment's own state, a scan over the segments turns them into the states that the segments
// start from, and a second pass makes the outputs.
#pragma once

#include "attn_fwd.cuh"  // kLog2e

namespace llsa {

struct LinearStream {
  const void* p;
  long long sb, sh, sn;  // strides in elements
};

struct LinearProblem {
  LinearStream x, y, z;
  void* out;          // [B, H, N, D] contiguous; rows at or past the length are written 0
  const float* init;  // M at the start: per segment [BH][nseg][D][D] (per_segment) or [BH][D][D]; null: 0
  float* state;       // M at the end, [BH][nseg][D][D] in the first pass over segments, else [BH][D][D]; null: not wanted
  float f1, f2, w;
  int rev;            // reversed time order
  int transpose;      // init holds M^T
  int exact;          // the caller gets the state (or one made from it) as fp32
};

struct LinearParams {
  LinearProblem p[3];
  int nprob;
  int H, N, nseg, seg;        // seg: tokens of a segment
  int per_segment;            // init is per segment
  const float* log_decay;     // [H]
  const int* lengths;         // [B] or null
};

// Tokens of batch row b that take part (a value outside [0, N] is recorded and clamped).
__device__ __forceinline__ int linear_length(const int* lengths, int b, int N) {
  if (!lengths) return N;
  const int n = __ldg(lengths + b);
  if (n < 0 || n > N) {
    record_error(LLSA_ERR_INTERNAL);
    return n < 0 ? 0 : N;
  }
  return n;
}

// log_decay, with -inf (no memory at all) replaced by a value whose exponential is 0, so that
// its product with a distance of 0 is 0 and not NaN.
__device__ __forceinline__ float linear_decay(const float* log_decay, int h) {
  const float a = __ldg(log_decay + h);
  return a < -1e5f ? -1e5f : a;
}


}  // namespace llsa
