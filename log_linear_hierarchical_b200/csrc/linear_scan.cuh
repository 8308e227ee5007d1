// The scan over a sequence's segments (linear attention with a decay for each head).
#pragma once

#include "linear_common.cuh"

namespace llsa {

// The states between segments, in place: slot s of [BH][nseg][D*D] holds segment s's own
// state on entry and the state that the segment starts from (time order: everything before
// it; reversed: everything after it) on return; `last` receives the state after all of them.
// Latency bounds it when there are few (batch, head) pairs: one value a thread (V = float),
// kScanAhead segments' values in flight before the first is used, addresses by addition (6 heads x 47
// segments of 64 x 64: 7.8 us, the launch's 3 included.  Sharing a value's segments out to 8 warps that
// meet in shared memory saved 2 us there and cost 10 at D = 128).  With many pairs the values themselves
// fill the GPU, and a thread takes four (V = float4).
constexpr int kScanThreads = 64;

__device__ __forceinline__ float scan_step(float m, float f, float own) { return fmaf(m, f, m) + own; }
__device__ __forceinline__ float4 scan_step(float4 m, float f, float4 own) {
  return make_float4(scan_step(m.x, f, own.x), scan_step(m.y, f, own.y), scan_step(m.z, f, own.z),
                     scan_step(m.w, f, own.w));
}

template <typename V>
__global__ void __launch_bounds__(kScanThreads)
    linear_scan_kernel(V* __restrict__ states, const V* __restrict__ init, V* __restrict__ last,
                       const float* __restrict__ log_decay, const int* __restrict__ lengths, int H, int N, int nseg,
                       int seg, int dd, int rev) {
  constexpr int kScanAhead = sizeof(V) == 4 ? 32 : 8;
  pdl_enter();
  const int per = dd / kScanThreads;  // CTAs of one (batch, head); dd: values V of a state
  const int bh = blockIdx.x / per, e = (blockIdx.x % per) * kScanThreads + threadIdx.x;
  const float a = linear_decay(log_decay, bh % H);
  const int len = linear_length(lengths, bh / H, N);
  // the segments' factors less 1, in scan order: whole ones before (reversed: after) place `part_at`,
  // a part of one there, none on its other side
  const int full = len / seg, part_at = rev ? nseg - 1 - full : full;
  const float whole = expm1f(a * (float)seg), part = expm1f(a * (float)(len - full * seg));
  const float before = rev ? 0.0f : whole, after = rev ? whole : 0.0f;
  V m{};
  if (init) m = init[(long long)bh * dd + e];
  const ptrdiff_t step = rev ? -(ptrdiff_t)dd : (ptrdiff_t)dd;
  V* in = states + ((long long)bh * nseg + (rev ? nseg - 1 : 0)) * dd + e;
  V* out = in;
  for (int i0 = 0; i0 < nseg; i0 += kScanAhead) {
    V own[kScanAhead];
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i) {
      if (i0 + i < nseg) own[i] = *in;
      in += step;
    }
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i) {
      if (i0 + i < nseg) {
        *out = m;
        m = scan_step(m, i0 + i == part_at ? part : (i0 + i < part_at ? before : after), own[i]);
      }
      out += step;
    }
  }
  if (last) last[(long long)bh * dd + e] = m;
}

}  // namespace llsa
