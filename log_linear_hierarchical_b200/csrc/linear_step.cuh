// One token of linear attention with a decay for each head, over a pool of states:
//   S = exp(log_decay[h]) pool[slots[b], h] + k v^T,  o = scale * S^T q,  pool[out_slots[b], h] = S.
// The states are fp32 and make up the traffic (8 D^2 bytes per batch row and head, read and
// written once), so HBM bounds it, or the launch's latency when there are few rows.  A CTA
// takes 32 of the D columns: 8 threads hold a row's 128 bytes as float4 and 16 groups of them
// the rows, so every access is a whole 128-byte line and all of a thread's D/16 loads are in
// flight together.
#pragma once

#include "linear_common.cuh"
#include "rotary.cuh"

namespace llsa {

constexpr int kStepThreads = 128;

struct StepParams {
  const void* q;
  const void* k;
  const void* v;  // [B, H, D] contiguous
  void* o;
  const float* log_decay;
  float* pool;             // [pool_rows, H, D, D]
  const int* slots;        // [B] or null: row b uses slot b
  const int* out_slots;    // [B] or null: as read
  int B, H, pool_rows;
  float scale;
};

// Rows with a negative slot take no part (o = 0).  A row with a slot outside the pool, or that
// would race with an earlier row of valid slots (one of the two writes what the other reads or
// writes), is recorded as LLSA_ERR_INTERNAL and takes no part either, so the first row with a
// slot has it.
__device__ __forceinline__ bool step_row_allowed(const StepParams& P, int b, int in, int out) {
  bool bad = false;
  if (P.slots || P.out_slots)
    for (int r = threadIdx.x; r < b; r += kStepThreads) {
      const int i = P.slots ? __ldg(P.slots + r) : r;
      const int o = P.out_slots ? __ldg(P.out_slots + r) : i;
      if (i >= 0 && o >= 0 && i < P.pool_rows && o < P.pool_rows) bad = bad || o == out || o == in || i == out;
    }
  bad = __syncthreads_or(bad);
  if (in < 0 || out < 0) return false;
  if (bad || in >= P.pool_rows || out >= P.pool_rows) {
    if (threadIdx.x == 0) record_error(LLSA_ERR_INTERNAL);
    return false;
  }
  return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(kStepThreads) linear_step_kernel(const StepParams P) {
  constexpr int R = D / 16;  // rows of one thread
  __shared__ float part[16][33];
  pdl_enter();
  const int slabs = D / 32;
  const int slab = blockIdx.x % slabs, bh = blockIdx.x / slabs;
  const int b = bh / P.H, h = bh % P.H;
  const int c = threadIdx.x % 8, g = threadIdx.x / 8;
  const int in = P.slots ? __ldg(P.slots + b) : b;
  const int out = P.out_slots ? __ldg(P.out_slots + b) : in;
  T* o = static_cast<T*>(P.o) + (long long)bh * D + slab * 32;
  if (!step_row_allowed(P, b, in, out)) {
    if (threadIdx.x < 32) o[threadIdx.x] = from_f32<T>(0.0f);
    return;
  }
  const float4* src = reinterpret_cast<const float4*>(P.pool + ((long long)in * P.H + h) * (D * D)) + slab * 8 + c;
  float4* dst = reinterpret_cast<float4*>(P.pool + ((long long)out * P.H + h) * (D * D)) + slab * 8 + c;
  float4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) s[i] = src[(long long)(g + 16 * i) * (D / 4)];
  const T* q = static_cast<const T*>(P.q) + (long long)bh * D;
  const T* k = static_cast<const T*>(P.k) + (long long)bh * D;
  const T* v = static_cast<const T*>(P.v) + (long long)bh * D + slab * 32 + 4 * c;
  const float fall = expm1f(linear_decay(P.log_decay, h));  // S + S (l - 1): l's own rounding would add up
  const float v0 = to_f32(v[0]), v1 = to_f32(v[1]), v2 = to_f32(v[2]), v3 = to_f32(v[3]);
  float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float kd = to_f32(k[g + 16 * i]), qd = to_f32(q[g + 16 * i]);
    s[i].x = fmaf(kd, v0, fmaf(s[i].x, fall, s[i].x));
    s[i].y = fmaf(kd, v1, fmaf(s[i].y, fall, s[i].y));
    s[i].z = fmaf(kd, v2, fmaf(s[i].z, fall, s[i].z));
    s[i].w = fmaf(kd, v3, fmaf(s[i].w, fall, s[i].w));
    a0 = fmaf(qd, s[i].x, a0);
    a1 = fmaf(qd, s[i].y, a1);
    a2 = fmaf(qd, s[i].z, a2);
    a3 = fmaf(qd, s[i].w, a3);
    dst[(long long)(g + 16 * i) * (D / 4)] = s[i];
  }
  part[g][4 * c] = a0;
  part[g][4 * c + 1] = a1;
  part[g][4 * c + 2] = a2;
  part[g][4 * c + 3] = a3;
  __syncthreads();
  if (threadIdx.x < 32) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += part[i][threadIdx.x];
    o[threadIdx.x] = from_f32<T>(P.scale * t);
  }
}

}  // namespace llsa
