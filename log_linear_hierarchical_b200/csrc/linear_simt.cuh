// Linear attention with a decay for each head, on the FP32 pipes: one CTA walks the chunks of
// one segment with the three token tiles, the masked products and the state in shared memory,
// all fp32 (see linear_common.cuh for the operation).
#pragma once

#include "linear_common.cuh"
#include "rotary.cuh"  // load8 / store8

namespace llsa {

constexpr int kLsThreads = 256;
constexpr int kLsChunk = 64;

template <int D>
constexpr int linear_simt_smem(bool out) {
  // z, y (and x, products) tiles with 4 floats of padding a row, the state, the row weights
  return 4 * (kLsChunk * (D + 4) * (out ? 3 : 2) + D * (D + 4) + (out ? kLsChunk * (kLsChunk + 4) : 0) + 2 * kLsChunk);
}

// OUT: the outputs and the state; otherwise only the state (the first pass over segments).
template <typename T, int D, bool OUT>
__global__ void __launch_bounds__(kLsThreads) linear_simt_kernel(const LinearParams P) {
  constexpr int C = kLsChunk, LD = D + 4, LP = C + 4, E = D / 64;
  extern __shared__ float4 ls_smem[];
  float* sy = reinterpret_cast<float*>(ls_smem);
  float* sz = sy + C * LD;
  float* sm = sz + C * LD;
  float* wy = sm + D * LD;   // weight of token j in the state's update
  float* wx = wy + C;        // weight of the state in output row i
  float* sx = wx + C;
  float* sp = sx + (OUT ? C * LD : 0);
  pdl_enter();
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const int prob = blockIdx.x % P.nprob;
  const int s = (blockIdx.x / P.nprob) % P.nseg, bh = blockIdx.x / P.nprob / P.nseg;
  const LinearProblem& Q = P.p[prob];
  const int b = bh / P.H, h = bh % P.H;
  const float a = linear_decay(P.log_decay, h), a2 = a * kLog2e;
  const int len = linear_length(P.lengths, b, P.N);
  const int lo = s * P.seg, top = min(P.N, lo + P.seg), hi = max(lo, min(top, len));

  // the state: M or its transpose
  {
    const float* init = Q.init ? Q.init + (P.per_segment ? (long long)bh * P.nseg + s : bh) * (D * D) : nullptr;
    for (int i = tid; i < D * D; i += kLsThreads) {
      const int r = i / D, c = i % D;
      const float v = init ? init[i] : 0.0f;
      if (Q.transpose)
        sm[c * LD + r] = v;
      else
        sm[r * LD + c] = v;
    }
  }
  auto load_tile = [&](const LinearStream& S, float* dst, int base, int n) {
    const T* src = static_cast<const T*>(S.p) + b * S.sb + h * S.sh;
    for (int i = tid; i < C * (D / 8); i += kLsThreads) {
      const int r = i / (D / 8), c = (i % (D / 8)) * 8;
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (r < n) load8<T>(src + (long long)(Q.rev ? base - r : base + r) * S.sn + c, v);
      store8<float>(dst + r * LD + c, v);
    }
  };

  for (int done = 0; done < hi - lo; done += C) {
    const int n = min(C, hi - lo - done);
    const int base = Q.rev ? hi - 1 - done : lo + done;  // token of row 0; row r is base +- r
    __syncthreads();
    load_tile(Q.y, sy, base, n);
    load_tile(Q.z, sz, base, n);
    if (OUT) load_tile(Q.x, sx, base, n);
    if (tid < C) {
      const int e = Q.rev ? 0 : 1;
      wy[tid] = tid < n ? Q.w * exp2f(a2 * (float)(n - tid - e)) : 0.0f;
      wx[tid] = exp2f(a2 * (float)(tid + e));
    }
    __syncthreads();
    float acc[4][E * 4];
    if (OUT) {
      float p[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) p[r][c] = 0.0f;
      for (int d = 0; d < D; d += 4) {
        float4 xa[4], yb[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) xa[r] = *reinterpret_cast<const float4*>(sx + (ty * 4 + r) * LD + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) yb[c] = *reinterpret_cast<const float4*>(sy + (tx + 16 * c) * LD + d);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            p[r][c] += xa[r].x * yb[c].x + xa[r].y * yb[c].y + xa[r].z * yb[c].z + xa[r].w * yb[c].w;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int i = ty * 4 + r, j = tx + 16 * c;
          sp[i * LP + j] = j <= i ? p[r][c] * exp2f(a2 * (float)(i - j)) : 0.0f;
        }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < E * 4; ++c) acc[r][c] = 0.0f;
      for (int d = 0; d < D; d += 4) {
        float xr[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 v = *reinterpret_cast<const float4*>(sx + (ty * 4 + r) * LD + d);
          xr[r][0] = v.x, xr[r][1] = v.y, xr[r][2] = v.z, xr[r][3] = v.w;
        }
#pragma unroll
        for (int dd = 0; dd < 4; ++dd)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float4 m = *reinterpret_cast<const float4*>(sm + (d + dd) * LD + tx * 4 + 64 * e);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              acc[r][4 * e] += xr[r][dd] * m.x;
              acc[r][4 * e + 1] += xr[r][dd] * m.y;
              acc[r][4 * e + 2] += xr[r][dd] * m.z;
              acc[r][4 * e + 3] += xr[r][dd] * m.w;
            }
          }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float f = Q.f2 * wx[ty * 4 + r];
#pragma unroll
        for (int c = 0; c < E * 4; ++c) acc[r][c] *= f;
      }
    }
    __syncthreads();  // the products are written, the state has been read
    if (OUT) {
      float acc1[4][E * 4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < E * 4; ++c) acc1[r][c] = 0.0f;
      for (int j = 0; j < n; ++j) {
        float pr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) pr[r] = sp[(ty * 4 + r) * LP + j];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float4 m = *reinterpret_cast<const float4*>(sz + j * LD + tx * 4 + 64 * e);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            acc1[r][4 * e] += pr[r] * m.x;
            acc1[r][4 * e + 1] += pr[r] * m.y;
            acc1[r][4 * e + 2] += pr[r] * m.z;
            acc1[r][4 * e + 3] += pr[r] * m.w;
          }
        }
      }
      T* out = static_cast<T*>(Q.out) + (long long)bh * P.N * D;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = ty * 4 + r;
        if (i < n) {
          T* dst = out + (long long)(Q.rev ? base - i : base + i) * D + tx * 4;
#pragma unroll
          for (int c = 0; c < E * 4; ++c)
            dst[64 * (c / 4) + c % 4] = from_f32<T>(Q.f1 * acc1[r][c] + acc[r][c]);
        }
      }
    }
    // the state: M + M (l^n - 1) rather than l^n M, so that a factor close to 1 repeated over
    // thousands of chunks does not add up its rounding
    const float fall = expm1f(a * (float)n);
#pragma unroll 1
    for (int u = 0; u < E; ++u) {
      float t[4][E * 4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < E * 4; ++c) t[r][c] = 0.0f;
      for (int j = 0; j < n; ++j) {
        const float4 yv = *reinterpret_cast<const float4*>(sy + j * LD + ty * 4 + 64 * u);
        const float yr[4] = {yv.x * wy[j], yv.y * wy[j], yv.z * wy[j], yv.w * wy[j]};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float4 m = *reinterpret_cast<const float4*>(sz + j * LD + tx * 4 + 64 * e);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            t[r][4 * e] += yr[r] * m.x;
            t[r][4 * e + 1] += yr[r] * m.y;
            t[r][4 * e + 2] += yr[r] * m.z;
            t[r][4 * e + 3] += yr[r] * m.w;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < E * 4; ++c) {
          float* m = sm + (ty * 4 + r + 64 * u) * LD + tx * 4 + 64 * (c / 4) + c % 4;
          *m = fmaf(*m, fall, *m) + t[r][c];
        }
    }
  }
  __syncthreads();
  if (OUT) {  // rows that take no part
    T* out = static_cast<T*>(Q.out) + ((long long)bh * P.N + hi) * D;
    for (long long i = tid; i < (long long)(top - hi) * D; i += kLsThreads) out[i] = from_f32<T>(0.0f);
  }
  if (Q.state) {
    float* dst = Q.state + (OUT ? (long long)bh : (long long)bh * P.nseg + s) * (D * D);
    for (int i = tid; i < D * D; i += kLsThreads) dst[i] = sm[(i / D) * LD + i % D];
  }
}

// The states between segments, in place: slot s of [BH][nseg][D*D] holds segment s's own
// state on entry and the state that the segment starts from (time order: everything before
// it; reversed: everything after it) on return; `last` receives the state after all of them.
// Latency bounds it: one value a thread, kScanAhead segments' values in flight before the first is
// used, addresses by addition (6 heads x 47 segments of 64 x 64: 7.8 us, the launch's 3 included.  Sharing
// a value's segments out to 8 warps that meet in shared memory saved 2 us there and cost 10 at D = 128,
// whose 4 times as many values fill the GPU by themselves).
constexpr int kScanThreads = 64, kScanAhead = 32;

__global__ void __launch_bounds__(kScanThreads)
    linear_scan_kernel(float* __restrict__ states, const float* __restrict__ init, float* __restrict__ last,
                       const float* __restrict__ log_decay, const int* __restrict__ lengths, int H, int N, int nseg,
                       int seg, int dd, int rev) {
  pdl_enter();
  const int per = dd / kScanThreads;  // CTAs of one (batch, head)
  const int bh = blockIdx.x / per, e = (blockIdx.x % per) * kScanThreads + threadIdx.x;
  const float a = linear_decay(log_decay, bh % H);
  const int len = linear_length(lengths, bh / H, N);
  // the segments' factors less 1, in scan order: whole ones before (reversed: after) place `part_at`,
  // a part of one there, none on its other side
  const int full = len / seg, part_at = rev ? nseg - 1 - full : full;
  const float whole = expm1f(a * (float)seg), part = expm1f(a * (float)(len - full * seg));
  const float before = rev ? 0.0f : whole, after = rev ? whole : 0.0f;
  float m = init ? init[(long long)bh * dd + e] : 0.0f;
  const ptrdiff_t step = rev ? -(ptrdiff_t)dd : (ptrdiff_t)dd;
  float* in = states + ((long long)bh * nseg + (rev ? nseg - 1 : 0)) * dd + e;
  float* out = in;
  for (int i0 = 0; i0 < nseg; i0 += kScanAhead) {
    float own[kScanAhead];
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i) {
      if (i0 + i < nseg) own[i] = *in;
      in += step;
    }
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i) {
      if (i0 + i < nseg) {
        *out = m;
        m = fmaf(m, i0 + i == part_at ? part : (i0 + i < part_at ? before : after), m) + own[i];
      }
      out += step;
    }
  }
  if (last) last[(long long)bh * dd + e] = m;
}

}  // namespace llsa
