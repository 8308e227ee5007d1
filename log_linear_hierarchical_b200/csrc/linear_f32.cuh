// Linear attention with a decay for each head for fp32 inputs: one CTA walks the 64-token chunks of
// one segment (see linear_common.cuh for the operation; reversed time order is the same walk over
// tokens taken from the segment's end).
//
// Products run on the tensor cores with fp32 accuracy: each factor is split into two TF32 terms,
// x = hi + lo (hi: x rounded to 11 bits; lo = x - hi exactly, of which TF32 keeps 11 bits), and
// lo hi + hi lo + hi hi of 8 channels at a time are formed on the tensor cores, smallest first, and
// added to the sums on the FP32 pipes: the tensor cores' own additions cut off instead of
// rounding, which over a chunk's sums cost 1.3e-6 of the result instead of 2e-7.  hi is rounded for the
// same reason: cut off, lo would always have x's sign and be twice as large, and what is lost of it
// and with lo lo would add up (7.4e-7 of the result; it is 8 % faster: B = 1, H = 6, N = 65536 forward
// 387 against 416 us at D = 64 and 1185 against 1280 at D = 128; the conversion instruction for
// the addition and mask took 459 and 1416).  mma.sync m16n8k8 does 509 multiply-adds a cycle and SM here, so
// three of them 170, against 128 of the FP32 pipes, with a quarter of their shared-memory reads (on those pipes
// with 4 x 4 register tiles this kernel took 3 to 4 times as long).  The accumulators are summed
// into the state, which lives in registers, in fp32 once a chunk.
//
// Bound: 64-token chunks cost (2 * 64 * D + 2 * D * D) * 64 * 3 multiply-adds, less the part of the
// masked products that is skipped, against 4 * 64 * D * 4 bytes: the tensor work is about twice the
// time of the bytes at D = 64 and three times at D = 128.
#pragma once

#include "linear_common.cuh"

namespace llsa {

constexpr int kLfChunk = 64;

template <int D>
constexpr int linear_f32_smem(bool out) {
  // y, z (x, products and the state's copy) tiles, powers of the decay, row weights
  return 4 * (kLfChunk * D * (out ? 3 : 2) + (out ? kLfChunk * kLfChunk + D * D : 0) + 3 * kLfChunk + 8);
}

// Tiles have rows of D floats whose 4-float pieces are permuted by the row, so that the two ways in
// which fragments read them -- 8 rows x 4 columns, and 4 rows x 8 columns -- both touch 32 banks.
__device__ __forceinline__ int lf_swz(int row) { return ((row & 3) << 3) | (row & 4); }

struct LfPair {
  uint32_t hi, lo;
};
// (From 2^128 (1 - 2^-12) on hi is infinite and the product NaN, as for an infinite x.  A NaN whose bits
// the addition carries past the sign still has a NaN for lo.)
__device__ __forceinline__ LfPair lf_split(float x) {
  const uint32_t hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  return LfPair{hi, __float_as_uint(x - __uint_as_float(hi))};
}

__device__ __forceinline__ void lf_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same without an addend.
__device__ __forceinline__ void lf_mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Fragments of one k step: A (rows r, r + 8; columns k, k + 4) and B (rows k, k + 4; column n).
struct LfA {
  uint32_t hi[4], lo[4];
  __device__ __forceinline__ void set(float v0, float v1, float v2, float v3) {
    const float v[4] = {v0, v1, v2, v3};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const LfPair p = lf_split(v[i]);
      hi[i] = p.hi;
      lo[i] = p.lo;
    }
  }
};
__device__ __forceinline__ void lf_mma3(float (&d)[4], const LfA& a, float b0, float b1) {
  const LfPair p = lf_split(b0), q = lf_split(b1);
  float t[4];
  lf_mma0(t, a.lo, p.hi, q.hi);
  lf_mma(t, a.hi, p.lo, q.lo);
  lf_mma(t, a.hi, p.hi, q.hi);
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] += t[e];
}

// OUT: the outputs and the state; otherwise only the state (the first pass over segments).
template <int D, bool OUT>
__global__ void __launch_bounds__(4 * D, D == 64 ? 2 : 1) linear_f32_kernel(const LinearParams P) {
  constexpr int C = kLfChunk;
  constexpr int T = 4 * D;                 // threads: 4 warps along the rows, WC along the columns
  constexpr int WC = D / 32;
  constexpr int MT = D / 64, NT = 4;       // a warp's tiles of the state: D / 4 rows, 32 columns
  extern __shared__ float4 lf_smem[];
  float* sy = reinterpret_cast<float*>(lf_smem);
  float* sz = sy + C * D;
  float* pw = sz + C * D;  // pw[n] = l^n, n = 0..64
  float* wy = pw + C + 8;  // weight of token j in the state's update
  float* wx = wy + C;      // weight of the state in output row i
  float* sx = wx + C;
  float* sp = sx + (OUT ? C * D : 0);
  float* sm = sp + (OUT ? C * C : 0);
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wr = warp / WC, wc = warp % WC;
  const int fr = lane >> 2, fc = lane & 3;  // fragment row and column
  const int prob = blockIdx.x % P.nprob;
  const int s = (blockIdx.x / P.nprob) % P.nseg, bh = blockIdx.x / P.nprob / P.nseg;
  const LinearProblem& Q = P.p[prob];
  const int b = bh / P.H, h = bh % P.H;
  const float a = linear_decay(P.log_decay, h), a2 = a * kLog2e;
  const int len = linear_length(P.lengths, b, P.N);
  const int lo = s * P.seg, top = min(P.N, lo + P.seg), hi = max(lo, min(top, len));
  if (tid <= C) pw[tid] = exp2f(a2 * (float)tid);

  // the state: rows wr D/4 .. of M, columns 32 wc .., as accumulator fragments
  float m[MT][NT][4];
  const float* init = Q.init ? Q.init + (P.per_segment ? (long long)bh * P.nseg + s : bh) * (D * D) : nullptr;
  auto each_m = [&](auto&& f) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f(m[t][u][e], wr * (D / 4) + 16 * t + fr + 8 * (e >> 1), 32 * wc + 8 * u + 2 * fc + (e & 1));
  };
  each_m([&](float& v, int r, int c) { v = init ? __ldg(init + (Q.transpose ? c * D + r : r * D + c)) : 0.0f; });
  auto copy_m = [&]() {
    each_m([&](float& v, int r, int c) { sm[r * D + (c ^ lf_swz(r))] = v; });
  };
  if (OUT) copy_m();

  auto load_tile = [&](const LinearStream& S, float* dst, int base, int n) {
    const float* src = static_cast<const float*>(S.p) + b * S.sb + h * S.sh;
#pragma unroll
    for (int i = tid; i < C * (D / 4); i += T) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < n) v = __ldg(reinterpret_cast<const float4*>(src + (long long)(Q.rev ? base - r : base + r) * S.sn + c));
      *reinterpret_cast<float4*>(dst + r * D + (c ^ lf_swz(r))) = v;
    }
  };
  // Fragment reads.  The permutations depend on fr or fc alone, so every address is a pointer made once
  // for each of four neighbouring 8-column groups, and a constant.
  // Eight rows from r0 on (a multiple of 8), columns 8g and 8g + 4 on: row_at(.., g % 4)[32 * (g / 4)] is element
  // (r0 + fr, 8g + fc), and (.., 8g + 4 + fc) with `half` 4.
  const int fs = lf_swz(fr), f24 = fs & 24;
  auto row_at = [&](const float* t, int ld, int r0, int g, int half) {
    return t + (r0 + fr) * ld + ((8 * g) ^ f24) + (fc ^ (fs & 4) ^ half);
  };
  // Rows k + fc (and k + 4 + fc with `half` 4), k a multiple of 8, columns c0 + 8g on (c0 a multiple of 32,
  // g < 4): col_at(.., g)[k * D].
  const int cx = fc << 3;
  auto col_at = [&](const float* t, int c0, int g, int half) {
    return t + (fc + half) * D + c0 + ((8 * g) ^ cx) + (fr ^ half);
  };
  const float *zp[4], *zq[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    zp[g] = col_at(sz, 32 * wc, g, 0);
    zq[g] = col_at(sz, 32 * wc, g, 4);
  }
  constexpr int kMinusZ = OUT ? C * D + 3 * C + 8 + C * D + C * C : 0;  // sm - sz

  for (int done = 0; done < hi - lo; done += C) {
    const int n = min(C, hi - lo - done);
    const int base = Q.rev ? hi - 1 - done : lo + done;  // token of row 0; row r is base +- r
    __syncthreads();
    load_tile(Q.y, sy, base, n);
    load_tile(Q.z, sz, base, n);
    if (OUT) load_tile(Q.x, sx, base, n);
    if (tid < C) {
      const int e = Q.rev ? 0 : 1;
      wy[tid] = tid < n ? Q.w * pw[n - tid - e] : 0.0f;
      wx[tid] = pw[tid + e];
    }
    __syncthreads();
    float acc[NT][4];  // output rows 16 wr .., columns 32 wc ..
    if (OUT) {
      const float *x0[4], *x4[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        x0[g] = row_at(sx, D, 16 * wr, g, 0);
        x4[g] = row_at(sx, D, 16 * wr, g, 4);
      }
      // P = f1 l^{i-j} X Y^T: rows 16 wr .., 8-column tiles wc, wc + WC, .., none past the diagonal
      constexpr int PT = 8 / WC;
      float p[PT][4];
#pragma unroll
      for (int u = 0; u < PT; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[u][e] = 0.0f;
      const int to_y = (int)(row_at(sy, D, 8 * wc, 0, 0) - x0[0]);
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          LfA x;
          x.set(x0[g][k], x0[g][k + 8 * D], x4[g][k], x4[g][k + 8 * D]);
          const float *y0 = x0[g] + to_y + k, *y4 = x4[g] + to_y + k;
#pragma unroll
          for (int u = 0; u < PT; ++u)
            if (wc + WC * u < 2 * wr + 2) lf_mma3(p[u], x, y0[8 * WC * u * D], y4[8 * WC * u * D]);
        }
      }
#pragma unroll
      for (int u = 0; u < PT; ++u)
        if (wc + WC * u < 2 * wr + 2) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 16 * wr + fr + 8 * (e >> 1), j = 8 * (WC * u + wc) + 2 * fc + (e & 1);
            sp[i * C + (j ^ lf_swz(i))] = j <= i ? p[u][e] * (Q.f1 * pw[i - j]) : 0.0f;
          }
        }
      // X M
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[u][e] = 0.0f;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          LfA x;
          x.set(x0[g][k], x0[g][k + 8 * D], x4[g][k], x4[g][k + 8 * D]);
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            const int off = kMinusZ + (k + 8 * g) * D;
            lf_mma3(acc[u], x, zp[u][off], zq[u][off]);
          }
        }
      }
      const float w0 = Q.f2 * wx[16 * wr + fr], w1 = Q.f2 * wx[16 * wr + fr + 8];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        acc[u][0] *= w0;
        acc[u][1] *= w0;
        acc[u][2] *= w1;
        acc[u][3] *= w1;
      }
      __syncthreads();  // the products are written, the state's copy has been read
      // + P Z, up to the diagonal and the last token
      const int last = min(n, 16 * wr + 16);
#pragma unroll 1
      for (int k = 0; k < last; k += 16) {  // (rows behind the last token are zeros)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          LfA q;
          const float *p0 = row_at(sp, C, 16 * wr, ((k >> 3) & 3) + g, 0) + (k & 32),
                      *p4 = row_at(sp, C, 16 * wr, ((k >> 3) & 3) + g, 4) + (k & 32);
          q.set(p0[0], p0[8 * C], p4[0], p4[8 * C]);
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            const int off = (k + 8 * g) * D;
            lf_mma3(acc[u], q, zp[u][off], zq[u][off]);
          }
        }
      }
      float* out = static_cast<float*>(Q.out) + (long long)bh * P.N * D + 32 * wc + 2 * fc;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 16 * wr + fr + 8 * e;
        if (i < n) {
          float* dst = out + (long long)(Q.rev ? base - i : base + i) * D;
#pragma unroll
          for (int u = 0; u < NT; ++u)
            *reinterpret_cast<float2*>(dst + 8 * u) = make_float2(acc[u][2 * e], acc[u][2 * e + 1]);
        }
      }
    }
    // T = (w Y)^T Z; M + M (l^n - 1) + T rather than l^n M + T, so that a factor close to 1 repeated
    // over thousands of chunks does not add up its rounding
    if (OUT && done + C >= hi - lo && Q.state == nullptr) break;  // no chunk follows and nobody asks
    const float fall = expm1f(a * (float)n);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float t[NT][4];
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[u][e] = 0.0f;
      const int r0 = wr * (D / 4) + 16 * i;
      const float *ya = col_at(sy, r0 & ~31, (r0 & 31) / 8, 0), *yb = col_at(sy, r0 & ~31, (r0 & 31) / 8 + 1, 0),
                  *ya4 = col_at(sy, r0 & ~31, (r0 & 31) / 8, 4), *yb4 = col_at(sy, r0 & ~31, (r0 & 31) / 8 + 1, 4);
#pragma unroll 1
      for (int k = 0; k < n; k += 16) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          LfA y;
          const int kr = k + 8 * g;
          const float w0 = wy[kr + fc], w1 = wy[kr + 4 + fc];
          y.set(w0 * ya[kr * D], w0 * yb[kr * D], w1 * ya4[kr * D], w1 * yb4[kr * D]);
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            const int off = kr * D;
            lf_mma3(t[u], y, zp[u][off], zq[u][off]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) m[i][u][e] = fmaf(m[i][u][e], fall, m[i][u][e]) + t[u][e];
    }
    if (OUT && done + C < hi - lo) copy_m();
  }
  if (OUT) {  // rows that take no part
    float4* out = reinterpret_cast<float4*>(static_cast<float*>(Q.out) + ((long long)bh * P.N + hi) * D);
    for (long long i = tid; i < (long long)(top - hi) * (D / 4); i += T) out[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (Q.state) {
    float* dst = Q.state + (OUT ? (long long)bh : (long long)bh * P.nseg + s) * (D * D);
    each_m([&](float& v, int r, int c) { dst[r * D + c] = v; });
  }
}

}  // namespace llsa
