// Rotary positions of one or two [B, H, N, D] tensors (a layer's q and k) in one launch.
//
// Pair c (x_a, x_b) of the rotated channels turns by t = position * frequency[c]:
//   y_a = s (x_a cos t - x_b sin t),  y_b = s (x_b cos t + x_a sin t),
// with a = first + c, b = first + rot/2 + c (half layout) or a = first + 2c, b = a + 1
// (interleaved); the other channels are copied.  The gradient is the same map with -t.
//
// Angles: position * frequency reaches 2^20 radians and more, where fp32 keeps no digit of
// the angle's place in its turn, and from about 2^30 on one rounding of the product to fp64 is as large
// as fp32's own.  So the product keeps its rounding's remainder and 1 / (2 pi) has two fp64 terms; the
// whole turns are taken off the large part exactly, and the rest (about half a turn at most, rounded to
// fp32 relative to itself) goes through sincospif.
//
// HBM streaming: each element is read once and written once.  The angles of a (batch row,
// token, 8 pairs) are computed once by one thread and used for its share of the heads of
// both tensors, so the sin/cos work is 1/(heads) of the elements; the launch gives a thread
// fewer heads when there are too few tokens to fill the GPU.
#pragma once

#include "llsa_common.cuh"

namespace llsa {

constexpr int kRotThreads = 128;

struct RotaryTensor {
  const void* x;
  void* y;               // [B, H, N, D] contiguous
  long long sb, sh, sn;  // strides of x in elements (channels are contiguous)
  int H;
  int x_vec, y_vec;      // rows are 16-byte aligned
};

struct RotaryParams {
  RotaryTensor t[2];
  int tensors;
  int B, N, D, rot, first;
  int interleaved, inverse, pos32;
  const void* positions;   // int64 (int32 with pos32), or null: token n has position n
  long long pos_stride;    // elements between batch rows of positions (0: shared)
  const double* freq;      // [rot / 2] radians per position
  float scale;
  int heads;               // heads of one thread (of each tensor)
};

__device__ __forceinline__ void rotary_angle(const RotaryParams& P, double pos, int c, float& cs, float& sn) {
  constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLow = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
  const double f = __ldg(P.freq + c);
  const double t = __dmul_rn(pos, f), t_low = fma(pos, f, -t);
  const double turns = fma(t, kTurn, -rint(__dmul_rn(t, kTurn))) + fma(t, kTurnLow, t_low * kTurn);
  sincospif(2.0f * (float)turns, &sn, &cs);
  cs *= P.scale;
  sn *= P.inverse ? -P.scale : P.scale;
}

__device__ __forceinline__ double rotary_position(const RotaryParams& P, int b, int n) {
  if (!P.positions) return (double)n;
  const long long i = (long long)b * P.pos_stride + n;
  return P.pos32 ? (double)__ldg(static_cast<const int*>(P.positions) + i)
                 : (double)__ldg(static_cast<const long long*>(P.positions) + i);
}

// 8 consecutive channels (16 or 32 bytes, 16-byte aligned) as they are stored.
template <typename T>
struct RotaryPiece;
template <>
struct RotaryPiece<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <>
struct RotaryPiece<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One thread's rows: heads [h0, h0 + heads) of the first tensor, then of the second.
struct RotaryRows {
  int h0, n0, n;
  __device__ __forceinline__ RotaryRows(const RotaryParams& P) {
    h0 = blockIdx.y * P.heads;
    n0 = max(0, min(P.heads, P.t[0].H - h0));
    n = n0 + (P.tensors > 1 ? max(0, min(P.heads, P.t[1].H - h0)) : 0);
  }
  template <typename T>
  __device__ __forceinline__ void at(const RotaryParams& P, int b, int n_tok, int q, const T*& x, T*& y) const {
    const RotaryTensor& X = P.t[q >= n0];
    const int h = h0 + (q >= n0 ? q - n0 : q);
    x = static_cast<const T*>(X.x) + b * X.sb + n_tok * X.sn + h * X.sh;
    y = static_cast<T*>(X.y) + (((long long)b * X.H + h) * P.N + n_tok) * P.D;
  }
};

// Vector form: first a multiple of 8, rot a multiple of 16, rows 16-byte aligned.  A row is
// D/16 units of two 8-channel pieces: unit u < rot/16 turns 8 pairs (half layout: piece u of
// either half; interleaved: pieces 2u and 2u + 1), the others copy the remaining pieces.
// kRotAhead rows' loads are in flight together, the first ones while the angles are computed.
// (65536 tokens, 6 heads of 64 bf16 channels, q and k, 201 MB: 36.0 us, 5.6 TB/s; 43.5 us with the
// loads after the angles, 45.8 with 4 rows ahead, whose registers leave too few CTAs on an SM.)
constexpr int kRotAhead = 2;

template <typename T>
__global__ void __launch_bounds__(kRotThreads) rotary_vec_kernel(const RotaryParams P) {
  pdl_enter();
  const int units = P.D / 16;
  const long long t = (long long)blockIdx.x * kRotThreads + threadIdx.x;
  if (t >= (long long)P.B * P.N * units) return;
  const int u = (int)(t & (units - 1));  // D / 16 is 4 or 8
  const long long row = t / units;
  const int b = (int)(row / P.N), n = (int)(row - (long long)b * P.N);
  const int turned = P.rot / 16;
  const bool turn = u < turned;
  int c0, c1;  // first channels of the unit's two pieces
  if (turn) {
    c0 = P.first + (P.interleaved ? 16 * u : 8 * u);
    c1 = c0 + (P.interleaved ? 8 : P.rot / 2);
  } else {
    c0 = 16 * (u - turned);
    c1 = c0 + 8;
    if (c0 >= P.first) c0 += P.rot;
    if (c1 >= P.first) c1 += P.rot;
  }
  const RotaryRows rows(P);
  RotaryPiece<T> p[kRotAhead], q[kRotAhead];
  T* y[kRotAhead];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kRotAhead; ++i)
      if (i0 + i < rows.n) {
        const T* x;
        rows.at(P, b, n, i0 + i, x, y[i]);
        p[i].load(x + c0);
        q[i].load(x + c1);
      }
  };
  load(0);
  float cs[8], sn[8];
  if (turn) {
    const double pos = rotary_position(P, b, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) rotary_angle(P, pos, 8 * u + i, cs[i], sn[i]);
  }
#pragma unroll 1
  for (int i0 = 0; i0 < rows.n; i0 += kRotAhead) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int k = 0; k < kRotAhead; ++k) {
      if (i0 + k >= rows.n) break;
      if (turn) {
        float v[8], w[8];
        p[k].get(v);
        q[k].get(w);
        if (P.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = v[2 * i], d = w[2 * i];
            v[2 * i] = a * cs[i] - v[2 * i + 1] * sn[i];
            v[2 * i + 1] = v[2 * i + 1] * cs[i] + a * sn[i];
            w[2 * i] = d * cs[4 + i] - w[2 * i + 1] * sn[4 + i];
            w[2 * i + 1] = w[2 * i + 1] * cs[4 + i] + d * sn[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = v[i];
            v[i] = a * cs[i] - w[i] * sn[i];
            w[i] = w[i] * cs[i] + a * sn[i];
          }
        }
        p[k].set(v);
        q[k].set(w);
      }
      p[k].store(y[k] + c0);
      q[k].store(y[k] + c1);
    }
  }
}

// Any even rot and first, any element alignment.  A CTA takes kAnyRows token rows and goes through its
// heads: a head's rows come into shared memory in 16-byte pieces (element by element where the tensor
// is not aligned to them), the pairs are turned there with angles from a table made once, and the
// rows leave the same way; the next head's pieces are on their way meanwhile.  (65536 tokens, 6 heads
// of 64 bf16 channels, q and k, 46 of them turned from channel 8 on; a thread for each pair, reading
// and writing global memory 2 bytes at a time, took 111 us.)
constexpr int kAnyRows = 32;

template <typename T, int D>
constexpr int rotary_any_smem(int pairs) {
  return kAnyRows * (pairs * 8 + D * (int)sizeof(T) + 4 * 8);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRotThreads) rotary_any_kernel(const RotaryParams P) {
  constexpr int E = 16 / (int)sizeof(T), row_pieces = D / E, pieces = kAnyRows * row_pieces / kRotThreads;
  extern __shared__ float4 any_smem[];
  T* tile = reinterpret_cast<T*>(any_smem);                             // [kAnyRows][D]
  long long* from = reinterpret_cast<long long*>(tile + kAnyRows * D);  // [2][kAnyRows] row offsets of x
  long long* to = from + 2 * kAnyRows;                                  // and of y
  float2* turn = reinterpret_cast<float2*>(to + 2 * kAnyRows);          // [kAnyRows][pairs] cos, sin
  pdl_enter();
  const int tid = threadIdx.x, pairs = P.rot / 2;
  const long long row0 = (long long)blockIdx.x * kAnyRows;
  const int rows = (int)min((long long)kAnyRows, (long long)P.B * P.N - row0);
  const RotaryRows share(P);
  for (int i = tid; i < 2 * rows; i += kRotThreads) {
    const int s = i / rows, r = i - s * rows;
    const RotaryTensor& X = P.t[s];
    const long long b = (row0 + r) / P.N, n = row0 + r - b * P.N;
    from[s * kAnyRows + r] = b * X.sb + n * X.sn;
    to[s * kAnyRows + r] = (b * X.H * P.N + n) * D;
  }
  for (int i = tid; i < rows * pairs; i += kRotThreads) {
    const int r = i / pairs, c = i - r * pairs;
    const long long b = (row0 + r) / P.N;
    rotary_angle(P, rotary_position(P, (int)b, (int)(row0 + r - b * P.N)), c, turn[i].x, turn[i].y);
  }
  __syncthreads();
  auto head = [&](int q) { return share.h0 + (q >= share.n0 ? q - share.n0 : q); };
  float4 held[pieces];  // the next head's pieces
  auto fetch = [&](int q) {
    const int s = q >= share.n0;
    const RotaryTensor& X = P.t[s];
    const T* x = static_cast<const T*>(X.x) + head(q) * X.sh;
#pragma unroll
    for (int k = 0; k < pieces; ++k) {
      const int i = tid + k * kRotThreads, r = i / row_pieces, c = (i % row_pieces) * E;
      if (r >= rows) break;
      const T* src = x + from[s * kAnyRows + r] + c;
      if (X.x_vec) {
        held[k] = *reinterpret_cast<const float4*>(src);
      } else {
        alignas(16) T v[E];  // read back as one float4
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = src[e];
        held[k] = *reinterpret_cast<const float4*>(v);
      }
    }
  };
  if (share.n > 0) fetch(0);
  for (int q = 0; q < share.n; ++q) {
    const int s = q >= share.n0;
    const RotaryTensor& X = P.t[s];
#pragma unroll
    for (int k = 0; k < pieces; ++k) {
      const int i = tid + k * kRotThreads;
      if (i / row_pieces < rows) reinterpret_cast<float4*>(tile)[i] = held[k];
    }
    if (q + 1 < share.n) fetch(q + 1);
    __syncthreads();
    int r = tid / pairs, c = tid - r * pairs;
    const int dr = kRotThreads / pairs, dc = kRotThreads - dr * pairs;
    for (int i = tid; i < rows * pairs; i += kRotThreads) {
      T* u = tile + r * D + P.first + (P.interleaved ? 2 * c : c);
      T* w = u + (P.interleaved ? 1 : pairs);
      const float a = to_f32(*u), d = to_f32(*w);
      const float2 t = turn[i];
      *u = from_f32<T>(a * t.x - d * t.y);
      *w = from_f32<T>(d * t.x + a * t.y);
      r += dr;
      c += dc;
      if (c >= pairs) {
        c -= pairs;
        ++r;
      }
    }
    __syncthreads();
    T* y = static_cast<T*>(X.y) + (long long)head(q) * P.N * D;
#pragma unroll
    for (int k = 0; k < pieces; ++k) {
      const int i = tid + k * kRotThreads, rr = i / row_pieces, cc = (i % row_pieces) * E;
      if (rr >= rows) break;
      T* dst = y + to[s * kAnyRows + rr] + cc;
      const float4 v = reinterpret_cast<const float4*>(tile)[i];
      if (X.y_vec) {
        *reinterpret_cast<float4*>(dst) = v;
      } else {
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int j = 0; j < E; ++j) dst[j] = e[j];
      }
    }
    // (a thread writes the pieces that it then overwrites: no barrier until the next turn)
  }
}

}  // namespace llsa
