// Rotary positions of one or two [B, H, N, D] tensors (a layer's q and k) in one launch.
//
// Pair c (x_a, x_b) of the rotated channels turns by t = position * frequency[c]:
//   y_a = s (x_a cos t - x_b sin t),  y_b = s (x_b cos t + x_a sin t),
// with a = first + c, b = first + rot/2 + c (half layout) or a = first + 2c, b = a + 1
// (interleaved); the other channels are copied.  The gradient is the same map with -t.
//
// Angles: position * frequency reaches 2^20 radians and more, where fp32 keeps no digit of
// the angle's place in its turn.  The product is formed in fp64 and reduced there to the
// nearest whole turn; the rest (at most half a turn, rounded to fp32 relative to itself)
// goes through sincospif.
//
// HBM streaming: each element is read once and written once.  The angles of a (batch row,
// token, 8 pairs) are computed once by one thread and used for its share of the heads of
// both tensors, so the sin/cos work is 1/(heads) of the elements; the launch gives a thread
// fewer heads when there are too few tokens to fill the GPU.
#pragma once

#include "llsa_common.cuh"

namespace llsa {

constexpr int kRotThreads = 256;

struct RotaryTensor {
  const void* x;
  void* y;               // [B, H, N, D] contiguous
  long long sb, sh, sn;  // strides of x in elements (channels are contiguous)
  int H;
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
  constexpr double kInv2Pi = 0.15915494309189533577;
  double turns = pos * __ldg(P.freq + c) * kInv2Pi;
  turns -= rint(turns);
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

// 8 consecutive channels as fp32 (16 or 32 bytes, 16-byte aligned).
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Vector form: first a multiple of 8, rot a multiple of 16, rows 16-byte aligned.  A row is
// D/16 units of two 8-channel pieces: unit u < rot/16 turns 8 pairs (half layout: piece u of
// either half; interleaved: pieces 2u and 2u + 1), the others copy the remaining pieces.
template <typename T>
__global__ void __launch_bounds__(kRotThreads) rotary_vec_kernel(const RotaryParams P) {
  pdl_enter();
  const int units = P.D / 16;
  const long long t = (long long)blockIdx.x * kRotThreads + threadIdx.x;
  if (t >= (long long)P.B * P.N * units) return;
  const int u = (int)(t % units);
  const long long row = t / units;
  const int n = (int)(row % P.N), b = (int)(row / P.N);
  const int turned = P.rot / 16;
  const bool turn = u < turned;
  int c0, c1;  // first channels of the unit's two pieces
  float cs[8], sn[8];
  if (turn) {
    c0 = P.first + (P.interleaved ? 16 * u : 8 * u);
    c1 = c0 + (P.interleaved ? 8 : P.rot / 2);
    const double pos = rotary_position(P, b, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) rotary_angle(P, pos, 8 * u + i, cs[i], sn[i]);
  } else {
    c0 = 16 * (u - turned);
    c1 = c0 + 8;
    if (c0 >= P.first) c0 += P.rot;
    if (c1 >= P.first) c1 += P.rot;
  }
#pragma unroll 1
  for (int s = 0; s < P.tensors; ++s) {
    const RotaryTensor& X = P.t[s];
    const int h0 = blockIdx.y * P.heads, h1 = min(X.H, h0 + P.heads);
    const T* x = static_cast<const T*>(X.x) + b * X.sb + n * X.sn;
    T* y = static_cast<T*>(X.y) + ((long long)b * X.H * P.N + n) * P.D;
#pragma unroll 2
    for (int h = h0; h < h1; ++h) {
      float p[8], q[8];
      load8<T>(x + h * X.sh + c0, p);
      load8<T>(x + h * X.sh + c1, q);
      if (turn) {
        float a[8], d[8];
        if (P.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[2 * i] = p[2 * i] * cs[i] - p[2 * i + 1] * sn[i];
            a[2 * i + 1] = p[2 * i + 1] * cs[i] + p[2 * i] * sn[i];
            d[2 * i] = q[2 * i] * cs[4 + i] - q[2 * i + 1] * sn[4 + i];
            d[2 * i + 1] = q[2 * i + 1] * cs[4 + i] + q[2 * i] * sn[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = p[i] * cs[i] - q[i] * sn[i];
            d[i] = q[i] * cs[i] + p[i] * sn[i];
          }
        }
        store8<T>(y + (long long)h * P.N * P.D + c0, a);
        store8<T>(y + (long long)h * P.N * P.D + c1, d);
      } else {
        store8<T>(y + (long long)h * P.N * P.D + c0, p);
        store8<T>(y + (long long)h * P.N * P.D + c1, q);
      }
    }
  }
}

// Any even rot and first, any element alignment: one pair, or one copied channel, per thread.
template <typename T>
__global__ void __launch_bounds__(kRotThreads) rotary_pair_kernel(const RotaryParams P) {
  pdl_enter();
  const int pairs = P.rot / 2, units = pairs + (P.D - P.rot);
  const long long t = (long long)blockIdx.x * kRotThreads + threadIdx.x;
  if (t >= (long long)P.B * P.N * units) return;
  const int u = (int)(t % units);
  const long long row = t / units;
  const int n = (int)(row % P.N), b = (int)(row / P.N);
  const bool turn = u < pairs;
  int c0, c1 = 0;
  float cs = 1.0f, sn = 0.0f;
  if (turn) {
    c0 = P.first + (P.interleaved ? 2 * u : u);
    c1 = c0 + (P.interleaved ? 1 : pairs);
    rotary_angle(P, rotary_position(P, b, n), u, cs, sn);
  } else {
    c0 = u - pairs;
    if (c0 >= P.first) c0 += P.rot;
  }
#pragma unroll 1
  for (int s = 0; s < P.tensors; ++s) {
    const RotaryTensor& X = P.t[s];
    const int h0 = blockIdx.y * P.heads, h1 = min(X.H, h0 + P.heads);
    const T* x = static_cast<const T*>(X.x) + b * X.sb + n * X.sn;
    T* y = static_cast<T*>(X.y) + ((long long)b * X.H * P.N + n) * P.D;
#pragma unroll 2
    for (int h = h0; h < h1; ++h) {
      const long long yo = (long long)h * P.N * P.D;
      if (turn) {
        const float p = to_f32(x[h * X.sh + c0]), q = to_f32(x[h * X.sh + c1]);
        y[yo + c0] = from_f32<T>(p * cs - q * sn);
        y[yo + c1] = from_f32<T>(q * cs + p * sn);
      } else {
        y[yo + c0] = x[h * X.sh + c0];
      }
    }
  }
}

}  // namespace llsa
