// Linear attention with a decay for each head on the tensor cores (tcgen05, bf16 inputs): one
// CTA walks the 128-token chunks of one segment (see linear_common.cuh for the operation).
//
// Per chunk, with the tokens' tiles X, Y, Z [128][D] brought in by TMA and the state M:
//   1. O = X M (M as bf16 in shared memory) and S = X Y^T                      (fp32, TMEM)
//   2. O <- f2 l^{i+1} O;  P = f1 l^{i-j} S where j <= i, else 0, as bf16 into TMEM;
//      Y <- w l^{n-1-j} Y, as two bf16 terms (the value and its rounding's remainder; the
//      second takes X's place)
//   3. O += P Z,  T = Y^T Z                                                    (fp32, TMEM)
//   4. M = l^n M + T in fp32 registers; O goes out as bf16 through X's place and a TMA store.
// Reversed time order mirrors the weights.  The first pass over segments (OUT = false) runs only
// the second half of 2, T and M.
//
// Roundings to bf16: P and the copy of M that X multiplies, which are tensor-core operands (2^-8
// of a term each, like the output's own rounding); the weighted Y would be a third, in the state
// itself, which is why it is split (2^-16).
//
// Weights: l^{i-j} over a 32-column block of P is (l^{i - last column}) (l^{last column - j}), two
// factors of at most 1, so one exponential a row and block serves 32 products and nothing
// overflows for any decay.  The 32 x 32 blocks on the diagonal take l^{i-j} from a table by
// distance; blocks past it are stored as zeros.
//
// Bound: a chunk moves 4 * 128 * D * 2 bytes (2 of them read in the first pass) and the
// tensor work is a quarter of that time, so HBM bounds it as long as the steps above overlap:
// at D = 64 two CTAs share an SM (104 KB of shared memory, 256 TMEM columns each); at D = 128 one
// CTA has two warpgroups that halve the columns (224 KB, 512 columns).
#pragma once

#include "linear_common.cuh"

namespace llsa {

constexpr int kLtChunk = 128;

template <int D, bool OUT>
struct LtCfg {
  static constexpr int G = D / 64;                // warpgroups, and 64-channel sub-tiles of a tile
  static constexpr int compute = 128 * G;
  static constexpr int threads = compute + 64;    // + TMA warp + MMA warp
  static constexpr int ctas_per_sm = D == 64 ? 2 : 1;
  static constexpr int sub = kLtChunk * 128;      // bytes of a sub-tile
  static constexpr int tile = G * sub;
  // a stage is Y, Z (and X); without OUT one more tile holds Y's second term
  static constexpr int stage = (OUT ? 3 : 2) * tile;
  static constexpr int mop = 2 * stage;           // M as bf16 (OUT), or Y's second term
  static constexpr int tab = mop + (OUT ? D * D * 2 : tile);
  static constexpr int bars = tab + (64 + 32) * 4;
  static constexpr int taddr = bars + 8 * 8;
  static constexpr int smem = 1024 + taddr + 16;
  // TMEM columns.  D = 64: P overlays S (a warp's P block jb only covers S columns that the same
  // warp has already read); D = 128: two warps share the lanes, so P has its own columns.
  static constexpr uint32_t col_s = 0, col_o = 128, col_t = OUT ? 128 + D : 0;
  static constexpr uint32_t col_p = D == 64 ? 0 : 384;
  static constexpr uint32_t cols = OUT ? (D == 64 ? 256 : 512) : (D == 64 ? 64 : 128);
};

enum : int { kLtFull = 0, kLtS = 2, kLtP = 3, kLtO = 4, kLtM = 5, kLtOut = 6 };

struct alignas(64) LinearTcParams {
  CUtensorMap map[7];
  LinearParams P;
  int ix[3], iy[3], iz[3], iout[3];  // maps of each problem's streams
};

// Shared-memory operand descriptors, 128-byte swizzle.  K-major: rows of 128 bytes, 8-row groups
// `1024` apart.  MN-major: the 64 contiguous elements are M or N; 8-row groups of K are 1024
// apart, 64-element groups of M or N `lbo` apart.
__device__ __forceinline__ uint64_t lt_desc(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::f16 instruction descriptor: fp32 accumulators, bf16 operands, MN-major flags.
__host__ __device__ constexpr uint32_t lt_idesc(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void lt_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A from TMEM (bf16 pairs, one row a lane).
__device__ __forceinline__ void lt_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void lt_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void lt_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void lt_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void lt_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

#define LT_R8(a, o) "=r"(a[o]), "=r"(a[o + 1]), "=r"(a[o + 2]), "=r"(a[o + 3]), "=r"(a[o + 4]), "=r"(a[o + 5]), "=r"(a[o + 6]), "=r"(a[o + 7])
#define LT_W8(a, o) "r"(a[o]), "r"(a[o + 1]), "r"(a[o + 2]), "r"(a[o + 3]), "r"(a[o + 4]), "r"(a[o + 5]), "r"(a[o + 6]), "r"(a[o + 7])

// 32 columns of this warp's TMEM lanes, one lane a thread; the wait is part of it, so the
// registers hold the values.
__device__ __forceinline__ void lt_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;"
      : LT_R8(r, 0), LT_R8(r, 8), LT_R8(r, 16), LT_R8(r, 24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void lt_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      LT_W8(r, 0), LT_W8(r, 8), LT_W8(r, 16), LT_W8(r, 24)
      : "memory");
}
__device__ __forceinline__ void lt_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      LT_W8(r, 0), LT_W8(r, 8)
      : "memory");
}
__device__ __forceinline__ void lt_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#undef LT_R8
#undef LT_W8

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// Waits for copies or products in flight after another wait has given up (bounded, and without
// the shortcut of mbar_wait that returns at once after a recorded timeout).
__device__ __forceinline__ void lt_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles / 2) return;
}

template <int D, bool OUT>
__global__ void __launch_bounds__(LtCfg<D, OUT>::threads, LtCfg<D, OUT>::ctas_per_sm)
    linear_tc_kernel(const __grid_constant__ LinearTcParams Q) {
  using Cfg = LtCfg<D, OUT>;
  constexpr int G = Cfg::G, C = kLtChunk;
  extern __shared__ uint8_t lt_smem[];
  uint8_t* base = lt_smem + ((1024u - (smem_u32(lt_smem) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(base), bars = sb + Cfg::bars;
  auto bar = [&](int i) { return bars + 8u * i; };
  float* tab = reinterpret_cast<float*>(base + Cfg::tab);  // tab[32 + n] = l^n (0 for n < 0)
  float* colf = tab + 64;                                  // weight of a block's column j at its edge
  uint32_t* taddr = reinterpret_cast<uint32_t*>(base + Cfg::taddr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const LinearParams& P = Q.P;

  const int prob = blockIdx.x % P.nprob;
  const int seg = (blockIdx.x / P.nprob) % P.nseg, bh = blockIdx.x / P.nprob / P.nseg;
  const LinearProblem& R = P.p[prob];
  const int b = bh / P.H, h = bh % P.H;
  const bool rev = R.rev;

  if (threadIdx.x == 0) {
    mbar_init(bar(kLtFull), 1);
    mbar_init(bar(kLtFull + 1), 1);
    mbar_init(bar(kLtS), 1);
    mbar_init(bar(kLtP), Cfg::compute);
    mbar_init(bar(kLtO), 1);
    mbar_init(bar(kLtM), Cfg::compute);
    mbar_init(bar(kLtOut), Cfg::compute);
    mbar_fence_init();
  }
  if (warp == 4 * G + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(taddr)),
                 "r"(Cfg::cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  const float a = linear_decay(P.log_decay, h), a2 = a * kLog2e;
  if (threadIdx.x < 64) {
    const int n = (int)threadIdx.x - 32;
    tab[threadIdx.x] = n < 0 ? 0.0f : exp2f(a2 * (float)n);
  } else if (threadIdx.x < 96) {
    const int j = (int)threadIdx.x - 64;
    colf[j] = exp2f(a2 * (float)(rev ? j : 31 - j));
  }
  lt_fence_before();
  __syncthreads();
  lt_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *taddr;

  const int len = linear_length(P.lengths, b, P.N);
  const int lo = seg * P.seg, top = min(P.N, lo + P.seg), hi = max(lo, min(top, len));
  const int chunks = (hi - lo + C - 1) / C;
  auto chunk_at = [&](int c) { return lo + (rev ? chunks - 1 - c : c) * C; };
  // the state after a chunk is needed by the next one, and after the last one if it is asked for
  auto wants_state = [&](int c) { return c + 1 < chunks || R.state != nullptr; };
  bool ok = true;

  if (warp == 4 * G) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0) {
      auto load = [&](int c, const CUtensorMap* m, int slot) {
        const uint32_t dst = sb + (c & 1) * Cfg::stage + slot * Cfg::tile;
#pragma unroll
        for (int g = 0; g < G; ++g) tma_load_4d(dst + g * Cfg::sub, m, 64 * g, chunk_at(c), h, b, bar(kLtFull + (c & 1)));
      };
      auto load_yz = [&](int c) {
        mbar_expect_tx(bar(kLtFull + (c & 1)), (OUT ? 3 : 2) * Cfg::tile);
        load(c, &Q.map[Q.iy[prob]], 0);
        load(c, &Q.map[Q.iz[prob]], 1);
      };
      int loaded = 0;
      for (; loaded < min(2, chunks); ++loaded) {
        load_yz(loaded);
        if (OUT) load(loaded, &Q.map[Q.ix[prob]], 2);
      }
      for (int c = 0; c < chunks; ++c) {
        if (OUT) {
          // the chunk's products are done and its output is staged in X's place
          ok = mbar_wait(bar(kLtOut), c & 1);
          if (!ok) break;
          const uint32_t src = sb + (c & 1) * Cfg::stage + 2 * Cfg::tile;
#pragma unroll
          for (int g = 0; g < G; ++g) tma_store_3d(&Q.map[Q.iout[prob]], 64 * g, chunk_at(c), bh, src + g * Cfg::sub);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          if (c + 2 < chunks) load_yz(c + 2);
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          if (c + 2 < chunks) {
            load(c + 2, &Q.map[Q.ix[prob]], 2);
            ++loaded;
          }
        } else {
          ok = mbar_wait(bar(kLtO), c & 1);
          if (!ok) break;
          if (c + 2 < chunks) {
            load_yz(c + 2);
            ++loaded;
          }
        }
      }
      if (!ok)  // no copy may be in flight when the CTA ends
        for (int c = max(0, loaded - 2); c < loaded; ++c) lt_drain(bar(kLtFull + (c & 1)), (c >> 1) & 1);
      if (OUT) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  } else if (warp == 4 * G + 1) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t id_s = lt_idesc(128, 128, 0, 0), id_m = lt_idesc(128, D, 0, 1), id_z = lt_idesc(128, D, 0, 1),
                         id_t = lt_idesc(D, D, 1, 1);
      constexpr uint32_t sub = Cfg::sub;
      uint32_t last = 0, last_parity = 0;
      for (int c = 0; c < chunks && ok; ++c) {
        const uint32_t st = sb + (c & 1) * Cfg::stage;
        const uint32_t y = st, z = st + Cfg::tile, x = st + 2 * Cfg::tile, m = sb + Cfg::mop;
        if (OUT) {
          ok = mbar_wait(bar(kLtFull + (c & 1)), (c >> 1) & 1) && mbar_wait(bar(kLtM), c & 1);
          if (!ok) break;
          lt_fence_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * sub + (k & 3) * 32;
            lt_mma(tmem + Cfg::col_s, lt_desc(x + off, 16), lt_desc(y + off, 16), id_s, k > 0);
          }
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * sub + (k & 3) * 32;
            lt_mma(tmem + Cfg::col_o, lt_desc(x + off, 16), lt_desc(m + k * 2048, D * 128), id_m, k > 0);
          }
          lt_commit(bar(kLtS));
          last = bar(kLtS), last_parity = c & 1;
        }
        ok = mbar_wait(bar(kLtP), c & 1);
        if (!ok) break;
        lt_fence_after();
        if (OUT) {
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            lt_mma_ts(tmem + Cfg::col_o, tmem + Cfg::col_p + 8 * k, lt_desc(z + k * 2048, sub), id_z, 1);
        }
        if (wants_state(c)) {
          const uint32_t y2 = OUT ? x : m;
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            lt_mma(tmem + Cfg::col_t, lt_desc(y + k * 2048, sub), lt_desc(z + k * 2048, sub), id_t, k > 0);
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            lt_mma(tmem + Cfg::col_t, lt_desc(y2 + k * 2048, sub), lt_desc(z + k * 2048, sub), id_t, 1);
        }
        lt_commit(bar(kLtO));
        last = bar(kLtO), last_parity = c & 1;
      }
      if (!ok && last) lt_drain(last, last_parity);
    }
  } else {
    // ---------------------------------------------------------------- weights, state, output
    const int quarter = warp & 3, g = warp >> 2;
    const int i = 32 * quarter + lane;                 // token row and TMEM lane
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    // state row of this thread's lane (M = 64 products use 16 lanes of each warp)
    const int sr = D == 64 ? 16 * quarter + (lane & 15) : i;
    const bool holds = D != 64 || lane < 16;
    auto wait = [&](int which, int parity) { ok = __all_sync(0xffffffffu, ok && mbar_wait(bar(which), parity)); };
    float m[64];                                       // columns 64 g .. of state row sr
    {
      const float* init = R.init ? R.init + (P.per_segment ? (long long)bh * P.nseg + seg : bh) * (D * D) : nullptr;
      if (!init) {
#pragma unroll
        for (int e = 0; e < 64; ++e) m[e] = 0.0f;
      } else if (R.transpose) {
#pragma unroll
        for (int e = 0; e < 64; ++e) m[e] = __ldg(init + (64 * g + e) * D + sr);
      } else {
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(init + sr * D + 64 * g + e));
          m[e] = v.x, m[e + 1] = v.y, m[e + 2] = v.z, m[e + 3] = v.w;
        }
      }
    }
    auto store_m = [&]() {  // M's copy for the tensor cores
      if (holds) {
        uint8_t* dst = base + Cfg::mop + g * (D * 128);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(dst + swz(sr, e)) =
              make_uint4(pack_bf16(m[8 * e], m[8 * e + 1]), pack_bf16(m[8 * e + 2], m[8 * e + 3]),
                         pack_bf16(m[8 * e + 4], m[8 * e + 5]), pack_bf16(m[8 * e + 6], m[8 * e + 7]));
      }
    };
    if (OUT) {
      store_m();
      __syncwarp();
      fence_proxy_async();
      lt_arrive(bar(kLtM));
    }
    for (int c = 0; c < chunks && ok; ++c) {
      const int n = min(C, hi - chunk_at(c));
      uint8_t* st = base + (c & 1) * Cfg::stage;
      wait(kLtFull + (c & 1), (c >> 1) & 1);  // this thread rewrites tokens that the copy brought in
      if (OUT) wait(kLtS, c & 1);
      if (!ok) break;
      lt_fence_after();
      if (OUT) {
        const float f = R.f2 * exp2f(a2 * (float)(rev ? max(0, n - 1 - i) : i + 1));
#pragma unroll
        for (int e = 0; e < 64; e += 32) {
          uint32_t r[32];
          lt_ld32(tmem + lanes + Cfg::col_o + 64 * g + e, r);
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * f);
          lt_st32(tmem + lanes + Cfg::col_o + 64 * g + e, r);
        }
#pragma unroll 1
        for (int jb = g * (4 / G); jb < (g + 1) * (4 / G); ++jb) {
          uint32_t p[16];
          const int past = rev ? quarter - jb : jb - quarter;  // > 0: only masked pairs
          if (past > 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = 0u;
          } else {
            uint32_t s[32];
            lt_ld32(tmem + lanes + Cfg::col_s + 32 * jb, s);
            float v[32];
            if (past < 0) {
              const float e = R.f1 * exp2f(a2 * (float)(rev ? 32 * jb - i : i - 32 * jb - 31));
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 w = *reinterpret_cast<const float4*>(colf + j);
                v[j] = __uint_as_float(s[j]) * (w.x * e);
                v[j + 1] = __uint_as_float(s[j + 1]) * (w.y * e);
                v[j + 2] = __uint_as_float(s[j + 2]) * (w.z * e);
                v[j + 3] = __uint_as_float(s[j + 3]) * (w.w * e);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const int dist = rev ? j - lane : lane - j;
                const float w = tab[32 + dist] * R.f1;
                v[j] = dist >= 0 ? __uint_as_float(s[j]) * w : 0.0f;
              }
            }
            if (n < C) {  // columns behind the last token hold anything
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 32 * jb + j < n ? v[j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
          }
          lt_st16(tmem + lanes + Cfg::col_p + 16 * jb, p);
        }
      }
      if (wants_state(c)) {
        const float w = R.w * exp2f(a2 * (float)(rev ? i + 1 : max(0, n - 1 - i)));
        uint8_t* y = st + g * Cfg::sub;
        uint8_t* y2 = (OUT ? st + 2 * Cfg::tile : base + Cfg::mop) + g * Cfg::sub;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint4* at = reinterpret_cast<uint4*>(y + swz(i, e));
          uint4* at2 = reinterpret_cast<uint4*>(y2 + swz(i, e));
          const uint4 v = *at;
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t one[4], two[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float u0 = __uint_as_float(in[k] << 16) * w, u1 = __uint_as_float(in[k] & 0xffff0000u) * w;
            one[k] = pack_bf16(u0, u1);
            two[k] = pack_bf16(u0 - __uint_as_float(one[k] << 16), u1 - __uint_as_float(one[k] & 0xffff0000u));
          }
          const bool in_use = i < n;
          *at = in_use ? make_uint4(one[0], one[1], one[2], one[3]) : make_uint4(0, 0, 0, 0);
          *at2 = in_use ? make_uint4(two[0], two[1], two[2], two[3]) : make_uint4(0, 0, 0, 0);
        }
      }
      if (i >= n) {  // a row behind the last token: its Z must not meet the products' zeros
        uint8_t* z = st + Cfg::tile + g * Cfg::sub;
#pragma unroll
        for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4*>(z + swz(i, e)) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
      if (OUT) lt_wait_st();
      fence_proxy_async();
      lt_fence_before();
      lt_arrive(bar(kLtP));
      wait(kLtO, c & 1);
      if (!ok) break;
      lt_fence_after();
      if (wants_state(c)) {
        // M + M (l^n - 1) rather than l^n M: a factor close to 1 repeated over thousands of
        // chunks would add up its rounding
        const float fall = expm1f(a * (float)n);
#pragma unroll
        for (int e = 0; e < 64; e += 32) {
          uint32_t t[32];
          lt_ld32(tmem + lanes + Cfg::col_t + 64 * g + e, t);
#pragma unroll
          for (int j = 0; j < 32; ++j) m[e + j] = fmaf(m[e + j], fall, m[e + j]) + __uint_as_float(t[j]);
        }
        if (OUT && c + 1 < chunks) store_m();
        __syncwarp();
      }
      if (OUT) {
        uint32_t o[32];
#pragma unroll
        for (int e = 0; e < 64; e += 32) {
          uint32_t r[32];
          lt_ld32(tmem + lanes + Cfg::col_o + 64 * g + e, r);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[e / 2 + j] = i < n ? pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])) : 0u;
        }
        fence_proxy_async();
        lt_fence_before();
        lt_arrive(bar(kLtM));
        uint8_t* dst = st + 2 * Cfg::tile + g * Cfg::sub;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(dst + swz(i, e)) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        fence_proxy_async();
        lt_arrive(bar(kLtOut));
      }
    }
    if (ok && R.state && holds) {
      float* dst = R.state + (OUT ? (long long)bh : (long long)bh * P.nseg + seg) * (D * D) + sr * D + 64 * g;
#pragma unroll
      for (int e = 0; e < 64; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(m[e], m[e + 1], m[e + 2], m[e + 3]);
    }
    if (OUT) {  // rows that take no part, behind the last chunk
      const int z0 = min(top, lo + chunks * C);
      uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(R.out) + ((long long)bh * P.N + z0) * D);
      for (long long e = threadIdx.x; e < (long long)(top - z0) * (D / 8); e += Cfg::compute) out[e] = make_uint4(0, 0, 0, 0);
    }
  }
  __syncthreads();
  if (warp == 4 * G + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Cfg::cols));
}

}  // namespace llsa
