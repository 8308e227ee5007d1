// Linear attention with a decay for each head on the tensor cores (tcgen05, bf16 inputs): one
// CTA walks the 128-token chunks of one segment (see linear_common.cuh for the operation).
//
// Per chunk, with the tokens' tiles X, Y, Z [128][D] brought in by TMA and the state M:
//   1. S = X Y^T and O = X M (M as bf16 in shared memory)                      (fp32, TMEM)
//   2. Y <- w l^{n-1-j} Y, as two bf16 terms (the value and its rounding's remainder; the
//      second takes X's place), then T = Y^T Z                                 (fp32, TMEM)
//      (three terms when the caller gets the state: the third in X's place, the second in that
//      of M's copy, which X M has read by then)
//   3. O <- f2 l^{i+1} O;  P = f1 l^{i-j} S where j <= i, else 0, as bf16 into TMEM, then
//      O += P Z while T is folded into M = l^n M + T (fp32 registers)
//   4. O goes out as bf16 through X's place and a TMA store.
// Reversed time order mirrors the weights.  The first pass over segments (OUT = false) runs
// only 2 and M, with the next chunk's weights applied while this chunk's T is formed.
//
// Roundings to bf16: P and the copy of M that X multiplies, which are tensor-core operands (2^-8
// of a term each, like the output's own rounding); the weighted Y would be a third, in the state
// itself, which is why it is split.  2^-16 is all that outputs can show, behind the rounding of M's
// copy; a state that is returned is fp32, so its tokens have three terms, 2^-24 (2.5e-6 -> 1.3e-7 of
// the state, for 5 to 20 % of the time: B = 8, H = 16, N = 1999, D = 128 71 -> 82 us, B = 32, H = 24,
// N = 2048, D = 64 175 -> 207 us).  At D = 64 two terms are the halves of one M = 128 product (M = 64 runs
// at half rate): lanes 0..63 hold the state's rows from the values, lanes 64..127 those from the
// remainders, both decay alike, X meets them as one 128-row operand, and they are added when the
// state leaves the kernel; with three terms a product of the third and half of the second precedes that
// of the first and half of the second.  At D = 128 they are products into one T.
//
// Weights: l^{i-j} over a 32-column block of P is (l^{i - last column}) (l^{last column - j}), two
// factors of at most 1, so one exponential a row and block serves 32 products and nothing
// overflows for any decay.  The 32 x 32 blocks on the diagonal take l^{i-j} from a table by
// distance, whose other half is 0; blocks past it are stored as zeros.  (So a NaN among a chunk's
// tokens reaches the chunk's other tokens, as through any tile of products.)
//
// Work split: a thread has one token row (a TMEM lane) and 32 of the D columns, so 8 warps at
// D = 64, where two CTAs share an SM (113 KB of shared memory, 256 TMEM columns each), and 16 at
// D = 128 (one CTA, 225 KB, 512 columns): 16 warps an SM either way.
//
// Measured at B = 1, H = 6, N = 65536 (47 segments of 11 chunks at D = 64, 24 of 22 at D = 128):
// first pass 24 us (100 MB, 4.2 TB/s) and 44 us (201 MB, 4.5 TB/s), second pass 45 us (201 MB, 4.5
// TB/s; 0.70 of the copy rate) and 83 us (403 MB, 4.9 TB/s); the three problems of a backward 124 and
// 220 us.  No unit is saturated in the second pass (tensor cores 30 / 43 % active, shared memory 39 / 40 %
// of its wavefronts from the warps and about as many again from the products' operands and the
// copies, issue slots 42 / 39 %): it is bound by the latency of the chain S -> P -> O and W -> T ->
// M -> O of a chunk, which the SM's other CTA (D = 64) or the other warps' phases (D = 128) cover in
// part.  Fewer, busier warps made it slower every time.  Weighting Y into TMEM as the products' first operand
// (no shared-memory writes) doubles the weighting at D = 64 and cost 20 us there.
#pragma once

#include "linear_common.cuh"

namespace llsa {

constexpr int kLtChunk = 128;
constexpr int kLtCols = 32;  // columns of a thread

template <int D, bool OUT>
struct LtCfg {
  static constexpr int G = D / kLtCols;           // threads of a row
  static constexpr int subs = D / 64;             // 64-channel sub-tiles of a tile
  static constexpr int compute = 128 * G;
  static constexpr int threads = compute + 64;    // + TMA warp + MMA warp
  static constexpr int ctas_per_sm = D == 64 ? 2 : 1;
  static constexpr int sub = kLtChunk * 128;      // bytes of a sub-tile
  static constexpr int tile = subs * sub;
  // a stage is Y, Z (and X); without OUT three more tiles hold Y's third terms and, by the chunk's
  // parity, its second ones
  static constexpr int stage = (OUT ? 3 : 2) * tile;
  static constexpr int mop = 2 * stage;           // [128][D] bf16: M (OUT), or Y's third terms
  static constexpr int tab = mop + (OUT ? 1 : 3) * tile;
  static constexpr int bars = tab + (132 + 64) * 4;
  static constexpr int taddr = tab + 130 * 4;     // (pw leaves three of its places free)
  static constexpr int smem = bars + 16 * 8;
  // TMEM columns.  P overlays the S columns of blocks 0 and 1 (both are in registers before
  // either is overwritten).  At D = 128 there are two O, so that a chunk's output leaves while the
  // next chunk's X M runs; at D = 64 the other CTA of the SM fills that time.  Without OUT there
  // are two T.
  static constexpr bool defer = OUT && D == 128;
  static constexpr uint32_t col_s = 0, col_p = 0, col_o = 128, col_t = OUT ? (defer ? 384 : 128 + D) : 0;
  static constexpr uint32_t cols = OUT ? (defer ? 512 : 256) : 2 * D;
};

// Barriers.  A wait is for a phase's parity, so nobody may fall two phases behind: a barrier's next
// phase always needs something that every waiter does after its wait.  Where chunks overlap (the
// first pass weights chunk c + 1 before it folds T of chunk c; the TMA warp runs beside both) that takes
// two of them: kLtY and kLtT by the chunk's parity, kLtFull, kLtFree (a stage's products are done) and
// kLtOut (its output is staged) by stage.  kLtThird (the first pass's third terms are read) needs one: its
// next phase needs every warp's weights, which each applies after its wait.
enum : int {
  kLtS, kLtX, kLtP, kLtO, kLtM, kLtY, kLtT = 7, kLtOut = 9, kLtFree = 11, kLtFull = 13, kLtThird = 15, kLtBars = 16
};

struct alignas(64) LinearTcParams {
  CUtensorMap map[7];
  LinearParams P;
  int ix[3], iy[3], iz[3], iout[3];  // maps of each problem's streams
};

// Shared-memory operand descriptors, 128-byte swizzle.  K-major: rows of 128 bytes, 8-row groups
// `1024` apart.  MN-major: the 64 contiguous elements are M or N; 8-row groups of K are 1024
// apart, 64-element groups of M or N `lbo` apart.
// The upper word is the same for all; the lower one is the address and lbo in 16-byte units, so
// the steps through a tile are additions of constants.
constexpr uint32_t kLtDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t lt_desc(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | (lbo >> 4 << 16); }
__device__ __forceinline__ uint64_t lt_desc64(uint32_t lo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kLtDescHi));
  return d;
}

// One thread of a converged warp.  (The products issued inside `if (lt_elect())` take the uniform
// data path; from a divergent `lane == 0` branch each cost about 100 cycles to issue, more than most take.)
__device__ __forceinline__ bool lt_elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n .reg .b32 r;\n elect.sync r|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}

// kind::f16 instruction descriptor: fp32 accumulators, bf16 operands, MN-major flags.
__host__ __device__ constexpr uint32_t lt_idesc(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void lt_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(lt_desc64(a)), "l"(lt_desc64(b)), "r"(idesc), "r"(acc)
      : "memory");
}
// A from TMEM (bf16 pairs, one row a lane).
__device__ __forceinline__ void lt_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(lt_desc64(b)), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void lt_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void lt_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void lt_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// One arrival for a warp, after all its lanes' writes and fences.
__device__ __forceinline__ void lt_arrive(uint32_t bar) {
  __syncwarp();
  if (lane_id() == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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

// Two fp32 products, or fused multiply-adds, in one instruction.
__device__ __forceinline__ float2 lt_mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 lt_fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 lt_add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 lt_f2(uint32_t lo, uint32_t hi) {
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ float2 lt_bf2(uint32_t v) { return lt_f2(v << 16, v & 0xffff0000u); }

// Barrier of `threads` threads (whole warps) among the CTA's, by number.
__device__ __forceinline__ void lt_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

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

// 227 KB of an SM's 228 are for its CTAs, which each take 1 KB more than they ask for.
static_assert(2 * (LtCfg<64, true>::smem + 1024) <= 228 * 1024 && 2 * (LtCfg<64, false>::smem + 1024) <= 228 * 1024 &&
                  LtCfg<128, true>::smem <= 227 * 1024 && LtCfg<128, false>::smem <= 227 * 1024,
              "shared memory of the CTAs that are to share an SM");

template <int D, bool OUT>
__global__ void __launch_bounds__(LtCfg<D, OUT>::threads, LtCfg<D, OUT>::ctas_per_sm)
    linear_tc_kernel(const __grid_constant__ LinearTcParams Q) {
  using Cfg = LtCfg<D, OUT>;
  constexpr int G = Cfg::G, C = kLtChunk, W = kLtCols;
  extern __shared__ __align__(1024) uint8_t lt_smem[];
  uint8_t* base = lt_smem;
  const uint32_t sb = smem_u32(base), bars = sb + Cfg::bars;
  auto bar = [&](int i) { return bars + 8u * i; };
  // Powers of l, made once: an exponential in the loop costs 20 instructions a thread.
  float* pw = reinterpret_cast<float*>(base + Cfg::tab);  // pw[n] = l^n, 0 <= n <= 128
  // f1 l^distance for the blocks of P: diag[column - row] in a block on the diagonal (0 past it), and
  // edge[column] from a block's column to its edge (the last column, or reversed the first).
  float* near = pw + 132;  // 64 values
  uint32_t* taddr = reinterpret_cast<uint32_t*>(base + Cfg::taddr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const LinearParams& P = Q.P;

  const int prob = blockIdx.x % P.nprob;
  const int seg = (blockIdx.x / P.nprob) % P.nseg, bh = blockIdx.x / P.nprob / P.nseg;
  const LinearProblem& R = P.p[prob];
  const int b = bh / P.H, h = bh % P.H;
  const bool rev = R.rev, exact = R.exact;
  const float *diag = near + (rev ? 32 : 31), *edge = near + (rev ? 32 : 0);

  if (threadIdx.x == 0) {
    if (sb & 1023u) record_error(LLSA_ERR_INTERNAL);  // the swizzle needs 1024-byte alignment
    for (int i = 0; i < kLtBars; ++i) {
      const bool warps = i == kLtP || i == kLtM || i == kLtY || i == kLtY + 1 || i == kLtOut || i == kLtOut + 1;
      mbar_init(bar(i), warps ? Cfg::compute / 32 : 1);
    }
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
  if (threadIdx.x < 129) pw[threadIdx.x] = exp2f(a2 * (float)threadIdx.x);
  if (threadIdx.x >= 192 && threadIdx.x < 256) {
    const int k = (int)threadIdx.x - 192, dist = rev ? k - 32 : 31 - k;
    near[k] = dist < 0 ? 0.0f : R.f1 * exp2f(a2 * (float)dist);
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
        for (int g = 0; g < Cfg::subs; ++g)
          tma_load_4d(dst + g * Cfg::sub, m, 64 * g, chunk_at(c), h, b, bar(kLtFull + (c & 1)));
      };
      auto expect = [&](int c) { mbar_expect_tx(bar(kLtFull + (c & 1)), (OUT ? 3 : 2) * Cfg::tile); };
      int loaded = 0;
      for (; loaded < min(2, chunks); ++loaded) {
        expect(loaded);
        load(loaded, &Q.map[Q.iy[prob]], 0);
        if (OUT) load(loaded, &Q.map[Q.ix[prob]], 2);
        load(loaded, &Q.map[Q.iz[prob]], 1);
      }
      for (int c = 0; c < (OUT ? chunks : chunks - 2); ++c) {
        const bool more = c + 2 < chunks;
        if (more) {  // the chunk's products are done: Y and Z are free
          ok = mbar_wait(bar(kLtFree + (c & 1)), c >> 1 & 1);
          if (!ok) break;
          expect(c + 2);
          ++loaded;
          load(c + 2, &Q.map[Q.iy[prob]], 0);
          load(c + 2, &Q.map[Q.iz[prob]], 1);
        }
        if (OUT) {  // X's place holds the chunk's output
          ok = mbar_wait(bar(kLtOut + (c & 1)), c >> 1 & 1);
          if (!ok) break;
          const uint32_t src = sb + (c & 1) * Cfg::stage + 2 * Cfg::tile;
#pragma unroll
          for (int g = 0; g < Cfg::subs; ++g)
            tma_store_3d(&Q.map[Q.iout[prob]], 64 * g, chunk_at(c), bh, src + g * Cfg::sub);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          if (more) {
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            load(c + 2, &Q.map[Q.ix[prob]], 2);
          }
        }
      }
      if (!ok)  // no copy may be in flight when the CTA ends
        for (int c = max(0, loaded - 2); c < loaded; ++c) lt_drain(bar(kLtFull + (c & 1)), (c >> 1) & 1);
      if (OUT) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  } else if (warp == 4 * G + 1) {
    // ---------------------------------------------------------------- MMA
    constexpr uint32_t id_s = lt_idesc(128, 128, 0, 0), id_o = lt_idesc(128, D, 0, 1), id_t = lt_idesc(128, D, 1, 1);
    constexpr uint32_t sub = Cfg::sub;
    auto wait = [&](int which, int parity) { ok = __all_sync(0xffffffffu, ok && mbar_wait(bar(which), parity)); };
    auto k_major = [](int k) { return (k >> 2) * (sub >> 4) + (k & 3) * 2; };  // 16 channels on, in 16-byte units
    auto mn_major = [](int k) { return k * 128; };                             // 16 rows on
    int last = -1, last_parity = 0;
    for (int c = 0; c < chunks && ok; ++c) {
      const uint32_t y = sb + (c & 1) * Cfg::stage, z = y + Cfg::tile, x = y + 2 * Cfg::tile, m = sb + Cfg::mop;
      const uint32_t o = tmem + Cfg::col_o + (Cfg::defer ? (c & 1) * D : 0);
      wait(kLtFull + (c & 1), c >> 1 & 1);
      if (!ok) break;
      if (OUT) {
        // S needs the last chunk's P read (its O complete); O needs M
        const uint32_t dx = lt_desc(x, 16), dy = lt_desc(y, 16), dm = lt_desc(m, sub);
        if (c > 0) wait(kLtO, (c - 1) & 1);
        if (!ok) break;
        lt_fence_after();
        if (lt_elect()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) lt_mma(tmem + Cfg::col_s, dx + k_major(k), dy + k_major(k), id_s, k > 0);
          lt_commit(bar(kLtS));
        }
        __syncwarp();
        last = kLtS, last_parity = c & 1;
        wait(kLtM, c & 1);
        if (!ok) break;
        lt_fence_after();
        if (lt_elect()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)  // D = 64: X against the rows of both terms
            lt_mma(o, dx + k_major(k & (D / 16 - 1)), dm + mn_major(k), id_o, k > 0);
          lt_commit(bar(kLtX));
        }
        __syncwarp();
        last = kLtX, last_parity = c & 1;
      }
      if (wants_state(c)) {
        wait(kLtY + (c & 1), c >> 1 & 1);
        if (!ok) break;
        lt_fence_after();
        const uint32_t y2 = OUT ? (exact ? m : x) : m + (1 + (c & 1)) * Cfg::tile, y3 = OUT ? x : m;
        const uint32_t t = tmem + Cfg::col_t + (OUT ? 0 : (c & 1) * D);
        if (lt_elect()) {
          const uint32_t dy = lt_desc(y, D == 64 ? y2 - y : sub), dy2 = lt_desc(y2, sub), dz = lt_desc(z, sub);
          if (exact) {  // smallest first: the third terms (D = 64: over the halves of the second ones)
            const uint32_t dy3 = lt_desc(y3, D == 64 ? y2 - y3 : sub);
#pragma unroll
            for (int k = 0; k < C / 16; ++k) lt_mma(t, dy3 + mn_major(k), dz + mn_major(k), id_t, k > 0);
            if (!OUT) lt_commit(bar(kLtThird));
            if (D == 128) {
#pragma unroll
              for (int k = 0; k < C / 16; ++k) lt_mma(t, dy2 + mn_major(k), dz + mn_major(k), id_t, 1);
            }
          }
#pragma unroll
          for (int k = 0; k < C / 16; ++k) lt_mma(t, dy + mn_major(k), dz + mn_major(k), id_t, exact || k > 0);
          if (D == 128 && !exact) {
#pragma unroll
            for (int k = 0; k < C / 16; ++k) lt_mma(t, dy2 + mn_major(k), dz + mn_major(k), id_t, 1);
          }
          lt_commit(bar(kLtT + (c & 1)));
          if (!OUT && c + 2 < chunks) lt_commit(bar(kLtFree + (c & 1)));
        }
        __syncwarp();
        last = kLtT + (c & 1), last_parity = c >> 1 & 1;
      }
      if (OUT) {
        wait(kLtP, c & 1);
        if (!ok) break;
        lt_fence_after();
        if (lt_elect()) {
          const uint32_t dz = lt_desc(z, sub);
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            lt_mma_ts(o, tmem + Cfg::col_p + 8 * k, dz + mn_major(k), id_o, 1);
          lt_commit(bar(kLtO));
          if (c + 2 < chunks) lt_commit(bar(kLtFree + (c & 1)));
        }
        __syncwarp();
        last = kLtO, last_parity = c & 1;
      }
    }
    if (!ok && last >= 0) lt_drain(bar(last), last_parity);
  } else {
    // ---------------------------------------------------------------- weights, state, output
    const int quarter = warp & 3, g = warp >> 2;
    const int i = 32 * quarter + lane;                 // token row, TMEM lane, row of the state's copy
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int sr = i & (D - 1);                        // state row
    const bool first_term = i < D;                     // at D = 64 lanes 64.. hold the second terms' rows
    // this thread's 32 columns in a tile: four 16-byte pieces from `piece` on of sub-tile `tile_off`
    const int tile_off = (W * g / 64) * Cfg::sub, piece = (W * g % 64) / 8;
    auto wait = [&](int which, int parity) { ok = __all_sync(0xffffffffu, ok && mbar_wait(bar(which), parity)); };
    const float fall_chunk = expm1f(a * (float)C);
    float2 m[W / 2];                                   // columns 32 g .. of state row sr
    {
      const float* init = R.init ? R.init + (P.per_segment ? (long long)bh * P.nseg + seg : bh) * (D * D) : nullptr;
#pragma unroll
      for (int e = 0; e < W / 2; ++e) m[e] = make_float2(0.0f, 0.0f);
      if (init && first_term) {
        if (R.transpose) {
#pragma unroll
          for (int e = 0; e < W / 2; ++e)
            m[e] = make_float2(__ldg(init + (W * g + 2 * e) * D + sr), __ldg(init + (W * g + 2 * e + 1) * D + sr));
        } else {
#pragma unroll
          for (int e = 0; e < W / 4; ++e) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(init + sr * D + W * g) + e);
            m[2 * e] = make_float2(v.x, v.y);
            m[2 * e + 1] = make_float2(v.z, v.w);
          }
        }
      }
    }
    auto store_m = [&]() {  // M's copy for the tensor cores
      uint8_t* dst = base + Cfg::mop + tile_off;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<uint4*>(dst + swz(i, piece + e)) =
            make_uint4(pack_bf16(m[4 * e].x, m[4 * e].y), pack_bf16(m[4 * e + 1].x, m[4 * e + 1].y),
                       pack_bf16(m[4 * e + 2].x, m[4 * e + 2].y), pack_bf16(m[4 * e + 3].x, m[4 * e + 3].y));
    };
    // Y's rows weighted, in place and in the other terms' tiles; rows behind the last token are
    // zeroed (with Z's: their contents must not meet a product's zeros)
    auto weight_y = [&](int c, int n) {
      uint8_t* y = base + (c & 1) * Cfg::stage + tile_off;
      uint8_t *x = y + 2 * Cfg::tile, *m_place = base + Cfg::mop + tile_off;
      uint8_t* y2 = OUT ? (exact ? m_place : x) : m_place + (1 + (c & 1)) * Cfg::tile;
      uint8_t* y3 = OUT ? x : m_place;
      if (i >= n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t at = swz(i, piece + e);
          *reinterpret_cast<uint4*>(y + at) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(y2 + at) = make_uint4(0, 0, 0, 0);
          if (exact) *reinterpret_cast<uint4*>(y3 + at) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(y + Cfg::tile + at) = make_uint4(0, 0, 0, 0);
        }
      } else if (wants_state(c)) {
        const float w1 = R.w * pw[rev ? i + 1 : n - 1 - i];
        const float2 w = make_float2(w1, w1), minus = make_float2(-1.0f, -1.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t at = swz(i, piece + e);
          const uint4 v = *reinterpret_cast<const uint4*>(y + at);
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t one[4], two[4];
          if (exact) {
            uint32_t three[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 u = lt_mul2(lt_bf2(in[k]), w);
              one[k] = pack_bf16(u.x, u.y);
              float2 rest = lt_fma2(lt_bf2(one[k]), minus, u);
              // D = 64: both products meet the second terms, so they are halved (exactly)
              const float2 part = D == 64 ? lt_mul2(rest, make_float2(0.5f, 0.5f)) : rest;
              two[k] = pack_bf16(part.x, part.y);
              rest = lt_fma2(lt_bf2(two[k]), D == 64 ? make_float2(-2.0f, -2.0f) : minus, rest);
              three[k] = pack_bf16(rest.x, rest.y);
            }
            *reinterpret_cast<uint4*>(y3 + at) = make_uint4(three[0], three[1], three[2], three[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 u = lt_mul2(lt_bf2(in[k]), w);
              one[k] = pack_bf16(u.x, u.y);
              const float2 rest = lt_fma2(lt_bf2(one[k]), minus, u);
              two[k] = pack_bf16(rest.x, rest.y);
            }
          }
          *reinterpret_cast<uint4*>(y + at) = make_uint4(one[0], one[1], one[2], one[3]);
          *reinterpret_cast<uint4*>(y2 + at) = make_uint4(two[0], two[1], two[2], two[3]);
        }
      }
      fence_proxy_async();
      lt_fence_before();
      lt_arrive(bar(kLtY + (c & 1)));
    };
    // M + M (l^n - 1) + T rather than l^n M + T: a factor close to 1 repeated over thousands of
    // chunks would add up its rounding
    auto fold_t = [&](int c, int n) {
      const float f1 = n == C ? fall_chunk : expm1f(a * (float)n);
      const float2 fall = make_float2(f1, f1);
      uint32_t t[W];
      lt_ld32(tmem + lanes + Cfg::col_t + (OUT ? 0 : (c & 1) * D) + W * g, t);
#pragma unroll
      for (int j = 0; j < W / 2; ++j) m[j] = lt_add2(lt_fma2(m[j], fall, m[j]), lt_f2(t[2 * j], t[2 * j + 1]));
    };
    // 32 columns of P
    auto p_block = [&](int jb, int n, uint32_t (&p)[16]) {
      const int past = rev ? quarter - jb : jb - quarter;  // > 0: only masked pairs
      if (past > 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) p[j] = 0u;
        return;
      }
      uint32_t s[32];
      lt_ld32(tmem + lanes + Cfg::col_s + 32 * jb, s);
      if (past < 0) {
        const float e1 = pw[rev ? 32 * jb - i : i - 32 * jb - 31];
        const float2 e = make_float2(e1, e1);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(edge + j);
          const float2 u = lt_mul2(lt_f2(s[j], s[j + 1]), lt_mul2(make_float2(w.x, w.y), e));
          const float2 v = lt_mul2(lt_f2(s[j + 2], s[j + 3]), lt_mul2(make_float2(w.z, w.w), e));
          s[j] = __float_as_uint(u.x), s[j + 1] = __float_as_uint(u.y);
          s[j + 2] = __float_as_uint(v.x), s[j + 3] = __float_as_uint(v.y);
        }
      } else {
        const float* w = diag - lane;
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j] = __float_as_uint(__uint_as_float(s[j]) * w[j]);
      }
      if (n < C) {  // columns behind the last token hold anything
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j] = 32 * jb + j < n ? s[j] : 0u;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) p[j] = pack_bf16(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
    };
    // A chunk's output, staged in X's place for the TMA warp
    auto write_out = [&](int c) {
      const int n = min(C, hi - chunk_at(c));
      uint32_t r[W], o[16];
      lt_ld32(tmem + lanes + Cfg::col_o + (Cfg::defer ? (c & 1) * D : 0) + W * g, r);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        o[j] = i < n ? pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])) : 0u;
      uint8_t* dst = base + (c & 1) * Cfg::stage + 2 * Cfg::tile + tile_off;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<uint4*>(dst + swz(i, piece + e)) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      fence_proxy_async();
      lt_fence_before();
      lt_arrive(bar(kLtOut + (c & 1)));
    };
    if (OUT) {
      store_m();
      fence_proxy_async();
      lt_arrive(bar(kLtM));
      for (int c = 0; c < chunks; ++c) {
        const int n = min(C, hi - chunk_at(c));
        if (Cfg::defer && c > 0) {
          wait(kLtO, (c - 1) & 1);
          if (!ok) break;
          lt_fence_after();
          write_out(c - 1);
        }
        wait(kLtFull + (c & 1), (c >> 1) & 1);  // this thread rewrites tokens that the copy brought in
        wait(kLtS, c & 1);
        wait(kLtX, c & 1);
        if (!ok) break;
        lt_fence_after();
        weight_y(c, n);
        uint32_t p[16];
        p_block(g, n, p);
        lt_bar(1 + quarter, 32 * G);  // S blocks 0 and 1 are read: P may overlay them
        lt_st16(tmem + lanes + Cfg::col_p + 16 * g, p);
        if (G == 2) {  // blocks 0 and 3 here, 1 and 2 there: at most two unmasked ones each
          p_block(3 - g, n, p);
          lt_st16(tmem + lanes + Cfg::col_p + 16 * (3 - g), p);
        }
        {
          const float f1 = R.f2 * pw[rev ? max(0, n - 1 - i) : i + 1];
          const float2 f = make_float2(f1, f1);
          const uint32_t at = tmem + lanes + Cfg::col_o + (Cfg::defer ? (c & 1) * D : 0) + W * g;
          uint32_t r[W];
          lt_ld32(at, r);
#pragma unroll
          for (int j = 0; j < W; j += 2) {
            const float2 v = lt_mul2(lt_f2(r[j], r[j + 1]), f);
            r[j] = __float_as_uint(v.x);
            r[j + 1] = __float_as_uint(v.y);
          }
          lt_st32(at, r);
        }
        lt_wait_st();
        lt_fence_before();
        lt_arrive(bar(kLtP));
        if (wants_state(c)) {
          wait(kLtT + (c & 1), c >> 1 & 1);
          if (!ok) break;
          lt_fence_after();
          fold_t(c, n);
          if (c + 1 < chunks) store_m();
        }
        if (!Cfg::defer) {
          wait(kLtO, c & 1);
          if (!ok) break;
          lt_fence_after();
          write_out(c);
        }
        fence_proxy_async();
        lt_fence_before();
        lt_arrive(bar(kLtM));
      }
      if (Cfg::defer && ok && chunks > 0) {
        wait(kLtO, (chunks - 1) & 1);
        lt_fence_after();
        if (ok) write_out(chunks - 1);
      }
      // a warp that gave up releases those that it shares its lanes with, whose next wait gives up too
      if (!ok) asm volatile("bar.arrive %0, %1;" ::"r"(1 + quarter), "n"(32 * G) : "memory");
    } else {
      for (int c = 0; c <= chunks; ++c) {
        if (c < chunks) {
          wait(kLtFull + (c & 1), (c >> 1) & 1);
          if (exact && c > 0) wait(kLtThird, (c - 1) & 1);
          if (!ok) break;
          weight_y(c, min(C, hi - chunk_at(c)));
        }
        if (c > 0) {
          wait(kLtT + ((c - 1) & 1), (c - 1) >> 1 & 1);
          if (!ok) break;
          lt_fence_after();
          fold_t(c - 1, min(C, hi - chunk_at(c - 1)));
        }
      }
    }
    if (R.state) {
      float* dst = R.state + (OUT ? (long long)bh : (long long)bh * P.nseg + seg) * (D * D) + sr * D + W * g;
      if (D == 64) {  // the two terms' halves meet in the copy's place, which no product reads now
        float2* other = reinterpret_cast<float2*>(base + Cfg::mop) + W / 2 * g * D + sr;  // [column pair][row]
        lt_bar(5, Cfg::compute);  // (without a chunk nothing else orders the copy's writes before these)
        if (!first_term) {
#pragma unroll
          for (int e = 0; e < W / 2; ++e) other[e * D] = m[e];
        }
        lt_bar(5, Cfg::compute);
        if (first_term) {
#pragma unroll
          for (int e = 0; e < W / 2; ++e) m[e] = make_float2(m[e].x + other[e * D].x, m[e].y + other[e * D].y);
        }
      }
      if (ok && first_term) {
#pragma unroll
        for (int e = 0; e < W / 4; ++e)
          reinterpret_cast<float4*>(dst)[e] = make_float4(m[2 * e].x, m[2 * e].y, m[2 * e + 1].x, m[2 * e + 1].y);
      }
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
