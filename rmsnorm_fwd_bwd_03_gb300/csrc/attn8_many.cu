// Attention over the 8-bit cache where sequences bring many rows (chunks of prompts, whole
// prompts): bound by the tensor cores, 4 D operations per pair of row and key, beside one
// exponential each.
//
// A block takes 256 rows (new tokens x heads of a group) of one K/V head as two tiles of
// 128, and 128 keys at a time:
//   * eight warps fetch codes, turn them into bf16 (exactly) and lay K and V in shared
//     memory, in the 128-byte swizzle that the tensor cores read;
//   * a thread per tile issues the products (tcgen05): S_t = Q_t K^T into tensor memory, later
//     O_t += P_t V with P_t read from tensor memory;
//   * four warps per tile turn S_t into P_t, a thread per row: no shuffles, and the row's
//     maximum, sum and rescaling stay in its registers.  P_t overwrites S_t.
// A tile's scores come 64 keys at a time into two places in turn: while one step's weights are
// computed, the products of the next step's scores and of the other tile run.  Tensor memory:
// the two tiles' scores, 2 x 64 columns each, and O_0, O_1, 128 columns each: all 512.
// Scores and sums are float32; weights times V's scales are rounded to bf16 (2^-8 at most) for their product:
// with fp16's range small weights would be lost beside large ones.
// Measured, 32 / 8 heads of 128: 2048 tokens over 32768 1.23 ms (870 TFLOP/s), 19 prompts of 32768 tokens
// 1.03 ms (690 TFLOP/s).  The tensor cores are busy 38% of the time, issue slots 54%, the shared-memory data pipe
// (operands of the products, codes, scales) 74%: that and a row's chain of tensor-memory loads, scales and
// exponentials bound a step; begin and end of a unit take 6 us.

#include <atomic>

#include "attn8.cuh"

namespace gbln {

namespace {

constexpr int kTile = 128;              // rows of a tile, keys that are fetched at a time
constexpr int kHalf = kTile / 2;        // keys of a step
constexpr int kManyRows = 2 * kTile;    // rows of a unit
static_assert(kManyRows == kManyUnit, "the joining kernel knows it too");
constexpr int kBegin = 1;               // tiles that a unit's begin counts for (19 prompts of 32768 tokens: 2 the same, 3 1.06 ms)
constexpr int kConvWarps = 8;
constexpr int kConvRows = kTile / kConvWarps / 8;  // keys of a converting thread
constexpr int kManyThreads = 640;      // five groups of four warps: rows twice, conversion twice, products
// Registers of a thread in each group; together what the block is launched with (640 x 96).  A launch with fewer would
// wait forever for the rest, so the host asks what the kernel was compiled to before its first one.
constexpr int kRegsRows = 128, kRegsConv = 72, kRegsMma = 80, kRegsLaunch = 96;
static_assert(2 * kRegsRows + 2 * kRegsConv + kRegsMma <= 5 * kRegsLaunch, "a larger sum would wait forever");

template <int D>
struct ManyShape {
  static constexpr int PLANES = (D + 63) / 64;      // of 64 values: 128 bytes of bf16
  static constexpr int PLANE = kTile * 128;         // bytes
  static constexpr int TILE = PLANES * PLANE;       // 128 rows or keys
  static constexpr int SMEM = 6 * TILE + 1024;      // Q_0, Q_1, two stages of K and of V; alignment
};

// Barriers of a block: K and V per stage, Q and results per tile of rows, scores and weights per tile and place.
enum { kKFull = 0, kKFree = 2, kVFull = 4, kVFree = 6, kQFull = 8, kODone = 10, kSFull = 12, kPFull = 16, kBars = 20 };

struct Shared {
  uint64_t bar[kBars], last[2];
  __align__(16) float scale[2][2][kTile];  // [stage][K times the softmax scale, V][key]
  Part plan;
  // Where the threads of the products and each converting warp are, and each warp of rows (now and next): kept
  // here, they leave the registers to the inner loops.
  Unit now[2 + kConvWarps], rows[8][2];
  uint32_t tmem;
};

// --- tcgen05 ---------------------------------------------------------------
// Shared memory matrix descriptor: 128-byte swizzle, eight rows of 128 bytes 1024 apart; the start and the
// leading offset in the low word, which steps through a tile by bytes / 16.
__device__ __forceinline__ uint64_t smem_desc(uint32_t low) {
  constexpr uint32_t high = (1024 >> 4) | 1u << 14 | 2u << 29;
  return (uint64_t)high << 32 | low;
}
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lead) { return (addr >> 4) | (lead >> 4) << 16; }
// Instruction descriptor: bf16 x bf16 + float32, M = 128, N = n; B with its N values contiguous where `nmajor`.
constexpr uint32_t inst_desc(int n, bool nmajor) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (nmajor ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (uint32_t)(kTile / 16) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
// `bar` completes when all products issued by this thread so far have.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define GBLN_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define GBLN_W8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
// 32 columns of the thread's lane.
__device__ __forceinline__ void tm_ld32(uint32_t (&v)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : GBLN_R8(v, 0), GBLN_R8(v, 8), GBLN_R8(v, 16), GBLN_R8(v, 24)
      : "r"(at));
}
__device__ __forceinline__ void tm_ld16(uint32_t (&v)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : GBLN_R8(v, 0), GBLN_R8(v, 8)
      : "r"(at));
}
// Values on their way from tensor memory have come: the compiler takes none of them before.
#define GBLN_T8(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7])
__device__ __forceinline__ void tm_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : GBLN_T8(v, 0), GBLN_T8(v, 8), GBLN_T8(v, 16), GBLN_T8(v, 24)::"memory");
}
__device__ __forceinline__ void tm_wait_ld(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : GBLN_T8(v, 0), GBLN_T8(v, 8)::"memory");
}
__device__ __forceinline__ void tm_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::GBLN_W8(v, 0), GBLN_W8(v, 8),
      "r"(at)
      : "memory");
}

// 16 bytes that come while other work goes on (zeros, and no read, where off).
__device__ __forceinline__ void cp_async16(uint32_t to, const void* from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// A whole sector: rows of results lie apart, and with half a sector per lane their stores took twice as long.
__device__ __forceinline__ void store_32b(void* to, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), GBLN_W8(v, 0) : "memory");
}

// A value that is not computed ahead of its place: all descriptors of a tile at once spill.
__device__ __forceinline__ uint32_t here(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}

// Bounded wait.  One that runs out (seconds; a legitimate one takes microseconds) is remembered in `late`, and
// the waits after it poll once: the block runs to its end on whatever it finds, all of it in bounds, and reports.
// (Leaving the loops instead put branches around everything that follows a wait.)
constexpr uint32_t kManyPolls = 1u << 20;
__device__ __forceinline__ void wait_for(const Shared& sh, int bar, uint32_t parity, uint32_t& late) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, %3;\n"
      "WAIT_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE_%=;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra WAIT_%=;\n"
      "DONE_%=:\n\t"
      "selp.u32 %0, 0, 1, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(&sh.bar[bar])), "r"(parity), "r"(late ? 1u : kManyPolls)
      : "memory");
  late |= ok;
}

// --- codes -> bf16 in shared memory ------------------------------------------
// Four codes as four bf16 values.  INT8: 0x4300 | (x & 0x7f) is 128 + the low seven bits, 0x4300 | (x & 0x80) is
// 128 or 256: their difference is the code.  E4M3: its exponent and fraction in bf16's places are the value
// times 2^-120 (a NaN code becomes 480: it comes with the scale NaN).
template <int FMT>
__device__ __forceinline__ uint2 codes4_bf16(uint32_t x) {
  uint2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t u, s;
    __nv_bfloat162 v;
    if constexpr (FMT == GBLN_Q8_INT8) {
      const uint32_t w = __byte_perm(x, 0x43u, 0x4140 + 0x0202 * i);
      u = w & 0xff7fff7fu;
      s = w & 0xff80ff80u;
      v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&s));
    } else {
      const uint32_t w = __byte_perm(x, 0u, 0x1404 + 0x2020 * i);
      u = (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u);
      s = 0x7b807b80u;  // 2^120
      v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u), *reinterpret_cast<const __nv_bfloat162*>(&s));
    }
    (i ? r.y : r.x) = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}
// Sixteen codes to the chunks 2 c and 2 c + 1 of row `row` of a plane.
template <int FMT>
__device__ __forceinline__ void store_codes(uint32_t plane, int row, int c, uint4 w) {
  const uint2 a = codes4_bf16<FMT>(w.x), b = codes4_bf16<FMT>(w.y), e = codes4_bf16<FMT>(w.z), f = codes4_bf16<FMT>(w.w);
  const uint32_t at = plane + row * 128;
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + 16 * ((2 * c) ^ (row & 7))), "r"(a.x), "r"(a.y), "r"(b.x), "r"(b.y) : "memory");
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + 16 * ((2 * c + 1) ^ (row & 7))), "r"(e.x), "r"(e.y), "r"(f.x), "r"(f.y) : "memory");
}

// The warps that bring K and V in.  Lane (r, c) = (lane / 4, lane % 4) of warp w has the chunks c, c + 4
// (16 codes each) of keys 16 w + r and 16 w + r + 8: a store instruction's eight lanes at a time hit all banks.
// Each tile's codes are on their way while the tile before is converted.
template <int D, int FMT>
__device__ __forceinline__ void convert(const AttnArgs& A, Shared& sh, uint32_t kv_smem, int w, uint32_t& late) {
  using M = ManyShape<D>;
  constexpr int NP = M::PLANES;
  const int lane = threadIdx.x & 31, c = lane & 3;
  const int row = 8 * kConvRows * w + (lane >> 2);  // + 8 i
  // The cursor runs two tiles ahead: a tile's pages are looked up while the codes of the one before it are on
  // their way and the one before that is converted.
  Unit& u = sh.now[2 + w];
  if (lane == 0) u = sh.plan.u;
  __syncwarp();
  int tile = sh.plan.tile;
  int64_t left = sh.plan.left;  // at the cursor
  int lo = u.lo, hi = u.hi, tiles = u.tiles, hg = u.hg;
  const int32_t* row_of = A.pages + (int64_t)u.b * A.max_pages;
  int page[kConvRows], h = 0;  // of the tile looked up last, as the table has it; place(): -1 no key, -2 outside the cache
  uint32_t off[kConvRows];     // kNoKey until then where there is no key: an entry of the table may be any number
  constexpr uint32_t kNoKey = 0xffffffffu;
  uint4 kr[kConvRows][NP], vr[kConvRows][NP];
  float sc[kConvRows];
  const auto look_up = [&]() {  // the pages of the cursor's tile; the cursor moves on
    if (left <= 0) return;
#pragma unroll
    for (int i = 0; i < kConvRows; ++i) {
      const int j = lo + tile * kTile + row + 8 * i;
      uint32_t q;
      A.page.split((uint32_t)j, q, off[i]);
      page[i] = j < hi ? __ldg(row_of + q) : -1;
      if (j >= hi) off[i] = kNoKey;
    }
    h = hg;
    --left;
    if (++tile == tiles && left > kBegin) {
      left -= kBegin;
      tile = 0;
      __syncwarp();
      if (lane == 0) next_unit<kManyRows, kTile>(A, u);
      __syncwarp();
      lo = u.lo;
      hi = u.hi;
      tiles = u.tiles;
      hg = u.hg;
      row_of = A.pages + (int64_t)u.b * A.max_pages;
    } else if (tile == tiles) {
      left = 0;
    }
  };
  const auto place = [&]() {
#pragma unroll
    for (int i = 0; i < kConvRows; ++i) {
      if (off[i] == kNoKey) {
        off[i] = 0;
      } else if (page[i] < 0 || page[i] >= A.n_pages) {
        page[i] = -2;
        atomicOr(A.err, kErrBadSlot);
      }
    }
  };
  const auto fetch = [&](const Cache& C, uint4 (&r)[kConvRows][NP]) {
#pragma unroll
    for (int i = 0; i < kConvRows; ++i) {
      const uint8_t* src = C.q + C.cq.at(max(page[i], 0), off[i], h) + 16 * c;
#pragma unroll
      for (int p = 0; p < NP; ++p)
        r[i][p] = page[i] >= 0 && 64 * p + 16 * c < D ? ld_stream(src + 64 * p) : make_uint4(0, 0, 0, 0);
    }
  };
  const auto scales = [&]() {  // of K for c = 0, of V for c = 1
#pragma unroll
    for (int i = 0; i < kConvRows; ++i) {
      sc[i] = page[i] == -2 ? __int_as_float(0x7fc00000) : 0.f;
      if (c < 2 && page[i] >= 0) sc[i] = c == 0 ? __ldg(A.K.sc + A.K.cs.at(page[i], off[i], h)) : __ldg(A.V.sc + A.V.cs.at(page[i], off[i], h));
    }
  };
  look_up();
  place();
  fetch(A.K, kr);
  fetch(A.V, vr);
  scales();
  bool more = left > 0;
  look_up();
  for (int64_t n = 0;; ++n) {
    const int st = (int)(n & 1);
    const uint32_t again = (uint32_t)(n >> 1 & 1) ^ 1u;
    wait_for(sh, kKFree + st, again, late);
    __syncwarp();
    const uint32_t ks = kv_smem + st * M::TILE, vs = kv_smem + (2 + st) * M::TILE;
#pragma unroll
    for (int i = 0; i < kConvRows; ++i)
#pragma unroll
      for (int p = 0; p < NP; ++p) store_codes<FMT>(ks + p * M::PLANE, row + 8 * i, c, kr[i][p]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.bar[kKFull + st]);
    if (more) {
      place();
      fetch(A.K, kr);
    }
    wait_for(sh, kVFree + st, again, late);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kConvRows; ++i) {
#pragma unroll
      for (int p = 0; p < NP; ++p) store_codes<FMT>(vs + p * M::PLANE, row + 8 * i, c, vr[i][p]);
      if (c < 2) sh.scale[st][c][row + 8 * i] = c == 0 ? sc[i] * A.scale2 : sc[i];
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.bar[kVFull + st]);
    if (!more) break;
    fetch(A.V, vr);
    scales();
    more = left > 0;
    look_up();
  }
}

// Steps of the block's tiles tile .. tile + nt - 1 of a unit: the last tile may end in its first half.
__device__ __forceinline__ int steps_of(const Unit& u, int tile, int nt) {
  return 2 * nt - (tile + nt == u.tiles && u.hi - u.lo - (u.tiles - 1) * kTile <= kHalf ? 1 : 0);
}

// The thread that issues the products of tile t of rows, one for each tile: neither's waits hold up the other's
// products.  A step's results, then the scores of the step after the next, which take its place.
template <int D>
__device__ __forceinline__ void products(const AttnArgs& A, Shared& sh, uint32_t q_smem, uint32_t kv_smem, int t, uint32_t& late) {
  using M = ManyShape<D>;
  constexpr uint32_t QK = inst_desc(kHalf, false), PV = inst_desc(D, true);
  const uint32_t s_at = sh.tmem + t * kTile, o_at = sh.tmem + 2 * kTile + t * kTile;
  const uint32_t q_low = desc_low(q_smem + t * M::TILE, 16), k_low = desc_low(kv_smem, 16), v_low = desc_low(kv_smem + 2 * M::TILE, M::PLANE);
  Unit& u = sh.now[t];
  u = sh.plan.u;
  int tile = sh.plan.tile;
  int64_t left = sh.plan.left;
  uint32_t n0 = 0;      // tiles of keys before the unit
  uint32_t rs = 0, rp = 0;  // steps whose scores, and whose results, have been issued
  uint32_t units = 0;
  for (;;) {
    const int nt = (int)min((int64_t)(u.tiles - tile), left);
    if (u.r0 + t * kTile < u.r1) {
      const int steps = steps_of(u, tile, nt);
      wait_for(sh, kQFull + t, units & 1, late);
      ++units;
#pragma unroll 1
      for (int j = -2; j < steps; ++j) {
        const uint32_t n = n0 + (j >> 1), st = n & 1, half = j & 1, ns = n + 1, sst = ns & 1;  // step j + 2 is of tile n + 1
        const bool s_on = j + 2 < steps;
        if (j >= 0) {
          if (half == 0) wait_for(sh, kVFull + st, n >> 1 & 1, late);
          const uint32_t b = rp & 1;
          wait_for(sh, kPFull + 2 * t + b, rp >> 1 & 1, late);
          ++rp;
          tc_after();
          const uint32_t v = here(v_low + ((st * M::TILE + half * kHalf * 128) >> 4)), w = here(s_at + b * kHalf);
#pragma unroll
          for (int i = 0; i < kHalf / 16; ++i)  // 16 keys: 16 rows of 128 bytes, 8 columns of weights
            mma_ts(o_at, w + 8 * i, smem_desc(v + (i * 2048 >> 4)), PV, j > 0 || i > 0);
          if (half == 1 || j + 1 == steps) mma_commit(&sh.bar[kVFree + st]);
        }
        if (s_on) {
          if (half == 0) wait_for(sh, kKFull + sst, ns >> 1 & 1, late);
          tc_after();
          const uint32_t b = rs & 1;
          ++rs;
          const uint32_t q = here(q_low), k = here(k_low + ((sst * M::TILE + half * kHalf * 128) >> 4)), d = here(s_at + b * kHalf);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t at = ((i / 4) * M::PLANE + (i % 4) * 32) >> 4;
            mma_ss(d, smem_desc(q + at), smem_desc(k + at), QK, i > 0);
          }
          mma_commit(&sh.bar[kSFull + 2 * t + b]);  // also after the results of step j
          if (half == 1 || j + 3 == steps) mma_commit(&sh.bar[kKFree + sst]);
        } else if (j >= 0) {
          mma_commit(&sh.bar[kODone + t]);  // of the last two steps, which no scores follow
        }
      }
    } else {  // no rows: keep step, so that no barrier gets two phases ahead
      for (int i = 0; i < nt; ++i) {
        const uint32_t n = n0 + i, st = n & 1, ph = n >> 1 & 1;
        wait_for(sh, kKFull + st, ph, late);
        mbar_arrive(&sh.bar[kKFree + st]);
        wait_for(sh, kVFull + st, ph, late);
        mbar_arrive(&sh.bar[kVFree + st]);
      }
    }
    n0 += nt;
    if (!go_on<kManyRows, kTile, kBegin>(A, u, tile, left, nt)) break;
  }
}

// Tile t of a unit's rows on their way into shared memory (zeros behind the last row), each of the tile's warps its own
// 32: eight lanes take a row's 128 bytes, no copy waits for another.
template <int D>
__device__ __forceinline__ void fetch_q(const AttnArgs& A, const Unit& u, int t, uint32_t q_smem, bool q16) {
  using M = ManyShape<D>;
  const int lane = threadIdx.x & 31, c = lane & 7, row0 = 32 * (warp_index() & 3) + (lane >> 3);
  const int r0 = u.r0 + t * kTile, r1 = u.r1, hg = u.hg;
  const bf16* q = (const bf16*)A.q + (int64_t)u.s.q0 * A.ldq + (int64_t)hg * A.G * D + 8 * c;
  const uint32_t to = q_smem + t * M::TILE;
#pragma unroll 4
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 4 * i;
    const bool on = r0 + row < r1;
    uint32_t tok, g;
    A.group.split((uint32_t)(on ? r0 + row : r0), tok, g);
    const bf16* src = q + (int64_t)tok * A.ldq + (int)g * D;
#pragma unroll
    for (int p = 0; p < M::PLANES; ++p) {
      if (64 * p + 8 * c >= D) continue;
      const uint32_t at = to + p * M::PLANE + row * 128 + 16 * (c ^ (row & 7));
      if (q16) {
        cp_async16(at, src + 64 * p, on);
      } else {
        uint32_t v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = on ? reinterpret_cast<const uint16_t*>(src)[64 * p + k] : 0;
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0] | v[1] << 16), "r"(v[2] | v[3] << 16), "r"(v[4] | v[5] << 16),
                     "r"(v[6] | v[7] << 16)
                     : "memory");
      }
    }
  }
}
__device__ __forceinline__ void q_has_come(Shared& sh, int t) {
  cp_wait_all();
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.bar[kQFull + t]);
}

// The largest of a row's scores: 32 columns from key col of the step on, times K's scales, of the keys it sees.
template <bool MASK>
__device__ __forceinline__ float top_of(const uint32_t (&s)[32], const float* ks, int col, int from, int to) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // chains side by side
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 k = *reinterpret_cast<const float4*>(ks + col + i);
    float2 a = mul2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), make_float2(k.x, k.y));
    float2 b = mul2(make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), make_float2(k.z, k.w));
    if constexpr (MASK) {
      if (col + i < from || col + i >= to) a.x = -INFINITY;
      if (col + i + 1 < from || col + i + 1 >= to) a.y = -INFINITY;
      if (col + i + 2 < from || col + i + 2 >= to) b.x = -INFINITY;
      if (col + i + 3 < from || col + i + 3 >= to) b.y = -INFINITY;
    }
    top[0] = fmaxf(top[0], a.x);
    top[1] = fmaxf(top[1], a.y);
    top[2] = fmaxf(top[2], b.x);
    top[3] = fmaxf(top[3], b.y);
  }
  return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}
// Their weights times V's scales, in bf16; sum takes the weights.
template <bool MASK>
__device__ __forceinline__ void weights_of(const uint32_t (&s)[32], const float* ks, const float* vs, int col, int from, int to, float ref, float2& sum,
                                           uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 k = *reinterpret_cast<const float4*>(ks + col + i), v = *reinterpret_cast<const float4*>(vs + col + i);
    float2 a = fma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), make_float2(k.x, k.y), both(-ref));
    float2 b = fma2(make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), make_float2(k.z, k.w), both(-ref));
    a = make_float2(ex2(a.x), ex2(a.y));
    b = make_float2(ex2(b.x), ex2(b.y));
    float2 x = mul2(a, make_float2(v.x, v.y)), y = mul2(b, make_float2(v.z, v.w));
    if constexpr (MASK) {  // whatever the scales of a key that is not seen
      if (col + i < from || col + i >= to) a.x = x.x = 0.f;
      if (col + i + 1 < from || col + i + 1 >= to) a.y = x.y = 0.f;
      if (col + i + 2 < from || col + i + 2 >= to) b.x = y.x = 0.f;
      if (col + i + 3 < from || col + i + 3 >= to) b.y = y.y = 0.f;
    }
    sum = add2(sum, add2(a, b));
    w[i / 2] = pack_bf16x2(x.x, x.y);
    w[i / 2 + 1] = pack_bf16x2(y.x, y.y);
  }
}

// The four warps of tile t of rows.
template <int D>
__device__ __forceinline__ void softmax(const AttnArgs& A, Shared& sh, uint32_t q_smem, int t, bool q16, int o_align, uint32_t& late) {
  const int warp = warp_index() & 3, lane = threadIdx.x & 31, row = 32 * warp + lane;
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  const uint32_t s_at = sh.tmem + t * kTile + lanes, o_at = sh.tmem + 2 * kTile + t * kTile + lanes;
  Unit* own = sh.rows[4 * t + warp];
  int which = 0;
  if (lane == 0) own[0] = sh.plan.u;
  __syncwarp();
  int tile = sh.plan.tile;
  int64_t left = sh.plan.left, num = sh.plan.at;
  uint32_t n = 0, rounds = 0, done = 0;  // tiles of keys, steps and phases of kODone so far
  if (own[0].r0 + t * kTile < own[0].r1) {
    fetch_q<D>(A, own[0], t, q_smem, q16);
    q_has_come(sh, t);
  }
  for (;;) {
    const Unit& u = own[which];
    const int nt = (int)min((int64_t)(u.tiles - tile), left);
    const bool before = tile > 0, behind = tile + nt < u.tiles, has = u.r0 + t * kTile < u.r1;
    // the next unit
    int64_t after = left;
    {
      int first_tile = tile;
      bool ok = false;
      if (lane == 0) {
        own[which ^ 1] = u;
        ok = go_on<kManyRows, kTile, kBegin>(A, own[which ^ 1], first_tile, after, nt);
      }
      after = __shfl_sync(0xffffffffu, (int)ok, 0) ? left - nt - kBegin : 0;
      __syncwarp();
    }
    const Unit& nu = own[which ^ 1];
    if (has) {
      const int r = u.r0 + t * kTile + row, first = u.s.kv - u.s.nq;
      const int pos = first + A.group.by(min(r, u.r1 - 1));
      const int wr = u.r0 + t * kTile + 32 * warp;  // the warp's rows
      const int pos_min = first + A.group.by(min(wr, u.r1 - 1)), pos_max = first + A.group.by(min(wr + 31, u.r1 - 1));
      const int hi = u.hi, key0 = u.lo + tile * kTile;
      float m = -INFINITY;
      float2 sum = make_float2(0.f, 0.f);
      const int steps = steps_of(u, tile, nt);
      for (int i = 0; i < steps; ++i, ++rounds) {
        const uint32_t g = n + (i >> 1), buf = rounds & 1, at = s_at + buf * kHalf;
        const int col0 = (i & 1) * kHalf, j0 = key0 + (i >> 1) * kTile + col0;
        wait_for(sh, kSFull + 2 * t + buf, rounds >> 1 & 1, late);
        if ((i & 1) == 0) wait_for(sh, kVFull + (g & 1), g >> 1 & 1, late);  // the scales
        __syncwarp();
        tc_after();
        const float *ks = sh.scale[g & 1][0] + col0, *vs = sh.scale[g & 1][1] + col0;
        const bool whole = j0 + kHalf <= hi && (!A.causal || j0 + kHalf - 1 <= pos_min) && (A.window <= 0 || j0 > pos_max - A.window);
        const int to = min(A.causal ? min(hi, pos + 1) : hi, j0 + kHalf) - j0, from = A.window > 0 ? pos - A.window + 1 - j0 : 0;
        uint32_t s[2][32];
        tm_ld32(s[0], at);
        tm_ld32(s[1], at + 32);
        tm_wait_ld(s[0]);
        tm_wait_ld(s[1]);
        if (i > 0 && i + 1 == steps) {  // no scores follow: a barrier of its own
          wait_for(sh, kODone + t, done & 1, late);
          __syncwarp();
          ++done;
          tc_after();
        }
        // Weights by the reference that the row has: while their sum stays below 2^10, no key can be far above
        // it, and neither the step's maximum nor a rescaling is needed.  That is the rule; a row that has no
        // reference yet, or whose sum says otherwise (or is not a number), takes the maximum and computes them
        // anew: each row for itself, whatever the others of its warp do.
        float2 part = make_float2(0.f, 0.f);
        const auto weigh = [&]() {
          const float ref = finite_or_zero(m);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[16];
            if (whole) weights_of<false>(s[c], ks, vs, 32 * c, from, to, ref, part, w);
            else weights_of<true>(s[c], ks, vs, 32 * c, from, to, ref, part, w);
            tm_st16(at + 16 * c, w);  // nobody reads them before the arrival below
          }
        };
        bool anew = true;
        if (i > 0) {
          weigh();
          anew = m == -INFINITY || !(part.x + part.y <= 1024.f);
        }
        if (__any_sync(0xffffffffu, anew)) {
          const float top = whole ? fmaxf(top_of<false>(s[0], ks, 0, from, to), top_of<false>(s[1], ks, 32, from, to))
                                  : fmaxf(top_of<true>(s[0], ks, 0, from, to), top_of<true>(s[1], ks, 32, from, to));
          const float up = anew ? fmaxf(m, top) : m, f = anew ? ex2(m - finite_or_zero(up)) : 1.f;
          m = up;
          sum = mul2(sum, both(f));
          if (i > 0) {
            // the results of the step before: the next scores' barrier comes after them
            if (i + 1 < steps) {
              wait_for(sh, kSFull + 2 * t + (buf ^ 1), (rounds + 1) >> 1 & 1, late);
              __syncwarp();
              tc_after();
            }
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tm_ld16(o, o_at + 16 * c);
              tm_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tm_st16(o_at + 16 * c, o);
            }
          }
          part = make_float2(0.f, 0.f);
          tm_wait_st();  // stores to tensor memory keep no order of their own: the first weights lie before the second come
          weigh();
        }
        sum = add2(sum, part);
        tm_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.bar[kPFull + 2 * t + buf]);
      }
      // the next unit's rows (the last scores have been read: the place is free) before this one's results
      const bool next = after > 0 && nu.r0 + t * kTile < nu.r1;
      if (next) fetch_q<D>(A, nu, t, q_smem, q16);
      wait_for(sh, kODone + t, done & 1, late);
      __syncwarp();
      if (next) q_has_come(sh, t);
      ++done;
      tc_after();
      const float l = sum.x + sum.y, inv = l == 0.f ? 0.f : 1.f / l;
      const int tok = A.group.by(r), hq = u.hg * A.G + r - tok * A.G;
      const bool split = before || behind;
      const int64_t at = (int64_t)(2 * blockIdx.x + (before ? 0 : 1)) * kManyRows + t * kTile + row;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t s[32];
        tm_ld32(s, o_at + 32 * c);
        tm_wait_ld(s);
        if (r >= u.r1) {
          // nothing to store
        } else if (split) {
          float4* dst = reinterpret_cast<float4*>(A.part_o + at * D + 32 * c);
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            dst[k / 4] = make_float4(__uint_as_float(s[k]), __uint_as_float(s[k + 1]), __uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]));
        } else {
          bf16* dst = (bf16*)A.out + (int64_t)(u.s.q0 + tok) * A.ldo + (int64_t)hq * D + 32 * c;
#pragma unroll
          for (int k = 0; k < 32; k += 16) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float a = __uint_as_float(s[k + 2 * e]) * inv, b = __uint_as_float(s[k + 2 * e + 1]) * inv;
              w[e] = l == 0.f ? 0u : pack_bf16x2(a, b);
            }
            if (o_align == 32) {
              store_32b(dst + k, w);
            } else if (o_align == 16) {
              reinterpret_cast<uint4*>(dst + k)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(dst + k)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) reinterpret_cast<uint16_t*>(dst + k)[e] = (uint16_t)(w[e / 2] >> 16 * (e & 1));
            }
          }
        }
        __syncwarp();  // the next load is the whole warp's
      }
      if (r < u.r1) {
        if (split) *reinterpret_cast<float2*>(A.part_ml + 2 * at) = make_float2(m, l);
        else if (A.lse) A.lse[(int64_t)(u.s.q0 + tok) * A.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
      tc_before();
    }
    if (t == 0 && behind && !before && row == 0) tell_join(A, u, parts_behind(sh.plan, num + (u.tiles - 1 - tile)));
    if (after <= 0) break;
    if (!has && nu.r0 + t * kTile < nu.r1) {
      fetch_q<D>(A, nu, t, q_smem, q16);
      q_has_come(sh, t);
    }
    n += nt;
    num += nt + kBegin;
    left = after;
    tile = 0;
    __syncwarp();  // all lanes are done with this unit: its place is the next but one's
    which ^= 1;
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kManyThreads, 1) attn8_many(const __grid_constant__ AttnArgs A, bool q16, int o_align) {
  using M = ManyShape<D>;
  extern __shared__ unsigned char many_smem[];
  __shared__ Shared sh;
  launch_dependents();
  const int warp = warp_index();
  const uint32_t q_smem = (smem_addr(many_smem) + 1023u) & ~1023u, kv_smem = q_smem + 2 * M::TILE;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      const bool conv = i < kKFree || (i >= kVFull && i < kVFree);                  // a converting warp each
      const bool rows = (i >= kQFull && i < kODone) || i >= kPFull;  // a warp of the tile each
      const bool free = (i >= kKFree && i < kVFull) || (i >= kVFree && i < kQFull);  // a thread of the products each
      mbar_init(&sh.bar[i], conv ? kConvWarps : rows ? 4 : free ? 2 : 1);
    }
    mbar_init_fence();
    A.info[blockIdx.x * kAttnInfo] = -1;
  }
  if (warp == 0) {
    Part p;
    plan_part<kManyRows, kTile, kBegin>(A, p);
    if ((threadIdx.x & 31) == 0) sh.plan = p;
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (sh.plan.left > 0) {
    uint32_t late = 0;
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
      softmax<D>(A, sh, q_smem, warp >> 2, q16, o_align, late);
    } else if (warp < 8 + kConvWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
      convert<D, FMT>(A, sh, kv_smem, warp - 8, late);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
      const int t = warp - 8 - kConvWarps;
      if (t < 2 && (threadIdx.x & 31) == 0) {
        products<D>(A, sh, q_smem, kv_smem, t, late);
        // all products are complete before the memory is given back, also where waits have run out
        mbar_init(&sh.last[t], 1);
        mbar_init_fence();
        mma_commit(&sh.last[t]);
        mbar_wait(&sh.last[t], 0, kWaitPolls);
      }
    }
    if (late) atomicOr(A.err, kErrWaitTimeout);
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh.tmem) : "memory");
}

template <int D, int FMT>
gbln_status many_go(const AttnArgs& A, int blocks, bool q16, int o_align, cudaStream_t s) {
  using M = ManyShape<D>;
  static std::atomic<uint64_t> ready{0};  // devices whose limit is raised
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GBLN_ERR_CUDA;
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    cudaFuncAttributes is{};
    if (cudaFuncGetAttributes(&is, attn8_many<D, FMT>) != cudaSuccess || is.numRegs < kRegsLaunch ||
        cudaFuncSetAttribute(attn8_many<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, M::SMEM) != cudaSuccess) {
      cudaGetLastError();
      return GBLN_ERR_CUDA;
    }
    ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  attn8_many<D, FMT><<<blocks, kManyThreads, M::SMEM, s>>>(A, q16, o_align);
  return cudaGetLastError() == cudaSuccess ? attn_join_launch(A, blocks, kManyRows, s) : GBLN_ERR_CUDA;
}

template <int FMT>
gbln_status many_typed(const AttnArgs& A, int blocks, bool q16, int o_align, cudaStream_t s) {
  return A.D == 64 ? many_go<64, FMT>(A, blocks, q16, o_align, s) : A.D == 96 ? many_go<96, FMT>(A, blocks, q16, o_align, s) : many_go<128, FMT>(A, blocks, q16, o_align, s);
}

}  // namespace

gbln_status attn_many_launch(const AttnArgs& A, int blocks, int fmt, cudaStream_t s) {
  const bool q16 = aligned16(A.q) && A.ldq % 8 == 0;
  const int o_align = (uintptr_t)A.out % 32 == 0 && A.ldo % 16 == 0 ? 32 : aligned16(A.out) && A.ldo % 8 == 0 ? 16 : 2;
  return fmt == GBLN_Q8_INT8 ? many_typed<GBLN_Q8_INT8>(A, blocks, q16, o_align, s) : many_typed<GBLN_Q8_E4M3>(A, blocks, q16, o_align, s);
}

}  // namespace gbln
