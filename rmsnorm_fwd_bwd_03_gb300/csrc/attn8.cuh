// What the attention kernels over the 8-bit cache share: the arguments, a sequence's
// rows and keys, and the plan by which the blocks of a launch share the work.
#pragma once

#include "cache8.cuh"

namespace gbln {

constexpr int kAttnInfo = 8;        // ints of info per block

constexpr int kManyUnit = 256;  // rows of a unit of the kernel for many rows

// Division of n < 2^31 by a fixed d < 2^31: (n m) >> s.
struct FastDiv {
  uint32_t d, m, s;
  __device__ __forceinline__ void split(uint32_t n, uint32_t& q, uint32_t& r) const {
    q = (uint32_t)(((uint64_t)n * m) >> s);
    r = n - q * d;
  }
  __device__ __forceinline__ int by(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> s); }
};

struct AttnArgs {
  const void* q;
  void* out;
  float* lse;  // may be null
  const int32_t* cu;
  const int32_t* kv;
  const int32_t* pages;  // [B, max_pages]
  int64_t max_pages;
  int64_t ldq, ldo;
  int T, B, Hq, Hk, G, D;
  float scale2;  // scale * log2(e)
  int causal, window;
  int n_pages;
  FastDiv page, group;  // by the slots of a page, by G
  Cache K, V;
  int HB, NHG;     // K/V heads of a block, groups of them
  float* part_o;   // [2 C, HB, rows, D]
  float* part_ml;  // [2 C, HB, rows, 2]
  int* info;       // [C, kAttnInfo]
  unsigned int* err;
};

// One sequence of the batch: its rows start at token q0, the last of its nq new tokens
// stands at position kv - 1.  Lengths outside their bounds are cut to them.
struct Seq {
  int q0, nq, kv;
};
__device__ __forceinline__ Seq seq_at(const AttnArgs& A, int b) {
  Seq s;
  s.q0 = min(max(__ldg(A.cu + b), 0), A.T);
  s.nq = min(max(__ldg(A.cu + b + 1), s.q0), A.T) - s.q0;
  const int64_t most = A.max_pages * (int64_t)A.page.d;
  s.kv = (int)min((int64_t)max(__ldg(A.kv + b), 0), most);
  return s;
}

// The keys [lo, hi) that any of a sequence's rows r0 .. r1 - 1 (row = token * G + head of the group) sees.
__device__ __forceinline__ void keys_of(const AttnArgs& A, const Seq& s, int r0, int r1, int& lo, int& hi) {
  const int first = s.kv - s.nq;
  lo = A.window > 0 ? max(0, first + A.group.by(r0) - A.window + 1) : 0;
  hi = A.causal ? min(s.kv, first + A.group.by(r1 - 1) + 1) : s.kv;
  hi = max(hi, lo);
}

// ---------------------------------------------------------------------------
// The plan.  A unit is one block of MR rows of a sequence's new tokens under one group of
// K/V heads; it takes as many tiles of TK keys as it sees (one at least, so that rows that
// see nothing are written too).  All units' tiles in a row are cut into as many equal
// parts as there are blocks: a long context is shared by many, a short one is a piece of
// one block's work, and no block waits for the longest sequence.  The begin of a unit counts as OV
// more tiles (its rows are fetched, the results before it stored).  Lengths are read on the
// device, so a captured graph follows them.  A unit that a cut divides leaves partial
// results, which a second kernel joins in the order of its parts.
// ---------------------------------------------------------------------------
struct Unit {
  int b, blk, hg;
  Seq s;
  int nblk, r0, r1, lo, hi, tiles;
};

template <int MR, int TK>
__device__ __forceinline__ void unit_range(const AttnArgs& A, Unit& u) {
  u.r0 = u.blk * MR;
  u.r1 = min(u.r0 + MR, u.s.nq * A.G);
  keys_of(A, u.s, u.r0, u.r1, u.lo, u.hi);
  const int lo = MR < kManyUnit ? u.lo & ~15 : u.lo;  // the kernel for few rows begins at multiples of sixteen keys
  u.tiles = max(1, (u.hi - lo + TK - 1) / TK);
}
// The next unit after u; false behind the last.
template <int MR, int TK>
__device__ __forceinline__ bool next_unit(const AttnArgs& A, Unit& u) {
  if (++u.hg < A.NHG) return true;
  u.hg = 0;
  if (++u.blk >= u.nblk) {
    u.blk = 0;
    do {
      if (++u.b >= A.B) return false;
      u.s = seq_at(A, u.b);
      u.nblk = (u.s.nq * A.G + MR - 1) / MR;
    } while (u.nblk == 0);
  }
  unit_range<MR, TK>(A, u);
  return true;
}

__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// One warp walks all row blocks, 32 at a time.  Returns the number of tiles of the whole batch
// (target < 0), or finds the unit that holds number `target` and the tile's number in it (negative:
// one of the OV that its begin counts for).
template <int MR, int TK, int OV>
__device__ __forceinline__ int64_t walk_units(const AttnArgs& A, int64_t target, Unit& u, int& tile) {
  const int lane = threadIdx.x & 31;
  int64_t run = 0;
  for (int b0 = 0; b0 < A.B; b0 += 32) {
    Seq s{0, 0, 0};
    if (b0 + lane < A.B) s = seq_at(A, b0 + lane);
    const int nblk = (s.nq * A.G + MR - 1) / MR;
    const int incl = warp_scan(nblk);
    const int all = __shfl_sync(0xffffffffu, incl, 31);
    for (int i0 = 0; i0 < all; i0 += 32) {
      const int i = i0 + lane;
      int at = 0;  // the sequence (lane) whose blocks hold number i: how many end at or before it
#pragma unroll
      for (int o = 16; o; o >>= 1)
        if (__shfl_sync(0xffffffffu, incl, at + o - 1) <= i) at += o;
      at = min(at, 31);
      Unit x;
      x.b = b0 + at;
      x.s.q0 = __shfl_sync(0xffffffffu, s.q0, at);
      x.s.nq = __shfl_sync(0xffffffffu, s.nq, at);
      x.s.kv = __shfl_sync(0xffffffffu, s.kv, at);
      x.nblk = __shfl_sync(0xffffffffu, nblk, at);
      x.blk = i - (__shfl_sync(0xffffffffu, incl, at) - x.nblk);
      x.hg = 0;
      x.tiles = 0;
      if (i < all) unit_range<MR, TK>(A, x);
      // in 64 bits: a block of rows alone may see 2^26 tiles
      int64_t mine = i < all ? (int64_t)(x.tiles + OV) * A.NHG : 0, sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += t;
      }
      const int64_t end = run + sum;
      if (target >= 0) {
        const unsigned hit = __ballot_sync(0xffffffffu, mine > 0 && target < end);
        if (hit) {
          const int l = __ffs(hit) - 1;
          u.b = __shfl_sync(0xffffffffu, x.b, l);
          u.blk = __shfl_sync(0xffffffffu, x.blk, l);
          u.nblk = __shfl_sync(0xffffffffu, x.nblk, l);
          u.s.q0 = __shfl_sync(0xffffffffu, x.s.q0, l);
          u.s.nq = __shfl_sync(0xffffffffu, x.s.nq, l);
          u.s.kv = __shfl_sync(0xffffffffu, x.s.kv, l);
          const int64_t in = target - (__shfl_sync(0xffffffffu, end, l) - __shfl_sync(0xffffffffu, mine, l));
          unit_range<MR, TK>(A, u);
          u.hg = (int)(in / (u.tiles + OV));
          tile = (int)(in - (int64_t)u.hg * (u.tiles + OV)) - OV;
          return run;
        }
      }
      run = __shfl_sync(0xffffffffu, end, 31);
    }
  }
  return run;
}

// A block's part of the plan: where it begins, and how many tiles are left to it.
struct Part {
  Unit u;
  int tile;
  int64_t at;    // the number of that tile among all
  int64_t left;  // tiles, the begins of further units among them
  int64_t total;
  int blocks;  // that have tiles: not more than there are numbers
};
template <int MR, int TK, int OV>
__device__ __forceinline__ void plan_part(const AttnArgs& A, Part& p) {
  p.total = walk_units<MR, TK, OV>(A, -1, p.u, p.tile);
  p.blocks = (int)min((int64_t)gridDim.x, p.total);
  p.at = p.left = 0;
  if ((int)blockIdx.x >= p.blocks) return;
  p.at = p.total * blockIdx.x / p.blocks;
  p.left = p.total * (blockIdx.x + 1) / p.blocks - p.at;
  walk_units<MR, TK, OV>(A, p.at, p.u, p.tile);
  if (p.tile < 0) {
    p.at -= p.tile;
    p.left += p.tile;
    p.tile = 0;
  }
}
// To the next unit, nt tiles having been done; false where the block's part ends.
template <int MR, int TK, int OV>
__device__ __forceinline__ bool go_on(const AttnArgs& A, Unit& u, int& tile, int64_t& left, int nt) {
  left -= nt + OV;
  tile = 0;
  return left > 0 && next_unit<MR, TK>(A, u);
}
// The blocks behind this one that hold tiles of the unit whose last tile is number `last`.
__device__ __forceinline__ int parts_behind(const Part& p, int64_t last) {
  // the block of number x: the smallest c with total (c + 1) / blocks > x
  int64_t c = ((last + 1) * p.blocks - 1) / p.total;
  while (p.total * (c + 1) / p.blocks <= last) ++c;
  while (c > 0 && p.total * c / p.blocks > last) --c;
  return (int)c - (int)blockIdx.x;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The reference b of ex2(a - b) where nothing has been seen yet (b = -infinity): a = -infinity then gives 0, not NaN.
__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

// What the joining kernel has to know of a unit that began in this block and was divided: the parts in
// the blocks behind, its rows, where its sequence begins, its heads.
__device__ __forceinline__ void tell_join(const AttnArgs& A, const Unit& u, int behind) {
  int* f = A.info + blockIdx.x * kAttnInfo;
  f[1] = u.r1 - u.r0;
  f[2] = u.r0;
  f[3] = u.s.q0;
  f[4] = u.hg;
  f[0] = behind;
}

// Let the kernel that joins the parts come up while this one runs, and wait there for it.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

constexpr int kAttnMaxHeads = 512;  // values of a head

// The kernel for many rows (attn8_many.cu), with the one that joins its parts.
gbln_status attn_many_launch(const AttnArgs& A, int blocks, int fmt, cudaStream_t s);
// Joins the parts of a launch of `blocks` blocks whose units have `rows` rows.
gbln_status attn_join_launch(const AttnArgs& A, int blocks, int rows, cudaStream_t s);

}  // namespace gbln
