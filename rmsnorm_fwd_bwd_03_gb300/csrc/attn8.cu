// Attention of the new tokens of a ragged batch over the paged 8-bit K/V cache.
//
// Operator: "Fast-LLM: 高效大语言模型训练框架", §三 框架结构 (attention with RoPE; heads /
// head_groups for grouped-query attention).  With codes k, v and scales a, b of key j:
//   s_j = scale a_j (q . k_j),   o = sum_j p_j b_j v_j / sum_j p_j,   p_j = 2^(s_j log2 e - m).
// INT8 and E4M3 codes are exact in fp16 and in bf16, so the products see the codes themselves:
// a_j goes onto the score, b_j onto the weight p_j, which is rounded to 16 bits for its product;
// scores, weights' sums and results are float32.  A row that sees a key of scale NaN is NaN; a
// key that it does not see has no part in it.
//
// Few rows per sequence (decode, drafts): bound by the cache's bytes, D + 4 per K or V head
// of a token.  A warp takes 8 or 16 rows (new tokens x heads of a group) of one K/V head and
// streams its keys, 16 at a time, through a ring in shared memory of its own, without any
// barrier between warps.  Keys are the 16 rows and queries the 8 columns of the 16 x 8 x 16
// products (S^T = K Q^T, O^T = V^T P^T): a decode step's few rows then waste little of them.
// Codes go straight from the ring into the fragments.  What bounds the kernel beside the memory
// are the integer instructions that turn codes into 16-bit values (in bf16, six for four codes,
// they kept that pipe busy at 45% of the memory's rate); in fp16 three are enough:
//   * INT8: (x & 0x00ff00ff) ^ 0x64806480 is 1152 + code of bytes 0 and 2, x >> 8 gives 1 and 3;
//   * E4M3: the conversion of two codes at a time.
// So the order of D within a product of Q and K is that of the bytes (Q is arranged to fit), V
// comes out of shared memory transposed, four keys to a word, and the rows of the scores are the
// keys in the order in which those words give them.  fp16's range: a row of Q is scaled by a
// power of two (exact) to below 2^15; a weight is at most 4 (the row's reference follows its
// maximum) and stands relative to R, a power of two above V's scales of the keys that the row has
// seen so far, times 2^13: it keeps 11 bits down to 2^-27 of R, half a step of what is below is 2^-38 of R.
// Every row has an R of its own: with one for the warp a scale that only a neighbour sees took bits from its weights.
// Measured: 64 sequences, 524288 cached tokens of 8 heads of 128, INT8 211 us (78% of the copy rate), E4M3
// 185 us (88%).

#include <cuda_fp16.h>

#include <atomic>

#include "attn8.cuh"

namespace gbln {

namespace {

constexpr int kStep = 16;  // keys of a warp's step
constexpr int kFewBegin = 4;  // tiles that a unit's begin counts for

// NT: columns of eight rows.  One leaves room for sixteen warps, two for eight.
template <int D, int NT>
struct FewShape {
  static constexpr int ROWS = 8 * NT;
  static constexpr int WARPS = NT == 1 && D <= 128 ? 16 : 8;
  static constexpr int STAGE = 2 * kStep * D + 2 * kStep * 4;  // K, V, their scales
  static constexpr int NS = (WARPS == 16 ? (D <= 64 ? 6 : D <= 96 ? 4 : 3) : (D <= 64 ? 8 : D <= 96 ? 7 : D <= 128 ? 6 : 3));
  static constexpr int WARP = NS * STAGE;  // holds a warp's results (ROWS x (D + 2) floats) at a unit's end
  static constexpr int SMEM = WARPS * WARP;
  static_assert(WARP >= ROWS * (D + 2) * 4 && SMEM <= 227 * 1024 - 512, "results fit the ring, the ring the SM");
  // Where chunk ch (16 bytes) of row r lies: the lanes that read at once hit different banks.  K is read 8 bytes a
  // lane, four lanes to each of the rows that key_row gives for four lane groups; V 16 bytes of eight rows at a time.
  template <int FMT>
  static __device__ __forceinline__ int k_at(int r, int ch) {
    const int x = FMT == GBLN_Q8_INT8 ? r >> 1 & 3 : (r & 1) | (r >> 1 & 2);
    if constexpr (D % 128 == 0) return r * D + 16 * (ch ^ (x << 1));
    else if constexpr (D == 64) return r * D + 16 * (ch ^ ((x >> 1) << 1));
    else return r * D + 16 * ch;
  }
  static __device__ __forceinline__ int v_at(int r, int ch) {
    if constexpr (D % 128 == 0) return r * D + 16 * (ch ^ (r & 7));
    else if constexpr (D == 64) return r * D + 16 * (ch ^ (r >> 1 & 3));
    else return r * D + 16 * ch;
  }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
// Four codes as two pairs of fp16 values: INT8 bytes (0, 2) and (1, 3), E4M3 bytes (0, 1) and (2, 3).
template <int FMT>
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t& a, uint32_t& b) {
  if constexpr (FMT == GBLN_Q8_INT8) {
    const __half2 k = __half2half2(__ushort_as_half(0x6480));  // 1152
    const uint32_t u = (x & 0x00ff00ffu) ^ 0x64806480u, v = ((x >> 8) & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&u), k), q = __hsub2(*reinterpret_cast<const __half2*>(&v), k);
    a = *reinterpret_cast<const uint32_t*>(&p);
    b = *reinterpret_cast<const uint32_t*>(&q);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(a), "=r"(b) : "r"(x));
  }
}
// The key of a step that row g (half 0) or g + 8 (half 1) of the scores stands for: the pairs above, of a word that
// holds keys 4 c .. 4 c + 3, are then the keys that a lane's weights have after their transposition.
template <int FMT>
__device__ __forceinline__ int key_row(int g, int half) {
  return FMT == GBLN_Q8_INT8 ? 2 * g + half : 4 * (g >> 1) + (g & 1) + 2 * half;
}
// NaN codes of E4M3 as zeros.
__device__ __forceinline__ uint32_t without_nan(uint32_t x) { return x & ~__vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu); }

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two 16 x 16 matrices of bytes, transposed: lane (g, c) gets columns g (words 0, 2) and g + 8 (1, 3), rows 4 c .. 4 c + 3.
// Lanes 0 .. 15 give the rows of the first, 16 .. 31 of the second.
__device__ __forceinline__ void ldm_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// P^T's fragment out of P's: an 8 x 8 matrix of 16-bit values transposed across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// 1 / x of a power of two from 2^-126 to 2^126.
__device__ __forceinline__ float power_inverse(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }
__device__ __forceinline__ float lds_f(uint32_t a) {
  float r;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(a));
  return r;
}

// The page and slot of key j of sequence b; -1: no key, -2: a page outside the cache.
struct KeyAt {
  int page;
  uint32_t off;
};
__device__ __forceinline__ KeyAt key_at(const AttnArgs& A, int b, int j, int lo, int hi) {
  KeyAt k{-1, 0};
  if (j >= lo && j < hi) {
    uint32_t p;
    A.page.split((uint32_t)j, p, k.off);
    k.page = __ldg(A.pages + (int64_t)b * A.max_pages + p);
    if (k.page < 0 || k.page >= A.n_pages) k.page = -2;
  }
  return k;
}

// A step's sixteen keys into a stage.  Where pages are multiples of sixteen slots the step lies in one page
// (ONE: k is the place of its first key that is seen, the same in all lanes, off of key 0); else k is the
// place of key (lane & 15).
template <int D, int FMT, int NT, bool ONE>
__device__ __forceinline__ void few_load(const AttnArgs& A, uint32_t stage, const KeyAt& k, int h, int j0, int lo, int hi) {
  using Sh = FewShape<D, NT>;
  const int lane = threadIdx.x & 31;
  constexpr int CH = D / 16;                 // chunks of a row
  constexpr int N = (kStep * CH + 31) / 32;  // of K (and of V) per lane
  static_assert(kStep * CH % 32 == 0, "whole passes");
  const bool there = k.page >= 0;
  const int64_t p = there ? k.page : 0, o = there ? k.off : 0;
  // lanes 0..15 K's scales, 16..31 V's
  const uint32_t at = stage + 2 * kStep * D + 4 * lane;
  const int key = lane & 15;
  const bool seen = !ONE || (j0 + key >= lo && j0 + key < hi);
  const int64_t so = ONE ? o + key : o;
  const float* src = lane < 16 ? A.K.sc + A.K.cs.at(p, so, h) : A.V.sc + A.V.cs.at(p, so, h);
  if (k.page == -2) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(0x7fc00000) : "memory");
  else cp4(at, src, there && seen);
  if constexpr (ONE) {
    const uint8_t *kq = A.K.q + A.K.cq.at(p, o, h), *vq = A.V.q + A.V.cq.at(p, o, h);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = i * 32 + lane, r = x / CH, ch = x - r * CH;
      const bool on = there && j0 + r >= lo && j0 + r < hi;
      cp16(stage + Sh::template k_at<FMT>(r, ch), kq + r * A.K.cq.slot + 16 * ch, on);
      cp16(stage + kStep * D + Sh::v_at(r, ch), vq + r * A.V.cq.slot + 16 * ch, on);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = i * 32 + lane, r = x / CH, ch = x - r * CH;
      const int page = __shfl_sync(0xffffffffu, k.page, r);
      const uint32_t off = __shfl_sync(0xffffffffu, k.off, r);
      const bool on = page >= 0;
      cp16(stage + Sh::template k_at<FMT>(r, ch), A.K.q + A.K.cq.at(on ? page : 0, on ? off : 0, h) + 16 * ch, on);
      cp16(stage + kStep * D + Sh::v_at(r, ch), A.V.q + A.V.cq.at(on ? page : 0, on ? off : 0, h) + 16 * ch, on);
    }
  }
}

// The plan's calls, S slices of the keys to a tile.
template <int ROWS>
__device__ __forceinline__ void few_plan(const AttnArgs& A, int S, Part& p) {
  switch (S) {
    case 16: plan_part<ROWS, 16 * kStep, kFewBegin>(A, p); break;
    case 8: plan_part<ROWS, 8 * kStep, kFewBegin>(A, p); break;
    case 4: plan_part<ROWS, 4 * kStep, kFewBegin>(A, p); break;
    case 2: plan_part<ROWS, 2 * kStep, kFewBegin>(A, p); break;
    default: plan_part<ROWS, kStep, kFewBegin>(A, p);
  }
}
template <int ROWS>
__device__ __forceinline__ bool few_go_on(const AttnArgs& A, int S, Unit& u, int& tile, int64_t& left, int nt) {
  switch (S) {
    case 16: return go_on<ROWS, 16 * kStep, kFewBegin>(A, u, tile, left, nt);
    case 8: return go_on<ROWS, 8 * kStep, kFewBegin>(A, u, tile, left, nt);
    case 4: return go_on<ROWS, 4 * kStep, kFewBegin>(A, u, tile, left, nt);
    case 2: return go_on<ROWS, 2 * kStep, kFewBegin>(A, u, tile, left, nt);
    default: return go_on<ROWS, kStep, kFewBegin>(A, u, tile, left, nt);
  }
}

template <int D, int FMT, int NT, bool ONE>
__global__ void __launch_bounds__(32 * FewShape<D, NT>::WARPS, 1) attn8_few(const __grid_constant__ AttnArgs A, bool q16) {
  using Sh = FewShape<D, NT>;
  constexpr int ROWS = Sh::ROWS, W = D / 32;  // words of a lane's slice of a key
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ Part plan;
  launch_dependents();
  const int lane = threadIdx.x & 31, warp = warp_index();
  const int g = lane >> 2, c = lane & 3;
  // warp -> K/V head of the block's group and slice of the keys
  const int S = Sh::WARPS / A.HB;
  const int wh = warp % A.HB, slice = warp / A.HB;
  if (warp == 0) {
    Part p;
    few_plan<ROWS>(A, S, p);
    if (lane == 0) plan = p;
  }
  __syncthreads();
  Unit u = plan.u;
  int tile = plan.tile;
  int64_t left = plan.left, num = plan.at;
  if (threadIdx.x == 0) A.info[blockIdx.x * kAttnInfo] = -1;
  if (left <= 0) return;
  const uint32_t mine = smem_addr(ring) + warp * Sh::WARP;
  float* res = reinterpret_cast<float*>(ring) + warp * (Sh::WARP / 4);

  for (;;) {
    const int t1 = (int)min((int64_t)u.tiles, tile + left);  // this block's tiles of the unit: tile .. t1 - 1
    const int h = u.hg * A.HB + wh;
    const bool on = h < A.Hk;
    const int nrows = u.r1 - u.r0;
    float m[NT][2], l[NT][2], o[NT][D / 16][4];
    float U[NT][2];  // 2^13 / R of each row, R a power of two above the scales of V that it has seen
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      U[n][0] = U[n][1] = 0x1p113f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    }
    if (on) {
      const int first = u.s.kv - u.s.nq;  // position of the sequence's first new token
      const int pos_min = first + A.group.by(u.r0), pos_max = first + A.group.by(u.r1 - 1);
      const int lo = u.lo, hi = u.hi;
      // steps begin at multiples of sixteen keys, which pages of such a size hold whole
      const int begin = (lo & ~(kStep - 1)) + slice * kStep;
      const auto base = [&](int t) { return begin + t * S * kStep; };
      const auto where = [&](int t) {
        const int j = base(t);
        if (t >= t1) return KeyAt{-1, 0};
        if constexpr (ONE) {
          KeyAt k = key_at(A, u.b, max(j, lo), lo, hi);
          k.off -= (uint32_t)(max(j, lo) - j);  // of the step's key 0
          return k;
        } else {
          return key_at(A, u.b, j + (lane & 15), lo, hi);
        }
      };
      // fill the ring
      KeyAt next = where(tile);
#pragma unroll
      for (int i = 0; i < Sh::NS - 1; ++i) {
        if (tile + i < t1) {
          const KeyAt k = next;
          next = where(tile + i + 1);
          if (k.page == -2) atomicOr(A.err, kErrBadSlot);
          few_load<D, FMT, NT, ONE>(A, mine + i * Sh::STAGE, k, h, base(tile + i), lo, hi);
        }
        cp_commit();
      }
      // Q^T: rows g + 8 n, values 32 i + 8 c .., times a power of two, in the codes' order
      uint32_t qb[NT][W][4];
      int pos[NT][2];
      float back[NT][2];  // the softmax scale and what undoes that power, of rows 2 c and 2 c + 1
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = min(u.r0 + g + 8 * n, u.r1 - 1), tok = A.group.by(r), hq = h * A.G + r - tok * A.G;
        const bf16* src = (const bf16*)A.q + (u.s.q0 + tok) * A.ldq + (int64_t)hq * D + 8 * c;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          if (q16) {
            const uint4 w = ld_reuse(src + 32 * i);
            qb[n][i][0] = w.x;
            qb[n][i][1] = w.y;
            qb[n][i][2] = w.z;
            qb[n][i][3] = w.w;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              qb[n][i][k] = reinterpret_cast<const uint16_t*>(src)[32 * i + 2 * k] | (uint32_t) reinterpret_cast<const uint16_t*>(src)[32 * i + 2 * k + 1] << 16;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, max(abs_bits(bf16_lo(qb[n][i][k])), abs_bits(bf16_hi(qb[n][i][k]))));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(14 - e) for a largest value of 2^e ..; 1 for a row of zeros, or one that is not finite anyway
        const int e = top == 0 || top >= kInfBits ? 14 : max((int)(top >> 23) - 127, -100);
        const float by = __uint_as_float((uint32_t)(127 + 14 - e) << 23), undo = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const float v[4] = {bf16_lo(qb[n][i][k]) * by, bf16_hi(qb[n][i][k]) * by, bf16_lo(qb[n][i][k + 1]) * by, bf16_hi(qb[n][i][k + 1]) * by};
            qb[n][i][k] = FMT == GBLN_Q8_INT8 ? pack_f16x2(v[0], v[2]) : pack_f16x2(v[0], v[1]);
            qb[n][i][k + 1] = FMT == GBLN_Q8_INT8 ? pack_f16x2(v[1], v[3]) : pack_f16x2(v[2], v[3]);
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          pos[n][k] = first + A.group.by(min(u.r0 + 8 * n + 2 * c + k, u.r1 - 1));
          back[n][k] = __shfl_sync(0xffffffffu, undo, 4 * (2 * c + k)) * A.scale2;
        }
      }
      const int key0 = key_row<FMT>(g, 0), key1 = key_row<FMT>(g, 1);
      int stage = 0;
#pragma unroll 1
      for (int t = tile; t < t1; ++t) {
        cp_wait<Sh::NS - 2>();
        __syncwarp();  // all lanes' copies have landed, all lanes are done with the stage that is filled next
        {
          const int f = t + Sh::NS - 1;
          if (f < t1) {
            const KeyAt k = next;
            next = where(f + 1);
            if (k.page == -2) atomicOr(A.err, kErrBadSlot);
            few_load<D, FMT, NT, ONE>(A, mine + (stage == 0 ? Sh::NS - 1 : stage - 1) * Sh::STAGE, k, h, base(f), lo, hi);
          }
          cp_commit();
        }
        const uint32_t st = mine + stage * Sh::STAGE;
        stage = stage + 1 == Sh::NS ? 0 : stage + 1;
        // scores: keys key0 and key1, rows 2 c and 2 c + 1
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const uint2 x = lds8(st + Sh::template k_at<FMT>(key0, 2 * i + (c >> 1)) + 8 * (c & 1));
          const uint2 y = lds8(st + Sh::template k_at<FMT>(key1, 2 * i + (c >> 1)) + 8 * (c & 1));
          uint32_t a0[4], a1[4];
          codes_f16<FMT>(x.x, a0[0], a0[2]);
          codes_f16<FMT>(y.x, a0[1], a0[3]);
          codes_f16<FMT>(x.y, a1[0], a1[2]);
          codes_f16<FMT>(y.y, a1[1], a1[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816(s[n], a0, qb[n][i][0], qb[n][i][1]);
            mma16816(s[n], a1, qb[n][i][2], qb[n][i][3]);
          }
        }
        const int j0 = base(t);
        const uint32_t sc = st + 2 * kStep * D;
        const float ks[2] = {lds_f(sc + 4 * key0), lds_f(sc + 4 * key1)}, vs[2] = {lds_f(sc + 64 + 4 * key0), lds_f(sc + 64 + 4 * key1)};
        const bool whole = j0 + kStep <= hi && (!A.causal || j0 + kStep - 1 <= pos_min) && (A.window <= 0 || j0 > pos_max - A.window);
        unsigned hide = 0;
        float top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = s[n][e] * ks[e >> 1] * back[n][e & 1];
          if (!whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = j0 + (e >> 1 ? key1 : key0), p = pos[n][e & 1];
              const bool seen = j < hi && (!A.causal || j <= p) && (A.window <= 0 || j > p - A.window);
              if (!seen) {
                s[n][e] = -INFINITY;
                hide |= 1u << (4 * n + e);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
            top[n][e] = x;
          }
        }
        // The reference of a row's weights follows its maximum only when that has grown by more than 2^2, R V's
        // scales when one is above it: weights have room for it, and the results are seldom rescaled.  A scale that is
        // above R brings the warp here also where no row sees its key; each row then goes by the keys that it sees.
        float vu[NT][4];
        bool up = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            vu[n][e] = vs[e >> 1] * U[n][e & 1];
            up = up || fabsf(vu[n][e]) > 8192.f;
          }
          up = up || top[n][0] > m[n][0] + 2.f || top[n][1] > m[n][1] + 2.f;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = hide & (1u << (4 * n + e)) ? 0.f : fabsf(vs[0]);
              v = fmaxf(v, hide & (1u << (4 * n + 2 + e)) ? 0.f : fabsf(vs[1]));
#pragma unroll
              for (int k = 4; k < 32; k <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
              const uint32_t r = (__float_as_uint(fminf(v, 0x1p120f)) & 0x7f800000u) + 0x00800000u;  // the power of two above v
              const float unit = fminf(U[n][e], power_inverse(__uint_as_float(r)) * 8192.f);
              const bool mv = top[n][e] > m[n][e] + 2.f;  // each row for itself
              const float to = mv ? top[n][e] : m[n][e], f = mv ? ex2(m[n][e] - to) : 1.f, fr = f * (unit * power_inverse(U[n][e]));
              U[n][e] = unit;
              vu[n][e] = vs[0] * unit;
              vu[n][e + 2] = vs[1] * unit;
              m[n][e] = to;
              l[n][e] *= f;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[n][i][e] *= fr;
                o[n][i][e + 2] *= fr;
              }
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // keys key0, key1
            const float p0 = ex2(s[n][2 * k] - finite_or_zero(m[n][0])), p1 = ex2(s[n][2 * k + 1] - finite_or_zero(m[n][1]));
            l[n][0] += p0;
            l[n][1] += p1;
            float w0 = p0 * vu[n][2 * k], w1 = p1 * vu[n][2 * k + 1];
            if (hide & (1u << (4 * n + 2 * k))) w0 = 0.f;  // whatever the scale of a key that is not seen
            if (hide & (1u << (4 * n + 2 * k + 1))) w1 = 0.f;
            pb[n][k] = transposed(pack_f16x2(w0, w1));
          }
        // results: values 16 i + g and + 8, rows 2 c and 2 c + 1
        const uint32_t vb = st + kStep * D;
#pragma unroll
        for (int i = 0; i < D / 16; i += 2) {
          uint32_t w[4];
          ldm_trans(w, vb + Sh::v_at(lane & 15, i + (lane >> 4)));
          if constexpr (FMT != GBLN_Q8_INT8) {
            if (!whole) {  // a NaN code of a key that some row does not see
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = without_nan(w[k]);
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t a[4];
            codes_f16<FMT>(w[2 * k], a[0], a[2]);
            codes_f16<FMT>(w[2 * k + 1], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(o[n][i + k], a, pb[n][0], pb[n][1]);
          }
        }
      }
      cp_wait<0>();
      __syncwarp();  // the ring is the results' now
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], k);
          const int r = 8 * n + 2 * c + e;
          const float back = power_inverse(U[n][e]);  // R / 2^13
          if (g == 0) *reinterpret_cast<float2*>(res + ROWS * D + 2 * r) = make_float2(m[n][e], l[n][e]);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            res[r * D + 16 * i + g] = o[n][i][e] * back;
            res[r * D + 16 * i + g + 8] = o[n][i][e + 2] * back;
          }
        }
    }
    const bool before = tile > 0, behind = t1 < u.tiles, split = before || behind;
    if (S > 1) __syncthreads();
    else __syncwarp();
    if (on) {  // a warp writes rows slice, slice + S, ... of its head: the slices joined in order
      const int slot = (int)blockIdx.x * 2 + (before ? 0 : 1);
      for (int r = slice; r < nrows; r += S) {
        const float* heads = reinterpret_cast<float*>(ring) + wh * (Sh::WARP / 4);
        const int next_slice = A.HB * (Sh::WARP / 4);
        float top = -INFINITY;
        for (int k = 0; k < S; ++k) top = fmaxf(top, heads[k * next_slice + ROWS * D + 2 * r]);
        const float ref = finite_or_zero(top);
        float sum = 0.f, acc[W];
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] = 0.f;
#pragma unroll 4
        for (int k = 0; k < S; ++k) {
          const float* a = heads + k * next_slice;
          const float f = ex2(a[ROWS * D + 2 * r] - ref);
          sum += a[ROWS * D + 2 * r + 1] * f;
#pragma unroll
          for (int i = 0; i < W; ++i) acc[i] += a[r * D + lane + 32 * i] * f;
        }
        if (split) {
          const int64_t at = ((int64_t)slot * A.HB + wh) * ROWS + r;
#pragma unroll
          for (int i = 0; i < W; ++i) A.part_o[at * D + lane + 32 * i] = acc[i];
          if (lane == 0) *reinterpret_cast<float2*>(A.part_ml + 2 * at) = make_float2(top, sum);
        } else {
          const int row = u.r0 + r, tok = A.group.by(row), hq = h * A.G + row - tok * A.G;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          bf16* dst = (bf16*)A.out + (u.s.q0 + tok) * A.ldo + (int64_t)hq * D;
#pragma unroll
          for (int i = 0; i < W; ++i) dst[lane + 32 * i] = __float2bfloat16_rn(sum == 0.f ? 0.f : acc[i] * inv);
          if (A.lse && lane == 0) A.lse[(int64_t)(u.s.q0 + tok) * A.Hq + hq] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        }
      }
    }
    if (behind && !before && threadIdx.x == 0) tell_join(A, u, parts_behind(plan, num + (u.tiles - 1 - tile)));
    const int nt = t1 - tile;
    num += nt + kFewBegin;
    if (!few_go_on<ROWS>(A, S, u, tile, left, nt)) break;
    if (S > 1) __syncthreads();
    else __syncwarp();
  }
}

// Parts first, first + step, ... n of a row: part 0 is of block c, its second place, the others of the blocks behind it, their
// first.  A lane has every 32nd value.
template <int D>
__device__ __forceinline__ void add_parts(const AttnArgs& A, int MR, int c, int n, int wh, int r, int first, int step, float& m, float& l,
                                          float (&acc)[D / 32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int k = first; k <= n; k += step) {
    const int64_t at = ((int64_t)(2 * (c + k) + (k == 0 ? 1 : 0)) * A.HB + wh) * MR + r;
    const float2 p = *reinterpret_cast<const float2*>(A.part_ml + 2 * at);
    float v[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) v[i] = A.part_o[at * D + lane + 32 * i];
    const float to = fmaxf(m, p.x), ref = finite_or_zero(to), f0 = ex2(m - ref), f1 = ex2(p.x - ref);
    m = to;
    l = l * f0 + p.y * f1;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = acc[i] * f0 + v[i] * f1;
  }
}

// Join the parts of the units that the plan divided.  A block takes one row after the other, its eight warps the
// row's parts in turns (all parts of a row are under way at once), a lane D / 32 of the values.  Where there are rows
// for more than two rounds, units have few parts, and each warp takes rows of its own (2048 tokens over 32768, 38912 rows of
// two or three parts: 76 us with a block per row, 17 so; 64
// sequences of one token 11 and 6 us).
template <int D>
__global__ void __launch_bounds__(256) attn8_join(const __grid_constant__ AttnArgs A, int MR, int blocks) {
  constexpr int W = D / 32;
  __shared__ int units[1024], count;  // the blocks of the primary kernel in which a divided unit began
  __shared__ float2 ml[8];
  __shared__ float part[8][D];
  const int lane = threadIdx.x & 31, warp = warp_index();
  wait_for_primary();
  if (warp == 0) {
    int n = 0;
    for (int c0 = 0; c0 < blocks; c0 += 32) {
      const bool first = c0 + lane < blocks && A.info[(c0 + lane) * kAttnInfo] > 0;
      const unsigned b = __ballot_sync(0xffffffffu, first);
      if (first) units[n + __popc(b & ((1u << lane) - 1u))] = c0 + lane;
      n += __popc(b);
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int per = MR * A.HB, total = count * per;
  const bool apart = total > 2 * (int)gridDim.x;
  for (int x = apart ? 8 * blockIdx.x + warp : blockIdx.x; x < total; x += apart ? 8 * gridDim.x : gridDim.x) {
    const int c = units[x / per], y = x % per, wh = y / MR, r = y - wh * MR;
    const int* f = A.info + c * kAttnInfo;
    const int n = f[0], nrows = f[1], row = f[2] + r, q0 = f[3], h = f[4] * A.HB + wh;
    if (r >= nrows || h >= A.Hk) continue;  // uniform in the block, or the warp
    float m = -INFINITY, l = 0.f, acc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.f;
    if (apart) {
      add_parts<D>(A, MR, c, n, wh, r, 0, 1, m, l, acc);
      const int tok = A.group.by(row), hq = h * A.G + row - tok * A.G;
      bf16* dst = (bf16*)A.out + (q0 + tok) * A.ldo + (int64_t)hq * D + lane;
#pragma unroll
      for (int i = 0; i < W; ++i) dst[32 * i] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[i] / l);
      if (A.lse && lane == 0) A.lse[(int64_t)(q0 + tok) * A.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      continue;
    }
    add_parts<D>(A, MR, c, n, wh, r, warp, 8, m, l, acc);
    if (lane == 0) ml[warp] = make_float2(m, l);
#pragma unroll
    for (int i = 0; i < W; ++i) part[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    if ((int)threadIdx.x < D) {
      float top = ml[0].x;
#pragma unroll
      for (int k = 1; k < 8; ++k) top = fmaxf(top, ml[k].x);
      const float ref = finite_or_zero(top);
      float sum = 0.f, v = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float e = ex2(ml[k].x - ref);
        sum += ml[k].y * e;
        v += part[k][threadIdx.x] * e;
      }
      const int tok = A.group.by(row), hq = h * A.G + row - tok * A.G;
      ((bf16*)A.out)[(q0 + tok) * A.ldo + (int64_t)hq * D + threadIdx.x] = __float2bfloat16_rn(sum == 0.f ? 0.f : v / sum);
      if (A.lse && threadIdx.x == 0) A.lse[(int64_t)(q0 + tok) * A.Hq + hq] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
    __syncthreads();
  }
}

// Any other rows (float32), head sizes and alignments.  A block per row, its warps on 32 keys at a time in turns: scores with a
// lane per key, W codes at a load (16 or 4 where sizes and strides are multiples of them, else 1), then lanes over the
// values, up to NVAL each; the warps' sums meet at the end.  Bound by instructions, about forty per key and warp.
// (64 sequences of 1024 keys, 32 / 8 heads: of 80 265 us, of 33 402; of 96 in the kernel above 51.)
constexpr int kElemWarps = 8;
template <typename T, int FMT, int W, int NVAL>
__global__ void __launch_bounds__(32 * kElemWarps, NVAL == 4 ? 4 : 3) attn8_elem(const __grid_constant__ AttnArgs A) {
  constexpr int VW = W >= 4 ? 4 : 1, NW = NVAL / VW;
  __shared__ __align__(16) float qs[32 * NVAL];
  __shared__ float part[kElemWarps][32 * NVAL], ml[kElemWarps][2];
  const int lane = threadIdx.x & 31, warp = warp_index();
  const int64_t rows = (int64_t)A.T * A.Hq;
  const int end = min(max(__ldg(A.cu + A.B), 0), A.T);
  for (int64_t x = blockIdx.x; x < rows; x += gridDim.x) {
    const int tok = (int)(x / A.Hq), hq = (int)(x - (int64_t)tok * A.Hq), h = hq / A.G;
    if (tok >= end) return;  // rows behind the last sequence
    // the last sequence that starts at or before the token
    int lo = 0, hi = A.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(A.cu + mid) <= tok) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo;
    const Seq s = seq_at(A, b);
    if (tok < s.q0 || tok >= s.q0 + s.nq) continue;
    const T* src = (const T*)A.q + tok * A.ldq + (int64_t)hq * A.D;
    __syncthreads();  // the row before is done
    for (int d = threadIdx.x; d < A.D; d += 32 * kElemWarps) qs[d] = to_f32(src[d]);
    __syncthreads();
    const int pos = s.kv - s.nq + tok - s.q0;
    const int first = A.window > 0 ? max(0, pos - A.window + 1) : 0, last = A.causal ? min(s.kv, pos + 1) : s.kv;
    float m = -INFINITY, l = 0.f, acc[NW][VW];
#pragma unroll
    for (int e = 0; e < NW; ++e)
#pragma unroll
      for (int k = 0; k < VW; ++k) acc[e][k] = 0.f;
    for (int64_t begin = (int64_t)first + 32 * warp; begin < last; begin += 32 * kElemWarps) {
      const int j0 = (int)begin;
      const KeyAt k = key_at(A, b, j0 + lane, first, last);
      if (k.page == -2) atomicOr(A.err, kErrBadSlot);
      float sc = -INFINITY, vs = 0.f;
      const uint8_t* vc = A.V.q;
      if (k.page >= 0) {
        const uint8_t* kc = A.K.q + A.K.cq.at(k.page, k.off, h);
        vc += A.V.cq.at(k.page, k.off, h);
        const float ks = A.K.sc[A.K.cs.at(k.page, k.off, h)];
        vs = A.V.sc[A.V.cs.at(k.page, k.off, h)];
        float dot[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (W == 1) {
          for (int d = 0; d < A.D; ++d) {
            float t[4];
            q8_decode4<FMT>(kc[d], t);
            dot[0] = fmaf(qs[d], t[0], dot[0]);
          }
        } else {
#pragma unroll 2
          for (int d = 0; d < A.D; d += W) {
            uint32_t w[W / 4];
            if constexpr (W == 16) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(kc + d);
            else w[0] = *reinterpret_cast<const uint32_t*>(kc + d);
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
              float t[4];
              q8_decode4<FMT>(w[i], t);
              const float4 q = *reinterpret_cast<const float4*>(qs + d + 4 * i);
              dot[0] = fmaf(q.x, t[0], dot[0]);
              dot[1] = fmaf(q.y, t[1], dot[1]);
              dot[2] = fmaf(q.z, t[2], dot[2]);
              dot[3] = fmaf(q.w, t[3], dot[3]);
            }
          }
        }
        sc = ((dot[0] + dot[1]) + (dot[2] + dot[3])) * (ks * A.scale2);
      } else if (k.page == -2) {
        sc = vs = __int_as_float(0x7fc00000);
      }
      float top = sc;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float to = fmaxf(m, top), ref = finite_or_zero(to), f = ex2(m - ref);
      m = to;
      const float p = ex2(sc - ref);
      l = l * f + p;
#pragma unroll
      for (int e = 0; e < NW; ++e)
#pragma unroll
        for (int i = 0; i < VW; ++i) acc[e][i] *= f;
      const float w = p * vs;
      const int n = min(32, last - j0);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const uint8_t* v = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, (unsigned long long)vc, i));
        const bool there = __shfl_sync(0xffffffffu, k.page, i) >= 0;
#pragma unroll
        for (int e = 0; e < NW; ++e) {
          const int d = VW * (lane + 32 * e);
          float t[4] = {0.f, 0.f, 0.f, 0.f};
          if (there && d < A.D) {
            if constexpr (VW == 4) q8_decode4<FMT>(*reinterpret_cast<const uint32_t*>(v + d), t);
            else q8_decode4<FMT>(v[d], t);
          }
#pragma unroll
          for (int c = 0; c < VW; ++c) acc[e][c] = fmaf(wi, t[c], acc[e][c]);
        }
      }
    }
    l = group_sum<32>(l);
    if (lane == 0) {
      ml[warp][0] = m;
      ml[warp][1] = l;
    }
#pragma unroll
    for (int e = 0; e < NW; ++e)
#pragma unroll
      for (int c = 0; c < VW; ++c) part[warp][VW * (lane + 32 * e) + c] = acc[e][c];
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kElemWarps; ++w) top = fmaxf(top, ml[w][0]);
    const float ref = finite_or_zero(top);
    float f[kElemWarps], sum = 0.f;
#pragma unroll
    for (int w = 0; w < kElemWarps; ++w) {
      f[w] = ex2(ml[w][0] - ref);
      sum += ml[w][1] * f[w];
    }
    T* dst = (T*)A.out + tok * A.ldo + (int64_t)hq * A.D;
    for (int d = threadIdx.x; d < A.D; d += 32 * kElemWarps) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kElemWarps; ++w) v += part[w][d] * f[w];
      dst[d] = from_f32<T>(sum == 0.f ? 0.f : v / sum);
    }
    if (A.lse && threadIdx.x == 0) A.lse[(int64_t)tok * A.Hq + hq] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  }
}

template <typename T, int FMT, int W>
void elem_sized(const AttnArgs& A, unsigned grid, cudaStream_t s) {
  if (A.D <= 128) attn8_elem<T, FMT, W, 4><<<grid, 32 * kElemWarps, 0, s>>>(A);
  else attn8_elem<T, FMT, W, 16><<<grid, 32 * kElemWarps, 0, s>>>(A);
}
template <typename T>
void elem_typed(const AttnArgs& A, int fmt, int w, unsigned grid, cudaStream_t s) {
  if (fmt == GBLN_Q8_INT8) {
    if (w == 16) elem_sized<T, GBLN_Q8_INT8, 16>(A, grid, s);
    else if (w == 4) elem_sized<T, GBLN_Q8_INT8, 4>(A, grid, s);
    else elem_sized<T, GBLN_Q8_INT8, 1>(A, grid, s);
  } else {
    if (w == 16) elem_sized<T, GBLN_Q8_E4M3, 16>(A, grid, s);
    else if (w == 4) elem_sized<T, GBLN_Q8_E4M3, 4>(A, grid, s);
    else elem_sized<T, GBLN_Q8_E4M3, 1>(A, grid, s);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return {d, (uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

// How the kernel for few rows is used: NT columns of eight rows, and the K/V heads of a block, 1, 2, 4 or 8.  All
// warps on heads of their own where the batch fills the GPU (neighbouring heads' scales share their sectors),
// fewer, with the keys of a head cut into slices, where it does not: less is left to be joined.
// (262144 cached tokens of 8 heads: 128 sequences 164 us with one head a block, 137 with eight; 4 sequences 136 and 152.  Two
// columns where a sequence has more than eight rows: 32 sequences of 4096 tokens, 8 rows each, 95 us with one column,
// 107 with two; 16 rows 140 and 122.)
struct FewUse {
  int nt, hb;
};
FewUse few_use(int64_t T, int64_t B, int G, int Hk, int sms) {
  FewUse f{T * G > 8 * B ? 2 : 1, 1};
  while (f.hb < 8 && f.hb < Hk && B * Hk >= (int64_t)sms * f.hb) f.hb *= 2;
  return f;
}

template <int D, int FMT, int NT, bool ONE>
gbln_status few_go(const AttnArgs& A, int blocks, bool q16, cudaStream_t s) {
  using Sh = FewShape<D, NT>;
  static std::atomic<uint64_t> ready{0};  // devices whose limit is raised
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GBLN_ERR_CUDA;
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    if (cudaFuncSetAttribute(attn8_few<D, FMT, NT, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM) != cudaSuccess) {
      cudaGetLastError();
      return GBLN_ERR_CUDA;
    }
    ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  attn8_few<D, FMT, NT, ONE><<<blocks, 32 * Sh::WARPS, Sh::SMEM, s>>>(A, q16);
  return cudaGetLastError() == cudaSuccess ? attn_join_launch(A, blocks, Sh::ROWS, s) : GBLN_ERR_CUDA;
}

template <int D, int FMT>
gbln_status few_sized(const AttnArgs& A, int nt, int blocks, bool q16, cudaStream_t s) {
  const bool one = A.page.d % kStep == 0;
  if (nt == 1) return one ? few_go<D, FMT, 1, true>(A, blocks, q16, s) : few_go<D, FMT, 1, false>(A, blocks, q16, s);
  return one ? few_go<D, FMT, 2, true>(A, blocks, q16, s) : few_go<D, FMT, 2, false>(A, blocks, q16, s);
}

template <int FMT>
gbln_status few_typed(const AttnArgs& A, int nt, int blocks, bool q16, cudaStream_t s) {
  switch (A.D) {
    case 64: return few_sized<64, FMT>(A, nt, blocks, q16, s);
    case 96: return few_sized<96, FMT>(A, nt, blocks, q16, s);
    case 128: return few_sized<128, FMT>(A, nt, blocks, q16, s);
    default: return few_sized<256, FMT>(A, nt, blocks, q16, s);
  }
}

// Rows for the tensor-core kernel: where a sequence brings more rows on average than the other
// kernel takes at once, so that K and V would be converted several times over there.
// (32 sequences of 4096 tokens, 4 heads a group: 24 rows each 157 us there, 190 here; 32 rows 204 and 190; 48 rows 332 and 231.)
bool many_rows(int64_t T, int32_t B, int G, int32_t D) { return D <= 128 && T * G >= 32 * (int64_t)B; }

bool fast_head(int32_t D, int io) { return io == GBLN_BF16 && (D == 64 || D == 96 || D == 128 || D == 256); }

bool attn_sizes_ok(int64_t T, int32_t B, int32_t Hq, int32_t Hk, int32_t D) {
  return T >= 0 && B >= 0 && Hk >= 1 && Hq >= 1 && Hq % Hk == 0 && D >= 1 && D <= kAttnMaxHeads && (int64_t)Hq * D <= (1 << 24) &&
         T <= (1LL << 30) / Hq;
}

}  // namespace

gbln_status attn_join_launch(const AttnArgs& A, int blocks, int rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks * 4);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = A.D == 64    ? cudaLaunchKernelEx(&cfg, attn8_join<64>, A, rows, blocks)
                        : A.D == 96  ? cudaLaunchKernelEx(&cfg, attn8_join<96>, A, rows, blocks)
                        : A.D == 128 ? cudaLaunchKernelEx(&cfg, attn8_join<128>, A, rows, blocks)
                                     : cudaLaunchKernelEx(&cfg, attn8_join<256>, A, rows, blocks);
  if (e == cudaSuccess) return GBLN_OK;
  cudaGetLastError();
  return GBLN_ERR_CUDA;
}

}  // namespace gbln

using namespace gbln;

extern "C" int64_t gbln_attn_cache8_workspace(int64_t T, int32_t B, int32_t Hq, int32_t Hk, int32_t D, gbln_dtype io) {
  if (!dtype_ok(io) || !attn_sizes_ok(T, B, Hq, Hk, D)) return -1;
  if (T == 0 || B == 0 || !fast_head(D, io)) return 0;
  const int sms = sm_count();
  if (sms <= 0) return -1;
  const FewUse f = few_use(T, B, Hq / Hk, Hk, sms);
  const int rows = many_rows(T, B, Hq / Hk, D) ? kManyUnit : f.hb * 8 * f.nt;
  return (int64_t)sms * (kAttnInfo * 4 + 2 * rows * (D + 2) * 4);
}

extern "C" gbln_status gbln_attn_cache8(const void* q, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                                        const int32_t* page_table, int64_t max_pages, const gbln_cache8* k_cache,
                                        const gbln_cache8* v_cache, void* out, float* lse, void* workspace,
                                        int64_t workspace_bytes, int64_t T, int32_t B, int32_t Hq, int32_t Hk, int32_t D,
                                        int64_t ld_q, int64_t ld_out, float scale, int32_t causal, int32_t window,
                                        gbln_q8 fmt, gbln_dtype io, gbln_stream_t stream) {
  if (!dtype_ok(io) || !q8_ok(fmt) || !attn_sizes_ok(T, B, Hq, Hk, D)) return GBLN_ERR_INVALID_ARG;
  // the scale is taken to powers of two: 2e38 * log2(e) is finite, 3e38 * log2(e) is not
  if (max_pages < 0 || window < 0 || !(scale >= -2.0e38f && scale <= 2.0e38f)) return GBLN_ERR_INVALID_ARG;
  if (!ld_fits(T, (int64_t)Hq * D, ld_q) || !ld_fits(T, (int64_t)Hq * D, ld_out)) return GBLN_ERR_INVALID_ARG;
  if (!cache_ok(k_cache, Hk, D) || !cache_ok(v_cache, Hk, D)) return GBLN_ERR_INVALID_ARG;
  if (k_cache->pages != v_cache->pages || k_cache->page_size != v_cache->page_size) return GBLN_ERR_INVALID_ARG;
  if (k_cache->pages >= (1LL << 31) || k_cache->page_size > (1LL << 30) || max_pages > (1LL << 30) / k_cache->page_size)
    return GBLN_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!q || !cu_seqlens_q || !kv_lens || !out || (max_pages > 0 && !page_table)) return GBLN_ERR_INVALID_ARG;
  if (k_cache->pages > 0 && (!k_cache->codes || !k_cache->scale || !v_cache->codes || !v_cache->scale)) return GBLN_ERR_INVALID_ARG;
  if (!aligned_to(cu_seqlens_q, 4) || !aligned_to(kv_lens, 4) || !aligned_to(page_table, 4) || !aligned_to(lse, 4)) return GBLN_ERR_INVALID_ARG;
  const int sms = sm_count();
  unsigned int* err = device_error_word();
  if (sms <= 0 || sms > 1024 || !err) return GBLN_ERR_CUDA;  // the joining kernel lists the blocks
  AttnArgs A{};
  A.q = q;
  A.out = out;
  A.lse = lse;
  A.cu = cu_seqlens_q;
  A.kv = kv_lens;
  A.pages = page_table;
  A.max_pages = max_pages;
  A.ldq = ld_q;
  A.ldo = ld_out;
  A.T = (int)T;
  A.B = B;
  A.Hq = Hq;
  A.Hk = Hk;
  A.G = Hq / Hk;
  A.D = D;
  A.scale2 = scale * 1.4426950408889634f;
  A.causal = causal != 0;
  A.window = window < (1 << 30) ? window : 0;  // no position is that far from another
  A.n_pages = (int)k_cache->pages;
  A.page = fast_div((uint32_t)k_cache->page_size);
  A.group = fast_div((uint32_t)A.G);
  A.K = cache_of(k_cache);
  A.V = cache_of(v_cache);
  A.err = err;
  cudaStream_t s = (cudaStream_t)stream;
  if (fast_head(D, io) && codes_aligned(k_cache, v_cache, 16)) {
    if (!workspace || !aligned16(workspace) || workspace_bytes < gbln_attn_cache8_workspace(T, B, Hq, Hk, D, io)) return GBLN_ERR_WORKSPACE;
    const bool many = many_rows(T, B, A.G, D);
    const FewUse f = few_use(T, B, A.G, Hk, sms);
    A.HB = many ? 1 : f.hb;
    A.NHG = (Hk + A.HB - 1) / A.HB;
    A.info = (int*)workspace;
    A.part_ml = (float*)workspace + (int64_t)sms * kAttnInfo;
    A.part_o = A.part_ml + (int64_t)sms * 2 * 2 * (many ? kManyUnit : A.HB * 8 * f.nt);
    if (many) return attn_many_launch(A, sms, fmt, s);
    const bool q16 = aligned16(q) && ld_q % 8 == 0;
    return fmt == GBLN_Q8_INT8 ? few_typed<GBLN_Q8_INT8>(A, f.nt, sms, q16, s) : few_typed<GBLN_Q8_E4M3>(A, f.nt, sms, q16, s);
  }
  const unsigned grid = grid_for(T * (int64_t)Hq, 1, (int64_t)sms * 32);
  const auto codes_by = [&](int n) { return D % n == 0 && codes_aligned(k_cache, v_cache, n); };
  const int w = codes_by(16) ? 16 : codes_by(4) ? 4 : 1;
  if (io == GBLN_F32) elem_typed<float>(A, fmt, w, grid, s);
  else elem_typed<bf16>(A, fmt, w, grid, s);
  return launch_status();
}
