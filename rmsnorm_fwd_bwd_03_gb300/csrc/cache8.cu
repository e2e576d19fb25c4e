// RoPE on Q and K with K and V quantised into a paged 8-bit cache in the same
// launch, and the read-back of any slots of that cache.
//
// Operator: "Fast-LLM: 高效大语言模型训练框架", §三 框架结构 (attention with RoPE; heads /
// head_groups / head_size for grouped-query attention) and 训练配置示例 (rotary);
// "LLaMA-Factory Kernels 系统" (fused RoPE); fusing the conversion into the pass
// that produces K, as "Kernels（自定义内核）" §Liger fuses a producer with what follows.
//
// A group is one head of one token: D codes (INT8 or E4M3) and one float32
// scale.  HBM-bound: Q is read and written once, K and V are read once and
// written as one byte per value; decode steps are bound by their single launch.

#include "cache8.cuh"

namespace gbln {

namespace {

template <typename T>
struct WriteArgs {
  const T* q;
  const T* k;
  const T* v;
  T* qo;
  const int32_t* pos;
  const float2* table;
  int64_t max_pos, rows;
  int Hq, Hk, D;
  int64_t ldq, ldk, ldv, ldqo;
  Slots S;
  Cache K, V;
  unsigned int* err;
};

// ---------------------------------------------------------------------------
// Vector path.  A warp works either on queries (up to kWriteQ head rows per lane:
// rotate and store) or on K and V (one or two heads of both per lane: rotate K,
// quantise both), one token after the other; where a token's heads leave lanes
// over, several tokens at a time.  A lane owns the vectors at v*VEC of both halves
// of a head row, whichever pairing, so a warp's accesses are whole lines: with
// rotate-half pairing they turn into each other by VEC table entries, with
// interleaved pairing each holds VEC / 2 pairs of its own.  A head row takes
// nu = D / (2 VEC) lanes out of a group of the next power of two, so 80 or 96 wide
// heads run here with idle lanes.  VEC fills 16 bytes, or 8 where a half head or an
// address is a multiple of 8 bytes only (bf16 heads of 40 or 72 values).  All of a lane's row loads are issued before
// anything that depends on the token's slot or position, and the maxima and
// divisions of its K and V heads run side by side.  (With queries, K and V taken
// alike, head after head, the chain of each one's reduction and division showed:
// 95 us instead of 79 for 32768 tokens of 16 / 8 heads of 128, 70 us at the copy
// rate.)  65536 tokens of 32 / 8 heads of 128: 223 us, 219 us at the copy rate; 16
// tokens 2.3 us.
// ---------------------------------------------------------------------------
// Head rows per lane and pass of a query warp: 8 measured 112 us, 6 119 and 4 117 for
// 32768 tokens of 32 / 8 heads of 128 (110 us at the copy rate).
constexpr int kWriteQ = 8;
constexpr int kMaxVecHeads = 1 << 17;  // Q, K and V heads: at most 2^14 rows of blocks
constexpr int kWriteWarps = 8;  // per block: chunks of a token, then tokens
// A warp walks its tokens and asks for the next ones' rows in L2 while it works
// on these.  Eight times the resident blocks leave a warp a few steps to do that
// for and the scheduler something to balance.
constexpr int kWriteBlocks = 2;               // resident per SM
constexpr int kWriteGrid = kWriteBlocks * 8;  // blocks per SM
// With 8-byte accesses half as many registers hold loads: three blocks measured 37 us
// for 16384 tokens of 8 / 8 heads of 72, two 50, four (spilling) 40.
constexpr int kWriteBlocks8 = 3;
// Few heads per token (a GPU's share of a model) leave most of a lane's registers
// idle: up to 32 bytes of each query half and one head of K and V per lane run four
// blocks per SM instead, at 64 registers.  32768 tokens, two and four blocks (copy
// rate): 8 / 2 heads of 128 42 and 33 us (28), 14 / 2 of 64 38 and 28 (21), 7 / 1 of 96
// 37 and 25 (16); five blocks spill, 51 us.  Beyond that the larger share per lane is
// faster (32 / 8 heads of 128: 113 and 127 us), except for so few tokens that every
// warp of the finer split runs at once (16 tokens: 3.0 and 2.4 us).
constexpr int kFewBlocks = 4;
constexpr int few_queries(int bytes) { return 32 / bytes; }  // per lane, in accesses of that many bytes

struct WriteShape {
  int nu, lg;         // lanes in use per head row, log2 of the lanes of its group
  int nq, qch, qlt;   // query chunks, head rows per lane in each, log2 of tokens per warp
  int nkv, kch, klt;  // the same of K and V heads
};

// (cos, sin) of a lane's pairs: entries ia.. (rotate-half), or half as many for
// each of its two vectors (interleaved); NaN for a position outside the table.
template <int VEC, bool IL>
__device__ __forceinline__ void load_turns(const float2* table, int half, int p, bool ok, bool on, int ia, float2 (&cs)[VEC]) {
  if (ok && on) {
    const float2* e = table + (size_t)p * half;
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      const int at = !IL ? ia + i : i < VEC / 2 ? ia / 2 + i : (half + ia) / 2 + i - VEC / 2;
      const float4 f = __ldg(reinterpret_cast<const float4*>(e + at));
      cs[i] = make_float2(f.x, f.y);
      cs[i + 1] = make_float2(f.z, f.w);
    }
  } else {
    const float x = ok ? 0.f : __int_as_float(0x7fc00000);
#pragma unroll
    for (int i = 0; i < VEC; ++i) cs[i] = make_float2(x, x);
  }
}
template <typename T, bool IL, int FMT, int VEC, int KP, int QP>
__global__ void __launch_bounds__(32 * kWriteWarps, QP < kWriteQ ? kFewBlocks : VEC * sizeof(T) == 16 ? kWriteBlocks : kWriteBlocks8)
cache8_write_vec(const WriteArgs<T> A, const WriteShape W) {
  using Run = HeadRun<T, VEC>;
  constexpr int LINE = 128 / sizeof(T);
  const int half = A.D / 2;
  const int lanes = 1 << W.lg;
  const int lane = threadIdx.x;
  const int v = lane & (lanes - 1);
  const bool on = v < W.nu;
  const int c = blockIdx.y * blockDim.y + threadIdx.y;
  if (c >= W.nq + W.nkv) return;  // uniform per warp
  const bool isq = c < W.nq;
  // the lanes of a group take a head of one of the warp's 2^lt tokens
  const int lt = isq ? W.qlt : W.klt, G = 32 >> (W.lg + lt);
  const int sub = (lane >> W.lg) >> (5 - W.lg - lt), g = (lane >> W.lg) & (G - 1);
  const int li = lane & ((32 >> lt) - 1);  // the lane's number among its token's
  const int64_t step = ((int64_t)gridDim.x * blockDim.z) << lt;
  int64_t t0 = ((int64_t)blockIdx.x * blockDim.z + threadIdx.z) << lt;
  if (t0 >= A.rows) return;
  const int64_t end = A.rows - 1;
  const int ia = v * VEC;
  const int64_t first = min(t0 + sub, end);
  int p = __ldg(A.pos + first);
  float2 cs[VEC];

  if (isq) {
    const int hf = G * c * W.qch, hb = hf + g;
    const int last = min(hf + G * W.qch, A.Hq) * A.D;
#pragma unroll 1
    for (; t0 < A.rows; t0 += step) {
      const int64_t t = t0 + sub;
      const bool live = on && t < A.rows;
      const T* qp = A.q + min(t, end) * A.ldq;
      T* qo = A.qo + min(t, end) * A.ldqo;
      Run a[QP], b[QP];
#pragma unroll
      for (int j = 0; j < QP; ++j) {
        const int h = hb + G * j;
        if (j < W.qch && live && h < A.Hq) {
          a[j].load(qp + h * A.D + ia);
          b[j].load(qp + h * A.D + ia + half);
        }
      }
      const bool ok = p >= 0 && (int64_t)p < A.max_pos;
      load_turns<VEC, IL>(A.table, half, p, ok, on, ia, cs);
      if (!ok && live && c == 0 && li == 0) atomicOr(A.err, kErrBadPosition);
      if (t0 + step < A.rows) {  // the warp's next tokens
        const int64_t n = min(t + step, end);
        p = __ldg(A.pos + n);
        for (int x = hf * A.D + li * LINE; x < last; x += (32 >> lt) * LINE) prefetch_line(A.q + n * A.ldq + x);
      }
#pragma unroll
      for (int j = 0; j < QP; ++j) {
        const int h = hb + G * j;
        if (j < W.qch && live && h < A.Hq) {
          float xa[VEC], xb[VEC];
          a[j].get(xa);
          b[j].get(xb);
          turn<VEC, IL>(xa, xb, cs);
          Run::store(qo + h * A.D + ia, xa);
          Run::store(qo + h * A.D + ia + half, xb);
        }
      }
    }
    return;
  }

  const int ck = c - W.nq;
  const int hf = G * ck * W.kch, hb = hf + g;
  const int last = min(hf + G * W.kch, A.Hk) * A.D;
  int64_t slot = __ldg(A.S.slots + first);
#pragma unroll 1
  for (; t0 < A.rows; t0 += step) {
    const int64_t t = t0 + sub;
    const bool live = on && t < A.rows;
    const T *kp = A.k + min(t, end) * A.ldk, *vp = A.v + min(t, end) * A.ldv;
    constexpr int N = 2 * KP;  // K of each head, then V of each
    Run a[N], b[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int h = hb + G * (j % KP);
      a[j].zero();
      b[j].zero();
      if (j % KP < W.kch && live && h < A.Hk) {
        const T* src = (j < KP ? kp : vp) + h * A.D + ia;
        a[j].load(src);
        b[j].load(src + half);
      }
    }
    const bool ok = p >= 0 && (int64_t)p < A.max_pos;
    load_turns<VEC, IL>(A.table, half, p, ok, on, ia, cs);
    int64_t off = 0;
    const int64_t page = A.S.page_of(slot, off);
    if (ck == 0 && li == 0 && live) {
      if (!ok && page >= 0) atomicOr(A.err, kErrBadPosition);
      if (page == -2) atomicOr(A.err, kErrBadSlot);
    }
    if (t0 + step < A.rows) {  // the warp's next tokens
      const int64_t n = min(t + step, end);
      p = __ldg(A.pos + n);
      slot = __ldg(A.S.slots + n);
      for (int x = hf * A.D + li * LINE; x < last; x += (32 >> lt) * LINE) {
        prefetch_line(A.k + n * A.ldk + x);
        prefetch_line(A.v + n * A.ldv + x);
      }
    }
    float xa[N][VEC], xb[N][VEC];
    uint32_t m[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      a[j].get(xa[j]);
      b[j].get(xb[j]);
      if (j < KP) turn<VEC, IL>(xa[j], xb[j], cs);
      m[j] = on ? max(abs_max_bits<VEC>(xa[j]), abs_max_bits<VEC>(xb[j])) : 0u;
    }
    float inv[N], sc[N];
    for (int o = 1; o < lanes; o <<= 1)
#pragma unroll
      for (int j = 0; j < N; ++j) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], o));
    if (lanes >= 2 * N) {
      // lanes 2 j and 2 j + 1 of a group divide for 1 / scale and for the scale of j
      uint32_t mine = m[0];
#pragma unroll
      for (int j = 1; j < N; ++j)
        if (((lane >> 1) & (N - 1)) == j) mine = m[j];
      const float am = q8_amax(mine);
      const float d = __fdiv_rn(lane & 1 ? am : Q8Max<FMT>::v, lane & 1 ? Q8Max<FMT>::v : am);
      const int base = lane & ~(lanes - 1);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        inv[j] = __shfl_sync(0xffffffffu, d, base | (2 * j));
        sc[j] = __shfl_sync(0xffffffffu, d, base | (2 * j + 1));
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float am = q8_amax(m[j]);
        inv[j] = q8_inv<FMT>(am);
        sc[j] = __fdiv_rn(am, Q8Max<FMT>::v);
      }
    }
    if (page < 0 || !live) continue;  // nothing to store; no shuffles below
    const int64_t kq = A.K.cq.at(page, off, hb) + ia, vq = A.V.cq.at(page, off, hb) + ia;
    const int64_t ks = A.K.cs.at(page, off, hb), vs = A.V.cs.at(page, off, hb);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = j % KP;
      if (i < W.kch && hb + G * i < A.Hk) {
        const bool isk = j < KP;
        uint8_t* dst = isk ? A.K.q + kq + G * i * A.K.cq.head : A.V.q + vq + G * i * A.V.cq.head;
        q8_store<FMT, VEC>(xa[j], inv[j], dst);
        q8_store<FMT, VEC>(xb[j], inv[j], dst + half);
        if (v == 0)
          *(isk ? A.K.sc + ks + G * i * A.K.cs.head : A.V.sc + vs + G * i * A.V.cs.head) =
              m[j] < kInfBits ? sc[j] : __int_as_float(0x7fc00000);
      }
    }
  }
}

// Element path (any alignment and stride, heads of up to 256 values): a warp takes
// four heads of one token, one value per access; lane l has the pairs l, l + 32, ...
// (K of them) of each, which wait in registers for the heads' maxima.  The heads share
// the token's slot, position and turns, and their loads, reductions and one
// division run side by side: 86 us for 16384 tokens of 8 / 8 heads of 72, where a
// warp per head, bound by its latency, took 174 and the 8-byte vector path takes 37
// (14 us at the copy rate).  16384 tokens of 12 / 3 heads of 100: 70 us.
constexpr int kElemHeads = 4;

template <typename T, bool IL, int FMT, int K>
__global__ void __launch_bounds__(256) cache8_write_elem(const WriteArgs<T> A, bool small) {
  constexpr int F = kElemHeads;
  const int half = A.D / 2, HR = A.Hq + A.Hk, HT = HR + A.Hk, nc = (HT + F - 1) / F;
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp_index(); item < A.rows * nc; item += step) {
    const int64_t t = small ? (int64_t)((uint32_t)item / (uint32_t)nc) : item / nc;
    const int h0 = (int)(item - t * nc) * F;
    const int64_t slot = __ldg(A.S.slots + t);
    const int p = __ldg(A.pos + t);
    T x1[F][K], x2[F][K];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int h = h0 + f;
      if (h >= HT) break;  // uniform per warp, as every test of h
      const T* src = h < A.Hq ? A.q + t * A.ldq + h * A.D
                     : h < HR ? A.k + t * A.ldk + (h - A.Hq) * A.D
                              : A.v + t * A.ldv + (h - HR) * A.D;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = lane + 32 * k;
        x1[f][k] = x2[f][k] = from_f32<T>(0.f);
        if (i < half) {
          x1[f][k] = src[IL ? 2 * i : i];
          x2[f][k] = src[IL ? 2 * i + 1 : half + i];
        }
      }
    }
    const bool ok = p >= 0 && (int64_t)p < A.max_pos;
    float2 cs[K];
    if (h0 < HR) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = lane + 32 * k;
        cs[k] = both(ok ? 0.f : __int_as_float(0x7fc00000));
        if (ok && i < half) cs[k] = __ldg(A.table + (size_t)p * half + i);
      }
    }
    int64_t off = 0;
    const int64_t page = A.S.page_of(slot, off);
    if (h0 == 0 && lane == 0) {
      if (!ok && (A.Hq > 0 || page >= 0)) atomicOr(A.err, kErrBadPosition);
      if (page == -2) atomicOr(A.err, kErrBadSlot);
    }
    float2 y[F][K];
    uint32_t mine = 0;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int h = h0 + f;
      if (h >= HT) break;
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float a = to_f32(x1[f][k]), b = to_f32(x2[f][k]);
        // V is not rotated: it is taken as it is, whatever it holds
        y[f][k] = h >= HR ? make_float2(a, b) : turn1(a, b, cs[k]);
        if (lane + 32 * k < half) m = max(m, max(abs_bits(y[f][k].x), abs_bits(y[f][k].y)));
      }
      if (h >= A.Hq) {
        m = group_max<32>(m);
        if (lane >> 1 == f) mine = m;  // lanes 2 f and 2 f + 1 divide for 1 / scale and scale
      }
    }
    const float am = q8_amax(mine);
    const float d = __fdiv_rn(lane & 1 ? am : Q8Max<FMT>::v, lane & 1 ? Q8Max<FMT>::v : am);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int h = h0 + f;
      const float inv = __shfl_sync(0xffffffffu, d, 2 * f);
      if (h >= HT) break;
      if (h < A.Hq) {
        T* dst = A.qo + t * A.ldqo + h * A.D;
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (const int i = lane + 32 * k; i < half) {
            dst[IL ? 2 * i : i] = from_f32<T>(y[f][k].x);
            dst[IL ? 2 * i + 1 : half + i] = from_f32<T>(y[f][k].y);
          }
      } else if (page >= 0) {
        const bool isk = h < HR;
        const int hk = h - (isk ? A.Hq : HR);
        uint8_t* dst = isk ? A.K.q + A.K.cq.at(page, off, hk) : A.V.q + A.V.cq.at(page, off, hk);
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (const int i = lane + 32 * k; i < half) {
            dst[IL ? 2 * i : i] = (uint8_t)q8_code1<FMT>(y[f][k].x, inv);
            dst[IL ? 2 * i + 1 : half + i] = (uint8_t)q8_code1<FMT>(y[f][k].y, inv);
          }
        if (lane == 2 * f + 1)
          *(isk ? A.K.sc + A.K.cs.at(page, off, hk) : A.V.sc + A.V.cs.at(page, off, hk)) =
              mine < kInfBits ? d : __int_as_float(0x7fc00000);
      }
    }
  }
}

// Heads too wide for that: a warp per head row, read twice, the second time from L1.
constexpr int kElemWidth = 256;

template <typename T, bool IL, int FMT>
__global__ void __launch_bounds__(256) cache8_write_wide(const WriteArgs<T> A, bool small) {
  const int half = A.D / 2, HR = A.Hq + A.Hk, HT = HR + A.Hk;
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp_index(); item < A.rows * HT; item += step) {
    const int64_t t = small ? (int64_t)((uint32_t)item / (uint32_t)HT) : item / HT;
    const int h = (int)(item - t * HT);
    const int64_t slot = __ldg(A.S.slots + t);
    const int p = __ldg(A.pos + t);
    const T* src = h < A.Hq ? A.q + t * A.ldq + (int64_t)h * A.D
                   : h < HR ? A.k + t * A.ldk + (int64_t)(h - A.Hq) * A.D
                            : A.v + t * A.ldv + (int64_t)(h - HR) * A.D;
    const bool ok = p >= 0 && (int64_t)p < A.max_pos;
    const float2* turns = A.table + (ok ? (size_t)p * half : 0);
    auto pair = [&](int i) {
      const float x1 = to_f32(src[IL ? 2 * i : i]), x2 = to_f32(src[IL ? 2 * i + 1 : half + i]);
      if (h >= HR) return make_float2(x1, x2);  // V is not rotated
      return turn1(x1, x2, ok ? __ldg(turns + i) : both(__int_as_float(0x7fc00000)));
    };
    int64_t off = 0;
    const int64_t page = A.S.page_of(slot, off);
    if (h == 0 && lane == 0) {
      if (!ok && (A.Hq > 0 || page >= 0)) atomicOr(A.err, kErrBadPosition);
      if (page == -2) atomicOr(A.err, kErrBadSlot);
    }
    if (h < A.Hq) {
      T* dst = A.qo + t * A.ldqo + (int64_t)h * A.D;
      for (int i = lane; i < half; i += 32) {
        const float2 v = pair(i);
        dst[IL ? 2 * i : i] = from_f32<T>(v.x);
        dst[IL ? 2 * i + 1 : half + i] = from_f32<T>(v.y);
      }
      continue;
    }
    if (page < 0) continue;
    uint32_t m = 0;
    for (int i = lane; i < half; i += 32) {
      const float2 v = pair(i);
      m = max(m, max(abs_bits(v.x), abs_bits(v.y)));
    }
    m = group_max<32>(m);
    const float am = q8_amax(m), inv = q8_inv<FMT>(am);
    const bool isk = h < HR;
    const int hk = h - (isk ? A.Hq : HR);
    uint8_t* dst = isk ? A.K.q + A.K.cq.at(page, off, hk) : A.V.q + A.V.cq.at(page, off, hk);
    for (int i = lane; i < half; i += 32) {
      const float2 v = pair(i);
      dst[IL ? 2 * i : i] = (uint8_t)q8_code1<FMT>(v.x, inv);
      dst[IL ? 2 * i + 1 : half + i] = (uint8_t)q8_code1<FMT>(v.y, inv);
    }
    if (lane == 0)
      *(isk ? A.K.sc + A.K.cs.at(page, off, hk) : A.V.sc + A.V.cs.at(page, off, hk)) = q8_scale<FMT>(am, m);
  }
}

// ---------------------------------------------------------------------------
// Read-back: a warp per token (several, where their heads leave lanes over), then
// the next one (the slot of which it has loaded by then).  A unit is N consecutive codes of one head: on the vector path
// as many as fill a 16-byte store (8 codes at bf16, 4 at float32), so that a
// warp's loads and its stores are both contiguous.  A head takes a power of two of
// lanes, which spares the units a division; four heads per lane of K and of V are
// in flight, in one block of code without branches (with a branch per load the
// INT8 form waited 40% longer).  66 us for 65536 tokens of 8 heads of 128, 60 us
// at the copy rate; two heads per lane at five blocks per SM 79, eight at two 76.
// ---------------------------------------------------------------------------
template <typename T>
struct ReadArgs {
  Slots S;
  Cache K, V;
  T* ko;
  T* vo;
  int64_t rows;
  int Hk, D;
  int64_t ldk, ldv;
  unsigned int* err;
};

// Blocks per SM, all resident: three at four heads of K and V per lane, four below.
constexpr int read_blocks(int heads) { return heads == 4 ? 3 : 4; }

template <typename T, int FMT, int N, int U>
__global__ void __launch_bounds__(256) cache8_read_kernel(const ReadArgs<T> A, int per, int lg, int lt) {
  const int lane = threadIdx.x & 31;
  const int64_t step = ((int64_t)gridDim.x * (blockDim.x >> 5)) << lt;
  int64_t t0 = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) << lt;
  if (t0 >= A.rows) return;  // uniform per warp
  // the lanes of a group take a head of one of the warp's 2^lt tokens
  const int lanes = 1 << lg, G = 32 >> (lg + lt);
  const int sub = (lane >> lg) >> (5 - lg - lt), hb = (lane >> lg) & (G - 1);
  const int d0 = lane & (lanes - 1);
  const bool lead = (lane & ((32 >> lt) - 1)) == 0;
  int64_t off = 0, page = -1;
  if (t0 + sub < A.rows) page = A.S.page_of(__ldg(A.S.slots + t0 + sub), off);
#pragma unroll 1
  for (; t0 < A.rows; t0 += step) {
    const int64_t t = t0 + sub;
    const int64_t next = t + step < A.rows ? __ldg(A.S.slots + t + step) : -1;
    if (t < A.rows) {
      T *ko = A.ko + t * A.ldk, *vo = A.vo + t * A.ldv;
      if (page >= 0) {
        const uint8_t *kq = A.K.q + A.K.cq.at(page, off, 0), *vq = A.V.q + A.V.cq.at(page, off, 0);
        const float *ks = A.K.sc + A.K.cs.at(page, off, 0), *vs = A.V.sc + A.V.cs.at(page, off, 0);
        for (int d = d0; d < per; d += lanes) {  // once, for heads of up to 32 units
          for (int h0 = hb; h0 < A.Hk; h0 += U * G) {
            Codes<FMT, N> kw[U], vw[U];
            float kc[U], vc[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
              const int h = min(h0 + j * G, A.Hk - 1);  // past the last head: that one again, not stored
              kw[j].load(kq + h * A.K.cq.head + d * N);
              vw[j].load(vq + h * A.V.cq.head + d * N);
              kc[j] = __ldg(ks + h * A.K.cs.head);
              vc[j] = __ldg(vs + h * A.V.cs.head);
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
              const int h = h0 + j * G;
              if (h < A.Hk) {
                float v[N];
                kw[j].get(v, kc[j]);
                store_n<T, N>(ko + h * A.D + d * N, v);
                vw[j].get(v, vc[j]);
                store_n<T, N>(vo + h * A.D + d * N, v);
              }
            }
          }
        }
      } else {  // no slot: zeros; a slot outside the cache: NaN
        if (page == -2 && lead) atomicOr(A.err, kErrBadSlot);
        float fill[N];
#pragma unroll
        for (int e = 0; e < N; ++e) fill[e] = page == -2 ? __int_as_float(0x7fc00000) : 0.f;
        for (int d = d0; d < per; d += lanes)
          for (int h = hb; h < A.Hk; h += G) {
            store_n<T, N>(ko + h * A.D + d * N, fill);
            store_n<T, N>(vo + h * A.D + d * N, fill);
          }
      }
    }
    page = A.S.page_of(next, off);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Whether runs of n values of a head row, and their codes, are aligned.
template <typename T>
bool runs_fit(const WriteArgs<T>& A, const gbln_cache8* k, const gbln_cache8* v, int n) {
  const auto row = [&](const void* p, int64_t ld) { return aligned_to(p, n * sizeof(T)) && ld % n == 0; };
  return A.D % (2 * n) == 0 && A.D / (2 * n) <= 32 && aligned16(A.table) && codes_aligned(k, v, n) &&
         (A.Hq == 0 || (row(A.q, A.ldq) && row(A.qo, A.ldqo))) && row(A.k, A.ldk) && row(A.v, A.ldv);
}

template <typename T, bool IL, int FMT, int VEC>
gbln_status write_vec_launch(const WriteArgs<T>& A, int sms, cudaStream_t s) {
  WriteShape W{};
  W.nu = A.D / (2 * VEC);
  while ((1 << W.lg) < W.nu) ++W.lg;
  const int lgG = 5 - W.lg, G = 1 << lgG;
  // log2 of the tokens whose n heads share a warp's G groups
  const auto tokens = [&](int n) {
    int lt = lgG;
    while (lt > 0 && (n << lt) > G) --lt;
    return lt;
  };
  const int Lq = (A.Hq + G - 1) / G, Lk = (A.Hk + G - 1) / G;  // head rows per lane and token
  constexpr int FQ = few_queries(VEC * sizeof(T));
  const int finer = (Lq + FQ - 1) / FQ + Lk;  // warps per token (and as many tokens as share one)
  const bool few = (Lq <= FQ && Lk <= 1) || A.rows * finer <= (int64_t)sms * kFewBlocks * kWriteWarps;
  const int QP = few ? FQ : kWriteQ;
  W.nq = (Lq + QP - 1) / QP;
  W.qch = W.nq ? (Lq + W.nq - 1) / W.nq : 0;
  W.qlt = W.nq ? tokens(A.Hq) : 0;
  W.nkv = few ? Lk : (Lk + 1) / 2;
  W.kch = (Lk + W.nkv - 1) / W.nkv;
  W.klt = tokens(A.Hk);
  const int n = W.nq + W.nkv, cy = n < kWriteWarps ? n : kWriteWarps, tz = kWriteWarps / cy;
  const dim3 grid(grid_for(A.rows, tz, (int64_t)sms * kWriteGrid), (unsigned)((n + cy - 1) / cy)), block(32, cy, tz);
  if (few) cache8_write_vec<T, IL, FMT, VEC, 1, FQ><<<grid, block, 0, s>>>(A, W);
  else if (W.kch == 1) cache8_write_vec<T, IL, FMT, VEC, 1, kWriteQ><<<grid, block, 0, s>>>(A, W);
  else cache8_write_vec<T, IL, FMT, VEC, 2, kWriteQ><<<grid, block, 0, s>>>(A, W);
  return launch_status();
}

// 16-byte runs where the sizes and addresses allow them, else 8-byte ones (heads of
// 40, 72 or 200 bf16 values), else single values.
template <typename T, bool IL, int FMT>
gbln_status write_launch(const WriteArgs<T>& A, const gbln_cache8* kc, const gbln_cache8* vc, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const int HT = A.Hq + 2 * A.Hk;
  const int sms = sm_count();
  if (sms <= 0) return GBLN_ERR_CUDA;
  if (HT <= kMaxVecHeads) {
    if (runs_fit(A, kc, vc, VEC)) return write_vec_launch<T, IL, FMT, VEC>(A, sms, s);
    if constexpr (VEC == 8)
      if (runs_fit(A, kc, vc, 4)) return write_vec_launch<T, IL, FMT, 4>(A, sms, s);
  }
  const int64_t items = A.rows * (A.D > kElemWidth ? HT : (HT + kElemHeads - 1) / kElemHeads);  // one per warp
  const unsigned grid = grid_for(items, 8, 1 << 20);
  const bool small = items <= 0xffffffffLL;
  if (A.D <= 64) cache8_write_elem<T, IL, FMT, 1><<<grid, 256, 0, s>>>(A, small);
  else if (A.D <= 128) cache8_write_elem<T, IL, FMT, 2><<<grid, 256, 0, s>>>(A, small);
  else if (A.D <= kElemWidth) cache8_write_elem<T, IL, FMT, 4><<<grid, 256, 0, s>>>(A, small);
  else cache8_write_wide<T, IL, FMT><<<grid, 256, 0, s>>>(A, small);
  return launch_status();
}

template <typename T>
gbln_status write_typed(const WriteArgs<T>& A, bool il, int fmt, const gbln_cache8* kc, const gbln_cache8* vc,
                        cudaStream_t s) {
  if (fmt == GBLN_Q8_INT8)
    return il ? write_launch<T, true, GBLN_Q8_INT8>(A, kc, vc, s) : write_launch<T, false, GBLN_Q8_INT8>(A, kc, vc, s);
  return il ? write_launch<T, true, GBLN_Q8_E4M3>(A, kc, vc, s) : write_launch<T, false, GBLN_Q8_E4M3>(A, kc, vc, s);
}

template <typename T>
gbln_status read_typed(const ReadArgs<T>& A, int fmt, bool cache_aligned, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const bool vec = A.D % VEC == 0 && cache_aligned && aligned16(A.ko) && aligned16(A.vo) &&
                   (A.ldk * (int64_t)sizeof(T)) % 16 == 0 && (A.ldv * (int64_t)sizeof(T)) % 16 == 0;
  const int sms = sm_count();
  if (sms <= 0) return GBLN_ERR_CUDA;
  const int per = A.D / (vec ? VEC : 1);  // units per head
  int lg = 0;
  while (lg < 5 && (1 << lg) < per) ++lg;
  int lt = 5 - lg;  // log2 of the tokens whose heads share a warp's groups
  while (lt > 0 && ((int64_t)A.Hk << (lt + lg)) > 32) --lt;
  const int G = 32 >> (lg + lt), steps = (A.Hk + G - 1) / G;  // heads per lane
  const int64_t warps = (A.rows + (1 << lt) - 1) >> lt;
#define GBLN_READ8_U(FMT, N, U) \
  cache8_read_kernel<T, FMT, N, U><<<grid_for(warps, 8, (int64_t)sms * read_blocks(U)), 256, 0, s>>>(A, per, lg, lt)
#define GBLN_READ8(FMT, N)                  \
  do {                                      \
    if (steps == 1) GBLN_READ8_U(FMT, N, 1);      \
    else if (steps == 2) GBLN_READ8_U(FMT, N, 2); \
    else GBLN_READ8_U(FMT, N, 4);                 \
  } while (0)
  if (fmt == GBLN_Q8_INT8) {
    if (vec) GBLN_READ8(GBLN_Q8_INT8, VEC);
    else GBLN_READ8(GBLN_Q8_INT8, 1);
  } else {
    if (vec) GBLN_READ8(GBLN_Q8_E4M3, VEC);
    else GBLN_READ8(GBLN_Q8_E4M3, 1);
  }
#undef GBLN_READ8
#undef GBLN_READ8_U
  return launch_status();
}

}  // namespace

}  // namespace gbln

using namespace gbln;

extern "C" gbln_status gbln_rope_fwd_cache8(const void* q, const void* k, const void* v, void* q_out,
                                            const int32_t* positions, const float* cos_sin,
                                            int64_t max_pos, const int64_t* slots,
                                            const gbln_cache8* k_cache, const gbln_cache8* v_cache,
                                            int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_q,
                                            int64_t ld_k, int64_t ld_v, int64_t ld_q_out,
                                            gbln_rope_pairing pairing, gbln_q8 fmt, gbln_dtype io,
                                            gbln_stream_t stream) {
  if (!dtype_ok(io) || !q8_ok(fmt) || (pairing != GBLN_ROPE_HALF && pairing != GBLN_ROPE_INTERLEAVED))
    return GBLN_ERR_INVALID_ARG;
  if (T < 0 || T > kMaxTokens || Hq < 0 || Hk <= 0 || D <= 0 || (D & 1) || max_pos < 0) return GBLN_ERR_INVALID_ARG;
  if (((int64_t)Hq + 2 * (int64_t)Hk) * D > (1 << 24)) return GBLN_ERR_INVALID_ARG;
  const int64_t qw = (int64_t)Hq * D, kw = (int64_t)Hk * D;
  if ((Hq > 0 && (!ld_fits(T, qw, ld_q) || !ld_fits(T, qw, ld_q_out))) || !ld_fits(T, kw, ld_k) || !ld_fits(T, kw, ld_v))
    return GBLN_ERR_INVALID_ARG;
  if (!cache_ok(k_cache, Hk, D) || !cache_ok(v_cache, Hk, D)) return GBLN_ERR_INVALID_ARG;
  if (k_cache->pages != v_cache->pages || k_cache->page_size != v_cache->page_size) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!k || !v || !positions || !cos_sin || !slots || (Hq > 0 && (!q || !q_out))) return GBLN_ERR_INVALID_ARG;
  if (k_cache->pages > 0 && (!k_cache->codes || !k_cache->scale || !v_cache->codes || !v_cache->scale))
    return GBLN_ERR_INVALID_ARG;
  if (!aligned_to(cos_sin, 8) || !aligned_to(slots, 8)) return GBLN_ERR_INVALID_ARG;  // float2, int64
  // one cache for both would leave either's codes with the other's scale
  if (k_cache->pages > 0 && (k_cache->codes == v_cache->codes || k_cache->scale == v_cache->scale)) return GBLN_ERR_INVALID_ARG;
  unsigned int* err = device_error_word();
  if (!err) return GBLN_ERR_CUDA;
  const bool il = pairing == GBLN_ROPE_INTERLEAVED;
  cudaStream_t s = (cudaStream_t)stream;
#define GBLN_WRITE_ARGS(TY)                                                                               \
  const WriteArgs<TY> A{(const TY*)q, (const TY*)k, (const TY*)v, (TY*)q_out, positions, (const float2*)cos_sin, \
                        max_pos, T, Hq, Hk, D, ld_q, ld_k, ld_v, ld_q_out, slots_of(k_cache, slots),       \
                        cache_of(k_cache), cache_of(v_cache), err}
  if (io == GBLN_F32) {
    GBLN_WRITE_ARGS(float);
    return write_typed<float>(A, il, fmt, k_cache, v_cache, s);
  }
  GBLN_WRITE_ARGS(bf16);
  return write_typed<bf16>(A, il, fmt, k_cache, v_cache, s);
#undef GBLN_WRITE_ARGS
}

extern "C" gbln_status gbln_cache8_read(const int64_t* slots, const gbln_cache8* k_cache,
                                        const gbln_cache8* v_cache, void* k_out, void* v_out, int64_t T,
                                        int32_t Hk, int32_t D, int64_t ld_k_out, int64_t ld_v_out,
                                        gbln_q8 fmt, gbln_dtype io, gbln_stream_t stream) {
  if (!dtype_ok(io) || !q8_ok(fmt)) return GBLN_ERR_INVALID_ARG;
  if (T < 0 || T > kMaxTokens || Hk <= 0 || D <= 0) return GBLN_ERR_INVALID_ARG;
  if (2 * (int64_t)Hk * D > (1 << 24)) return GBLN_ERR_INVALID_ARG;
  const int64_t kw = (int64_t)Hk * D;
  if (!ld_fits(T, kw, ld_k_out) || !ld_fits(T, kw, ld_v_out)) return GBLN_ERR_INVALID_ARG;
  if (!cache_ok(k_cache, Hk, D) || !cache_ok(v_cache, Hk, D)) return GBLN_ERR_INVALID_ARG;
  if (k_cache->pages != v_cache->pages || k_cache->page_size != v_cache->page_size) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!slots || !k_out || !v_out || !aligned_to(slots, 8)) return GBLN_ERR_INVALID_ARG;
  if (k_cache->pages > 0 && (!k_cache->codes || !k_cache->scale || !v_cache->codes || !v_cache->scale))
    return GBLN_ERR_INVALID_ARG;
  unsigned int* err = device_error_word();
  if (!err) return GBLN_ERR_CUDA;
  const bool ca = codes_aligned(k_cache, v_cache, io == GBLN_F32 ? 4 : 8);
  cudaStream_t s = (cudaStream_t)stream;
#define GBLN_READ_ARGS(TY)                                                                             \
  const ReadArgs<TY> A{slots_of(k_cache, slots), cache_of(k_cache), cache_of(v_cache), (TY*)k_out, (TY*)v_out, \
                       T, Hk, D, ld_k_out, ld_v_out, err}
  if (io == GBLN_F32) {
    GBLN_READ_ARGS(float);
    return read_typed<float>(A, fmt, ca, s);
  }
  GBLN_READ_ARGS(bf16);
  return read_typed<bf16>(A, fmt, ca, s);
#undef GBLN_READ_ARGS
}
