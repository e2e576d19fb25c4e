// What stands between the QKV projection and attention, in one pass: the RMSNorm of
// every head of Q and K (optional), the rotary embedding with one to four position
// axes, and (serving) K and V quantised into the paged 8-bit cache; the backward
// pass of norm and rotation with the gradients of both norm weights.
//
// Operator: "Fast-LLM: 高效大语言模型训练框架", §三 框架结构 (attention with RoPE; heads /
// head_groups / head_size) and 训练配置示例 (rms_norm, rotary); "LLaMA-Factory Kernels 系统"
// (fused RMSNorm, fused RoPE); one pass instead of two, as "Kernels（自定义内核）" §Liger.
//
// With x one head of one token, w its weight, (c, s) the turn of a pair:
//   u = (x rstd) w,  rstd = 1 / sqrt(mean x^2 + eps),  y = (u1 c - u2 s, u2 c + u1 s)
// and with d = dy turned back and g = d w:
//   dx = rstd (g - n mean(g n)),  n = x rstd,  dW = sum over tokens and heads of d n.
// rstd is not stored: the backward pass reads x anyway, and the sums of x^2 and g x
// go through the same shuffles.  HBM-bound: forward 2, backward 3 accesses per value.
// Measured, bf16 heads of 128: 32761 tokens of 64 / 8 heads with three axes 212 us forward, 349
// backward (84 and 76% of the copy rate); 16384 of 16 / 8 heads 48 and 65 us (62 and 68%: issue slots
// half used, warps waiting for their rows); axes alone, 65536 of 32 / 8 heads 205 us (96%); the
// cache's write, 32768 tokens of 32 / 8 heads, three axes, 152 us.

#include <type_traits>

#include "cache8.cuh"

namespace gbln {

namespace {

constexpr int kAxes = 4;         // position axes
constexpr int kMaxHead = 512;    // values of a head
constexpr int kHeadWarps = 8;    // per block
constexpr int kMaxRows = 4096;   // heads of a token on the vector path

// The position axis of each pair, two bits each.
struct AxisMap {
  uint32_t bits[kMaxHead / 2 / 16];
  int n;
  int64_t ld;  // between the axes' position rows
  // of `run` pairs from i on (they lie in one word)
  __device__ __forceinline__ uint32_t of(int i, int run) const {
    return (bits[i >> 4] >> (2 * (i & 15))) & ((1u << (2 * run)) - 1u);
  }
};

template <typename T>
struct HeadArgs {
  const T* q;
  const T* k;
  const T* v;
  T* qo;
  T* ko;
  const T* dq;  // backward: the gradients of the rotated heads
  const T* dk;
  const void* wq;  // null: no norm
  const void* wk;
  float* part;  // [P, 2 D]
  const int32_t* pos;
  const float2* table;
  int64_t max_pos, rows;
  int64_t ldq, ldk, ldv, ldqo, ldko, lddq, lddk;
  int Hq, Hk, D;
  float eps, sign;  // sign of the angles
  int w32;          // weights are float32
  AxisMap ax;
  Slots S;
  Cache K, V;
  unsigned int* err;
};

struct Pos {
  int p[kAxes];
  __device__ __forceinline__ void load(const int32_t* pos, const AxisMap& ax, int64_t t) {
    p[0] = __ldg(pos + t);
#pragma unroll
    for (int a = 1; a < kAxes; ++a) p[a] = a < ax.n ? __ldg(pos + a * ax.ld + t) : p[0];
  }
  __device__ __forceinline__ bool ok(int64_t max_pos) const {
    bool r = true;
#pragma unroll
    for (int a = 0; a < kAxes; ++a) r = r && p[a] >= 0 && (int64_t)p[a] < max_pos;
    return r;
  }
  __device__ __forceinline__ int at(uint32_t axis) const {
    const int lo = axis & 1 ? p[1] : p[0], hi = axis & 1 ? p[3] : p[2];
    return axis & 2 ? hi : lo;
  }
};

// (cos, sin) of a lane's pairs: entries ia.. (rotate-half), or half as many for each of
// its two vectors (interleaved); NaN where a position is outside the table.  One axis
// reads two entries at a time; several read each pair's entry from its axis' row.
template <int VEC, bool IL>
__device__ __forceinline__ void load_axes(const float2* table, int half, const Pos& p, const AxisMap& ax, uint32_t codes,
                                          bool ok, bool on, int ia, float sign, float2 (&cs)[VEC]) {
  if (ok && on) {
    if (ax.n == 1) {
      const float2* e = table + (size_t)p.p[0] * half;
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        const int at = !IL ? ia + i : i < VEC / 2 ? ia / 2 + i : (half + ia) / 2 + i - VEC / 2;
        const float4 f = __ldg(reinterpret_cast<const float4*>(e + at));
        cs[i] = make_float2(f.x, f.y);
        cs[i + 1] = make_float2(f.z, f.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int at = !IL ? ia + i : i < VEC / 2 ? ia / 2 + i : (half + ia) / 2 + i - VEC / 2;
        cs[i] = __ldg(table + (size_t)p.at(codes >> (2 * i)) * half + at);
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) cs[i].y *= sign;
  } else {
    const float x = ok ? 0.f : __int_as_float(0x7fc00000);
#pragma unroll
    for (int i = 0; i < VEC; ++i) cs[i] = make_float2(x, x);
  }
}

// turn() two values an instruction: the same roundings, each for itself.
template <int VEC, bool IL>
__device__ __forceinline__ void turn2(float (&xa)[VEC], float (&xb)[VEC], const float2 (&cs)[VEC]) {
  if constexpr (IL) {
    turn<VEC, true>(xa, xb, cs);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 a = make_float2(xa[e], xa[e + 1]), b = make_float2(xb[e], xb[e + 1]);
      const float2 c = make_float2(cs[e].x, cs[e + 1].x), s = make_float2(cs[e].y, cs[e + 1].y);
      const float2 p = mul2(b, s), y = fma2(a, c, make_float2(-p.x, -p.y)), z = fma2(b, c, mul2(a, s));
      xa[e] = y.x;
      xa[e + 1] = y.y;
      xb[e] = z.x;
      xb[e + 1] = z.y;
    }
  }
}
// v times r, then times w (each product rounded); without r: times w.
template <int VEC>
__device__ __forceinline__ void times(float (&v)[VEC], const float (&w)[VEC], float r) {
#pragma unroll
  for (int e = 0; e < VEC; e += 2) {
    const float2 y = mul2(mul2(make_float2(v[e], v[e + 1]), both(r)), make_float2(w[e], w[e + 1]));
    v[e] = y.x;
    v[e + 1] = y.y;
  }
}
template <int VEC>
__device__ __forceinline__ void times(float (&v)[VEC], const float (&w)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; e += 2) {
    const float2 y = mul2(make_float2(v[e], v[e + 1]), make_float2(w[e], w[e + 1]));
    v[e] = y.x;
    v[e + 1] = y.y;
  }
}

__device__ __forceinline__ float weight_at(const void* w, int w32, int i) {
  return w32 ? __ldg((const float*)w + i) : to_f32(((const bf16*)w)[i]);
}
// VEC weights from i on; single loads where the weights are not aligned (w16).
template <int VEC>
__device__ __forceinline__ void weights_at(const void* w, int w32, bool w16, int i, float (&v)[VEC]) {
  if (!w16) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = weight_at(w, w32, i + e);
  } else if (w32) {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>((const float*)w + i + e));
      v[e] = f.x;
      v[e + 1] = f.y;
      v[e + 2] = f.z;
      v[e + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const uint2 f = __ldg(reinterpret_cast<const uint2*>((const bf16*)w + i + e));
      v[e] = bf16_lo(f.x);
      v[e + 1] = bf16_hi(f.x);
      v[e + 2] = bf16_lo(f.y);
      v[e + 3] = bf16_hi(f.y);
    }
  }
}
template <int VEC>
__device__ __forceinline__ void load_weights(const void* w, int w32, int ia, int half, bool on, float (&wa)[VEC], float (&wb)[VEC]) {
  if (w && on) {
    const bool w16 = (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
    weights_at<VEC>(w, w32, w16, ia, wa);
    weights_at<VEC>(w, w32, w16, half + ia, wb);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) wa[e] = wb[e] = 1.f;
  }
}
template <int VEC>
__device__ __forceinline__ float sum_squares(const float (&a)[VEC], const float (&b)[VEC]) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < VEC; e += 2) {
    s = fma2(make_float2(a[e], a[e + 1]), make_float2(a[e], a[e + 1]), s);
    s = fma2(make_float2(b[e], b[e + 1]), make_float2(b[e], b[e + 1]), s);
  }
  return s.x + s.y;
}
__device__ __forceinline__ float rstd_of(float sum, int D, float eps) {
  return rsqrtf(__fadd_rn(__fdiv_rn(sum, (float)D), eps));
}

// How a launch's warps share the work: every token has nq chunks of query head rows
// and nk of K (and V) head rows; warp w of all has chunk w % (nq + nk) of the tokens
// w / (nq + nk), that + stride, ...  Neighbouring warps so read one token's row together.
// (Warps given to the two kinds by their rows, the kinds apart, wasted none of them on small
// chunks, but read Q and K of a token at different times: 65536 tokens of 32 / 8 heads of 128, axes alone, 230 and 244 us at the time.)
struct Split {
  int nu, lg;         // lanes in use per head row, log2 of the lanes of its group
  int nq, qch, qlt;   // chunks, head rows per lane in each, log2 of the tokens a warp takes at once
  int nk, kch, klt;
  int64_t stride;     // warps per chunk
};

// The lane's place in its warp's work.
struct Place {
  int v, ia, G, sub, g, li, lt;
  bool on;
  __device__ __forceinline__ Place(const Split& W, int lt_, int VEC) : lt(lt_) {
    const int lane = threadIdx.x & 31;
    v = lane & ((1 << W.lg) - 1);
    on = v < W.nu;
    ia = v * VEC;
    G = 32 >> (W.lg + lt);
    sub = (lane >> W.lg) >> (5 - W.lg - lt);
    g = (lane >> W.lg) & (G - 1);
    li = lane & ((32 >> lt) - 1);
  }
};

// Whole-warp: ask for the head rows hf .. of token n in L2.
template <typename T>
__device__ __forceinline__ void ask_ahead(const T* row, int first, int last, int li, int lanes) {
  constexpr int LINE = 128 / sizeof(T);
  for (int x = first + li * LINE; x < last; x += lanes * LINE) prefetch_line(row + x);
}

// ---------------------------------------------------------------------------
// Forward, vector path.  A lane owns the vectors at ia = v VEC of both halves of a head
// row, whichever pairing (as the cache's write), and keeps the weights and turns of its
// pairs across the rows it takes: up to NQ rows of Q (or of K where it is not cached),
// or KP heads of K and V to be quantised.  All row loads of a pass are issued before
// anything depends on them; the sums of all rows go through the shuffles side by side.
// ---------------------------------------------------------------------------
template <typename T, bool IL, int VEC, int NQ, bool NORM>
__device__ __forceinline__ void heads_rows(const HeadArgs<T>& A, const Split& W, const T* x, int64_t ldx, T* y, int64_t ldy,
                                           const void* w, int H, int c, int ch, int lt, int64_t first, bool report) {
  using Run = HeadRun<T, VEC>;
  const Place P(W, lt, VEC);
  const int half = A.D / 2, lanes = 1 << W.lg;
  const int hf = P.G * c * ch, hb = hf + P.g;
  const int last = min(hf + P.G * ch, H) * A.D;
  const int64_t end = A.rows - 1, step = W.stride << lt;
  int64_t t0 = first << lt;
  if (t0 >= A.rows) return;
  uint32_t codes = 0;
  if (A.ax.n > 1 && P.on)
    codes = !IL ? A.ax.of(P.ia, VEC) : A.ax.of(P.ia / 2, VEC / 2) | A.ax.of((half + P.ia) / 2, VEC / 2) << VEC;
  Pos p;
  p.load(A.pos, A.ax, min(t0 + P.sub, end));
  float wa[VEC], wb[VEC];
  bool have = false;  // the weights: asked for behind the first rows, as most warps have one step
#pragma unroll 1
  for (; t0 < A.rows; t0 += step) {
    const int64_t t = t0 + P.sub;
    const bool live = P.on && t < A.rows;
    const T* src = x + min(t, end) * ldx + P.ia;
    T* dst = y + min(t, end) * ldy + P.ia;
    Run a[NQ], b[NQ];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const int h = hb + P.G * j;
      a[j].zero();
      b[j].zero();
      if (j < ch && live && h < H) {
        a[j].load(src + h * A.D);
        b[j].load(src + h * A.D + half);
      }
    }
    if constexpr (NORM) {
      if (!have) load_weights<VEC>(w, A.w32, P.ia, half, P.on, wa, wb);
      have = true;
    }
    const bool ok = p.ok(A.max_pos);
    float2 cs[VEC];
    load_axes<VEC, IL>(A.table, half, p, A.ax, codes, ok, P.on, P.ia, A.sign, cs);
    if (!ok && live && report && P.li == 0) atomicOr(A.err, kErrBadPosition);
    if (t0 + step < A.rows) {  // the warp's next tokens
      const int64_t n = min(t + step, end);
      p.load(A.pos, A.ax, n);
      ask_ahead(x + n * ldx, hf * A.D, last, P.li, 32 >> lt);
    }
    float ss[NQ];
    if (NORM && w) {
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        float xa[VEC], xb[VEC];
        a[j].get(xa);
        b[j].get(xb);
        ss[j] = sum_squares<VEC>(xa, xb);
      }
      for (int o = 1; o < lanes; o <<= 1)
#pragma unroll
        for (int j = 0; j < NQ; ++j) ss[j] += __shfl_xor_sync(0xffffffffu, ss[j], o);
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      const int h = hb + P.G * j;
      if (j < ch && live && h < H) {
        float xa[VEC], xb[VEC];
        a[j].get(xa);
        b[j].get(xb);
        if (NORM && w) {
          const float r = rstd_of(ss[j], A.D, A.eps);
          times<VEC>(xa, wa, r);
          times<VEC>(xb, wb, r);
        }
        turn2<VEC, IL>(xa, xb, cs);
        Run::store(dst + h * A.D, xa);
        Run::store(dst + h * A.D + half, xb);
      }
    }
  }
}

template <typename T, bool IL, int FMT, int VEC, int KP>
__device__ __forceinline__ void heads_cache(const HeadArgs<T>& A, const Split& W, int c, int64_t first) {
  using Run = HeadRun<T, VEC>;
  const Place P(W, W.klt, VEC);
  const int half = A.D / 2, lanes = 1 << W.lg, lane = threadIdx.x & 31;
  const int hf = P.G * c * W.kch, hb = hf + P.g;
  const int last = min(hf + P.G * W.kch, A.Hk) * A.D;
  const int64_t end = A.rows - 1, step = W.stride << P.lt;
  int64_t t0 = first << P.lt;
  if (t0 >= A.rows) return;
  uint32_t codes = 0;
  if (A.ax.n > 1 && P.on)
    codes = !IL ? A.ax.of(P.ia, VEC) : A.ax.of(P.ia / 2, VEC / 2) | A.ax.of((half + P.ia) / 2, VEC / 2) << VEC;
  Pos p;
  p.load(A.pos, A.ax, min(t0 + P.sub, end));
  int64_t slot = __ldg(A.S.slots + min(t0 + P.sub, end));
  float wa[VEC], wb[VEC];
  bool have = false;
#pragma unroll 1
  for (; t0 < A.rows; t0 += step) {
    const int64_t t = t0 + P.sub;
    const bool live = P.on && t < A.rows;
    const T *kp = A.k + min(t, end) * A.ldk, *vp = A.v + min(t, end) * A.ldv;
    constexpr int N = 2 * KP;  // K of each head, then V of each
    Run a[N], b[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int h = hb + P.G * (j % KP);
      a[j].zero();
      b[j].zero();
      if (j % KP < W.kch && live && h < A.Hk) {
        const T* src = (j < KP ? kp : vp) + h * A.D + P.ia;
        a[j].load(src);
        b[j].load(src + half);
      }
    }
    if (!have) load_weights<VEC>(A.wk, A.w32, P.ia, half, P.on, wa, wb);
    have = true;
    const bool ok = p.ok(A.max_pos);
    float2 cs[VEC];
    load_axes<VEC, IL>(A.table, half, p, A.ax, codes, ok, P.on, P.ia, 1.f, cs);
    int64_t off = 0;
    const int64_t page = A.S.page_of(slot, off);
    if (c == 0 && P.li == 0 && live) {
      if (!ok && page >= 0) atomicOr(A.err, kErrBadPosition);
      if (page == -2) atomicOr(A.err, kErrBadSlot);
    }
    if (t0 + step < A.rows) {  // the warp's next tokens
      const int64_t n = min(t + step, end);
      p.load(A.pos, A.ax, n);
      slot = __ldg(A.S.slots + n);
      ask_ahead(A.k + n * A.ldk, hf * A.D, last, P.li, 32 >> P.lt);
      ask_ahead(A.v + n * A.ldv, hf * A.D, last, P.li, 32 >> P.lt);
    }
    float xa[N][VEC], xb[N][VEC], ss[KP];
    uint32_t m[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      a[j].get(xa[j]);
      b[j].get(xb[j]);
      if (j < KP) {
        ss[j] = sum_squares<VEC>(xa[j], xb[j]);
        times<VEC>(xa[j], wa);  // rstd is the head's: it goes into the scale
        times<VEC>(xb[j], wb);
        turn2<VEC, IL>(xa[j], xb[j], cs);
      }
      m[j] = P.on ? max(abs_max_bits<VEC>(xa[j]), abs_max_bits<VEC>(xb[j])) : 0u;
    }
    for (int o = 1; o < lanes; o <<= 1) {
#pragma unroll
      for (int j = 0; j < N; ++j) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], o));
#pragma unroll
      for (int j = 0; j < KP; ++j) ss[j] += __shfl_xor_sync(0xffffffffu, ss[j], o);
    }
    float inv[N], sc[N], r[KP];
#pragma unroll
    for (int j = 0; j < KP; ++j) r[j] = A.wk ? rstd_of(ss[j], A.D, A.eps) : 1.f;
    if (lanes >= 2 * N) {
      // lanes 2 j and 2 j + 1 of a group divide for 1 / scale and for the scale of j
      uint32_t mine = m[0];
      float mr = r[0];
#pragma unroll
      for (int j = 1; j < N; ++j)
        if (((lane >> 1) & (N - 1)) == j) {
          mine = m[j];
          mr = j < KP ? r[j < KP ? j : 0] : 1.f;
        }
      const float am = q8_amax(mine);
      const float d = __fdiv_rn(lane & 1 ? __fmul_rn(am, mr) : Q8Max<FMT>::v, lane & 1 ? Q8Max<FMT>::v : am);
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
        sc[j] = __fdiv_rn(j < KP ? __fmul_rn(am, r[j < KP ? j : 0]) : am, Q8Max<FMT>::v);
      }
    }
    if (page < 0 || !live) continue;  // nothing to store; no shuffles below
    const int64_t kq = A.K.cq.at(page, off, hb) + P.ia, vq = A.V.cq.at(page, off, hb) + P.ia;
    const int64_t ks = A.K.cs.at(page, off, hb), vs = A.V.cs.at(page, off, hb);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = j % KP;
      if (i < W.kch && hb + P.G * i < A.Hk) {
        const bool isk = j < KP;
        uint8_t* dst = isk ? A.K.q + kq + P.G * i * A.K.cq.head : A.V.q + vq + P.G * i * A.V.cq.head;
        q8_store<FMT, VEC>(xa[j], inv[j], dst);
        q8_store<FMT, VEC>(xb[j], inv[j], dst + half);
        if (P.v == 0)
          *(isk ? A.K.sc + ks + P.G * i * A.K.cs.head : A.V.sc + vs + P.G * i * A.V.cs.head) =
              m[j] < kInfBits ? sc[j] : __int_as_float(0x7fc00000);
      }
    }
  }
}

// Rows per lane and blocks per SM: a large share of a token, or a small one where tokens
// are few or narrow.  (16 tokens of 16 / 8 heads of 128, bf16: small 3.5 us, large 3.8, into the cache 3.9
// and 4.5; 1024 tokens of 64 / 8 float32 heads 13.7 and 12.7, 4096 into the cache 26.1 and 22.2.)
constexpr int kRowsLarge = 4, kRowsSmall = 2, kSmallBlocks = 3;
constexpr int rows_of(bool small, int bytes) { return (small ? kRowsSmall : kRowsLarge) * (16 / bytes); }

// Rotations alone have no weights to hold: three blocks where norms leave room for two (65536 tokens of 32 / 8 heads of
// 128, three axes: 205 us, with two blocks 226).
constexpr int kRotate = -2;  // in the place of a format (-1: no cache): neither cache nor norms
constexpr int fwd_blocks(int fmt, bool small) { return small ? kSmallBlocks : fmt == kRotate ? 3 : 2; }

template <typename T, bool IL, int FMT, int VEC, bool SMALL>
__global__ void __launch_bounds__(32 * kHeadWarps, fwd_blocks(FMT, SMALL))
heads_fwd_vec(const __grid_constant__ HeadArgs<T> A, const Split W) {
  constexpr int NQ = rows_of(SMALL, VEC * sizeof(T));
  const int64_t w = (int64_t)blockIdx.x * kHeadWarps + warp_index();
  const int n = W.nq + W.nk;
  const int64_t first = w / n;
  const int c = (int)(w - first * n);
  if (first >= W.stride) return;
  if (c < W.nq) {
    heads_rows<T, IL, VEC, NQ, FMT != kRotate>(A, W, A.q, A.ldq, A.qo, A.ldqo, A.wq, A.Hq, c, W.qch, W.qlt, first, c == 0);
  } else if constexpr (FMT < 0) {
    heads_rows<T, IL, VEC, NQ, FMT != kRotate>(A, W, A.k, A.ldk, A.ko, A.ldko, A.wk, A.Hk, c - W.nq, W.kch, W.klt, first, c == 0);
  } else {
    heads_cache<T, IL, FMT, VEC, SMALL ? 1 : 2>(A, W, c - W.nq, first);
  }
}

// ---------------------------------------------------------------------------
// Backward, vector path: the same lanes and chunks; a lane adds up d n of its pairs over
// all its rows and tokens, in order, and the block its warps' sums, warp after warp: the
// partial rows are the same on every run.
// ---------------------------------------------------------------------------
template <typename T, bool IL, int VEC, int NB>
__device__ __forceinline__ void heads_rows_bwd(const HeadArgs<T>& A, const Split& W, const Place& P, const T* dy, int64_t ldd,
                                               const T* x, int64_t ldx, T* dx, int64_t ldo, const void* w, int H, int c,
                                               int ch, int64_t first, bool report, float (&da)[VEC], float (&db)[VEC]) {
  using Run = HeadRun<T, VEC>;
  const int half = A.D / 2, lanes = 1 << W.lg;
  const int hf = P.G * c * ch, hb = hf + P.g;
  const int last = min(hf + P.G * ch, H) * A.D;
  const int64_t end = A.rows - 1, step = W.stride << P.lt;
  int64_t t0 = first << P.lt;
  if (t0 >= A.rows) return;
  uint32_t codes = 0;
  if (A.ax.n > 1 && P.on)
    codes = !IL ? A.ax.of(P.ia, VEC) : A.ax.of(P.ia / 2, VEC / 2) | A.ax.of((half + P.ia) / 2, VEC / 2) << VEC;
  Pos p;
  p.load(A.pos, A.ax, min(t0 + P.sub, end));
  float wa[VEC], wb[VEC];
  load_weights<VEC>(w, A.w32, P.ia, half, P.on, wa, wb);
  const float inv_d = 1.f / (float)A.D;
#pragma unroll 1
  for (; t0 < A.rows; t0 += step) {
    const int64_t t = t0 + P.sub;
    const bool live = P.on && t < A.rows;
    const T* gs = dy + min(t, end) * ldd + P.ia;
    const T* xs = x + min(t, end) * ldx + P.ia;
    T* dst = dx + min(t, end) * ldo + P.ia;
    Run ga[NB], gb[NB], ra[NB], rb[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int h = hb + P.G * j;
      ga[j].zero();
      gb[j].zero();
      ra[j].zero();
      rb[j].zero();
      if (j < ch && live && h < H) {
        ga[j].load(gs + h * A.D);
        gb[j].load(gs + h * A.D + half);
        ra[j].load(xs + h * A.D);
        rb[j].load(xs + h * A.D + half);
      }
    }
    const bool ok = p.ok(A.max_pos);
    float2 cs[VEC];
    load_axes<VEC, IL>(A.table, half, p, A.ax, codes, ok, P.on, P.ia, -1.f, cs);
    if (!ok && live && report && P.li == 0) atomicOr(A.err, kErrBadPosition);
    if (t0 + step < A.rows) {  // the warp's next tokens
      const int64_t n = min(t + step, end);
      p.load(A.pos, A.ax, n);
      ask_ahead(dy + n * ldd, hf * A.D, last, P.li, 32 >> P.lt);
      ask_ahead(x + n * ldx, hf * A.D, last, P.li, 32 >> P.lt);
    }
    float s1[NB], s2[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float xa[VEC], xb[VEC], ya[VEC], yb[VEC];
      ra[j].get(xa);
      rb[j].get(xb);
      ga[j].get(ya);
      gb[j].get(yb);
      turn<VEC, IL>(ya, yb, cs);
      s1[j] = sum_squares<VEC>(xa, xb);
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        s = fma2(mul2(make_float2(ya[e], yb[e]), make_float2(wa[e], wb[e])), make_float2(xa[e], xb[e]), s);
      s2[j] = s.x + s.y;
    }
    for (int o = 1; o < lanes; o <<= 1)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        s1[j] += __shfl_xor_sync(0xffffffffu, s1[j], o);
        s2[j] += __shfl_xor_sync(0xffffffffu, s2[j], o);
      }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int h = hb + P.G * j;
      if (j < ch && live && h < H) {
        float xa[VEC], xb[VEC], ya[VEC], yb[VEC];
        ra[j].get(xa);
        rb[j].get(xb);
        ga[j].get(ya);
        gb[j].get(yb);
        turn<VEC, IL>(ya, yb, cs);
        const float r = rstd_of(s1[j], A.D, A.eps);
        const float m = r * s2[j] * inv_d;  // mean(g n)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 n = mul2(make_float2(xa[e], xb[e]), both(r)), d = make_float2(ya[e], yb[e]);
          const float2 acc = fma2(d, n, make_float2(da[e], db[e]));
          da[e] = acc.x;
          db[e] = acc.y;
          const float2 o = mul2(both(r), fma2(n, both(-m), mul2(d, make_float2(wa[e], wb[e]))));
          ya[e] = o.x;
          yb[e] = o.y;
        }
        Run::store(dst + h * A.D, ya);
        Run::store(dst + h * A.D + half, yb);
      }
    }
  }
}

// Add the warps' sums (lane values da, db at element ia of both halves; which = 0 Q, 1 K,
// -1 none) to the block's row of partials, in the order of the warps.
template <int VEC>
__device__ __forceinline__ void flush_dw(float* acc, int D, int which, bool first_group, int ia, const float (&da)[VEC],
                                         const float (&db)[VEC], float* out) {
  for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) acc[i] = 0.f;
  for (int w = 0; w < kHeadWarps; ++w) {
    __syncthreads();
    if ((threadIdx.x >> 5) == w && which >= 0 && first_group) {
      float* a = acc + which * D + ia;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        a[e] += da[e];
        a[D / 2 + e] += db[e];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) out[i] = acc[i];
}

// Two rows of bf16 spill 456 bytes a thread at 128 registers (the compiler keeps the first pass' unpacked rows); float32 none.
// Small where every warp has one chunk at most: 16 tokens of 16 / 8 heads of 128 6.2 us, large 6.9; 4096 23.7 and 19.4.
constexpr int kRowsBwd = 2, kRowsBwdSmall = 1;
constexpr int kBwdBlocks = 2;  // per SM
constexpr int rows_bwd(bool small, int bytes) { return (small ? kRowsBwdSmall : kRowsBwd) * (16 / bytes); }

template <typename T, bool IL, int VEC, bool SMALL>
__global__ void __launch_bounds__(32 * kHeadWarps, kBwdBlocks)
heads_bwd_vec(const __grid_constant__ HeadArgs<T> A, const Split W) {
  constexpr int NB = rows_bwd(SMALL, VEC * sizeof(T));
  __shared__ float acc[2 * kMaxHead];
  const int64_t w = (int64_t)blockIdx.x * kHeadWarps + warp_index();
  const int n = W.nq + W.nk;
  const int64_t first = w / n;
  const int c = (int)(w - first * n);
  const bool isq = c < W.nq, runs = first < W.stride;
  const Place P(W, isq ? W.qlt : W.klt, VEC);
  float da[VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) da[e] = db[e] = 0.f;
  if (runs) {
    if (isq)
      heads_rows_bwd<T, IL, VEC, NB>(A, W, P, A.dq, A.lddq, A.q, A.ldq, A.qo, A.ldqo, A.wq, A.Hq, c, W.qch, first, c == 0, da, db);
    else
      heads_rows_bwd<T, IL, VEC, NB>(A, W, P, A.dk, A.lddk, A.k, A.ldk, A.ko, A.ldko, A.wk, A.Hk, c - W.nq, W.kch, first, c == 0, da, db);
  }
  for (int o = 1 << W.lg; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      da[e] += __shfl_xor_sync(0xffffffffu, da[e], o);
      db[e] += __shfl_xor_sync(0xffffffffu, db[e], o);
    }
  flush_dw<VEC>(acc, A.D, runs ? (isq ? 0 : 1) : -1, P.on && (threadIdx.x & 31) < (1 << W.lg), P.ia, da, db,
                A.part + (size_t)blockIdx.x * 2 * A.D);
}

// ---------------------------------------------------------------------------
// Element path: any alignment and stride.  A warp takes one head row after the other,
// lane l the pairs l, l + 32, ... (K of them).
// ---------------------------------------------------------------------------
template <bool IL, int K>
__device__ __forceinline__ void elem_turns(const float2* table, int half, const Pos& p, const AxisMap& ax, bool ok, float sign,
                                           float2 (&cs)[K]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int i = lane + 32 * k;
    cs[k] = both(ok ? 0.f : __int_as_float(0x7fc00000));
    if (ok && i < half) {
      cs[k] = __ldg(table + (size_t)(ax.n == 1 ? p.p[0] : p.at(ax.of(i, 1))) * half + i);
      cs[k].y *= sign;
    }
  }
}

template <typename T, bool IL, int FMT, int K>
__global__ void __launch_bounds__(256) heads_fwd_elem(const __grid_constant__ HeadArgs<T> A) {
  const int half = A.D / 2, HR = A.Hq + A.Hk, HT = HR + (FMT < 0 ? 0 : A.Hk);
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kHeadWarps;
  for (int64_t item = (int64_t)blockIdx.x * kHeadWarps + warp_index(); item < A.rows * HT; item += step) {
    const int64_t t = item / HT;
    const int h = (int)(item - t * HT);  // uniform per warp, as every test of it
    const T* src = h < A.Hq ? A.q + t * A.ldq + h * A.D : h < HR ? A.k + t * A.ldk + (h - A.Hq) * A.D : A.v + t * A.ldv + (h - HR) * A.D;
    Pos p;
    p.load(A.pos, A.ax, t);
    const bool ok = p.ok(A.max_pos);
    int64_t off = 0, page = 0;
    if constexpr (FMT >= 0) page = A.S.page_of(__ldg(A.S.slots + t), off);
    if (h == 0 && lane == 0) {
      if (!ok && (A.Hq > 0 || page >= 0)) atomicOr(A.err, kErrBadPosition);
      if (page == -2) atomicOr(A.err, kErrBadSlot);
    }
    float2 y[K], cs[K];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = lane + 32 * k;
      y[k] = make_float2(0.f, 0.f);
      if (i < half) y[k] = make_float2(to_f32(src[IL ? 2 * i : i]), to_f32(src[IL ? 2 * i + 1 : half + i]));
      ss = fmaf(y[k].x, y[k].x, fmaf(y[k].y, y[k].y, ss));
    }
    const void* w = h < A.Hq ? A.wq : A.wk;
    const bool stored = FMT >= 0 && h >= A.Hq;  // rstd goes into the scale
    float r = 1.f;
    if (h < HR) {
      elem_turns<IL, K>(A.table, half, p, A.ax, ok, A.sign, cs);
      if (w) r = rstd_of(group_sum<32>(ss), A.D, A.eps);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = lane + 32 * k;
        if (w && i < half) {
          const float u = stored ? 1.f : r;
          y[k].x = __fmul_rn(__fmul_rn(y[k].x, u), weight_at(w, A.w32, IL ? 2 * i : i));
          y[k].y = __fmul_rn(__fmul_rn(y[k].y, u), weight_at(w, A.w32, IL ? 2 * i + 1 : half + i));
        }
        y[k] = turn1(y[k].x, y[k].y, cs[k]);
      }
    }
    if (!stored) {
      T* dst = h < A.Hq ? A.qo + t * A.ldqo + h * A.D : A.ko + t * A.ldko + (h - A.Hq) * A.D;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (const int i = lane + 32 * k; i < half) {
          dst[IL ? 2 * i : i] = from_f32<T>(y[k].x);
          dst[IL ? 2 * i + 1 : half + i] = from_f32<T>(y[k].y);
        }
    } else if constexpr (FMT >= 0) {
      if (page < 0) continue;
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (lane + 32 * k < half) m = max(m, max(abs_bits(y[k].x), abs_bits(y[k].y)));
      m = group_max<32>(m);
      const float am = q8_amax(m), inv = q8_inv<FMT>(am);
      const bool isk = h < HR;
      const int hk = h - (isk ? A.Hq : HR);
      uint8_t* dst = isk ? A.K.q + A.K.cq.at(page, off, hk) : A.V.q + A.V.cq.at(page, off, hk);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (const int i = lane + 32 * k; i < half) {
          dst[IL ? 2 * i : i] = (uint8_t)q8_code1<FMT>(y[k].x, inv);
          dst[IL ? 2 * i + 1 : half + i] = (uint8_t)q8_code1<FMT>(y[k].y, inv);
        }
      if (lane == 0)
        *(isk ? A.K.sc + A.K.cs.at(page, off, hk) : A.V.sc + A.V.cs.at(page, off, hk)) =
            m < kInfBits ? __fdiv_rn(isk ? __fmul_rn(am, r) : am, Q8Max<FMT>::v) : __int_as_float(0x7fc00000);
    }
  }
}

template <typename T, bool IL, int K>
__global__ void __launch_bounds__(256) heads_bwd_elem(const __grid_constant__ HeadArgs<T> A) {
  __shared__ float acc[2 * kMaxHead];
  const int half = A.D / 2, HR = A.Hq + A.Hk;
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kHeadWarps;
  float2 dw[2][K];
#pragma unroll
  for (int k = 0; k < K; ++k) dw[0][k] = dw[1][k] = make_float2(0.f, 0.f);
  for (int64_t item = (int64_t)blockIdx.x * kHeadWarps + warp_index(); item < A.rows * HR; item += step) {
    const int64_t t = item / HR;
    const int h = (int)(item - t * HR);  // uniform per warp, as every test of it
    const bool isq = h < A.Hq;
    const int hh = isq ? h : h - A.Hq;
    const T* xs = (isq ? A.q + t * A.ldq : A.k + t * A.ldk) + hh * A.D;
    const T* gs = (isq ? A.dq + t * A.lddq : A.dk + t * A.lddk) + hh * A.D;
    T* dst = (isq ? A.qo + t * A.ldqo : A.ko + t * A.ldko) + hh * A.D;
    const void* w = isq ? A.wq : A.wk;
    Pos p;
    p.load(A.pos, A.ax, t);
    const bool ok = p.ok(A.max_pos);
    if (!ok && h == 0 && lane == 0) atomicOr(A.err, kErrBadPosition);
    float2 x[K], d[K], g[K], cs[K];
    elem_turns<IL, K>(A.table, half, p, A.ax, ok, -1.f, cs);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = lane + 32 * k, i1 = IL ? 2 * i : i, i2 = IL ? 2 * i + 1 : half + i;
      x[k] = d[k] = g[k] = make_float2(0.f, 0.f);
      if (i < half) {
        x[k] = make_float2(to_f32(xs[i1]), to_f32(xs[i2]));
        d[k] = turn1(to_f32(gs[i1]), to_f32(gs[i2]), cs[k]);
        g[k] = make_float2(d[k].x * weight_at(w, A.w32, i1), d[k].y * weight_at(w, A.w32, i2));
      }
      s1 = fmaf(x[k].x, x[k].x, fmaf(x[k].y, x[k].y, s1));
      s2 = fmaf(g[k].x, x[k].x, fmaf(g[k].y, x[k].y, s2));
    }
    const float r = rstd_of(group_sum<32>(s1), A.D, A.eps);
    const float m = r * group_sum<32>(s2) / (float)A.D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = lane + 32 * k;
      const float2 n = make_float2(x[k].x * r, x[k].y * r);
      if (isq) dw[0][k] = fma2(d[k], n, dw[0][k]);
      else dw[1][k] = fma2(d[k], n, dw[1][k]);
      if (i < half) {
        dst[IL ? 2 * i : i] = from_f32<T>(r * fmaf(-m, n.x, g[k].x));
        dst[IL ? 2 * i + 1 : half + i] = from_f32<T>(r * fmaf(-m, n.y, g[k].y));
      }
    }
  }
  for (int i = threadIdx.x; i < 2 * A.D; i += blockDim.x) acc[i] = 0.f;
  for (int w = 0; w < kHeadWarps; ++w) {
    __syncthreads();
    if ((threadIdx.x >> 5) == w) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (const int i = lane + 32 * k; i < half) {
          const int i1 = IL ? 2 * i : i, i2 = IL ? 2 * i + 1 : half + i;
          acc[i1] += dw[0][k].x;
          acc[i2] += dw[0][k].y;
          acc[A.D + i1] += dw[1][k].x;
          acc[A.D + i2] += dw[1][k].y;
        }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * A.D; i += blockDim.x) A.part[(size_t)blockIdx.x * 2 * A.D + i] = acc[i];
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Whether runs of n values of every head row are aligned.
template <typename T>
bool heads_fit(const HeadArgs<T>& A, const gbln_cache8* kc, const gbln_cache8* vc, int n) {
  const auto row = [&](const void* p, int64_t ld) { return !p || (aligned_to(p, n * sizeof(T)) && ld % n == 0); };
  return A.D % (2 * n) == 0 && A.D / (2 * n) <= 32 && aligned16(A.table) && A.Hq + 2 * A.Hk <= kMaxRows &&
         row(A.q, A.ldq) && row(A.qo, A.ldqo) && row(A.k, A.ldk) && row(A.ko, A.ldko) && row(A.v, A.ldv) &&
         row(A.dq, A.lddq) && row(A.dk, A.lddk) && (!kc || codes_aligned(kc, vc, n));
}

// rows: head rows per lane of a query (or plain K) chunk; kp: of a K chunk.
Split split_of(int Hq, int Hk, int D, int VEC, int rows, int kp) {
  Split W{};
  W.nu = D / (2 * VEC);
  while ((1 << W.lg) < W.nu) ++W.lg;
  const int lgG = 5 - W.lg, G = 1 << lgG;
  // log2 of the tokens whose n heads share a warp's G groups
  const auto tokens = [&](int n) {
    int lt = lgG;
    while (lt > 0 && (n << lt) > G) --lt;
    return lt;
  };
  const int Lq = (Hq + G - 1) / G, Lk = (Hk + G - 1) / G;  // head rows per lane and token
  W.nq = (Lq + rows - 1) / rows;
  W.qch = W.nq ? (Lq + W.nq - 1) / W.nq : 0;
  W.qlt = W.nq ? tokens(Hq) : 0;
  W.nk = (Lk + kp - 1) / kp;
  W.kch = W.nk ? (Lk + W.nk - 1) / W.nk : 0;
  W.klt = W.nk ? tokens(Hk) : 0;
  return W;
}
// Token groups of the chunk with the most: a chunk whose warps take several tokens at once has fewer.
int64_t token_groups(const Split& W, int64_t T) {
  const int lt = !W.nq ? W.klt : !W.nk ? W.qlt : W.qlt < W.klt ? W.qlt : W.klt;
  return (T + (1LL << lt) - 1) >> lt;
}

template <typename T, bool IL, int FMT, int VEC>
gbln_status fwd_vec_launch(const HeadArgs<T>& A, int sms, cudaStream_t s) {
  constexpr int B = VEC * sizeof(T), SQ = rows_of(true, B), LQ = rows_of(false, B);
  Split W = split_of(A.Hq, A.Hk, A.D, VEC, SQ, FMT < 0 ? SQ : 1);
  const int64_t warps = token_groups(W, A.rows) * (W.nq + W.nk);
  bool small = warps <= (int64_t)sms * kSmallBlocks * kHeadWarps;
  if constexpr (B != 16) small = small || W.nq + W.nk <= (FMT < 0 ? 1 : 2);
  if (!small) W = split_of(A.Hq, A.Hk, A.D, VEC, LQ, FMT < 0 ? LQ : 2);
  const int n = W.nq + W.nk;
  // eight times the resident blocks leave a warp a few steps to ask ahead for and the scheduler something to balance
  const unsigned grid = grid_for(token_groups(W, A.rows) * n, kHeadWarps, (int64_t)sms * fwd_blocks(FMT, small) * 8 + (n + kHeadWarps - 1) / kHeadWarps);
  W.stride = (int64_t)grid * kHeadWarps / n;
  if (small) heads_fwd_vec<T, IL, FMT, VEC, true><<<grid, 32 * kHeadWarps, 0, s>>>(A, W);
  else heads_fwd_vec<T, IL, FMT, VEC, false><<<grid, 32 * kHeadWarps, 0, s>>>(A, W);
  return launch_status();
}

template <typename T, bool IL, int FMT>
gbln_status fwd_launch(const HeadArgs<T>& A, const gbln_cache8* kc, const gbln_cache8* vc, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const int sms = sm_count();
  if (sms <= 0) return GBLN_ERR_CUDA;
  if (heads_fit(A, kc, vc, VEC)) return fwd_vec_launch<T, IL, FMT, VEC>(A, sms, s);
  if constexpr (VEC == 8)
    if (heads_fit(A, kc, vc, 4)) return fwd_vec_launch<T, IL, FMT, 4>(A, sms, s);
  const unsigned grid = grid_for(A.rows * (A.Hq + (FMT < 0 ? 1 : 2) * A.Hk), kHeadWarps, (int64_t)sms * 64);
  constexpr int F = FMT < 0 ? -1 : FMT;
  if (A.D <= 128) heads_fwd_elem<T, IL, F, 2><<<grid, 256, 0, s>>>(A);
  else heads_fwd_elem<T, IL, F, 8><<<grid, 256, 0, s>>>(A);
  return launch_status();
}

template <typename T>
gbln_status fwd_typed(const HeadArgs<T>& A, bool il, int fmt, const gbln_cache8* kc, const gbln_cache8* vc, cudaStream_t s) {
  if (fmt < 0 && !A.wq && !A.wk) return il ? fwd_launch<T, true, kRotate>(A, kc, vc, s) : fwd_launch<T, false, kRotate>(A, kc, vc, s);
  if (fmt < 0) return il ? fwd_launch<T, true, -1>(A, kc, vc, s) : fwd_launch<T, false, -1>(A, kc, vc, s);
  if (fmt == GBLN_Q8_INT8)
    return il ? fwd_launch<T, true, GBLN_Q8_INT8>(A, kc, vc, s) : fwd_launch<T, false, GBLN_Q8_INT8>(A, kc, vc, s);
  return il ? fwd_launch<T, true, GBLN_Q8_E4M3>(A, kc, vc, s) : fwd_launch<T, false, GBLN_Q8_E4M3>(A, kc, vc, s);
}

// Blocks (partial rows) of the backward pass: by the sizes alone, whatever path the addresses allow.
int64_t bwd_blocks(int64_t T, int32_t Hq, int32_t Hk, int sms) {
  const int64_t rows = (int64_t)Hq + Hk, few = (rows + 15) / 16 + 1;  // a warp at least for every chunk of two rows
  const int64_t P = grid_for(T * rows, 4 * kHeadWarps, (int64_t)sms * kBwdBlocks);
  return rows <= kMaxRows && P < few ? few : P;
}

template <typename T, bool IL, int VEC>
gbln_status bwd_vec_launch(const HeadArgs<T>& A, int64_t P, int sms, cudaStream_t s) {
  constexpr int B = VEC * sizeof(T), SB = rows_bwd(true, B), LB = rows_bwd(false, B);
  Split W = split_of(A.Hq, A.Hk, A.D, VEC, SB, SB);
  const bool small = token_groups(W, A.rows) * (W.nq + W.nk) <= P * kHeadWarps;
  if (!small) W = split_of(A.Hq, A.Hk, A.D, VEC, LB, LB);
  W.stride = P * kHeadWarps / (W.nq + W.nk);
  if (small) heads_bwd_vec<T, IL, VEC, true><<<(unsigned)P, 32 * kHeadWarps, 0, s>>>(A, W);
  else heads_bwd_vec<T, IL, VEC, false><<<(unsigned)P, 32 * kHeadWarps, 0, s>>>(A, W);
  return launch_status();
}

template <typename T, bool IL>
gbln_status bwd_launch(const HeadArgs<T>& A, int64_t P, int sms, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  if (heads_fit(A, nullptr, nullptr, VEC)) return bwd_vec_launch<T, IL, VEC>(A, P, sms, s);
  if constexpr (VEC == 8)
    if (heads_fit(A, nullptr, nullptr, 4)) return bwd_vec_launch<T, IL, 4>(A, P, sms, s);
  if (A.D <= 128) heads_bwd_elem<T, IL, 2><<<(unsigned)P, 256, 0, s>>>(A);
  else heads_bwd_elem<T, IL, 8><<<(unsigned)P, 256, 0, s>>>(A);
  return launch_status();
}

bool axes_ok(int32_t n, const uint8_t* axis, int32_t D, int64_t ld, int64_t T) {
  if (n < 1 || n > kAxes || (n > 1 && (!axis || ld < T || ld > kLim))) return false;
  if (n > 1)
    for (int i = 0; i < D / 2; ++i)
      if (axis[i] >= n) return false;
  return true;
}
AxisMap axes_of(int32_t n, const uint8_t* axis, int32_t D, int64_t ld) {
  AxisMap m{};
  m.n = n;
  m.ld = ld;
  if (n > 1)
    for (int i = 0; i < D / 2; ++i) m.bits[i >> 4] |= (uint32_t)axis[i] << (2 * (i & 15));
  return m;
}
bool sizes_ok(int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t max_pos) {
  return T >= 0 && T <= kMaxTokens && Hq >= 0 && Hk >= 0 && D > 0 && !(D & 1) && D <= kMaxHead && max_pos >= 0 &&
         ((int64_t)Hq + 2 * (int64_t)Hk) * D <= (1 << 24);
}
bool types_ok(int io, int wt) {
  return (io == GBLN_F32 && wt == GBLN_F32) || (io == GBLN_BF16 && (wt == GBLN_F32 || wt == GBLN_BF16));
}

struct Common {
  const void *q, *k;
  void *qo, *ko;
  const int32_t* pos;
  int32_t n_axes;
  const uint8_t* axis;
  int64_t ld_pos;
  const float* table;
  int64_t max_pos, T;
  int32_t Hq, Hk, D;
  int64_t ldq, ldk, ldqo, ldko;
};
template <typename T>
HeadArgs<T> args_of(const Common& c, unsigned int* err) {
  HeadArgs<T> A{};
  if (c.Hq > 0) {
    A.q = (const T*)c.q;
    A.qo = (T*)c.qo;
  }
  if (c.Hk > 0) {
    A.k = (const T*)c.k;
    A.ko = (T*)c.ko;
  }
  A.pos = c.pos;
  A.table = (const float2*)c.table;
  A.max_pos = c.max_pos;
  A.rows = c.T;
  A.ldq = c.ldq;
  A.ldk = c.ldk;
  A.ldqo = c.ldqo;
  A.ldko = c.ldko;
  A.Hq = c.Hq;
  A.Hk = c.Hk;
  A.D = c.D;
  A.sign = 1.f;
  A.ax = axes_of(c.n_axes, c.axis, c.D, c.ld_pos);
  A.err = err;
  return A;
}
// Sizes, strides and axes of a call; its pointers too where it has tokens.
bool common_ok(const Common& c, bool ko) {
  if (!sizes_ok(c.T, c.Hq, c.Hk, c.D, c.max_pos) || !axes_ok(c.n_axes, c.axis, c.D, c.ld_pos, c.T)) return false;
  const int64_t qw = (int64_t)c.Hq * c.D, kw = (int64_t)c.Hk * c.D;
  if (c.Hq > 0 && (!ld_fits(c.T, qw, c.ldq) || !ld_fits(c.T, qw, c.ldqo))) return false;
  if (c.Hk > 0 && (!ld_fits(c.T, kw, c.ldk) || (ko && !ld_fits(c.T, kw, c.ldko)))) return false;
  if (c.T == 0) return true;
  if (!c.pos || !c.table || !aligned_to(c.table, 8) || (c.Hq > 0 && (!c.q || !c.qo)) || (c.Hk > 0 && (!c.k || (ko && !c.ko)))) return false;
  return true;
}
bool pairing_ok(int p) { return p == GBLN_ROPE_HALF || p == GBLN_ROPE_INTERLEAVED; }

gbln_status rope_axes(const Common& c, float sign, int pairing, int io, cudaStream_t s) {
  if (!dtype_ok(io) || !pairing_ok(pairing) || !common_ok(c, true) || c.Hq < 1) return GBLN_ERR_INVALID_ARG;
  if (c.T == 0) return GBLN_OK;
  unsigned int* err = device_error_word();
  if (!err) return GBLN_ERR_CUDA;
  const bool il = pairing == GBLN_ROPE_INTERLEAVED;
  if (io == GBLN_F32) {
    HeadArgs<float> A = args_of<float>(c, err);
    A.sign = sign;
    return fwd_typed<float>(A, il, -1, nullptr, nullptr, s);
  }
  HeadArgs<bf16> A = args_of<bf16>(c, err);
  A.sign = sign;
  return fwd_typed<bf16>(A, il, -1, nullptr, nullptr, s);
}

}  // namespace

}  // namespace gbln

using namespace gbln;

extern "C" gbln_status gbln_rope_axes_fwd(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions,
                                          int64_t ld_positions, int32_t n_axes, const uint8_t* axis, const float* cos_sin,
                                          int64_t max_pos, int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_q,
                                          int64_t ld_k, int64_t ld_q_out, int64_t ld_k_out, gbln_rope_pairing pairing,
                                          gbln_dtype io, gbln_stream_t stream) {
  return rope_axes({q, k, q_out, k_out, positions, n_axes, axis, ld_positions, cos_sin, max_pos, T, Hq, Hk, D, ld_q, ld_k, ld_q_out, ld_k_out},
                   1.f, pairing, io, (cudaStream_t)stream);
}

extern "C" gbln_status gbln_rope_axes_bwd(const void* dq, const void* dk, void* dq_in, void* dk_in, const int32_t* positions,
                                          int64_t ld_positions, int32_t n_axes, const uint8_t* axis, const float* cos_sin,
                                          int64_t max_pos, int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_dq,
                                          int64_t ld_dk, int64_t ld_dq_in, int64_t ld_dk_in, gbln_rope_pairing pairing,
                                          gbln_dtype io, gbln_stream_t stream) {
  return rope_axes({dq, dk, dq_in, dk_in, positions, n_axes, axis, ld_positions, cos_sin, max_pos, T, Hq, Hk, D, ld_dq, ld_dk, ld_dq_in, ld_dk_in},
                   -1.f, pairing, io, (cudaStream_t)stream);
}

extern "C" gbln_status gbln_qk_norm_rope_fwd(const void* q, const void* k, const void* q_weight, const void* k_weight,
                                             void* q_out, void* k_out, const int32_t* positions, int64_t ld_positions,
                                             int32_t n_axes, const uint8_t* axis, const float* cos_sin, int64_t max_pos,
                                             int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_q, int64_t ld_k,
                                             int64_t ld_q_out, int64_t ld_k_out, float eps, gbln_rope_pairing pairing,
                                             gbln_dtype io, gbln_dtype wt, gbln_stream_t stream) {
  const Common c{q, k, q_out, k_out, positions, n_axes, axis, ld_positions, cos_sin, max_pos, T, Hq, Hk, D, ld_q, ld_k, ld_q_out, ld_k_out};
  if (!types_ok(io, wt)) return GBLN_ERR_UNSUPPORTED;
  if (!pairing_ok(pairing) || !common_ok(c, true) || Hq < 1 || !(eps >= 0.f) || !(eps <= 3.0e38f)) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;
  if (!q_weight || (Hk > 0 && !k_weight)) return GBLN_ERR_INVALID_ARG;
  unsigned int* err = device_error_word();
  if (!err) return GBLN_ERR_CUDA;
  const bool il = pairing == GBLN_ROPE_INTERLEAVED;
  const auto go = [&](auto A) {
    A.wq = q_weight;
    A.wk = k_weight;
    A.w32 = wt == GBLN_F32;
    A.eps = eps;
    return fwd_typed(A, il, -1, nullptr, nullptr, (cudaStream_t)stream);
  };
  return io == GBLN_F32 ? go(args_of<float>(c, err)) : go(args_of<bf16>(c, err));
}

extern "C" int64_t gbln_qk_norm_rope_bwd_num_partials(int64_t T, int32_t Hq, int32_t Hk, int32_t D) {
  if (!sizes_ok(T, Hq, Hk, D, 0) || Hq < 1) return -1;
  if (T == 0) return 0;
  const int sms = sm_count();
  return sms <= 0 ? -1 : bwd_blocks(T, Hq, Hk, sms);
}

extern "C" gbln_status gbln_qk_norm_rope_bwd(const void* dq, const void* dk, const void* q, const void* k,
                                             const void* q_weight, const void* k_weight, void* dq_in, void* dk_in,
                                             float* dw_partial, int64_t P_cap, const int32_t* positions,
                                             int64_t ld_positions, int32_t n_axes, const uint8_t* axis,
                                             const float* cos_sin, int64_t max_pos, int64_t T, int32_t Hq, int32_t Hk,
                                             int32_t D, int64_t ld_dq, int64_t ld_dk, int64_t ld_q, int64_t ld_k,
                                             int64_t ld_dq_in, int64_t ld_dk_in, float eps, gbln_rope_pairing pairing,
                                             gbln_dtype io, gbln_dtype wt, gbln_stream_t stream) {
  const Common c{q, k, dq_in, dk_in, positions, n_axes, axis, ld_positions, cos_sin, max_pos, T, Hq, Hk, D, ld_q, ld_k, ld_dq_in, ld_dk_in};
  if (!types_ok(io, wt)) return GBLN_ERR_UNSUPPORTED;
  if (!pairing_ok(pairing) || !common_ok(c, true) || Hq < 1 || !(eps >= 0.f) || !(eps <= 3.0e38f)) return GBLN_ERR_INVALID_ARG;
  if (!ld_fits(T, (int64_t)Hq * D, ld_dq) || (Hk > 0 && !ld_fits(T, (int64_t)Hk * D, ld_dk))) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;
  if (!dq || !q_weight || !dw_partial || !aligned_to(dw_partial, 4) || (Hk > 0 && (!dk || !k_weight))) return GBLN_ERR_INVALID_ARG;
  const int sms = sm_count();
  unsigned int* err = device_error_word();
  if (sms <= 0 || !err) return GBLN_ERR_CUDA;
  const int64_t P = bwd_blocks(T, Hq, Hk, sms);
  if (P_cap < P) return GBLN_ERR_WORKSPACE;
  const auto go = [&](auto A) {
    using TY = typename std::remove_const<typename std::remove_pointer<decltype(A.q)>::type>::type;
    A.dq = (const TY*)dq;
    if (Hk > 0) A.dk = (const TY*)dk;
    A.lddq = ld_dq;
    A.lddk = ld_dk;
    A.wq = q_weight;
    A.wk = k_weight;
    A.w32 = wt == GBLN_F32;
    A.eps = eps;
    A.part = dw_partial;
    return pairing == GBLN_ROPE_INTERLEAVED ? bwd_launch<TY, true>(A, P, sms, (cudaStream_t)stream)
                                            : bwd_launch<TY, false>(A, P, sms, (cudaStream_t)stream);
  };
  return io == GBLN_F32 ? go(args_of<float>(c, err)) : go(args_of<bf16>(c, err));
}

extern "C" gbln_status gbln_qk_norm_dw_finalize(const float* dw_partial, int64_t P, int32_t D, float* dwq, float* dwk,
                                                int accumulate, gbln_stream_t stream) {
  if (P < 0 || P > (1LL << 31) || D <= 0 || D > kMaxHead || !dwq || !dwk || (P > 0 && !dw_partial)) return GBLN_ERR_INVALID_ARG;
  colsum_kernel<0><<<(2 * D + 31) / 32, 32 * kColSumStripes, 0, (cudaStream_t)stream>>>(dw_partial, P, 2 * D, 2 * D, dwq, dwk, D, accumulate);
  return launch_status();
}

extern "C" gbln_status gbln_qk_norm_rope_fwd_cache8(const void* q, const void* k, const void* v, const void* q_weight,
                                                    const void* k_weight, void* q_out, const int32_t* positions,
                                                    int64_t ld_positions, int32_t n_axes, const uint8_t* axis,
                                                    const float* cos_sin, int64_t max_pos, const int64_t* slots,
                                                    const gbln_cache8* k_cache, const gbln_cache8* v_cache, int64_t T,
                                                    int32_t Hq, int32_t Hk, int32_t D, int64_t ld_q, int64_t ld_k,
                                                    int64_t ld_v, int64_t ld_q_out, float eps, gbln_rope_pairing pairing,
                                                    gbln_q8 fmt, gbln_dtype io, gbln_dtype wt, gbln_stream_t stream) {
  const Common c{q, k, q_out, nullptr, positions, n_axes, axis, ld_positions, cos_sin, max_pos, T, Hq, Hk, D, ld_q, ld_k, ld_q_out, 0};
  if (!types_ok(io, wt)) return GBLN_ERR_UNSUPPORTED;
  if (!q8_ok(fmt) || !pairing_ok(pairing) || !common_ok(c, false) || Hk < 1 || !(eps >= 0.f) || !(eps <= 3.0e38f)) return GBLN_ERR_INVALID_ARG;
  if (!ld_fits(T, (int64_t)Hk * D, ld_v) || !cache_ok(k_cache, Hk, D) || !cache_ok(v_cache, Hk, D)) return GBLN_ERR_INVALID_ARG;
  if (k_cache->pages != v_cache->pages || k_cache->page_size != v_cache->page_size) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;
  if (!v || !slots || !aligned_to(slots, 8) || (Hq > 0 && !q_weight != !k_weight)) return GBLN_ERR_INVALID_ARG;
  if (k_cache->pages > 0 && (!k_cache->codes || !k_cache->scale || !v_cache->codes || !v_cache->scale ||
                             k_cache->codes == v_cache->codes || k_cache->scale == v_cache->scale))
    return GBLN_ERR_INVALID_ARG;
  unsigned int* err = device_error_word();
  if (!err) return GBLN_ERR_CUDA;
  const bool il = pairing == GBLN_ROPE_INTERLEAVED;
  const auto go = [&](auto A) {
    using TY = typename std::remove_const<typename std::remove_pointer<decltype(A.q)>::type>::type;
    A.v = (const TY*)v;
    A.ldv = ld_v;
    A.wq = q_weight;
    A.wk = k_weight;
    A.w32 = wt == GBLN_F32;
    A.eps = eps;
    A.S = slots_of(k_cache, slots);
    A.K = cache_of(k_cache);
    A.V = cache_of(v_cache);
    return fwd_typed(A, il, fmt, k_cache, v_cache, (cudaStream_t)stream);
  };
  return io == GBLN_F32 ? go(args_of<float>(c, err)) : go(args_of<bf16>(c, err));
}
