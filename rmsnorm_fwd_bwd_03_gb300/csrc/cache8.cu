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

#include "q8.cuh"

namespace gbln {

namespace {

// Where a cache's slot and head lie (strides in elements).
struct CacheAt {
  int64_t page, slot, head;
  __device__ __forceinline__ int64_t at(int64_t p, int64_t o, int h) const {
    return p * page + o * slot + (int64_t)h * head;
  }
};
struct Cache {
  uint8_t* q;
  float* sc;
  CacheAt cq, cs;
};

struct Slots {
  const int64_t* slots;
  int64_t total, page_size;  // total = pages * page_size
  bool small;                // slots fit 32 bits
  // The page of slot s and the slot's place in it; -1 for "none" (negative), -2
  // for a slot outside the cache.
  __device__ __forceinline__ int64_t page_of(int64_t s, int64_t& off) const {
    if (s < 0) return -1;
    if (s >= total) return -2;
    if (small) {
      const uint32_t p = (uint32_t)s / (uint32_t)page_size;
      off = (int64_t)((uint32_t)s - p * (uint32_t)page_size);
      return p;
    }
    const int64_t p = s / page_size;
    off = s - p * page_size;
    return p;
  }
};

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
  __device__ __forceinline__ const T* src(int64_t t, int h) const {
    if (h < Hq) return q + t * ldq + (int64_t)h * D;
    if (h < Hq + Hk) return k + t * ldk + (int64_t)(h - Hq) * D;
    return v + t * ldv + (int64_t)(h - Hq - Hk) * D;
  }
};

// ---------------------------------------------------------------------------
// Vector path: a warp takes one token and up to kWriteHeads head rows per lane.
// A lane owns the vectors at v*VEC of both halves of a head row, whichever
// pairing, so a warp's accesses are whole lines: with rotate-half pairing they
// turn into each other by VEC table entries, with interleaved pairing each holds
// VEC / 2 pairs of its own.  A head row takes nu = D / (2 VEC) lanes out of a group
// of the next power of two, so 80 or 96 wide heads run here with idle lanes.  The
// table entries are loaded once per token and lane, and all of a lane's row
// loads are issued before anything that depends on the token's slot or position.
// ---------------------------------------------------------------------------
// Six head rows per lane (two blocks of 256 threads per SM) measured faster than
// four (three blocks): 236 against 247 us for 65536 tokens of 32 / 8 heads of 128.
constexpr int kWriteHeads = 6;
constexpr int kWriteWarps = 8;  // per block: chunks of a token, then tokens
// A warp walks tokens t, t + step, ... and asks for the next one's rows in L2
// while it works on this one.  Eight times the resident blocks leave a warp a
// few tokens to do that for and the scheduler something to balance: 236 us, with
// one token per warp 283, with the resident blocks alone 266.
constexpr int kWriteGrid = 2 * 8;  // blocks per SM

template <typename T, bool IL, int FMT>
__global__ void __launch_bounds__(32 * kWriteWarps, 2)
cache8_write_vec(const WriteArgs<T> A, int nu, int lg, int ch) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int LINE = 128 / sizeof(T);
  const int half = A.D / 2, HR = A.Hq + A.Hk, HT = HR + A.Hk;
  const int lanes = 1 << lg, G = 32 >> lg;
  const int lane = threadIdx.x;
  const int v = lane & (lanes - 1);
  const bool on = v < nu;
  const int c = blockIdx.y * blockDim.y + threadIdx.y;
  const int hf = G * c * ch, hb = (lane >> lg) + hf;
  const int64_t step = (int64_t)gridDim.x * blockDim.z;
  int64_t t = (int64_t)blockIdx.x * blockDim.z + threadIdx.z;
  if (t >= A.rows || hf >= HT) return;  // uniform per warp
  const int ia = v * VEC, ib = half + ia;
  int p = __ldg(A.pos + t);
  int64_t slot = __ldg(A.S.slots + t);
#pragma unroll 1
  for (; t < A.rows; t += step) {
    // rows of the three inputs, offset so that head h is at + h * D in each
    const T* qp = A.q + t * A.ldq;
    const T* kp = A.k + t * A.ldk - (int64_t)A.Hq * A.D;
    const T* vp = A.v + t * A.ldv - (int64_t)HR * A.D;
    uint4 a[kWriteHeads], b[kWriteHeads];
#pragma unroll
    for (int j = 0; j < kWriteHeads; ++j) {
      const int h = hb + G * j;
      a[j] = b[j] = make_uint4(0, 0, 0, 0);
      if (j < ch && on && h < HT) {
        const T* src = (h < A.Hq ? qp : h < HR ? kp : vp) + h * A.D + ia;
        a[j] = ld_stream(src);
        b[j] = ld_stream(src + half);
      }
    }
    const bool ok = p >= 0 && (int64_t)p < A.max_pos;
    // (cos, sin) of the lane's pairs: entries v*VEC.. (rotate-half), or half as many
    // for each of its two vectors (interleaved)
    float2 cs[VEC];
    if (ok && on) {
      const float2* e = A.table + (size_t)p * half;
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        const int at = !IL ? ia + i : i < VEC / 2 ? ia / 2 + i : ib / 2 + i - VEC / 2;
        const float4 f = __ldg(reinterpret_cast<const float4*>(e + at));
        cs[i] = make_float2(f.x, f.y);
        cs[i + 1] = make_float2(f.z, f.w);
      }
    } else {
      const float x = ok ? 0.f : __int_as_float(0x7fc00000);
#pragma unroll
      for (int i = 0; i < VEC; ++i) cs[i] = make_float2(x, x);
    }
    int64_t off = 0;
    const int64_t page = A.S.page_of(slot, off);
    // the warp's next token: its position and slot, and its rows on their way to L2
    if (t + step < A.rows) {
      p = __ldg(A.pos + t + step);
      slot = __ldg(A.S.slots + t + step);
      const int last = min(hf + G * ch, HT) * A.D;
      for (int x = hf * A.D + lane * LINE; x < last; x += 32 * LINE)
        prefetch_line((x < A.Hq * A.D ? qp + step * A.ldq : x < HR * A.D ? kp + step * A.ldk : vp + step * A.ldv) + x);
    }
    if (c == 0 && lane == 0) {
      if (!ok && (A.Hq > 0 || page >= 0)) atomicOr(A.err, kErrBadPosition);
      if (page == -2) atomicOr(A.err, kErrBadSlot);
    }
    T* qo = A.qo + t * A.ldqo + ia;
#pragma unroll
    for (int j = 0; j < kWriteHeads; ++j) {
      if (j >= ch) break;
      const int h = hb + G * j;
      float xa[VEC], xb[VEC];
      unpack<VEC>(a[j], xa);
      unpack<VEC>(b[j], xb);
      if (h < HR) {
        float ya[VEC], yb[VEC];
        if constexpr (IL) {
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const float2 f = cs[e / 2], f2 = cs[VEC / 2 + e / 2];
            ya[e] = xa[e] * f.x - xa[e + 1] * f.y;
            ya[e + 1] = xa[e + 1] * f.x + xa[e] * f.y;
            yb[e] = xb[e] * f2.x - xb[e + 1] * f2.y;
            yb[e + 1] = xb[e + 1] * f2.x + xb[e] * f2.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            ya[e] = xa[e] * cs[e].x - xb[e] * cs[e].y;
            yb[e] = xb[e] * cs[e].x + xa[e] * cs[e].y;
          }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          xa[e] = ya[e];
          xb[e] = yb[e];
        }
      }
      if (h < A.Hq && on) {
        T* dst = qo + h * A.D;
        st_vec(dst, pack<T, VEC>(xa));
        st_vec(dst + half, pack<T, VEC>(xb));
      }
      const bool kv = h >= A.Hq && h < HT && page >= 0;
      if (__any_sync(0xffffffffu, kv)) {  // a warp's head rows may be both Q and K
        uint32_t m = on ? max(abs_max_bits<VEC>(xa), abs_max_bits<VEC>(xb)) : 0u;
        for (int o = lanes >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        // even lanes divide for 1 / scale, odd ones for the scale
        const float am = q8_amax(m);
        const bool odd = (lane & 1) != 0;
        const float d = __fdiv_rn(odd ? am : Q8Max<FMT>::v, odd ? Q8Max<FMT>::v : am);
        float inv = __shfl_sync(0xffffffffu, d, lane & ~1);
        float scale = d;
        if (lanes == 1) {  // a head per lane: both divisions are its own
          inv = q8_inv<FMT>(am);
          scale = __fdiv_rn(am, Q8Max<FMT>::v);
        }
        if (kv && on) {
          const bool isk = h < HR;
          const int hk = h - (isk ? A.Hq : HR);
          uint8_t* dst = (isk ? A.K.q : A.V.q) + (isk ? A.K.cq.at(page, off, hk) : A.V.cq.at(page, off, hk)) + ia;
          q8_store<FMT, VEC>(xa, inv, dst);
          q8_store<FMT, VEC>(xb, inv, dst + half);
          if (v == (lanes == 1 ? 0 : 1)) {
            float* sc = isk ? A.K.sc + A.K.cs.at(page, off, hk) : A.V.sc + A.V.cs.at(page, off, hk);
            *sc = m < kInfBits ? scale : __int_as_float(0x7fc00000);
          }
        }
      }
    }
  }
}

// Element path (any head size, alignment and stride): a warp per head row, a
// lane the pairs l, l + 32, ...; K and V are read twice, the second time from L1.
template <typename T, bool IL, int FMT>
__global__ void __launch_bounds__(256) cache8_write_elem(const WriteArgs<T> A) {
  const int half = A.D / 2, HR = A.Hq + A.Hk, HT = HR + A.Hk;
  const int lane = threadIdx.x & 31;
  const int64_t step = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; item < A.rows * HT; item += step) {
    const int64_t t = item / HT;
    const int h = (int)(item - t * HT);
    int64_t off = 0;
    const int64_t page = A.S.page_of(__ldg(A.S.slots + t), off);
    const int p = __ldg(A.pos + t);
    const bool ok = p >= 0 && (int64_t)p < A.max_pos;
    if (h == 0 && lane == 0) {
      if (!ok && (A.Hq > 0 || page >= 0)) atomicOr(A.err, kErrBadPosition);
      if (page == -2) atomicOr(A.err, kErrBadSlot);
    }
    if (h >= A.Hq && page < 0) continue;
    const T* src = A.src(t, h);
    auto pair = [&](int i, float& y1, float& y2) {
      const float x1 = to_f32(src[IL ? 2 * i : i]), x2 = to_f32(src[IL ? 2 * i + 1 : half + i]);
      if (h < HR) {
        const float qnan = __int_as_float(0x7fc00000);
        const float2 f = ok ? __ldg(A.table + (size_t)p * half + i) : make_float2(qnan, qnan);
        y1 = x1 * f.x - x2 * f.y;
        y2 = x2 * f.x + x1 * f.y;
      } else {
        y1 = x1;
        y2 = x2;
      }
    };
    if (h < A.Hq) {
      T* dst = A.qo + t * A.ldqo + (int64_t)h * A.D;
      for (int i = lane; i < half; i += 32) {
        float y1, y2;
        pair(i, y1, y2);
        dst[IL ? 2 * i : i] = from_f32<T>(y1);
        dst[IL ? 2 * i + 1 : half + i] = from_f32<T>(y2);
      }
      continue;
    }
    uint32_t m = 0;
    for (int i = lane; i < half; i += 32) {
      float y1, y2;
      pair(i, y1, y2);
      m = max(m, max(abs_bits(y1), abs_bits(y2)));
    }
    m = group_max<32>(m);
    const float am = q8_amax(m), inv = q8_inv<FMT>(am);
    const bool isk = h < HR;
    const int hk = h - (isk ? A.Hq : HR);
    const Cache& C = isk ? A.K : A.V;
    uint8_t* dst = C.q + C.cq.at(page, off, hk);
    for (int i = lane; i < half; i += 32) {
      float y1, y2;
      pair(i, y1, y2);
      dst[IL ? 2 * i : i] = (uint8_t)q8_code1<FMT>(y1, inv);
      dst[IL ? 2 * i + 1 : half + i] = (uint8_t)q8_code1<FMT>(y2, inv);
    }
    if (lane == 0) C.sc[C.cs.at(page, off, hk)] = q8_scale<FMT>(am, m);
  }
}

// ---------------------------------------------------------------------------
// Read-back: a warp per token, then the next one (the slot of which it has
// loaded by then).  A unit is N consecutive codes of one head: on the vector path
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

constexpr int kReadHeads = 4;
constexpr int kReadGrid = 3;  // blocks per SM, all resident

template <typename T, int FMT, int N>
__global__ void __launch_bounds__(256) cache8_read_kernel(const ReadArgs<T> A, int per, int lg) {
  constexpr int U = kReadHeads;
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
  int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= A.rows) return;  // uniform per warp
  const int lanes = 1 << lg, G = 32 >> lg;
  const int d0 = lane & (lanes - 1), hb = lane >> lg;
  int64_t off = 0, page = A.S.page_of(__ldg(A.S.slots + t), off);
#pragma unroll 1
  for (; t < A.rows; t += step) {
    const bool more = t + step < A.rows;
    const int64_t next = more ? __ldg(A.S.slots + t + step) : -1;
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
      if (page == -2 && lane == 0) atomicOr(A.err, kErrBadSlot);
      float fill[N];
#pragma unroll
      for (int e = 0; e < N; ++e) fill[e] = page == -2 ? __int_as_float(0x7fc00000) : 0.f;
      for (int d = d0; d < per; d += lanes)
        for (int h = hb; h < A.Hk; h += G) {
          store_n<T, N>(ko + h * A.D + d * N, fill);
          store_n<T, N>(vo + h * A.D + d * N, fill);
        }
    }
    page = A.S.page_of(next, off);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int64_t kLim = 1LL << 40;  // strides and sizes (elements)
constexpr int64_t kMaxTokens = 1LL << 33;

// Whether the pages, slots and heads of a cache lie apart: each stride reaches
// past all that the smaller ones span (dimensions of size 1 have no stride).
bool apart(int64_t pages, int64_t page, int64_t slots, int64_t slot, int64_t heads, int64_t head, int64_t width) {
  int64_t n[3] = {pages, slots, heads}, st[3] = {page, slot, head};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) {
        const int64_t a = n[i], b = st[i];
        n[i] = n[j]; st[i] = st[j];
        n[j] = a; st[j] = b;
      }
  double span = (double)width;  // 2^62 and more would overflow an integer
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < 0 || (double)st[i] < span) return false;
    span += (double)st[i] * (double)(n[i] - 1);
  }
  return span < 1.0e18;
}

bool cache_ok(const gbln_cache8* c, int32_t Hk, int32_t D) {
  if (!c || c->pages < 0 || c->page_size <= 0 || c->pages > kLim || c->page_size > kLim) return false;
  if (c->pages > 0 && c->page_size > kLim / c->pages) return false;
  return apart(c->pages, c->page_stride, c->page_size, c->slot_stride, Hk, c->head_stride, D) &&
         apart(c->pages, c->scale_page_stride, c->page_size, c->scale_slot_stride, Hk, c->scale_head_stride, 1);
}

// A token stride: at least the row's width, the last row far from overflow.
bool ld_fits(int64_t T, int64_t w, int64_t ld) { return ld >= w && ld <= kLim && (double)T * (double)ld < 1.0e18; }

Cache cache_of(const gbln_cache8* c) {
  return {c->codes, c->scale, {c->page_stride, c->slot_stride, c->head_stride},
          {c->scale_page_stride, c->scale_slot_stride, c->scale_head_stride}};
}
bool strides_multiple(const gbln_cache8* c, int n) {
  return c->page_stride % n == 0 && c->slot_stride % n == 0 && c->head_stride % n == 0;
}
// Whether every head starts at a multiple of the codes of one access.
bool codes_aligned(const gbln_cache8* k, const gbln_cache8* v, gbln_dtype io) {
  const int n = io == GBLN_F32 ? 4 : 8;
  return aligned_to(k->codes, n) && aligned_to(v->codes, n) && strides_multiple(k, n) && strides_multiple(v, n);
}
Slots slots_of(const gbln_cache8* c, const int64_t* slots) {
  const int64_t total = c->pages * c->page_size;
  return {slots, total, c->page_size, total < (1LL << 31) && c->page_size < (1LL << 31)};
}

template <typename T, bool IL, int FMT>
gbln_status write_launch(const WriteArgs<T>& A, bool cache_aligned, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const int HT = A.Hq + 2 * A.Hk;
  const auto row16 = [](const void* p, int64_t ld) { return aligned16(p) && (ld * (int64_t)sizeof(T)) % 16 == 0; };
  const bool vec = A.D % (2 * VEC) == 0 && A.D / (2 * VEC) <= 32 && aligned16(A.table) && cache_aligned &&
                   (A.Hq == 0 || (row16(A.q, A.ldq) && row16(A.qo, A.ldqo))) && row16(A.k, A.ldk) && row16(A.v, A.ldv);
  if (vec) {
    const int nu = A.D / (2 * VEC);
    int lg = 0;
    while ((1 << lg) < nu) ++lg;
    const int G = 32 >> lg, L = (HT + G - 1) / G;  // head rows per lane and token
    const int nchunk = (L + kWriteHeads - 1) / kWriteHeads;
    const int ch = (L + nchunk - 1) / nchunk;
    const int cy = nchunk < kWriteWarps ? nchunk : kWriteWarps, tz = kWriteWarps / cy;
    const int sms = sm_count();
    if (sms <= 0) return GBLN_ERR_CUDA;
    const int64_t gy = (nchunk + cy - 1) / cy;
    if (gy <= 65535) {
      const unsigned gx = grid_for(A.rows, tz, (int64_t)sms * kWriteGrid);
      cache8_write_vec<T, IL, FMT><<<dim3(gx, (unsigned)gy), dim3(32, cy, tz), 0, s>>>(A, nu, lg, ch);
      return launch_status();
    }
  }
  cache8_write_elem<T, IL, FMT><<<grid_for(A.rows * HT, 8, 1 << 20), 256, 0, s>>>(A);
  return launch_status();
}

template <typename T>
gbln_status write_typed(const WriteArgs<T>& A, bool il, int fmt, bool cache_aligned, cudaStream_t s) {
  if (fmt == GBLN_Q8_INT8)
    return il ? write_launch<T, true, GBLN_Q8_INT8>(A, cache_aligned, s)
              : write_launch<T, false, GBLN_Q8_INT8>(A, cache_aligned, s);
  return il ? write_launch<T, true, GBLN_Q8_E4M3>(A, cache_aligned, s)
            : write_launch<T, false, GBLN_Q8_E4M3>(A, cache_aligned, s);
}

template <typename T>
gbln_status read_typed(const ReadArgs<T>& A, int fmt, bool cache_aligned, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const bool vec = A.D % VEC == 0 && cache_aligned && aligned16(A.ko) && aligned16(A.vo) &&
                   (A.ldk * (int64_t)sizeof(T)) % 16 == 0 && (A.ldv * (int64_t)sizeof(T)) % 16 == 0;
  const int sms = sm_count();
  if (sms <= 0) return GBLN_ERR_CUDA;
  const unsigned grid = grid_for(A.rows, 8, (int64_t)sms * kReadGrid);
  const int per = A.D / (vec ? VEC : 1);  // units per head
  int lg = 0;
  while (lg < 5 && (1 << lg) < per) ++lg;
#define GBLN_READ8(FMT, N) cache8_read_kernel<T, FMT, N><<<grid, 256, 0, s>>>(A, per, lg)
  if (fmt == GBLN_Q8_INT8) {
    if (vec) GBLN_READ8(GBLN_Q8_INT8, VEC);
    else GBLN_READ8(GBLN_Q8_INT8, 1);
  } else {
    if (vec) GBLN_READ8(GBLN_Q8_E4M3, VEC);
    else GBLN_READ8(GBLN_Q8_E4M3, 1);
  }
#undef GBLN_READ8
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
  unsigned int* err = device_error_word();
  if (!err) return GBLN_ERR_CUDA;
  const bool il = pairing == GBLN_ROPE_INTERLEAVED;
  const bool ca = codes_aligned(k_cache, v_cache, io);
  cudaStream_t s = (cudaStream_t)stream;
#define GBLN_WRITE_ARGS(TY)                                                                               \
  const WriteArgs<TY> A{(const TY*)q, (const TY*)k, (const TY*)v, (TY*)q_out, positions, (const float2*)cos_sin, \
                        max_pos, T, Hq, Hk, D, ld_q, ld_k, ld_v, ld_q_out, slots_of(k_cache, slots),       \
                        cache_of(k_cache), cache_of(v_cache), err}
  if (io == GBLN_F32) {
    GBLN_WRITE_ARGS(float);
    return write_typed<float>(A, il, fmt, ca, s);
  }
  GBLN_WRITE_ARGS(bf16);
  return write_typed<bf16>(A, il, fmt, ca, s);
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
  const bool ca = codes_aligned(k_cache, v_cache, io);
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
