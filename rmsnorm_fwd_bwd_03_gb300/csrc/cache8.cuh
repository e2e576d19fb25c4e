// What the kernels of the paged 8-bit K/V cache share: where its slots lie, runs of a
// head's values, the rotation with its roundings written out, and the host's checks.
#pragma once

#include "q8.cuh"

namespace gbln {

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

// VEC consecutive values of a head row: 16 bytes, or 8 of them.
template <typename T, int VEC, bool WIDE = (VEC * sizeof(T) == 16)>
struct HeadRun;
template <typename T, int VEC>
struct HeadRun<T, VEC, true> {
  uint4 r;
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const T* p) { r = ld_stream(p); }
  __device__ __forceinline__ void get(float (&v)[VEC]) const { unpack<VEC>(r, v); }
  static __device__ __forceinline__ void store(T* p, const float (&v)[VEC]) { st_vec(p, pack<T, VEC>(v)); }
};
template <>
struct HeadRun<bf16, 4, false> {
  uint32_t a, b;
  __device__ __forceinline__ void zero() { a = b = 0; }
  __device__ __forceinline__ void load(const bf16* p) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "l"(p));
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = bf16_lo(a);
    v[1] = bf16_hi(a);
    v[2] = bf16_lo(b);
    v[3] = bf16_hi(b);
  }
  static __device__ __forceinline__ void store(bf16* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
};
// x1 c - x2 s and x2 c + x1 s, f = (c, s).  The roundings are written out (one product
// rounded, the other exact within the multiply-add): chosen by the compiler they were
// not the same in every kernel, and a token's codes depended on the call that stored it.
__device__ __forceinline__ float2 turn1(float x1, float x2, float2 f) {
  return make_float2(__fmaf_rn(x1, f.x, -__fmul_rn(x2, f.y)), __fmaf_rn(x2, f.x, __fmul_rn(x1, f.y)));
}
template <int VEC, bool IL>
__device__ __forceinline__ void turn(float (&xa)[VEC], float (&xb)[VEC], const float2 (&cs)[VEC]) {
  if constexpr (IL) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 a = turn1(xa[e], xa[e + 1], cs[e / 2]), b = turn1(xb[e], xb[e + 1], cs[VEC / 2 + e / 2]);
      xa[e] = a.x;
      xa[e + 1] = a.y;
      xb[e] = b.x;
      xb[e + 1] = b.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float2 a = turn1(xa[e], xb[e], cs[e]);
      xa[e] = a.x;
      xb[e] = a.y;
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int64_t kLim = 1LL << 40;  // strides and sizes (elements)
constexpr int64_t kMaxTokens = 1LL << 33;

// Whether the pages, slots and heads of a cache lie apart: each stride reaches
// past all that the smaller ones span (dimensions of size 1 have no stride).
inline bool apart(int64_t pages, int64_t page, int64_t slots, int64_t slot, int64_t heads, int64_t head, int64_t width) {
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

inline bool cache_ok(const gbln_cache8* c, int32_t Hk, int32_t D) {
  if (!c || c->pages < 0 || c->page_size <= 0 || c->pages > kLim || c->page_size > kLim) return false;
  if (c->pages > 0 && c->page_size > kLim / c->pages) return false;
  return apart(c->pages, c->page_stride, c->page_size, c->slot_stride, Hk, c->head_stride, D) &&
         apart(c->pages, c->scale_page_stride, c->page_size, c->scale_slot_stride, Hk, c->scale_head_stride, 1);
}

// A token stride: at least the row's width, the last row far from overflow.
inline bool ld_fits(int64_t T, int64_t w, int64_t ld) { return ld >= w && ld <= kLim && (double)T * (double)ld < 1.0e18; }

inline Cache cache_of(const gbln_cache8* c) {
  return {c->codes, c->scale, {c->page_stride, c->slot_stride, c->head_stride},
          {c->scale_page_stride, c->scale_slot_stride, c->scale_head_stride}};
}
inline bool strides_multiple(const gbln_cache8* c, int n) {
  return c->page_stride % n == 0 && c->slot_stride % n == 0 && c->head_stride % n == 0;
}
// Whether every head starts at a multiple of n codes.
inline bool codes_aligned(const gbln_cache8* k, const gbln_cache8* v, int n) {
  return aligned_to(k->codes, n) && aligned_to(v->codes, n) && strides_multiple(k, n) && strides_multiple(v, n);
}
inline Slots slots_of(const gbln_cache8* c, const int64_t* slots) {
  const int64_t total = c->pages * c->page_size;
  return {slots, total, c->page_size, total < (1LL << 31) && c->page_size < (1LL << 31)};
}

}  // namespace gbln
