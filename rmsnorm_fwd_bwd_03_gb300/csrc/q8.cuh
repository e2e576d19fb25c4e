// 8-bit storage with float32 scales: INT8 or E4M3 codes and one scale per group
// of values (a whole row, 128 consecutive values of a row, one head of one
// token).  Every operation below is a float32 operation rounded to nearest, and
// none may be contracted or reassociated: together they define the codes.
//
//   a     = max(max |v|, 2^-100)       (the floor keeps qmax / a finite)
//   inv   = qmax / a                   qmax = 127 (INT8), 448 (E4M3)
//   code  = RNE(v * inv)               to an integer / to E4M3
//   scale = a / qmax                   value = code * scale
//
// |v * inv| <= qmax (1 + 2^-22), which rounds to at most qmax: no clamp.  A
// group that holds an infinity or a NaN gets the scale NaN, so that all of it
// reads back as NaN.  INT8 is off by at most a / 254 per value and E4M3 by the larger
// of 2^-4 of the value and a / 448 * 2^-10 (half a step of its subnormals), each plus
// 2^-21 of the value: the roundings of inv, of v * inv, of the scale and of code * scale.
#pragma once

#include "common.cuh"

namespace gbln {

constexpr float kQ8AmaxMin = 7.888609052210118e-31f;  // 2^-100
constexpr int kCkptGroup = 128;                       // values per checkpoint scale
constexpr uint32_t kInfBits = 0x7f800000u;

template <int FMT>
struct Q8Max {
  static constexpr float v = FMT == GBLN_Q8_INT8 ? 127.0f : 448.0f;
};

inline bool q8_ok(int fmt) { return fmt == GBLN_Q8_INT8 || fmt == GBLN_Q8_E4M3; }

// Two float32 operations in one instruction (each rounded to nearest even by
// itself): the codes cost two to three operations per value beside the kernels'
// own arithmetic, and every instruction stands between a warp's loads.
#define GBLN_F2_OP(name, op)                                                                           \
  __device__ __forceinline__ float2 name(float2 a, float2 b) {                                         \
    float2 r;                                                                                          \
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t" op             \
        " z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"                                                       \
        : "=f"(r.x), "=f"(r.y)                                                                         \
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));                                                     \
    return r;                                                                                          \
  }
GBLN_F2_OP(mul2, "mul.rn.f32x2")
GBLN_F2_OP(add2, "add.rn.f32x2")
#undef GBLN_F2_OP
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Magnitudes are compared as the bit patterns of |v|: an unsigned maximum
// orders finite < infinity < NaN, so a NaN is never lost.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// max(|a|, |b|, |c|) in one instruction; a NaN wins.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int N>
__device__ __forceinline__ uint32_t abs_max_bits(const float (&v)[N]) {
  if constexpr (N == 1) {
    return abs_bits(v[0]);
  } else {
    float m = max3_abs(v[0], v[1], v[N > 2 ? 2 : 1]);
#pragma unroll
    for (int e = 3; e < N; e += 2) m = max3_abs(m, v[e], v[e + 1 < N ? e + 1 : e]);
    return __float_as_uint(m);
  }
}

// Maximum over groups of W consecutive lanes; every lane gets it.
template <int W>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (W == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o, W));
    return v;
  }
}

// The same of values as they lie in memory, without unpacking: bf16 magnitudes
// are compared two at a time (a NaN wins, as above).  part() of the words of a
// thread, join() across threads, bits() of the result as float32.
template <typename T>
struct AbsMax;
template <>
struct AbsMax<float> {
  static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t part(uint4 w) {
    const uint32_t k = 0x7fffffffu;
    return max(max(w.x & k, w.y & k), max(w.z & k, w.w & k));
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
};
template <>
struct AbsMax<bf16> {
  static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  static __device__ __forceinline__ uint32_t part(uint4 w) {
    const uint32_t k = 0x7fff7fffu;
    return join(join(w.x & k, w.y & k), join(w.z & k, w.w & k));
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) { return max(m & 0xffffu, m >> 16) << 16; }
};

__device__ __forceinline__ float q8_amax(uint32_t amax_bits) {
  return fmaxf(__uint_as_float(amax_bits), kQ8AmaxMin);
}
template <int FMT>
__device__ __forceinline__ float q8_inv(float a) { return __fdiv_rn(Q8Max<FMT>::v, a); }
// The stored scale; NaN where the group is not finite.
template <int FMT>
__device__ __forceinline__ float q8_scale(float a, uint32_t amax_bits) {
  return amax_bits < kInfBits ? __fdiv_rn(a, Q8Max<FMT>::v) : __int_as_float(0x7fc00000);
}

// Adding 1.5 * 2^23 rounds |t| <= 2^22 to the nearest integer (ties to even)
// and leaves its two's complement in the low bits of the sum.
constexpr float kRoundMagic = 12582912.0f;

// Codes of N values, packed little-endian.
template <int FMT>
__device__ __forceinline__ uint32_t q8_code1(float v, float inv) {
  const float t = __fmul_rn(v, inv);
  if constexpr (FMT == GBLN_Q8_INT8) return __float_as_uint(__fadd_rn(t, kRoundMagic)) & 0xffu;
  else return e4m3x2(t, 0.f) & 0xffu;
}
template <int FMT>
__device__ __forceinline__ uint32_t q8_code4(float v0, float v1, float v2, float v3, float inv) {
  if constexpr (FMT == GBLN_Q8_INT8) {
    // Single multiplications: a paired one followed by the paired addition came
    // out fused (one rounding instead of two), which moves codes next to a tie.
    const float2 t = add2(make_float2(__fmul_rn(v0, inv), __fmul_rn(v1, inv)), both(kRoundMagic));
    const float2 u = add2(make_float2(__fmul_rn(v2, inv), __fmul_rn(v3, inv)), both(kRoundMagic));
    return __byte_perm(__byte_perm(__float_as_uint(t.x), __float_as_uint(t.y), 0x0040),
                       __byte_perm(__float_as_uint(u.x), __float_as_uint(u.y), 0x0040), 0x5410);
  } else {
    const float2 t = mul2(make_float2(v0, v1), both(inv)), u = mul2(make_float2(v2, v3), both(inv));
    return e4m3x2(t.x, t.y) | (e4m3x2(u.x, u.y) << 16);
  }
}
// N consecutive codes to q, aligned to N bytes when N > 1.
template <int FMT, int N>
__device__ __forceinline__ void q8_store(const float (&v)[N], float inv, uint8_t* q) {
  static_assert(N == 1 || N == 4 || N == 8, "1, 4 or 8 codes");
  if constexpr (N == 1) *q = (uint8_t)q8_code1<FMT>(v[0], inv);
  else if constexpr (N == 4) *reinterpret_cast<uint32_t*>(q) = q8_code4<FMT>(v[0], v[1], v[2], v[3], inv);
  else
    *reinterpret_cast<uint2*>(q) = make_uint2(q8_code4<FMT>(v[0], v[1], v[2], v[3], inv),
                                              q8_code4<FMT>(v[4], v[5], v[6], v[7], inv));
}

// Four codes as float32 (not yet scaled).  INT8: the byte, biased by 128, becomes
// the low mantissa byte of 2^23 + byte, from which 2^23 + 128 is subtracted.
template <int FMT>
__device__ __forceinline__ void q8_decode4(uint32_t w, float* v) {
  if constexpr (FMT == GBLN_Q8_INT8) {
    const uint32_t x = w ^ 0x80808080u;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float2 f = add2(make_float2(__uint_as_float(__byte_perm(x, 0x4b000000u, 0x7540 + e)),
                                        __uint_as_float(__byte_perm(x, 0x4b000000u, 0x7541 + e))),
                            both(-8388736.0f));
      v[e] = f.x;
      v[e + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * e)), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * e] = f.x;
      v[2 * e + 1] = f.y;
    }
  }
}

// N codes kept packed between load and use.
template <int FMT, int N>
struct Codes {
  static_assert(N == 1 || N == 4 || N == 8, "1, 4 or 8 codes");
  uint32_t w[N == 8 ? 2 : 1];
  __device__ __forceinline__ void zero() {
    w[0] = 0;
    if constexpr (N == 8) w[1] = 0;
  }
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (N == 8) {
      asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else if constexpr (N == 4) {
      asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    } else {
      w[0] = *p;
    }
  }
  // code * scale, rounded to float32
  __device__ __forceinline__ void get(float (&v)[N], float scale) const {
    float t[N == 1 ? 4 : N];
    q8_decode4<FMT>(w[0], t);
    if constexpr (N == 8) q8_decode4<FMT>(w[1], t + 4);
    if constexpr (N == 1) {
      v[0] = __fmul_rn(t[0], scale);
    } else {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float2 f = mul2(make_float2(t[e], t[e + 1]), both(scale));
        v[e] = f.x;
        v[e + 1] = f.y;
      }
    }
  }
};

// Ask for the line at p (any alignment) in L2 ahead of use.
__device__ __forceinline__ void prefetch_line(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// The warp's number in its block, in a form that the compiler knows to be the
// same in all lanes: what follows from it needs no divergence handling.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace gbln
