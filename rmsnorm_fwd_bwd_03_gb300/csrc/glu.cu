// Gated MLP units (SwiGLU and its GeLU / ReLU siblings) and plain activations,
// forward and backward.
//
// Operator: "Fast-LLM: 高效大语言模型训练框架", §三 "支持的 MLP 变体" (dense MLP, gated
// or not, SiLU / GeLU / ReLU) and "训练配置示例" (gated: true, activation: silu,
// intermediate_size); "LLaMA-Factory Kernels 系统" (fused SwiGLU);
// "Kernels（自定义内核）" §Liger.
//
// Pure streaming: 2 reads + 1 write (gated forward), 3 reads + 2 writes (gated
// backward), 1 + 1 and 2 + 1 for the plain activation, 128-bit accesses,
// UNROLL independent vectors in flight per thread, grid sized to the resident
// capacity of the GPU.  Contiguous tensors are walked as one flat index space;
// row-strided ones (gate and up as the two halves of a packed [T, 2I]
// projection output, for instance) by (row group, column block) units.  The
// activation is recomputed in the backward pass; nothing is saved.  The gated
// forward can also deliver its output as MXFP8 (E4M3 codes and one E8M0 scale
// per 32 values of a row) or as E4M3 with one float32 scale per row for the down
// projection, and save gate and up as 8-bit checkpoints (one float32 scale per
// 128 values of a row) that a backward pass reads.

#include <atomic>
#include <type_traits>

#include <cooperative_groups.h>

#include "q8.cuh"

namespace gbln {

namespace {

constexpr int kGluBlock = 256;

// bf16 I/O moves only 2 bytes per element, so the arithmetic per element must
// stay within a few instructions for the kernels to remain HBM-bound.  Their
// exponentials and reciprocals therefore go straight to the hardware's base-2
// exponential and reciprocal approximations in flush-to-zero form
// (ex2.approx.ftz, rcp.approx.ftz), with e^a = 2^(a log2 e).  Their relative
// errors are a few float32 ulp, far below bf16 rounding, and none of the
// formulas needs denormals (a denormal exponential or reciprocal is far below
// bf16 resolution wherever it appears); dropping the denormal handling saves
// instructions.  float32 I/O keeps the accurate library functions.
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// e^a for the bf16 paths (a * log2 e rounded once, then ex2).
__device__ __forceinline__ float exp_fast(float a) { return ex2_ftz(a * kLog2e); }

// sigmoid(g) = 1 / (1 + exp(-g)): expf and an IEEE division for float32 I/O.
// For g < ~-88, exp(-g) = inf and both forms give 0 (the reciprocal of inf is 0).
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 4) {
    return 1.0f / (1.0f + expf(-g));
  } else {
    return rcp_ftz(1.0f + exp_fast(-g));
  }
}

// GeLU, tanh form: 0.5 x (1 + tanh(z)) with z = sqrt(2/pi) (x + 0.044715 x^3).
// Since 0.5 (1 + tanh(z)) = sigmoid(2 z), it is evaluated as x * sigmoid(2 z),
// which has no cancellation for negative x.
constexpr float kGeluK = 1.5957691216057308f;   // 2 * sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;  // 1 / sqrt(2 pi)

// Normal CDF for the bf16 path from the rational approximation of erfc in
// Abramowitz & Stegun, Handbook of Mathematical Functions, formula 7.1.26
// (absolute error of erf below 1.5e-7): for z >= 0, erfc(z) ~ (a1 t + a2 t^2 +
// a3 t^3 + a4 t^4 + a5 t^5) e^{-z^2} with t = 1 / (1 + p z).  With z = |x| /
// sqrt(2): Phi(x) = erfc(z) / 2 for x < 0 (no cancellation) and 1 - erfc(z) / 2
// for x >= 0.  ex receives e^{-z^2} = e^{-x^2/2}, the Gaussian density's
// exponential, which the backward pass needs as well.  About half the
// instructions of erff; float32 I/O keeps erff.
constexpr float kAsP = 0.3275911f;
constexpr float kAsA1 = 0.254829592f, kAsA2 = -0.284496736f, kAsA3 = 1.421413741f,
                kAsA4 = -1.453152027f, kAsA5 = 1.061405429f;

__device__ __forceinline__ float gauss_cdf_as(float x, float& ex) {
  const float z = fabsf(x) * kInvSqrt2;
  const float t = rcp_ftz(fmaf(kAsP, z, 1.0f));
  ex = exp_fast(-z * z);
  const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, kAsA5, kAsA4), kAsA3), kAsA2), kAsA1);
  const float half_erfc = 0.5f * poly * ex;
  return x >= 0.f ? __fsub_rn(1.0f, half_erfc) : half_erfc;
}

// 2 z of the tanh form.
__device__ __forceinline__ float gelu_arg(float x) { return kGeluK * fmaf(kGeluC * x * x, x, x); }

// Activation value f(x) and, for the backward pass, f(x) and f'(x) together.
template <typename T, int ACT>
__device__ __forceinline__ float act_f(float x) {
  if constexpr (ACT == GBLN_ACT_SILU) {
    if constexpr (sizeof(T) == 4) return x / (1.0f + expf(-x));
    else return x * rcp_ftz(1.0f + exp_fast(-x));
  } else if constexpr (ACT == GBLN_ACT_GELU_TANH) {
    return x * sigmoid<T>(gelu_arg(x));
  } else if constexpr (ACT == GBLN_ACT_GELU_ERF) {
    if constexpr (sizeof(T) == 4) {
      return 0.5f * x * (1.0f + erff(x * kInvSqrt2));
    } else {
      float ex;
      return x * gauss_cdf_as(x, ex);
    }
  } else {
    return x > 0.f ? x : 0.f;
  }
}

template <typename T, int ACT>
__device__ __forceinline__ void act_fd(float x, float& f, float& d) {
  if constexpr (ACT == GBLN_ACT_SILU) {
    const float s = sigmoid<T>(x);
    f = x * s;
    d = s * (1.0f + x * (1.0f - s));
  } else if constexpr (ACT == GBLN_ACT_GELU_TANH) {
    const float s = sigmoid<T>(gelu_arg(x));
    f = x * s;
    d = s + x * s * (1.0f - s) * kGeluK * (1.0f + 3.0f * kGeluC * x * x);
  } else if constexpr (ACT == GBLN_ACT_GELU_ERF) {
    if constexpr (sizeof(T) == 4) {
      const float cdf = 0.5f * (1.0f + erff(x * kInvSqrt2));
      f = x * cdf;
      d = cdf + x * kInvSqrt2Pi * expf(-0.5f * x * x);
    } else {
      float ex;
      const float cdf = gauss_cdf_as(x, ex);
      f = x * cdf;
      d = cdf + x * kInvSqrt2Pi * ex;
    }
  } else {
    f = x > 0.f ? x : 0.f;
    d = x > 0.f ? 1.f : 0.f;
  }
}

// ---------------------------------------------------------------------------
// Contiguous tensors: flat index over n / VEC vectors.  Packed 16-byte loads
// stay packed in registers until used, so UNROLL vectors per tensor can be in
// flight without spilling.
// ---------------------------------------------------------------------------
template <typename T, int ACT, int UNROLL>
__global__ void __launch_bounds__(kGluBlock)
glu_fwd_vec(const T* gate, const T* up, T* out, int64_t nvec) {
  constexpr int VEC = VecOf<T>::N;
  const int64_t step = (int64_t)gridDim.x * kGluBlock * UNROLL;
  for (int64_t b = (int64_t)blockIdx.x * kGluBlock * UNROLL + threadIdx.x; b < nvec; b += step) {
    uint4 g[UNROLL], u[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int64_t i = b + (int64_t)k * kGluBlock;
      if (i < nvec) {
        g[k] = ld_stream(gate + i * VEC);
        u[k] = ld_stream(up + i * VEC);
      }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int64_t i = b + (int64_t)k * kGluBlock;
      if (i < nvec) {
        float gf[VEC], uf[VEC], o[VEC];
        unpack<VEC>(g[k], gf);
        unpack<VEC>(u[k], uf);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = act_f<T, ACT>(gf[e]) * uf[e];
        st_vec(out + i * VEC, pack<T, VEC>(o));
      }
    }
  }
}

template <typename T, int ACT, int UNROLL>
__global__ void __launch_bounds__(kGluBlock)
glu_bwd_vec(const T* dout, const T* gate, const T* up, T* dgate, T* dup, int64_t nvec) {
  constexpr int VEC = VecOf<T>::N;
  const int64_t step = (int64_t)gridDim.x * kGluBlock * UNROLL;
  for (int64_t b = (int64_t)blockIdx.x * kGluBlock * UNROLL + threadIdx.x; b < nvec; b += step) {
    uint4 d[UNROLL], g[UNROLL], u[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int64_t i = b + (int64_t)k * kGluBlock;
      if (i < nvec) {
        d[k] = ld_stream(dout + i * VEC);
        g[k] = ld_stream(gate + i * VEC);
        u[k] = ld_stream(up + i * VEC);
      }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int64_t i = b + (int64_t)k * kGluBlock;
      if (i < nvec) {
        float df[VEC], gf[VEC], uf[VEC], dg[VEC], du[VEC];
        unpack<VEC>(d[k], df);
        unpack<VEC>(g[k], gf);
        unpack<VEC>(u[k], uf);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float f, fp;
          act_fd<T, ACT>(gf[e], f, fp);
          du[e] = df[e] * f;
          dg[e] = df[e] * uf[e] * fp;
        }
        st_vec(dgate + i * VEC, pack<T, VEC>(dg));
        st_vec(dup + i * VEC, pack<T, VEC>(du));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Row-strided tensors.  A unit is (group of UNROLL consecutive rows, block of
// blockDim.x column vectors); thread t takes column vector j * blockDim.x + t
// of each row of the group, so a warp's accesses stay contiguous within a row.
// The host picks the block width so that the column blocks tile the row.
// VEC = 1 is the element-wise path (unaligned pointers or strides).
// ---------------------------------------------------------------------------
template <typename T, int VEC, int ACT, int UNROLL>
__global__ void __launch_bounds__(kGluBlock)
glu_fwd_rows(const T* gate, const T* up, T* out, int64_t T_, int64_t ncol, int64_t ldg,
             int64_t ldu, int64_t ldo) {
  const int cb = blockDim.x;
  const int64_t ncb = (ncol + cb - 1) / cb;
  const int64_t units = (T_ + UNROLL - 1) / UNROLL * ncb;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t rg = u / ncb;
    const int64_t c = (u - rg * ncb) * cb + threadIdx.x;
    if (c >= ncol) continue;
    const int64_t r0 = rg * UNROLL;
    Packed<T, VEC> g[UNROLL], v[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (r0 + k < T_) {
        g[k].load(gate + (r0 + k) * ldg + c * VEC);
        v[k].load(up + (r0 + k) * ldu + c * VEC);
      }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (r0 + k < T_) {
        float gf[VEC], uf[VEC], o[VEC];
        g[k].get(gf);
        v[k].get(uf);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = act_f<T, ACT>(gf[e]) * uf[e];
        store_n<T, VEC>(out + (r0 + k) * ldo + c * VEC, o);
      }
    }
  }
}

template <typename T, int VEC, int ACT, int UNROLL>
__global__ void __launch_bounds__(kGluBlock)
glu_bwd_rows(const T* dout, const T* gate, const T* up, T* dgate, T* dup, int64_t T_,
             int64_t ncol, int64_t ldd, int64_t ldg, int64_t ldu, int64_t lddg, int64_t lddu) {
  const int cb = blockDim.x;
  const int64_t ncb = (ncol + cb - 1) / cb;
  const int64_t units = (T_ + UNROLL - 1) / UNROLL * ncb;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t rg = u / ncb;
    const int64_t c = (u - rg * ncb) * cb + threadIdx.x;
    if (c >= ncol) continue;
    const int64_t r0 = rg * UNROLL;
    Packed<T, VEC> d[UNROLL], g[UNROLL], v[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (r0 + k < T_) {
        d[k].load(dout + (r0 + k) * ldd + c * VEC);
        g[k].load(gate + (r0 + k) * ldg + c * VEC);
        v[k].load(up + (r0 + k) * ldu + c * VEC);
      }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (r0 + k < T_) {
        float df[VEC], gf[VEC], uf[VEC], dg[VEC], du[VEC];
        d[k].get(df);
        g[k].get(gf);
        v[k].get(uf);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float f, fp;
          act_fd<T, ACT>(gf[e], f, fp);
          du[e] = df[e] * f;
          dg[e] = df[e] * uf[e] * fp;
        }
        store_n<T, VEC>(dgate + (r0 + k) * lddg + c * VEC, dg);
        store_n<T, VEC>(dup + (r0 + k) * lddu + c * VEC, du);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Plain activation y = f(x), dx = dy * f'(x) over n contiguous elements.
// ---------------------------------------------------------------------------
template <typename T, int VEC, int ACT, int UNROLL>
__global__ void __launch_bounds__(kGluBlock)
act_fwd_kernel(const T* x, T* y, int64_t nv) {
  const int64_t step = (int64_t)gridDim.x * kGluBlock * UNROLL;
  for (int64_t b = (int64_t)blockIdx.x * kGluBlock * UNROLL + threadIdx.x; b < nv; b += step) {
    Packed<T, VEC> a[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int64_t i = b + (int64_t)k * kGluBlock;
      if (i < nv) a[k].load(x + i * VEC);
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int64_t i = b + (int64_t)k * kGluBlock;
      if (i < nv) {
        float v[VEC];
        a[k].get(v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = act_f<T, ACT>(v[e]);
        store_n<T, VEC>(y + i * VEC, v);
      }
    }
  }
}

template <typename T, int VEC, int ACT, int UNROLL>
__global__ void __launch_bounds__(kGluBlock)
act_bwd_kernel(const T* dy, const T* x, T* dx, int64_t nv) {
  const int64_t step = (int64_t)gridDim.x * kGluBlock * UNROLL;
  for (int64_t b = (int64_t)blockIdx.x * kGluBlock * UNROLL + threadIdx.x; b < nv; b += step) {
    Packed<T, VEC> a[UNROLL], d[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int64_t i = b + (int64_t)k * kGluBlock;
      if (i < nv) {
        a[k].load(x + i * VEC);
        d[k].load(dy + i * VEC);
      }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int64_t i = b + (int64_t)k * kGluBlock;
      if (i < nv) {
        float v[VEC], dv[VEC];
        a[k].get(v);
        d[k].get(dv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float f, fp;
          act_fd<T, ACT>(v[e], f, fp);
          v[e] = dv[e] * fp;
        }
        store_n<T, VEC>(dx + i * VEC, v);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Forward with MXFP8 output (codes [T, I] and one scale byte per 32 values of
// a row), for the down projection's FP8 operand.  Same units as glu_fwd_rows;
// I is a multiple of 32, so an MX block is 32 / VEC consecutive column
// vectors, held by consecutive lanes.  Every lane runs the quantisation (its
// warp shuffles need all 32), inactive lanes with nothing to store.
// ---------------------------------------------------------------------------
template <typename T, int VEC, int ACT, int UNROLL>
__global__ void __launch_bounds__(kGluBlock)
glu_fwd_mx(const T* gate, const T* up, MxOut mx, int64_t T_, int64_t ncol, int64_t ldg,
           int64_t ldu) {
  constexpr int LB = kMxBlock / VEC;
  const int64_t I = ncol * VEC;
  const int cb = blockDim.x;
  const int64_t ncb = (ncol + cb - 1) / cb;
  const int64_t units = (T_ + UNROLL - 1) / UNROLL * ncb;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t rg = u / ncb;
    const int64_t c = (u - rg * ncb) * cb + threadIdx.x;
    const bool colok = c < ncol;
    const int64_t r0 = rg * UNROLL;
    Packed<T, VEC> g[UNROLL], v[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (colok && r0 + k < T_) {
        g[k].load(gate + (r0 + k) * ldg + c * VEC);
        v[k].load(up + (r0 + k) * ldu + c * VEC);
      }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (r0 + k >= T_) break;  // uniform across the block
      float o[VEC];
      if (colok) {
        float gf[VEC], uf[VEC];
        g[k].get(gf);
        v[k].get(uf);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = act_f<T, ACT>(gf[e]) * uf[e];
      }
      mx_store<VEC>(o, colok, c % LB == 0, mx.q + (r0 + k) * I + c * VEC,
                    mx.sc + (r0 + k) * (I / kMxBlock) + c / LB);
    }
  }
}

// f(gate) * up of N values for the kernels that also quantise.  With bf16 inputs
// the multiplications and additions of act_f go two at a time; the exponentials and
// reciprocals stay single.  Where a product meets a sum, both write out whether it is
// rounded in between (the tanh form's argument: no; 1 - erfc / 2: yes), so that they
// give the same bits: out is glu_fwd's, and codes do not depend on a row's alignment.
template <int ACT>
__device__ __forceinline__ float2 act_f2(float2 x) {
  if constexpr (ACT == GBLN_ACT_RELU) {
    return make_float2(x.x > 0.f ? x.x : 0.f, x.y > 0.f ? x.y : 0.f);
  } else if constexpr (ACT == GBLN_ACT_GELU_ERF) {
    const float2 z = mul2(make_float2(fabsf(x.x), fabsf(x.y)), both(kInvSqrt2));
    const float2 pz = fma2(both(kAsP), z, both(1.0f));
    const float2 t = make_float2(rcp_ftz(pz.x), rcp_ftz(pz.y));
    const float2 a = mul2(mul2(make_float2(-z.x, -z.y), z), both(kLog2e));
    const float2 ex = make_float2(ex2_ftz(a.x), ex2_ftz(a.y));
    const float2 poly = mul2(t, fma2(t, fma2(t, fma2(t, fma2(t, both(kAsA5), both(kAsA4)), both(kAsA3)), both(kAsA2)), both(kAsA1)));
    const float2 h = mul2(mul2(both(0.5f), poly), ex);
    const float2 up = make_float2(__fsub_rn(1.0f, h.x), __fsub_rn(1.0f, h.y));  // a paired sum may be fused
    return mul2(x, make_float2(x.x >= 0.f ? up.x : h.x, x.y >= 0.f ? up.y : h.y));
  } else {
    float2 a;  // argument of the sigmoid
    if constexpr (ACT == GBLN_ACT_SILU) {
      a = x;
    } else {
      a = mul2(both(kGeluK), fma2(mul2(mul2(both(kGeluC), x), x), x, x));
    }
    const float2 n = mul2(make_float2(-a.x, -a.y), both(kLog2e));
    const float2 d = add2(both(1.0f), make_float2(ex2_ftz(n.x), ex2_ftz(n.y)));
    return mul2(x, make_float2(rcp_ftz(d.x), rcp_ftz(d.y)));
  }
}
template <typename T, int ACT, int N>
__device__ __forceinline__ void glu_values(const float (&g)[N], const float (&u)[N], float (&o)[N]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 r = mul2(act_f2<ACT>(make_float2(g[e], g[e + 1])), make_float2(u[e], u[e + 1]));
      o[e] = r.x;
      o[e + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = act_f<T, ACT>(g[e]) * u[e];
  }
}

// ---------------------------------------------------------------------------
// Forward with row-scaled E4M3 output.  The scale needs the whole row's maximum
// before the first code, so the outputs wait for it in float32 registers (VPT
// vectors per thread): gate and up are read once.  TPR threads per row and
// block: several rows per block when TPR is a warp; one row per block beyond;
// one row per cluster of CL blocks for rows beyond 1024 threads' registers, whose
// maxima meet through distributed shared memory.  32768 x 14336 bf16, SiLU: 345 us
// (346 us at the copy rate); GeLU-erf 406 us: half as many instructions again, and 1.5
// warps wait for an arithmetic pipe at every issue (0.4 in the unaligned SiLU form).
// ---------------------------------------------------------------------------
template <typename T, int ACT, int TPR, int VPT, int RPB, int CL>
__device__ __forceinline__ void glu_row8(const T* gate, const T* up, uint8_t* q, float* sc, int64_t rows,
                                         int I, int64_t ldg, int64_t ldu) {
  static_assert((RPB == 1 || TPR == 32) && (CL == 1 || RPB == 1), "row split");
  constexpr int VEC = VecOf<T>::N;
  constexpr int FMT = GBLN_Q8_E4M3;
  constexpr int STEP = TPR * CL;  // vectors between two of a thread's
  __shared__ uint32_t redm[TPR / 32];
  __shared__ uint32_t blockm;
  const int64_t row = CL > 1 ? blockIdx.x / CL : (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row >= rows) return;  // uniform per warp; never with one row per block or cluster
  const int nvec = I / VEC, l = (CL > 1 ? (int)(blockIdx.x % CL) * TPR : 0) + threadIdx.x % TPR;
  uint4 ga[VPT], ua[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int iv = l + v * STEP;
    if (iv < nvec) {
      ga[v] = ld_stream(gate + row * ldg + (int64_t)iv * VEC);
      ua[v] = ld_stream(up + row * ldu + (int64_t)iv * VEC);
    }
  }
  float o[VPT][VEC];
  uint32_t m = 0;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (l + v * STEP < nvec) {
      float g[VEC], u[VEC];
      unpack<VEC>(ga[v], g);
      unpack<VEC>(ua[v], u);
      glu_values<T, ACT, VEC>(g, u, o[v]);
      m = max(m, abs_max_bits<VEC>(o[v]));
    }
  }
  m = group_max<32>(m);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) redm[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) m = max(m, redm[i]);
  }
  if constexpr (CL > 1) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    if (threadIdx.x == 0) blockm = m;
    cluster.sync();
#pragma unroll
    for (int i = 0; i < CL; ++i) m = max(m, *cluster.map_shared_rank(&blockm, i));
    cluster.barrier_arrive();  // this block has read its peers; waited for before it ends
  }
  const float a = q8_amax(m), inv = q8_inv<FMT>(a);
  if (l == 0) sc[row] = q8_scale<FMT>(a, m);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int iv = l + v * STEP;
    if (iv < nvec) q8_store<FMT, VEC>(o[v], inv, q + row * I + (int64_t)iv * VEC);
  }
  if constexpr (CL > 1) cooperative_groups::this_cluster().barrier_wait();
}

template <typename T, int ACT, int TPR, int VPT, int RPB>
__global__ void __launch_bounds__(TPR * RPB)
glu_fwd_row8(const T* gate, const T* up, uint8_t* q, float* sc, int64_t rows, int I, int64_t ldg,
             int64_t ldu) {
  glu_row8<T, ACT, TPR, VPT, RPB, 1>(gate, up, q, sc, rows, I, ldg, ldu);
}
template <typename T, int ACT, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(512)
glu_fwd_row8_cluster(const T* gate, const T* up, uint8_t* q, float* sc, int64_t rows, int I, int64_t ldg,
                     int64_t ldu) {
  glu_row8<T, ACT, 512, 4, 1, CL>(gate, up, q, sc, rows, I, ldg, ldu);
}

// ---------------------------------------------------------------------------
// Row-scaled output for many rows of 2049 to 4096 vectors (bf16: up to 32768
// values).  One such row fills an SM's registers while it waits for its maximum,
// so no second block covers the wait with loads of its own.  Here a persistent
// block keeps HBM busy itself: a producer warp streams gate and up of this row
// and the next through a ring of shared-memory stages (TMA bulk copies, 512
// vectors of each per stage), and 512 consumer threads turn a stage into float32
// outputs in registers, meet once per row for the maximum, and store the codes.
// 16383 x 28672 bf16: 331 us (346 us at the copy rate; this pass mostly reads),
// with a block of 1024 threads per row 497 us; 4000 rows of 16640 67 us (49), of 32768
// 101 us (97).
// ---------------------------------------------------------------------------
constexpr int kRingThreads = 512;                             // consumers
constexpr int kRingStages = 12;                               // 16 KB each
constexpr int kRingBytes = kRingThreads * 16;                 // of gate, and of up, per stage
constexpr int kRingVpt = 8;                                   // stages per row, at most

struct RingBarriers {
  uint64_t full[kRingStages], empty[kRingStages];
  uint32_t maxima[2][kRingThreads / 32];
};
constexpr size_t kRingSmem = (size_t)kRingStages * 2 * kRingBytes + sizeof(RingBarriers);

template <typename T, int ACT>
__global__ void __launch_bounds__(kRingThreads + 32, 1)
glu_fwd_row8_ring(const T* gate, const T* up, uint8_t* q, float* sc, int64_t rows, int I, int64_t ldg,
                  int64_t ldu, unsigned int* err) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int FMT = GBLN_Q8_E4M3;
  extern __shared__ __align__(128) unsigned char ring[];
  RingBarriers& B = *reinterpret_cast<RingBarriers*>(ring + (size_t)kRingStages * 2 * kRingBytes);
  const int nvec = I / VEC, per = (nvec + kRingThreads - 1) / kRingThreads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRingStages; ++s) {
      mbar_init(&B.full[s], 1);
      mbar_init(&B.empty[s], kRingThreads / 32);
    }
    mbar_init_fence();
  }
  __syncthreads();

  if (warp == kRingThreads / 32) {  // producer: one thread
    if (lane != 0) return;
    int stage = 0;
    uint32_t round = 0;  // times the ring has been filled
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
      for (int v = 0; v < per; ++v) {
        if (round > 0 && !mbar_wait(&B.empty[stage], (round - 1) & 1, kWaitPolls)) {
          atomicOr(err, kErrWaitTimeout);
          row = rows;  // nothing more is issued
          break;
        }
        const int n = nvec - v * kRingThreads < kRingThreads ? nvec - v * kRingThreads : kRingThreads;
        unsigned char* dst = ring + (size_t)stage * 2 * kRingBytes;
        const int64_t at = (int64_t)v * kRingThreads * VEC;
        mbar_arrive_expect_tx(&B.full[stage], (uint32_t)n * 32);
        bulk_load(dst, gate + row * ldg + at, (uint32_t)n * 16, &B.full[stage]);
        bulk_load(dst + kRingBytes, up + row * ldu + at, (uint32_t)n * 16, &B.full[stage]);
        if (++stage == kRingStages) {
          stage = 0;
          ++round;
        }
      }
    }
    // The block's memory outlives its copies: wait for those still in flight.
    for (int s = 0; s < kRingStages; ++s) {
      const uint32_t fills = round + (s < stage ? 1 : 0);
      if (fills > 0 && !mbar_wait(&B.full[s], (fills - 1) & 1, kWaitPolls)) atomicOr(err, kErrWaitTimeout);
    }
    return;
  }

  int stage = 0;
  uint32_t phase = 0;
  int par = 0;
  bool good = true;  // false: a wait ran out, results are void, nothing waits any more
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, par ^= 1) {
    float o[kRingVpt][VEC];
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < kRingVpt; ++v) {
      if (v < per) {
        if (good && !mbar_wait(&B.full[stage], phase, kWaitPolls)) {
          good = false;
          atomicOr(err, kErrWaitTimeout);
        }
        const unsigned char* src = ring + (size_t)stage * 2 * kRingBytes + (size_t)threadIdx.x * 16;
        const uint4 ga = ld_shared_v4(src), ua = ld_shared_v4(src + kRingBytes);
        float g[VEC], u[VEC];
        unpack<VEC>(ga, g);
        unpack<VEC>(ua, u);
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.empty[stage]);
        if (++stage == kRingStages) {
          stage = 0;
          phase ^= 1;
        }
        glu_values<T, ACT, VEC>(g, u, o[v]);
        if (v * kRingThreads + (int)threadIdx.x < nvec) m = max(m, abs_max_bits<VEC>(o[v]));
      }
    }
    m = group_max<32>(m);
    if (lane == 0) B.maxima[par][warp] = m;
    // a buffer is written again two rows later, past the next barrier
    bar_sync_named(1, kRingThreads);
#pragma unroll
    for (int i = 0; i < kRingThreads / 32; ++i) m = max(m, B.maxima[par][i]);
    const float a = q8_amax(m), inv = q8_inv<FMT>(a);
    if (threadIdx.x == 0) sc[row] = q8_scale<FMT>(a, m);
#pragma unroll
    for (int v = 0; v < kRingVpt; ++v) {
      const int iv = v * kRingThreads + threadIdx.x;
      if (v < per && iv < nvec) q8_store<FMT, VEC>(o[v], inv, q + row * I + (int64_t)iv * VEC);
    }
  }
}

// Runs of 128 consecutive values of a row for the element-wise paths: lane l holds
// the values l, l + 32, l + 64, l + 96 (offsets are immediates); rem = values from
// the lane's first one to the row's end, looked at where the run is not FULL.
template <bool FULL, typename T>
__device__ __forceinline__ void load_run(const T* p, int rem, T (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = FULL || 32 * e < rem ? p[32 * e] : T(0.f);
}
template <bool FULL>
__device__ __forceinline__ uint32_t load_run_codes(const uint8_t* p, int rem) {
  uint32_t b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = FULL || 32 * e < rem ? (uint32_t)p[32 * e] : 0u;
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}
template <bool FULL, typename T>
__device__ __forceinline__ void store_run(T* p, int rem, const float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (FULL || 32 * e < rem) p[32 * e] = from_f32<T>(v[e]);
}
template <bool FULL, int FMT>
__device__ __forceinline__ void store_run_codes(uint8_t* p, int rem, const float (&v)[4], float inv) {
  const uint32_t q = q8_code4<FMT>(v[0], v[1], v[2], v[3], inv);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (FULL || 32 * e < rem) p[32 * e] = (uint8_t)(q >> (8 * e));
}

// The same for any alignment and width.  A warp takes runs of 128 values, lane l
// the values l, l + 32, l + 64, l + 96 of each; up to kRow8Runs runs per warp wait
// in registers (blocks of up to 1024 threads: 16384 values), wider rows are read
// a second time to write the codes.  8190 x 4097 bf16 38 us (25 us at the copy
// rate): one value per lane and access, 70% of the issue slots and half of an SM's
// warps in use, which wait for their loads.
constexpr int kRow8Runs = 4;

template <typename T, int ACT, bool FITS>
__global__ void __launch_bounds__(1024)
glu_fwd_row8_elem(const T* gate, const T* up, uint8_t* q, float* sc, int64_t rows, int64_t I,
                  int64_t ldg, int64_t ldu) {
  constexpr int FMT = GBLN_Q8_E4M3;
  __shared__ uint32_t redm[32];
  const int64_t row = blockIdx.x;
  const int nw = blockDim.x / 32, warp = warp_index(), lane = threadIdx.x & 31;
  const int j0 = warp * 128;  // the warp's first run
  const T* gr = gate + row * ldg;
  const T* ur = up + row * ldu;
  uint8_t* qr = q + row * I;
  float o[FITS ? kRow8Runs : 1][4];
  uint32_t m = 0;
  if constexpr (FITS) {
    T g[kRow8Runs][4], u[kRow8Runs][4];
#pragma unroll
    for (int k = 0; k < kRow8Runs; ++k) {
      const int j = j0 + k * nw * 128;
      if (j + 128 <= I) {
        load_run<true>(gr + j + lane, 0, g[k]);
        load_run<true>(ur + j + lane, 0, u[k]);
      } else {
        load_run<false>(gr + j + lane, (int)I - j - lane, g[k]);
        load_run<false>(ur + j + lane, (int)I - j - lane, u[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kRow8Runs; ++k)
      if (j0 + k * nw * 128 < I) {
        float gf[4], uf[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          gf[e] = to_f32(g[k][e]);
          uf[e] = to_f32(u[k][e]);
        }
        glu_values<T, ACT, 4>(gf, uf, o[k]);
        m = max(m, abs_max_bits<4>(o[k]));
      }
  } else {
    for (int64_t j = threadIdx.x; j < I; j += blockDim.x)
      m = max(m, abs_bits(act_f<T, ACT>(to_f32(gr[j])) * to_f32(ur[j])));
  }
  m = group_max<32>(m);
  if ((threadIdx.x & 31) == 0) redm[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int i = 0; i < nw; ++i) m = max(m, redm[i]);
  const float a = q8_amax(m), inv = q8_inv<FMT>(a);
  if (threadIdx.x == 0) sc[row] = q8_scale<FMT>(a, m);
  if constexpr (FITS) {
#pragma unroll
    for (int k = 0; k < kRow8Runs; ++k)
      if (const int j = j0 + k * nw * 128; j + 128 <= I) store_run_codes<true, FMT>(qr + j + lane, 0, o[k], inv);
      else if (j < I) store_run_codes<false, FMT>(qr + j + lane, (int)I - j - lane, o[k], inv);
  } else {
    for (int64_t j = threadIdx.x; j < I; j += blockDim.x)
      qr[j] = (uint8_t)q8_code1<FMT>(act_f<T, ACT>(to_f32(gr[j])) * to_f32(ur[j]), inv);
  }
}

// ---------------------------------------------------------------------------
// Forward that also saves gate and up as 8-bit checkpoints.  Units as in
// glu_fwd_rows; a checkpoint group is LPG = 128 / VEC consecutive column vectors,
// held by consecutive lanes (blockDim is a multiple of 32, so column blocks start
// at a group), and every lane takes part in the reductions.
//
// Four rows of gate and up give a lane eight groups to reduce.  Each halving step
// of the reduction also halves the number of groups a lane looks after, so that
// eight reductions cost eight shuffles instead of thirty-two, and leave each
// group's maximum with two lanes (four at float32): one divides for 1 / scale,
// the other for the scale.  With a reduction and two divisions per lane and
// group instead, the kernel ran at 81% of the copy rate.
// 32768 x 14336 bf16, SiLU: 555 us (558 us at the copy rate).
// ---------------------------------------------------------------------------
struct GluCkpt {
  uint8_t* gq;
  float* gs;
  uint8_t* uq;
  float* us;
};
struct GluCkptIn {
  const uint8_t* gq;
  const float* gs;
  const uint8_t* uq;
  const float* us;
};

constexpr int kCkptRows = 4;
// Blocks per SM, far more than are resident: blocks that end and start at different
// times keep loads and stores mixed, where resident ones that loop over all the
// units fall into step (forward 549..556 us from 64 to 128 blocks, 573 at 24, 620
// at the 3 that are resident; 32768 x 14336 bf16, 558 us at the copy rate).  With
// one unit per block the GeLU forms lose what the loop overlaps (655 us).
constexpr int kCkptGrid = 64;

// u / n of unit numbers, which fit 32 bits in all but absurd sizes (a 64-bit
// division takes as long as a dozen values).
__device__ __forceinline__ int64_t unit_div(int64_t u, int64_t n, bool small) {
  return small ? (int64_t)((uint32_t)u / (uint32_t)n) : u / n;
}

template <typename T, int ACT, int FMT>
__global__ void __launch_bounds__(kGluBlock, 3)
glu_fwd_ckpt(const T* gate, const T* up, T* out, const GluCkpt C, int64_t T_, int64_t ncol, int64_t ldg,
             int64_t ldu, int64_t ldo) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int LPG = kCkptGroup / VEC;  // 16 or 32 lanes per group
  constexpr int U = kCkptRows;
  constexpr int SH = LPG == 16 ? 1 : 2;  // lane bits below those that name a group
  const int64_t I = ncol * VEC, ng = (ncol + LPG - 1) / LPG;
  const int cb = blockDim.x, lane = threadIdx.x & 31;
  const int64_t ncb = (ncol + cb - 1) / cb;
  const int64_t units = (T_ + U - 1) / U * ncb;
  const bool small = units <= 0xffffffffLL;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t rg = unit_div(u, ncb, small);
    const int64_t c = (u - rg * ncb) * cb + threadIdx.x;
    const bool on = c < ncol;
    const int64_t r0 = rg * U;
    const int nr = (int)(T_ - r0 < U ? T_ - r0 : (int64_t)U);
    uint4 g[U], v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      g[k] = v[k] = make_uint4(0, 0, 0, 0);
      if (on && k < nr) {
        g[k] = ld_stream(gate + (r0 + k) * ldg + c * VEC);
        v[k] = ld_stream(up + (r0 + k) * ldu + c * VEC);
      }
    }
    // The block's next unit on its way to L2: cb / 8 lines of each row and tensor, one
    // per thread.
    if (u + gridDim.x < units) {
      const int64_t un = u + gridDim.x, rn = unit_div(un, ncb, small);
      const int n = cb / 8, row8 = threadIdx.x / n, line = threadIdx.x - row8 * n;
      const int64_t col = ((un - rn * ncb) * cb + line * 8) * VEC, r = rn * U + (row8 >> 1);
      if (r < T_ && col < I) prefetch_line((row8 & 1 ? up + r * ldu : gate + r * ldg) + col);
    }
    uint32_t m[2 * U];  // gate and up of row 0, of row 1, ...
#pragma unroll
    for (int k = 0; k < U; ++k) {
      m[2 * k] = AbsMax<T>::part(g[k]);
      m[2 * k + 1] = AbsMax<T>::part(v[k]);
    }
#pragma unroll
    for (int n = U, o = LPG / 2; n >= 1; n /= 2, o /= 2) {  // n groups kept per lane
      const bool hi = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? m[i] : m[i + n], o);
        m[i] = AbsMax<T>::join(hi ? m[i + n] : m[i], got);
      }
    }
#pragma unroll
    for (int o = 1 << (SH - 1); o > 0; o >>= 1) m[0] = AbsMax<T>::join(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    const int mine = (lane & (LPG - 1)) >> SH;  // the group left with this lane: 2 * row + (up)
    const uint32_t bits = AbsMax<T>::bits(m[0]);
    const float a = q8_amax(bits);
    const bool scales = (lane & 1) != 0;
    const float d = __fdiv_rn(scales ? a : Q8Max<FMT>::v, scales ? Q8Max<FMT>::v : a);
    if (scales && (SH == 1 || (lane & 2) == 0) && (mine >> 1) < nr && (c & ~(int64_t)(LPG - 1)) < ncol)
      (mine & 1 ? C.us : C.gs)[(r0 + (mine >> 1)) * ng + c / LPG] = bits < kInfBits ? d : __int_as_float(0x7fc00000);
    const int base = lane & ~(LPG - 1);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float gi = __shfl_sync(0xffffffffu, d, base | ((2 * k) << SH));
      const float ui = __shfl_sync(0xffffffffu, d, base | ((2 * k + 1) << SH));
      if (on && k < nr) {
        float gf[VEC], uf[VEC], o[VEC];
        unpack<VEC>(g[k], gf);
        unpack<VEC>(v[k], uf);
        q8_store<FMT, VEC>(gf, gi, C.gq + (r0 + k) * I + c * VEC);
        q8_store<FMT, VEC>(uf, ui, C.uq + (r0 + k) * I + c * VEC);
        glu_values<T, ACT, VEC>(gf, uf, o);
        st_vec(out + (r0 + k) * ldo + c * VEC, pack<T, VEC>(o));
      }
    }
  }
}

// Any alignment and width: a warp takes four consecutive checkpoint groups of a row,
// lane l the values l, l + 32, l + 64, l + 96 of each; the groups share one division
// and the 64-bit addresses, which two groups of their own addresses spent a tenth of
// the time on.  8190 x 4097 bf16 55 us (that form 62), the backward 60 (68), of 40 us
// at the copy rate: issue slots 56 and 63%, 40 and 50% of an SM's warps, waiting for loads.
constexpr int kElemGroups = 4;

// unit(F, FULL, first value, values) over a warp's `left` values: four groups at once
// where they are whole, else one by one.
template <typename Unit>
__device__ __forceinline__ void row_groups(int left, Unit unit) {
  using One = std::integral_constant<int, 1>;
  if (left == kElemGroups * kCkptGroup) {
    unit(std::integral_constant<int, kElemGroups>{}, std::true_type{}, 0, left);
  } else {
    int c = 0;
    for (; c + kCkptGroup <= left; c += kCkptGroup) unit(One{}, std::true_type{}, c, kCkptGroup);
    if (c < left) unit(One{}, std::false_type{}, c, left - c);
  }
}

template <typename T, int ACT, int FMT, int F, bool FULL>
__device__ __forceinline__ void glu_fwd_ckpt_unit(const T* gp, const T* up, T* op, uint8_t* gq, uint8_t* uq,
                                                  float* gs, float* us, int left, int lane) {
  T g[F][4], v[F][4];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    load_run<FULL>(gp + f * kCkptGroup, left - f * kCkptGroup - lane, g[f]);
    load_run<FULL>(up + f * kCkptGroup, left - f * kCkptGroup - lane, v[f]);
  }
  // Lane 4 f divides for 1 / scale of gate's group f, lane 4 f + 2 of up's, the lane
  // after each for the scale.
  uint32_t mine = 0;
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const float gf[4] = {to_f32(g[f][0]), to_f32(g[f][1]), to_f32(g[f][2]), to_f32(g[f][3])};
    const float uf[4] = {to_f32(v[f][0]), to_f32(v[f][1]), to_f32(v[f][2]), to_f32(v[f][3])};
    const uint32_t gm = group_max<32>(abs_max_bits<4>(gf)), um = group_max<32>(abs_max_bits<4>(uf));
    if (lane >> 2 == f) mine = lane & 2 ? um : gm;
  }
  const float a = q8_amax(mine);
  const float d = __fdiv_rn(lane & 1 ? a : Q8Max<FMT>::v, lane & 1 ? Q8Max<FMT>::v : a);
  if (lane < 4 * F && (lane & 1) && (FULL || (lane >> 2) * kCkptGroup < left))
    (lane & 2 ? us : gs)[lane >> 2] = mine < kInfBits ? d : __int_as_float(0x7fc00000);
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const float gi = __shfl_sync(0xffffffffu, d, 4 * f), ui = __shfl_sync(0xffffffffu, d, 4 * f + 2);
    const float gf[4] = {to_f32(g[f][0]), to_f32(g[f][1]), to_f32(g[f][2]), to_f32(g[f][3])};
    const float uf[4] = {to_f32(v[f][0]), to_f32(v[f][1]), to_f32(v[f][2]), to_f32(v[f][3])};
    const int rem = left - f * kCkptGroup - lane;
    float o[4];
    glu_values<T, ACT, 4>(gf, uf, o);
    store_run<FULL>(op + f * kCkptGroup, rem, o);
    store_run_codes<FULL, FMT>(gq + f * kCkptGroup, rem, gf, gi);
    store_run_codes<FULL, FMT>(uq + f * kCkptGroup, rem, uf, ui);
  }
}

template <typename T, int ACT, int FMT>
__global__ void __launch_bounds__(kGluBlock)
glu_fwd_ckpt_elem(const T* gate, const T* up, T* out, const GluCkpt C, int64_t T_, int64_t I, int64_t ldg,
                  int64_t ldu, int64_t ldo) {
  constexpr int W = kElemGroups * kCkptGroup;  // values per unit
  const int lane = threadIdx.x & 31;
  const int64_t ng = (I + kCkptGroup - 1) / kCkptGroup, nu = (I + W - 1) / W, n = T_ * nu;
  const bool small = n <= 0xffffffffLL;
  const int64_t step = (int64_t)gridDim.x * (kGluBlock / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kGluBlock / 32) + warp_index(); u < n; u += step) {
    const int64_t row = unit_div(u, nu, small), c = (u - row * nu) * W;
    const int left = I - c < W ? (int)(I - c) : W;
    const T *gp = gate + row * ldg + c + lane, *vp = up + row * ldu + c + lane;
    T* op = out + row * ldo + c + lane;
    const int64_t at = row * I + c + lane, sc = row * ng + c / kCkptGroup;
    auto unit = [&](auto f, auto full, int at0, int n) {
      glu_fwd_ckpt_unit<T, ACT, FMT, f.value, full.value>(gp + at0, vp + at0, op + at0, C.gq + at + at0, C.uq + at + at0,
                                                          C.gs + sc + at0 / kCkptGroup, C.us + sc + at0 / kCkptGroup, n, lane);
    };
    row_groups(left, unit);
  }
}

// ---------------------------------------------------------------------------
// Backward from the checkpoints, units as in glu_fwd_ckpt (four rows at a time
// keep twice the loads in flight of glu_bwd_rows' two: 563 against 573 us).  A
// lane's VEC columns lie in one group: VEC divides 128.  32768 x 14336 bf16, SiLU:
// 557 us, GeLU-erf 575 us (558 us at the copy rate).
// ---------------------------------------------------------------------------
template <typename T, int ACT, int FMT, int UNROLL>
__global__ void __launch_bounds__(kGluBlock)
glu_bwd_ckpt(const T* dout, const GluCkptIn C, T* dgate, T* dup, int64_t T_, int64_t ncol, int64_t ldd,
             int64_t lddg, int64_t lddu) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int LPG = kCkptGroup / VEC;
  const int64_t I = ncol * VEC, ng = (ncol + LPG - 1) / LPG;
  const int cb = blockDim.x;
  const int64_t ncb = (ncol + cb - 1) / cb;
  const int64_t units = (T_ + UNROLL - 1) / UNROLL * ncb;
  const bool small = units <= 0xffffffffLL;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t rg = unit_div(u, ncb, small);
    const int64_t c = (u - rg * ncb) * cb + threadIdx.x;
    if (c >= ncol) continue;
    const int64_t r0 = rg * UNROLL;
    Packed<T, VEC> d[UNROLL];
    Codes<FMT, VEC> g[UNROLL], v[UNROLL];
    float gs[UNROLL], us[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (r0 + k < T_) {
        d[k].load(dout + (r0 + k) * ldd + c * VEC);
        g[k].load(C.gq + (r0 + k) * I + c * VEC);
        v[k].load(C.uq + (r0 + k) * I + c * VEC);
        gs[k] = __ldg(C.gs + (r0 + k) * ng + c / LPG);
        us[k] = __ldg(C.us + (r0 + k) * ng + c / LPG);
      }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (r0 + k < T_) {
        float df[VEC], gf[VEC], uf[VEC], dg[VEC], du[VEC];
        d[k].get(df);
        g[k].get(gf, gs[k]);
        v[k].get(uf, us[k]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float f, fp;
          act_fd<T, ACT>(gf[e], f, fp);
          du[e] = df[e] * f;
          dg[e] = df[e] * uf[e] * fp;
        }
        store_n<T, VEC>(dgate + (r0 + k) * lddg + c * VEC, dg);
        store_n<T, VEC>(dup + (r0 + k) * lddu + c * VEC, du);
      }
    }
  }
}

// Any alignment and width, as glu_fwd_ckpt_elem.
template <typename T, int ACT, int FMT, int F, bool FULL>
__device__ __forceinline__ void glu_bwd_ckpt_unit(const T* dp, const uint8_t* gq, const uint8_t* uq, const float* gs,
                                                  const float* us, T* dgp, T* dup, int left, int lane) {
  T d[F][4];
  uint32_t g[F], v[F];
  float sg[F], su[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int rem = left - f * kCkptGroup - lane;
    load_run<FULL>(dp + f * kCkptGroup, rem, d[f]);
    g[f] = load_run_codes<FULL>(gq + f * kCkptGroup, rem);
    v[f] = load_run_codes<FULL>(uq + f * kCkptGroup, rem);
    const bool in = FULL || f * kCkptGroup < left;
    sg[f] = in ? __ldg(gs + f) : 0.f;
    su[f] = in ? __ldg(us + f) : 0.f;
  }
#pragma unroll
  for (int f = 0; f < F; ++f) {
    float gf[4], uf[4], dg[4], du[4];
    q8_decode4<FMT>(g[f], gf);
    q8_decode4<FMT>(v[f], uf);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float df = to_f32(d[f][e]);
      float fx, fp;
      act_fd<T, ACT>(__fmul_rn(gf[e], sg[f]), fx, fp);
      du[e] = df * fx;
      dg[e] = df * __fmul_rn(uf[e], su[f]) * fp;
    }
    const int rem = left - f * kCkptGroup - lane;
    store_run<FULL>(dgp + f * kCkptGroup, rem, dg);
    store_run<FULL>(dup + f * kCkptGroup, rem, du);
  }
}

template <typename T, int ACT, int FMT>
__global__ void __launch_bounds__(kGluBlock)
glu_bwd_ckpt_elem(const T* dout, const GluCkptIn C, T* dgate, T* dup, int64_t T_, int64_t I, int64_t ldd,
                  int64_t lddg, int64_t lddu) {
  constexpr int W = kElemGroups * kCkptGroup;
  const int lane = threadIdx.x & 31;
  const int64_t ng = (I + kCkptGroup - 1) / kCkptGroup, nu = (I + W - 1) / W, n = T_ * nu;
  const bool small = n <= 0xffffffffLL;
  const int64_t step = (int64_t)gridDim.x * (kGluBlock / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kGluBlock / 32) + warp_index(); u < n; u += step) {
    const int64_t row = unit_div(u, nu, small), c = (u - row * nu) * W;
    const int left = I - c < W ? (int)(I - c) : W;
    const T* dp = dout + row * ldd + c + lane;
    T *gp = dgate + row * lddg + c + lane, *vp = dup + row * lddu + c + lane;
    const int64_t at = row * I + c + lane, sc = row * ng + c / kCkptGroup;
    auto unit = [&](auto f, auto full, int at0, int n) {
      glu_bwd_ckpt_unit<T, ACT, FMT, f.value, full.value>(dp + at0, C.gq + at + at0, C.uq + at + at0,
                                                          C.gs + sc + at0 / kCkptGroup, C.us + sc + at0 / kCkptGroup,
                                                          gp + at0, vp + at0, n, lane);
    };
    row_groups(left, unit);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

unsigned resident_grid(int64_t units, int threads = kGluBlock) {
  const int sms = sm_count();
  const int64_t cap = (int64_t)(sms > 0 ? sms : 1) * (2048 / threads);
  return grid_for(units, 1, cap);
}

// Threads per block of the row-strided kernels: the multiple of 32 in
// [128, kGluBlock] whose column blocks cover a row of ncol units with the
// fewest idle lanes, the widest on a tie.  A bf16 row of 3072 values (384
// vectors) gets two blocks of 192 instead of one and a half of 256.
int col_block(int64_t ncol) {
  int best = kGluBlock;
  int64_t best_slots = -1;
  for (int b = kGluBlock; b >= 128; b -= 32) {
    const int64_t slots = (ncol + b - 1) / b * b;
    if (best_slots < 0 || slots < best_slots) {
      best = b;
      best_slots = slots;
    }
  }
  return best;
}

template <typename T, int ACT>
void glu_fwd_launch(const void* g, const void* u, void* o, int64_t rows, int64_t I, int64_t ldg,
                    int64_t ldu, int64_t ldo, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const bool contiguous = ldg == I && ldu == I && ldo == I;
  const bool aligned = aligned16(g) && aligned16(u) && aligned16(o);
  if (contiguous && aligned && (rows * I) % VEC == 0) {
    constexpr int U = 4;
    const int64_t nvec = rows * I / VEC;
    glu_fwd_vec<T, ACT, U><<<resident_grid((nvec + U - 1) / U / kGluBlock + 1), kGluBlock, 0, s>>>(
        (const T*)g, (const T*)u, (T*)o, nvec);
  } else if (aligned && I % VEC == 0 && ldg % VEC == 0 && ldu % VEC == 0 && ldo % VEC == 0) {
    constexpr int U = 4;
    const int64_t ncol = I / VEC;
    const int cb = col_block(ncol);
    const int64_t units = (rows + U - 1) / U * ((ncol + cb - 1) / cb);
    glu_fwd_rows<T, VEC, ACT, U><<<resident_grid(units, cb), cb, 0, s>>>(
        (const T*)g, (const T*)u, (T*)o, rows, ncol, ldg, ldu, ldo);
  } else {
    constexpr int U = 4;
    const int cb = col_block(I);
    const int64_t units = (rows + U - 1) / U * ((I + cb - 1) / cb);
    glu_fwd_rows<T, 1, ACT, U><<<resident_grid(units, cb), cb, 0, s>>>(
        (const T*)g, (const T*)u, (T*)o, rows, I, ldg, ldu, ldo);
  }
}

template <typename T, int ACT>
void glu_fwd_mx_launch(const void* g, const void* u, MxOut mx, int64_t rows, int64_t I, int64_t ldg,
                       int64_t ldu, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int U = 4;
  const bool vec = aligned16(g) && aligned16(u) && ldg % VEC == 0 && ldu % VEC == 0 &&
                   reinterpret_cast<uintptr_t>(mx.q) % VEC == 0;  // VEC codes per lane
  if (vec) {
    const int64_t ncol = I / VEC;
    const int cb = col_block(ncol);
    const int64_t units = (rows + U - 1) / U * ((ncol + cb - 1) / cb);
    glu_fwd_mx<T, VEC, ACT, U><<<resident_grid(units, cb), cb, 0, s>>>((const T*)g, (const T*)u, mx,
                                                                          rows, ncol, ldg, ldu);
  } else {
    const int cb = col_block(I);
    const int64_t units = (rows + U - 1) / U * ((I + cb - 1) / cb);
    glu_fwd_mx<T, 1, ACT, U><<<resident_grid(units, cb), cb, 0, s>>>((const T*)g, (const T*)u, mx,
                                                                        rows, I, ldg, ldu);
  }
}

template <typename T, int ACT>
void glu_bwd_launch(const void* d, const void* g, const void* u, void* dg, void* du, int64_t rows,
                    int64_t I, int64_t ldd, int64_t ldg, int64_t ldu, int64_t lddg, int64_t lddu,
                    cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const bool contiguous = ldd == I && ldg == I && ldu == I && lddg == I && lddu == I;
  const bool aligned = aligned16(d) && aligned16(g) && aligned16(u) && aligned16(dg) && aligned16(du);
  if (contiguous && aligned && (rows * I) % VEC == 0) {
    constexpr int U = 4;
    const int64_t nvec = rows * I / VEC;
    glu_bwd_vec<T, ACT, U><<<resident_grid((nvec + U - 1) / U / kGluBlock + 1), kGluBlock, 0, s>>>(
        (const T*)d, (const T*)g, (const T*)u, (T*)dg, (T*)du, nvec);
  } else if (aligned && I % VEC == 0 && ldd % VEC == 0 && ldg % VEC == 0 && ldu % VEC == 0 &&
             lddg % VEC == 0 && lddu % VEC == 0) {
    constexpr int U = 2;
    const int64_t ncol = I / VEC;
    const int cb = col_block(ncol);
    const int64_t units = (rows + U - 1) / U * ((ncol + cb - 1) / cb);
    glu_bwd_rows<T, VEC, ACT, U><<<resident_grid(units, cb), cb, 0, s>>>(
        (const T*)d, (const T*)g, (const T*)u, (T*)dg, (T*)du, rows, ncol, ldd, ldg, ldu, lddg, lddu);
  } else {
    constexpr int U = 2;
    const int cb = col_block(I);
    const int64_t units = (rows + U - 1) / U * ((I + cb - 1) / cb);
    glu_bwd_rows<T, 1, ACT, U><<<resident_grid(units, cb), cb, 0, s>>>(
        (const T*)d, (const T*)g, (const T*)u, (T*)dg, (T*)du, rows, I, ldd, ldg, ldu, lddg, lddu);
  }
}

template <typename T, int ACT>
void act_fwd_launch(const void* x, void* y, int64_t n, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int U = 4;
  if (aligned16(x) && aligned16(y) && n % VEC == 0) {
    const int64_t nv = n / VEC;
    act_fwd_kernel<T, VEC, ACT, U><<<resident_grid((nv + U - 1) / U / kGluBlock + 1), kGluBlock, 0, s>>>(
        (const T*)x, (T*)y, nv);
  } else {
    act_fwd_kernel<T, 1, ACT, U><<<resident_grid((n + U - 1) / U / kGluBlock + 1), kGluBlock, 0, s>>>(
        (const T*)x, (T*)y, n);
  }
}

template <typename T, int ACT>
void act_bwd_launch(const void* dy, const void* x, void* dx, int64_t n, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int U = 4;
  if (aligned16(x) && aligned16(dy) && aligned16(dx) && n % VEC == 0) {
    const int64_t nv = n / VEC;
    act_bwd_kernel<T, VEC, ACT, U><<<resident_grid((nv + U - 1) / U / kGluBlock + 1), kGluBlock, 0, s>>>(
        (const T*)dy, (const T*)x, (T*)dx, nv);
  } else {
    act_bwd_kernel<T, 1, ACT, U><<<resident_grid((n + U - 1) / U / kGluBlock + 1), kGluBlock, 0, s>>>(
        (const T*)dy, (const T*)x, (T*)dx, n);
  }
}

template <typename T, int ACT>
gbln_status glu_fwd_row8_ring_launch(const T* g, const T* u, uint8_t* q, float* sc, int64_t rows, int I, int64_t ldg,
                                     int64_t ldu, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};  // one bit per device
  int dev = 0;
  unsigned int* err = device_error_word();
  if (!err || cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return GBLN_ERR_CUDA; }
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(glu_fwd_row8_ring<T, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingSmem) !=
        cudaSuccess) {
      cudaGetLastError();
      return GBLN_ERR_CUDA;
    }
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  glu_fwd_row8_ring<T, ACT><<<grid_for(rows, 1, sms), kRingThreads + 32, kRingSmem, s>>>(g, u, q, sc, rows, I, ldg,
                                                                                         ldu, err);
  return launch_status();
}

// Row-scaled output: a warp per row up to 128 vectors, then a block of 64 to 1024
// threads with four vectors each, then a cluster of 512-thread blocks.
template <typename T, int ACT>
gbln_status glu_fwd_row8_launch(const void* g, const void* u, uint8_t* q, float* sc, int64_t rows, int64_t I,
                                int64_t ldg, int64_t ldu, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return GBLN_ERR_CUDA;
  constexpr int VEC = VecOf<T>::N;
  constexpr int64_t kMaxGrid = 0x7fffffff;
  const int64_t nvec = I / VEC;
  const int cl = nvec <= 4096 ? 1 : nvec <= 8192 ? 4 : 8;
  const bool vec = I % VEC == 0 && nvec <= 8 * 2048 && rows * cl <= kMaxGrid && aligned16(g) && aligned16(u) &&
                   ldg % VEC == 0 && ldu % VEC == 0 && aligned_to(q, VEC);
  const T *gt = (const T*)g, *ut = (const T*)u;
  if (!vec) {
    const int64_t nw = (I + 128 * kRow8Runs - 1) / (128 * kRow8Runs);
    if (nw <= 32)
      glu_fwd_row8_elem<T, ACT, true><<<(unsigned)rows, (int)nw * 32, 0, s>>>(gt, ut, q, sc, rows, I, ldg, ldu);
    else
      glu_fwd_row8_elem<T, ACT, false><<<(unsigned)rows, 512, 0, s>>>(gt, ut, q, sc, rows, I, ldg, ldu);
    return launch_status();
  }
#define GBLN_ROW8(TPR, VPT, RPB) \
  glu_fwd_row8<T, ACT, TPR, VPT, RPB><<<(unsigned)((rows + RPB - 1) / RPB), TPR * RPB, 0, s>>>(gt, ut, q, sc, rows, (int)I, ldg, ldu)
#define GBLN_ROW8_CLUSTER(CL) \
  glu_fwd_row8_cluster<T, ACT, CL><<<(unsigned)(rows * CL), 512, 0, s>>>(gt, ut, q, sc, rows, (int)I, ldg, ldu)
  if (nvec <= 32) GBLN_ROW8(32, 1, 8);
  else if (nvec <= 64) GBLN_ROW8(32, 2, 8);
  else if (nvec <= 128) GBLN_ROW8(32, 4, 8);
  else if (nvec <= 256) GBLN_ROW8(64, 4, 1);
  else if (nvec <= 512) GBLN_ROW8(128, 4, 1);
  else if (nvec <= 1024) GBLN_ROW8(256, 4, 1);
  else if (nvec <= 2048) GBLN_ROW8(512, 4, 1);
  else if (cl == 1 && rows > sms)  // a row for each SM: 6.7 us either way; 2000 rows of 28672: 48 against 66 us
    return glu_fwd_row8_ring_launch<T, ACT>(gt, ut, q, sc, rows, (int)I, ldg, ldu, sms, s);
  else if (cl == 1) GBLN_ROW8(1024, 4, 1);
  else if (cl == 4) GBLN_ROW8_CLUSTER(4);
  else GBLN_ROW8_CLUSTER(8);
#undef GBLN_ROW8
#undef GBLN_ROW8_CLUSTER
  return launch_status();
}

template <typename T, int ACT, int FMT>
void glu_fwd_ckpt_launch(const void* g, const void* u, void* o, GluCkpt C, int64_t rows, int64_t I,
                         int64_t ldg, int64_t ldu, int64_t ldo, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const bool vec = I % VEC == 0 && aligned16(g) && aligned16(u) && aligned16(o) && ldg % VEC == 0 &&
                   ldu % VEC == 0 && ldo % VEC == 0 && aligned_to(C.gq, VEC) && aligned_to(C.uq, VEC);
  if (vec) {
    const int64_t ncol = I / VEC;
    const int cb = col_block(ncol);
    const int64_t units = (rows + kCkptRows - 1) / kCkptRows * ((ncol + cb - 1) / cb);
    glu_fwd_ckpt<T, ACT, FMT><<<grid_for(units, 1, (int64_t)sm_count() * kCkptGrid), cb, 0, s>>>((const T*)g, (const T*)u, (T*)o, C,
                                                                        rows, ncol, ldg, ldu, ldo);
  } else {
    const int64_t units = rows * ((I + kElemGroups * kCkptGroup - 1) / (kElemGroups * kCkptGroup)), per = kGluBlock / 32;
    glu_fwd_ckpt_elem<T, ACT, FMT><<<grid_for((units + per - 1) / per, 1, (int64_t)sm_count() * kCkptGrid), kGluBlock, 0, s>>>(
        (const T*)g, (const T*)u, (T*)o, C, rows, I, ldg, ldu, ldo);
  }
}

template <typename T, int ACT, int FMT>
void glu_bwd_ckpt_launch(const void* d, GluCkptIn C, void* dg, void* du, int64_t rows, int64_t I,
                         int64_t ldd, int64_t lddg, int64_t lddu, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int U = kCkptRows;
  const bool vec = I % VEC == 0 && aligned16(d) && aligned16(dg) && aligned16(du) && ldd % VEC == 0 &&
                   lddg % VEC == 0 && lddu % VEC == 0 && aligned_to(C.gq, VEC) && aligned_to(C.uq, VEC);
  if (vec) {
    const int64_t ncol = I / VEC;
    const int cb = col_block(ncol);
    const unsigned grid = grid_for((rows + U - 1) / U * ((ncol + cb - 1) / cb), 1, (int64_t)sm_count() * kCkptGrid);
    glu_bwd_ckpt<T, ACT, FMT, U><<<grid, cb, 0, s>>>((const T*)d, C, (T*)dg, (T*)du, rows, ncol, ldd, lddg, lddu);
  } else {
    const int64_t units = rows * ((I + kElemGroups * kCkptGroup - 1) / (kElemGroups * kCkptGroup)), per = kGluBlock / 32;
    glu_bwd_ckpt_elem<T, ACT, FMT><<<grid_for((units + per - 1) / per, 1, (int64_t)sm_count() * kCkptGrid), kGluBlock, 0, s>>>(
        (const T*)d, C, (T*)dg, (T*)du, rows, I, ldd, lddg, lddu);
  }
}

// Dispatch on (io, act) to a templated launcher F<T, ACT>::run(args...).
#define GBLN_DISPATCH_ACT(T, act, CALL)                       \
  switch (act) {                                              \
    case GBLN_ACT_SILU: CALL(T, GBLN_ACT_SILU); break;        \
    case GBLN_ACT_GELU_TANH: CALL(T, GBLN_ACT_GELU_TANH); break; \
    case GBLN_ACT_GELU_ERF: CALL(T, GBLN_ACT_GELU_ERF); break; \
    default: CALL(T, GBLN_ACT_RELU); break;                   \
  }

bool act_ok(int a) { return a >= GBLN_ACT_SILU && a <= GBLN_ACT_RELU; }

bool sizes_ok(int64_t T, int64_t I) {
  if (T < 0 || I <= 0) return false;
  return T <= (INT64_MAX / 16) / I;  // T * I * 16 bytes does not overflow
}

// Strides: at least the row width, and the last row's end must not overflow.
bool ld_ok(int64_t T, int64_t I, int64_t ld) {
  return ld >= I && (T == 0 || ld <= (INT64_MAX / 16 - I) / (T > 1 ? T - 1 : 1));
}

}  // namespace

}  // namespace gbln

using namespace gbln;

extern "C" gbln_status gbln_glu_fwd(const void* gate, const void* up, void* out, int64_t T,
                                    int64_t I, int64_t ld_gate, int64_t ld_up, int64_t ld_out,
                                    gbln_act act, gbln_dtype io, gbln_stream_t stream) {
  if (!dtype_ok(io) || !act_ok(act) || !sizes_ok(T, I)) return GBLN_ERR_INVALID_ARG;
  if (!ld_ok(T, I, ld_gate) || !ld_ok(T, I, ld_up) || !ld_ok(T, I, ld_out)) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!gate || !up || !out) return GBLN_ERR_INVALID_ARG;
  if (sm_count() <= 0) return GBLN_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
#define GBLN_GLU_FWD(TY, A) glu_fwd_launch<TY, A>(gate, up, out, T, I, ld_gate, ld_up, ld_out, s)
  if (io == GBLN_F32) {
    GBLN_DISPATCH_ACT(float, act, GBLN_GLU_FWD)
  } else {
    GBLN_DISPATCH_ACT(bf16, act, GBLN_GLU_FWD)
  }
#undef GBLN_GLU_FWD
  return launch_status();
}

extern "C" gbln_status gbln_glu_fwd_mxfp8(const void* gate, const void* up, uint8_t* out_e4m3,
                                          uint8_t* out_scale, int64_t T, int64_t I,
                                          int64_t ld_gate, int64_t ld_up, gbln_act act,
                                          gbln_dtype io, gbln_stream_t stream) {
  if (!dtype_ok(io) || !act_ok(act) || !sizes_ok(T, I) || I % kMxBlock != 0) return GBLN_ERR_INVALID_ARG;
  if (!ld_ok(T, I, ld_gate) || !ld_ok(T, I, ld_up)) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!gate || !up || !out_e4m3 || !out_scale) return GBLN_ERR_INVALID_ARG;
  if (sm_count() <= 0) return GBLN_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  const MxOut mx{out_e4m3, out_scale};
#define GBLN_GLU_FWD_MX(TY, A) glu_fwd_mx_launch<TY, A>(gate, up, mx, T, I, ld_gate, ld_up, s)
  if (io == GBLN_F32) {
    GBLN_DISPATCH_ACT(float, act, GBLN_GLU_FWD_MX)
  } else {
    GBLN_DISPATCH_ACT(bf16, act, GBLN_GLU_FWD_MX)
  }
#undef GBLN_GLU_FWD_MX
  return launch_status();
}

extern "C" gbln_status gbln_glu_bwd(const void* dout, const void* gate, const void* up,
                                    void* dgate, void* dup, int64_t T, int64_t I,
                                    int64_t ld_dout, int64_t ld_gate, int64_t ld_up,
                                    int64_t ld_dgate, int64_t ld_dup, gbln_act act,
                                    gbln_dtype io, gbln_stream_t stream) {
  if (!dtype_ok(io) || !act_ok(act) || !sizes_ok(T, I)) return GBLN_ERR_INVALID_ARG;
  if (!ld_ok(T, I, ld_dout) || !ld_ok(T, I, ld_gate) || !ld_ok(T, I, ld_up) ||
      !ld_ok(T, I, ld_dgate) || !ld_ok(T, I, ld_dup))
    return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!dout || !gate || !up || !dgate || !dup) return GBLN_ERR_INVALID_ARG;
  if (sm_count() <= 0) return GBLN_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
#define GBLN_GLU_BWD(TY, A) \
  glu_bwd_launch<TY, A>(dout, gate, up, dgate, dup, T, I, ld_dout, ld_gate, ld_up, ld_dgate, ld_dup, s)
  if (io == GBLN_F32) {
    GBLN_DISPATCH_ACT(float, act, GBLN_GLU_BWD)
  } else {
    GBLN_DISPATCH_ACT(bf16, act, GBLN_GLU_BWD)
  }
#undef GBLN_GLU_BWD
  return launch_status();
}

extern "C" gbln_status gbln_swiglu_fwd(const void* gate, const void* up, void* out, int64_t T,
                                       int64_t I, gbln_dtype io, gbln_stream_t stream) {
  return gbln_glu_fwd(gate, up, out, T, I, I, I, I, GBLN_ACT_SILU, io, stream);
}

extern "C" gbln_status gbln_swiglu_bwd(const void* dout, const void* gate, const void* up,
                                       void* dgate, void* dup, int64_t T, int64_t I,
                                       gbln_dtype io, gbln_stream_t stream) {
  return gbln_glu_bwd(dout, gate, up, dgate, dup, T, I, I, I, I, I, I, GBLN_ACT_SILU, io, stream);
}

extern "C" gbln_status gbln_act_fwd(const void* x, void* y, int64_t n, gbln_act act,
                                    gbln_dtype io, gbln_stream_t stream) {
  if (!dtype_ok(io) || !act_ok(act) || !sizes_ok(n, 1)) return GBLN_ERR_INVALID_ARG;
  if (n == 0) return GBLN_OK;
  if (!x || !y) return GBLN_ERR_INVALID_ARG;
  if (sm_count() <= 0) return GBLN_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
#define GBLN_ACT_FWD(TY, A) act_fwd_launch<TY, A>(x, y, n, s)
  if (io == GBLN_F32) {
    GBLN_DISPATCH_ACT(float, act, GBLN_ACT_FWD)
  } else {
    GBLN_DISPATCH_ACT(bf16, act, GBLN_ACT_FWD)
  }
#undef GBLN_ACT_FWD
  return launch_status();
}

extern "C" gbln_status gbln_act_bwd(const void* dy, const void* x, void* dx, int64_t n,
                                    gbln_act act, gbln_dtype io, gbln_stream_t stream) {
  if (!dtype_ok(io) || !act_ok(act) || !sizes_ok(n, 1)) return GBLN_ERR_INVALID_ARG;
  if (n == 0) return GBLN_OK;
  if (!dy || !x || !dx) return GBLN_ERR_INVALID_ARG;
  if (sm_count() <= 0) return GBLN_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
#define GBLN_ACT_BWD(TY, A) act_bwd_launch<TY, A>(dy, x, dx, n, s)
  if (io == GBLN_F32) {
    GBLN_DISPATCH_ACT(float, act, GBLN_ACT_BWD)
  } else {
    GBLN_DISPATCH_ACT(bf16, act, GBLN_ACT_BWD)
  }
#undef GBLN_ACT_BWD
  return launch_status();
}

extern "C" gbln_status gbln_glu_fwd_fp8(const void* gate, const void* up, uint8_t* out_e4m3,
                                        float* out_scale, int64_t T, int64_t I, int64_t ld_gate,
                                        int64_t ld_up, gbln_act act, gbln_dtype io,
                                        gbln_stream_t stream) {
  if (!dtype_ok(io) || !act_ok(act) || !sizes_ok(T, I) || T > (1LL << 31) - 1) return GBLN_ERR_INVALID_ARG;
  if (!ld_ok(T, I, ld_gate) || !ld_ok(T, I, ld_up)) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!gate || !up || !out_e4m3 || !out_scale) return GBLN_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
#define GBLN_GLU_FWD_FP8(TY, A) \
  return glu_fwd_row8_launch<TY, A>(gate, up, out_e4m3, out_scale, T, I, ld_gate, ld_up, s)
  if (io == GBLN_F32) {
    GBLN_DISPATCH_ACT(float, act, GBLN_GLU_FWD_FP8)
  } else {
    GBLN_DISPATCH_ACT(bf16, act, GBLN_GLU_FWD_FP8)
  }
#undef GBLN_GLU_FWD_FP8
}

extern "C" gbln_status gbln_glu_fwd_ckpt8(const void* gate, const void* up, void* out, uint8_t* gate8,
                                          float* gate_scale, uint8_t* up8, float* up_scale, int64_t T,
                                          int64_t I, int64_t ld_gate, int64_t ld_up, int64_t ld_out,
                                          gbln_act act, gbln_q8 fmt, gbln_dtype io,
                                          gbln_stream_t stream) {
  if (!dtype_ok(io) || !act_ok(act) || !q8_ok(fmt) || !sizes_ok(T, I)) return GBLN_ERR_INVALID_ARG;
  if (!ld_ok(T, I, ld_gate) || !ld_ok(T, I, ld_up) || !ld_ok(T, I, ld_out)) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!gate || !up || !out || !gate8 || !gate_scale || !up8 || !up_scale) return GBLN_ERR_INVALID_ARG;
  if (sm_count() <= 0) return GBLN_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  const GluCkpt C{gate8, gate_scale, up8, up_scale};
#define GBLN_GLU_FWD_CKPT(TY, A)                                                              \
  fmt == GBLN_Q8_INT8                                                                         \
      ? glu_fwd_ckpt_launch<TY, A, GBLN_Q8_INT8>(gate, up, out, C, T, I, ld_gate, ld_up, ld_out, s) \
      : glu_fwd_ckpt_launch<TY, A, GBLN_Q8_E4M3>(gate, up, out, C, T, I, ld_gate, ld_up, ld_out, s)
  if (io == GBLN_F32) {
    GBLN_DISPATCH_ACT(float, act, GBLN_GLU_FWD_CKPT)
  } else {
    GBLN_DISPATCH_ACT(bf16, act, GBLN_GLU_FWD_CKPT)
  }
#undef GBLN_GLU_FWD_CKPT
  return launch_status();
}

extern "C" gbln_status gbln_glu_bwd_ckpt8(const void* dout, const uint8_t* gate8, const float* gate_scale,
                                          const uint8_t* up8, const float* up_scale, void* dgate,
                                          void* dup, int64_t T, int64_t I, int64_t ld_dout,
                                          int64_t ld_dgate, int64_t ld_dup, gbln_act act, gbln_q8 fmt,
                                          gbln_dtype io, gbln_stream_t stream) {
  if (!dtype_ok(io) || !act_ok(act) || !q8_ok(fmt) || !sizes_ok(T, I)) return GBLN_ERR_INVALID_ARG;
  if (!ld_ok(T, I, ld_dout) || !ld_ok(T, I, ld_dgate) || !ld_ok(T, I, ld_dup)) return GBLN_ERR_INVALID_ARG;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!dout || !gate8 || !gate_scale || !up8 || !up_scale || !dgate || !dup) return GBLN_ERR_INVALID_ARG;
  if (sm_count() <= 0) return GBLN_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  const GluCkptIn C{gate8, gate_scale, up8, up_scale};
#define GBLN_GLU_BWD_CKPT(TY, A)                                                                   \
  fmt == GBLN_Q8_INT8                                                                              \
      ? glu_bwd_ckpt_launch<TY, A, GBLN_Q8_INT8>(dout, C, dgate, dup, T, I, ld_dout, ld_dgate, ld_dup, s) \
      : glu_bwd_ckpt_launch<TY, A, GBLN_Q8_E4M3>(dout, C, dgate, dup, T, I, ld_dout, ld_dgate, ld_dup, s)
  if (io == GBLN_F32) {
    GBLN_DISPATCH_ACT(float, act, GBLN_GLU_BWD_CKPT)
  } else {
    GBLN_DISPATCH_ACT(bf16, act, GBLN_GLU_BWD_CKPT)
  }
#undef GBLN_GLU_BWD_CKPT
  return launch_status();
}
