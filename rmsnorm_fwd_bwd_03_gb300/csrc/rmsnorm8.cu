// RMSNorm with 8-bit results: the forward (fused residual add) whose output is
// E4M3 with one float32 scale per row, the forward that also saves its input as
// an 8-bit checkpoint (INT8 or E4M3, one float32 scale per 128 values of a row),
// and the backward that reads the checkpoint.
//
// Operator: "Fast-LLM: 高效大语言模型训练框架", §三 技术架构, "Transformer Block 结构"
// (normalization RMSNorm); fused form as in "LLaMA-Factory Kernels 系统" (fused
// RMSNorm) and "Kernels（自定义内核）" §Liger (fusion saves memory and traffic).
//
// HBM-bound, as the plain operator: every row is read once, held in registers
// across its reduction, and written once.
//
// Row scale: with u = w h, the output is y = u rstd and its largest magnitude is
// rstd max|u|.  rstd cancels out of the codes, RNE(u * 448 / max|u|), so the sum
// of squares and the maximum come out of ONE reduction over the row, and the
// scale is max|u| rstd / 448.
//
// Checkpoint: 128 values are 16 lanes of 16-byte bf16 vectors (32 of float32);
// their maximum takes 4 shuffles (one redux), and the codes are written from the
// registers that hold h.  The backward reads 1.03 bytes per value instead of 2
// or 4.

#include "q8.cuh"

namespace gbln {

namespace {

// What a forward writes in 8 bits.
enum Mode { kRowE4m3 = 0, kCkptInt8 = 1, kCkptE4m3 = 2 };
constexpr int mode_fmt(int m) { return m == kCkptInt8 ? GBLN_Q8_INT8 : GBLN_Q8_E4M3; }

template <typename T, typename W>
struct Fwd8 {
  const T* x;
  const T* r;
  const W* w;
  T* y;  // may be null with kRowE4m3
  T* hout;
  float* rstd;
  uint8_t* q;
  float* sc;
  int64_t rows;
  int H;
  int ng;  // scales per row
  float inv_H, eps;
};

template <typename T, typename W>
struct Bwd8 {
  const T* dy;
  const T* dres;
  const uint8_t* hq;
  const float* hs;
  const W* w;
  const float* rstd;
  T* dx;
  float* partial;
  int64_t rows;
  int H;
  int ng;
  float inv_H;
};

// Sum and maximum over the TPR threads of a row in one barrier pair (TPR > 32:
// one row per block).
template <int TPR>
__device__ __forceinline__ void row_sum_max(float& s, uint32_t& m, float* red, uint32_t* redm) {
  s = group_sum<32>(s);
  m = group_max<32>(m);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
      red[warp] = s;
      redm[warp] = m;
    }
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) {
      s += red[i];
      m = max(m, redm[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// Forward, vector path: TPR threads per row, VPT 16-byte vectors per thread,
// BLOCK / TPR rows per block; no loop over rows, so the block scheduler keeps the
// loads of other rows in flight while one is reduced.  h stays packed: it is
// exact in T.  HBM-bound: 65536 x 4096 bf16 with a residual, row-scaled output 271
// us and checkpoint 348 us (277 and 357 us at the copy rate); 16384 rows of 1024
// 21.7 and 26.5 us (17.3 and 22.3), of which about 2 us are the launch.
// ---------------------------------------------------------------------------
template <typename T, typename W, int TPR, int VPT, int BLOCK, bool RES, int MODE>
__global__ void __launch_bounds__(BLOCK) rms8_fwd_vec(const Fwd8<T, W> A) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int FMT = mode_fmt(MODE);
  constexpr int LPG = kCkptGroup / VEC;  // lanes per checkpoint group
  __shared__ float red[TPR / 32];
  __shared__ uint32_t redm[TPR / 32];
  const int g = threadIdx.x / TPR, l = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (BLOCK / TPR) + g;
  if (row >= A.rows) return;  // uniform per row group; one row per block when TPR > 32
  const int nvec = A.H / VEC;
  const size_t base = (size_t)row * A.H;

  uint4 xa[VPT], ra[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int iv = l + v * TPR;
    if (iv < nvec) {
      xa[v] = ld_stream(A.x + base + (size_t)iv * VEC);
      if constexpr (RES) ra[v] = ld_stream(A.r + base + (size_t)iv * VEC);
    }
  }
  float ss = 0.f;
  uint32_t am = 0;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int iv = l + v * TPR;
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = 0.f;
    if (iv < nvec) {
      unpack<VEC>(xa[v], h);
      if constexpr (RES) {
        float b[VEC];
        unpack<VEC>(ra[v], b);
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] += b[e];
        xa[v] = pack<T, VEC>(h);  // the stored h is what gets normalised and saved
        unpack<VEC>(xa[v], h);
        st_vec(A.hout + base + (size_t)iv * VEC, xa[v]);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(h[e], h[e], ss);
    }
    if constexpr (MODE == kRowE4m3) {
      if (iv < nvec) {
        float wv[VEC];
        load_weight<W, VEC>(A.w, iv, wv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) am = max(am, abs_bits(__fmul_rn(wv[e], h[e])));
      }
    } else {
      // All lanes of a warp take part; those past the row's end hold zeros.
      const uint32_t gm = group_max<LPG>(abs_max_bits<VEC>(h));
      if (iv < nvec) {
        const float a = q8_amax(gm);
        q8_store<FMT, VEC>(h, q8_inv<FMT>(a), A.q + base + (size_t)iv * VEC);
        if (iv % LPG == 0) A.sc[(size_t)row * A.ng + iv / LPG] = q8_scale<FMT>(a, gm);
      }
    }
  }
  if constexpr (MODE == kRowE4m3) {
    row_sum_max<TPR>(ss, am, red, redm);
  } else {
    ss = row_sum<TPR>(ss, red);
  }
  const float rs = rsqrtf(ss * A.inv_H + A.eps);
  if (l == 0) A.rstd[row] = rs;
  float inv = 0.f;
  if constexpr (MODE == kRowE4m3) {
    const float a = q8_amax(am);
    inv = q8_inv<FMT>(a);
    if (l == 0) A.sc[row] = q8_scale<FMT>(__fmul_rn(a, rs), am);
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int iv = l + v * TPR;
    if (iv < nvec) {
      float h[VEC], wv[VEC], o[VEC];
      unpack<VEC>(xa[v], h);
      load_weight<W, VEC>(A.w, iv, wv);
      if (MODE != kRowE4m3 || A.y) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = wv[e] * (h[e] * rs);
        st_vec(A.y + base + (size_t)iv * VEC, pack<T, VEC>(o));
      }
      if constexpr (MODE == kRowE4m3) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = __fmul_rn(wv[e], h[e]);
        q8_store<FMT, VEC>(o, inv, A.q + base + (size_t)iv * VEC);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Forward, element path (any alignment, rows of up to 16384 values).  A warp
// takes chunks of 128 consecutive values, lane l the values l, l + 32, l + 64,
// l + 96: every access of a warp is contiguous, and a chunk is a checkpoint
// group.  NW warps per row take `per` consecutive chunks each, at most kElemChunks,
// which stay in registers.  Offsets from a warp's first value are immediates and
// only a row's last chunk is predicated: at one value per lane and access a warp
// issues 40 instructions per 32 values and has few bytes in flight.  Nothing is full
// (issue slots 60 to 63%, load/store pipe 50%, half of an SM's warps): the warps wait
// for their loads.  65536 x 1021 bf16: row scale 113 us, checkpoint 119 us (69 and 89 us
// at the copy rate).
// ---------------------------------------------------------------------------
constexpr int kElemChunks = 4;

// Values l, l + 32, l + 64, l + 96 of a chunk; rem = values from the lane's first
// one to the row's end (FULL: the chunk is whole).
template <bool FULL, typename T>
__device__ __forceinline__ void load_chunk(const T* p, int rem, T (&v)[4]) {
#pragma unroll
  for (int m = 0; m < 4; ++m) v[m] = FULL || 32 * m < rem ? p[32 * m] : from_f32<T>(0.f);
}
template <bool FULL>
__device__ __forceinline__ void load_chunk(const uint8_t* p, int rem, uint8_t (&v)[4]) {
#pragma unroll
  for (int m = 0; m < 4; ++m) v[m] = FULL || 32 * m < rem ? p[32 * m] : (uint8_t)0;
}
template <bool FULL, typename T>
__device__ __forceinline__ void store_chunk(T* p, int rem, const float2 (&v)[2]) {
  const float f[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
#pragma unroll
  for (int m = 0; m < 4; ++m)
    if (FULL || 32 * m < rem) p[32 * m] = from_f32<T>(f[m]);
}
template <bool FULL, int FMT>
__device__ __forceinline__ void store_codes(uint8_t* p, int rem, const float2 (&v)[2], float inv) {
  const uint32_t q = q8_code4<FMT>(v[0].x, v[0].y, v[1].x, v[1].y, inv);
#pragma unroll
  for (int m = 0; m < 4; ++m)
    if (FULL || 32 * m < rem) p[32 * m] = (uint8_t)(q >> (8 * m));
}
// Round to T and back.
template <typename T>
__device__ __forceinline__ float2 round2(float2 v) {
  if constexpr (sizeof(T) == 4) return v;
  const uint32_t w = pack_bf16x2(v.x, v.y);
  return make_float2(bf16_lo(w), bf16_hi(w));
}
// Run f(true_type) for a whole chunk, f(false_type) for a row's last, shorter one.
struct FullChunk { static constexpr bool v = true; };
struct PartChunk { static constexpr bool v = false; };
template <typename F>
__device__ __forceinline__ void chunk_of(int c0, int H, F&& f) {
  if (c0 + kCkptGroup <= H) f(FullChunk{});
  else if (c0 < H) f(PartChunk{});
}

template <typename T, typename W, bool RES, int MODE>
__global__ void __launch_bounds__(1024) rms8_fwd_elem(const Fwd8<T, W> A, int NW, int per) {
  constexpr int FMT = mode_fmt(MODE);
  __shared__ float red[32];
  __shared__ uint32_t redm[32];
  const int lane = threadIdx.x & 31, warp = warp_index();
  const int g = warp / NW, wi = warp - g * NW;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / (32 * NW)) + g;
  const bool live = row < A.rows;  // the barrier below is reached by every warp
  const int H = live ? A.H : 0;
  const size_t at = (size_t)(live ? row : 0) * A.H + wi * per * kCkptGroup + lane;
  const int c0 = wi * per * kCkptGroup;  // the warp's first chunk
  const int end = min(c0 + per * kCkptGroup, H);

  T xr[kElemChunks][4], rr[kElemChunks][4];
#pragma unroll
  for (int k = 0; k < kElemChunks; ++k)
    chunk_of(c0 + k * kCkptGroup, end, [&](auto full) {
      const int rem = end - (c0 + k * kCkptGroup) - lane;
      load_chunk<decltype(full)::v>(A.x + at + k * kCkptGroup, rem, xr[k]);
      if constexpr (RES) load_chunk<decltype(full)::v>(A.r + at + k * kCkptGroup, rem, rr[k]);
    });
  float2 h[kElemChunks][2];  // values l and l + 32, l + 64 and l + 96
  float2 sq = both(0.f);
  uint32_t am = 0, cm[kElemChunks];
#pragma unroll
  for (int k = 0; k < kElemChunks; ++k) {
    cm[k] = 0;
    chunk_of(c0 + k * kCkptGroup, end, [&](auto full) {
      [[maybe_unused]] constexpr bool FULL = decltype(full)::v;
      [[maybe_unused]] const int rem = end - (c0 + k * kCkptGroup) - lane;
      h[k][0] = make_float2(to_f32(xr[k][0]), to_f32(xr[k][1]));
      h[k][1] = make_float2(to_f32(xr[k][2]), to_f32(xr[k][3]));
      if constexpr (RES) {
        h[k][0] = round2<T>(add2(h[k][0], make_float2(to_f32(rr[k][0]), to_f32(rr[k][1]))));
        h[k][1] = round2<T>(add2(h[k][1], make_float2(to_f32(rr[k][2]), to_f32(rr[k][3]))));
        store_chunk<FULL>(A.hout + at + k * kCkptGroup, rem, h[k]);
      }
      sq = fma2(h[k][0], h[k][0], fma2(h[k][1], h[k][1], sq));
      if constexpr (MODE == kRowE4m3) {
        W w[4];
        load_chunk<FULL>(A.w + c0 + k * kCkptGroup + lane, rem, w);
        const float2 u = mul2(make_float2(to_f32(w[0]), to_f32(w[1])), h[k][0]);
        const float2 v = mul2(make_float2(to_f32(w[2]), to_f32(w[3])), h[k][1]);
        am = max(am, __float_as_uint(max3_abs(max3_abs(u.x, u.y, v.x), v.y, v.y)));
      } else {
        cm[k] = group_max<32>(__float_as_uint(
            max3_abs(max3_abs(h[k][0].x, h[k][0].y, h[k][1].x), h[k][1].y, h[k][1].y)));
      }
    });
  }
  if constexpr (MODE != kRowE4m3) {
    // Lanes 2 k and 2 k + 1 divide for chunk k's 1 / scale and scale: one division
    // per lane instead of two per chunk.
    static_assert(kElemChunks == 4, "two lane bits name a chunk");
    const uint32_t mine = lane & 4 ? (lane & 2 ? cm[3] : cm[2]) : (lane & 2 ? cm[1] : cm[0]);
    const float a = q8_amax(mine);
    const float d = __fdiv_rn(lane & 1 ? a : Q8Max<FMT>::v, lane & 1 ? Q8Max<FMT>::v : a);
    if (lane < 8 && (lane & 1) && c0 + (lane >> 1) * kCkptGroup < end)
      A.sc[(size_t)row * A.ng + wi * per + (lane >> 1)] = mine < kInfBits ? d : __int_as_float(0x7fc00000);
#pragma unroll
    for (int k = 0; k < kElemChunks; ++k) {
      const float inv = __shfl_sync(0xffffffffu, d, 2 * k);
      chunk_of(c0 + k * kCkptGroup, end, [&](auto full) {
        store_codes<decltype(full)::v, FMT>(A.q + at + k * kCkptGroup, end - (c0 + k * kCkptGroup) - lane, h[k], inv);
      });
    }
  }
  float ss = group_sum<32>(sq.x + sq.y);
  if constexpr (MODE == kRowE4m3) am = group_max<32>(am);
  if (NW > 1) {
    if (lane == 0) {
      red[warp] = ss;
      redm[warp] = am;
    }
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < NW; ++i) {
      ss += red[g * NW + i];
      am = max(am, redm[g * NW + i]);
    }
  }
  const float rs = rsqrtf(ss * A.inv_H + A.eps);
  if (live && wi == 0 && lane == 0) A.rstd[row] = rs;
  float inv = 0.f;
  if constexpr (MODE == kRowE4m3) {
    const float a = q8_amax(am);
    inv = q8_inv<FMT>(a);
    if (live && wi == 0 && lane == 0) A.sc[row] = q8_scale<FMT>(__fmul_rn(a, rs), am);
  }
#pragma unroll
  for (int k = 0; k < kElemChunks; ++k)
    chunk_of(c0 + k * kCkptGroup, end, [&](auto full) {
      constexpr bool FULL = decltype(full)::v;
      const int rem = end - (c0 + k * kCkptGroup) - lane;
      W w[4];
      load_chunk<FULL>(A.w + c0 + k * kCkptGroup + lane, rem, w);
      const float2 w0 = make_float2(to_f32(w[0]), to_f32(w[1])), w1 = make_float2(to_f32(w[2]), to_f32(w[3]));
      if (MODE != kRowE4m3 || A.y) {
        const float2 o[2] = {mul2(w0, mul2(h[k][0], both(rs))), mul2(w1, mul2(h[k][1], both(rs)))};
        store_chunk<FULL>(A.y + at + k * kCkptGroup, rem, o);
      }
      if constexpr (MODE == kRowE4m3) {
        const float2 o[2] = {mul2(w0, h[k][0]), mul2(w1, h[k][1])};
        store_codes<FULL, FMT>(A.q + at + k * kCkptGroup, rem, o, inv);
      }
    });
}

// Forward for rows too wide for the registers of either path: one block per row,
// which it reads a second time for the output (its own stores, where there is a
// residual).  Chunks as above; compensated sums, since a thread may add up tens
// of thousands of terms.
constexpr int kWideBlock = 512;

template <typename T, typename W, bool RES, int MODE>
__global__ void __launch_bounds__(kWideBlock) rms8_fwd_wide(const Fwd8<T, W> A) {
  constexpr int FMT = mode_fmt(MODE), NW = kWideBlock / 32;
  __shared__ float red[NW];
  __shared__ uint32_t redm[NW];
  const int lane = threadIdx.x & 31, warp = warp_index();
  const int64_t row = blockIdx.x;
  const size_t base = (size_t)row * A.H;
  KahanSum ks;
  uint32_t am = 0;
  for (int c0 = warp * kCkptGroup; c0 < A.H; c0 += NW * kCkptGroup) {
    float h[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int j = c0 + 32 * m + lane;
      h[m] = 0.f;
      if (j < A.H) {
        h[m] = to_f32(A.x[base + j]);
        if constexpr (RES) {
          const T hv = from_f32<T>(h[m] + to_f32(A.r[base + j]));
          A.hout[base + j] = hv;
          h[m] = to_f32(hv);
        }
        ks.add(h[m] * h[m]);
        if constexpr (MODE == kRowE4m3) am = max(am, abs_bits(__fmul_rn(to_f32(A.w[j]), h[m])));
      }
    }
    if constexpr (MODE != kRowE4m3) {
      const uint32_t gm = group_max<32>(abs_max_bits<4>(h));
      const float a = q8_amax(gm);
      const float2 hp[2] = {make_float2(h[0], h[1]), make_float2(h[2], h[3])};
      store_codes<false, FMT>(A.q + base + c0 + lane, A.H - c0 - lane, hp, q8_inv<FMT>(a));
      if (lane == 0) A.sc[(size_t)row * A.ng + c0 / kCkptGroup] = q8_scale<FMT>(a, gm);
    }
  }
  float ss = ks.s;
  row_sum_max<kWideBlock>(ss, am, red, redm);
  const float rs = rsqrtf(ss * A.inv_H + A.eps);
  if (threadIdx.x == 0) A.rstd[row] = rs;
  float inv = 0.f;
  if constexpr (MODE == kRowE4m3) {
    const float a = q8_amax(am);
    inv = q8_inv<FMT>(a);
    if (threadIdx.x == 0) A.sc[row] = q8_scale<FMT>(__fmul_rn(a, rs), am);
  }
  for (int c0 = warp * kCkptGroup; c0 < A.H; c0 += NW * kCkptGroup) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int j = c0 + 32 * m + lane;
      if (j < A.H) {
        const float h = RES ? to_f32(A.hout[base + j]) : to_f32(A.x[base + j]);  // own write
        const float wv = to_f32(A.w[j]);
        if (MODE != kRowE4m3 || A.y) A.y[base + j] = from_f32<T>(wv * (h * rs));
        if constexpr (MODE == kRowE4m3) A.q[base + j] = (uint8_t)q8_code1<FMT>(__fmul_rn(wv, h), inv);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward, vector path.  gridDim.x = P blocks; block p owns the contiguous rows
// [p*rows/P, (p+1)*rows/P), its GPB groups of TPR threads take every GPB-th of
// them.  dW is accumulated per thread in float32 registers, then the groups'
// sums are added in order: no atomics, one partial row per block.  Only packed
// inputs stay in registers across the row's reduction.  65536 x 4096 bf16 284 us
// (278 us at the copy rate); 65536 x 768 63 us (52), 16384 x 1024 24 us (17): with
// few vectors per thread the wait for a row's sum shows.  Three blocks of 256
// threads per SM at up to 85 registers measured faster than four at 64 (27 us at
// 16384 x 1024), and more blocks than are resident only add partial rows.
// ---------------------------------------------------------------------------
template <typename T, typename W, int TPR, int VPT, int GPB, bool DRES, int FMT>
__global__ void __launch_bounds__(TPR * GPB, GPB > 1 ? 3 : 512 / TPR) rms8_bwd_vec(const Bwd8<T, W> A, bool prefetch) {
  constexpr int VEC = VecOf<T>::N;
  constexpr int LPG = kCkptGroup / VEC;
  constexpr int NWG = TPR / 32;
  __shared__ float red[GPB][2][NWG];
  const int g = threadIdx.x / TPR, l = threadIdx.x % TPR, lane = threadIdx.x & 31;
  const int nvec = A.H / VEC;
  const int64_t P = gridDim.x, p = blockIdx.x;
  const int64_t r0 = p * A.rows / P, r1 = (p + 1) * A.rows / P;

  float2 acc[VPT][VEC / 2];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) acc[v][e] = both(0.f);

  int par = 0;
  for (int64_t row = r0 + g; row < r1; row += GPB) {
    const size_t base = (size_t)row * A.H;
    // The group's next row is asked for in L2 while this one is processed: by one
    // bulk prefetch per tensor where a block has one row, else line by line.
    if constexpr (GPB > 1) {
      constexpr int LINE = 128 / sizeof(T), SEG = TPR / 4;  // at most SEG lines per tensor
      const int seg = l / SEG, i = l % SEG;
      if (row + GPB < r1) {
        const size_t nb = base + (size_t)GPB * A.H;
        if (seg == 0 && i * LINE < A.H) prefetch_line(A.dy + nb + i * LINE);
        if (DRES && seg == 1 && i * LINE < A.H) prefetch_line(A.dres + nb + i * LINE);
        if (seg == 2 && i * 128 < A.H) prefetch_line(A.hq + nb + i * 128);
      }
    } else {
      if (threadIdx.x == 0 && row + 1 < r1) {
        const size_t nb = base + A.H;
        const uint32_t rb = (uint32_t)(A.H * sizeof(T));
        prefetch_l2(A.dy + nb, rb);
        if constexpr (DRES) prefetch_l2(A.dres + nb, rb);
        if (prefetch) prefetch_l2(A.hq + nb, (uint32_t)A.H);
      }
    }
    uint4 dya[VPT], dra[VPT];
    Codes<FMT, VEC> ha[VPT];
    float hs[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int iv = l + v * TPR;
      if (iv < nvec) {
        dya[v] = ld_stream(A.dy + base + (size_t)iv * VEC);
        ha[v].load(A.hq + base + (size_t)iv * VEC);
        if constexpr (DRES) dra[v] = ld_stream(A.dres + base + (size_t)iv * VEC);
        hs[v] = __ldg(A.hs + (size_t)row * A.ng + iv / LPG);
      }
    }
    const float rs = __ldg(A.rstd + row);
    float2 dot2 = both(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int iv = l + v * TPR;
      if (iv < nvec) {
        float d[VEC], n[VEC], wv[VEC];
        unpack<VEC>(dya[v], d);
        ha[v].get(n, hs[v]);
        load_weight<W, VEC>(A.w, iv, wv);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 d2 = make_float2(d[e], d[e + 1]), n2 = mul2(make_float2(n[e], n[e + 1]), both(rs));
          dot2 = fma2(mul2(d2, make_float2(wv[e], wv[e + 1])), n2, dot2);
          acc[v][e / 2] = fma2(d2, n2, acc[v][e / 2]);
        }
      }
    }
    float dot = group_sum<32>(dot2.x + dot2.y);
    if constexpr (TPR > 32) {
      // red is double-buffered: a buffer is written again only after the group's
      // next barrier, which every thread reaches after reading it.
      if (lane == 0) red[g][par][l / 32] = dot;
      bar_sync_named(1 + g, TPR);
      dot = red[g][par][0];
#pragma unroll
      for (int k = 1; k < NWG; ++k) dot += red[g][par][k];
      par ^= 1;
    }
    const float2 mc = both(-dot * A.inv_H);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int iv = l + v * TPR;
      if (iv < nvec) {
        float d[VEC], n[VEC], wv[VEC], o[VEC];
        unpack<VEC>(dya[v], d);
        ha[v].get(n, hs[v]);
        load_weight<W, VEC>(A.w, iv, wv);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 g2 = mul2(make_float2(d[e], d[e + 1]), make_float2(wv[e], wv[e + 1]));
          const float2 o2 = mul2(both(rs), fma2(mul2(make_float2(n[e], n[e + 1]), both(rs)), mc, g2));
          o[e] = o2.x;
          o[e + 1] = o2.y;
        }
        if constexpr (DRES) {
          float d2[VEC];
          unpack<VEC>(dra[v], d2);
#pragma unroll
          for (int e = 0; e < VEC; ++e) o[e] += d2[e];
        }
        st_vec(A.dx + base + (size_t)iv * VEC, pack<T, VEC>(o));
      }
    }
  }

  float* prow = A.partial + (size_t)p * A.H;
  if constexpr (GPB == 1) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int iv = l + v * TPR;
      if (iv < nvec) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
          *reinterpret_cast<float4*>(prow + (size_t)iv * VEC + e) =
              make_float4(acc[v][e / 2].x, acc[v][e / 2].y, acc[v][e / 2 + 1].x, acc[v][e / 2 + 1].y);
      }
    }
  } else {
    __shared__ __align__(16) float sacc[GPB][TPR * VPT * VEC];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int iv = l + v * TPR;
      if (iv < nvec) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) *reinterpret_cast<float2*>(&sacc[g][iv * VEC + e]) = acc[v][e / 2];
      }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < A.H; j += TPR * GPB) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < GPB; ++q) s += sacc[q][j];
      prow[j] = s;
    }
  }
}

// ---------------------------------------------------------------------------
// Backward, element path: chunks of 128 values per warp as in rms8_fwd_elem, two
// per warp: with their weights, dW sums and inputs they fill 64 registers, and
// 1024 threads per SM are resident.  The warp asks for its next row in L2 while
// it works on this one.  As there, the warps wait for their loads: 65536 x 1021 bf16
// 118 us (69 us at the copy rate; 123 with every NW-th chunk, whose addresses are not
// immediates), 8194 x 4095 81 us (35).  A block of 18 warps is alone on its SM: 7708 x
// 4353 110 us (35), with 28% of an SM's warps and 37% of its issue slots in use.
// ---------------------------------------------------------------------------
constexpr int kElemBwdChunks = 2;

template <typename T, typename W, bool DRES, int FMT, int BLOCK>
__global__ void __launch_bounds__(BLOCK, 1024 / BLOCK) rms8_bwd_elem(const Bwd8<T, W> A, int NW, int per) {
  constexpr int C = kElemBwdChunks;
  constexpr int LINE = 128 / sizeof(T);
  extern __shared__ float sacc[];  // several row groups: one row of dW sums
  __shared__ float red[2][BLOCK / 32];
  const int lane = threadIdx.x & 31, warp = warp_index();
  const int GPB = (int)blockDim.x / (32 * NW);
  const int g = warp / NW, wi = warp - g * NW;
  const int H = A.H;
  const int64_t P = gridDim.x, p = blockIdx.x;
  const int64_t r0 = p * A.rows / P, r1 = (p + 1) * A.rows / P;
  const int c0 = wi * per * kCkptGroup, end = min(c0 + per * kCkptGroup, H);

  float2 acc[C][2], w[C][2];
#pragma unroll
  for (int k = 0; k < C; ++k) {
    acc[k][0] = acc[k][1] = w[k][0] = w[k][1] = both(0.f);
    chunk_of(c0 + k * kCkptGroup, end, [&](auto full) {
      W v[4];
      load_chunk<decltype(full)::v>(A.w + c0 + k * kCkptGroup + lane, end - (c0 + k * kCkptGroup) - lane, v);
      w[k][0] = make_float2(to_f32(v[0]), to_f32(v[1]));
      w[k][1] = make_float2(to_f32(v[2]), to_f32(v[3]));
    });
  }

  int par = 0;
  for (int64_t row = r0 + g; row < r1; row += GPB) {
    const size_t base = (size_t)row * H, at = base + c0 + lane;
    T dy[C][4], dr[C][4];
    float2 n[C][2];
    const float rs = __ldg(A.rstd + row);
#pragma unroll
    for (int k = 0; k < C; ++k)
      chunk_of(c0 + k * kCkptGroup, end, [&](auto full) {
        constexpr bool FULL = decltype(full)::v;
        const int rem = end - (c0 + k * kCkptGroup) - lane;
        load_chunk<FULL>(A.dy + at + k * kCkptGroup, rem, dy[k]);
        if constexpr (DRES) load_chunk<FULL>(A.dres + at + k * kCkptGroup, rem, dr[k]);
      });
#pragma unroll
    for (int k = 0; k < C; ++k)
      chunk_of(c0 + k * kCkptGroup, end, [&](auto full) {
        const int rem = end - (c0 + k * kCkptGroup) - lane;
        uint8_t b[4];
        load_chunk<decltype(full)::v>(A.hq + at + k * kCkptGroup, rem, b);
        const float sc = __ldg(A.hs + (size_t)row * A.ng + wi * per + k);
        float v[4];
        q8_decode4<FMT>(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410), v);
        n[k][0] = mul2(mul2(make_float2(v[0], v[1]), both(sc)), both(rs));
        n[k][1] = mul2(mul2(make_float2(v[2], v[3]), both(sc)), both(rs));
      });
    if (row + GPB < r1) {
      const size_t nb = base + (size_t)GPB * H;
      for (int j = wi * 32 * LINE + lane * LINE; j < H; j += NW * 32 * LINE) {
        prefetch_line(A.dy + nb + j);
        if constexpr (DRES) prefetch_line(A.dres + nb + j);
      }
      for (int j = (wi * 32 + lane) * 128; j < H; j += NW * 32 * 128) prefetch_line(A.hq + nb + j);
    }
    float2 dot2 = both(0.f);
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (c0 + k * kCkptGroup < end) {
        const float2 d0 = make_float2(to_f32(dy[k][0]), to_f32(dy[k][1]));
        const float2 d1 = make_float2(to_f32(dy[k][2]), to_f32(dy[k][3]));
        dot2 = fma2(mul2(d0, w[k][0]), n[k][0], fma2(mul2(d1, w[k][1]), n[k][1], dot2));
        acc[k][0] = fma2(d0, n[k][0], acc[k][0]);
        acc[k][1] = fma2(d1, n[k][1], acc[k][1]);
      }
    float dot = group_sum<32>(dot2.x + dot2.y);
    if (NW > 1) {  // double-buffered as in rms8_bwd_vec
      if (lane == 0) red[par][warp] = dot;
      bar_sync_named(1 + g, 32 * NW);
      dot = 0.f;
      for (int i = 0; i < NW; ++i) dot += red[par][g * NW + i];
      par ^= 1;
    }
    const float2 mc = both(-dot * A.inv_H);
#pragma unroll
    for (int k = 0; k < C; ++k)
      chunk_of(c0 + k * kCkptGroup, end, [&](auto full) {
        const int rem = end - (c0 + k * kCkptGroup) - lane;
        float2 o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 d = make_float2(to_f32(dy[k][2 * i]), to_f32(dy[k][2 * i + 1]));
          o[i] = mul2(both(rs), fma2(n[k][i], mc, mul2(d, w[k][i])));
          if constexpr (DRES) o[i] = add2(o[i], make_float2(to_f32(dr[k][2 * i]), to_f32(dr[k][2 * i + 1])));
        }
        store_chunk<decltype(full)::v>(A.dx + at + k * kCkptGroup, rem, o);
      });
  }

  float* prow = A.partial + (size_t)p * H + c0 + lane;
  float* srow = sacc + c0 + lane;
  for (int t = 0; t < GPB; ++t) {  // groups add in order
    if (t == g) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const float a[4] = {acc[k][0].x, acc[k][0].y, acc[k][1].x, acc[k][1].y};
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (c0 + k * kCkptGroup + 32 * m + lane < end) {
            const int j = k * kCkptGroup + 32 * m;
            const float v = t == 0 ? a[m] : srow[j] + a[m];
            if (t == GPB - 1) prow[j] = v;
            else srow[j] = v;
          }
      }
    }
    __syncthreads();
  }
}

// Backward for wider rows: one block per row at a time, read twice; dW sums are
// kept in the block's partial row.
template <typename T, typename W, bool DRES, int FMT>
__global__ void __launch_bounds__(kWideBlock) rms8_bwd_wide(const Bwd8<T, W> A) {
  __shared__ float red[kWideBlock / 32];
  const int H = A.H;
  const int64_t P = gridDim.x, p = blockIdx.x;
  const int64_t r0 = p * A.rows / P, r1 = (p + 1) * A.rows / P;
  float* prow = A.partial + (size_t)p * H;
  for (int j = threadIdx.x; j < H; j += kWideBlock) prow[j] = 0.f;
  for (int64_t row = r0; row < r1; ++row) {
    const size_t base = (size_t)row * H;
    const float rs = __ldg(A.rstd + row);
    const auto norm = [&](int j) {
      Codes<FMT, 1> q;
      float v[1];
      q.load(A.hq + base + j);
      q.get(v, __ldg(A.hs + (size_t)row * A.ng + j / kCkptGroup));
      return v[0] * rs;
    };
    KahanSum ks;
    for (int j = threadIdx.x; j < H; j += kWideBlock)
      ks.add(to_f32(A.dy[base + j]) * to_f32(A.w[j]) * norm(j));
    const float c = row_sum<kWideBlock>(ks.s, red) * A.inv_H;
    for (int j = threadIdx.x; j < H; j += kWideBlock) {
      const float d = to_f32(A.dy[base + j]), n = norm(j);
      float o = rs * (d * to_f32(A.w[j]) - n * c);
      if constexpr (DRES) o += to_f32(A.dres[base + j]);
      prow[j] = fmaf(d, n, prow[j]);
      A.dx[base + j] = from_f32<T>(o);
    }
  }
}

// ---------------------------------------------------------------------------
// Launch geometry.
// ---------------------------------------------------------------------------
constexpr int64_t kMaxH = 1 << 24;
constexpr int64_t kMaxRows = (1LL << 31) - 1;
constexpr int64_t kMaxVecPerRow = 2048;  // 512 threads x 4 vectors

// Element path: as few warps per row (up to 32) as hold it with at most `chunks`
// chunks each, and rows for about eight warps per block; wider rows do not fit the
// registers.
struct Elem {
  bool fits;
  int nw;      // warps per row
  int per;     // chunks per warp
  int block;   // threads
  int groups;  // rows per block and pass
};
Elem elem_geometry(int64_t H, int chunks) {
  const int64_t nchunk = (H + kCkptGroup - 1) / kCkptGroup;
  if (nchunk > 32 * chunks) return {false, kWideBlock / 32, 0, kWideBlock, 1};
  const int nw = (int)((nchunk + chunks - 1) / chunks);
  const int groups = nw < 8 ? 8 / nw : 1;
  return {true, nw, (int)((nchunk + nw - 1) / nw), 32 * nw * groups, groups};
}

bool vec_width(int64_t H, size_t io) {
  return (H * (int64_t)io) % 16 == 0 && H * (int64_t)io / 16 <= kMaxVecPerRow;
}

struct BwdGeometry {
  int tpr, vpt, gpb;  // tpr 0: element path
  int bps;            // blocks per SM
};
BwdGeometry bwd_geometry(int64_t H, size_t io) {
  if (!vec_width(H, io)) {
    const Elem e = elem_geometry(H, kElemBwdChunks);
    // At 64 registers each of an SM's four partitions holds eight warps, and a
    // block's warps go to them in turn: five warps fit four times, not six (counting
    // six took a quarter longer for 30476 rows of 1101 values, now 90 us).
    return {0, 0, e.groups, e.fits ? 8 / ((e.block + 127) / 128) : 2};
  }
  const int64_t nvec = H * (int64_t)io / 16;
  if (nvec <= 32) return {32, 1, 8, 3};
  if (nvec <= 64) return {32, 2, 8, 3};
  if (nvec <= 128) return {64, 2, 4, 3};
  int tpr = 64;
  while ((int64_t)tpr * 4 < nvec) tpr *= 2;
  return {tpr, 4, 1, 512 / tpr > 0 ? 512 / tpr : 1};
}

int64_t partials_for(int64_t T, const BwdGeometry& g, int sms) {
  if (T <= 0) return 0;
  int64_t P = (int64_t)sms * g.bps;
  const int64_t groups = (T + g.gpb - 1) / g.gpb;
  if (P > groups) P = groups;
  return P < 1 ? 1 : P;
}

template <typename T, typename W, bool RES, int MODE>
gbln_status fwd_launch(const Fwd8<T, W>& A, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const bool vec = vec_width(A.H, sizeof(T)) && aligned16(A.x) && aligned16(A.w) && aligned16(A.y) &&
                   (!RES || (aligned16(A.r) && aligned16(A.hout))) && aligned_to(A.q, VEC);
  if (!vec) {
    const Elem e = elem_geometry(A.H, kElemChunks);
    const int64_t blocks = (A.rows + e.groups - 1) / e.groups;
    if (e.fits) rms8_fwd_elem<T, W, RES, MODE><<<(unsigned)blocks, e.block, 0, s>>>(A, e.nw, e.per);
    else rms8_fwd_wide<T, W, RES, MODE><<<(unsigned)A.rows, kWideBlock, 0, s>>>(A);
    return launch_status();
  }
  const int nvec = A.H / VEC;
#define GBLN_FWD8(TPR, VPT, BLOCK) \
  rms8_fwd_vec<T, W, TPR, VPT, BLOCK, RES, MODE><<<(unsigned)((A.rows + BLOCK / TPR - 1) / (BLOCK / TPR)), BLOCK, 0, s>>>(A)
  if (nvec <= 32) GBLN_FWD8(32, 1, 256);
  else if (nvec <= 64) GBLN_FWD8(32, 2, 256);
  else if (nvec <= 128) GBLN_FWD8(32, 4, 256);
  else if (nvec <= 256) GBLN_FWD8(64, 4, 64);
  else if (nvec <= 512) GBLN_FWD8(128, 4, 128);
  else if (nvec <= 1024) GBLN_FWD8(256, 4, 256);
  else GBLN_FWD8(512, 4, 512);
#undef GBLN_FWD8
  return launch_status();
}

template <typename T, typename W, int MODE>
gbln_status fwd_typed(const void* x, const void* r, const void* w, void* y, void* ho, float* rstd,
                      uint8_t* q, float* sc, int64_t rows, int64_t H, float eps, cudaStream_t s) {
  const Fwd8<T, W> A{(const T*)x, (const T*)r, (const W*)w, (T*)y, (T*)ho, rstd, q, sc, rows, (int)H,
                     (int)((H + kCkptGroup - 1) / kCkptGroup), 1.0f / (float)H, eps};
  return r ? fwd_launch<T, W, true, MODE>(A, s) : fwd_launch<T, W, false, MODE>(A, s);
}

template <typename T, typename W, bool DRES, int FMT>
gbln_status bwd_launch(const Bwd8<T, W>& A, int64_t P, cudaStream_t s) {
  constexpr int VEC = VecOf<T>::N;
  const BwdGeometry g = bwd_geometry(A.H, sizeof(T));
  const bool vec = g.tpr && aligned16(A.dy) && aligned16(A.w) && aligned16(A.dx) && aligned16(A.partial) &&
                   (!DRES || aligned16(A.dres)) && aligned_to(A.hq, VEC);
  const unsigned grid = (unsigned)P;
  if (!vec) {
    const Elem e = elem_geometry(A.H, kElemBwdChunks);
    const size_t smem = e.groups > 1 ? (size_t)A.H * sizeof(float) : 0;  // at most 1024 values
    if (e.fits && e.block <= 256) rms8_bwd_elem<T, W, DRES, FMT, 256><<<grid, e.block, smem, s>>>(A, e.nw, e.per);
    else if (e.fits && e.block <= 512) rms8_bwd_elem<T, W, DRES, FMT, 512><<<grid, e.block, 0, s>>>(A, e.nw, e.per);
    else if (e.fits) rms8_bwd_elem<T, W, DRES, FMT, 1024><<<grid, e.block, 0, s>>>(A, e.nw, e.per);
    else rms8_bwd_wide<T, W, DRES, FMT><<<grid, kWideBlock, 0, s>>>(A);
    return launch_status();
  }
  const bool prefetch = aligned16(A.hq) && A.H % 16 == 0;
#define GBLN_BWD8(TPR, VPT, GPB) rms8_bwd_vec<T, W, TPR, VPT, GPB, DRES, FMT><<<grid, TPR * GPB, 0, s>>>(A, prefetch)
  if (g.tpr == 32 && g.vpt == 1) GBLN_BWD8(32, 1, 8);
  else if (g.tpr == 32) GBLN_BWD8(32, 2, 8);
  else if (g.vpt == 2) GBLN_BWD8(64, 2, 4);
  else if (g.tpr == 64) GBLN_BWD8(64, 4, 1);
  else if (g.tpr == 128) GBLN_BWD8(128, 4, 1);
  else if (g.tpr == 256) GBLN_BWD8(256, 4, 1);
  else GBLN_BWD8(512, 4, 1);
#undef GBLN_BWD8
  return launch_status();
}

template <typename T, typename W>
gbln_status bwd_typed(const void* dy, const void* dr, const uint8_t* hq, const float* hs, const void* w,
                      const float* rstd, void* dx, float* partial, int64_t P, int64_t rows, int64_t H,
                      int fmt, cudaStream_t s) {
  const Bwd8<T, W> A{(const T*)dy, (const T*)dr, hq, hs, (const W*)w, rstd, (T*)dx, partial, rows, (int)H,
                     (int)((H + kCkptGroup - 1) / kCkptGroup), 1.0f / (float)H};
  if (fmt == GBLN_Q8_INT8)
    return dr ? bwd_launch<T, W, true, GBLN_Q8_INT8>(A, P, s) : bwd_launch<T, W, false, GBLN_Q8_INT8>(A, P, s);
  return dr ? bwd_launch<T, W, true, GBLN_Q8_E4M3>(A, P, s) : bwd_launch<T, W, false, GBLN_Q8_E4M3>(A, P, s);
}

gbln_status sizes_and_types(int64_t T, int64_t H, int io, int wt) {
  if (!dtype_ok(io) || !dtype_ok(wt)) return GBLN_ERR_INVALID_ARG;
  if (T < 0 || T > kMaxRows || H <= 0 || H > kMaxH) return GBLN_ERR_INVALID_ARG;
  const bool pair = (io == GBLN_F32 && wt == GBLN_F32) || io == GBLN_BF16;
  return pair ? GBLN_OK : GBLN_ERR_UNSUPPORTED;
}

template <int MODE>
gbln_status fwd_entry(const void* x, const void* residual, const void* w, void* y, uint8_t* q, float* sc,
                      void* residual_out, float* rstd, int64_t T, int64_t H, float eps, gbln_dtype io,
                      gbln_dtype wt, gbln_stream_t stream) {
  if (!(eps >= 0.0f && eps <= 3.4028235e38f)) return GBLN_ERR_INVALID_ARG;  // also rejects NaN
  const gbln_status st = sizes_and_types(T, H, io, wt);
  if (st != GBLN_OK) return st;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!x || !w || !q || !sc || !rstd || (MODE != kRowE4m3 && !y)) return GBLN_ERR_INVALID_ARG;
  if (residual && !residual_out) return GBLN_ERR_INVALID_ARG;
  void* ho = residual ? residual_out : nullptr;
  cudaStream_t s = (cudaStream_t)stream;
  if (io == GBLN_F32) return fwd_typed<float, float, MODE>(x, residual, w, y, ho, rstd, q, sc, T, H, eps, s);
  if (wt == GBLN_BF16) return fwd_typed<bf16, bf16, MODE>(x, residual, w, y, ho, rstd, q, sc, T, H, eps, s);
  return fwd_typed<bf16, float, MODE>(x, residual, w, y, ho, rstd, q, sc, T, H, eps, s);
}

}  // namespace

}  // namespace gbln

using namespace gbln;

extern "C" gbln_status gbln_rmsnorm_fwd_fp8(const void* x, const void* residual, const void* weight,
                                            void* y, uint8_t* y_e4m3, float* y_scale,
                                            void* residual_out, float* rstd, int64_t T, int64_t H,
                                            float eps, gbln_dtype io, gbln_dtype wt,
                                            gbln_stream_t stream) {
  return fwd_entry<kRowE4m3>(x, residual, weight, y, y_e4m3, y_scale, residual_out, rstd, T, H, eps, io,
                             wt, stream);
}

extern "C" gbln_status gbln_rmsnorm_fwd_ckpt8(const void* x, const void* residual, const void* weight,
                                              void* y, void* residual_out, float* rstd, uint8_t* h8,
                                              float* h8_scale, int64_t T, int64_t H, float eps,
                                              gbln_q8 fmt, gbln_dtype io, gbln_dtype wt,
                                              gbln_stream_t stream) {
  if (!q8_ok(fmt)) return GBLN_ERR_INVALID_ARG;
  if (fmt == GBLN_Q8_INT8)
    return fwd_entry<kCkptInt8>(x, residual, weight, y, h8, h8_scale, residual_out, rstd, T, H, eps, io,
                                wt, stream);
  return fwd_entry<kCkptE4m3>(x, residual, weight, y, h8, h8_scale, residual_out, rstd, T, H, eps, io, wt,
                              stream);
}

extern "C" int64_t gbln_rmsnorm_bwd_ckpt8_num_partials(int64_t T, int64_t H, gbln_dtype io) {
  if (!dtype_ok(io) || T < 0 || T > kMaxRows || H <= 0 || H > kMaxH) return -1;
  if (T == 0) return 0;
  const int sms = sm_count();
  if (sms <= 0) return -1;
  return partials_for(T, bwd_geometry(H, dtype_size(io)), sms);
}

extern "C" gbln_status gbln_rmsnorm_bwd_ckpt8(const void* dy, const void* dresidual_out,
                                              const uint8_t* h8, const float* h8_scale,
                                              const void* weight, const float* rstd, void* dx,
                                              float* dw_partial, int64_t P_cap, int64_t T, int64_t H,
                                              gbln_q8 fmt, gbln_dtype io, gbln_dtype wt,
                                              gbln_stream_t stream) {
  if (!q8_ok(fmt) || P_cap < 0) return GBLN_ERR_INVALID_ARG;
  const gbln_status st = sizes_and_types(T, H, io, wt);
  if (st != GBLN_OK) return st;
  if (T == 0) return GBLN_OK;  // nothing is read or written: pointers are not examined
  if (!dy || !h8 || !h8_scale || !weight || !rstd || !dx || !dw_partial) return GBLN_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return GBLN_ERR_CUDA;
  const int64_t P = partials_for(T, bwd_geometry(H, dtype_size(io)), sms);
  if (P_cap < P) return GBLN_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  if (io == GBLN_F32)
    return bwd_typed<float, float>(dy, dresidual_out, h8, h8_scale, weight, rstd, dx, dw_partial, P, T, H, fmt, s);
  if (wt == GBLN_BF16)
    return bwd_typed<bf16, bf16>(dy, dresidual_out, h8, h8_scale, weight, rstd, dx, dw_partial, P, T, H, fmt, s);
  return bwd_typed<bf16, float>(dy, dresidual_out, h8, h8_scale, weight, rstd, dx, dw_partial, P, T, H, fmt, s);
}
