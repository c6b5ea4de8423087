// Quantisation to E4M3 codes with one fp32 scale for each block of 128:
//   amax  = max(|v| over the block, 2^-100)
//   scale = amax / 448                 (fp32, rounded to nearest)
//   code  = E4M3(v * (448 / amax))     (both fp32 operations rounded to nearest,
//                                       then to nearest even)
// rows      blocks of 1 x 128 along K; scales [K blocks][rows], so that a GEMM
//           tile reads the scales of its rows from consecutive addresses
// transpose the same of the transposed matrix: blocks of 128 x 1 down the rows
// weights   blocks of 128 x 128, codes as they lie and, on demand, transposed
// All three read their input once; they are bound by memory.  The factor of a
// block is one division, an element costs one product and half a conversion.
// bf16: rows of 8192 x 8192 32 us (6.4 TB/s), with squared ReLU 45056 x 5120
// 105 us (6.6 TB/s); transposed 4096 x 8192 and 4096 x 2048 together 30 us (4.2
// TB/s); 2048 x 8192 weights both ways 20 us (3.4 TB/s).
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace lmoe {

namespace {

constexpr float kF8Max = 448.f;
constexpr float kF8Floor = 0x1p-100f;

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// two values times a factor as two E4M3 codes (nearest even, saturating)
__device__ __forceinline__ uint32_t codes2(float a, float b, float q) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a * q, b * q), __NV_SATFINITE, __NV_E4M3);
}

// 8 elements as they lie in memory; zeros past the row
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
  __device__ __forceinline__ void load_tail(const __nv_bfloat16* p, int n) {
    const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (2 * i < n ? u[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)u[2 * i + 1] << 16 : 0u);
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  // the largest |v| (RELU: the largest v, at least 0); NaN does not count
  template <bool RELU> __device__ __forceinline__ float amax() const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
    __nv_bfloat162 m = RELU ? __hmax2(h[0], __nv_bfloat162(__nv_bfloat16(0.f), __nv_bfloat16(0.f))) : __habs2(h[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2(m, RELU ? h[i] : __habs2(h[i]));
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), 0.f);
  }
};
template <> struct Raw8<float> {
  float w[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ void load_tail(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? p[i] : 0.f;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.f;
  }
  __device__ __forceinline__ float at(int i) const { return w[i]; }
  template <bool RELU> __device__ __forceinline__ float amax() const {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, RELU ? w[i] : fabsf(w[i]));
    return m;
  }
};

// 8 elements of a row from column c on
template <typename T>
__device__ __forceinline__ void load_row8(const T* row, int c, int K, bool vec, Raw8<T>& r) {
  if (c + 8 <= K && vec) r.load(row + c);
  else if (c < K) r.load_tail(row + c, K - c);
  else r.zero();
}

__device__ __forceinline__ float relu2_nan(float v) {          // max(v, 0)^2, NaN stays NaN
  float m;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(m) : "f"(v));
  return m * m;
}

template <bool RELU2, typename T>
__device__ __forceinline__ uint2 codes8(const Raw8<T>& r, float q) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = RELU2 ? relu2_nan(r.at(i)) : r.at(i);
  return make_uint2(codes2(f[0], f[1], q) | codes2(f[2], f[3], q) << 16,
                    codes2(f[4], f[5], q) | codes2(f[6], f[7], q) << 16);
}

__device__ __forceinline__ void store_codes8(uint8_t* row, int c, int K, uint2 v) {
  if (c + 8 <= K) {
    *reinterpret_cast<uint2*>(row + c) = v;
  } else {
    for (int j = 0; c + j < K && j < 8; ++j)
      row[c + j] = (uint8_t)((j < 4 ? v.x >> (8 * j) : v.y >> (8 * (j - 4))) & 0xffu);
  }
}

// 16 codes at row r, column c of a matrix of `rows` x `cols` codes
__device__ __forceinline__ void store_codes16(uint8_t* codes, long ld, const uint8_t* from, int r,
                                              int rows, int c, int cols) {
  if (r >= rows || c >= cols) return;
  const uint4 w = *reinterpret_cast<const uint4*>(from);
  uint8_t* out = codes + (long)r * ld;
  if (c + 16 <= cols) {
    *reinterpret_cast<uint4*>(out + c) = w;
  } else {
    store_codes8(out, c, cols, make_uint2(w.x, w.y));
    store_codes8(out, c + 8, cols, make_uint2(w.z, w.w));
  }
}

struct QuantArgs {
  const void* x;
  long ldx;
  int rows, K;             // of the output (rows) / of the input (transpose, weights)
  const int32_t* perm;     // rows: input row of output row r is perm[r] / k (NULL: r)
  int k, x_rows;
  uint8_t* codes;
  long ldc;
  float* scales;
  long lds;
  uint8_t* codes_t;
  long ldct;
  float* scales_t;
  int vec;                 // rows of x start on 16 bytes (transpose: on two elements)
};

// rows: 16 lanes per block of 128 (8 elements each), kQRows rows x kQBlocks
// blocks per CTA.  The 16 lanes reduce their kQBlocks maxima by halving
// exchanges, after which lane pair b holds block b's and does its two
// divisions, once for the 16 lanes; the factors come back by shuffle.
constexpr int kQRows = 16, kQBlocks = 8;

template <typename T, bool RELU2>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2)
quant_rows_kernel(const QuantArgs a) {
  __shared__ float s_scale[kQBlocks][kQRows + 1];
  const int sub = threadIdx.x & 15, rl = threadIdx.x >> 4;
  let_next();
  after_previous();
  const int kb0 = blockIdx.x * kQBlocks, nkb = (a.K + 127) >> 7;
  for (long r0 = (long)blockIdx.y * kQRows; r0 < a.rows; r0 += (long)gridDim.y * kQRows) {
    const long r = r0 + rl;
    long src = r;
    if (r < a.rows && a.perm) {
      const int p = a.perm[r];
      src = p >= 0 && p / a.k < a.x_rows ? p / a.k : -1;
    }
    const bool ok = r < a.rows && src >= 0;
    const T* row = static_cast<const T*>(a.x) + (ok ? src : 0) * a.ldx;
    Raw8<T> v[kQBlocks];
    float m[kQBlocks];
    if (a.vec && (kb0 + kQBlocks) * 128 <= a.K && ok) {
#pragma unroll
      for (int b = 0; b < kQBlocks; ++b) v[b].load(row + (kb0 + b) * 128 + sub * 8);
    } else {
#pragma unroll
      for (int b = 0; b < kQBlocks; ++b) load_row8(row, (kb0 + b) * 128 + sub * 8, ok ? a.K : 0, a.vec, v[b]);
    }
#pragma unroll
    for (int b = 0; b < kQBlocks; ++b) m[b] = v[b].template amax<RELU2>();
#pragma unroll
    for (int n = 4, bit = 8; n >= 1; n >>= 1, bit >>= 1) {
      const bool up = sub & bit;
#pragma unroll
      for (int i = 0; i < n; ++i)
        m[i] = fmaxf(up ? m[i + n] : m[i], __shfl_xor_sync(0xffffffffu, up ? m[i] : m[i + n], bit));
    }
    float top = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));    // of block sub / 2
    if (RELU2) top *= top;                    // rounding is monotone: the largest square
    top = fmaxf(top, kF8Floor);
    const float q = __fdiv_rn(kF8Max, top);
    if (!(sub & 1)) s_scale[sub >> 1][rl] = __fdiv_rn(top, kF8Max);
#pragma unroll
    for (int b = 0; b < kQBlocks; ++b) {
      const float qb = __shfl_sync(0xffffffffu, q, 2 * b, 16);
      const int c = (kb0 + b) * 128 + sub * 8;
      if (r < a.rows && c < a.K) store_codes8(a.codes + r * a.ldc, c, a.K, codes8<RELU2>(v[b], qb));
    }
    __syncthreads();
    if (threadIdx.x < kQBlocks * kQRows) {
      const int b = threadIdx.x / kQRows, i = threadIdx.x % kQRows;
      if (kb0 + b < nkb && r0 + i < a.rows) a.scales[(kb0 + b) * a.lds + r0 + i] = s_scale[b][i];
    }
    __syncthreads();
  }
}

// transpose: a CTA takes 128 rows x 64 columns of x, a warp 16 of the rows, a
// lane two neighbouring columns (a warp's loads are whole 128- or 256-byte
// runs).  A lane ends up with 16 consecutive bytes of two output rows; they go
// through shared memory so that a store instruction writes 128-byte runs (16
// bytes to each of 32 rows took twice the whole kernel's time).
template <typename T>
__global__ void __launch_bounds__(256)
quant_cols_kernel(const QuantArgs a) {
  __shared__ float s_max[8][64];
  __shared__ float s_q[64];
  __shared__ __align__(16) uint8_t s_t[64][128 + 16];
  let_next();
  after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 64 + 2 * lane;
  const long r0 = (long)blockIdx.y * 128 + 16 * warp;
  const T* x = static_cast<const T*>(a.x);
  float v[2][16], m0 = 0.f, m1 = 0.f;
  if (a.vec && (blockIdx.x + 1) * 64 <= a.K && r0 + 16 <= a.rows) {   // uniform in the warp:
    const T* p = x + r0 * a.ldx + c;                                  // 16 loads in flight
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (sizeof(T) == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p + i * a.ldx);
        v[0][i] = __uint_as_float(w << 16);
        v[1][i] = __uint_as_float(w & 0xffff0000u);
      } else {
        const float2 w = *reinterpret_cast<const float2*>(p + i * a.ldx);
        v[0][i] = w.x;
        v[1][i] = w.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool in = r0 + i < a.rows;
      v[0][i] = in && c < a.K ? ld1(x + (r0 + i) * a.ldx + c) : 0.f;
      v[1][i] = in && c + 1 < a.K ? ld1(x + (r0 + i) * a.ldx + c + 1) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) { m0 = fmaxf(m0, fabsf(v[0][i])); m1 = fmaxf(m1, fabsf(v[1][i])); }
  s_max[warp][2 * lane] = m0;
  s_max[warp][2 * lane + 1] = m1;
  __syncthreads();
  if (threadIdx.x < 64) {
    float m = kF8Floor;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, s_max[w][threadIdx.x]);
    s_q[threadIdx.x] = __fdiv_rn(kF8Max, m);
    const int cc = blockIdx.x * 64 + threadIdx.x;
    if (cc < a.K) a.scales[(long)blockIdx.y * a.lds + cc] = __fdiv_rn(m, kF8Max);
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float q = s_q[2 * lane + h];
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = codes2(v[h][4 * i], v[h][4 * i + 1], q) | codes2(v[h][4 * i + 2], v[h][4 * i + 3], q) << 16;
    *reinterpret_cast<uint4*>(&s_t[2 * lane + h][16 * warp]) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    store_codes16(a.codes, a.ldc, &s_t[(threadIdx.x >> 3) + 32 * i][16 * (threadIdx.x & 7)],
                  blockIdx.x * 64 + (threadIdx.x >> 3) + 32 * i, a.K,
                  blockIdx.y * 128 + 16 * (threadIdx.x & 7), a.rows);
}

// 4 x 4 bytes: w[i] holds row i's four columns; afterwards column i's four rows
__device__ __forceinline__ void transpose4(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  const uint32_t t0 = __byte_perm(a, b, 0x5140), t1 = __byte_perm(a, b, 0x7362);
  const uint32_t u0 = __byte_perm(c, d, 0x5140), u1 = __byte_perm(c, d, 0x7362);
  a = __byte_perm(t0, u0, 0x5410);
  b = __byte_perm(t0, u0, 0x7632);
  c = __byte_perm(t1, u1, 0x5410);
  d = __byte_perm(t1, u1, 0x7632);
}

// weights: a CTA per 128 x 128 block; a thread holds 8 rows x 8 columns, whose
// codes it transposes in registers
template <typename T>
__global__ void __launch_bounds__(256)
quant_square_kernel(const QuantArgs a) {
  __shared__ float s_max[8];
  __shared__ __align__(16) uint8_t s_t[128][128 + 16];
  let_next();
  after_previous();
  const int nb = blockIdx.x, kb = blockIdx.y;
  const long mat = blockIdx.z;
  const int NB = (a.rows + 127) >> 7, KB = (a.K + 127) >> 7;
  const T* x = static_cast<const T*>(a.x) + mat * a.rows * a.ldx;
  const int sub = threadIdx.x & 15, rl = threadIdx.x >> 4;
  const int r0 = nb * 128 + 8 * rl, c0 = kb * 128 + 8 * sub;
  Raw8<T> v[8];
  float m = 0.f;
  if (a.vec && (nb + 1) * 128 <= a.rows && (kb + 1) * 128 <= a.K) {    // no branch between the loads
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i].load(x + (long)(r0 + i) * a.ldx + c0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) load_row8(x + (long)(r0 + i) * a.ldx, c0, r0 + i < a.rows ? a.K : 0, a.vec, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, v[i].template amax<false>());
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = kF8Floor;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, s_max[i]);
  const float q = __fdiv_rn(kF8Max, m);
  if (threadIdx.x == 0) {
    const float s = __fdiv_rn(m, kF8Max);
    a.scales[(mat * NB + nb) * KB + kb] = s;
    if (a.scales_t) a.scales_t[(mat * KB + kb) * NB + nb] = s;
  }
  uint8_t* codes = a.codes + mat * a.rows * a.ldc;
  uint32_t lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint2 w = codes8<false>(v[i], q);
    lo[i] = w.x;
    hi[i] = w.y;
    if (r0 + i < a.rows && c0 < a.K) store_codes8(codes + (r0 + i) * a.ldc, c0, a.K, w);
  }
  if (!a.codes_t) return;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    transpose4(lo[i], lo[i + 1], lo[i + 2], lo[i + 3]);
    transpose4(hi[i], hi[i + 1], hi[i + 2], hi[i + 3]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    *reinterpret_cast<uint2*>(&s_t[8 * sub + j][8 * rl]) = make_uint2(lo[j], lo[j + 4]);
    *reinterpret_cast<uint2*>(&s_t[8 * sub + 4 + j][8 * rl]) = make_uint2(hi[j], hi[j + 4]);
  }
  __syncthreads();
  uint8_t* codes_t = a.codes_t + mat * a.K * a.ldct;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int cc = (threadIdx.x >> 3) + 32 * i, at = 16 * (threadIdx.x & 7);
    store_codes16(codes_t, a.ldct, &s_t[cc][at], kb * 128 + cc, a.K, nb * 128 + at, a.rows);
  }
}

bool rows16(const void* p, long ld, moe_dtype dt) {
  const long es = dt == MOE_BF16 ? 2 : 4;
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0;
}

}  // namespace

cudaError_t launch_quantize_fp8_rows(const void* x, moe_dtype dt, int rows, int K, long ldx,
                                     const int32_t* perm, int k, int x_rows, int relu2,
                                     uint8_t* codes, long ldc, float* scales, long lds,
                                     cudaStream_t st) {
  QuantArgs a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.K = K; a.perm = perm; a.k = k; a.x_rows = x_rows;
  a.codes = codes; a.ldc = ldc; a.scales = scales; a.lds = lds; a.vec = rows16(x, ldx, dt);
  const int gy = ceil_div(rows, kQRows);
  const dim3 grid(ceil_div(K, 128 * kQBlocks), gy < 65535 ? gy : 65535);
  cudaError_t e;
  if (dt == MOE_BF16) {
    if (relu2) e = launch_early(quant_rows_kernel<__nv_bfloat16, true>, grid, 256, 0, st, a);
    else e = launch_early(quant_rows_kernel<__nv_bfloat16, false>, grid, 256, 0, st, a);
  } else {
    if (relu2) e = launch_early(quant_rows_kernel<float, true>, grid, 256, 0, st, a);
    else e = launch_early(quant_rows_kernel<float, false>, grid, 256, 0, st, a);
  }
  return e;
}

cudaError_t launch_quantize_fp8_cols(const void* x, moe_dtype dt, int rows, int K, long ldx,
                                     uint8_t* codes, long ldc, float* scales, long lds,
                                     cudaStream_t st) {
  QuantArgs a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.K = K;
  a.codes = codes; a.ldc = ldc; a.scales = scales; a.lds = lds;
  a.vec = ldx % 2 == 0 && (reinterpret_cast<uintptr_t>(x) & (dt == MOE_BF16 ? 3u : 7u)) == 0;
  const dim3 grid(ceil_div(K, 64), ceil_div(rows, 128));
  cudaError_t e;
  if (dt == MOE_BF16) e = launch_early(quant_cols_kernel<__nv_bfloat16>, grid, 256, 0, st, a);
  else e = launch_early(quant_cols_kernel<float>, grid, 256, 0, st, a);
  return e;
}

cudaError_t launch_quantize_fp8_weight(const void* w, moe_dtype dt, int n_mat, int N, int K,
                                       long ldx, uint8_t* codes, long ldc, float* scales,
                                       uint8_t* codes_t, long ldct, float* scales_t,
                                       cudaStream_t st) {
  QuantArgs a{};
  a.x = w; a.ldx = ldx; a.rows = N; a.K = K; a.codes = codes; a.ldc = ldc; a.scales = scales;
  a.codes_t = codes_t; a.ldct = ldct; a.scales_t = scales_t; a.vec = rows16(w, ldx, dt);
  const dim3 grid(ceil_div(N, 128), ceil_div(K, 128), n_mat);
  cudaError_t e;
  if (dt == MOE_BF16) e = launch_early(quant_square_kernel<__nv_bfloat16>, grid, 256, 0, st, a);
  else e = launch_early(quant_square_kernel<float>, grid, 256, 0, st, a);
  return e;
}

}  // namespace lmoe
