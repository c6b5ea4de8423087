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
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace lmoe {

namespace {

constexpr float kF8Max = 448.f;
constexpr float kF8Floor = 0x1p-100f;

// four values, scaled, as four E4M3 codes
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// 8 elements of a row from column c on: vector loads where the row is aligned
// and whole, zeros past K
template <typename T>
__device__ __forceinline__ void load_row8(const T* row, int c, int K, bool vec, float (&f)[8]) {
  if (vec && c + 8 <= K) {
    load8(row + c, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = c + j < K ? ld1(row + c + j) : 0.f;
  }
}

__device__ __forceinline__ void store_codes8(uint8_t* row, int c, int K, uint32_t lo, uint32_t hi) {
  if (c + 8 <= K) {
    *reinterpret_cast<uint2*>(row + c) = make_uint2(lo, hi);
  } else {
    for (int j = 0; c + j < K && j < 8; ++j)
      row[c + j] = (uint8_t)((j < 4 ? lo >> (8 * j) : hi >> (8 * (j - 4))) & 0xffu);
  }
}

struct QuantArgs {
  const void* x;
  long ldx;
  int rows, K;             // of the output (rows) / of the input (transpose, weights)
  const int32_t* perm;     // rows: input row of output row r is perm[r] / k (NULL: r)
  int k, x_rows, relu2;
  uint8_t* codes;
  long ldc;
  float* scales;
  long lds;
  uint8_t* codes_t;
  long ldct;
  float* scales_t;
  int vec;                 // rows of x start on 16 bytes
};

// 16 lanes per block of 128, kQRows rows x kQBlocks blocks per CTA
constexpr int kQRows = 16, kQBlocks = 4;

template <typename T, bool RELU2>
__global__ void __launch_bounds__(256)
quant_rows_kernel(const QuantArgs a) {
  __shared__ float s_scale[kQBlocks][kQRows];
  const int sub = threadIdx.x & 15, rl = threadIdx.x >> 4;
  const int kb0 = blockIdx.x * kQBlocks, nkb = ceil_div(a.K, 128);
  for (long r0 = (long)blockIdx.y * kQRows; r0 < a.rows; r0 += (long)gridDim.y * kQRows) {
    const long r = r0 + rl;
    long src = r;
    if (r < a.rows && a.perm) {
      const int p = a.perm[r];
      src = p >= 0 && p / a.k < a.x_rows ? p / a.k : -1;
    }
    const bool ok = r < a.rows && src >= 0;
    const T* row = static_cast<const T*>(a.x) + (ok ? src : 0) * a.ldx;
    float f[kQBlocks][8];
#pragma unroll
    for (int b = 0; b < kQBlocks; ++b) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[b][j] = 0.f;
      if (ok) load_row8(row, (kb0 + b) * 128 + sub * 8, a.K, a.vec, f[b]);
    }
#pragma unroll
    for (int b = 0; b < kQBlocks; ++b) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (RELU2) { const float v = f[b][j] > 0.f ? f[b][j] : (f[b][j] != f[b][j] ? f[b][j] : 0.f); f[b][j] = v * v; }
        m = fmaxf(m, fabsf(f[b][j]));
      }
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      m = fmaxf(m, kF8Floor);
      const float q = __fdiv_rn(kF8Max, m);
      const int c = (kb0 + b) * 128 + sub * 8;
      if (r < a.rows && c < a.K)
        store_codes8(a.codes + r * a.ldc, c, a.K,
                     pack4(f[b][0] * q, f[b][1] * q, f[b][2] * q, f[b][3] * q),
                     pack4(f[b][4] * q, f[b][5] * q, f[b][6] * q, f[b][7] * q));
      if (sub == 0) s_scale[b][rl] = __fdiv_rn(m, kF8Max);
    }
    __syncthreads();
    if (threadIdx.x < kQBlocks * kQRows) {
      const int b = threadIdx.x / kQRows, i = threadIdx.x % kQRows;
      if (kb0 + b < nkb && r0 + i < a.rows) a.scales[(kb0 + b) * a.lds + r0 + i] = s_scale[b][i];
    }
    __syncthreads();
  }
}

// transpose: a CTA takes 128 rows x 64 columns of x; thread = (column, quarter
// of the rows).  Codes of column c go to row c of the output.
template <typename T>
__global__ void __launch_bounds__(256)
quant_cols_kernel(const QuantArgs a) {
  __shared__ T s_x[128][64 + 8];
  __shared__ float s_max[4][64];
  const int c0 = blockIdx.x * 64;
  const int r0 = blockIdx.y * 128;
  for (int i = threadIdx.x; i < 128 * 8; i += 256) {
    const int r = i >> 3, c = (i & 7) * 8;
    const T* row = static_cast<const T*>(a.x) + (long)min(r0 + r, a.rows - 1) * a.ldx;
    float f[8];
    load_row8(row, c0 + c, r0 + r < a.rows ? a.K : 0, a.vec, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) store_val(&s_x[r][c + j], f[j]);       // exact: back to x's type
  }
  __syncthreads();
  const int c = threadIdx.x & 63, quarter = threadIdx.x >> 6;
  float m = 0.f;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(ld1(&s_x[quarter * 32 + i][c])));
  s_max[quarter][c] = m;
  __syncthreads();
  m = fmaxf(fmaxf(fmaxf(s_max[0][c], s_max[1][c]), fmaxf(s_max[2][c], s_max[3][c])), kF8Floor);
  if (c0 + c >= a.K) return;
  const float q = __fdiv_rn(kF8Max, m);
  uint8_t* out = a.codes + (long)(c0 + c) * a.ldc;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = ld1(&s_x[quarter * 32 + i + j][c]) * q;
    store_codes8(out, r0 + quarter * 32 + i, a.rows, pack4(f[0], f[1], f[2], f[3]),
                 pack4(f[4], f[5], f[6], f[7]));
  }
  if (quarter == 0) a.scales[(long)blockIdx.y * a.lds + c0 + c] = __fdiv_rn(m, kF8Max);
}

// weights: a CTA per 128 x 128 block; 256 threads hold 64 elements each
template <typename T>
__global__ void __launch_bounds__(256)
quant_square_kernel(const QuantArgs a) {
  __shared__ float s_max[8];
  __shared__ uint8_t s_t[128][128 + 4];
  const int nb = blockIdx.x, kb = blockIdx.y;
  const long mat = blockIdx.z;
  const int NB = ceil_div(a.rows, 128), KB = ceil_div(a.K, 128);
  const T* x = static_cast<const T*>(a.x) + mat * a.rows * a.ldx;
  const int sub = threadIdx.x & 15, rl = threadIdx.x >> 4;
  float f[8][8], m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = nb * 128 + rl + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    if (r < a.rows) load_row8(x + r * a.ldx, kb * 128 + sub * 8, a.K, a.vec, f[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[i][j]));
  }
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
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rr = rl + 16 * i, r = nb * 128 + rr, c = kb * 128 + sub * 8;
    const uint32_t lo = pack4(f[i][0] * q, f[i][1] * q, f[i][2] * q, f[i][3] * q);
    const uint32_t hi = pack4(f[i][4] * q, f[i][5] * q, f[i][6] * q, f[i][7] * q);
    if (r < a.rows && c < a.K) store_codes8(codes + r * a.ldc, c, a.K, lo, hi);
    if (a.codes_t) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s_t[sub * 8 + j][rr] = (uint8_t)(lo >> (8 * j));
        s_t[sub * 8 + 4 + j][rr] = (uint8_t)(hi >> (8 * j));
      }
    }
  }
  if (!a.codes_t) return;
  __syncthreads();
  uint8_t* codes_t = a.codes_t + mat * a.K * a.ldct;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int cc = rl + 16 * i, c = kb * 128 + cc, r = nb * 128 + sub * 8;
    if (c >= a.K || r >= a.rows) continue;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&s_t[cc][sub * 8]);
    store_codes8(codes_t + c * a.ldct, r, a.rows, w[0], w[1]);
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
  if (dt == MOE_BF16) {
    if (relu2) quant_rows_kernel<__nv_bfloat16, true><<<grid, 256, 0, st>>>(a);
    else quant_rows_kernel<__nv_bfloat16, false><<<grid, 256, 0, st>>>(a);
  } else {
    if (relu2) quant_rows_kernel<float, true><<<grid, 256, 0, st>>>(a);
    else quant_rows_kernel<float, false><<<grid, 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_quantize_fp8_cols(const void* x, moe_dtype dt, int rows, int K, long ldx,
                                     uint8_t* codes, long ldc, float* scales, long lds,
                                     cudaStream_t st) {
  QuantArgs a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.K = K;
  a.codes = codes; a.ldc = ldc; a.scales = scales; a.lds = lds; a.vec = rows16(x, ldx, dt);
  const dim3 grid(ceil_div(K, 64), ceil_div(rows, 128));
  if (dt == MOE_BF16) quant_cols_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  else quant_cols_kernel<float><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_quantize_fp8_weight(const void* w, moe_dtype dt, int n_mat, int N, int K,
                                       long ldx, uint8_t* codes, long ldc, float* scales,
                                       uint8_t* codes_t, long ldct, float* scales_t,
                                       cudaStream_t st) {
  QuantArgs a{};
  a.x = w; a.ldx = ldx; a.rows = N; a.K = K; a.codes = codes; a.ldc = ldc; a.scales = scales;
  a.codes_t = codes_t; a.ldct = ldct; a.scales_t = scales_t; a.vec = rows16(w, ldx, dt);
  const dim3 grid(ceil_div(N, 128), ceil_div(K, 128), n_mat);
  if (dt == MOE_BF16) quant_square_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  else quant_square_kernel<float><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace lmoe
