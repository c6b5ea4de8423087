// What stands between two blocks of a residual stream, in one pass:
//   n = y * ry * w_post,  ry = 1 / sqrt(mean(y^2) + eps)     (n = y without w_post)
//   r = alpha * x + g * n            the new residual, rounded to its type
//   h = r * rr * w_pre,   rr = 1 / sqrt(mean(r^2) + eps)     (next block's input)
// g: nothing, one factor per channel, per row, or per element.  h reads r as it
// is stored, so that a program which norms the stored stream gets the same h
// and the gradient, which has only the stored r, belongs to the same function.
// Sums are fp32, r and h are rounded once.
//
// Gradient, from dr and dh:
//   v  = dh * w_pre                     d  = dr + rr (v - r rr^2 mean(v r))
//   dx = alpha d                        q  = d g w_post
//   dy = ry (q - y ry^2 mean(q y))      (d g without w_post)
//   dw_pre = sum_t dh r rr,  dw_post = sum_t d g y ry,  dg = [sums of] d n
// mean(q y) needs d, which needs mean(v r).  With b = g w_post y the dot product
// splits, sum q y = sum (dr + rr v) b - rr^3 mean(v r) sum r b, so one block
// reduction of three sums serves both means.
#include "common.cuh"
#include "kernels.h"

namespace lmoe {

namespace {

constexpr int kVec = 8;                       // elements per thread and step

template <typename T> struct Pack;            // 8 elements as they lie in memory
template <> struct Pack<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(h[i]);
      f[2 * i] = t.x; f[2 * i + 1] = t.y;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
};
template <> struct Pack<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Sums of N values over the block; every thread gets them.  buf holds N x 32
// floats and must not be the one of the previous call (a fast warp may already
// write the next sums while a slow one reads these).
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
  if (lane == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) buf[n * 32 + warp] = v[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float s = lane < nw ? buf[n * 32 + lane] : 0.f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    v[n] = s;
  }
}

__device__ __forceinline__ float rstd_of(float sum, int D, float eps) {
  return 1.0f / sqrtf(sum / (float)D + eps);
}

template <typename T, int VPT>
__global__ void __launch_bounds__(1024)
norm_fwd_kernel(const moe_norm_args a) {
  __shared__ float s_red[2][32];
  const int D = a.D, nv = D / kVec;
  const long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* y = static_cast<const T*>(a.y) + row * a.ldy;
  const T* gate = static_cast<const T*>(a.gate);
  const T* wpost = static_cast<const T*>(a.post_weight);
  const T* wpre = static_cast<const T*>(a.pre_weight);
  T* r = static_cast<T*>(a.r) + row * a.ldr;
  Pack<T> py[VPT], px[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    py[i].zero(); px[i].zero();
    if (v < nv) { py[i].load(y + v * kVec); px[i].load(x + v * kVec); }
  }
  float ry = 1.f;
  if (wpost) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
      py[i].get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(f[j], f[j], s[0]);
    }
    block_sum<1>(s, s_red[0]);
    ry = rstd_of(s[0], D, a.eps);
    if (a.rstd_y && threadIdx.x == 0) a.rstd_y[row] = ry;
  }
  const float gt = a.gate_kind == MOE_GATE_TOKEN ? to_f32(gate[row * a.ldg]) : 1.f;
  float s2[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) continue;
    float fy[8], fx[8], w[8];
    py[i].get(fy);
    px[i].get(fx);
    Pack<T> p;
    if (wpost) {
      p.load(wpost + v * kVec);
      p.get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) fy[j] = fy[j] * ry * w[j];
    }
    if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL) {
      p.load(gate + (a.gate_kind == MOE_GATE_FULL ? row * a.ldg : 0) + v * kVec);
      p.get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) fy[j] *= w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) fy[j] *= gt;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) fx[j] = fmaf(a.residual_scale, fx[j], fy[j]);
    px[i].set(fx);
    px[i].store(r + v * kVec);
    px[i].get(fx);                               // as stored
#pragma unroll
    for (int j = 0; j < 8; ++j) s2[0] = fmaf(fx[j], fx[j], s2[0]);
  }
  if (!wpre) return;
  block_sum<1>(s2, s_red[1]);
  const float rr = rstd_of(s2[0], D, a.eps);
  if (a.rstd_r && threadIdx.x == 0) a.rstd_r[row] = rr;
  T* h = static_cast<T*>(a.h) + row * a.ldh;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) continue;
    float f[8], w[8];
    px[i].get(f);
    Pack<T> p;
    p.load(wpre + v * kVec);
    p.get(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * rr * w[j];
    p.set(f);
    p.store(h + v * kVec);
  }
}

// One block walks rows blockIdx.x, + gridDim.x, ...; thread i keeps the column
// sums of its VPT vectors in registers and writes one partial row per block and
// weight at the end (parts [3][grid][D]: post, pre, gate), which a second
// kernel adds in block order.
template <typename T, int VPT>
__global__ void __launch_bounds__(1024)
norm_bwd_kernel(const moe_norm_args a, float* parts) {
  __shared__ float s_red[2][3 * 32];
  const int D = a.D, nv = D / kVec;
  const T* gate = static_cast<const T*>(a.gate);
  const T* wpost = static_cast<const T*>(a.post_weight);
  const T* wpre = static_cast<const T*>(a.pre_weight);
  const bool gvec = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL;
  // sums of d y ry (a channel gate: dgate and dpost are multiples of it), of
  // d g y ry otherwise; and of dh r rr
  float ca[VPT][8], cb[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ca[i][j] = cb[i][j] = 0.f;
  int it = 0;
  for (long row = blockIdx.x; row < a.T; row += gridDim.x, ++it) {
    const T* y = static_cast<const T*>(a.y) + row * a.ldy;
    const T* r = static_cast<const T*>(a.r) + row * a.ldr;
    const T* dr = a.dr ? static_cast<const T*>(a.dr) + row * a.lddr : nullptr;
    const T* dh = wpre ? static_cast<const T*>(a.dh) + row * a.lddh : nullptr;
    const float ry = wpost ? a.rstd_y[row] : 1.f, rr = wpre ? a.rstd_r[row] : 0.f;
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? to_f32(gate[row * a.ldg]) : 1.f;
    Pack<T> py[VPT], pr[VPT], pd[VPT], ph[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      py[i].zero(); pr[i].zero(); pd[i].zero(); ph[i].zero();
      if (v < nv) {
        py[i].load(y + v * kVec);
        if (dr) pd[i].load(dr + v * kVec);
        if (wpre) { pr[i].load(r + v * kVec); ph[i].load(dh + v * kVec); }
      }
    }
    // sum v r; sum (dr + rr v) b; sum r b, with b = w_post y [gate vector]
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nv) continue;
      float fy[8], fr[8], fd[8], fh[8], w[8];
      Pack<T> p;
      py[i].get(fy); pr[i].get(fr); pd[i].get(fd); ph[i].get(fh);
      if (wpre) {
        p.load(wpre + v * kVec);
        p.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          fh[j] *= w[j];
          s[0] = fmaf(fh[j], fr[j], s[0]);
          fd[j] = fmaf(rr, fh[j], fd[j]);
        }
      }
      if (wpost) {
        p.load(wpost + v * kVec);
        p.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) fy[j] *= w[j];
      }
      if (gvec) {
        p.load(gate + (a.gate_kind == MOE_GATE_FULL ? row * a.ldg : 0) + v * kVec);
        p.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) fy[j] *= w[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[1] = fmaf(fd[j], fy[j], s[1]);
        s[2] = fmaf(fr[j], fy[j], s[2]);
      }
    }
    block_sum<3>(s, s_red[it & 1]);
    const float m1 = rr * rr * rr * (s[0] / (float)D);     // d = dr + rr v - m1 r
    const float dot = s[1] - m1 * s[2];                    // sum d b
    const float m2 = wpost ? ry * ry * ry * gt * (dot / (float)D) : 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0)
      static_cast<float*>(a.dgate)[row] = ry * dot;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
    T* dy = static_cast<T*>(a.dy) + row * a.lddy;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nv) continue;
      float fy[8], fr[8], d[8], f[8], w[8], g[8];
      Pack<T> p;
      py[i].get(fy); pr[i].get(fr); pd[i].get(d); ph[i].get(f);
      if (wpre) {
        p.load(wpre + v * kVec);
        p.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          cb[i][j] = fmaf(f[j] * rr, fr[j], cb[i][j]);
          d[j] = fmaf(rr, f[j] * w[j], d[j]) - m1 * fr[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = a.residual_scale * d[j];
      p.set(f);
      p.store(dx + v * kVec);
#pragma unroll
      for (int j = 0; j < 8; ++j) { g[j] = gt; w[j] = 1.f; }
      if (gvec) {
        p.load(gate + (a.gate_kind == MOE_GATE_FULL ? row * a.ldg : 0) + v * kVec);
        p.get(g);
      }
      if (wpost) { p.load(wpost + v * kVec); p.get(w); }
      if (a.gate_kind == MOE_GATE_FULL) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = d[j] * fy[j] * ry * w[j];
        p.set(f);
        p.store(static_cast<T*>(a.dgate) + row * a.lddg + v * kVec);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dn = d[j] * g[j];
        ca[i][j] = fmaf(a.gate_kind == MOE_GATE_CHANNEL ? d[j] : dn, fy[j] * ry, ca[i][j]);
        f[j] = wpost ? fmaf(ry, dn * w[j], -m2 * fy[j]) : dn;
      }
      p.set(f);
      p.store(dy + v * kVec);
    }
  }
  // partial column sums of this block
  const size_t plane = (size_t)gridDim.x * D;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) continue;
    float* o = parts + (size_t)blockIdx.x * D + v * kVec;
    *reinterpret_cast<float4*>(o) = make_float4(ca[i][0], ca[i][1], ca[i][2], ca[i][3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(ca[i][4], ca[i][5], ca[i][6], ca[i][7]);
    if (wpre) {
      o += plane;
      *reinterpret_cast<float4*>(o) = make_float4(cb[i][0], cb[i][1], cb[i][2], cb[i][3]);
      *reinterpret_cast<float4*>(o + 4) = make_float4(cb[i][4], cb[i][5], cb[i][6], cb[i][7]);
    }
  }
}

// Column sums of the blocks' partial rows, in block order within each of 32
// strands and then over the strands: 32 columns x 32 strands per block.
template <typename T>
__global__ void __launch_bounds__(1024)
norm_bwd_reduce_kernel(const moe_norm_args a, const float* __restrict__ parts, int nblk) {
  __shared__ float s_a[32][33], s_b[32][33];
  const int c = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  const size_t plane = (size_t)nblk * a.D;
  float va = 0.f, vb = 0.f;
  if (col < a.D)
    for (int b = strand; b < nblk; b += 32) {
      va += parts[(size_t)b * a.D + col];
      if (a.pre_weight) vb += parts[plane + (size_t)b * a.D + col];
    }
  s_a[strand][c] = va;
  s_b[strand][c] = vb;
  __syncthreads();
  if (strand != 0 || col >= a.D) return;
  va = vb = 0.f;
  for (int s = 0; s < 32; ++s) { va += s_a[s][c]; vb += s_b[s][c]; }
  if (a.pre_weight) static_cast<float*>(a.dpre_weight)[col] = vb;
  if (a.gate_kind == MOE_GATE_CHANNEL) {
    const float w = a.post_weight ? to_f32(static_cast<const T*>(a.post_weight)[col]) : 1.f;
    static_cast<float*>(a.dgate)[col] = va * w;
    va *= to_f32(static_cast<const T*>(a.gate)[col]);
  }
  if (a.post_weight) static_cast<float*>(a.dpost_weight)[col] = va;
}

// threads and vectors per thread for D / 8 vectors
struct Shape { int threads, vpt; };
Shape shape_for(int D, int want) {
  const int nv = D / kVec;
  int vpt = want;
  while (ceil_div(nv, vpt) > 1024) vpt *= 2;
  return {(ceil_div(nv, vpt) + 31) / 32 * 32, vpt};
}

template <typename T>
cudaError_t fwd_t(const moe_norm_args& a, cudaStream_t st) {
  const Shape s = shape_for(a.D, 1);
  if (s.vpt == 1) norm_fwd_kernel<T, 1><<<a.T, s.threads, 0, st>>>(a);
  else norm_fwd_kernel<T, 2><<<a.T, s.threads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(const moe_norm_args& a, float* ws, int nblk, cudaStream_t st) {
  const Shape s = shape_for(a.D, 1);
  if (s.vpt == 1) norm_bwd_kernel<T, 1><<<nblk, s.threads, 0, st>>>(a, ws);
  else norm_bwd_kernel<T, 2><<<nblk, s.threads, 0, st>>>(a, ws);
  if (a.post_weight || a.pre_weight || a.gate_kind == MOE_GATE_CHANNEL)
    norm_bwd_reduce_kernel<T><<<ceil_div(a.D, 32), 1024, 0, st>>>(a, ws, nblk);
  return cudaGetLastError();
}

}  // namespace

int norm_bwd_blocks(int T) { return T < 296 ? T : 296; }

size_t norm_bwd_workspace(int T, int D) { return (size_t)2 * norm_bwd_blocks(T) * D * 4; }

cudaError_t launch_norm_fwd(const moe_norm_args& a, cudaStream_t st) {
  return a.dtype == MOE_BF16 ? fwd_t<__nv_bfloat16>(a, st) : fwd_t<float>(a, st);
}

cudaError_t launch_norm_bwd(const moe_norm_args& a, void* ws, cudaStream_t st) {
  const int nblk = norm_bwd_blocks(a.T);
  return a.dtype == MOE_BF16 ? bwd_t<__nv_bfloat16>(a, static_cast<float*>(ws), nblk, st)
                             : bwd_t<float>(a, static_cast<float*>(ws), nblk, st);
}

}  // namespace lmoe
