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
#include <atomic>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace lmoe {

namespace {

__device__ int g_norm_err;                    // DEV_ERR_TIMEOUT

constexpr int kVec = 8;                       // elements per thread and step
constexpr int kMaxStages = 4;
constexpr int kMaxRing = 216 << 10;           // bytes of the backward's ring of rows

// `bytes` contiguous bytes into shared memory, completion signalled on `bar`
__device__ __forceinline__ void bulk_row(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(sm100::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes),
        "r"(sm100::smem_u32(bar))
      : "memory");
}

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
  // as four pairs
  __device__ __forceinline__ void get2(uint64_t (&f)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pack2(w[i] << 16, w[i] & 0xffff0000u);
  }
  __device__ __forceinline__ void set2(const uint64_t (&f)[4]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpack2(f[i], lo, hi);
      h[i] = __floats2bfloat162_rn(lo, hi);
    }
  }
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
  __device__ __forceinline__ void get2(uint64_t (&f)[4]) const {
    f[0] = pack2(a.x, a.y); f[1] = pack2(a.z, a.w); f[2] = pack2(b.x, b.y); f[3] = pack2(b.z, b.w);
  }
  __device__ __forceinline__ void set2(const uint64_t (&f)[4]) {
    unpack2(f[0], a.x, a.y); unpack2(f[1], a.z, a.w); unpack2(f[2], b.x, b.y); unpack2(f[3], b.z, b.w);
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
__global__ void __launch_bounds__(512)
norm_fwd_kernel(const moe_norm_args a) {
  __shared__ float s_red[2][32];
  let_next();
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

// One block walks rows blockIdx.x, + gridDim.x, ...  A row's inputs (y; r and dh;
// dr; a full gate) arrive by bulk copies into a ring of rows in shared memory,
// issued ahead by thread 0; the weights' vectors and the column sums stay in
// registers.  A stage is refilled after the next row's block barrier, which
// every thread reaches only when it is through with the stage.  Rows too long
// for two stages are read from global memory directly (stages = 0).  What is
// absent is filled in so that one formula serves: no w_post or gate is 1, no
// w_pre is dh = r = 0.  At the end a block writes one partial row per kind of
// column sum (parts [2][grid][D]), which a second kernel adds in block order.
// Two sums per column are enough: with a channel gate dgate = w_post S and
// dpost = g S, S = sum_t d y ry.
//
// Six rows of D move per row; an element costs about 17 instructions in packed
// fp32 pairs (30 unpacked, which bounded the kernel).  T = D = 8192 bf16: 152 us
// (5.3 TB/s), the 64 partial rows' sum 5 us more.
template <typename T, int VPT, bool FULL, bool RING>
__global__ void __launch_bounds__(512)
norm_bwd_kernel(const moe_norm_args a, float* parts, const int stages) {
  extern __shared__ __align__(16) uint8_t s_ring[];
  __shared__ float s_red[2][3 * 32];
  __shared__ uint64_t s_full[kMaxStages];
  constexpr bool kHold = VPT <= 2;                         // weights in registers
  const int D = a.D, nv = D / kVec;
  const uint32_t row_bytes = D * sizeof(T);
  const T* wpost = static_cast<const T*>(a.post_weight);
  const T* wpre = static_cast<const T*>(a.pre_weight);
  const T* gvec = a.gate_kind == MOE_GATE_CHANNEL ? static_cast<const T*>(a.gate) : nullptr;
  // a row's arrays, in this order: y, [r, dh], [dr], [gate]
  const int n_dr = wpre ? 3 : 1, n_gate = n_dr + (a.dr != nullptr);
  const uint32_t stage_bytes = (n_gate + FULL) * row_bytes;

  auto source = [&](int k, long row) -> const T* {
    if (k == 0) return static_cast<const T*>(a.y) + row * a.ldy;
    if (wpre && k == 1) return static_cast<const T*>(a.r) + row * a.ldr;
    if (wpre && k == 2) return static_cast<const T*>(a.dh) + row * a.lddh;
    if (a.dr && k == n_dr) return static_cast<const T*>(a.dr) + row * a.lddr;
    return static_cast<const T*>(a.gate) + row * a.ldg;
  };
  auto fetch = [&](long row, int st) {
    sm100::mbar_arrive_expect_tx(&s_full[st], stage_bytes);
    for (int k = 0; k < n_gate + FULL; ++k)
      bulk_row(s_ring + (size_t)st * stage_bytes + k * row_bytes, source(k, row), row_bytes, &s_full[st]);
  };
  let_next();
  if (RING && threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) sm100::mbar_init(&s_full[i], 1);
    sm100::fence_mbar_init();
    sm100::fence_proxy_async();
    for (int i = 0; i < stages; ++i) {
      const long row = blockIdx.x + (long)i * gridDim.x;
      if (row < a.T) fetch(row, i);
    }
  }
  const uint64_t one = both(1.f);
  // w_pre, and w_post times a channel gate (ones where there is none)
  auto weights = [&](int v, uint64_t (&we)[4], uint64_t (&wg)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) we[j] = wg[j] = one;
    if (v >= nv) return;
    Pack<T> p;
    if (wpre) { p.load(wpre + v * kVec); p.get2(we); }
    if (wpost) { p.load(wpost + v * kVec); p.get2(wg); }
    if (gvec) {
      uint64_t g[4];
      p.load(gvec + v * kVec);
      p.get2(g);
#pragma unroll
      for (int j = 0; j < 4; ++j) wg[j] = mul2(wg[j], g[j]);
    }
  };
  uint64_t we_[kHold ? VPT : 1][4], wg_[kHold ? VPT : 1][4], ca[VPT][4], cb[VPT][4];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if constexpr (kHold) weights(threadIdx.x + i * blockDim.x, we_[i], wg_[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) ca[i][j] = cb[i][j] = 0;
  }
  auto scalars = [&](long row, float& ry, float& rr, float& gt) {
    ry = wpost ? a.rstd_y[row] : 1.f;
    rr = wpre ? a.rstd_r[row] : 0.f;
    gt = a.gate_kind == MOE_GATE_TOKEN ? to_f32(static_cast<const T*>(a.gate)[row * a.ldg]) : 1.f;
  };
  float ry, rr, gt;
  scalars(blockIdx.x, ry, rr, gt);
  __syncthreads();                                         // the barriers exist
  int st = 0, phase = 0, it = 0;
  for (long row = blockIdx.x; row < a.T; row += gridDim.x, it ^= 1) {
    // a bulk copy that never lands is reported, not waited for without end
    if (RING && !sm100::mbar_wait(&s_full[st], phase)) atomicOr(&g_norm_err, DEV_ERR_TIMEOUT);
    const T* ring = reinterpret_cast<const T*>(s_ring + (size_t)st * stage_bytes);
    // vector v of the row's array k
    auto get = [&](int k, int v, uint64_t (&f)[4]) {
      Pack<T> p;
      if constexpr (RING) p.load(ring + k * D + v * kVec);
      else p.load(source(k, row) + v * kVec);
      p.get2(f);
    };
    // r, dh and dr of vector v (zeros where absent), y, the weights; with a full
    // gate wg is w_post times it
    auto vector = [&](int i, int v, uint64_t (&fr)[4], uint64_t (&fh)[4], uint64_t (&fd)[4],
                      uint64_t (&fy)[4], uint64_t (&we)[4], uint64_t (&wg)[4], uint64_t (&g)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) fr[j] = fh[j] = fd[j] = 0;
      get(0, v, fy);
      if (wpre) { get(1, v, fr); get(2, v, fh); }
      if (a.dr) get(n_dr, v, fd);
      if constexpr (kHold) {
#pragma unroll
        for (int j = 0; j < 4; ++j) { we[j] = we_[i][j]; wg[j] = wg_[i][j]; }
      } else {
        weights(v, we, wg);
      }
      if constexpr (FULL) {
        get(n_gate, v, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) wg[j] = mul2(wg[j], g[j]);
      }
    };
    // sum v r; sum (dr + rr v) b; sum r b, with b = w_post y [gate vector]
    uint64_t s0 = 0, s1 = 0, s2 = 0;
    const uint64_t rr2 = both(rr);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nv) continue;
      uint64_t fr[4], fh[4], fd[4], fy[4], we[4], wg[4], g[4];
      vector(i, v, fr, fh, fd, fy, we, wg, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t vv = mul2(fh[j], we[j]), b = mul2(fy[j], wg[j]);
        s0 = fma2(vv, fr[j], s0);
        s1 = fma2(fma2(rr2, vv, fd[j]), b, s1);
        s2 = fma2(fr[j], b, s2);
      }
    }
    float s[3], hi;
    unpack2(s0, s[0], hi); s[0] += hi;
    unpack2(s1, s[1], hi); s[1] += hi;
    unpack2(s2, s[2], hi); s[2] += hi;
    block_sum<3>(s, s_red[it]);
    if (RING && threadIdx.x == 0 && row >= (long)gridDim.x) {          // the last row's stage
      const long next = row + (long)(stages - 1) * gridDim.x;
      if (next < a.T) fetch(next, st ? st - 1 : stages - 1);
    }
    // d = dr + rr v - m1 r.  One factor at a time: a mean of products with y or r
    // is of the size of its partner over ry, so the first factor brings it back
    // into range, where ry^3 by itself leaves it from |y| = 1e13 on.
    const float m1 = rr * (rr * (rr * (s[0] / (float)D)));
    const float dot = s[1] - m1 * s[2];                    // sum d b
    const float m2 = wpost ? gt * (ry * (ry * (ry * (dot / (float)D)))) : 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0)
      static_cast<float*>(a.dgate)[row] = ry * dot;
    const uint64_t m12 = both(-m1), m22 = both(-m2), ry2 = both(ry), gt2 = both(gt),
                   rg2 = both(ry * gt), al2 = both(a.residual_scale);
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
    T* dy = static_cast<T*>(a.dy) + row * a.lddy;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nv) continue;
      uint64_t fr[4], fh[4], d[4], fy[4], we[4], wg[4], g[4];
      vector(i, v, fr, fh, d, fy, we, wg, g);
      Pack<T> p;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        fh[j] = mul2(fh[j], rr2);
        cb[i][j] = fma2(fh[j], fr[j], cb[i][j]);
        d[j] = fma2(m12, fr[j], fma2(fh[j], we[j], d[j]));
        fr[j] = mul2(al2, d[j]);
        fh[j] = mul2(fy[j], ry2);                          // y ry
      }
      p.set2(fr);
      p.store(dx + v * kVec);
      if constexpr (FULL) {
        uint64_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = one;
        if (wpost) { Pack<T> q; q.load(wpost + v * kVec); q.get2(w); }
#pragma unroll
        for (int j = 0; j < 4; ++j) fr[j] = mul2(mul2(d[j], fh[j]), w[j]);
        p.set2(fr);
        p.store(static_cast<T*>(a.dgate) + row * a.lddg + v * kVec);
#pragma unroll
        for (int j = 0; j < 4; ++j) fh[j] = mul2(fh[j], g[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // S of a channel gate; otherwise the gate (gt, g) belongs to dpost's sum
        ca[i][j] = fma2(mul2(d[j], gt2), fh[j], ca[i][j]);
        fr[j] = fma2(m22, fy[j], mul2(mul2(d[j], wg[j]), rg2));
      }
      p.set2(fr);
      p.store(dy + v * kVec);
    }
    if (RING && ++st == stages) { st = 0; phase ^= 1; }
    scalars(min(row + (long)gridDim.x, (long)a.T - 1), ry, rr, gt);       // the next row's
  }
  // partial column sums of this block
  const size_t plane = (size_t)gridDim.x * D;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) continue;
    Pack<float> p;
    p.set2(ca[i]);
    p.store(parts + (size_t)blockIdx.x * D + v * kVec);
    if (wpre) {
      p.set2(cb[i]);
      p.store(parts + plane + (size_t)blockIdx.x * D + v * kVec);
    }
  }
}

// Column sums of the blocks' partial rows, in block order within each of 32
// strands and then over the strands: 32 columns x 32 strands per block.
template <typename T>
__global__ void __launch_bounds__(1024)
norm_bwd_reduce_kernel(const moe_norm_args a, const float* parts, int nblk) {
  __shared__ float s_a[32][33], s_b[32][33];
  let_next();
  after_previous();
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

// Forward: about 256 threads a row, so that several rows are under way on an SM
// (D = 8192: 128 -> 94 us at 8192 rows against 1024 threads); with fewer rows
// than that fills, as many threads as the row has vectors (64 rows: 5.8 -> 4.2 us).
template <typename T>
cudaError_t fwd_t(const moe_norm_args& a, cudaStream_t st) {
  const int nv = a.D / kVec;
  const int vpt = a.T <= 296 ? (nv <= 512 ? 1 : nv <= 1024 ? 2 : 4) : nv <= 256 ? 1 : nv <= 512 ? 2 : 4;
  const int threads = (ceil_div(nv, vpt) + 31) / 32 * 32;
  if (vpt == 1) norm_fwd_kernel<T, 1><<<a.T, threads, 0, st>>>(a);
  else if (vpt == 2) norm_fwd_kernel<T, 2><<<a.T, threads, 0, st>>>(a);
  else norm_fwd_kernel<T, 4><<<a.T, threads, 0, st>>>(a);
  return cudaGetLastError();
}

// Backward: vectors per thread, threads, blocks per SM and ring stages.  Two
// vectors a thread (four past 1024 vectors, so that a block has at most 512
// threads) keep the weights and sums in registers; the SM's shared memory is
// shared out over enough blocks for 512 threads.
struct BwdShape { int vpt, threads, blocks, stages; size_t smem; };
BwdShape bwd_shape(const moe_norm_args& a) {
  BwdShape s;
  const int nv = a.D / kVec, es = a.dtype == MOE_BF16 ? 2 : 4;
  s.vpt = nv <= 256 ? 1 : nv <= 1024 ? 2 : 4;
  s.threads = (ceil_div(nv, s.vpt) + 31) / 32 * 32;
  int per_sm = 512 / s.threads;
  per_sm = per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm;
  const int arrays = 1 + (a.pre_weight ? 2 : 0) + (a.dr ? 1 : 0) + (a.gate_kind == MOE_GATE_FULL ? 1 : 0);
  const size_t row = (size_t)arrays * a.D * es, room = size_t(216) << 10;
  // (777 x 2056 fp32 with a full gate: three blocks an SM leave less than two stages)
  const size_t n = room / per_sm / row;
  s.stages = n < 2 ? 0 : n > kMaxStages ? kMaxStages : (int)n;
  s.smem = row * s.stages;
  const long blocks = 148L * per_sm;
  s.blocks = (int)(a.T < blocks ? a.T : blocks);
  return s;
}

template <typename T, int VPT, bool FULL, bool RING>
cudaError_t bwd_v(const moe_norm_args& a, const BwdShape& s, float* ws, cudaStream_t st) {
  auto kern = norm_bwd_kernel<T, VPT, FULL, RING>;
  static std::atomic<bool> configured[64];        // several threads may call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRing)) != cudaSuccess)
      return e;
    configured[dev] = true;
  }
  kern<<<s.blocks, s.threads, s.smem, st>>>(a, ws, s.stages);
  return cudaGetLastError();
}

template <typename T, bool FULL>
cudaError_t bwd_f(const moe_norm_args& a, const BwdShape& s, float* ws, cudaStream_t st) {
  if (s.vpt == 1) return bwd_v<T, 1, FULL, true>(a, s, ws, st);    // at most 2048 columns
  if (s.stages) return s.vpt == 2 ? bwd_v<T, 2, FULL, true>(a, s, ws, st) : bwd_v<T, 4, FULL, true>(a, s, ws, st);
  return s.vpt == 2 ? bwd_v<T, 2, FULL, false>(a, s, ws, st) : bwd_v<T, 4, FULL, false>(a, s, ws, st);
}

template <typename T>
cudaError_t bwd_t(const moe_norm_args& a, float* ws, cudaStream_t st) {
  const BwdShape s = bwd_shape(a);
  cudaError_t e = a.gate_kind == MOE_GATE_FULL ? bwd_f<T, true>(a, s, ws, st)
                                               : bwd_f<T, false>(a, s, ws, st);
  if (e == cudaSuccess && (a.post_weight || a.pre_weight || a.gate_kind == MOE_GATE_CHANNEL)) {
    e = launch_early(norm_bwd_reduce_kernel<T>, ceil_div(a.D, 32), 1024, 0, st, a, ws, s.blocks);
  }
  return e;
}

}  // namespace

// two partial rows for each block of any shape
size_t norm_bwd_workspace(int T, int D) {
  const int nv = D / kVec, threads = (ceil_div(nv, nv <= 256 ? 1 : nv <= 1024 ? 2 : 4) + 31) / 32 * 32;
  int per_sm = 512 / threads;
  per_sm = per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm;
  const long blocks = 148L * per_sm;
  return (size_t)2 * (T < blocks ? T : blocks) * D * 4;
}

cudaError_t norm_take_error(int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_norm_err, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && *word) e = cudaMemcpyToSymbol(g_norm_err, &zero, sizeof(int));
  return e;
}

cudaError_t launch_norm_fwd(const moe_norm_args& a, cudaStream_t st) {
  return a.dtype == MOE_BF16 ? fwd_t<__nv_bfloat16>(a, st) : fwd_t<float>(a, st);
}

cudaError_t launch_norm_bwd(const moe_norm_args& a, void* ws, cudaStream_t st) {
  return a.dtype == MOE_BF16 ? bwd_t<__nv_bfloat16>(a, static_cast<float*>(ws), st)
                             : bwd_t<float>(a, static_cast<float*>(ws), st);
}

}  // namespace lmoe
