// Stand-alone routing: top-k experts of given router logits, the gradient of
// the logits, and the grouping of the chosen pairs by expert.
//
// Forward, one row of logits l[E] with selection bias b[E]:
//   s_e = 1 / (1 + exp(-l_e))            or   exp(l_e - m) / sum_i exp(l_i - m)
//   c_e = s_e + b_e                      (both fp32; s evaluated in fp64, rounded once)
//   groups: E / n_group consecutive experts, scored by the fp32 sum of their two
//           largest c; the topk_group best stay eligible (ties: lower group)
//   idx = the k eligible experts of largest c (ties: lower expert)
//   w_j = s_idx / (sum s_idx + 1e-20) * scale     or   s_idx * scale
// A logit of -inf or NaN takes its expert out: score 0, never eligible.  Slots
// that no eligible expert is left for take the lowest experts not yet taken,
// with weight 0, so every row names k different experts in range.
//
// Why fp64 scores: selection compares neighbouring values, and an fp32 sigmoid
// or softmax is off by several units in the last place, enough to swap them.
#include "common.cuh"
#include "kernels.h"
#include "router_math.cuh"

namespace lmoe {

namespace {

__device__ int g_group_err;            // DEV_ERR_INDEX: an expert index out of range

constexpr int kRows = 8;               // rows (warps) per CTA

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// The layer's sigmoid without its clamp at +-80: beyond +-110 the fp32 result
// is 1 or 0 anyway, and inside +-80 the bits are the layer's.
__device__ __forceinline__ float sigmoid_score(float l) {
  const double a = -fmin(fmax((double)l, -110.0), 110.0);
  return __double2float_rn(__ddiv_rn(1.0, __dadd_rn(1.0, exp_fixed(a))));
}

// exp(l - m) for l <= m: below -700 the quotient rounds to 0 in fp32; l == m
// covers rows whose maximum is +inf.
__device__ __forceinline__ double softmax_term(float l, float m) {
  if (l == m) return 1.0;
  return exp_fixed(fmax((double)l - (double)m, -700.0));
}

__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);        // -0 orders as +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Keys order as choice scores do; experts out of the selection and experts
// already taken come below every score.
constexpr uint32_t kKeyOut = 1u, kKeyTaken = 0u;

// Group step for one row held by a warp (lane: experts lane + 32 i).
template <int EPL>
__device__ void drop_groups(float (&c)[EPL], int E, int n_group, int topk_group, int lane, float* gs) {
  const int G = E / n_group;
  for (int g = 0; g < n_group; ++g) {
    float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e >= g * G && e < (g + 1) * G) { m1 = fmaxf(m1, fminf(m0, c[i])); m0 = fmaxf(m0, c[i]); }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      const float o0 = __shfl_xor_sync(0xffffffffu, m0, off), o1 = __shfl_xor_sync(0xffffffffu, m1, off);
      m1 = fmaxf(fminf(m0, o0), fmaxf(m1, o1));
      m0 = fmaxf(m0, o0);
    }
    if (lane == 0) gs[g] = __fadd_rn(m0, m1);
  }
  __syncwarp();
  uint64_t keep = 0;
  for (int g0 = 0; g0 < n_group; g0 += 32) {
    const int g = g0 + lane;
    bool kg = false;
    if (g < n_group) {
      int r = 0;
      for (int o = 0; o < n_group; ++o) r += (gs[o] > gs[g] || (gs[o] == gs[g] && o < g)) ? 1 : 0;
      kg = r < topk_group;
    }
    keep |= (uint64_t)__ballot_sync(0xffffffffu, kg) << g0;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    if (e < E && !((keep >> (e / G)) & 1ull)) c[i] = -INFINITY;
  }
  __syncwarp();
}

struct TopkArgs {
  const void* logits;
  long ld;
  const float* bias;
  int T, E, k;
  int n_group, topk_group, renorm;
  float scale;
  int32_t* idx;
  float* w;
};

template <typename TL, int EPL, bool SOFTMAX>
__global__ void __launch_bounds__(32 * kRows)
route_topk_kernel(const TopkArgs a) {
  __shared__ float s_sel[kRows][64];
  __shared__ float s_grp[kRows][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kRows + warp;
  if (t >= a.T) return;
  const TL* row = static_cast<const TL*>(a.logits) + (size_t)t * a.ld;
  float s[EPL], c[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    s[i] = e < a.E ? load_logit(row + e) : -INFINITY;
    if (!(s[i] > -INFINITY)) s[i] = -INFINITY;             // NaN counts as -inf
  }
  uint32_t live = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) live |= (s[i] > -INFINITY ? 1u : 0u) << i;
  if (SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) m = fmaxf(m, s[i]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (live >> i & 1u) sum += softmax_term(s[i], m);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      s[i] = live >> i & 1u ? __double2float_rn(__ddiv_rn(softmax_term(s[i], m), sum)) : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = live >> i & 1u ? sigmoid_score(s[i]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    c[i] = -INFINITY;
    if (live >> i & 1u) c[i] = a.bias ? __fadd_rn(s[i], a.bias[e]) : s[i];
    if (!(c[i] > -INFINITY)) c[i] = -INFINITY;             // a NaN bias takes its expert out
  }
  if (a.n_group > 1) drop_groups<EPL>(c, a.E, a.n_group, a.topk_group, lane, s_grp[warp]);
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = e >= a.E ? kKeyTaken : c[i] > -INFINITY ? order_key(c[i]) : kKeyOut;
  }
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) { best = key[i]; bi = i; }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? (unsigned)(lane + 32 * bi) : 0xffffffffu);
    if ((e & 31) == lane) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i == e >> 5) { v = top > kKeyOut ? s[i] : 0.f; key[i] = kKeyTaken; }
      s_sel[warp][j] = v;
      a.idx[(size_t)t * a.k + j] = e;
    }
  }
  __syncwarp();
  float den = 1.f;
  if (a.renorm) {
    float S = 0.f;
    for (int j = 0; j < a.k; ++j) S = __fadd_rn(S, s_sel[warp][j]);
    den = __fadd_rn(S, 1e-20f);
  }
  for (int j = lane; j < a.k; j += 32)
    a.w[(size_t)t * a.k + j] = __fmul_rn(__fdiv_rn(s_sel[warp][j], den), a.scale);
}

// ---------------------------------------------------------------------------
// Gradient of the logits.  With p_j = s_j / (S + eps), u_j = dw_j * scale and
// ubar = sum_j u_j p_j over the slots that carry a weight:
//   renormalised:  s_j ds_j = p_j (u_j - ubar)
//   otherwise:     s_j ds_j = s_j u_j
//   sigmoid:  dl_e = s_e ds_e (1 - s_e)              (chosen experts only)
//   softmax:  dl_e = s_e ds_e - s_e C,  C = sum_j s_j ds_j
// Renormalised, C = ubar (1 - sum p) = ubar eps / (S + eps): taken from that
// form, since the difference of the sums would be rounding noise.  The slots
// behind a masked row carry weight 0 and give no gradient.
// ---------------------------------------------------------------------------
struct TopkBwdArgs {
  const void* logits;
  long ld;
  const int32_t* idx;
  const float *w, *dw;
  int T, E, k, renorm;
  float scale;
  void* dl;
  long ldd;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <typename TL, int EPL, bool SOFTMAX>
__global__ void __launch_bounds__(32 * kRows)
route_topk_bwd_kernel(const TopkBwdArgs a) {
  extern __shared__ float s_row[];                     // [kRows][E]: s_e ds_e of the chosen experts
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kRows + warp;
  if (t >= a.T) return;
  float* g = s_row + (size_t)warp * a.E;
  const TL* row = static_cast<const TL*>(a.logits) + (size_t)t * a.ld;
  float l[EPL], m = 0.f, inv = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (lane + 32 * i < a.E) g[lane + 32 * i] = 0.f;
  if (SOFTMAX) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < a.E ? load_logit(row + e) : -INFINITY;
      m = fmaxf(m, l[i]);                              // fmaxf drops a NaN
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      l[i] = l[i] == m ? 1.f : l[i] > -INFINITY ? expf(l[i] - m) : 0.f;
      z += l[i];
    }
    z = warp_sum(z);
    inv = m > -INFINITY ? 1.f / z : 0.f;
  }
  // up to two slots per lane (k <= 64)
  float s[2], u[2], q[2];
  int e[2];
  float S = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 32 * h;
    s[h] = u[h] = q[h] = 0.f;
    e[h] = -1;
    if (j < a.k) {
      const size_t p = (size_t)t * a.k + j;
      const int x = a.idx[p];
      if (x >= 0 && x < a.E && a.w[p] != 0.f) {
        e[h] = x;
        u[h] = a.dw[p] * a.scale;
        const float lx = load_logit(row + x);
        if (SOFTMAX) {
          s[h] = (lx == m ? 1.f : expf(lx - m)) * inv;
        } else {
          // s and 1 - s, each without cancellation
          const float ex = expf(-fabsf(lx)), d = 1.f / (1.f + ex);
          s[h] = lx >= 0.f ? d : ex * d;
          q[h] = lx >= 0.f ? ex * d : d;
        }
      }
    }
    S += s[h];
  }
  float C = 0.f, ubar = 0.f;
  const float den = a.renorm ? warp_sum(S) + 1e-20f : 1.f;
  const float p0 = s[0] / den, p1 = s[1] / den;
  const float up = warp_sum(u[0] * p0 + u[1] * p1);
  if (a.renorm) { ubar = up; C = up * (1e-20f / den); } else { C = up; }
  __syncwarp();
  const float pp[2] = {p0, p1};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (e[h] >= 0) g[e[h]] = pp[h] * (u[h] - ubar) * (SOFTMAX ? 1.f : q[h]);
  __syncwarp();
  TL* out = static_cast<TL*>(a.dl) + (size_t)t * a.ldd;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int x = lane + 32 * i;
    if (x < a.E) store_val(out + x, SOFTMAX ? g[x] - l[i] * inv * C : g[x]);
  }
}

template <typename TL, bool SOFTMAX>
cudaError_t topk_launch(const TopkArgs& a, cudaStream_t st) {
  const int grid = ceil_div(a.T, kRows), epl = ceil_div(a.E, 32);
  if (epl <= 1) route_topk_kernel<TL, 1, SOFTMAX><<<grid, 32 * kRows, 0, st>>>(a);
  else if (epl <= 4) route_topk_kernel<TL, 4, SOFTMAX><<<grid, 32 * kRows, 0, st>>>(a);
  else if (epl <= 8) route_topk_kernel<TL, 8, SOFTMAX><<<grid, 32 * kRows, 0, st>>>(a);
  else if (epl <= 16) route_topk_kernel<TL, 16, SOFTMAX><<<grid, 32 * kRows, 0, st>>>(a);
  else route_topk_kernel<TL, 32, SOFTMAX><<<grid, 32 * kRows, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename TL, bool SOFTMAX>
cudaError_t topk_bwd_launch(const TopkBwdArgs& a, cudaStream_t st) {
  const int grid = ceil_div(a.T, kRows), epl = ceil_div(a.E, 32);
  const size_t sm = (size_t)kRows * a.E * sizeof(float);          // at most 32 KB
  if (epl <= 1) route_topk_bwd_kernel<TL, 1, SOFTMAX><<<grid, 32 * kRows, sm, st>>>(a);
  else if (epl <= 4) route_topk_bwd_kernel<TL, 4, SOFTMAX><<<grid, 32 * kRows, sm, st>>>(a);
  else if (epl <= 8) route_topk_bwd_kernel<TL, 8, SOFTMAX><<<grid, 32 * kRows, sm, st>>>(a);
  else if (epl <= 16) route_topk_bwd_kernel<TL, 16, SOFTMAX><<<grid, 32 * kRows, sm, st>>>(a);
  else route_topk_bwd_kernel<TL, 32, SOFTMAX><<<grid, 32 * kRows, sm, st>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Grouping: a stable counting sort of the pairs p = t k + j by expert.  Blocks
// of kPairs consecutive pairs count their experts, one block scans the counts
// of every (expert, block), and the blocks place their pairs.  A pair's rank
// among its block's pairs of the same expert is the number of such pairs in
// earlier warps (a column of s_cnt) plus those in lower lanes (match mask), so
// the order never depends on the order in which atomics arrive.  Pairs with an
// index outside [0, E) go nowhere: pos -1, and the tail of perm that they leave
// is -1 too.
// ---------------------------------------------------------------------------
constexpr int kPairs = 1024;

struct GroupArgs {
  const int32_t* idx;
  long P;
  int E, nblk;
  int32_t *counts, *offsets, *perm, *pos;
  int32_t* blk;                    // [E][nblk]: counts, then exclusive prefixes
};

__global__ void __launch_bounds__(kPairs)
group_count_kernel(const GroupArgs a) {
  extern __shared__ int32_t s_hist[];                  // [E]
  for (int e = threadIdx.x; e < a.E; e += kPairs) s_hist[e] = 0;
  __syncthreads();
  const long p = (long)blockIdx.x * kPairs + threadIdx.x;
  if (p < a.P) {
    const int e = a.idx[p];
    if (e >= 0 && e < a.E) atomicAdd(&s_hist[e], 1);
    else atomicOr(&g_group_err, DEV_ERR_INDEX);
    a.perm[p] = -1;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kPairs) a.blk[(size_t)e * a.nblk + blockIdx.x] = s_hist[e];
}

__global__ void __launch_bounds__(1024)
group_scan_kernel(const GroupArgs a) {
  __shared__ int s_tot[1024], s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = warp; e < a.E; e += 32) {
    int run = 0;
    for (int b0 = 0; b0 < a.nblk; b0 += 32) {
      const int b = b0 + lane;
      const int v = b < a.nblk ? a.blk[(size_t)e * a.nblk + b] : 0;
      int x = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (b < a.nblk) a.blk[(size_t)e * a.nblk + b] = run + x - v;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_tot[e] = run;
  }
  __syncthreads();
  const int e = threadIdx.x, v = e < a.E ? s_tot[e] : 0;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < warp; ++i) before += s_warp[i];
  if (e < a.E) { a.counts[e] = v; a.offsets[e + 1] = before + x; }
  if (e == 0) a.offsets[0] = 0;
}

__global__ void __launch_bounds__(kPairs)
group_place_kernel(const GroupArgs a) {
  extern __shared__ uint8_t s_cnt[];                   // [32 warps][E] pairs of a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < 8 * a.E; i += kPairs) reinterpret_cast<uint32_t*>(s_cnt)[i] = 0u;
  __syncthreads();
  const long p = (long)blockIdx.x * kPairs + threadIdx.x;
  int e = p < a.P ? a.idx[p] : -1;
  if (e >= a.E) e = -1;
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const int below = __popc(same & ((1u << lane) - 1u));
  if (e >= 0 && below == 0) s_cnt[warp * a.E + e] = (uint8_t)__popc(same);
  __syncthreads();
  if (p >= a.P) return;
  if (e < 0) { a.pos[p] = -1; return; }
  int q = a.offsets[e] + a.blk[(size_t)e * a.nblk + blockIdx.x] + below;
  for (int i = 0; i < warp; ++i) q += s_cnt[i * a.E + e];
  a.pos[p] = q;
  a.perm[q] = (int32_t)p;
}

}  // namespace

cudaError_t launch_route_topk(const void* logits, moe_dtype dt, long ld, const float* bias, int T,
                              int E, int k, moe_score score, int n_group, int topk_group,
                              int renorm, float scale, int32_t* idx, float* w, cudaStream_t st) {
  const TopkArgs a{logits, ld, bias, T, E, k, n_group, topk_group, renorm, scale, idx, w};
  if (dt == MOE_BF16)
    return score == MOE_SCORE_SOFTMAX ? topk_launch<__nv_bfloat16, true>(a, st)
                                      : topk_launch<__nv_bfloat16, false>(a, st);
  return score == MOE_SCORE_SOFTMAX ? topk_launch<float, true>(a, st)
                                    : topk_launch<float, false>(a, st);
}

cudaError_t launch_route_topk_bwd(const void* logits, moe_dtype dt, long ld, const int32_t* idx,
                                  const float* w, const float* dw, int T, int E, int k,
                                  moe_score score, int renorm, float scale, void* dl, long ldd,
                                  cudaStream_t st) {
  const TopkBwdArgs a{logits, ld, idx, w, dw, T, E, k, renorm, scale, dl, ldd};
  if (dt == MOE_BF16)
    return score == MOE_SCORE_SOFTMAX ? topk_bwd_launch<__nv_bfloat16, true>(a, st)
                                      : topk_bwd_launch<__nv_bfloat16, false>(a, st);
  return score == MOE_SCORE_SOFTMAX ? topk_bwd_launch<float, true>(a, st)
                                    : topk_bwd_launch<float, false>(a, st);
}

size_t route_group_workspace(long P, int E) { return (size_t)E * ceil_div(P, kPairs) * 4; }

cudaError_t launch_route_group(const int32_t* idx, long P, int E, int32_t* counts,
                               int32_t* offsets, int32_t* perm, int32_t* pos, void* ws,
                               cudaStream_t st) {
  const GroupArgs a{idx, P, E, ceil_div(P, kPairs), counts, offsets, perm, pos,
                    static_cast<int32_t*>(ws)};
  group_count_kernel<<<a.nblk, kPairs, (size_t)E * 4, st>>>(a);
  group_scan_kernel<<<1, 1024, 0, st>>>(a);
  group_place_kernel<<<a.nblk, kPairs, (size_t)E * 32, st>>>(a);
  return cudaGetLastError();
}

cudaError_t route_group_take_error(int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_group_err, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && *word) e = cudaMemcpyToSymbol(g_group_err, &zero, sizeof(int));
  return e;
}

}  // namespace lmoe
