// Stand-alone routing: top-k experts of given router logits, the gradient of
// the logits, and the grouping of the chosen pairs by expert.
//
// Forward, one row of logits l[E] with selection bias b[E]:
//   s_e = 1 / (1 + exp(-l_e))            or   exp(l_e - m) / sum_i exp(l_i - m)
//   c_e = s_e + b_e                      (both fp32; s evaluated in fp64, rounded once)
//   groups: E / n_group consecutive experts, scored by the fp32 sum of their two
//           largest c, -inf without two eligible experts; the topk_group best
//           stay eligible (ties: lower group)
//   idx = the k eligible experts of largest c (ties: lower expert)
//   w_j = s_idx / (sum s_idx + 1e-20) * scale     or   s_idx * scale
// A logit of -inf or NaN takes its expert out: score 0, never eligible.  Slots
// that no eligible expert is left for take the lowest experts not yet taken,
// with weight 0, so every row names k different experts in range.
//
// Why fp64 scores: selection compares neighbouring values, and an fp32 sigmoid
// or softmax is off by several units in the last place, enough to swap them.
#include <float.h>

#include "common.cuh"
#include "kernels.h"
#include "router_math.cuh"

namespace lmoe {

namespace {

__device__ int g_group_err;            // DEV_ERR_INDEX: an expert index out of range

constexpr int kRows = 8;               // rows (warps) per CTA, at most
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// The layer's sigmoid without its clamp at +-80: beyond +-110 the fp32 result
// is 1 or 0 anyway, and inside +-80 the bits are the layer's.
__device__ __forceinline__ float sigmoid_score(float l) {
  const double a = -fmin(fmax((double)l, -110.0), 110.0);
  return __double2float_rn(__ddiv_rn(1.0, __dadd_rn(1.0, exp_fixed(a))));
}

// exp(l - m) in fp64 for l <= m: a = n ln 2 + r, |r| <= ln 2 / 2, and the Taylor
// polynomial of degree 13 (truncated below 2^-57).  Below -700 the quotient by
// the sum rounds to 0 in fp32; l == m covers rows whose maximum is +inf.
__device__ __forceinline__ double softmax_term(float l, float m) {
  if (l == m) return 1.0;
  const double a = fmax((double)l - (double)m, -700.0);
  const double n = rint(a * 0x1.71547652b82fep+0);
  const double r = fma(n, -0x1.a39ef35793c76p-33, fma(n, -0x1.62e42fee00000p-1, a));
  double p = 1.0 / 6227020800.0;
  p = fma(p, r, 1.0 / 479001600.0);
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return p * __longlong_as_double((long long)((int)n + 1023) << 52);
}

__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);        // -0 orders as +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// Keys order as choice scores do; experts out of the selection and experts
// already taken come below every score.
constexpr uint32_t kKeyOut = 1u, kKeyTaken = 0u;

__device__ __forceinline__ float rcp_approx(float v) {     // within 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
  return v;
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

// The two largest of each group of G consecutive experts, added: lane g returns
// the sums of groups g and g + 32.  A group without a second eligible expert has
// -inf, whatever the first is: +inf (by its bias) - inf would be a NaN, which
// counts neither as better nor as worse than the other groups.  c goes through
// shared memory, a group's stretch starting G | 1 floats behind the last one's (an
// odd stride, so lanes reading their own groups meet no bank conflicts).
template <int EPL>
__device__ __forceinline__ void group_sums(const float (&c)[EPL], int E, int n_group, int lane,
                                           float* buf, float (&sum)[2]) {
  const int G = E / n_group, st = G | 1;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    if (e < E) buf[e / G * st + e % G] = c[i];
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float m0 = -INFINITY, m1 = -INFINITY;
    if (lane + 32 * h < n_group)
      for (int j = 0; j < G; ++j) {
        const float v = buf[(lane + 32 * h) * st + j];
        m1 = fmaxf(m1, fminf(m0, v));
        m0 = fmaxf(m0, v);
      }
    sum[h] = m1 > -INFINITY ? __fadd_rn(m0, m1) : -INFINITY;
  }
  __syncwarp();
}

// bit mask of the topk_group best groups (ties: lower group)
__device__ __forceinline__ uint64_t best_groups(const float (&sum)[2], int n_group, int topk_group, int lane) {
  int r0 = 0, r1 = 0;
  for (int o = 0; o < n_group; ++o) {
    const float v = __shfl_sync(kAll, o < 32 ? sum[0] : sum[1], o & 31);
    r0 += v > sum[0] || (v == sum[0] && o < lane);
    r1 += v > sum[1] || (v == sum[1] && o < lane + 32);
  }
  const unsigned k0 = __ballot_sync(kAll, lane < n_group && r0 < topk_group);
  const unsigned k1 = __ballot_sync(kAll, lane + 32 < n_group && r1 < topk_group);
  return (uint64_t)k1 << 32 | k0;
}

// The weights of one row from its scores in slot order; sel is zero from slot k
// to the next multiple of 4.
__device__ __forceinline__ void write_weights(const TopkArgs& a, long t, const float* sel, int lane) {
  float den = 1.f;
  if (a.renorm) {
    float S = 0.f;
    for (int j = 0; j < a.k; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(sel + j);
      S = __fadd_rn(__fadd_rn(__fadd_rn(__fadd_rn(S, v.x), v.y), v.z), v.w);
    }
    den = __fadd_rn(S, 1e-20f);
  }
  for (int j = lane; j < a.k; j += 32) {
    const float v = a.renorm ? __fdiv_rn(sel[j], den) : sel[j];
    a.w[t * a.k + j] = __fmul_rn(v, a.scale);
  }
}

// One row, every score evaluated exactly and k rounds of a warp arg-max: rows
// that the quick way cannot decide (more than 32 experts next to the border,
// fewer eligible experts than slots, k > 32, groups whose order the bounds
// leave open).  16384 x 512: 123 us where all logits are equal, 176 with k = 40.
template <typename TL, int EPL, bool SOFTMAX>
__device__ __noinline__ void select_exact(const TopkArgs& a, long t, int lane, float* sel, float* buf) {
  const TL* row = static_cast<const TL*>(a.logits) + (size_t)t * a.ld;
  float s[EPL], c[EPL];
  uint32_t live = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    s[i] = e < a.E ? load_logit(row + e) : -INFINITY;
    live |= (s[i] > -INFINITY ? 1u : 0u) << i;               // NaN is out as well
  }
  if (SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) m = fmaxf(m, s[i]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (live >> i & 1u) sum += softmax_term(s[i], m);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      s[i] = live >> i & 1u ? __double2float_rn(__ddiv_rn(softmax_term(s[i], m), sum)) : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = live >> i & 1u ? sigmoid_score(s[i]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    c[i] = -INFINITY;
    if (live >> i & 1u) c[i] = a.bias ? __fadd_rn(s[i], a.bias[lane + 32 * i]) : s[i];
    if (!(c[i] > -INFINITY)) c[i] = -INFINITY;               // a NaN bias takes its expert out
  }
  if (a.n_group > 1) {
    float gs[2];
    group_sums<EPL>(c, a.E, a.n_group, lane, buf, gs);
    const uint64_t keep = best_groups(gs, a.n_group, a.topk_group, lane);
    const int G = a.E / a.n_group;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && !(keep >> (e / G) & 1)) c[i] = -INFINITY;
    }
  }
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    key[i] = lane + 32 * i >= a.E ? kKeyTaken : c[i] > -INFINITY ? order_key(c[i]) : kKeyOut;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) { best = key[i]; bi = i; }
    const uint32_t top = __reduce_max_sync(kAll, best);
    const int e = (int)__reduce_min_sync(kAll, best == top ? (unsigned)(lane + 32 * bi) : kAll);
    if ((e & 31) == lane) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i == e >> 5) { v = top > kKeyOut ? s[i] : 0.f; key[i] = kKeyTaken; }
      sel[j] = v;
      a.idx[t * a.k + j] = e;
    }
  }
  if (lane < 3 && a.k + lane < 64) sel[a.k + lane] = 0.f;
  __syncwarp();
  write_weights(a, t, sel, lane);
}

// A row per warp.  Exact scores of all experts are not needed to find the top k:
// an order value c~ per expert, within d of a value that orders as the choice
// scores do, leaves only the experts next to the border open.
//   1. c~ = s~ + b from fp32 arithmetic; for softmax without a bias the logit
//      itself (the score rises with it)
//   2. tau that at least k experts reach (c~ >= tau), by bisection between the
//      smallest lane maximum, which 32 experts reach, and the largest value (1 to 5
//      steps; from fp32's lowest value, where a lane has no eligible expert, about
//      130: 160 experts 21 us, of which 3 of 8 groups are kept 83).  An expert of
//      c~ < tau - 2 d is beaten by k others
//   3. the rest, at most 32, one per lane: exact score in fp64, rank by counting
//      (score descending, expert ascending), slot = rank
// so a row costs one fp64 score per lane and not E / 32.
//
// Bounds.  Sigmoid: the argument of ex2.approx, |l| log2 e in fp32, is off by
// half a unit and by the constant's rounding, together 1.2e-6 of the exponential
// at |l| = 16 and 4.9e-6 at 80; ex2.approx, the sum and the quotient add 4.1e-7:
// s~ is within kappa s, kappa = 2^-19 up to 16 and 2^-17 up to 80.  Below -80 the
// argument stays there: s and s~ are under 2e-35.  Softmax has its exponentials
// from fp64, for the sum: four fp32 roundings, kappa = 2^-21.  The roundings of
// c~, s and c are 2^-24 of |c| and s each, so d = kappa (2 max s + max |b|) + 1e-34
// covers every expert.  Logits as order values: scores whose logits differ by
// 2^-20 differ by 2^-20 of themselves and round to different fp32 numbers while
// they are normal, which holds for l - m > -80 (a sum of at most 1024).
//
// A row takes about 1200 warp instructions at 512 experts (issue slots 68 % taken,
// the rest waits of dependent ones): 16384 x 512, k = 22, 30 us, against 92 us for fp64
// scores of all experts and k arg-max rounds.
// FULL: E == 32 EPL, no lane has an index past the row.
template <typename TL, int EPL, bool SOFTMAX, bool FULL>
__global__ void __launch_bounds__(32 * kRows, EPL <= 8 ? 5 : EPL == 16 ? 4 : 2)
route_topk_kernel(const TopkArgs a) {
  extern __shared__ float s_dyn[];
  __shared__ __align__(16) float s_sel[kRows][64];
  __shared__ __align__(16) uint64_t s_key[kRows][32];
  let_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  float* buf = s_dyn + (size_t)warp * (a.E + 64);          // n_group > 1 only
  float* sel = s_sel[warp];
  uint64_t* keys = s_key[warp];
  auto in = [&](int i) { return FULL || lane + 32 * i < a.E; };
  float b[EPL], bmax = 0.f;
  bool odd = false;                                        // a NaN or -inf bias
  const bool by_logit = SOFTMAX && !a.bias && a.n_group == 1;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    b[i] = a.bias && in(i) ? a.bias[lane + 32 * i] : 0.f;
    if (b[i] > -INFINITY) bmax = fmaxf(bmax, fabsf(b[i]));   // an expert out by its bias has no say
    else odd = true;
  }
  bmax = warp_max(bmax);
  odd = __any_sync(kAll, odd);

  for (long t = (long)blockIdx.x * warps + warp; t < a.T; t += (long)gridDim.x * warps) {
    const TL* row = static_cast<const TL*>(a.logits) + (size_t)t * a.ld;
    float c[EPL];                                          // -inf: not eligible
    float m = -INFINITY, d;
    double sum = 1.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = in(i) ? load_logit(row + lane + 32 * i) : -INFINITY;
    if (SOFTMAX) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) m = fmaxf(m, c[i]);
      m = warp_max(m);
      sum = 0.0;
      if (by_logit) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          if (c[i] > -INFINITY) sum += softmax_term(c[i], m);
          else c[i] = -INFINITY;                           // NaN
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
        d = 0x1p-21f;
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const double e = c[i] > -INFINITY ? softmax_term(c[i], m) : 0.0;
          c[i] = c[i] > -INFINITY ? (float)e : -INFINITY;
          sum += e;
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
        const float inv = 1.f / (float)sum;                // the largest score as well
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = fmaf(c[i], inv, b[i]);
        d = 0x1p-21f * (2.f * inv + bmax) + 1e-34f;
      }
    } else {
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float l = c[i], x = fmaxf(l, -80.f);
        big = fmaxf(big, fabsf(x));
        c[i] = l > -INFINITY ? rcp_approx(1.f + __expf(-x)) + b[i] : -INFINITY;
      }
      d = (__any_sync(kAll, big > 16.f) ? 0x1p-17f : 0x1p-19f) * (2.f + bmax) + 1e-34f;
    }
    if (odd) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!(c[i] > -INFINITY)) c[i] = -INFINITY;
    }
    bool open = !(d < INFINITY) || a.k > 32;               // an infinite bias
    if (a.n_group > 1) {
      float gs[2];
      group_sums<EPL>(c, a.E, a.n_group, lane, buf, gs);
      const uint64_t keep = best_groups(gs, a.n_group, a.topk_group, lane);
      // the worst kept and the best dropped group have to differ by more than
      // twice the error of a sum of two scores, whose rounding d covers too
      float kept = INFINITY, dropped = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < a.n_group) {
          if (keep >> (lane + 32 * h) & 1) kept = fminf(kept, gs[h]);
          else dropped = fmaxf(dropped, gs[h]);
        }
      kept = -warp_max(-kept);
      dropped = warp_max(dropped);
      open |= a.topk_group < a.n_group && !(kept - dropped > 8.f * d);
      const int G = a.E / a.n_group;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        if (in(i) && !(keep >> (e / G) & 1)) c[i] = -INFINITY;
      }
    }
    float top = -INFINITY, low = INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      top = fmaxf(top, c[i]);
      if (in(i)) low = fminf(low, c[i]);
    }
    int n = a.E;                                           // eligible experts
    if (!__all_sync(kAll, low > -INFINITY)) {
      n = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) n += c[i] > -INFINITY;
      n = __reduce_add_sync(kAll, n);
    }
    open |= n < a.k;
    float cut = -FLT_MAX;                                  // candidates: c >= cut
    if (!open && n > 32) {
      // a lane without an eligible expert: start at fp32's lowest value
      float lo = fmaxf(-warp_max(-top), -FLT_MAX), hi = warp_max(top);
      while (true) {
        // raise lo: to the middle, or down towards it while fewer than k reach
        // that, until at most 32 experts are left above it
        bool moved = false;
        while (true) {
          const float x = 0.5f * lo + 0.5f * hi;
          if (!(x > lo && x < hi)) break;
          int r = 0;
#pragma unroll
          for (int i = 0; i < EPL; ++i) r += c[i] >= x;
          r = __reduce_add_sync(kAll, r);
          if (r < a.k) { hi = x; continue; }
          lo = x;
          moved = true;
          if (r <= 32) break;
        }
        cut = lo - 2.f * d;
        n = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) n += c[i] >= cut;
        n = __reduce_add_sync(kAll, n);
        if (n <= 32) {
          open = by_logit && lo - m < -80.f;
          break;
        }
        if (!moved) { open = true; break; }
      }
    } else if (by_logit) {
      open |= __any_sync(kAll, low > -INFINITY && low - m < -80.f);
    }
    if (open) {
      select_exact<TL, EPL, SOFTMAX>(a, t, lane, sel, buf);
      __syncwarp();
      continue;
    }
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) mask |= (c[i] >= cut ? 1u : 0u) << i;
    const int own = __popc(mask);
    int at = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kAll, at, off);
      if (lane >= off) at += v;
    }
    at -= own;
    int* cand = reinterpret_cast<int*>(sel);
    for (; mask; mask &= mask - 1) cand[at++] = lane + 32 * (__ffs(mask) - 1);
    __syncwarp();
    const int e = cand[lane < n ? lane : 0];
    float s = 0.f;
    uint64_t key = 0;
    if (lane < n) {
      const float l = load_logit(row + e);
      s = SOFTMAX ? __double2float_rn(__ddiv_rn(softmax_term(l, m), sum)) : sigmoid_score(l);
      const float v = a.bias ? __fadd_rn(s, a.bias[e]) : s;
      key = (uint64_t)order_key(v) << 32 | (uint32_t)(0xffff - e);
    }
    keys[lane] = key;                                      // 0, below all, past n
    __syncwarp();
    int rank = 0;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(keys + j);
      rank += v.x > key;
      rank += v.y > key;
    }
    if (lane < n && rank < a.k) {
      sel[rank] = s;
      a.idx[t * a.k + rank] = e;
    }
    if (lane < 3 && a.k + lane < 64) sel[a.k + lane] = 0.f;
    __syncwarp();
    write_weights(a, t, sel, lane);
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// Gradient of the logits.  With p_j = s_j / (S + eps), u_j = dw_j * scale and
// C = sum_j u_j p_j over the slots that carry a weight (p = s where the weights
// are not renormalised):
//   sigmoid:  dl_e = p_e (u_e - C) (1 - s_e), renormalised; s_e u_e (1 - s_e)
//   softmax:  dl_e = p_e (u_e - C) - s_e C eps / (S + eps), renormalised;
//             s_e (u_e - C)                              (u_e = 0 if not chosen)
// Where one slot has nearly all of the weight, u_e - C by itself is the rounding
// of C.  With u* of the slot of the largest p and r = 1 - sum p (eps / (S + eps),
// or the softmax's mass outside the slots, added up as such)
//   u_e - C = (u_e - u*) + B,   B = u* r - sum_j p_j (u_j - u*),
// whose terms are as small as the result.  That form costs a maximum and, for
// the mass outside the slots, a pass over the row in shared memory: 16384 x 512,
// k 22, softmax 18.6 -> 22.7 us, sigmoid renormalised 10.5 -> 12.1; 8192 x 128
// bf16 is as fast (8.3).  The arithmetic is fp32: scores and gradients are off by
// a few units of their own terms.  The slots behind a masked row carry weight 0
// and give no gradient.
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
  extern __shared__ float s_row[];                     // [kRows][E]: gradients of the chosen experts
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long t = (long)blockIdx.x * kRows + warp;      // the last block's may pass 2^31
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
  // the slot of the largest score (scores are not negative: they order as their bits do)
  const unsigned big = __float_as_uint(fmaxf(s[0], s[1])), most = __reduce_max_sync(kAll, big);
  const float top = __shfl_sync(kAll, __float_as_uint(s[0]) == big ? u[0] : u[1],
                                __ffs(__ballot_sync(kAll, big == most)) - 1);
  const float den = a.renorm ? warp_sum(S) + 1e-20f : 1.f;
  const float p[2] = {s[0] / den, s[1] / den};
  float B = 0.f, C = 0.f;                              // C: what the softmax's experts lose a score
  if (SOFTMAX || a.renorm) {
    float rest = 1e-20f / den;
    if (SOFTMAX && !a.renorm) {
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (e[h] >= 0) g[e[h]] = 1.f;
      __syncwarp();
      rest = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {                  // a chosen expert's score is out of l
        if (lane + 32 * i < a.E && g[lane + 32 * i] != 0.f) l[i] = 0.f;
        rest += l[i];
      }
      rest = warp_sum(rest) * inv;
    }
    B = top * rest - warp_sum(p[0] * (u[0] - top) + p[1] * (u[1] - top));
    C = (top - B) * (a.renorm ? rest : 1.f);
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (e[h] >= 0) g[e[h]] = p[h] * (SOFTMAX || a.renorm ? (u[h] - top) + B : u[h]) * (SOFTMAX ? 1.f : q[h]);
  __syncwarp();
  TL* out = static_cast<TL*>(a.dl) + (size_t)t * a.ldd;
  C *= inv;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int x = lane + 32 * i;
    if (x < a.E) store_val(out + x, SOFTMAX ? fmaf(-l[i], C, g[x]) : g[x]);
  }
}

template <typename TL, int EPL, bool SOFTMAX>
cudaError_t topk_epl(const TopkArgs& a, cudaStream_t st) {
  // few rows: one warp per CTA, so that each has an SM's issue slots to itself
  const int warps = a.T >= 2048 ? kRows : a.T >= 512 ? 4 : 1;
  const int need = ceil_div(a.T, warps), grid = need < 148 * 8 ? need : 148 * 8;
  const size_t sm = a.n_group > 1 ? (size_t)warps * (a.E + 64) * 4 : 0;      // at most 34 KB
  if (a.E == 32 * EPL) route_topk_kernel<TL, EPL, SOFTMAX, true><<<grid, 32 * warps, sm, st>>>(a);
  else route_topk_kernel<TL, EPL, SOFTMAX, false><<<grid, 32 * warps, sm, st>>>(a);
  return cudaGetLastError();
}

template <typename TL, bool SOFTMAX>
cudaError_t topk_launch(const TopkArgs& a, cudaStream_t st) {
  const int epl = ceil_div(a.E, 32);
  return epl <= 1 ? topk_epl<TL, 1, SOFTMAX>(a, st) : epl <= 4 ? topk_epl<TL, 4, SOFTMAX>(a, st)
       : epl <= 8 ? topk_epl<TL, 8, SOFTMAX>(a, st) : epl <= 16 ? topk_epl<TL, 16, SOFTMAX>(a, st)
                                                    : topk_epl<TL, 32, SOFTMAX>(a, st);
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
// of kPairs consecutive pairs count their experts, a warp per expert scans its
// counts over the blocks, and the blocks place their pairs.  A pair's rank
// among its block's pairs of the same expert is the number of such pairs in
// earlier warps (a column of s_cnt) plus those in lower lanes (match mask), so
// the order never depends on the order in which atomics arrive.  Pairs with an
// index outside [0, E) go nowhere: pos -1, and the tail of perm that they leave
// is -1 too.
// ---------------------------------------------------------------------------
constexpr int kPairs = 1024, kPairWarps = kPairs / 32;

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
  let_next();
  after_previous();
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

// a warp per expert: its counts over the blocks become exclusive prefixes
__global__ void __launch_bounds__(256)
group_scan_kernel(const GroupArgs a) {
  const int lane = threadIdx.x & 31, e = blockIdx.x * 8 + (threadIdx.x >> 5);
  let_next();
  after_previous();
  if (e >= a.E) return;
  int32_t* c = a.blk + (size_t)e * a.nblk;
  int run = 0;
  for (int b0 = 0; b0 < a.nblk; b0 += 32) {
    const int b = b0 + lane;
    const int v = b < a.nblk ? c[b] : 0;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (b < a.nblk) c[b] = run + x - v;
    run += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) a.counts[e] = run;
}

// exclusive prefix of v over the block's 1024 threads
__device__ __forceinline__ int block_prefix(int v, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = lane < warp ? s_warp[lane] : 0;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
  return before + x - v;
}

// places a block's pairs; every block adds up the experts' counts for itself,
// the first writes them out as offsets
__global__ void __launch_bounds__(kPairs)
group_place_kernel(const GroupArgs a) {
  extern __shared__ uint16_t s_cnt[];                  // [kPairWarps][E] pairs of a warp, then before it
  __shared__ int s_base[1024], s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kPairWarps / 2 * a.E; i += kPairs) reinterpret_cast<uint32_t*>(s_cnt)[i] = 0u;
  let_next();
  after_previous();
  const int c = threadIdx.x < a.E ? a.counts[threadIdx.x] : 0;
  const int off = block_prefix(c, s_warp);             // (a barrier: s_cnt is cleared)
  if (threadIdx.x < a.E) {
    s_base[threadIdx.x] = off + a.blk[(size_t)threadIdx.x * a.nblk + blockIdx.x];
    if (blockIdx.x == 0) {
      a.offsets[threadIdx.x] = off;
      if (threadIdx.x == a.E - 1) a.offsets[a.E] = off + c;
    }
  }
  const long p = (long)blockIdx.x * kPairs + threadIdx.x;
  int e = p < a.P ? a.idx[p] : -1;
  if (e >= a.E) e = -1;
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const int below = __popc(same & ((1u << lane) - 1u));
  if (e >= 0 && below == 0) s_cnt[warp * a.E + e] = (uint16_t)__popc(same);
  __syncthreads();
  // a column per thread: the pairs of its expert in earlier warps
  if (threadIdx.x < a.E) {
    int run = 0;
#pragma unroll 8
    for (int i = 0; i < kPairWarps; ++i) {
      const int v = s_cnt[i * a.E + threadIdx.x];
      s_cnt[i * a.E + threadIdx.x] = (uint16_t)run;
      run += v;
    }
  }
  __syncthreads();
  if (p >= a.P) return;
  if (e < 0) { a.pos[p] = -1; return; }
  const int q = s_base[e] + s_cnt[warp * a.E + e] + below;
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
  cudaError_t e = launch_early(group_count_kernel, a.nblk, kPairs, (size_t)E * 4, st, a);
  if (e == cudaSuccess) e = launch_early(group_scan_kernel, ceil_div(E, 8), 256, 0, st, a);
  const size_t sm = (size_t)E * kPairWarps * 2;               // at most 64 KB
  if (e == cudaSuccess && sm > 48 * 1024 - 4500)
    e = cudaFuncSetAttribute(group_place_kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
  return e == cudaSuccess ? launch_early(group_place_kernel, a.nblk, kPairs, sm, st, a) : e;
}

cudaError_t route_group_take_error(int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_group_err, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && *word) e = cudaMemcpyToSymbol(g_group_err, &zero, sizeof(int));
  return e;
}

}  // namespace lmoe
