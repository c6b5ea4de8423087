// Products of E4M3 operands with one fp32 scale for each block of 128 along K:
//   out[m, n] = sum_kb sa[kb][m] sb[kb][n] sum_{k in block kb} a[m, k] b[n, k]
// a: activations (a scale per row and K block).  b: weights with a scale per
// 128 x 128 block, or a second matrix of the first kind (the weight gradient).
// Rows of a may be grouped, group g taking weight matrix g.
//
// The inner sum of 128 products is one tcgen05 accumulation (kind::f8f6f4, four
// K = 32 MMAs) into one of a ring of TMEM buffers.  The tensor core cannot apply
// an fp32 scale, so "promoting" warps read every 128-K partial back and add
// scale * partial to fp32 registers (packed pairs) while the tensor core fills
// the other buffers.  Per 128-K step of a pair's 256 x 256 tile the MMAs take 512
// cycles and each SM's 32768 FMAs 256, so the promotion hides behind the products.
//
// Two forms of the tile:
//   wide  an SM pair's 256 activation rows x 256 weight rows; a thread owns one
//         activation row, and its scale product is one number for each 128
//         columns (per column in the weight gradient, where it owns four rows and
//         a quarter of the columns).  8192 x 10240 x 8192:
//         620 us, 2.2 PFLOP/s, in a short run; under steady load, where the clock
//         falls (power), about 720 us, 1.9 PFLOP/s, and the promotion's TMEM reads
//         and FMAs share it with the products.
//   tall  MMA rows = 128 weight rows, MMA columns = 16..64 activation rows: for
//         few rows, where streaming the weights is the work.  Two CTAs per SM
//         keep more loads in flight; when the tiles cannot fill the GPU, K is
//         split over the CTAs of a cluster, which add their sums in rank order
//         through distributed shared memory (no atomics: one order).
//         64 x 10240 x 8192 with cold weights: 21.4 us, 4.0 TB/s; 8 rows 17.2, 4.9.
//
// Roles: a producer thread (TMA tiles), a warp that lays scale products into a
// ring of their own (the promotion reads them after the tile's stage is free
// again; the wide form's row scales are read by the promoting threads), two MMA
// threads, 4 (tall) or 8 promoting warps.  Scales are read by ordinary loads: the
// kernel may start while the one that writes them still runs, so they are not
// constant for its whole life, which a non-coherent load would ask for.  Every wait
// is bounded; one that runs out sets DEV_ERR_TIMEOUT, and its whole warp unwinds.
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "pair_sm100.cuh"
#include "sm100.cuh"

namespace lmoe {

namespace {

using namespace sm100;

__device__ int g_fp8_err;

constexpr int kRowsP = 128;               // MMA rows of a tile
constexpr int kKB = 128;                  // K elements (bytes) per step
constexpr int kPBytes = kRowsP * kKB;
constexpr int kMaxGroups = 1024;

struct Fp8Args {
  const float* sa;          // [KB][ldsa]
  long ldsa;
  const float* sb;          // block scales [G][NB][KB], or [KB][ldsb]
  long ldsb;
  const int32_t* offsets;   // [G + 1] or NULL
  void* out;
  long ldo;
  int M, N, KB, G, NB;
  int split;                // CTAs per tile (cluster size), TALL only
  int vec;                  // out rows start on 16 bytes and are whole 16 bytes (TMA stores)
};

__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate));
}

// fp32 accumulator, E4M3 operands (format 0), both K-major
__device__ __forceinline__ uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 32 lanes x 64 columns as fragments: thread t gets, for each group i of 8 columns
// and lane t / 4 + 8 n, columns 8 i + 2 (t % 4) and + 1 in r[n / 2][4 i + 2 (n % 2)]
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[2][32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=r"(r[h][0]), "=r"(r[h][1]), "=r"(r[h][2]), "=r"(r[h][3]), "=r"(r[h][4]), "=r"(r[h][5]),
          "=r"(r[h][6]), "=r"(r[h][7]), "=r"(r[h][8]), "=r"(r[h][9]), "=r"(r[h][10]), "=r"(r[h][11]),
          "=r"(r[h][12]), "=r"(r[h][13]), "=r"(r[h][14]), "=r"(r[h][15]), "=r"(r[h][16]),
          "=r"(r[h][17]), "=r"(r[h][18]), "=r"(r[h][19]), "=r"(r[h][20]), "=r"(r[h][21]),
          "=r"(r[h][22]), "=r"(r[h][23]), "=r"(r[h][24]), "=r"(r[h][25]), "=r"(r[h][26]),
          "=r"(r[h][27]), "=r"(r[h][28]), "=r"(r[h][29]), "=r"(r[h][30]), "=r"(r[h][31])
        : "r"(taddr + ((uint32_t)(16 * h) << 16)));
}

// Arrival on a barrier of either CTA of the pair, for hand-overs of TMEM alone:
// what it orders are this warp's finished TMEM reads (tcgen05.wait::ld and the
// fence before it), so no memory has to become visible to the other SM.  The
// cluster-scope release form costs about 1300 cycles per arrival.
__device__ __forceinline__ void arrive_tmem(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// a staged box of 32 rows x 128 bytes to the output matrix; columns past its
// width are not written
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

constexpr int kScaleSteps = 4;             // steps per slot of the tall form's scale ring

template <int NT>
struct TCfg {
  static constexpr int kQBytes = NT * kKB;
  static constexpr int kStageBytes = kPBytes + kQBytes;
  static constexpr int kStages = NT <= 32 ? 5 : 4;              // two CTAs share an SM: its shared
  static constexpr int kBufs = 4;                               // memory, and its 512 TMEM columns,
  static constexpr int kSlots = 3;                              // for the partial sums
  static constexpr int kWarps = 4;                              // promoting warps (64 rows: eight of
                                                                // 80 registers were 9 % slower)
  static constexpr int kThreads = 128 + 32 * kWarps;
  static constexpr int kStepFloats = NT;                        // the columns' scale products
  static constexpr uint32_t kTmemCols = kBufs * NT;
  // The promotion waits on a stage's `done`, which completes again when the stage
  // is used again: the MMAs must not get that far ahead of it, and what holds
  // them back is the number of buffers.
  static_assert(kBufs <= kStages, "a done phase could pass unseen");
  static constexpr int kScaleOffset = kStages * kStageBytes;
  static constexpr int kBarOffset = kScaleOffset + kSlots * kScaleSteps * kStepFloats * 4;
  static constexpr int kTableOffset = kBarOffset + 512;
  static constexpr int bytes(int groups) {         // groups: 0 for a plain product
    return kTableOffset + (groups ? 2 * (groups + 1) * 4 : 0) + 1024;
  }
};

// A wait of a whole warp: every lane gets the same answer, so that a wait that ran
// out is left by all of them (the tcgen05 loads that follow need the whole warp).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ bool warp_aborted(const volatile int* flag) {
  return __any_sync(0xffffffffu, *flag != 0);
}

struct Tile {
  int grp;
  int m0, rows;      // activation rows [m0, m0 + rows)
  int n0, cols;      // weight rows [n0, n0 + cols) of the group's matrix
};

// Tile t: the weight blocks of a group run fastest over its row tiles, so that
// the CTAs in flight share weight blocks and row tiles through L2.
template <int RM, int RN>
__device__ __forceinline__ bool decode(const Fp8Args& a, const int* s_tiles, const int* s_off, int t,
                                       Tile& o) {
  const int nn = (a.N + RN - 1) / RN;
  int lo = 0, base = 0, cnt = a.M;
  if (a.offsets) {
    int hi = a.G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_tiles[mid] <= t) lo = mid; else hi = mid;
    }
    base = s_off[lo];
    cnt = s_off[lo + 1] - base;
    t -= s_tiles[lo];
  }
  const int nm = (cnt + RM - 1) / RM;
  if (nm <= 0) return false;
  int im, in;
  if (RM < 256) {
    in = t / nm; im = t - in * nm;
  } else {
    // bands of 8 row tiles: a wave's tiles form a block, not a strip
    const int band = t / (8 * nn), left = nm - band * 8, h = left < 8 ? left : 8;
    const int u = t - band * 8 * nn;
    in = u / h; im = band * 8 + u - in * h;
  }
  if (in >= nn || im >= nm) return false;
  o.grp = lo;
  o.m0 = base + im * RM;
  o.rows = min(RM, cnt - im * RM);
  o.n0 = in * RN;
  o.cols = min(RN, a.N - in * RN);
  return true;
}

// tile offsets [G + 1] and row offsets [G + 1] of the groups.  Offsets are
// clamped to [0, M] and made ascending, so that whatever the caller's array
// holds, every tile lies inside a, b and out.
template <int RM, int RN>
__device__ void load_groups(const Fp8Args& a, int* s_tiles, int* s_off) {
  if (!a.offsets) return;
  const int nn = (a.N + RN - 1) / RN;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int top = 0, tiles = 0;
    for (int g0 = 0; g0 <= a.G; g0 += 32) {
      const int g = g0 + lane;
      int v = g <= a.G ? min(max(a.offsets[g], 0), a.M) : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v = max(v, y);
      }
      v = max(v, top);
      int prev = __shfl_up_sync(0xffffffffu, v, 1);
      if (lane == 0) prev = g0 == 0 ? v : top;
      // tiles of group g - 1 lie before tile offset g
      int n = g <= a.G && g > 0 ? (v - prev + RM - 1) / RM * nn : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, n, off);
        if (lane >= off) n += y;
      }
      if (g <= a.G) { s_off[g] = v; s_tiles[g] = tiles + n; }
      tiles += __shfl_sync(0xffffffffu, n, 31);
      top = __shfl_sync(0xffffffffu, v, 31);
    }
  }
}

template <int NT, typename TO>
__global__ void __launch_bounds__(TCfg<NT>::kThreads, 2)
fp8_tall_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                const Fp8Args a, const int n_tiles) {
  using C = TCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_scale = reinterpret_cast<float*>(smem + C::kScaleOffset);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* done = full + C::kStages;             // a step's products are finished
  uint64_t* sfull = done + C::kStages;
  uint64_t* sempty = sfull + C::kSlots;
  uint64_t* tempty = sempty + C::kSlots;
  uint64_t* mma_done = tempty + C::kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_tiles = reinterpret_cast<int*>(smem + C::kTableOffset);
  int* s_off = s_tiles + a.G + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = a.split;
  const uint32_t rank = split > 1 ? pair2::cluster_rank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&done[s], 1); }
    for (int s = 0; s < C::kSlots; ++s) { mbar_init(&sfull[s], 32); mbar_init(&sempty[s], C::kWarps); }
    for (int b = 0; b < C::kBufs; ++b) mbar_init(&tempty[b], C::kWarps);
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&amap);
    tma_prefetch_desc(&bmap);
  }
  if (warp == 1) { tmem_alloc(tmem_slot, C::kTmemCols); tmem_relinquish(); }
  let_next();
  after_previous();
  load_groups<NT, kRowsP>(a, s_tiles, s_off);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int ntiles = a.offsets ? s_tiles[a.G] : n_tiles;
  const int kb0 = (int)((long)a.KB * rank / split), kb1 = (int)((long)a.KB * (rank + 1) / split);
  const int first = blockIdx.x / split, step = gridDim.x / split;

  auto fail = [&]() {
    atomicOr(&g_fp8_err, DEV_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp < 4) {
    if (warp == 0) {
      // ---------------- tiles by TMA ----------------
      if (lane == 0) {
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; t < ntiles && ok && !*abort_flag; t += step) {
          Tile ti;
          if (!decode<NT, kRowsP>(a, s_tiles, s_off, t, ti)) break;
          const int brow = ti.grp * a.N + ti.n0;
          for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const uint32_t st = it % C::kStages;
            if (!mbar_wait(&done[st], ((it / C::kStages) & 1) ^ 1)) { ok = false; fail(); break; }
            mbar_arrive_expect_tx(&full[st], C::kStageBytes);
            uint8_t* sp = smem + st * C::kStageBytes;
            tma_load_2d(sp, &bmap, &full[st], kb * kKB, brow);
            tma_load_2d(sp + kPBytes, &amap, &full[st], kb * kKB, ti.m0);
          }
        }
        // nothing may be in flight into this CTA's memory when it ends
        const uint32_t n = it < (uint32_t)C::kStages ? it : (uint32_t)C::kStages;
        for (uint32_t j = 0; j < n && ok; ++j) {
          const uint32_t i = it - 1 - j;
          if (!mbar_wait(&done[i % C::kStages], (i / C::kStages) & 1)) { ok = false; fail(); }
        }
        if (!ok)
          for (uint32_t j = 0; j < n; ++j) {
            const uint32_t i = it - 1 - j;
            mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1);
          }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- scale products, kScaleSteps steps at a time ----------------
      uint32_t sl = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok && !warp_aborted(abort_flag); t += step) {
        Tile ti;
        if (!decode<NT, kRowsP>(a, s_tiles, s_off, t, ti)) break;
        const float* sb = a.sb + ((size_t)ti.grp * a.NB + ti.n0 / 128) * a.KB;
        const float* sa = a.sa + (size_t)kb0 * a.ldsa + ti.m0;
        constexpr int PL = (NT + 31) / 32;                 // columns per lane
        for (int kb = kb0; kb < kb1; kb += kScaleSteps, ++sl) {
          const uint32_t ss = sl % C::kSlots;
          float v[kScaleSteps][PL];
#pragma unroll
          for (int k = 0; k < kScaleSteps; ++k, sa += a.ldsa) {
            const bool in = kb + k < kb1;
            const float bs = in ? sb[kb + k] : 0.f;
#pragma unroll
            for (int i = 0; i < PL; ++i)
              v[k][i] = in && lane + 32 * i < ti.rows ? sa[lane + 32 * i] * bs : 0.f;
          }
          ok = warp_wait(&sempty[ss], ((sl / C::kSlots) & 1) ^ 1);
          if (!ok) { fail(); break; }
          float* sc = s_scale + ss * kScaleSteps * C::kStepFloats;
#pragma unroll
          for (int k = 0; k < kScaleSteps; ++k)
#pragma unroll
            for (int i = 0; i < PL; ++i)
              if (lane + 32 * i < NT) sc[k * NT + lane + 32 * i] = v[k][i];
          mbar_arrive(&sfull[ss]);
        }
      }
    } else if (lane == 0) {
      // ---------------- MMA issuers: warp 1 the even steps, warp 3 the odd ones ----------------
      const uint32_t odd = warp >> 1;
      const uint64_t desc0 = sw128_desc(smem_u32(smem));
      uint32_t it = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok && !*abort_flag; t += step) {
        Tile ti;
        if (!decode<NT, kRowsP>(a, s_tiles, s_off, t, ti)) break;
        const uint32_t idesc = idesc_f8(kRowsP, (ti.rows + 15) & ~15);
        const uint32_t end = it + (kb1 - kb0);
        for (it += (it ^ odd) & 1; it < end; it += 2) {
          const uint32_t st = it % C::kStages, b = it % C::kBufs;
          const uint64_t pd = desc0 + (uint64_t)(st * (C::kStageBytes >> 4));
          const uint64_t qd = pd + (uint64_t)(kPBytes >> 4);
          if (!mbar_wait(&tempty[b], ((it / C::kBufs) & 1) ^ 1) ||
              !mbar_wait(&full[st], (it / C::kStages) & 1)) { ok = false; fail(); break; }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f8_ss(tmem + b * NT, pd + 2 * k, qd + 2 * k, idesc, k > 0);
          mma_commit(&done[st]);
        }
        it = end;
      }
      mma_commit(mma_done);                  // nothing may write TMEM once it is freed
      if (!mbar_wait(mma_done, 0)) fail();
    }
    __syncwarp();
  } else {
    // ---------------- promotion and store ----------------
    const int q = warp & 3;                                // TMEM lane quarter
    const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16);
    const int prow = 32 * q + lane;                        // this thread's weight row
    uint32_t it = 0, sl = 0;
    bool ok = true;
    TO* out = static_cast<TO*>(a.out);
    for (int t = first; t < ntiles && ok && !warp_aborted(abort_flag); t += step) {
      Tile ti;
      if (!decode<NT, kRowsP>(a, s_tiles, s_off, t, ti)) break;
      uint64_t acc[NT / 2];
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) acc[j] = 0;
      for (int kb = kb0; kb < kb1 && ok; kb += kScaleSteps, ++sl) {
        const uint32_t ss = sl % C::kSlots;
        if (!warp_wait(&sfull[ss], (sl / C::kSlots) & 1)) { ok = false; fail(); break; }
        const float* sc = s_scale + ss * kScaleSteps * C::kStepFloats;
        const int steps = min(kScaleSteps, kb1 - kb);
        for (int k = 0; k < steps; ++k, ++it, sc += C::kStepFloats) {
          const uint32_t st = it % C::kStages, b = it % C::kBufs;
          if (!warp_wait(&done[st], (it / C::kStages) & 1)) { ok = false; fail(); break; }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < NT; c += 16) {
            uint32_t r[16];
            tmem_ld16(tbase + b * NT + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const uint4 w = *reinterpret_cast<const uint4*>(sc + c + j);
              uint64_t* s = &acc[(c + j) >> 1];
              s[0] = fma2(pack2(r[j], r[j + 1]), pack2(w.x, w.y), s[0]);
              s[1] = fma2(pack2(r[j + 2], r[j + 3]), pack2(w.z, w.w), s[1]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[b]);
        }
        if (lane == 0) mbar_arrive(&sempty[ss]);
      }
      if (!ok) break;
      if (split > 1) {
        // this CTA's sums for the cluster: [column][row] over the stages, whose
        // loads have all been consumed (one tile per CTA when split)
        float* red = reinterpret_cast<float*>(smem) + prow;
#pragma unroll
        for (int j = 0; j < NT; j += 2) unpack2(acc[j >> 1], red[j * kRowsP], red[(j + 1) * kRowsP]);
      } else if (prow < ti.cols) {
        TO* o = out + (size_t)ti.m0 * a.ldo + ti.n0 + prow;
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          float lo, hi;
          unpack2(acc[j >> 1], lo, hi);
          if (j < ti.rows) store_val(o + (size_t)j * a.ldo, lo);
          if (j + 1 < ti.rows) store_val(o + (size_t)(j + 1) * a.ldo, hi);
        }
      }
    }
  }
  if (split > 1) {
    __syncwarp();
    pair2::cluster_sync();
    Tile ti;
    if (first < ntiles && decode<NT, kRowsP>(a, s_tiles, s_off, first, ti)) {
      // columns [j0, j1) are this CTA's, one per warp at a time; a lane adds four
      // rows of it over the ranks, all of whose loads are under way at once
      const int j0 = NT * (int)rank / split, j1 = min(NT * ((int)rank + 1) / split, ti.rows);
      TO* out = static_cast<TO*>(a.out);
      const float* red = reinterpret_cast<const float*>(smem);
      for (int j = j0 + warp; j < j1; j += C::kThreads / 32) {
        float4 v[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < split) v[s] = ld_cluster4(pair2::map_to_rank(red + j * kRowsP + 4 * lane, s));
        float4 x = v[0];
#pragma unroll
        for (int s = 1; s < 8; ++s)
          if (s < split) { x.x += v[s].x; x.y += v[s].y; x.z += v[s].z; x.w += v[s].w; }
        TO* o = out + (size_t)(ti.m0 + j) * a.ldo + ti.n0 + 4 * lane;
        const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * lane + i < ti.cols) store_val(o + i, f[i]);
      }
    }
    __syncwarp();
    pair2::cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) { tc_fence_after(); tmem_dealloc(tmem, C::kTmemCols); }
}

// ---------------------------------------------------------------------------
// Wide form: 256 activation rows x 256 weight rows on an SM pair.
// ---------------------------------------------------------------------------
constexpr int kWN = 256;                       // weight rows per tile
constexpr int kWStages = 4;
constexpr int kWWarps = 8;                     // promoting warps per CTA
constexpr int kWCols = 128;                    // columns per promoting thread
constexpr int kWThreads = 128 + 32 * kWWarps;
// registers: the launch gives 384 x 168 = 64512; the first warpgroup keeps 40 a thread
// (128 x 40), which leaves the promoting two 232 (256 x 232)
constexpr int kWRegsLow = 40, kWRegsHigh = 232;
constexpr int kWStageBytes = 2 * kPBytes;      // 128 activation rows and 128 weight rows
static_assert(2 <= kWStages, "two TMEM buffers: a done phase could pass unseen");
constexpr int kWOutBytes = 32 * 128;           // output staging: 32 rows of 128 bytes

constexpr int kWScaleSlots = 8;                // scale ring: a slot per step

template <bool ROWS>
struct WCfg {
  // a slot's scales: of 256 columns and of this CTA's 128 rows
  static constexpr int kScaleFloats = ROWS ? kWN + kRowsP : 0;
  static constexpr int kOutOffset = kWStages * kWStageBytes;
  static constexpr int kScaleOffset = kOutOffset + kWWarps * 2 * kWOutBytes;
  static constexpr int kBarOffset = kScaleOffset + kWScaleSlots * kScaleFloats * 4;
  static constexpr int kTableOffset = kBarOffset + 512;
  static constexpr int bytes(int groups) {
    return kTableOffset + (groups ? 2 * (groups + 1) * 4 : 0) + 1024;
  }
};

__device__ __forceinline__ void mma_pair_f8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate));
}

// p[i, i + 4), zeros from n on; vec: p is aligned to 16 bytes
__device__ __forceinline__ float4 four(const float* p, int i, int n, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec && i + 4 <= n) return *reinterpret_cast<const float4*>(p + i);
  if (i < n) v.x = p[i];
  if (i + 1 < n) v.y = p[i + 1];
  if (i + 2 < n) v.z = p[i + 2];
  if (i + 3 < n) v.w = p[i + 3];
  return v;
}

// MMA columns of a pair tile: the valid ones rounded up to 32 (each CTA holds half)
__device__ __forceinline__ int pair_cols(int cols) { return (cols + 31) & ~31; }

template <bool ROWS, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWThreads, 1)
fp8_pair_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                const __grid_constant__ CUtensorMap omap, const Fp8Args a, const int n_tiles) {
  using C = WCfg<ROWS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_scale = reinterpret_cast<float*>(smem + C::kScaleOffset);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);   // the leader's are used
  uint64_t* done = full + kWStages;                                      // a step's products are
                                                                         // finished: both CTAs
  uint64_t* sfull = done + kWStages;                                     // own scales
  uint64_t* sempty = sfull + kWScaleSlots;
  uint64_t* tempty = sempty + kWScaleSlots;                              // [2] the leader's are used
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_tiles = reinterpret_cast<int*>(smem + C::kTableOffset);
  int* s_off = s_tiles + a.G + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = pair2::cluster_rank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kWStages; ++s) { mbar_init(&full[s], 1); mbar_init(&done[s], 1); }
    for (int s = 0; s < kWScaleSlots; ++s) { mbar_init(&sfull[s], 32); mbar_init(&sempty[s], kWWarps); }
    for (int b = 0; b < 2; ++b) mbar_init(&tempty[b], 2 * kWWarps);
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&amap);
    tma_prefetch_desc(&bmap);
  }
  if (warp == 1) { pair2::tmem_alloc_pair(tmem_slot, 512); pair2::tmem_relinquish_pair(); }
  let_next();
  after_previous();
  load_groups<2 * kRowsP, kWN>(a, s_tiles, s_off);
  tc_fence_before();
  __syncthreads();
  pair2::cluster_sync();                 // both CTAs' barriers exist before any remote use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int ntiles = a.offsets ? s_tiles[a.G] : n_tiles;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const uint32_t peer_abort = pair2::map_to_rank(const_cast<int*>(abort_flag), rank ^ 1u);

  auto fail = [&]() {
    atomicOr(&g_fp8_err, DEV_ERR_TIMEOUT);
    *abort_flag = 1;
    pair2::store_remote_u32(peer_abort, 1u);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWRegsLow));
    if (warp == 0) {
      // ---------------- tiles by TMA (both CTAs) ----------------
      if (lane == 0) {
        const uint32_t full_leader = pair2::map_to_rank(full, 0);
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; t < ntiles && ok && !*abort_flag; t += step) {
          Tile ti;
          if (!decode<2 * kRowsP, kWN>(a, s_tiles, s_off, t, ti)) break;
          const int arow = ti.m0 + (int)rank * kRowsP;
          const int brow = ti.grp * a.N + ti.n0 + (int)rank * (pair_cols(ti.cols) >> 1);
          for (int kb = 0; kb < a.KB; ++kb, ++it) {
            const uint32_t st = it % kWStages;
            if (!mbar_wait(&done[st], ((it / kWStages) & 1) ^ 1)) { ok = false; fail(); break; }
            uint8_t* sp = smem + st * kWStageBytes;
            if (leader) mbar_arrive_expect_tx(&full[st], 2 * kWStageBytes);
            const uint32_t fb = full_leader + st * (uint32_t)sizeof(uint64_t);
            pair2::tma_load_2d_pair(sp, &amap, fb, kb * kKB, arow);
            pair2::tma_load_2d_pair(sp + kPBytes, &bmap, fb, kb * kKB, brow);
          }
        }
        // nothing may be in flight into the pair's memory when it ends
        const uint32_t n = it < (uint32_t)kWStages ? it : (uint32_t)kWStages;
        for (uint32_t j = 0; j < n && ok; ++j) {
          const uint32_t i = it - 1 - j;
          if (!mbar_wait(&done[i % kWStages], (i / kWStages) & 1)) { ok = false; fail(); }
        }
        if (!ok && leader)
          for (uint32_t j = 0; j < n; ++j) {
            const uint32_t i = it - 1 - j;
            mbar_wait(&full[i % kWStages], (i / kWStages) & 1);
          }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- scales (both CTAs) ----------------
      if constexpr (ROWS) {
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; t < ntiles && ok && !warp_aborted(abort_flag); t += step) {
          Tile ti;
          if (!decode<2 * kRowsP, kWN>(a, s_tiles, s_off, t, ti)) break;
          const int row0 = (int)rank * kRowsP;
          const float* sb = a.sb + ti.n0;
          const float* sa = a.sa + ti.m0 + row0;
          // whole 16 bytes where the rows of scales allow it
          const bool vec_b = a.ldsb % 4 == 0 && (reinterpret_cast<uintptr_t>(sb) & 15u) == 0;
          const bool vec_a = a.ldsa % 4 == 0 && (reinterpret_cast<uintptr_t>(sa) & 15u) == 0;
          for (int kb = 0; kb < a.KB; ++kb, ++it, sb += a.ldsb, sa += a.ldsa) {
            const uint32_t ss = it % kWScaleSlots;
            const float4 v0 = four(sb, 4 * lane, ti.cols, vec_b);
            const float4 v1 = four(sb, 4 * lane + 128, ti.cols, vec_b);
            const float4 v2 = four(sa, 4 * lane, ti.rows - row0, vec_a);
            ok = warp_wait(&sempty[ss], ((it / kWScaleSlots) & 1) ^ 1);
            if (!ok) { fail(); break; }
            float4* sc = reinterpret_cast<float4*>(s_scale + ss * C::kScaleFloats) + lane;
            sc[0] = v0;
            sc[32] = v1;
            sc[64] = v2;
            mbar_arrive(&sfull[ss]);
          }
        }
      }
    } else if (leader && lane == 0) {
      // ---------------- MMA issuers: warp 1 the even steps, warp 3 the odd ones ----------------
      // (a step's sum is its own, so the steps need no order among each other)
      const uint32_t b = warp >> 1;
      const uint64_t desc0 = sw128_desc(smem_u32(smem));
      const uint32_t d = tmem + b * kWN;
      uint32_t it = 0;
      bool ok = true;
      for (int t = first; t < ntiles && ok && !*abort_flag; t += step) {
        Tile ti;
        if (!decode<2 * kRowsP, kWN>(a, s_tiles, s_off, t, ti)) break;
        const uint32_t idesc = idesc_f8(2 * kRowsP, pair_cols(ti.cols));
        const uint32_t end = it + a.KB;
        for (it += (it ^ b) & 1; it < end; it += 2) {
          const uint32_t st = it % kWStages;
          if (!mbar_wait(&tempty[b], ((it >> 1) & 1) ^ 1) ||
              !mbar_wait(&full[st], (it / kWStages) & 1)) { ok = false; fail(); break; }
          tc_fence_after();
          const uint64_t ad = desc0 + (uint64_t)(st * (kWStageBytes >> 4));
          const uint64_t bd = ad + (uint64_t)(kPBytes >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_pair_f8(d, ad + 2 * k, bd + 2 * k, idesc, k > 0);
          pair2::commit_pair_both(&done[st]);
        }
        it = end;
      }
      pair2::commit_pair_local(mma_done);
      if (!mbar_wait(mma_done, 0)) fail();
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWRegsHigh));
    // ---------------- promotion and store (both CTAs) ----------------
    const int q = warp & 3, half = (warp - 4) >> 2, c0 = half * kWCols;
    const uint32_t tbase = tmem + ((uint32_t)(32 * q) << 16) + c0;
    const uint32_t tempty_leader = pair2::map_to_rank(tempty, 0);
    const int r0 = (int)rank * kRowsP + 32 * q;            // this warp's first row of a tile
    uint8_t* stage = smem + C::kOutOffset + (warp - 4) * 2 * kWOutBytes;
    TO* out = static_cast<TO*>(a.out);
    uint32_t it = 0;
    // Block scales: a thread owns one row; its scale (times its 128 columns' block
    // scale) is read three steps ahead, the next tile's first ones before this tile
    // is written out.
    // Column scales: a thread reads TMEM as 16 x 8 fragments and owns four rows
    // (lane / 4 + 8 n) and a quarter of the columns, so that it takes 32 column
    // scales and 4 row scales a step from shared memory, not 128 column scales, whose
    // broadcasts took 1024 cycles of it (2048 x 8192 x 4096: 160 -> 139 us).  What
    // bounds this form is two operations an element instead of one, the product of
    // the scales and the FMA.
    const float *pa = nullptr, *pb = nullptr;
    float sa[3], sb[3];
    auto open = [&](const Tile& ti) {
      if (ROWS) return;
      const int row = r0 + lane;
      pa = a.sa + ti.m0 + (row < ti.rows ? row : 0);
      pb = a.sb + ((size_t)ti.grp * a.NB + ti.n0 / 128 + (c0 < ti.cols ? half : 0)) * a.KB;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        sa[i] = i < a.KB ? pa[(size_t)i * a.ldsa] : 0.f;
        sb[i] = i < a.KB ? pb[i] : 0.f;
      }
      pa += 3 * a.ldsa;
      pb += 3;
    };
    Tile ti;
    int t = first;
    bool ok = t < ntiles && decode<2 * kRowsP, kWN>(a, s_tiles, s_off, t, ti);
    if (ok) open(ti);
    while (ok && !warp_aborted(abort_flag)) {
      const int qn = ti.cols, nc = qn - c0;                // columns of this half
      uint64_t acc[kWCols / 2];
#pragma unroll
      for (int j = 0; j < kWCols / 2; ++j) acc[j] = 0;
      for (int kb = 0; kb < a.KB; ++kb, ++it) {
        const uint32_t ss = it % kWScaleSlots, b = it & 1;
        uint64_t rs = 0;
        if constexpr (!ROWS) {
          rs = both(sa[0] * sb[0]);
          sa[0] = sa[1]; sa[1] = sa[2]; sb[0] = sb[1]; sb[1] = sb[2];
          if (kb + 3 < a.KB) {
            sa[2] = *pa;
            pa += a.ldsa;
            sb[2] = *pb++;
          }
        }
        if ((ROWS && !warp_wait(&sfull[ss], (it / kWScaleSlots) & 1)) ||
            !warp_wait(&done[it % kWStages], (it / kWStages) & 1)) {
          ok = false;
          fail();
          break;
        }
        tc_fence_after();
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_tmem(tempty_leader + b * (uint32_t)sizeof(uint64_t));
        };
        const float* cs = s_scale + ss * C::kScaleFloats;
        uint64_t rr[4];
        if constexpr (ROWS) {
#pragma unroll
          for (int n = 0; n < 4; ++n) rr[n] = both(cs[kWN + 32 * q + (lane >> 2) + 8 * n]);
          cs += c0 + 2 * (lane & 3);
        }
        // the buffer is given back once its last columns are read, before they are
        // added (8192 x 10240 x 8192: 647 -> 634 us)
        bool held = true;
#pragma unroll
        for (int c = 0; c < kWCols; c += 64) {
          if (c >= nc) break;                              // uniform in the warp
          uint32_t r[2][32];
          if constexpr (ROWS) {
            tmem_ld_frag(tbase + b * kWN + c, r);
          } else {
            pair2::tmem_ld32(tbase + b * kWN + c, r[0]);
            pair2::tmem_ld32(tbase + b * kWN + c + 32, r[1]);
          }
          tmem_ld_wait();
          if (c + 64 >= kWCols) { release(); held = false; }
          uint64_t* s = &acc[c >> 1];
          if constexpr (ROWS) {
            // s[4 i + n]: columns c + 8 i + 2 (lane % 4) and + 1, row lane / 4 + 8 n
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint64_t w = *reinterpret_cast<const uint64_t*>(cs + c + 8 * i);
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                const uint32_t* v = &r[n >> 1][4 * i + 2 * (n & 1)];
                s[4 * i + n] = fma2(pack2(v[0], v[1]), mul2(rr[n], w), s[4 * i + n]);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 64; j += 2)
              s[j >> 1] = fma2(pack2(r[j >> 5][j & 31], r[j >> 5][(j & 31) + 1]), rs, s[j >> 1]);
          }
        }
        if (held) release();
        if (ROWS) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[ss]);
        }
      }
      if (!ok) break;
      const Tile cur = ti;
      t += step;
      ok = t < ntiles && decode<2 * kRowsP, kWN>(a, s_tiles, s_off, t, ti);
      if (ok) open(ti);
      // out: 128 bytes of each of the warp's 32 rows at a time through shared
      // memory (16-byte pieces, exclusive-or swizzled as the output map says); 32
      // whole rows leave by one TMA store, behind which the warp goes on (16-byte
      // stores to 32 rows each held it about 6500 cycles a tile, whole-run
      // stores 4000).  The last rows of a group are stored row by row: what lies
      // behind them is not this group's.  The two staging buffers alternate within a
      // tile; its first pass waits for all earlier stores, since a tile with an odd
      // number of passes ends on the buffer that the next one begins with.  (A count
      // of passes over the whole kernel, with no such wait, needs a register through
      // the main loop and addresses at run time: 8192 x 10240 x 8192 624 us against
      // 612, the column-scale product 148 against 139.)
      constexpr int V = 16 / sizeof(TO), W = 8 * V;        // columns per 16 bytes, per pass
      const int rows = cur.rows - r0;
#pragma unroll
      for (int c = 0; c < kWCols; c += W) {
        if (c0 + c >= qn) break;
        uint8_t* buf = stage + ((c / W) & 1) * kWOutBytes;
        if (lane == 0) {                                   // buf's last store has read it
          if (c == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        }
        __syncwarp();
        if constexpr (ROWS) {
          const int l = lane >> 2, x = 2 * (lane & 3);     // row of 8, column of 8
          const uint32_t off = l * 128 + (((x / V) ^ l) << 4) + x % V * sizeof(TO);
#pragma unroll
          for (int i = 0; i < W / 8; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              uint8_t* at = buf + 1024 * n + (off ^ ((8 * i / V) << 4));
              float lo, hi;
              unpack2(acc[(c + 8 * i) / 2 + n], lo, hi);
              if constexpr (sizeof(TO) == 2) *reinterpret_cast<__nv_bfloat162*>(at) = __floats2bfloat162_rn(lo, hi);
              else *reinterpret_cast<float2*>(at) = make_float2(lo, hi);
            }
        } else {
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            uint4 v;
            TO* e = reinterpret_cast<TO*>(&v);
#pragma unroll
            for (int i = 0; i < V; i += 2) {
              float lo, hi;
              unpack2(acc[(c + h * V + i) >> 1], lo, hi);
              if constexpr (sizeof(TO) == 2) *reinterpret_cast<__nv_bfloat162*>(e + i) = __floats2bfloat162_rn(lo, hi);
              else { e[i] = lo; e[i + 1] = hi; }
            }
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((h ^ (lane & 7)) << 4)) = v;
          }
        }
        const bool whole = a.vec && rows >= 32;
        if (whole) fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          if (whole) tma_store_2d(&omap, buf, cur.n0 + c0 + c, cur.m0 + r0);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        if (!whole) {
          const int h = lane & 7, col = c0 + c + h * V;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            const uint4 v = *reinterpret_cast<const uint4*>(buf + r * 128 + ((h ^ (r & 7)) << 4));
            if (r < rows) {
              TO* o = out + (size_t)(cur.m0 + r0 + r) * a.ldo + cur.n0 + col;
              if (a.vec && col + V <= qn) {
                *reinterpret_cast<uint4*>(o) = v;
              } else {
                const TO* e = reinterpret_cast<const TO*>(&v);
#pragma unroll
                for (int x = 0; x < V; ++x)
                  if (col + x < qn) o[x] = e[x];
              }
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  pair2::cluster_sync();                 // the leader's MMAs and both CTAs' loads are done
  if (warp == 1) { tc_fence_after(); pair2::tmem_dealloc_pair(tmem, 512); }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, from the driver that is loaded
EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(p) : nullptr;
  }();
  return fn;
}

// a matrix of `rows` rows, `pitch` bytes apart (a multiple of 16), by boxes of
// box_rows x 128 bytes in the 128-byte swizzle
bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, long rows, int cols,
            long pitch, int es, int box_rows, CUtensorMapL2promotion l2) {
  const EncodeFn fn = encoder();
  if (!fn || !base || rows <= 0 || cols <= 0 || pitch < (long)cols * es || pitch % 16) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows}, step[2] = {1, 1};
  return fn(map, type, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 8-bit codes: those past a row's K read as zeros
bool make_tmap_codes(CUtensorMap* map, const void* base, long rows, int K, long pitch, int box_rows) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rows, K, pitch, 1, box_rows,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// the output matrix, rows `ld` elements apart
bool make_tmap_out(CUtensorMap* map, void* base, long rows, int cols, long ld, moe_dtype dt) {
  const bool half = dt == MOE_BF16;
  const int es = half ? 2 : 4;
  return encode(map, half ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base,
                rows, cols, ld * es, es, 32, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

constexpr int kMaxDevices = 64;

Fp8Args args_of(const moe_fp8_gemm& g) {
  const long es = g.out_dtype == MOE_BF16 ? 2 : 4;
  Fp8Args a{};
  a.sa = g.a_scales; a.ldsa = g.lda_scales; a.sb = g.b_scales; a.ldsb = g.ldb_scales;
  a.offsets = g.offsets; a.out = g.out; a.ldo = g.ldo; a.M = g.M; a.N = g.N;
  a.KB = ceil_div(g.K, 128); a.G = g.offsets ? g.n_groups : 1; a.NB = ceil_div(g.N, 128);
  a.split = 1;
  // a TMA store writes whole 16 bytes at the matrix's right edge
  a.vec = (g.ldo * es) % 16 == 0 && (g.N * es) % 16 == 0 && (reinterpret_cast<uintptr_t>(g.out) & 15u) == 0;
  return a;
}

// setmaxnreg.inc takes its registers from those that the launch gave the block:
// a kernel compiled to fewer than its split counts on would wait for ever, so it
// is not launched
template <typename K>
cudaError_t check_registers(K kern, int threads, int need) {
  cudaFuncAttributes at;
  const cudaError_t e = cudaFuncGetAttributes(&at, kern);
  if (e != cudaSuccess) return e;
  return at.numRegs * threads >= need ? cudaSuccess : cudaErrorInvalidConfiguration;
}

// Tall form, two CTAs per SM.  A product of few tiles splits K over the CTAs of a
// cluster: the split, up to 8, with the fewest steps one behind the other.  A
// step takes nearly twice as long where two CTAs share an SM (they share its
// loads), a CTA more in the cluster's sum a fifth of a step.  2048 x 8192: M = 128
// as 4 CTAs a tile 13.9 us, as 8 15.7; M = 256 as 2 21.5, as 4 18.9; 1024 x 1024,
// M = 8: as 4 6.3, as 8 5.8.  A
// second wave, whose clusters must find their SMs free together, costs twelve
// steps more: M = 384 as 5 31.4, as 2 27.9.  The runtime's count of resident clusters (74 of 2,
// 45 of 3, 33 of 4, 22 of 6, 15 of 8) takes one CTA per SM for kernels that
// allocate TMEM; the GPU holds two, so beyond the count SMs are shared, and beyond
// twice the count there is another wave: 80 clusters of 3 overlap (13 us for
// 16 x 10240 x 8192 in L2).
constexpr double kSharedStep = 1.95, kSumStep = 0.2, kWaveSteps = 12;
template <int NT, typename TO>
cudaError_t tall_t(const moe_fp8_gemm& g, int n_tiles, int sms, int dev, cudaStream_t st) {
  using C = TCfg<NT>;
  auto kern = fp8_tall_kernel<NT, TO>;
  static std::atomic<int> clusters[kMaxDevices][9];      // resident clusters of each size (0: not asked)
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::bytes(g.offsets ? g.n_groups : 0);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  if (!clusters[dev][1]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::bytes(kMaxGroups));
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
    for (int c = 8; c >= 1; --c) {
      at[0].val.clusterDim.x = c;
      cfg.gridDim = dim3(c * (sms / c));
      int n = 0;
      if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
      clusters[dev][c] = n > 0 ? n : 1;
    }
  }
  Fp8Args a = args_of(g);
  if (!g.offsets) {
    double best = 1e30;
    for (int c = 1; c <= 8 && c <= a.KB; ++c) {
      const int held = clusters[dev][c];
      const double step = n_tiles > held ? kSharedStep : 1.0;
      const double cost = ceil_div(n_tiles, 2 * held) * (step * ceil_div(a.KB, c) + kSumStep * c + kWaveSteps);
      if (cost < best) { best = cost; a.split = c; }
    }
  }
  CUtensorMap am, bm;
  if (!make_tmap_codes(&am, g.a, g.M, g.K, g.lda, NT) ||
      !make_tmap_codes(&bm, g.b, (long)a.G * g.N, g.K, g.ldb, kRowsP))
    return cudaErrorInvalidValue;
  cfg.gridDim = dim3(a.split > 1 ? n_tiles * a.split : (n_tiles < 2 * sms ? n_tiles : 2 * sms));
  at[0].val.clusterDim.x = a.split;
  cfg.attrs = a.split > 1 ? at : at + 1;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, am, bm, a, n_tiles);
}

template <int NT>
cudaError_t tall(const moe_fp8_gemm& g, int n_tiles, int sms, int dev, cudaStream_t st) {
  return g.out_dtype == MOE_BF16 ? tall_t<NT, __nv_bfloat16>(g, n_tiles, sms, dev, st)
                                 : tall_t<NT, float>(g, n_tiles, sms, dev, st);
}

template <bool ROWS, typename TO>
cudaError_t wide_t(const moe_fp8_gemm& g, int n_tiles, int sms, int dev, cudaStream_t st) {
  using C = WCfg<ROWS>;
  auto kern = fp8_pair_kernel<ROWS, TO>;
  static std::atomic<int> pairs[kMaxDevices];    // co-resident pairs (0: not asked yet)
  if (!pairs[dev]) {
    cudaError_t e = check_registers(kern, kWThreads, 128 * kWRegsLow + 256 * kWRegsHigh);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::bytes(kMaxGroups));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (sms / 2));
    cfg.blockDim = dim3(kWThreads);
    cfg.dynamicSmemBytes = C::bytes(kMaxGroups);
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
    pairs[dev] = n > 0 ? n : 1;
  }
  const Fp8Args a = args_of(g);
  CUtensorMap am, bm, om = {};
  if (!make_tmap_codes(&am, g.a, g.M, g.K, g.lda, kRowsP) ||
      !make_tmap_codes(&bm, g.b, (long)a.G * g.N, g.K, g.ldb, kRowsP) ||
      (a.vec && !make_tmap_out(&om, g.out, g.M, g.N, g.ldo, g.out_dtype)))
    return cudaErrorInvalidValue;
  const int room = pairs[dev], n = n_tiles < room ? n_tiles : room;
  return launch_early(kern, 2 * n, kWThreads, C::bytes(g.offsets ? g.n_groups : 0), st, am, bm, om, a, n_tiles);
}

template <bool ROWS>
cudaError_t wide(const moe_fp8_gemm& g, int n_tiles, int sms, int dev, cudaStream_t st) {
  return g.out_dtype == MOE_BF16 ? wide_t<ROWS, __nv_bfloat16>(g, n_tiles, sms, dev, st)
                                 : wide_t<ROWS, float>(g, n_tiles, sms, dev, st);
}

}  // namespace

cudaError_t launch_fp8_gemm(const moe_fp8_gemm& g, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int G = g.offsets ? g.n_groups : 1, KB = ceil_div(g.K, 128);
  const int mean = (g.M + G - 1) / G;                     // rows per group on average
  // an upper bound of the tile count: a grouped kernel reads the exact one from
  // the offsets
  auto tiles = [&](int rm, int rn) {
    const long t = ((long)g.M / rm + G) * ceil_div(g.N, rn);
    const long d = (long)ceil_div(g.M, rm) * ceil_div(g.N, rn);
    const long n = g.offsets ? t : d;
    return n > 0x7fffffff ? 0x7fffffff : (int)n;
  };
  if (g.ldb_scales > 0) return wide<true>(g, tiles(256, 256), sms, dev, st);
  // Tall or wide.  Up to 64 rows (a group's mean, when grouped) the weights are
  // what costs, and they are streamed: 64 groups of 5120 x 2048, mean 11 / 44 / 64
  // / 90 rows: tall 110 / 122 / 160 / 207 us, wide 196 / 199 / 198 / 200;
  // 16 of 2048 x 5120: 32 / 35 / 55 / 58, and 53 wide from 64 rows on.  A popular
  // group among idle ones reads its weights again for each tile of its rows, from
  // L2: with 90 % of the rows in one of 64 groups, mean 11 / 44 / 90 / 704, 130 /
  // 172 / 251 / 629 us, where even ones take 109 / 122 / 205 / 556.
  // Plain products of more rows take the form that by its steps is the shorter: a
  // tall CTA does 0.4 us a step, 0.75 where two share an SM, and 6.5 us besides, most
  // of them the cluster's sum; a wide pair 0.53 us a step and 4.5.
  bool use_tall = mean <= 64;
  if (!use_tall && !g.offsets) {
    const int nt = tiles(64, 128), nw = tiles(256, 256), pairs = sms / 2;
    int split = 2 * sms / nt;
    split = split < 1 ? 1 : split > 8 ? 8 : split;
    const double step = (long)nt * split > sms ? 0.75 : 0.4;
    const double tall_us = 6.5 + step * ceil_div((long)nt * split, 2 * sms) * ceil_div(KB, split);
    const double wide_us = 4.5 + 0.53 * ceil_div(nw, pairs) * KB;
    use_tall = tall_us < wide_us;
  }
  if (!use_tall) return wide<false>(g, tiles(256, 256), sms, dev, st);
  if (mean <= 16) return tall<16>(g, tiles(16, 128), sms, dev, st);
  if (mean <= 32) return tall<32>(g, tiles(32, 128), sms, dev, st);
  return tall<64>(g, tiles(64, 128), sms, dev, st);
}

cudaError_t fp8_gemm_take_error(int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_fp8_err, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && *word) e = cudaMemcpyToSymbol(g_fp8_err, &zero, sizeof(int));
  return e;
}

}  // namespace lmoe
