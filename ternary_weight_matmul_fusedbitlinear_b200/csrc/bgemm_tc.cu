// Training contractions on the 5th-generation tensor cores (tcgen05 kind::f16,
// bf16 operands, fp32 accumulators in tensor memory).
//
// The gradients of a ternary layer y = gamma (q . w) / s are two products
// ("MatMul-free language models", DataCamp blog, "Memory efficiency": the
// models are trained with fused GPU kernels; no formula is printed, these are
// the derivatives with the two roundings passed straight through):
//   dx^[t, k] = gamma sum_n dy[t, n] w[n, k]        form dx
//   dW [n, k] = sum_t dy[t, n] q[t, k] / s[t]       form dw
// The ternary codes w, and the int8 codes q, are exact in bf16, so the only
// rounded operand is the gradient (or, for a caller's bf16 gradient, q / s).
// An fp32 gradient comes as three bf16 planes g = g0 + g1 + g2 (24 bits); the
// smallest plane is multiplied first.
//
// Operands stay as they lie in memory. For dx the gradient is K-major (its
// reduction index n is contiguous); every other operand has the reduction
// index as its row, i.e. is MN-major, which the MMA takes directly (no
// transposed copies): a 64 x 64 box per 128-byte swizzle column block.
//
// What bounds it: feeding the tensor cores. A 128 x 256 tile per SM takes 48 KB
// of operands per 64 reduction steps; CTAS = 2 pairs the two SMs of a cluster on
// a 256 x 256 tile (cta_group::2), each loading its own 128 rows of A and half
// of B, 32 KB. 8192 x 2048 x 8192, gradient of the input: 181 us on pairs (1.52
// PFLOP/s), 200 us on single SMs (1.38), which stay for products whose tiles
// fill them better.
//
// Persistent: TMA ring (4 x 48 KB or 6 x 32 KB), two TMEM accumulators, so a
// tile's epilogue runs under the next tile's main loop. The last column tile
// shrinks the MMA to the columns there are. Too few tiles for the SMs: the
// reduction is cut in `splits` ranges, each writing its own fp32 slice for the
// kernel that reads the result to add up in order (no atomics, same result
// each run).
//
// Even shares: tiles rarely fill the last round (160 tiles on 74 pairs are 2.16
// rounds of work in 3 rounds of time). With `even` the whole rounds go as
// before and the tiles left over are cut so that every group gets the same
// share of their reduction, in order: a group ends one tile and begins the
// next. Parts of tiles go to fp32 slots (two per group), which a second kernel
// adds in order of the reduction. 4096 x 2560 x 13824, gradient of the input:
// 225 -> 185 us.
//
// One launch can run both products of a backward, dx's tiles before dw's: small
// ones share the SMs, one start-up and one launch.
//
// Chained products: the reduction is cut in units (32 k-steps of one segment; 4 for fp32
// planes) whose sums leave tensor memory one by one and are added in registers,
// each times its segment's gamma. For several layers of one input that is the
// sum over layers in one launch; for fp32 it bounds the error: the tensor
// core's running sum is truncated at every step (measured 2e-8 relative per 16
// reduction steps), the register sum is rounded.
#include "kernels.cuh"
#include "umma.cuh"

namespace mmf {

namespace {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int A_BYTES = BM * BK * 2, BOX_BYTES = 64 * 64 * 2;
constexpr int kEpiWarps = 8, kEpiWarp0 = 2;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr int kChainF32 = 4, kChainBf16 = 32;   // k-steps per unit

template <int CTAS>
struct __align__(1024) Smem {
  static constexpr int NS = CTAS == 2 ? 6 : 4;
  static constexpr int B_BYTES = BN / CTAS * BK * 2;
  uint8_t a[NS][A_BYTES];
  uint8_t b[NS][B_BYTES];
  uint8_t stage[kEpiWarps][4096];   // one fp32 box of 32 x 32, or two bf16 ones
  uint64_t full[NS], empty[NS], tmem_full[2], tmem_empty[2], mma_drain;
  uint32_t tmem_base;
  int abort_flag;
};

// kind::f16 with bf16 operands and fp32 accumulators; a set bit marks an
// MN-major operand.
__device__ __forceinline__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// MN-major operand, 128-byte swizzle: 64 MN elements x 8 reduction rows per
// 1024-byte atom; the next 8 rows follow at 1024 bytes, the next 64 MN
// elements at one 64 x 64 box.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(BOX_BYTES >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

template <int CTAS>
__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accum) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum)
        : "memory");
}

// Completion of the MMAs issued so far: arrives at the barrier, in both CTAs of a pair.
template <int CTAS>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    umma_commit(bar);
}

// Address of the pair's first CTA's copy of a shared variable.
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}

// TMA load into this CTA's shared memory; a pair's loads all count on its first
// CTA's barrier (`bar`: its shared::cluster address).
template <int CTAS>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Several 64-column blocks in one load: a 3-D map {64, rows, cols / 64}.
template <int CTAS>
__device__ __forceinline__ void load_blocks(void* dst, const CUtensorMap* map, int y, int block, uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(block), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(block), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// mbar_wait with cluster scope, for a barrier that the other CTA of the pair arrives at.
__device__ __noinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          long long limit) {
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > limit) {
      *abort_flag = 1;
      if (status) atomicExch(status, 1);
      return false;
    }
  }
}

// What the kernel reads of a product (BGemmArgs without its operands).
struct ProbArgs {
  int a_plane, planes, I, J, R, splits, slice_rows, seg_pitch, seg_rows;
  bool out_f32, accumulate;
  const void* out[3];
  const float *gamma[3], *inv_gamma[3], *row_scale;
  const int8_t* dot_q;
  float* dot_part;
};
struct Prob {
  ProbArgs g;
  int i_tiles, j_tiles;
  int nk, cl, ups, units;   // k-steps per segment; k-steps per unit; units per segment and in all
  bool wide_a, wide_b;      // MN-major operands loaded by 64-column blocks (widths that are multiples of 64)
};
struct KArgs {
  Prob pr[2];               // dx, dw
  int tiles0, tiles;        // dx's tiles; all tiles that go whole
  int shared;               // even shares (one product): tiles after those, cut among all groups
  int* status;
  long long wait_cycles;
};
struct Maps {
  CUtensorMap a[2], b[2], o[4];   // outputs: dx, then dw's segments
  CUtensorMap slots;              // even shares: fp32 [2 groups][tile rows][256]
};

// Group c's share of `total` units in `groups` equal parts.
__host__ __device__ __forceinline__ long long share_begin(long long total, int groups, int c) {
  return total * c / groups;
}

// KIND 0: nothing chained; 1: dx chained (several layers); 2: both (fp32 planes).
// MODE 0: dx alone, 1: dw alone, 2: both.
template <int KIND, int CTAS, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    bgemm_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ KArgs p) {
  using S = Smem<CTAS>;
  constexpr int NS = S::NS;
  extern __shared__ uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const int rank = CTAS == 2 ? blockIdx.x & 1 : 0;
  const int first = blockIdx.x / CTAS, stride = gridDim.x / CTAS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.tmem_full[a], 1);
      mbar_init(&sm.tmem_empty[a], CTAS * kEpiWarps);
    }
    mbar_init(&sm.mma_drain, 1);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    const int d = MODE == 2 ? (first < p.tiles0 ? 0 : 1) : MODE;
    prefetch_tmap(&maps.a[d]);
    prefetch_tmap(&maps.b[d]);
  }
  if (warp == 1) {
    if constexpr (CTAS == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();   // barriers of both CTAs are set up
  tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;
  pdl_trigger();
  pdl_wait();

  // tile -> product, (split, i tile, j tile), j fastest: neighbours share their
  // rows of A; its range of units; whether units are drained one by one
  struct Place {
    bool dw, chain;
    int sp, it, jt, lo, hi;
    int slot;   // part of a tile: where its sums go (-1: a whole tile)
  };
  auto place = [&](int tile) {
    Place t;
    t.dw = MODE == 2 ? tile >= p.tiles0 : MODE == 1;
    const Prob& q = p.pr[t.dw];
    const int id = MODE == 2 && t.dw ? tile - p.tiles0 : tile;
    // one division in the usual case: between tiles the MMA thread's own
    // arithmetic is time the tensor cores lose
    const unsigned row = (unsigned)id / (unsigned)q.j_tiles;
    t.jt = id - (int)row * q.j_tiles;
    t.it = (int)row;
    t.sp = 0;
    t.lo = 0;
    t.hi = q.units;
    if (q.g.splits > 1) {
      t.sp = (int)(row / (unsigned)q.i_tiles);
      t.it = (int)row - t.sp * q.i_tiles;
      t.lo = (int)((long long)q.units * t.sp / q.g.splits);
      t.hi = (int)((long long)q.units * (t.sp + 1) / q.g.splits);
    }
    t.chain = KIND == 2 || (KIND == 1 && !t.dw);
    t.slot = -1;
    return t;
  };
  // This group's work in order: whole tiles, then its share of the others.
  struct Walk {
    int tile;
    long long u, end;
  };
  auto begin = [&]() {
    Walk w;
    w.tile = first;
    w.u = w.end = 0;
    if (MODE < 2 && p.shared > 0) {
      const long long total = (long long)p.shared * p.pr[MODE == 1].units;
      w.u = share_begin(total, stride, first);
      w.end = share_begin(total, stride, first + 1);
    }
    return w;
  };
  auto next = [&](Walk& w, Place& t) {
    if (w.tile < p.tiles) {
      t = place(w.tile);
      w.tile += stride;
      return true;
    }
    if (MODE == 2 || w.u >= w.end) return false;
    const int units = p.pr[MODE == 1].units, k = (int)(w.u / units);
    t = place(p.tiles + k);   // splits is 1: sp = 0
    t.lo = (int)(w.u - (long long)k * units);
    t.hi = (int)min((long long)units, t.lo + (w.end - w.u));
    t.slot = t.lo == 0 && t.hi == units ? -1 : 2 * first + (t.lo == 0 ? 1 : 0);
    w.u += t.hi - t.lo;
    return true;
  };
  // MMA columns of a tile: a multiple of 16, for a pair of 32 (each CTA holds half
  // of B), of 128 where B comes in blocks
  auto cols_of = [&](const Prob& q, int jt) {
    const int n = min(BN, q.g.J - jt * BN);
    return CTAS == 1 ? n : q.wide_b ? (n + 127) / 128 * 128 : (n + 31) / 32 * 32;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // One thread feeds the ring; its instructions per step are on the critical
    // path (a few more of them cost 5 % of the product), hence the running
    // stage and phase and the few wide loads.
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 1, n = 0;
      bool ok = true;
      const uint32_t bar0 = CTAS == 2 ? leader_addr(&sm.full[0]) : smem_u32(&sm.full[0]);
      Place t;
      for (Walk w = begin(); ok && next(w, t);) {
        const Prob& q = p.pr[t.dw];
        const CUtensorMap *ma = &maps.a[t.dw], *mb = &maps.b[t.dw];
        const int half = cols_of(q, t.jt) / CTAS;
        const bool wide_a = q.wide_a, wide_b = q.wide_b;
        const int boxes = wide_b ? BN / CTAS / 64 : (half + 63) / 64;
        const uint32_t bytes = CTAS * (A_BYTES + boxes * BOX_BYTES);
        const int i0 = (t.it * CTAS + rank) * BM, j0 = t.jt * BN + rank * half;
        // k-step at reduction row r of B, row (or column) ra of A
        auto step = [&](int ra_x, int ra_y, int r) {
          if (!mbar_try_wait(&sm.empty[s], ph) && !mbar_wait(&sm.empty[s], ph, abort_flag, p.status, p.wait_cycles))
            return false;
          const uint32_t bar = bar0 + 8 * s;
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], bytes);
          if (t.dw && wide_a) {
            load_blocks<CTAS>(sm.a[s], ma, ra_y, i0 / 64, bar);
          } else if (t.dw) {
            load_box<CTAS>(sm.a[s], ma, i0, ra_y, bar);
            load_box<CTAS>(sm.a[s] + BOX_BYTES, ma, i0 + 64, ra_y, bar);
          } else {
            load_box<CTAS>(sm.a[s], ma, ra_x, ra_y, bar);
          }
          if (wide_b) {
            load_blocks<CTAS>(sm.b[s], mb, r, j0 / 64, bar);
          } else {
            for (int b = 0; b < boxes; ++b) load_box<CTAS>(sm.b[s] + b * BOX_BYTES, mb, j0 + 64 * b, r, bar);
          }
          if (++s == NS) {
            s = 0;
            ph ^= 1;
          }
          ++n;
          return true;
        };
        if (!t.chain) {
          for (int r = t.lo * BK; r < t.hi * BK && ok; r += BK) ok = step(r, t.dw ? r : i0, r);
        } else {
          for (int u = t.lo; u < t.hi && ok; ++u) {
            const int seg = u / q.ups, kb0 = (u - seg * q.ups) * q.cl, kb1 = min(kb0 + q.cl, q.nk);
            for (int pl = q.g.planes - 1; pl >= 0 && ok; --pl)
              for (int kb = kb0; kb < kb1 && ok; ++kb) {
                const int r = seg * q.g.R + kb * BK;
                ok = step(r, pl * q.g.a_plane + (t.dw ? kb * BK : i0), r);
              }
          }
        }
      }
      // let every copy land before the CTA (the pair) can exit
      if (rank == 0)
        for (uint32_t j = (n > NS ? n - NS : 0); j < n; ++j) mbar_drain(&sm.full[j % NS], (j / NS) & 1, p.wait_cycles);
      if (CTAS == 2 && !ok) {   // gave up: the other CTA's copies count on barriers that nobody waits at any more
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the pair's first CTA)
    if (lane == 0 && rank == 0) {
      int s = 0;
      uint32_t ph = 0, na = 0;   // ring phase; accumulators begun
      bool ok = true;
      Place t;
      for (Walk w = begin(); ok && next(w, t);) {
        const Prob& q = p.pr[t.dw];
        const uint32_t idesc = idesc_bf16(BM * CTAS, cols_of(q, t.jt), t.dw, true);
        // 16 reduction steps: 2 row groups (MN-major) or 32 bytes (K-major)
        const uint32_t astep = t.dw ? 128 : 2;
        // `steps` ring stages into the next accumulator
        auto accumulate = [&](int steps) {
          const int acc = na & 1;
          const uint32_t eph = ((na >> 1) & 1) ^ 1;
          const bool got = CTAS == 2 ? wait_cluster(&sm.tmem_empty[acc], eph, abort_flag, p.status, p.wait_cycles)
                                     : mbar_wait(&sm.tmem_empty[acc], eph, abort_flag, p.status, p.wait_cycles);
          if (!got) return false;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * BN;
          for (int st = 0; st < steps; ++st) {
            if (!mbar_try_wait(&sm.full[s], ph) && !mbar_wait(&sm.full[s], ph, abort_flag, p.status, p.wait_cycles))
              return false;
            tc_fence_after();
            const uint64_t ad = t.dw ? desc_mn_sw128(smem_u32(sm.a[s])) : umma_desc_sw128(smem_u32(sm.a[s]));
            const uint64_t bd = desc_mn_sw128(smem_u32(sm.b[s]));
#pragma unroll
            for (int j = 0; j < BK / 16; ++j)
              umma_f16<CTAS>(d_tmem, ad + (uint64_t)(astep * j), bd + (uint64_t)(128 * j), idesc, st + j);
            commit<CTAS>(&sm.empty[s]);
            if (++s == NS) {
              s = 0;
              ph ^= 1;
            }
          }
          commit<CTAS>(&sm.tmem_full[acc]);
          ++na;
          return true;
        };
        if (!t.chain) {
          ok = accumulate(t.hi - t.lo);
        } else {
          for (int u = t.lo; u < t.hi && ok; ++u) {
            const int kb0 = (u % q.ups) * q.cl;
            ok = accumulate((min(kb0 + q.cl, q.nk) - kb0) * q.g.planes);
          }
        }
      }
      // every MMA this thread issued has finished before TMEM can be released
      if constexpr (CTAS == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_u32(&sm.mma_drain))
                     : "memory");
      else
        umma_commit(&sm.mma_drain);
      mbar_drain(&sm.mma_drain, 0, p.wait_cycles);
    }
  } else {
    // ------------------------------------------------------------ epilogue (8 warps)
    const int ew = warp - kEpiWarp0;
    const int quarter = warp & 3, group = ew >> 2;
    const uint32_t empty_at[2] = {CTAS == 2 ? leader_addr(&sm.tmem_empty[0]) : smem_u32(&sm.tmem_empty[0]),
                                  CTAS == 2 ? leader_addr(&sm.tmem_empty[1]) : smem_u32(&sm.tmem_empty[1])};
    uint32_t na = 0;
    int nst = 0;
    bool last_bf16 = false;
    auto wait_full = [&]() {
      const bool got = mbar_wait(&sm.tmem_full[na & 1], (na >> 1) & 1, abort_flag, p.status, p.wait_cycles);
      __syncwarp();
      const bool all = __all_sync(0xffffffffu, got);
      tc_fence_after();
      return all;
    };
    auto release_acc = [&]() {   // one arrival per warp, at the issuing CTA
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CTAS == 2)
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(empty_at[na & 1]) : "memory");
        else
          mbar_arrive(&sm.tmem_empty[na & 1]);
      }
      ++na;
    };
    Place t;
    for (Walk walk = begin(); next(walk, t);) {
      const Prob& q = p.pr[t.dw];
      const int i0 = (t.it * CTAS + rank) * BM + quarter * 32;   // this warp's 32 rows of the result
      const int i = i0 + lane;
      // where the rows go: a slice of partial sums, or segment `seg` of dW
      int seg = 0, y = t.sp * q.g.slice_rows + i0;
      float sc = 1.0f;
      bool rows_ok = i0 < q.g.I;
      if (t.dw) {
        if (q.g.splits == 1) {
          seg = i0 / q.g.seg_pitch;
          y = i0 - seg * q.g.seg_pitch;
          rows_ok = rows_ok && seg < 3 && q.g.out[seg < 3 ? seg : 0] != nullptr;
          if (rows_ok && q.g.inv_gamma[seg] != nullptr) sc = 1.0f / fold_gamma(*q.g.inv_gamma[seg]);
        }
      } else {
        if (!t.chain && q.g.gamma[0] != nullptr) sc = *q.g.gamma[0];
        if (q.g.row_scale != nullptr && i < q.g.I) sc *= q.g.row_scale[i];
      }
      const CUtensorMap* mo = &maps.o[t.dw ? 1 + (rows_ok ? seg : 0) : 0];
      const bool part = MODE < 2 && t.slot >= 0;
      const bool f32 = MODE == 0 || part ? true : q.g.out_f32;
      const bool add = q.g.accumulate && !part;
      if (part) {   // rows of a slot, scaled as the result would be
        mo = &maps.slots;
        y = (t.slot * CTAS + rank) * BM + quarter * 32;
      }
      const int jo = part ? t.jt * BN : 0;   // a slot's columns count from the tile's
      const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
      const int jg = t.jt * BN + group * 128;                    // this warp's first column

      // One staging area per warp: an fp32 box, or two bf16 ones. Boxes of both
      // sizes may follow one another, so a bf16 box waits for all but the last
      // store only when that was a bf16 one too.
      auto put = [&](const float (&out)[32], int j0) {
        uint8_t* buf = sm.stage[ew];
        const bool two = !f32 && last_bf16;
        if (lane == 0) {
          if (two) bulk_wait_read_le1();
          else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        __syncwarp();
        if (f32) {
          stage_row(buf, lane, out, (float*)nullptr);
        } else {
          buf += (nst & 1) * 2048;
          stage_row(buf, lane, out, (bf16*)nullptr);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (f32 && add) tma_add_2d(mo, buf, j0 - jo, y);
          else tma_store_2d(mo, buf, j0 - jo, y);
        }
        last_bf16 = !f32;
        ++nst;
      };

      if (KIND > 0 && t.chain) {
        float acc[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c][j] = 0.0f;
        bool alive = true;
        for (int u = t.lo; u < t.hi; ++u) {
          if (!(alive = wait_full())) break;
          float g = sc;
          if (!t.dw && q.g.gamma[u / q.ups] != nullptr) g *= *q.g.gamma[u / q.ups];
          const uint32_t tbase = tmem_base + lanes + (na & 1) * BN + group * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (jg + 32 * c < q.g.J) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                uint32_t r[16];
                tmem_ld16(tbase + 32 * c + h, r);
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[c][h + j] = fmaf(__uint_as_float(r[j]), g, acc[c][h + j]);
              }
            }
          release_acc();
        }
        if (!alive) break;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (rows_ok && jg + 32 * c < q.g.J) put(acc[c], jg + 32 * c);
      } else if (KIND < 2) {
        const bool dots = MODE == 0 && KIND == 0 && q.g.dot_q != nullptr && !part;
        uint4 codes[8];   // this row's codes under the tile's columns, fetched ahead of the accumulator
        if (dots) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const bool in = i < q.g.I && jg + 16 * c < q.g.J;   // J is a multiple of 16
            codes[c] = in ? __ldg(reinterpret_cast<const uint4*>(q.g.dot_q + (size_t)i * q.g.J + jg + 16 * c))
                          : make_uint4(0, 0, 0, 0);
          }
        }
        if (!wait_full()) break;
        const uint32_t tbase = tmem_base + lanes + (na & 1) * BN + group * 128;
        if (dots) {
          float dot = 0.0f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (jg + 32 * c < q.g.J && rows_ok) {
              uint32_t r[32];
              tmem_ld32(tbase + 32 * c, r);
              float out[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                out[j] = __uint_as_float(r[j]) * sc;
                const uint32_t w = (&codes[2 * c + j / 16].x)[j / 4 % 4];
                if (jg + 32 * c + j / 16 * 16 < q.g.J)   // past J the accumulator was never written
                  dot = fmaf(out[j], (float)((int)(w << (24 - 8 * (j & 3))) >> 24), dot);
              }
              put(out, jg + 32 * c);
            }
          }
          if (i < q.g.I && jg < q.g.J) q.g.dot_part[(size_t)(2 * t.jt + group) * q.g.I + i] = dot;
        } else {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            if (jg + 32 * c >= q.g.J || !rows_ok) break;
            uint32_t r[32];
            tmem_ld32(tbase + 32 * c, r);
            float out[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) out[j] = __uint_as_float(r[j]) * sc;
            put(out, jg + 32 * c);
          }
        }
        release_acc();
      }
    }
    // the staging areas have been read; the stores themselves end with the kernel
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();   // the first CTA's MMAs have read this one's shared memory
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (CTAS == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
  }
}

// Even shares: adds up the parts of each tile that was cut, in order of the
// reduction, into the result. A block has 4 rows x 256 columns, a thread 4
// columns. With codes it also leaves the rows' partial dots that whole tiles
// left in the epilogue.
struct ShareArgs {
  ProbArgs g;
  int i_tiles, j_tiles, units, tile0, tiles, groups, tile_rows;
  const float* slots;
};

template <typename OUT>
__global__ void __launch_bounds__(256) share_join_kernel(const __grid_constant__ ShareArgs a) {
  pdl_trigger();
  pdl_wait();
  const long long total = (long long)a.tiles * a.units, t0 = (long long)blockIdx.x * a.units, t1 = t0 + a.units;
  // the groups whose shares meet this tile
  int c0 = (int)(t0 * a.groups / total);
  while (share_begin(total, a.groups, c0 + 1) <= t0) ++c0;
  if (share_begin(total, a.groups, c0) <= t0 && share_begin(total, a.groups, c0 + 1) >= t1) return;   // whole
  const int tile = a.tile0 + blockIdx.x, jt = tile % a.j_tiles, it = tile / a.j_tiles;
  const int row = threadIdx.x / 64 + 4 * blockIdx.y, i = it * a.tile_rows + row;
  if (i >= a.g.I) return;
  void* out = nullptr;
  size_t at = 0;
  if (a.g.seg_pitch > 0) {
    const int seg = i / a.g.seg_pitch, n = i - seg * a.g.seg_pitch;
    if (seg >= 3 || n >= a.g.seg_rows) return;
    out = const_cast<void*>(a.g.out[seg]);
    at = (size_t)n * a.g.J;
  } else {
    out = const_cast<void*>(a.g.out[0]);
    at = (size_t)i * a.g.J;
  }
  if (out == nullptr) return;
  const int jl = threadIdx.x % 64 * 4, j = jt * BN + jl;   // J is a multiple of 16
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float dot = 0.0f;
  if (j < a.g.J) {
    for (int c = c0; c < a.groups; ++c) {
      const long long lo = share_begin(total, a.groups, c);
      if (lo >= t1) break;
      if (share_begin(total, a.groups, c + 1) <= max(lo, t0)) continue;   // an empty share
      const int slot = 2 * c + (lo <= t0 ? 1 : 0);   // began the tile, or went on with it
      const float4 w = *reinterpret_cast<const float4*>(a.slots + ((size_t)slot * a.tile_rows + row) * BN + jl);
      v[0] += w.x;
      v[1] += w.y;
      v[2] += w.z;
      v[3] += w.w;
    }
    if (a.g.dot_q != nullptr) {
      const int w = *reinterpret_cast<const int*>(a.g.dot_q + at + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) dot = fmaf(v[e], (float)((w << (24 - 8 * e)) >> 24), dot);
    }
    OUT* o = static_cast<OUT*>(out) + at + j;
    if constexpr (sizeof(OUT) == 4) {
      if (a.g.accumulate) {
        const float4 w = *reinterpret_cast<const float4*>(o);
        v[0] += w.x;
        v[1] += w.y;
        v[2] += w.z;
        v[3] += w.w;
      }
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      __nv_bfloat162 x = __floats2bfloat162_rn(v[0], v[1]), y = __floats2bfloat162_rn(v[2], v[3]);
      uint2 u;
      u.x = *reinterpret_cast<uint32_t*>(&x);
      u.y = *reinterpret_cast<uint32_t*>(&y);
      *reinterpret_cast<uint2*>(o) = u;
    }
  }
  if (a.g.dot_q != nullptr) {   // a warp has 128 columns of one row
    const int h = threadIdx.x % 64 / 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (threadIdx.x % 32 == 0 && jt * BN + 128 * h < a.g.J) a.g.dot_part[(size_t)(2 * jt + h) * a.g.I + i] = dot;
  }
}

template <int KIND, int CTAS, int MODE>
cudaError_t launch_form(const Maps& m, const KArgs& p, cudaStream_t stream) {
  auto kern = bgemm_tc_kernel<KIND, CTAS, MODE>;
  const size_t smem = sizeof(Smem<CTAS>) + 1024;
  static_assert(sizeof(Smem<CTAS>) + 1024 <= 227 * 1024, "shared memory");
  static SmemOptIn opt;
  const cudaError_t e = opt.set(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int groups = p.shared > 0 ? num_sms() / CTAS : std::min(p.tiles, num_sms() / CTAS);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(groups * CTAS);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CTAS == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, m, p);
}

template <int KIND, int CTAS>
cudaError_t launch_mode(int mode, const Maps& m, const KArgs& p, cudaStream_t stream) {
  if constexpr (KIND != 1)
    if (mode == 1) return launch_form<KIND, CTAS, 1>(m, p, stream);
  return mode == 0 ? launch_form<KIND, CTAS, 0>(m, p, stream) : launch_form<KIND, CTAS, 2>(m, p, stream);
}

bool is_chain(int planes, int nseg) { return planes > 1 || nseg > 1; }
int chain_steps(int planes, int nseg) { return !is_chain(planes, nseg) ? 1 : planes > 1 ? kChainF32 : kChainBf16; }

}  // namespace

namespace {

// Model of one product's time on one B200: groups (SMs, or pairs) take tiles in
// turn; a tile takes its share of the reduction and a start-up; fp32 slices are
// written and read again. Measured: a pair 0.32 us per 64 steps of 256 x 256,
// an SM 0.36 us of 128 x 256, about 2 us per tile.
struct Model {
  bool pair;
  int groups;
  double step_us, tile_us;
  explicit Model(bool two) : pair(two) {
    groups = two ? num_sms() / 2 : num_sms();
    step_us = two ? 0.32 : 0.36;
    tile_us = 2.0;
  }
  long long tiles(const BGemmShape& s) const {
    return (long long)ceil_div(s.I, pair ? 2 * BM : BM) * ceil_div(s.J, BN);
  }
  double tile_time(const BGemmShape& s, int splits) const {
    return (double)ceil_div(s.R, BK) * s.planes * s.nseg / splits * step_us + tile_us;
  }
};
double slices_us(const BGemmShape& s, int splits, bool dw) {
  return splits == 1 ? 0.0 : (dw ? 3.0 : 0.0) + (double)splits * s.I * s.J * 8 / 4e6;
}
const int kTry[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32};
bool may_split(const BGemmShape& s, int splits) {   // at least 8 k-steps in each
  return splits == 1 || (splits <= bgemm_units(s) && ceil_div(s.R, BK) * s.planes * s.nseg >= 8 * splits);
}

}  // namespace

// Tile shape, splits, and whether both products go in one launch: they do when
// all their tiles run at once (small products: one launch and one start-up
// less, a one-token backward 29 -> 16 us), and not when they take rounds (the
// 370M GLU's 540 us in four launches, 548 us in two: the operands of both then
// compete for L2).
BGemmPlan bgemm_plan(const BGemmShape& dx, const BGemmShape& dw) {
  BGemmPlan best = {};
  best.together = true;
  double best_t = 1e30;
  for (int pair = 0; pair < 2; ++pair) {
    const Model m(pair != 0);
    const long long n0 = m.tiles(dx), n1 = m.tiles(dw);
    // one round either way: single SMs start quicker and split the rows finer
    if (n0 + n1 > m.groups || best_t < 1e30) continue;
    for (int s0 : kTry) {
      if (n0 * s0 + n1 > m.groups || !may_split(dx, s0)) break;
      for (int s1 : kTry) {
        if (n0 * s0 + n1 * s1 > m.groups || !may_split(dw, s1)) break;
        const double t = std::max(m.tile_time(dx, s0), m.tile_time(dw, s1)) + slices_us(dx, s0, false) +
                         slices_us(dw, s1, true);
        if (t < best_t) {
          best_t = t;
          best.pair[0] = best.pair[1] = pair != 0;
          best.splits[0] = s0;
          best.splits[1] = s1;
        }
      }
    }
  }
  if (best_t < 1e30) return best;
  best = {};
  const BGemmShape* sh[2] = {&dx, &dw};
  for (int i = 0; i < 2; ++i) {
    best_t = 1e30;
    for (int pair = 0; pair < 2; ++pair) {
      const Model m(pair != 0);
      const long long n = m.tiles(*sh[i]);
      for (int s : kTry) {
        if (s > 1 && (n * s > 4 * m.groups || !may_split(*sh[i], s))) break;
        const double t = (double)((n * s + m.groups - 1) / m.groups) * m.tile_time(*sh[i], s) + slices_us(*sh[i], s, i == 1);
        if (t < best_t) {
          best_t = t;
          best.pair[i] = pair != 0;
          best.splits[i] = s;
          best.even[i] = false;
        }
      }
      // even shares of the last round: their parts are written and read once more, and
      // groups at different places of the reduction share fewer operands in L2
      // (1024 x 2816 x 16384, 44 tiles: 94 us, in 3 splits 88 us)
      const long long left = n % m.groups;
      const double parts_us = 12.0 + (double)(m.groups + left) * (pair ? 2 : 1) * BM * BN * 8 / 4e6;
      const double t = (double)(n / m.groups) * m.tile_time(*sh[i], 1) +
                       (m.tile_time(*sh[i], 1) - m.tile_us) * left / m.groups + 2 * m.tile_us + parts_us;
      if (left > 0 && t < best_t && left * bgemm_units(*sh[i]) >= 8 * m.groups) {
        best_t = t;
        best.pair[i] = pair != 0;
        best.splits[i] = 1;
        best.even[i] = true;
      }
    }
  }
  return best;
}

// Two slots per group: the same size for pairs and for single SMs.
size_t bgemm_slot_floats() { return (size_t)2 * num_sms() * BM * BN; }

int bgemm_slice_rows(int I) { return ceil_div(I, 32) * 32; }

int bgemm_units(const BGemmShape& s) {
  return s.nseg * ceil_div(ceil_div(s.R, BK), chain_steps(s.planes, s.nseg));
}

cudaError_t launch_bgemm_tc(const BGemmArgs* dx, const BGemmArgs* dw, bool pair, int* status, cudaStream_t stream) {
  Maps m;
  KArgs p = {};
  const BGemmArgs* args[2] = {dx, dw};
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  bool chain[2] = {};
  int tiles[2] = {};
  for (int d = 0; d < 2; ++d) {
    if (args[d] == nullptr || args[d]->sh.I == 0 || args[d]->sh.J == 0) continue;
    const BGemmArgs& g = *args[d];
    const BGemmShape& s = g.sh;
    const uint64_t a_rows = (uint64_t)(s.planes - 1) * g.a_plane + (d ? s.R : s.I);
    const uint64_t a_cols = d ? s.I : (uint64_t)s.nseg * s.R;
    const uint64_t b_rows = (uint64_t)s.nseg * s.R;
    Prob& q = p.pr[d];
    q.wide_a = d && s.I % 64 == 0;
    q.wide_b = s.J % 64 == 0;
    const bool ok_a = q.wide_a ? make_tma_blocks(&m.a[d], g.a, a_cols, a_rows, 64, BM / 64, (uint64_t)g.lda * 2)
                               : make_tma_2d(&m.a[d], g.a, BF, 2, a_cols, a_rows, 64, d ? 64 : BM,
                                             CU_TENSOR_MAP_SWIZZLE_128B, (uint64_t)g.lda * 2);
    const bool ok_b = q.wide_b ? make_tma_blocks(&m.b[d], g.b, (uint64_t)s.J, b_rows, 64, pair ? BN / 128 : BN / 64,
                                                 (uint64_t)g.ldb * 2)
                               : make_tma_2d(&m.b[d], g.b, BF, 2, (uint64_t)s.J, b_rows, 64, 64,
                                             CU_TENSOR_MAP_SWIZZLE_128B, (uint64_t)g.ldb * 2);
    if (!ok_a || !ok_b) return cudaErrorInvalidValue;
    for (int i = 0; i < (d ? 3 : 1); ++i) {
      if (g.out[i] == nullptr) continue;   // a segment without an output is skipped
      const uint64_t rows = d && g.splits == 1 ? (uint64_t)g.seg_rows : (uint64_t)g.splits * g.slice_rows;
      if (!make_tma_2d(&m.o[d + i], g.out[i], g.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : BF, g.out_f32 ? 4 : 2,
                       (uint64_t)s.J, rows, 32, 32, g.out_f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    }
    q.g.a_plane = g.a_plane;
    q.g.planes = s.planes;
    q.g.I = s.I;
    q.g.J = s.J;
    q.g.R = s.R;
    q.g.splits = g.splits;
    q.g.slice_rows = g.slice_rows;
    q.g.out_f32 = g.out_f32;
    q.g.accumulate = g.accumulate;
    q.g.seg_pitch = g.seg_pitch;
    q.g.seg_rows = g.seg_rows;
    for (int i = 0; i < 3; ++i) {
      q.g.out[i] = g.out[i];
      q.g.gamma[i] = g.gamma[i];
      q.g.inv_gamma[i] = g.inv_gamma[i];
    }
    q.g.row_scale = g.row_scale;
    q.g.dot_q = g.dot_q;
    q.g.dot_part = g.dot_part;
    q.i_tiles = ceil_div(s.I, pair ? 2 * BM : BM);
    q.j_tiles = ceil_div(s.J, BN);
    q.nk = ceil_div(s.R, BK);
    chain[d] = is_chain(s.planes, s.nseg);
    q.cl = chain_steps(s.planes, s.nseg);
    q.ups = ceil_div(q.nk, q.cl);
    q.units = s.nseg * q.ups;
    if (g.splits < 1 || g.splits > q.units) return cudaErrorInvalidValue;
    tiles[d] = g.splits * q.i_tiles * q.j_tiles;
  }
  p.tiles0 = tiles[0];
  p.tiles = tiles[0] + tiles[1];
  if (p.tiles == 0) return cudaSuccess;
  p.status = status;
  p.wait_cycles = wait_limit_cycles();
  const int kind = chain[1] ? 2 : chain[0] ? (args[0]->sh.planes > 1 ? 2 : 1) : 0;
  const int groups = num_sms() / (pair ? 2 : 1), one = tiles[0] > 0 ? 0 : 1;
  const float* slots = args[one] != nullptr ? args[one]->slots : nullptr;
  if (slots != nullptr && (tiles[0] == 0 || tiles[1] == 0) && args[one]->splits == 1) {
    p.shared = p.tiles % groups;
    p.tiles -= p.shared;
    if (p.shared > 0 && !make_tma_2d(&m.slots, slots, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, BN,
                                     (uint64_t)2 * groups * BM * (pair ? 2 : 1), 32, 32, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  const int mode = tiles[1] == 0 ? 0 : tiles[0] == 0 ? 1 : 2;
  cudaError_t e;
  if (pair)
    e = kind == 0 ? launch_mode<0, 2>(mode, m, p, stream)
                  : kind == 1 ? launch_mode<1, 2>(mode, m, p, stream) : launch_mode<2, 2>(mode, m, p, stream);
  else
    e = kind == 0 ? launch_mode<0, 1>(mode, m, p, stream)
                  : kind == 1 ? launch_mode<1, 1>(mode, m, p, stream) : launch_mode<2, 1>(mode, m, p, stream);
  if (e != cudaSuccess || p.shared == 0) return e;
  const Prob& q = p.pr[one];
  ShareArgs a;
  a.g = q.g;
  if (one == 0) a.g.seg_pitch = 0;
  a.i_tiles = q.i_tiles;
  a.j_tiles = q.j_tiles;
  a.units = q.units;
  a.tile0 = p.tiles;
  a.tiles = p.shared;
  a.groups = groups;
  a.tile_rows = BM * (pair ? 2 : 1);
  a.slots = slots;
  const dim3 grid(p.shared, a.tile_rows / 4), block(256);
  return q.g.out_f32 ? launch_pdl(share_join_kernel<float>, grid, block, 0, stream, a)
                     : launch_pdl(share_join_kernel<bf16>, grid, block, 0, stream, a);
}

}  // namespace mmf
