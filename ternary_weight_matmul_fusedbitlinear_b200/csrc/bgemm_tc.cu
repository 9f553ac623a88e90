// Training contractions on the 5th-generation tensor cores (tcgen05 kind::f16,
// bf16 operands, fp32 accumulators in tensor memory).
//
// The gradients of a ternary layer y = gamma (q . w) / s are two products
// ("MatMul-free language models", DataCamp blog, "Memory efficiency": the
// models are trained with fused GPU kernels; no formula is printed, these are
// the derivatives with the two roundings passed straight through):
//   dx^[t, k] = gamma sum_n dy[t, n] w[n, k]        form kDx
//   dW [n, k] = sum_t dy[t, n] q[t, k] / s[t]       form kDw
// The ternary codes w, and the int8 codes q, are exact in bf16, so the only
// rounded operand is the gradient (or, for a caller's bf16 gradient, q / s).
// An fp32 gradient comes as three bf16 planes g = g0 + g1 + g2 (24 bits), whose
// products accumulate in the same tensor memory: "planes" extends the
// reduction, plane p's rows of A starting p * a_plane rows further down.
//
// Operands stay as they lie in memory. For kDx the gradient is K-major (its
// reduction index n is contiguous); every other operand has the reduction
// index as its row, i.e. is MN-major, which the MMA takes directly (no
// transposed copies): a 64 x 64 box per 128-byte swizzle column block.
//
// Tile 128 x 256 x 64, persistent, one CTA per SM, 4-stage TMA ring of 48 KB,
// two TMEM accumulators so that a tile's epilogue runs under the next tile's
// main loop. The last column tile shrinks the MMA to the columns there are.
// Too few tiles for the SMs (short batches, small matrices): the reduction is
// cut in `splits` equal ranges, each writing its own fp32 slice for the kernel
// that reads the result to add up in order (no atomics, same result each run).
#include "kernels.cuh"
#include "umma.cuh"

namespace mmf {

namespace {

constexpr int BM = 128, BN = 256, BK = 64, NS = 4;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, BOX_BYTES = 64 * 64 * 2;
constexpr int kEpiWarps = 8, kEpiWarp0 = 2;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kTmemCols = 512;

struct __align__(1024) Smem {
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

__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum)
      : "memory");
}

__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

struct KArgs {
  BGemmArgs g;
  int i_tiles, j_tiles, nk, steps;   // nk: k-steps per plane; steps: planes * nk
  int* status;
  long long wait_cycles;
};

template <bool DW, typename OUT>
__global__ void __launch_bounds__(kThreads, 1)
    bgemm_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_o0, const __grid_constant__ CUtensorMap map_o1,
                    const __grid_constant__ CUtensorMap map_o2, const KArgs p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const int tiles = p.g.splits * p.i_tiles * p.j_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.tmem_full[a], 1);
      mbar_init(&sm.tmem_empty[a], kEpiWarps * 32);
    }
    mbar_init(&sm.mma_drain, 1);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;
  pdl_trigger();
  pdl_wait();

  // tile -> (split, i tile, j tile), j fastest: neighbours share their rows of A
  auto place = [&](int tile, int& sp, int& it, int& jt, int& lo, int& hi) {
    jt = tile % p.j_tiles;
    it = tile / p.j_tiles % p.i_tiles;
    sp = tile / (p.j_tiles * p.i_tiles);
    lo = (int)((long long)p.steps * sp / p.g.splits);
    hi = (int)((long long)p.steps * (sp + 1) / p.g.splits);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        int sp, it, jt, lo, hi;
        place(tile, sp, it, jt, lo, hi);
        const int boxes = min(BN / 64, ceil_div(p.g.J - jt * BN, 64));
        for (int st = lo; st < hi; ++st, ++n) {
          const int s = n % NS;
          const int plane = st / p.nk, r0 = (st % p.nk) * BK;
          if (!mbar_wait(&sm.empty[s], ((n / NS) & 1) ^ 1, abort_flag, p.status, p.wait_cycles)) { ok = false; break; }
          mbar_arrive_expect_tx(&sm.full[s], A_BYTES + boxes * BOX_BYTES);
          if constexpr (DW) {
            tma_load_2d(sm.a[s], &map_a, it * BM, plane * p.g.a_plane + r0, &sm.full[s]);
            tma_load_2d(sm.a[s] + BOX_BYTES, &map_a, it * BM + 64, plane * p.g.a_plane + r0, &sm.full[s]);
          } else {
            tma_load_2d(sm.a[s], &map_a, r0, plane * p.g.a_plane + it * BM, &sm.full[s]);
          }
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(sm.b[s] + b * BOX_BYTES, &map_b, jt * BN + 64 * b, r0, &sm.full[s]);
        }
      }
      // let every copy this thread issued land before the CTA can exit
      for (uint32_t j = (n > NS ? n - NS : 0); j < n; ++j) mbar_drain(&sm.full[j % NS], (j / NS) & 1, p.wait_cycles);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t n = 0, tl = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, ++tl) {
        int sp, it, jt, lo, hi;
        place(tile, sp, it, jt, lo, hi);
        const int acc = tl & 1;
        if (!mbar_wait(&sm.tmem_empty[acc], ((tl >> 1) & 1) ^ 1, abort_flag, p.status, p.wait_cycles)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        const uint32_t idesc = idesc_bf16(BM, min(BN, p.g.J - jt * BN), DW, true);   // J % 16 == 0
        for (int st = lo; st < hi; ++st, ++n) {
          const int s = n % NS;
          if (!mbar_wait(&sm.full[s], (n / NS) & 1, abort_flag, p.status, p.wait_cycles)) { ok = false; break; }
          tc_fence_after();
          const uint64_t ad = DW ? desc_mn_sw128(smem_u32(sm.a[s])) : umma_desc_sw128(smem_u32(sm.a[s]));
          const uint64_t bd = desc_mn_sw128(smem_u32(sm.b[s]));
#pragma unroll
          for (int j = 0; j < BK / 16; ++j)   // 16 reduction steps: 2 row groups (MN-major) or 32 bytes (K-major)
            umma_f16(d_tmem, ad + (uint64_t)(DW ? 128 * j : 2 * j), bd + (uint64_t)(128 * j), idesc,
                     (st > lo) || (j > 0));
          umma_commit(&sm.empty[s]);
        }
        if (ok) umma_commit(&sm.tmem_full[acc]);
      }
      umma_commit(&sm.mma_drain);
      mbar_drain(&sm.mma_drain, 0, p.wait_cycles);
    }
  } else {
    // ------------------------------------------------------------ epilogue (8 warps)
    const int ew = warp - kEpiWarp0;
    const int quarter = warp & 3, group = ew >> 2;
    uint32_t tl = 0;
    int nst = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++tl) {
      int sp, it, jt, lo, hi;
      place(tile, sp, it, jt, lo, hi);
      const int acc = tl & 1;
      const bool got = mbar_wait(&sm.tmem_full[acc], (tl >> 1) & 1, abort_flag, p.status, p.wait_cycles);
      __syncwarp();
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const int i0 = it * BM + quarter * 32;   // this warp's 32 rows of the result
      const int i = i0 + lane;
      // where the rows go: a slice of partial sums, or segment `seg` of the result
      int seg = 0, y = i0;
      float sc = 1.0f;
      if constexpr (DW) {
        if (p.g.splits > 1 || p.g.seg_pitch == 0) {
          y = sp * p.g.slice_rows + i0;
        } else {
          seg = i0 / p.g.seg_pitch;
          y = i0 - seg * p.g.seg_pitch;
        }
        if (p.g.splits == 1 && p.g.inv_gamma[seg < 3 ? seg : 0] != nullptr)
          sc = 1.0f / fold_gamma(*p.g.inv_gamma[seg < 3 ? seg : 0]);
      } else {
        y = sp * p.g.slice_rows + i0;
        if (p.g.gamma != nullptr) sc = *p.g.gamma;
        if (p.g.row_scale != nullptr && i < p.g.I) sc *= p.g.row_scale[i];
      }
      const CUtensorMap* mo = seg == 0 ? &map_o0 : (seg == 1 ? &map_o1 : &map_o2);
      const bool rows_ok = i0 < p.g.I && seg < 3 && p.g.out[seg < 3 ? seg : 0] != nullptr;
      const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * BN;
      for (int c = group * 4; c < group * 4 + 4; ++c) {
        const int j0 = jt * BN + 32 * c;
        if (j0 >= p.g.J || !rows_ok) break;
        uint32_t r[32];
        tmem_ld32(tbase + 32 * c, r);
        float out[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) out[j] = __uint_as_float(r[j]) * sc;
        uint8_t* buf = sm.stage[ew];
        if constexpr (sizeof(OUT) == 2) {
          if (lane == 0) bulk_wait_read_le1();
          buf += (nst & 1) * 2048;
        } else {
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        __syncwarp();
        stage_row(buf, lane, out, (OUT*)nullptr);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (sizeof(OUT) == 4 && p.g.accumulate) tma_add_2d(mo, buf, j0, y);
          else tma_store_2d(mo, buf, j0, y);
        }
        ++nst;
      }
      tc_fence_before();
      mbar_arrive(&sm.tmem_empty[acc]);
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols)
                 : "memory");
  }
}

template <bool DW, typename OUT>
cudaError_t launch_form(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap (&mo)[3], const KArgs& p,
                        cudaStream_t stream) {
  auto kern = bgemm_tc_kernel<DW, OUT>;
  const size_t smem = sizeof(Smem) + 1024;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(p.g.splits * p.i_tiles * p.j_tiles, num_sms());
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, stream, ma, mb, mo[0], mo[1], mo[2], p);
}

}  // namespace

// Splits of the reduction: enough tiles for the SMs, at least 8 k-steps (512
// reduction rows) per split so that a split's fp32 slice costs less than it
// saves, and no more slices than `most`.
int bgemm_splits(int I, int J, int R, int planes, int most) {
  const long long tiles = (long long)ceil_div(I, BM) * ceil_div(J, BN);
  const long long steps = (long long)planes * ceil_div(R, BK);
  long long s = num_sms() / std::max(1LL, tiles);
  s = std::min(s, steps / 8);
  return (int)std::max(1LL, std::min(s, (long long)most));
}

int bgemm_slice_rows(int I) { return ceil_div(I, BM) * BM; }

cudaError_t launch_bgemm_tc(const BGemmArgs& g, int* status, cudaStream_t stream) {
  if (g.I == 0 || g.J == 0) return cudaSuccess;
  CUtensorMap ma, mb, mo[3];
  const uint64_t a_rows = g.dw ? (uint64_t)(g.planes - 1) * g.a_plane + g.R : (uint64_t)(g.planes - 1) * g.a_plane + g.I;
  const uint64_t a_cols = g.dw ? g.I : g.R;
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!make_tma_2d(&ma, g.a, BF, 2, a_cols, a_rows, 64, g.dw ? 64 : BM, CU_TENSOR_MAP_SWIZZLE_128B, (uint64_t)g.lda * 2) ||
      !make_tma_2d(&mb, g.b, BF, 2, (uint64_t)g.J, (uint64_t)g.R, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, (uint64_t)g.ldb * 2))
    return cudaErrorInvalidValue;
  const bool f32 = g.out_f32;
  void* any = g.out[0] != nullptr ? g.out[0] : (g.out[1] != nullptr ? g.out[1] : g.out[2]);
  for (int i = 0; i < 3; ++i) {
    void* base = g.out[i] != nullptr ? g.out[i] : any;   // a segment without an output is skipped
    const uint64_t rows = g.seg_pitch != 0 && g.splits == 1 ? (uint64_t)g.seg_rows : (uint64_t)g.splits * g.slice_rows;
    if (!make_tma_2d(&mo[i], base, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : BF, f32 ? 4 : 2, (uint64_t)g.J, rows, 32, 32,
                     f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  KArgs p;
  p.g = g;
  p.i_tiles = ceil_div(g.I, BM);
  p.j_tiles = ceil_div(g.J, BN);
  p.nk = ceil_div(g.R, BK);
  p.steps = p.nk * g.planes;
  p.status = status;
  p.wait_cycles = wait_limit_cycles();
  if (g.dw) return f32 ? launch_form<true, float>(ma, mb, mo, p, stream) : launch_form<true, bf16>(ma, mb, mo, p, stream);
  return launch_form<false, float>(ma, mb, mo, p, stream);
}

}  // namespace mmf
