// mx4_pair.cu -- the 4-bit product for many rows, on CTA pairs.
//
// The arithmetic of mx4_gemm.cu with tcgen05.mma.cta_group::2: a pair's tile is
// 256 x 256, the even CTA holding rows 0..127 of it, the odd one rows
// 128..255.  Each CTA loads its own 128 rows of x (codes and scales, one box)
// and its own 128 weight rows; per SM a 256-element step of K moves 35 KB for
// 128 x 256 x 256 products, half of what 128 x 128 tiles move (at 4 bits the
// delivery from L2 sets the pace long before the tensor core does).  The MMA
// reads both CTAs' codes, but each CTA's scales from its own TMEM: so each
// loads the weight scales of both halves (1 KB more).
//
// TMEM (512 columns): two accumulators of 256 overlap in 64 columns, columns
// [0, 256) and [192, 448), which leaves [448, 496) for two sets of scales.  The
// epilogue drains the shared 64 columns first (each of the two warps of a lane
// quarter 32 of them) and reports them on a barrier of their own: the next
// tile's MMAs start one chunk into the epilogue, not after it.  The
// copies of scales and the MMAs of one thread execute in the order of their
// issue; with two sets in turn a copy need not wait for the MMAs just before
// it.
//
// Persistent clusters of two CTAs, roles as in gemm2sm.cu.  No load uses
// multicast.  Every wait is bounded; a pair that gives up meets at the cluster
// barrier and frees its TMEM.
#include <algorithm>

#include "gemm_common.cuh"
#include "mx4_common.cuh"

namespace w8a8 {
namespace {

constexpr int kPairStages = 5;
constexpr int kTileRows128 = kMxTileBytes / 128;   // a tile as 136 rows of 128 bytes
constexpr int kScaleRows128 = kMxScaleBytes / 128;  // 8
constexpr int kAccOverlap = 64;
constexpr uint32_t kScaleSets = 2, kScaleSetCols = 24;  // x: 2 x 4, weights: 2 x 8
constexpr uint32_t kScaleBase = 512 - kAccOverlap;

struct PairSmem {
  // one stage: tile of x | codes of this CTA's weight rows | weight scales of both halves
  static constexpr int kW = kMxTileBytes;
  static constexpr int kWS = kW + kMxCodeBytes;
  static constexpr int kStageBytes = kWS + 2 * kMxScaleBytes;  // 35 KB
  static constexpr int kOut = kPairStages * kStageBytes;
  static constexpr int kBias = kOut + kEpiWarps * kEpiStagePerWarp;  // 8 x 128 bf16
  static constexpr int kBars = kBias + kEpiWarps * 128 * 2;
  // full[S], empty[S], tfull[2], tempty[2], tshared[2], done
  static constexpr int kMisc = kBars + (2 * kPairStages + 7) * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
};
static_assert(PairSmem::kStageBytes % 1024 == 0 && PairSmem::kAlloc <= 232448, "one CTA's shared memory");
static_assert(kScaleBase + kScaleSets * kScaleSetCols <= 512, "TMEM columns");

// ACT, IMAGE: the activation (a w8a8_act) and the form of the output, fixed so
// that the epilogue's code is short: it runs a few times a launch, and its
// instructions are fetched for each (see mx4_gemm.cu).
template <int ACT, bool IMAGE>
__global__ void __maxnreg__(kGemmRegs)
    mx4_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                    const __grid_constant__ CUtensorMap tmap_ws, const __grid_constant__ CUtensorMap tmap_y,
                    const Mx4Args args) {
  using L = PairSmem;
  constexpr int S = kPairStages;
  constexpr uint32_t kIdesc = idesc_mx4(256, 256);

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *empty = full + S;
  uint64_t *tfull = empty + S;
  uint64_t *tempty = tfull + 2;
  uint64_t *tshared = tempty + 2;
  uint64_t *mma_done = tshared + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: the even CTA, which issues the MMAs
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 2);  // one expect_tx arrival from each CTA
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
      mbar_init(&tshared[b], 2 * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_w);
    prefetch_tmap(&tmap_ws);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int num_tiles = args.tiles_m * args.tiles_n;
  const int slot = (int)(blockIdx.x >> 1), nslots = (int)(gridDim.x >> 1);
  const int my_tiles = slot < num_tiles ? (num_tiles - 1 - slot) / nslots + 1 : 0;
  const int kt = args.kt;
  const uint32_t full0 = map_to_cta(smem_addr(full), 0);
  const uint32_t tempty0 = map_to_cta(smem_addr(tempty), 0);
  const uint32_t tshared0 = map_to_cta(smem_addr(tshared), 0);
  auto acc_col = [](uint32_t b) { return b * (256 - kAccOverlap); };
  auto coords = [&](int i, int &mb, int &nb) {
    const int tile = slot + i * nslots;
    if (args.row_major) {
      mb = tile / args.tiles_n;
      nb = tile - mb * args.tiles_n;
    } else {
      nb = tile / args.tiles_m;
      mb = tile - nb * args.tiles_m;
    }
  };

  if (threadIdx.x == kGemmThreads) {
    // ---------------- producer (both CTAs) ----------------
    struct Cursor {
      int i, k;
      int a, w, w0, w1;  // first 128-byte rows: tile of x, own weight tile, the two weight tiles
    };
    auto enter = [&](int i) {
      Cursor c{i, 0, 0, 0, 0, 0};
      if (i < my_tiles) {
        int mb, nb;
        coords(i, mb, nb);
        c.a = (mb * 2 + (int)rank) * kt * kTileRows128;
        c.w0 = nb * 2 * kt * kTileRows128;
        c.w1 = c.w0 + kt * kTileRows128;
        c.w = rank ? c.w1 : c.w0;
      }
      return c;
    };
    auto load = [&](const Cursor &c, uint32_t s) {
      uint8_t *st = smem + s * L::kStageBytes;
      const uint32_t bar = full0 + s * 8;
      const int k = c.k * kTileRows128;
      mbar_arrive_expect_tx_cluster(bar, L::kStageBytes);
      tma_load_2d_pair(st, &tmap_a, 0, c.a + k, bar);
      tma_load_2d_pair(st + L::kW, &tmap_w, 0, c.w + k, bar);
      tma_load_2d_pair(st + L::kWS, &tmap_ws, 0, c.w0 + k + 128, bar);
      tma_load_2d_pair(st + L::kWS + kMxScaleBytes, &tmap_ws, 0, c.w1 + k + 128, bar);
    };
    const int64_t total = (int64_t)my_tiles * kt;
    Cursor cur = enter(0);
    griddep_wait();
    uint32_t s = 0, ph = 0;
    int64_t issued = 0;
    for (; issued < total; ++issued) {
      if (issued >= S && !mbar_wait(&empty[s], ph ^ 1, abort_flag, args.status)) break;
      load(cur, s);
      if (++cur.k == kt) cur = enter(cur.i + 1);
      if (++s == (uint32_t)S) {
        s = 0;
        ph ^= 1;
      }
    }
    // Every stage this CTA filled is consumed before it may leave: the commits
    // that say so arrive here too (bounded).
    if (issued == total)
      for (int64_t sl = 0; sl < S && sl < issued; ++sl) {
        const int64_t last = sl + ((issued - 1 - sl) / S) * S;
        volatile int no_abort = 0;
        (void)mbar_wait_bounded(&empty[sl], (uint32_t)((last / S) & 1), &no_abort, args.status);
      }
    else if (rank == 0)  // gave up: the pair's copies land before it leaves (bounded)
      for (int64_t sl = 0; sl < S && sl < issued; ++sl) {
        const int64_t last = sl + ((issued - 1 - sl) / S) * S;
        volatile int no_abort = 0;
        (void)mbar_wait_bounded(&full[sl], (uint32_t)((last / S) & 1), &no_abort, args.status);
      }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------- MMA issuer (even CTA) ----------------
      // The whole warp walks the steps and waits; one elected lane issues.
      griddep_wait();  // the bounded waits below start when the data may come
      const bool lead = elect_one();
      const uint64_t a_desc0 = sw128_kmajor_desc(smem), sc_desc0 = mx4_scale_desc(smem);
      const uint32_t sf0 = tmem_base + kScaleBase;
      uint32_t s = 0, ph = 0, step = 0;
      bool ok = true;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, args.status)) != 0;
      };
      for (int i = 0; ok && i < my_tiles; ++i) {
        const uint32_t b = i & 1, bph = (i >> 1) & 1;
        // the accumulator's previous tile is drained, and of the other
        // accumulator's tile the columns they share
        ok = wait(&tempty[b], bph ^ 1) && (i == 0 || wait(&tshared[b ^ 1], ((i - 1) >> 1) & 1));
        if (!ok) break;
        const uint32_t d_tmem = tmem_base + acc_col(b);
        for (int k = 0; k < kt; ++k, ++step) {
          ok = wait(&full[s], ph);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
            // (a descriptor's address field is the shared-memory address / 16:
            // one addition a stage, the rest are constants)
            const uint64_t at = (uint64_t)(s * (L::kStageBytes >> 4));
            const uint64_t a_desc = a_desc0 + at, sc_desc = sc_desc0 + at;
            const uint32_t sfa = sf0 + (step & 1) * kScaleSetCols, sfb = sfa + 8;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              copy_scales_pair(sfa + 4 * g, sc_desc + ((kMxCodeBytes + g * kMxGroupBytes) >> 4));
              copy_scales_pair(sfb + 8 * g, sc_desc + ((L::kWS + g * kMxGroupBytes) >> 4));
              copy_scales_pair(sfb + 8 * g + 4,
                               sc_desc + ((L::kWS + kMxScaleBytes + g * kMxGroupBytes) >> 4));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_mx4_pair(d_tmem, a_desc + 2 * j, a_desc + ((L::kW >> 4) + 2 * j),
                           kIdesc | ((j & 1) ? kMxSecondPair : 0u), sfa + 4 * (j >> 1), sfb + 8 * (j >> 1),
                           (k | j) != 0);
            mma_commit_pair(&empty[s], 0x3);
          }
          __syncwarp();
          if (++s == (uint32_t)S) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok && lead) mma_commit_pair(&tfull[b], 0x3);
        __syncwarp();
      }
      if (lead) {  // nothing in flight when the pair leaves (bounded)
        mma_commit_pair(mma_done, 0x1);
        volatile int no_abort = 0;
        (void)mbar_wait_bounded(mma_done, 0, &no_abort, args.status);
      }
    }
    __syncwarp();
  } else if (warp >= 2 && threadIdx.x < kGemmThreads) {
    // ---------------- epilogue (warps 2..9, both CTAs) ----------------
    griddep_wait();
    const EpiWarp ew(warp);
    uint16_t *s_bias = reinterpret_cast<uint16_t *>(smem + L::kBias) + (warp - 2) * 128;
    uint8_t *stage = smem + L::kOut + (warp - 2) * kEpiStagePerWarp;
    const int n_end = IMAGE ? args.y_kt * kMxTileK : args.N;
    for (int i = 0; i < my_tiles; ++i) {
      int mb, nb;
      coords(i, mb, nb);
      const int row0 = mb * 256 + (int)rank * 128 + ew.quarter * 32;
      const uint32_t b = i & 1, bph = (i >> 1) & 1;
      // this warp's four chunks of 32 columns: one of the shared 64, three of the rest
      const int c_shared = (b ? 0 : 256 - kAccOverlap) + ew.half * 32;
      const int c_rest = (b ? kAccOverlap : 0) + ew.half * 96;
      auto column = [&](int c) { return c == 0 ? c_shared : c_rest + (c - 1) * 32; };
      {
        const int j = lane * 4;  // 4 bias values a lane: chunk j / 32
        const int n = nb * 256 + column(j >> 5) + (j & 31);
        uint2 v = make_uint2(0, 0);
        if (args.bias && n < args.N) v = *reinterpret_cast<const uint2 *>(args.bias + n);
        *reinterpret_cast<uint2 *>(s_bias + j) = v;
      }
      __syncwarp();
      int ok = 0;
      if (lane == 0) ok = mbar_wait(&tfull[b], bph, abort_flag, args.status);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + acc_col(b) + ((uint32_t)(ew.quarter * 32) << 16);
      auto emit = [&](const uint32_t(&v)[32], int c) {
        const int n0 = nb * 256 + column(c);
        if (n0 >= n_end) return;
        uint4 out[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) out[g] = mx4_finish8<ACT>(v + 8 * g, s_bias + c * 32 + 8 * g);
        if constexpr (IMAGE) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (n0 + 8 * g >= args.N) out[g] = make_uint4(0, 0, 0, 0);
          uint4 codes;
          const uint32_t sc = mx4_encode_block(out, codes);
          const int row = row0 + lane;
          if (row < args.M) {
            uint8_t *tile = args.y_image + ((size_t)(row >> 7) * args.y_kt + nb) * kMxTileBytes;
            const int r = row & 127, blk = (n0 & 255) >> 5;
            *reinterpret_cast<uint4 *>(tile + mx4_chunk_offset(r, blk)) = codes;
            tile[mx4_scale_offset(r, blk)] = (uint8_t)sc;
          }
        } else {
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<uint4 *>(stage + swz64_offset(lane, g)) = out[g];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmap_y, stage, n0, row0);
            bulk_commit_group();
          }
        }
      };
      uint32_t v0[32], v1[32];
      tmem_ld_32x32b_x32(taddr + column(0), v0);
      tmem_ld_wait_regs(v0);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tshared0 + b * 8);  // the next tile may start
      tmem_ld_32x32b_x32(taddr + column(1), v1);
      emit(v0, 0);
      __syncwarp();
      tmem_ld_wait_regs(v1);
      tmem_ld_32x32b_x32(taddr + column(2), v0);
      emit(v1, 1);
      __syncwarp();
      tmem_ld_wait_regs(v0);
      tmem_ld_32x32b_x32(taddr + column(3), v1);
      emit(v0, 2);
      __syncwarp();
      tmem_ld_wait_regs(v1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + b * 8);
      emit(v1, 3);
      __syncwarp();
    }
    if (lane == 0) bulk_wait_group_all();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();  // no CTA leaves while its peer may still touch its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

FuncAttrOnce g_mx_pair_attr[4];

}  // namespace

w8a8_status launch_mx4_pair(Mx4Args a, cudaStream_t stream) {
  CUtensorMap ta, tw, tws, ty = {};
  const uint64_t rows_a = (uint64_t)mx4_slabs(a.M) * a.kt * kTileRows128;
  const uint64_t rows_w = (uint64_t)mx4_slabs(a.N) * a.kt * kTileRows128;
  // (128-byte rows past an image read as zeros: the odd CTA's half of a last tile)
  if (!make_tmap_u8_2d_plain(&ta, a.a, rows_a, 128, 128, kTileRows128, 128) ||
      !make_tmap_u8_2d_plain(&tw, a.w, rows_w, 128, 128, 128, 128) ||
      !make_tmap_u8_2d_plain(&tws, a.w, rows_w, 128, 128, kScaleRows128, 128))
    return W8A8_ERR_CUDA;
  if (a.y && !make_tmap_out_bf16(&ty, a.y, (uint64_t)a.M, (uint64_t)a.N)) return W8A8_ERR_CUDA;
  const int form = (a.act != W8A8_ACT_NONE ? 1 : 0) + (a.y_image ? 2 : 0);
  auto k = form == 0   ? mx4_pair_kernel<W8A8_ACT_NONE, false>
           : form == 1 ? mx4_pair_kernel<W8A8_ACT_GELU_TANH, false>
           : form == 2 ? mx4_pair_kernel<W8A8_ACT_NONE, true>
                       : mx4_pair_kernel<W8A8_ACT_GELU_TANH, true>;
  if (g_mx_pair_attr[form].ensure([&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, PairSmem::kAlloc);
      }) != cudaSuccess)
    return W8A8_ERR_CUDA;
  a.tiles_m = (int)(((int64_t)a.M + 255) / 256);
  a.tiles_n = (int)(((int64_t)a.N + 255) / 256);
  a.row_major = a.M > a.N ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::max(1, std::min(a.tiles_m * a.tiles_n, sm_count() / 2))));
  cfg.blockDim = dim3(kGemmThreads + 1);
  cfg.dynamicSmemBytes = (size_t)PairSmem::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, ta, tw, tws, ty, a);
  if (e == cudaSuccess) count_launch();
  return from_cuda(e);
}

}  // namespace w8a8
