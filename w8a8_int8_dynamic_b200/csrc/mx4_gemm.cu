// mx4_gemm.cu -- the product of two microscaled 4-bit images on the sm_100a
// tensor cores, and the entry points of the 4-bit layers.
//
//   y[m, n] = act(sum over blocks of 2^(ea + ew) * sum of 32 qa * qw  + bias[n])
//
// tcgen05.mma kind::mxf4 applies both block scales itself: the codes come from
// shared memory, the scales from TMEM, where tcgen05.cp puts them from the
// same pipeline stage.  A stage is one 256-element tile of either operand,
// codes and scales together (one contiguous copy each, mx4_common.cuh).  The
// accumulators are fp32 in TMEM, double-buffered, and leave through the
// epilogue: bias, optional GELU, one rounding to bf16, then either TMA stores
// of y or, for a layer that feeds another 4-bit layer, the MX codes of y.
// A thread of the epilogue holds 32 consecutive outputs of one row, which is
// one block: its maximum, scale and codes need no other thread.  Activation
// and form of the output are fixed at compile time: with both in one kernel the
// epilogue jumped over the code of the other forms, and fetching instructions
// cost 0.5 to 1 us a launch (256 x 4096 x 4096: 11.3 us, now 10.0).
//
// Scale columns: every stage has its own TMEM columns (16: two groups of four
// for either operand), written when the stage's MMAs are issued, so they are
// overwritten only after the MMAs that read them released the stage.
//
// Persistent, one CTA per SM, roles as in gemm.cu: the producer is a lone
// thread in a last warp, warp 1 issues the copies to TMEM and the MMAs, warps
// 2..9 are the epilogue.  Every wait is bounded.
#include <algorithm>

#include "gemm_common.cuh"
#include "mx4_common.cuh"

namespace w8a8 {
namespace {

constexpr int kMxBN = 128;
constexpr int kMxStages = 6;
constexpr int kMxStageBytes = 2 * kMxTileBytes;  // 34 KB

struct MxSmem {
  static constexpr int kStage = 0;
  static constexpr int kOut = kMxStages * kMxStageBytes;           // 8 x 2 KB output boxes
  static constexpr int kBias = kOut + kEpiWarps * kEpiStagePerWarp;  // 8 x 64 bf16
  static constexpr int kBars = kBias + kEpiWarps * (kMxBN / 2) * 2;
  static constexpr int kMisc = kBars + (2 * kMxStages + 5) * 8;
  static constexpr int kUsed = kMisc + 16;
  static constexpr int kAlloc = kUsed + 1024;
};
static_assert(MxSmem::kAlloc <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void mx4_tile_coords(const Mx4Args &a, int tile, int &mb, int &nb) {
  if (a.row_major) {
    mb = tile / a.tiles_n;
    nb = tile - mb * a.tiles_n;
  } else {
    nb = tile / a.tiles_m;
    mb = tile - nb * a.tiles_m;
  }
}

// ACT, IMAGE: the activation (a w8a8_act) and the form of the output, fixed so
// that the epilogue's code is short.
template <int ACT, bool IMAGE>
__global__ void __maxnreg__(kGemmRegs)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmap_y, const Mx4Args args) {
  using L = MxSmem;
  constexpr uint32_t kScaleCols = 16;                    // TMEM columns of one stage's scales
  constexpr uint32_t kScaleBase = 2 * kMxBN;
  constexpr uint32_t kTmemCols = 512;                    // 2 x 128 + 6 x 16, a power of two
  constexpr uint32_t kIdesc = idesc_mx4(128, kMxBN);

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *empty = full + kMxStages;
  uint64_t *tfull = empty + kMxStages;
  uint64_t *tempty = tfull + 2;
  uint64_t *mma_done = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int num_tiles = args.tiles_m * args.tiles_n;
  const int nslots = (int)gridDim.x, slot = (int)blockIdx.x;
  const int kt = args.kt;
  const int my_tiles = slot < num_tiles ? (num_tiles - 1 - slot) / nslots + 1 : 0;
  const int w_slabs = (args.N + 127) >> 7;

  if (threadIdx.x == kGemmThreads) {
    // ---------------- producer ----------------
    struct Cursor {
      int i, k;
      const uint8_t *a, *w;
    };
    auto enter = [&](int i) {
      Cursor c{i, 0, args.a, args.w};
      if (i < my_tiles) {
        int mb, nb;
        mx4_tile_coords(args, slot + i * nslots, mb, nb);
        // (an image's last 128 columns may have no weight slab: their
        // accumulators are not used, any slab will do)
        nb = min(nb, w_slabs - 1);
        c.a = args.a + (size_t)mb * kt * kMxTileBytes;
        c.w = args.w + (size_t)nb * kt * kMxTileBytes;
      }
      return c;
    };
    auto next = [&](Cursor &c) {
      if (++c.k == kt) {
        c = enter(c.i + 1);
      } else {
        c.a += kMxTileBytes;
        c.w += kMxTileBytes;
      }
    };
    auto weights = [&](const Cursor &c, uint32_t s) {
      bulk_load(smem + s * kMxStageBytes + kMxTileBytes, c.w, kMxTileBytes, &full[s]);
    };
    auto acts = [&](const Cursor &c, uint32_t s) {
      bulk_load(smem + s * kMxStageBytes, c.a, kMxTileBytes, &full[s]);
    };
    const int64_t total = (int64_t)my_tiles * kt;
    const uint32_t pre = total < kMxStages ? (uint32_t)total : (uint32_t)kMxStages;
    int64_t issued = 0;
    Cursor cur = enter(0);
    // before the wait for the preceding kernel, the first weights are only
    // asked into L2 (see mx4_stream.cu)
    if (total > 0) bulk_prefetch_l2(cur.w, (uint32_t)(min(kt, kMxStages) * kMxTileBytes));
    griddep_wait();
    for (uint32_t s = 0; s < pre; ++s) {
      mbar_arrive_expect_tx(&full[s], kMxStageBytes);
      weights(cur, s);
      acts(cur, s);
      next(cur);
    }
    uint32_t s = 0, ph = 1;
    for (issued = pre; issued < total; ++issued) {
      if (!mbar_wait(&empty[s], ph ^ 1, abort_flag, args.status)) break;
      mbar_arrive_expect_tx(&full[s], kMxStageBytes);
      weights(cur, s);
      acts(cur, s);
      next(cur);
      if (++s == (uint32_t)kMxStages) {
        s = 0;
        ph ^= 1;
      }
    }
    // every copy issued has landed before the CTA leaves (bounded)
    for (int64_t sl = 0; sl < kMxStages && sl < issued; ++sl) {
      const int64_t last = sl + ((issued - 1 - sl) / kMxStages) * kMxStages;
      volatile int no_abort = 0;
      (void)mbar_wait_bounded(&full[sl], (uint32_t)((last / kMxStages) & 1), &no_abort, args.status);
    }
  } else if (warp == 0) {
    // idle
  } else if (warp == 1) {
    // ---------------- MMA issuer: the warp waits, one elected lane issues ----
    griddep_wait();  // the bounded waits below start when the data may come
    const bool lead = elect_one();
    const uint64_t a_desc0 = sw128_kmajor_desc(smem), sc_desc0 = mx4_scale_desc(smem);
    uint32_t s = 0, ph = 0;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, args.status)) != 0;
    };
    for (int i = 0; ok && i < my_tiles; ++i) {
      const uint32_t b = i & 1, bph = (i >> 1) & 1;
      ok = wait(&tempty[b], bph ^ 1);
      if (!ok) break;
      const uint32_t d_tmem = tmem_base + b * kMxBN;
      for (int k = 0; k < kt; ++k) {
        ok = wait(&full[s], ph);
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          // (a descriptor's address field is the shared-memory address / 16)
          const uint64_t at = (uint64_t)(s * (kMxStageBytes >> 4));
          const uint64_t a_desc = a_desc0 + at, sc_desc = sc_desc0 + at;
          const uint32_t sfa = tmem_base + kScaleBase + s * kScaleCols, sfb = sfa + 8;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            copy_scales(sfa + 4 * g, sc_desc + ((kMxCodeBytes + g * kMxGroupBytes) >> 4));
            copy_scales(sfb + 4 * g, sc_desc + ((kMxTileBytes + kMxCodeBytes + g * kMxGroupBytes) >> 4));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_mx4(d_tmem, a_desc + 2 * j, a_desc + ((kMxTileBytes >> 4) + 2 * j),
                    kIdesc | ((j & 1) ? kMxSecondPair : 0u), sfa + 4 * (j >> 1), sfb + 4 * (j >> 1),
                    (k | j) != 0);
          mma_commit(&empty[s]);
        }
        __syncwarp();
        if (++s == (uint32_t)kMxStages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (ok && lead) mma_commit(&tfull[b]);
      __syncwarp();
    }
    if (lead) {  // nothing of this CTA is in flight when it leaves (bounded)
      mma_commit(mma_done);
      volatile int no_abort = 0;
      (void)mbar_wait_bounded(mma_done, 0, &no_abort, args.status);
    }
    __syncwarp();
  } else {
    // ---------------- epilogue (warps 2..9) ----------------
    griddep_wait();
    constexpr int kCols = kMxBN / 2;
    const EpiWarp ew(warp);
    uint16_t *s_bias = reinterpret_cast<uint16_t *>(smem + L::kBias) + (warp - 2) * kCols;
    uint8_t *stage = smem + L::kOut + (warp - 2) * kEpiStagePerWarp;
    const int n_end = IMAGE ? args.y_kt * kMxTileK : args.N;
    for (int i = 0; i < my_tiles; ++i) {
      int mb, nb;
      mx4_tile_coords(args, slot + i * nslots, mb, nb);
      const int row0 = mb * 128 + ew.quarter * 32;
      const int n0 = nb * kMxBN + ew.half * kCols;
      const uint32_t b = i & 1, bph = (i >> 1) & 1;
      for (int j = lane * 8; j < kCols; j += 256) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (args.bias && n0 + j < args.N) v = *reinterpret_cast<const uint4 *>(args.bias + n0 + j);
        *reinterpret_cast<uint4 *>(s_bias + j) = v;
      }
      __syncwarp();
      int ok = 0;
      if (lane == 0) ok = mbar_wait(&tfull[b], bph, abort_flag, args.status);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + b * kMxBN + ew.half * kCols + ((uint32_t)(ew.quarter * 32) << 16);
      for_tmem_chunks<kCols / 32>(
          taddr, [&](int c) { return n0 + c * 32 < n_end; },
          [&](const uint32_t(&v)[32], int c) {
            uint4 out[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) out[g] = mx4_finish8<ACT>(v + 8 * g, s_bias + c * 32 + 8 * g);
            const int nc = n0 + c * 32;
            if constexpr (IMAGE) {
#pragma unroll
              for (int g = 0; g < 4; ++g)
                if (nc + 8 * g >= args.N) out[g] = make_uint4(0, 0, 0, 0);
              uint4 codes;
              const uint32_t sc = mx4_encode_block(out, codes);
              const int row = row0 + lane;
              if (row < args.M) {
                uint8_t *tile = args.y_image + ((size_t)mb * args.y_kt + (nc >> 8)) * kMxTileBytes;
                const int r = row & 127, blk = (nc & 255) >> 5;
                *reinterpret_cast<uint4 *>(tile + mx4_chunk_offset(r, blk)) = codes;
                tile[mx4_scale_offset(r, blk)] = (uint8_t)sc;
              }
            } else {
              if (lane == 0) bulk_wait_group_read<0>();  // the box's previous store
              __syncwarp();
#pragma unroll
              for (int g = 0; g < 4; ++g)
                *reinterpret_cast<uint4 *>(stage + swz64_offset(lane, g)) = out[g];
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&tmap_y, stage, nc, row0);
                bulk_commit_group();
              }
            }
          });
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
    }
    if (lane == 0) bulk_wait_group_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

FuncAttrOnce g_mx_smem_attr[4];

w8a8_status launch_mx4_1sm(const CUtensorMap &ty, Mx4Args a, cudaStream_t stream) {
  const int form = (a.act != W8A8_ACT_NONE ? 1 : 0) + (a.y_image ? 2 : 0);
  auto k = form == 0   ? mx4_gemm_kernel<W8A8_ACT_NONE, false>
           : form == 1 ? mx4_gemm_kernel<W8A8_ACT_GELU_TANH, false>
           : form == 2 ? mx4_gemm_kernel<W8A8_ACT_NONE, true>
                       : mx4_gemm_kernel<W8A8_ACT_GELU_TANH, true>;
  if (g_mx_smem_attr[form].ensure([&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, MxSmem::kAlloc);
      }) != cudaSuccess)
    return W8A8_ERR_CUDA;
  a.tiles_m = (int)mx4_slabs(a.M);
  // an output image's columns are written to the end of its last tile
  a.tiles_n = a.y_image ? a.y_kt * (kMxTileK / kMxBN) : (int)mx4_slabs(a.N);
  if ((int64_t)a.tiles_m * a.tiles_n > 0x7FFFFFFF) return W8A8_ERR_UNSUPPORTED_SHAPE;
  a.row_major = a.M > a.N ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(a.tiles_m * a.tiles_n, sm_count()));
  cfg.blockDim = dim3(kGemmThreads + 1);
  cfg.dynamicSmemBytes = MxSmem::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, ty, a);
  if (e == cudaSuccess) count_launch();
  return from_cuda(e);
}

// Up to 64 rows the weight stream sets the time (mx4_stream.cu).  Up to 128 it
// is worth its longer end where clusters that split K save 18 steps of it or
// more (us, stream and single CTAs, 128 rows: N = 5120, K = 13824 15.1, 18.3;
// 1024, 8192 8.6, 11.9; 2048, 6144, which saves 18, 8.2, 9.9; 8192, 8192, 16,
// 14.0, 13.5; 5120, 5120, 13, 10.9, 10.0).
bool use_stream(const Mx4Args &a) {
  const int p = forced_path();
  if (p != 0 || a.M > kStreamRows) return p == 2;
  if (a.M <= 64) return true;
  const int C = (int)std::min<int64_t>(kMaxStreamCluster, sm_count() / mx4_slabs(a.N));
  return C > 1 && a.kt - (a.kt + C - 1) / C >= 18;
}

// Pairs with 256 x 256 tiles or single CTAs with 128 x 128 ones: by the rounds
// of tiles, a step of K taking 0.365 us in the one and 0.27 us in the other
// when all SMs are busy, and 1 us more to start and end the pair kernel.
// Measured (pair, single): 512 x 4096 x 4096 13.7, 11.2 us; 1024 x 4096 x 4096
// 14.4, 16.8; 256 x 12288 x 4096 13.2, 15.0; 300 x 5120 x 13824 23.2, 19.7;
// 2048^3 9.9, 10.3; 128 x 27648 x 5120 23.1, 20.2; 4096 x 12288 x 4096 76, 98.
bool use_pair(const Mx4Args &a) {
  const int p = forced_path();
  // (the pair kernel's box coordinates are 32-bit rows of 128 bytes)
  const int64_t most = (std::max(mx4_slabs(a.M), mx4_slabs(a.N)) + 2) * a.kt * (kMxTileBytes / 128);
  if (most > 0x7FFFFFFF || (p != 0 && p != 5 && p != 7)) return false;
  if (p != 0) return true;
  auto rounds = [](int64_t tiles, int64_t slots) { return (double)((tiles + slots - 1) / slots); };
  const int64_t sms = sm_count();
  const double pair = rounds((((int64_t)a.M + 255) / 256) * (((int64_t)a.N + 255) / 256), sms / 2) * a.kt * 0.365 + 1.0;
  const double single = rounds(mx4_slabs(a.M) * mx4_slabs(a.N), sms) * a.kt * 0.27;
  return pair < single;
}

// x (with ldx; a layer of few rows): quantised by the product itself, in place of a_image.
w8a8_status launch_mx4(const void *a_image, const void *w_image, const void *bias, void *y,
                       void *y_image, int64_t M, int64_t N, int64_t K, int act, const void *x,
                       int64_t ldx, cudaStream_t stream) {
  Mx4Args a{};
  a.a = static_cast<const uint8_t *>(a_image);
  a.w = static_cast<const uint8_t *>(w_image);
  a.bias = static_cast<const uint16_t *>(bias);
  a.y = static_cast<uint16_t *>(y);
  a.y_image = static_cast<uint8_t *>(y_image);
  a.M = (int)M;
  a.N = (int)N;
  a.kt = (int)mx4_ktiles(K);
  a.y_kt = (int)mx4_ktiles(N);
  a.act = act;
  a.status = status_word();
  if (!a.status) return W8A8_ERR_CUDA;
  if (forced_path() == 2 && M > kStreamRows) return W8A8_ERR_INVALID_ARG;
  if (x || use_stream(a)) return launch_mx4_stream(a, x, ldx, K, stream);
  if (use_pair(a)) return launch_mx4_pair(a, stream);
  CUtensorMap ty = {};
  if (y && !make_tmap_out_bf16(&ty, y, (uint64_t)M, (uint64_t)N)) return W8A8_ERR_CUDA;
  return launch_mx4_1sm(ty, a, stream);
}

// The checks that every product shares.  `image`: the output is an image (the
// next product's left operand, whose K is this N).
w8a8_status check_product(const void *w_image, const void *bias, const void *y, const void *y_image,
                          bool image, int64_t M, int64_t N, int64_t K, int act) {
  if (!w_image || (image ? !y_image : !y) || M < 1 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFFF ||
      K < 1 || (act != W8A8_ACT_NONE && act != W8A8_ACT_GELU_TANH))
    return W8A8_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > kMaxK || N % (image ? 16 : 8) != 0 || (image && N > kMaxK))
    return W8A8_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(w_image) || (bias && !aligned16(bias)) || !aligned16(image ? y_image : y))
    return W8A8_ERR_ALIGNMENT;
  return W8A8_OK;
}

bool overlap(const void *p, size_t np, const void *q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + nq && b < a + np;
}

size_t output_bytes(bool image, int64_t M, int64_t N) {
  return image ? (size_t)mx4_image_bytes(M, N) : (size_t)M * N * 2;
}

// What a product writes while it still reads its operands.
bool over_weights(const void *out, size_t bytes, const void *w_image, const void *bias, int64_t N, int64_t K) {
  return overlap(out, bytes, w_image, (size_t)mx4_image_bytes(N, K)) || overlap(out, bytes, bias, (size_t)N * 2);
}

w8a8_status product(const void *a_image, const void *w_image, const void *bias, void *y, void *y_image,
                    size_t y_image_bytes, bool image, int64_t M, int64_t N, int64_t K, int act,
                    w8a8_stream_t stream) {
  if (!a_image) return W8A8_ERR_INVALID_ARG;
  if (const w8a8_status s = check_product(w_image, bias, y, y_image, image, M, N, K, act)) return s;
  if (!aligned16(a_image)) return W8A8_ERR_ALIGNMENT;
  if (image && y_image_bytes < (size_t)mx4_image_bytes(M, N)) return W8A8_ERR_BUFFER_TOO_SMALL;
  const void *out = image ? y_image : y;
  const size_t out_bytes = output_bytes(image, M, N);
  if (overlap(out, out_bytes, a_image, (size_t)mx4_image_bytes(M, K)) ||
      over_weights(out, out_bytes, w_image, bias, N, K))
    return W8A8_ERR_INVALID_ARG;
  return launch_mx4(a_image, w_image, bias, image ? nullptr : y, image ? y_image : nullptr, M, N, K,
                    act, nullptr, 0, reinterpret_cast<cudaStream_t>(stream));
}

// A layer's workspace: the image of x, which up to 16 rows the product forms
// itself (whatever path is set).
int64_t layer_workspace_bytes(int64_t M, int64_t K) {
  return M <= kStreamQuantRows ? 0 : mx4_image_bytes(M, K);
}

w8a8_status layer(const void *x, int64_t ldx, const void *w_image, const void *bias, void *y,
                  void *y_image, size_t y_image_bytes, bool image, int64_t M, int64_t N, int64_t K,
                  int act, void *workspace, size_t ws_bytes, w8a8_stream_t stream) {
  if (!x || ldx < K) return W8A8_ERR_INVALID_ARG;
  if (const w8a8_status s = check_product(w_image, bias, y, y_image, image, M, N, K, act)) return s;
  if (!aligned16(x) || ldx % 8 != 0 || !aligned16(workspace)) return W8A8_ERR_ALIGNMENT;
  if ((image && y_image_bytes < (size_t)mx4_image_bytes(M, N)) ||
      (workspace ? ws_bytes : 0) < (size_t)layer_workspace_bytes(M, K))
    return W8A8_ERR_BUFFER_TOO_SMALL;
  const void *out = image ? y_image : y;
  const size_t out_bytes = output_bytes(image, M, N), a_bytes = (size_t)mx4_image_bytes(M, K);
  const size_t x_bytes = (size_t)((M - 1) * ldx + K) * 2;
  // A layer in place: the kernel that quantises x itself would write y where
  // other CTAs still read x, so x is quantised first, as with more rows.
  const bool fused = M <= kStreamQuantRows && !overlap(out, out_bytes, x, x_bytes);
  if (over_weights(out, out_bytes, w_image, bias, N, K) ||
      (!fused && ((workspace ? ws_bytes : 0) < a_bytes || overlap(workspace, a_bytes, x, x_bytes) ||
                  overlap(workspace, a_bytes, out, out_bytes))))
    return W8A8_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!fused)
    if (const w8a8_status r = launch_mx4_quant(x, M, K, ldx, workspace, s)) return r;
  return launch_mx4(workspace, w_image, bias, image ? nullptr : y, image ? y_image : nullptr, M, N, K, act,
                    fused ? x : nullptr, ldx, s);
}

}  // namespace
}  // namespace w8a8

using namespace w8a8;

extern "C" {

w8a8_status w8a8_mx4_scaled_mm(const void *a_image, const void *w_image, const void *bias, void *y,
                               int64_t M, int64_t N, int64_t K, int act, w8a8_stream_t stream) {
  return product(a_image, w_image, bias, y, nullptr, 0, false, M, N, K, act, stream);
}

w8a8_status w8a8_mx4_scaled_mm_quant(const void *a_image, const void *w_image, const void *bias,
                                     void *y_image, size_t y_image_bytes, int64_t M, int64_t N,
                                     int64_t K, int act, w8a8_stream_t stream) {
  return product(a_image, w_image, bias, nullptr, y_image, y_image_bytes, true, M, N, K, act, stream);
}

w8a8_status w8a8_mx4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t *bytes) {
  if (!bytes || M < 1 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFFF || K < 1) return W8A8_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > kMaxK || N % 8 != 0) return W8A8_ERR_UNSUPPORTED_SHAPE;
  *bytes = (size_t)layer_workspace_bytes(M, K);
  return W8A8_OK;
}

w8a8_status w8a8_mx4_linear(const void *x, int64_t ldx, const void *w_image, const void *bias, void *y,
                            int64_t M, int64_t N, int64_t K, int act, void *workspace, size_t ws_bytes,
                            w8a8_stream_t stream) {
  return layer(x, ldx, w_image, bias, y, nullptr, 0, false, M, N, K, act, workspace, ws_bytes, stream);
}

w8a8_status w8a8_mx4_linear_quant(const void *x, int64_t ldx, const void *w_image, const void *bias,
                                  void *y_image, size_t y_image_bytes, int64_t M, int64_t N, int64_t K,
                                  int act, void *workspace, size_t ws_bytes, w8a8_stream_t stream) {
  return layer(x, ldx, w_image, bias, nullptr, y_image, y_image_bytes, true, M, N, K, act, workspace,
               ws_bytes, stream);
}

}  // extern "C"
