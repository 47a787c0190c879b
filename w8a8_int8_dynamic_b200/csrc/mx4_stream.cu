// mx4_stream.cu -- the 4-bit product for few rows: every SM streams its share
// of the weights.
//
// With few rows (M <= 64, and to 128 where K is long and there are few slabs)
// the weights are most of the bytes, so they set the time.
// Swap-AB: a 128-row weight tile is the MMA's M operand and the rows of x (16,
// 32, 64 or 128 of them) its N operand.  A pipeline stage is one weight tile
// (17 KB, one copy, codes and scales) and the rows' codes of the same 256
// elements.  From 64 rows on the epilogue has two sets of four warps, which
// take the chunks of 16 rows in turn (128 x 27648 x 5120 26.1 us, now 20.8).
//
// Work split: a cluster of C CTAs (1 to 4) takes a 128-row weight slab,
// each CTA a C-th of its K; clusters are persistent over the slabs.  The
// partial sums are joined through distributed shared memory: the rows of x are
// finished in chunks of 16, chunk q by the CTA of rank q mod C; the others send
// it those columns of their accumulators, and it adds the C parts in rank
// order.  So equal calls
// give equal bits, and no workspace, counter or fence in global memory is
// needed.  (Slabs split evenly over all SMs and joined through global memory
// had a tail of 3 to 7 us: 13 x 5120 x 13824 took 15.7 us in a graph.)
//
// QUANT (the layer, M <= 16): x comes as bf16 and eight more warps form its
// codes and scales, a block of 32 in one lane, straight into the pipeline
// stage: no quantisation launch, no image of x in memory.  Each CTA forms the
// tiles that it needs.
//
// Before the wait for the preceding kernel of the stream, whose output x (or
// even the weights) may be, the first weight tiles are only asked into L2,
// where they are coherent; every read and write follows the wait.
#include <algorithm>
#include <atomic>

#include "gemm_common.cuh"
#include "mx4_common.cuh"

namespace w8a8 {
namespace {

template <int NT>
struct StreamCfg {
  static constexpr int kStages = NT == 16 ? 9 : NT == 32 ? 8 : NT == 64 ? 7 : 4;
  static constexpr int kSets = NT >= 64 ? 2 : 1;  // of four epilogue warps
  static constexpr int kThreads = 64 + 128 * kSets;
  static constexpr int kQ = kMxTileBytes;             // codes of NT rows of x
  static constexpr int kS = kQ + NT * 128;            // their scales
  static constexpr int kStageBytes = kS + kMxScaleBytes;  // a multiple of 1024
  static constexpr int kRecv = kStages * kStageBytes;  // the parts of the cluster's CTAs
  static constexpr int kChunks = NT == 128 ? 9 : 4;  // C * ceil(NT / 16 / C) of them at most
  static constexpr int kBars = kRecv + kChunks * 16 * 128 * 4;
  // full[S], empty[S], tfull[2], tempty[2], recv, sent, done
  static constexpr int kMisc = kBars + (2 * kStages + 7) * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  // TMEM: two accumulators of NT columns, then each stage's scale columns
  static constexpr uint32_t kTmemCols = NT == 128 ? 512 : 256;
  static_assert(kStageBytes % 1024 == 0 && kAlloc <= 232448 && 2 * NT + kStages * 16 <= (int)kTmemCols,
                "one CTA's shared memory and TMEM");
};

struct StreamArgs {
  Mx4Args p;          // p.a: the image of x, without QUANT
  const uint16_t *x;  // QUANT
  int64_t ldx;
  int K;
  int C;              // CTAs of a cluster: 1 to 4
  int slabs;          // 128-row slabs of the weight
};

// Bytes a microsecond that DRAM delivers, and that one SM's copies do.
constexpr double kDramBytesPerUs = 6.5e6, kSmBytesPerUs = 8e4, kJoinUs = 1.0;

// A CTA's weight tiles asked into L2 before the wait for the preceding kernel:
// half of its own, at most 16 (40 MB in all).  More take DRAM time from that
// kernel's own last reads, fewer leave DRAM idle in the change (1 row, product
// on codes: 8192 x 8192, all / half / 4 tiles 10.2, 9.6, 9.8 us; 27648 x 5120,
// at most 16 / 8 / 4 tiles 12.6, 13.0, 14.1).
constexpr int kPrefetchTiles = 16;
constexpr int kQuantWarps = 8;

// ---- distributed shared memory -------------------------------------------------
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
// A phase known to be complete, acquired at cluster scope.
__device__ __forceinline__ bool acquire_cluster(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return __all_sync(0xFFFFFFFFu, done != 0) != 0;
}
__device__ __forceinline__ void arrive_release_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// One row of a slab's 128 outputs into the image of y: the warp's 32 values
// (bf16 bits, zero past N) are one block.
__device__ __noinline__ void image_row(const Mx4Args &p, int row, int nb, int quarter, int lane,
                                       uint32_t bits) {
  uint8_t *tile = p.y_image + (size_t)(nb >> 1) * kMxTileBytes;
  const int blk = (nb & 1) * 4 + quarter;
  const bool pad = !(nb & 1) && (nb + 1) * 128 >= p.N;  // the tile's other half has no slab
  const uint32_t code = mx4_scale_code(__reduce_max_sync(0xFFFFFFFFu, bits & 0x7FFFu));
  uint32_t word = mx4_code1(__uint_as_float(bits << 16), code) << (4 * (lane & 7));
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
  if ((lane & 7) == 0) {
    *reinterpret_cast<uint32_t *>(tile + mx4_chunk_offset(row, blk) + (lane >> 3) * 4) = word;
    if (pad) *reinterpret_cast<uint32_t *>(tile + mx4_chunk_offset(row, blk + 4) + (lane >> 3) * 4) = 0u;
  }
  if (lane == 0) {
    tile[mx4_scale_offset(row, blk)] = (uint8_t)code;
    if (pad) tile[mx4_scale_offset(row, blk + 4)] = 0;
  }
  __syncwarp();
}

template <int NT, bool QUANT>
__global__ void __launch_bounds__(StreamCfg<NT>::kThreads + (QUANT ? 32 * kQuantWarps : 0), 1)
    mx4_stream_kernel(const StreamArgs args) {
  using L = StreamCfg<NT>;
  constexpr int S = L::kStages;
  constexpr uint32_t kIdesc = idesc_mx4(128, NT);
  // A quantising warp has seen the MMAs of the stage's round before last end
  // (its own last tile waited for later ones), which a barrier's parity needs.
  static_assert(!QUANT || kQuantWarps <= S, "quantising warps and the ring");

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *empty = full + S;
  uint64_t *tfull = empty + S;
  uint64_t *tempty = tfull + 2;
  uint64_t *recv = tempty + 2;  // the other CTAs' parts of a slab are in
  uint64_t *sent = recv + 1;    // the other CTAs have read what this one sent
  uint64_t *mma_done = sent + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = args.C;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], QUANT ? 2 : 1);  // the copies; the codes of x
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4 * L::kSets);
    }
    mbar_init(recv, 4 * L::kSets * (C > 1 ? C - 1 : 1));
    mbar_init(sent, 4 * L::kSets * (C > 1 ? C - 1 : 1));
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, L::kTmemCols);
  tc_fence_before();
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int kt = args.p.kt;
  const int k_begin = (int)((int64_t)kt * rank / C), k_end = (int)((int64_t)kt * (rank + 1) / C);
  const int nk = k_end - k_begin;  // tiles of a slab for this CTA: at least one, as C <= kt
  const int first = (int)blockIdx.x / C, step = (int)gridDim.x / C;
  const int nseg = first < args.slabs ? (args.slabs - 1 - first) / step + 1 : 0;
  const int64_t total = (int64_t)nseg * nk;

  auto wait_all = [&](uint64_t *bar, uint32_t parity) {  // by a whole warp
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, args.p.status)) != 0;
  };
  if (warp == 0) {
    // ---------------- producer: the warp waits, one elected lane issues ----
    const bool lead = elect_one();
    const uint64_t evict_first = policy_evict_first();
    const size_t slab_bytes = (size_t)kt * kMxTileBytes;
    const uint8_t *w0 = args.p.w + (size_t)first * slab_bytes + (size_t)k_begin * kMxTileBytes;
    // before the wait: DRAM to L2 only, in the order of the copies
    if (lead)
      for (int64_t i = 0, left = min((int64_t)kPrefetchTiles, (total + 1) / 2); i < nseg && left > 0; ++i, left -= nk)
        bulk_prefetch_l2(w0 + (size_t)i * step * slab_bytes,
                         (uint32_t)(min((int64_t)nk, left) * kMxTileBytes));
    __syncwarp();
    griddep_wait();
    uint32_t s = 0, ph = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int i = 0; ok && i < nseg; ++i) {
      const uint8_t *w = w0 + (size_t)i * step * slab_bytes;
      for (int k = 0; k < nk; ++k, ++issued) {
        ok = issued < S || wait_all(&empty[s], ph ^ 1);
        if (!ok) break;
        if (lead) {
          uint8_t *st = smem + s * L::kStageBytes;
          mbar_arrive_expect_tx(&full[s], kMxTileBytes + (QUANT ? 0 : NT * 128 + kMxScaleBytes));
          bulk_load_hint(st, w + (size_t)k * kMxTileBytes, kMxTileBytes, &full[s], evict_first);
          if (!QUANT) {
            const uint8_t *t = args.p.a + (size_t)(k_begin + k) * kMxTileBytes;
            bulk_load(st + L::kQ, t, NT * 128, &full[s]);
            bulk_load(st + L::kS, t + kMxCodeBytes, kMxScaleBytes, &full[s]);
          }
        }
        __syncwarp();
        if (++s == (uint32_t)S) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // Every copy issued lands before the CTA leaves, whatever gave up.  (With
    // QUANT a stage whose codes never came stays incomplete: bounded too.)
    if (lead)
      for (int64_t sl = 0; sl < S && sl < issued; ++sl) {
        const int64_t last = sl + ((issued - 1 - sl) / S) * S;
        volatile int no_abort = 0;
        (void)mbar_wait_bounded(&full[sl], (uint32_t)((last / S) & 1), &no_abort, args.p.status);
      }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer: the warp waits, one elected lane issues ----
    griddep_wait();  // the bounded waits below start when the data may come
    const bool lead = elect_one();
    const uint64_t desc0 = sw128_kmajor_desc(smem), sc_desc0 = mx4_scale_desc(smem);
    uint32_t s = 0, ph = 0;
    bool ok = true;
    for (int i = 0; ok && i < nseg; ++i) {
      const uint32_t b = i & 1, bph = (i >> 1) & 1;
      ok = wait_all(&tempty[b], bph ^ 1);
      if (!ok) break;
      const uint32_t d_tmem = tmem_base + b * NT;
      for (int k = 0; k < nk; ++k) {
        ok = wait_all(&full[s], ph);
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          // (a descriptor's address field is the shared-memory address / 16)
          const uint64_t at = (uint64_t)(s * (L::kStageBytes >> 4));
          const uint64_t wd = desc0 + at, sd = sc_desc0 + at;
          const uint32_t sfw = tmem_base + 2 * NT + s * 16, sfq = sfw + 8;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            copy_scales(sfw + 4 * g, sd + ((kMxCodeBytes + g * kMxGroupBytes) >> 4));
            copy_scales(sfq + 4 * g, sd + ((L::kS + g * kMxGroupBytes) >> 4));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_mx4(d_tmem, wd + 2 * j, wd + ((L::kQ >> 4) + 2 * j),
                    kIdesc | ((j & 1) ? kMxSecondPair : 0u), sfw + 4 * (j >> 1), sfq + 4 * (j >> 1),
                    (k | j) != 0);
          mma_commit(&empty[s]);
        }
        __syncwarp();
        if (++s == (uint32_t)S) {
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
      (void)mbar_wait_bounded(mma_done, 0, &no_abort, args.p.status);
    }
    __syncwarp();
  } else if (warp < L::kThreads / 32) {
    // ---- epilogue (one or two sets of four warps): one output column per thread ----
    griddep_wait();
    const int quarter = warp & 3, set = (warp - 2) >> 2;
    const int n_local = quarter * 32 + lane;
    const int M = args.p.M, N = args.p.N;
    // 16 rows of x a chunk; chunk q is finished by the CTA of rank q % C
    const int chunks = (M + 15) >> 4;
    // parts[chunk / C][rank][16][128]
    float *parts = reinterpret_cast<float *>(smem + L::kRecv) + n_local;
    const uint32_t parts_addr = smem_addr(parts);
    const uint32_t recv_addr = smem_addr(recv), sent_addr = smem_addr(sent);
    for (int i = 0; i < nseg; ++i) {
      const int nb = first + i * step;
      const uint32_t b = i & 1, bph = (i >> 1) & 1;
      const int n = nb * 128 + n_local;
      const float bv =
          (args.p.bias && n < N) ? __uint_as_float((uint32_t)args.p.bias[n] << 16) : 0.0f;
      if (!wait_all(&tfull[b], bph)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + b * NT;
      // the parts that other CTAs finish go to them
      if (C > 1) {
        // (they have read the previous ones)
        if (i > 0 && !(wait_all(sent, (uint32_t)(i - 1) & 1) && acquire_cluster(sent, (uint32_t)(i - 1) & 1))) break;
        for (int q = set; q < chunks; q += L::kSets) {
          const int to = q % C;
          if (to == rank) continue;
          uint32_t v[16];
          tmem_ld_32x32b_x16(taddr + q * 16, v);
          tmem_ld_wait();
          const uint32_t at = map_to_cta(parts_addr, (uint32_t)to) +
                              (uint32_t)((q / C * C + rank) * (16 * 512));
#pragma unroll
          for (int m = 0; m < 16; ++m)
            if (q * 16 + m < M) st_cluster_f32(at + m * 512, __uint_as_float(v[m]));
        }
        fence_cluster();
        __syncwarp();
        if (lane < C && lane != rank) arrive_release_cluster(map_to_cta(recv_addr, (uint32_t)lane));
        if (!(wait_all(recv, (uint32_t)i & 1) && acquire_cluster(recv, (uint32_t)i & 1))) break;
      }
      // Few rows: a short loop, since this code runs once a slab and unrolled
      // over all 16 rows its instructions take longer to fetch than to execute
      // (1 x 4096 x 4096: 7.3 us, four rows at a time 6.5).  With more rows the
      // latencies of a short loop cost more (64 x 27648 x 5120: two rows at a
      // time 22.7 us, eight 20.0, sixteen 18.2).
      for (int q = rank + set * C; q < chunks; q += L::kSets * C) {
        const int m0 = q * 16, rows = min(16, M - m0);
        float *part = parts + (C > 1 ? q / C * C : set) * (16 * 128);
        {
          uint32_t v[16];
          tmem_ld_32x32b_x16(taddr + m0, v);
          tmem_ld_wait();
#pragma unroll
          for (int m = 0; m < 16; ++m)
            if (m < rows) part[(rank * 16 + m) * 128] = __uint_as_float(v[m]);
        }
        uint16_t *y = args.p.y + (int64_t)m0 * N + n;
        constexpr int kRows = NT == 16 ? 4 : 16;  // at a time
#pragma unroll 1
        for (int m = 0; m < rows; m += kRows) {
          float t[kRows];
#pragma unroll
          for (int j = 0; j < kRows; ++j) t[j] = 0.0f;
          // the parts in rank order (rows past the last one are not used)
          for (int r = 0; r < C; ++r)
#pragma unroll
            for (int j = 0; j < kRows; ++j) t[j] += part[(r * 16 + m + j) * 128];
#pragma unroll
          for (int j = 0; j < kRows; ++j) t[j] = __fadd_rn(t[j], bv);
          if (args.p.act != W8A8_ACT_NONE) {
#pragma unroll
            for (int j = 0; j < kRows; j += 2) apply_act_pair(t[j], t[j + 1], args.p.act);
          }
#pragma unroll
          for (int j = 0; j < kRows; j += 2) {
            const uint32_t out = n < N ? pack_bf16x2(t[j], t[j + 1]) : 0u;
            const bool one = m + j < rows, two = m + j + 1 < rows;
            if (args.p.y_image) {
              if (one) image_row(args.p, m0 + m + j, nb, quarter, lane, out & 0xFFFFu);
              if (two) image_row(args.p, m0 + m + j + 1, nb, quarter, lane, out >> 16);
            } else if (n < N) {
              if (one) y[(m + j) * (int64_t)N] = (uint16_t)out;
              if (two) y[(m + j + 1) * (int64_t)N] = (uint16_t)(out >> 16);
            }
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
      if (C > 1 && lane < C && lane != rank) arrive_release_cluster(map_to_cta(sent_addr, (uint32_t)lane));
    }
  } else if (QUANT) {
    // ---------------- quantisation (warps 6..13): every eighth tile a warp ------
    // A lane takes block lane & 7 of every fourth row, all its loads in flight
    // together; a warp has the time of eight stages for its one.
    griddep_wait();
    const int qw = warp - L::kThreads / 32;
    const int M = args.p.M, blk = lane & 7;
    uint32_t s = 0, ph = 0;  // the ring's first round needs no wait
    bool ok = true;
    int k = 0;
    for (int64_t i = 0; ok && i < total; ++i) {
      if ((int)(i & (kQuantWarps - 1)) == qw) {
        uint8_t *st = smem + s * L::kStageBytes;
        const int col = (k_begin + k) * kMxTileK + blk * 32;
        uint4 v[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int row = (lane >> 3) + 4 * j;
            v[j][g] = make_uint4(0, 0, 0, 0);
            if (row < M && col + g * 8 < args.K)
              v[j][g] = *reinterpret_cast<const uint4 *>(args.x + (int64_t)row * args.ldx + col + g * 8);
          }
        if (i >= S) {  // the stage's previous MMAs are done
          ok = wait_all(&empty[s], ph ^ 1);
          if (!ok) break;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = (lane >> 3) + 4 * j;
          if (row >= M) continue;
          uint4 codes;
          const uint32_t c = mx4_encode_block(v[j], codes);
          *reinterpret_cast<uint4 *>(st + L::kQ + mx4_chunk_offset(row, blk)) = codes;
          st[L::kS + mx4_scale_offset(row, blk) - kMxCodeBytes] = (uint8_t)c;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
      if (++k == nk) k = 0;
      if (++s == (uint32_t)S) {
        s = 0;
        ph ^= 1;
      }
    }
  }

  tc_fence_before();
  if (C > 1)
    cluster_sync();  // no CTA leaves while another may still write to it
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
}

FuncAttrOnce g_stream_attr[5];

template <int NT, bool QUANT>
cudaError_t allow_smem() {
  return g_stream_attr[QUANT ? 0 : NT == 16 ? 1 : NT == 32 ? 2 : NT == 64 ? 3 : 4].ensure([] {
    return cudaFuncSetAttribute(mx4_stream_kernel<NT, QUANT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                StreamCfg<NT>::kAlloc);
  });
}

// Clusters of C CTAs that the device holds at once (0: not that size), asked
// once per device.  Of the instance without QUANT for both, so that the layer
// splits K, and rounds its sums, as the product on codes does.
template <int NT>
int max_clusters(int C) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxStreamCluster + 1];  // + 1
  const int dev = current_device();
  const bool keep = dev >= 0 && dev < kDevices;
  int n = keep ? known[dev][C].load(std::memory_order_relaxed) - 1 : -1;
  if (n >= 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C);
  cfg.blockDim = dim3(StreamCfg<NT>::kThreads);
  cfg.dynamicSmemBytes = StreamCfg<NT>::kAlloc;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (allow_smem<NT, false>() != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, mx4_stream_kernel<NT, false>, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  if (keep) known[dev][C].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int NT, bool QUANT>
w8a8_status run(StreamArgs a, cudaStream_t stream) {
  if (allow_smem<NT, QUANT>() != cudaSuccess) return W8A8_ERR_CUDA;
  // The cluster size with the least estimated time: rounds of slabs, each
  // round at the rate of DRAM or of one SM's copies, whichever is slower, and
  // the time to join a split slab.
  double best = 1e30;
  int best_clusters = 0;
  for (int C = 1; C <= kMaxStreamCluster && C <= a.p.kt; ++C) {
    // (of 64 rows, the parts of three CTAs would not fit in shared memory)
    const int clusters = C * ((NT / 16 + C - 1) / C) <= StreamCfg<NT>::kChunks ? max_clusters<NT>(C) : 0;
    if (clusters < 1) continue;
    const int tiles = (a.p.kt + C - 1) / C;
    auto round_us = [&](int n) {
      return tiles * kMxTileBytes * std::max(1.0 / kSmBytesPerUs, n * C / kDramBytesPerUs);
    };
    const int whole = a.slabs / clusters, rest = a.slabs % clusters;
    const double us = (C > 1 ? kJoinUs * (whole + (rest > 0)) : 0.0) + whole * round_us(clusters) +
                      (rest ? round_us(rest) : 0.0);
    if (us < best) {
      best = us;
      best_clusters = std::min(a.slabs, clusters);
      a.C = C;
    }
  }
  if (!best_clusters) return W8A8_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(best_clusters * a.C));
  cfg.blockDim = dim3(StreamCfg<NT>::kThreads + (QUANT ? 32 * kQuantWarps : 0));
  cfg.dynamicSmemBytes = (size_t)StreamCfg<NT>::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, mx4_stream_kernel<NT, QUANT>, a);
  if (e == cudaSuccess) count_launch();
  return from_cuda(e);
}

}  // namespace

w8a8_status launch_mx4_stream(const Mx4Args &p, const void *x, int64_t ldx, int64_t K, cudaStream_t stream) {
  StreamArgs a{};
  a.p = p;
  a.x = static_cast<const uint16_t *>(x);
  a.ldx = ldx;
  a.K = (int)K;
  a.slabs = (int)mx4_slabs(p.N);
  if (x) return run<16, true>(a, stream);
  if (p.M <= 16) return run<16, false>(a, stream);
  if (p.M <= 32) return run<32, false>(a, stream);
  if (p.M <= 64) return run<64, false>(a, stream);
  return run<128, false>(a, stream);
}

}  // namespace w8a8
