// mx4_stream.cu -- the 4-bit product for few rows: every SM streams its share
// of the weights.
//
// With M <= 128 rows the weights are most of the bytes, so they set the time.
// Swap-AB: a 128-row weight tile is the MMA's M operand and the rows of x (16,
// 32, 64 or 128 of them) its N operand.  A work unit is two consecutive tiles
// of one 128-row weight slab (34 KB, one copy, codes and scales); the units
// are split evenly over all SMs, so that N and K need not fill the chip.  A
// slab whose units belong to several CTAs is finished by the last of them to
// arrive (call-tagged counters, as in decode.cu: no clearing, no waits
// between CTAs).  The fp32 partial sums of a slab are always added in the
// same order, from the last contributor to the first, whoever adds them: equal
// calls give equal bits.  A CTA that finds every other contributor done when
// it starts on a slab (as the first contributor, which works on it last,
// usually does) reads their partials while its own MMAs run.
//
// QUANT (the layer, M <= 16): x comes as bf16 and four more warps form its
// codes and scales, a block of 32 in one lane, straight into the pipeline
// stage: no quantisation launch, no image of x in memory.  Each CTA forms the
// tiles that its units need.
//
// Before the wait for the preceding kernel of the stream, whose output x (or
// even the weights) may be, the first weight units are only asked into L2,
// where they are coherent; every read and write follows the wait.
#include <algorithm>

#include "gemm_common.cuh"
#include "mx4_common.cuh"

namespace w8a8 {
namespace {

constexpr int kUnitTiles = 2;

template <int NT>
struct StreamCfg {
  static constexpr int kStages = NT <= 32 ? 5 : NT == 64 ? 4 : 3;
  static constexpr int kCodes = NT * 128;  // bytes of the activation codes of one tile
  static constexpr int kW = 0;
  static constexpr int kQ = kUnitTiles * kMxTileBytes;
  static constexpr int kS = kQ + kUnitTiles * kCodes;
  static constexpr int kStageBytes = kS + kUnitTiles * kMxScaleBytes;  // a multiple of 1024
  static constexpr int kBars = kStages * kStageBytes;
  static constexpr int kMisc = kBars + (2 * kStages + 5) * 8;
  static constexpr int kAlloc = kMisc + 32 + 1024;
  // TMEM: two accumulators of NT columns, then each stage's scale columns
  static constexpr uint32_t kScaleCols = kUnitTiles * 16;
  static constexpr uint32_t kNeeded = 2 * NT + kStages * kScaleCols;
  static constexpr uint32_t kTmemCols = kNeeded <= 256 ? 256 : 512;
  static_assert(kAlloc <= 232448 && kNeeded <= 512, "one CTA's shared memory and TMEM");
};

struct StreamArgs {
  Mx4Args p;           // p.a: the image of x, without QUANT
  const uint16_t *x;   // QUANT
  int64_t ldx;
  int K;
  int num_ku;          // units per slab
  int64_t units;
  int max_contrib;
  float *partials;               // [slabs][max_contrib][NT][128]
  unsigned long long *counters;  // [slabs]
  unsigned long long tag;
};

__device__ __forceinline__ int64_t stream_begin(int64_t units, int grid, int c) { return units * c / grid; }

// The CTA whose units contain unit u.
__device__ __forceinline__ int stream_cta_of(int64_t units, int grid, int64_t u) {
  int c = (int)((u * grid) / units);
  while (c + 1 < grid && stream_begin(units, grid, c + 1) <= u) ++c;
  while (c > 0 && stream_begin(units, grid, c) > u) --c;
  return c;
}

constexpr int kPrefetchUnits = 8;  // 272 KB a CTA, 40 MB in all
constexpr int kStreamThreads = 192;
constexpr int kQuantWarps = 4;

template <int NT, bool QUANT>
__global__ void __launch_bounds__(kStreamThreads + (QUANT ? 32 * kQuantWarps : 0), 1)
    mx4_stream_kernel(const StreamArgs args) {
  using L = StreamCfg<NT>;
  constexpr int S = L::kStages;
  constexpr uint32_t kIdesc = idesc_mx4(128, NT);
  constexpr int kChunk = NT < 32 ? NT : 32;  // accumulator columns read at a time

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars);
  uint64_t *empty = full + S;
  uint64_t *tfull = empty + S;
  uint64_t *tempty = tfull + 2;
  uint64_t *mma_done = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
  volatile int *shared_word = reinterpret_cast<volatile int *>(smem + L::kMisc + 8);  // [4]

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], QUANT ? 2 : 1);  // the copies; the codes of x
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, L::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int grid = (int)gridDim.x;
  const int64_t u_begin = stream_begin(args.units, grid, blockIdx.x);
  const int64_t u_end = stream_begin(args.units, grid, blockIdx.x + 1);
  const int64_t n_units = u_end - u_begin;
  const int kt = args.p.kt, nku = args.num_ku;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- producer ----------------
      const uint64_t evict_first = policy_evict_first();
      struct Cur {
        int k0;  // first tile of the unit
        const uint8_t *w;
      };
      auto next = [&](Cur &c) {
        const int left = kt - c.k0;
        c.w += (size_t)min(kUnitTiles, left) * kMxTileBytes;  // slabs follow one another
        c.k0 = left <= kUnitTiles ? 0 : c.k0 + kUnitTiles;
      };
      auto tiles = [&](const Cur &c) { return min(kUnitTiles, kt - c.k0); };
      auto bytes = [&](int nk) {
        return (uint32_t)(nk * (kMxTileBytes + (QUANT ? 0 : L::kCodes + kMxScaleBytes)));
      };
      auto weights = [&](const Cur &c, uint32_t s, int nk) {
        bulk_load_hint(smem + s * L::kStageBytes + L::kW, c.w, (uint32_t)(nk * kMxTileBytes), &full[s],
                       evict_first);
      };
      auto acts = [&](const Cur &c, uint32_t s, int nk) {
        if (QUANT) return;
        for (int h = 0; h < nk; ++h) {
          const uint8_t *t = args.p.a + (size_t)(c.k0 + h) * kMxTileBytes;
          uint8_t *st = smem + s * L::kStageBytes;
          bulk_load(st + L::kQ + h * L::kCodes, t, L::kCodes, &full[s]);
          bulk_load(st + L::kS + h * kMxScaleBytes, t + kMxCodeBytes, kMxScaleBytes, &full[s]);
        }
      };
      const uint32_t pre = n_units < S ? (uint32_t)n_units : (uint32_t)S;
      Cur cur;
      {
        const int nb = (int)(u_begin / nku);
        cur.k0 = (int)(u_begin - (int64_t)nb * nku) * kUnitTiles;
        cur.w = args.p.w + ((size_t)nb * kt + cur.k0) * kMxTileBytes;
      }
      // before the wait: DRAM to L2 only, in the order of the copies
      {
        Cur c = cur;
        for (int64_t i = 0; i < n_units && i < kPrefetchUnits; ++i) {
          bulk_prefetch_l2(c.w, (uint32_t)(tiles(c) * kMxTileBytes));
          next(c);
        }
      }
      griddep_wait();
      for (uint32_t s = 0; s < pre; ++s) {
        const int nk = tiles(cur);
        mbar_arrive_expect_tx(&full[s], bytes(nk));
        weights(cur, s, nk);
        acts(cur, s, nk);
        next(cur);
      }
      uint32_t s = 0, ph = 1;
      int64_t issued = pre;
      for (; issued < n_units; ++issued) {
        const int nk = tiles(cur);
        if (!mbar_wait(&empty[s], ph ^ 1, abort_flag, args.p.status)) break;
        mbar_arrive_expect_tx(&full[s], bytes(nk));
        weights(cur, s, nk);
        acts(cur, s, nk);
        next(cur);
        if (++s == (uint32_t)S) {
          s = 0;
          ph ^= 1;
        }
      }
      // Every copy issued lands before the CTA leaves, whatever gave up.  (With
      // QUANT a stage whose codes never came stays incomplete: bounded too.)
      for (int64_t sl = 0; sl < S && sl < issued; ++sl) {
        const int64_t last = sl + ((issued - 1 - sl) / S) * S;
        volatile int no_abort = 0;
        (void)mbar_wait_bounded(&full[sl], (uint32_t)((last / S) & 1), &no_abort, args.p.status);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer: the warp waits, one elected lane issues ----
    const bool lead = elect_one();
    const uint64_t desc0 = sw128_kmajor_desc(smem), sc_desc0 = mx4_scale_desc(smem);
    uint32_t s = 0, ph = 0, seg = 0;
    bool ok = true;
    int64_t u = u_begin;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, args.p.status)) != 0;
    };
    while (ok && u < u_end) {
      const int64_t nb = u / nku;
      const int64_t seg_end = min(u_end, (nb + 1) * nku);
      const uint32_t b = seg & 1, bph = (seg >> 1) & 1;
      ok = wait(&tempty[b], bph ^ 1);
      if (!ok) break;
      const uint32_t d_tmem = tmem_base + b * NT;
      uint32_t acc = 0;
      for (int k0 = (int)(u - nb * nku) * kUnitTiles; u < seg_end; ++u, k0 += kUnitTiles) {
        ok = wait(&full[s], ph);
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          // (a descriptor's address field is the shared-memory address / 16)
          const uint64_t at = (uint64_t)(s * (L::kStageBytes >> 4));
          const int nk = min(kUnitTiles, kt - k0);
          for (int h = 0; h < nk; ++h) {
            const uint64_t wd = desc0 + at + (uint64_t)(h * (kMxTileBytes >> 4));
            const uint64_t qd = desc0 + at + (uint64_t)((L::kQ + h * L::kCodes) >> 4);
            const uint64_t ws = sc_desc0 + at + (uint64_t)((h * kMxTileBytes + kMxCodeBytes) >> 4);
            const uint64_t qs = sc_desc0 + at + (uint64_t)((L::kS + h * kMxScaleBytes) >> 4);
            const uint32_t sfw = tmem_base + 2 * NT + s * L::kScaleCols + h * 16, sfq = sfw + 8;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              copy_scales(sfw + 4 * g, ws + ((g * kMxGroupBytes) >> 4));
              copy_scales(sfq + 4 * g, qs + ((g * kMxGroupBytes) >> 4));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma_mx4(d_tmem, wd + 2 * j, qd + 2 * j, kIdesc | ((j & 1) ? kMxSecondPair : 0u),
                      sfw + 4 * (j >> 1), sfq + 4 * (j >> 1), acc);
              acc = 1;
            }
          }
          mma_commit(&empty[s]);
        }
        acc = 1;
        __syncwarp();
        if (++s == (uint32_t)S) {
          s = 0;
          ph ^= 1;
        }
      }
      if (ok && lead) mma_commit(&tfull[b]);
      __syncwarp();
      ++seg;
    }
    if (lead) {  // nothing of this CTA is in flight when it leaves (bounded)
      mma_commit(mma_done);
      volatile int no_abort = 0;
      (void)mbar_wait_bounded(mma_done, 0, &no_abort, args.p.status);
    }
    __syncwarp();
  } else if (warp < 6) {
    // ---------------- epilogue (warps 2..5): one output column per thread ----
    // The four warps take every decision together: thread 0 of the group
    // decides and publishes behind a named barrier.
    griddep_wait();
    const int quarter = warp & 3;
    const int et = threadIdx.x - 64;
    const int M = args.p.M, N = args.p.N;
    const int nchunks = (M + kChunk - 1) / kChunk;  // chunks of columns that hold rows of x
    uint32_t seg = 0;
    int64_t u = u_begin;
    auto decide = [&](uint32_t word, int v) {  // et == 0's v, to the group
      if (et == 0) shared_word[word] = v;
      __syncwarp();
      named_barrier_sync(1, 128);
      return (int)shared_word[word];
    };
    while (u < u_end) {
      const int nb = (int)(u / nku);
      const int64_t slab_begin = (int64_t)nb * nku, slab_end = slab_begin + nku;
      const int64_t seg_end = min(u_end, slab_end);
      const bool whole = (u == slab_begin) && (seg_end == slab_end);
      const uint32_t b = seg & 1, bph = (seg >> 1) & 1;
      const int n_local = quarter * 32 + lane;
      const int n = nb * 128 + n_local;
      const float bv =
          (args.p.bias && n < N) ? __uint_as_float((uint32_t)__ldg(args.p.bias + n) << 16) : 0.0f;
      int contributors = 1, rank = 0;
      if (!whole) {
        const int first_cta = stream_cta_of(args.units, grid, slab_begin);
        contributors = stream_cta_of(args.units, grid, slab_end - 1) - first_cta + 1;
        rank = blockIdx.x - first_cta;
      }
      float *slots = args.partials + (size_t)nb * args.max_contrib * (128 * NT) + n_local;
      auto others_done = [&]() {  // et == 0: whether every other contributor has arrived
        const unsigned long long v = ld_acquire_gpu(args.counters + nb);
        const bool in = (v >> 8) == args.tag && (uint32_t)(v & 0xFF) == (uint32_t)(contributors - 1);
        // no other arrival can follow: this call is done with the word (a
        // replayed graph has the same tag and must find it at zero)
        if (in) args.counters[nb] = 0ull;
        return in;
      };
      // Adds the partials of contributors hi, hi - 1, ..., lo + 1 in that order
      // (chunk c), the loads of kGroup of them in flight together: one after
      // another they cost a round trip to L2 each, at the kernel's tail
      // (13 x 5120 x 13824, 5 contributors a slab: 7 us of 16.6 us).
      constexpr int kGroup = kChunk == 16 ? 4 : 2;
      auto add_parts = [&](float (&sum)[kChunk], int hi, int lo, int c) {
        const float *base = slots + c * kChunk * 128;
        for (int o = hi; o > lo; o -= kGroup) {
          float v[kGroup][kChunk];
#pragma unroll
          for (int g = 0; g < kGroup; ++g)
#pragma unroll
            for (int m = 0; m < kChunk; ++m)
              v[g][m] = o - g > lo ? __ldcg(base + (size_t)(o - g) * (128 * NT) + m * 128) : 0.0f;
#pragma unroll
          for (int g = 0; g < kGroup; ++g)
            if (o - g > lo) {
#pragma unroll
              for (int m = 0; m < kChunk; ++m) sum[m] += v[g][m];
            }
        }
      };
      // While this CTA's MMAs run: the later contributors' partials, if all are in.
      bool finish = whole;
      float pre[kChunk];
      bool have_pre = false;
      if (!whole && NT <= 16) {
        finish = decide(b, (et == 0 && others_done()) ? 1 : 0) != 0;
        if (finish) {
          have_pre = true;
#pragma unroll
          for (int m = 0; m < kChunk; ++m) pre[m] = 0.0f;
          add_parts(pre, contributors - 1, rank, 0);
        }
      }
      if (!decide(2 + b, et == 0 ? (mbar_wait(&tfull[b], bph, abort_flag, args.p.status) ? 1 : 0) : 0)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + b * NT;
      auto load = [&](int c, float (&r)[kChunk]) {
        uint32_t v[kChunk];
        if constexpr (kChunk == 16)
          tmem_ld_32x32b_x16(taddr + c * kChunk, v);
        else
          tmem_ld_32x32b_x32(taddr + c * kChunk, v);
        tmem_ld_wait();
#pragma unroll
        for (int m = 0; m < kChunk; ++m) r[m] = __uint_as_float(v[m]);
      };
      if (!finish) {
        finish = decide(b, (et == 0 && others_done()) ? 1 : 0) != 0;
        if (!finish) {  // publish this CTA's part
          float *o = slots + (size_t)rank * (128 * NT);
          for (int c = 0; c < nchunks; ++c) {
            float r[kChunk];
            load(c, r);
#pragma unroll
            for (int m = 0; m < kChunk; ++m) __stcg(o + (c * kChunk + m) * 128, r[m]);
          }
          __threadfence();
          __syncwarp();
          named_barrier_sync(1, 128);
          bool last = false;
          if (et == 0) {
            last = arrive_tagged(args.counters + nb, args.tag) == (uint32_t)contributors;
            if (last) {
              args.counters[nb] = 0ull;
              __threadfence();
            }
          }
          finish = decide(b, last ? 1 : 0) != 0;
        }
      }
      if (finish) {
        for (int c = 0; c < nchunks; ++c) {
          float r[kChunk];
          load(c, r);
          if (!whole) {
            float sum[kChunk];
#pragma unroll
            for (int m = 0; m < kChunk; ++m) sum[m] = have_pre ? pre[m] : 0.0f;
            if (!have_pre) add_parts(sum, contributors - 1, rank, c);
#pragma unroll
            for (int m = 0; m < kChunk; ++m) sum[m] += r[m];
            add_parts(sum, rank - 1, -1, c);
#pragma unroll
            for (int m = 0; m < kChunk; ++m) r[m] = sum[m];
          }
          // bias, activation, rounding, in pairs of rows
          uint32_t out[kChunk / 2];
#pragma unroll
          for (int m = 0; m < kChunk; m += 2) {
            float t0 = __fadd_rn(r[m], bv), t1 = __fadd_rn(r[m + 1], bv);
            apply_act_pair(t0, t1, args.p.act);
            out[m / 2] = n < N ? pack_bf16x2(t0, t1) : 0u;
          }
          const int m0 = c * kChunk;
          if (args.p.y_image) {
            // a block is the warp's 32 columns of one row of y
            uint8_t *tile = args.p.y_image + (size_t)(nb >> 1) * kMxTileBytes;
            const int blk = (nb & 1) * 4 + quarter;
            const bool pad = !(nb & 1) && (nb + 1) * 128 >= N;  // the tile's other half has no slab
#pragma unroll
            for (int m = 0; m < kChunk; ++m) {
              if (m0 + m >= M) break;
              const uint32_t bits = (m & 1) ? out[m / 2] >> 16 : out[m / 2] & 0xFFFFu;
              const uint32_t code = mx4_scale_code(__reduce_max_sync(0xFFFFFFFFu, bits & 0x7FFFu));
              const uint32_t q = code == 255u ? 0u
                                              : mx4_codes8(__uint_as_float(bits << 16) * mx4_inverse_scale(code),
                                                           0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f) & 15u;
              uint32_t word = q << (4 * (lane & 7));
              word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
              word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
              word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
              const int row = m0 + m;
              if ((lane & 7) == 0) {
                *reinterpret_cast<uint32_t *>(tile + mx4_chunk_offset(row, blk) + (lane >> 3) * 4) = word;
                if (pad)
                  *reinterpret_cast<uint32_t *>(tile + mx4_chunk_offset(row, blk + 4) + (lane >> 3) * 4) = 0u;
              }
              if (lane == 0) {
                tile[mx4_scale_offset(row, blk)] = (uint8_t)code;
                if (pad) tile[mx4_scale_offset(row, blk + 4)] = 0;
              }
            }
          } else if (n < N) {
#pragma unroll
            for (int m = 0; m < kChunk; ++m)
              if (m0 + m < M)
                args.p.y[(int64_t)(m0 + m) * N + n] =
                    (uint16_t)((m & 1) ? out[m / 2] >> 16 : out[m / 2] & 0xFFFFu);
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
      u = seg_end;
      ++seg;
    }
  } else if (QUANT) {
    // ---------------- quantisation (warps 6..9): every fourth unit a warp -------
    // A unit is 16 blocks of each row: a lane takes block lane & 15 of every
    // second row.  The loads of up to eight rows are in flight together, and a
    // warp has the time of four units for its one (with all four warps on
    // every unit, each paid a round trip to L2: slower than the weights).
    griddep_wait();
    const int qw = warp - kStreamThreads / 32;
    const int M = args.p.M, blk = lane & 7, h = (lane >> 3) & 1;
    const int nb0 = (int)(u_begin / nku);
    int k0 = (int)(u_begin - (int64_t)nb0 * nku) * kUnitTiles;
    uint32_t s = 0, ph = 0;  // the ring's first round needs no wait
    bool ok = true;
    constexpr int kRows = 4;  // rows of a lane in flight
    for (int64_t i = 0; ok && i < n_units; ++i) {
      if ((int)(i & (kQuantWarps - 1)) == qw) {
        uint8_t *st = smem + s * L::kStageBytes;
        const int k = (k0 + h) * kMxTileK + blk * 32;
        const bool in_tile = k0 + h < kt;
        for (int r0 = lane >> 4; r0 < M || r0 < 2; r0 += 2 * kRows) {
          uint4 v[kRows][4];
#pragma unroll
          for (int j = 0; j < kRows; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const int row = r0 + 2 * j;
              v[j][g] = make_uint4(0, 0, 0, 0);
              if (row < M && k + g * 8 < args.K)
                v[j][g] = *reinterpret_cast<const uint4 *>(args.x + (int64_t)row * args.ldx + k + g * 8);
            }
          if (r0 < 2 && i >= S) {  // the stage's previous MMAs are done
            int done = 0;
            if (lane == 0) done = mbar_wait(&empty[s], ph ^ 1, abort_flag, args.p.status);
            ok = __shfl_sync(0xFFFFFFFFu, done, 0) != 0;
            if (!ok) break;
          }
#pragma unroll
          for (int j = 0; j < kRows; ++j) {
            const int row = r0 + 2 * j;
            if (row >= M || !in_tile) continue;
            uint4 codes;
            const uint32_t c = mx4_encode_block(v[j], codes);
            *reinterpret_cast<uint4 *>(st + L::kQ + h * L::kCodes + mx4_chunk_offset(row, blk)) = codes;
            st[L::kS + h * kMxScaleBytes + mx4_scale_offset(row, blk) - kMxCodeBytes] = (uint8_t)c;
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
      k0 = kt - k0 <= kUnitTiles ? 0 : k0 + kUnitTiles;
      if (++s == (uint32_t)S) {
        s = 0;
        ph ^= 1;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
}

struct Geometry {
  int64_t slabs, ku, units;
  int grid, contrib;
};

Geometry geometry(int64_t N, int64_t K) {
  Geometry g;
  g.slabs = mx4_slabs(N);
  g.ku = (mx4_ktiles(K) + kUnitTiles - 1) / kUnitTiles;
  g.units = g.slabs * g.ku;
  g.grid = (int)std::min<int64_t>(g.units, sm_count());
  const int64_t per = g.units / g.grid;  // the shortest share of a CTA
  g.contrib = (int)((g.ku + per - 1) / per + 1);
  return g;
}

int rows_of(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

FuncAttrOnce g_stream_attr[5];

template <int NT, bool QUANT>
cudaError_t run(const StreamArgs &a, int grid, cudaStream_t stream, int slot) {
  using L = StreamCfg<NT>;
  auto k = mx4_stream_kernel<NT, QUANT>;
  cudaError_t e = g_stream_attr[slot].ensure([&] {
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kStreamThreads + (QUANT ? 32 * kQuantWarps : 0));
  cfg.dynamicSmemBytes = (size_t)L::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

int64_t mx4_stream_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const Geometry g = geometry(N, K);
  return round_up(g.slabs * 8, 256) + g.slabs * g.contrib * 128 * rows_of(M) * 4;
}

w8a8_status launch_mx4_stream(const Mx4Args &p, const void *x, int64_t ldx, int64_t K, void *workspace,
                              cudaStream_t stream) {
  const Geometry g = geometry(p.N, K);
  StreamArgs a{};
  a.p = p;
  a.x = static_cast<const uint16_t *>(x);
  a.ldx = ldx;
  a.K = (int)K;
  a.num_ku = (int)g.ku;
  a.units = g.units;
  a.max_contrib = g.contrib;
  a.counters = static_cast<unsigned long long *>(workspace);
  a.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + round_up(g.slabs * 8, 256));
  a.tag = next_call_tag();
  if (x) return from_cuda(run<16, true>(a, g.grid, stream, 0));
  switch (rows_of(p.M)) {
    case 16: return from_cuda(run<16, false>(a, g.grid, stream, 1));
    case 32: return from_cuda(run<32, false>(a, g.grid, stream, 2));
    case 64: return from_cuda(run<64, false>(a, g.grid, stream, 3));
    default: return from_cuda(run<128, false>(a, g.grid, stream, 4));
  }
}

}  // namespace w8a8
