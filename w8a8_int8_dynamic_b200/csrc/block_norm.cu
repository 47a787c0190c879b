// block_norm.cu -- the step between two blocks of a transformer in one kernel:
// the norm after the block, its gate, the residual sum with its scale, the
// norm before the next block with its modulation, and the codes of the next
// quantised layer.
//
//   u = post(x)                       (or x)
//   v = residual_scale * residual + gate[g] * u,  rounded to the residual's type
//   h = pre(v) * (1 + scale[g]) + shift[g]
//   rms(t)   = t * rsqrt(mean(t^2) + eps) * w + b
//   layer(t) = (t - mean) * rsqrt(mean((t - mean)^2) + eps) * w + b
//   y = bf16(h);  int8 codes and row scale of y;  MX 4-bit image of y
//
// A CTA of W warps takes a run of rows, each lane holding CPL chunks of eight
// elements: x and the residual are read once and everything until the stores
// stays in registers in fp32.  The loads of the next row are in flight while
// the CTA works on this one.
//
// What is shared by a group's rows is folded once per run of rows of a group,
// into fp32 vectors in shared memory: gate * post weight, pre weight * (1 +
// scale), pre bias * (1 + scale) + shift.  A row then costs two or three
// multiply-adds an element for them; widening up to seven bf16 vectors again
// for every row made the kernel instruction-bound (52 instructions an element,
// 8192 x 4096: 76 us).  The arithmetic runs on paired fp32 instructions.
// Memory-bound: (2 + r) bytes read and (r + 2 | 1 | 17/32) written an element,
// r the bytes of the residual's type.
//
// The mean and the sum of squared differences of a row take one barrier: each
// warp forms both of its own part (the mean first, so nothing cancels), and
// the parts are joined as sum(m2) + sum(n (mean - total mean)^2).  (The mean of
// what is left of a part, added to the part's, would make the row's mean exact
// to roundings of its spread, but made the row's code so much longer that
// 8192 x 4096 with both norms took 98 us for 59.)
//
// A programmatic dependent that releases the next kernel at its start and
// touches memory only after its own wait; no load takes the read-only path
// (the kernel ahead may be writing what this one reads when it starts, and the
// residual may be updated in place).
#include <algorithm>

#include "mx4_common.cuh"
#include "quant_common.cuh"

namespace w8a8 {
namespace {

struct NormArgs {
  const uint16_t *x;
  const void *residual;
  void *residual_out;
  uint16_t *y;
  int8_t *q;
  float *a_scale;
  uint8_t *image;
  const uint16_t *post_w, *post_b, *pre_w, *pre_b;
  const uint16_t *gate, *scale, *shift;
  const int32_t *group_index;
  int64_t ldx, ldr, ldro, ldy, ld_gate, ld_scale, ld_shift;
  int64_t rows_per_group, groups;
  int M, K, kt;
  int post_kind, pre_kind;
  int residual_f32;
  float residual_scale, post_eps, pre_eps, inv_k;
  int W;        // warps per row
  int folded;   // which folded vectors there are (kFold*)
  int padded;   // chunks of a folded vector: W * 32 * chunks per lane
};

// Eight values as four fp32 pairs.
struct Eight {
  uint64_t p[4];
};

__device__ __forceinline__ uint64_t widen(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ Eight widen8(const uint4 &v) {
  return {{widen(v.x), widen(v.y), widen(v.z), widen(v.w)}};
}
__device__ __forceinline__ uint32_t narrow(uint64_t p) {
  float lo, hi;
  f2_unpack(p, lo, hi);
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint4 narrow8(const Eight &e) {
  return make_uint4(narrow(e.p[0]), narrow(e.p[1]), narrow(e.p[2]), narrow(e.p[3]));
}
__device__ __forceinline__ float pair_sum(uint64_t p) {
  float lo, hi;
  f2_unpack(p, lo, hi);
  return lo + hi;
}

constexpr int kMaxWarps = 16;  // of a row: lanes 0..15 join their parts

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum over lanes 0..15 (in every one of them and, of zeros, above), the same everywhere.
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return __shfl_sync(0xFFFFFFFFu, v, 0);
}

// Where a warp stands: its part of the row.
struct Place {
  int w, W, lane, c0, nchunks;
  float own_count;   // elements of the row in this warp's part: at least eight
  float lane_count;  // elements in the part of warp `lane` (0: no such warp)
};

// A row's norm as t -> t * rstd + offset, for t with this warp's mean taken off.
struct Stat {
  uint64_t rstd, offset;
};

// Takes the mean of the warp's part off t and joins the warps' parts.  `line`:
// shared memory of this call and row parity, so one barrier a call is enough.
template <int CPL>
__device__ __forceinline__ Stat centre(Eight (&t)[CPL], int kind, float eps, float inv_k, float2 *line,
                                       const Place &at) {
  float own = 0.0f;
  const bool layer = kind == W8A8_NORM_LAYER;
  if (layer) {
    uint64_t s[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < CPL; ++j)
      if (at.c0 + 32 * j < at.nchunks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = f2_add(s[i], t[j].p[i]);
      }
    const float sum = warp_sum(pair_sum(f2_add(f2_add(s[0], s[1]), f2_add(s[2], s[3]))));
    // the quotient by a step of reciprocal refinement (quant_common.cuh): exact where it is a
    // float, so a constant row is taken off whole, and 1 / sqrt(eps) has nothing to enlarge
    const float inv = __fdividef(1.0f, at.own_count);
    own = __fmul_rn(sum, inv);
    own = __fmaf_rn(__fmaf_rn(-own, at.own_count, sum), inv, own);
    const uint64_t neg = f2_splat(-own);
#pragma unroll
    for (int j = 0; j < CPL; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) t[j].p[i] = f2_add(t[j].p[i], neg);
  }
  uint64_t q[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < CPL; ++j)
    if (at.c0 + 32 * j < at.nchunks) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = f2_fma(t[j].p[i], t[j].p[i], q[i]);
    }
  float m2 = warp_sum(pair_sum(f2_add(f2_add(q[0], q[1]), f2_add(q[2], q[3])))), offset = 0.0f;
  if (at.W > 1) {
    if (at.lane == 0) line[at.w] = make_float2(own, m2);
    __syncthreads();
    // (a lane without a part stands at the first one's mean: its distance, times a count of zero, is no NaN)
    float2 part = line[at.lane < at.W ? at.lane : 0];
    if (at.lane >= at.W) part.y = 0.0f;
    if (layer) {
      // by the parts' distances from the first one's mean: roundings of the spread, not of the mean
      const float first = line[0].x, d = part.x - first;
      const float mean = half_sum(d * at.lane_count) * inv_k;  // of the distances
      const float e = d - mean;
      part.y = __fmaf_rn(e * e, at.lane_count, part.y);
      offset = (own - first) - mean;
    }
    m2 = half_sum(part.y);
  }
  const float rstd = rsqrtf(__fmaf_rn(m2, inv_k, eps));
  return {f2_splat(rstd), f2_splat(offset * rstd)};
}

// Folded vectors in shared memory, present or not.  A vector is stored by 32
// chunks at a time: the first four values of each of the 32, then the last
// four, so that a warp's 16-byte reads are consecutive and all of a lane's are
// at constant offsets from one address.  It is as long as the warps' parts
// (a.padded chunks); what is past the row is never written and never used.
enum { kFoldBranch = 1, kFoldBranchAdd = 2, kFoldMul = 4, kFoldAdd = 8 };

// `v`: this lane's address in the vector, for its chunk j.
__device__ __forceinline__ Eight load_fold(const ulonglong2 *v, int j) {
  const ulonglong2 lo = v[j * 64], hi = v[j * 64 + 32];
  return {{lo.x, lo.y, hi.x, hi.y}};
}
__device__ __forceinline__ void store_fold(ulonglong2 *v, int c, const Eight &e) {
  v += (c >> 5) * 64 + (c & 31);
  v[0] = make_ulonglong2(e.p[0], e.p[1]);
  v[32] = make_ulonglong2(e.p[2], e.p[3]);
}

// Folds the vectors of group g (all threads of the CTA; the caller syncs).
// The loads of a chunk's vectors are in flight together.
__device__ __forceinline__ void fold(const NormArgs &a, ulonglong2 *v, int64_t g) {
  const int nchunks = a.K >> 3;
  const uint64_t one = f2_splat(1.0f);
  const uint16_t *gp = a.gate ? a.gate + g * a.ld_gate : nullptr;
  const uint16_t *sp = a.scale ? a.scale + g * a.ld_scale : nullptr;
  const uint16_t *tp = a.shift ? a.shift + g * a.ld_shift : nullptr;
  for (int c = threadIdx.x; c < nchunks; c += blockDim.x) {
    auto get = [&](const uint16_t *p, uint4 &d) {
      if (p) d = reinterpret_cast<const uint4 *>(p)[c];
    };
    uint4 gate, pw, pb, sc, w, b, sh;
    get(gp, gate);
    get(a.post_w, pw);
    get(a.post_b, pb);
    get(sp, sc);
    get(a.pre_w, w);
    get(a.pre_b, b);
    get(tp, sh);
    ulonglong2 *to = v;
    auto emit = [&](const Eight &e) {
      store_fold(to, c, e);
      to += a.padded * 2;
    };
    Eight e{{one, one, one, one}};
    if (gp) e = widen8(gate);
    Eight f = e;
    if (a.post_w) {
      const Eight m = widen8(pw);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.p[i] = f2_mul(f.p[i], m.p[i]);
    }
    if (a.folded & kFoldBranch) emit(f);
    if (a.folded & kFoldBranchAdd) {
      f = widen8(pb);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.p[i] = f2_mul(f.p[i], e.p[i]);
      emit(f);
    }
    e = {{one, one, one, one}};
    if (sp) {
      e = widen8(sc);
#pragma unroll
      for (int i = 0; i < 4; ++i) e.p[i] = f2_add(e.p[i], one);
    }
    f = e;
    if (a.pre_w) {
      const Eight m = widen8(w);
#pragma unroll
      for (int i = 0; i < 4; ++i) f.p[i] = f2_mul(f.p[i], m.p[i]);
    }
    if (a.folded & kFoldMul) emit(f);
    if (a.folded & kFoldAdd) {
      f = {{0, 0, 0, 0}};
      if (tp) f = widen8(sh);
      if (a.pre_b) {
        const Eight m = widen8(b);
#pragma unroll
        for (int i = 0; i < 4; ++i) f.p[i] = f2_fma(m.p[i], e.p[i], f.p[i]);
      }
      emit(f);
    }
  }
}

enum { kNoResidual = 0, kResidualBf16 = 1, kResidualF32 = 2 };

// A row as it was loaded.
template <int CPL, int RES>
struct Raw {
  uint4 x[CPL];
  uint4 r0[RES == kNoResidual ? 1 : CPL], r1[RES == kResidualF32 ? CPL : 1];
};

// x, r: this lane's first chunk of the row (elements past the row read as zeros).
template <int CPL, int RES>
__device__ __forceinline__ void fetch(const uint8_t *x, const uint8_t *r, const Place &at, Raw<CPL, RES> &d) {
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const bool in = at.c0 + 32 * j < at.nchunks;
    d.x[j] = make_uint4(0, 0, 0, 0);
    if (in) d.x[j] = ld_once_u4(x + j * 512);
    if constexpr (RES == kResidualF32) {
      d.r0[j] = d.r1[j] = make_uint4(0, 0, 0, 0);
      if (in) {
        d.r0[j] = ld_once_u4(r + j * 1024);
        d.r1[j] = ld_once_u4(r + j * 1024 + 16);
      }
    } else if constexpr (RES == kResidualBf16) {
      d.r0[j] = make_uint4(0, 0, 0, 0);
      if (in) d.r0[j] = ld_once_u4(r + j * 512);
    }
  }
}

template <int CPL, int RES, int REGS>
__global__ void __maxnreg__(REGS) block_norm_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ ulonglong2 folded[];
  __shared__ float2 lines[2][2][kMaxWarps];     // [row parity][norm][warp]
  __shared__ uint32_t max_lines[2][kMaxWarps];  // [row parity][warp]
  griddep_launch_dependents();
  griddep_wait();
  Place at;
  at.lane = threadIdx.x & 31;
  at.w = threadIdx.x >> 5;
  at.W = a.W;
  at.nchunks = a.K >> 3;
  at.c0 = at.w * 32 * CPL + at.lane;
  auto count = [&](int w) { return (float)(max(0, min(at.nchunks - w * 32 * CPL, 32 * CPL)) * 8); };
  at.own_count = count(at.w);
  at.lane_count = at.lane < at.W ? count(at.lane) : 0.0f;
  // this lane's place in a folded vector, of which `before` are stored ahead
  auto place = [&](int before) {
    return folded + (at.w * 64 * CPL + at.lane) + __popc(a.folded & before) * a.padded * 2;
  };

  constexpr int kRes = RES == kResidualF32 ? 4 : 2;  // bytes of the residual's type
  int have = -1;   // the group whose vectors are folded
  int parity = 0;  // of the rows computed: each leaves the other its barrier lines
  int row = (int)((int64_t)a.M * blockIdx.x / gridDim.x);
  const int end = (int)((int64_t)a.M * (blockIdx.x + 1) / gridDim.x);
  while (row < end) {
    // a run of rows of one group
    int group = 0, run = end;
    if (a.group_index) {
      group = a.group_index[row];
      for (run = row + 1; run < end && a.group_index[run] == group;) ++run;
      if (group < 0 || group >= a.groups) {  // padding rows: their outputs keep what they hold
        row = run;
        continue;
      }
    } else if (a.rows_per_group) {
      group = (int)(row / a.rows_per_group);
      run = (int)min((int64_t)end, (group + 1) * a.rows_per_group);
    }
    auto load = [&](int i, Raw<CPL, RES> &d) {
      fetch<CPL, RES>(reinterpret_cast<const uint8_t *>(a.x + i * a.ldx + at.c0 * 8),
                      static_cast<const uint8_t *>(a.residual) + (i * a.ldr + at.c0 * 8) * kRes, at, d);
    };
    Raw<CPL, RES> next;
    load(row, next);  // in flight while the vectors are folded
    if (a.folded && group != have) {
      __syncthreads();
      fold(a, folded, group);
      __syncthreads();
      have = group;
    }
    for (; row < run; ++row) {
      const Raw<CPL, RES> cur = next;
      if (row + 1 < run) load(row + 1, next);
      parity ^= 1;
      Eight t[CPL];
#pragma unroll
      for (int j = 0; j < CPL; ++j) t[j] = widen8(cur.x[j]);

      if constexpr (RES != kNoResidual) {
        uint8_t *ro = static_cast<uint8_t *>(a.residual_out) + (row * a.ldro + at.c0 * 8) * kRes;
        const bool post = a.post_kind != W8A8_NORM_NONE;
        Stat st = {};
        if (post) st = centre<CPL>(t, a.post_kind, a.post_eps, a.inv_k, lines[parity][0], at);
        const uint64_t rs = f2_splat(a.residual_scale);
        // (No branch on a chunk past the row: it computes on what it finds and is
        // not stored, so that the chunks' reads of shared memory can be in flight
        // together.)
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
          const bool in = at.c0 + 32 * j < at.nchunks;
          if (post) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[j].p[i] = f2_fma(t[j].p[i], st.rstd, st.offset);
          }
          Eight r;
          if constexpr (RES == kResidualF32) {
            r.p[0] = f2_pack(__uint_as_float(cur.r0[j].x), __uint_as_float(cur.r0[j].y));
            r.p[1] = f2_pack(__uint_as_float(cur.r0[j].z), __uint_as_float(cur.r0[j].w));
            r.p[2] = f2_pack(__uint_as_float(cur.r1[j].x), __uint_as_float(cur.r1[j].y));
            r.p[3] = f2_pack(__uint_as_float(cur.r1[j].z), __uint_as_float(cur.r1[j].w));
          } else {
            r = widen8(cur.r0[j]);
          }
          if (a.folded & kFoldBranchAdd) {
            const Eight e = load_fold(place(kFoldBranch), j);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.p[i] = f2_fma(r.p[i], rs, e.p[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) r.p[i] = f2_mul(r.p[i], rs);
          }
          if (a.folded & kFoldBranch) {
            const Eight e = load_fold(place(0), j);
#pragma unroll
            for (int i = 0; i < 4; ++i) t[j].p[i] = f2_fma(t[j].p[i], e.p[i], r.p[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[j].p[i] = f2_add(t[j].p[i], r.p[i]);
          }
          if constexpr (RES == kResidualF32) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_unpack(t[j].p[i], f[2 * i], f[2 * i + 1]);
            if (in) {
              float4 *p = reinterpret_cast<float4 *>(ro + j * 1024);
              p[0] = make_float4(f[0], f[1], f[2], f[3]);
              p[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
          } else {
            const uint4 v = narrow8(t[j]);
            if (in) *reinterpret_cast<uint4 *>(ro + j * 512) = v;
            t[j] = widen8(v);  // the norm is of the stream as it is stored
          }
        }
        if (a.pre_kind == W8A8_NORM_NONE) continue;
      }

      const Stat st = centre<CPL>(t, a.pre_kind, a.pre_eps, a.inv_k, lines[parity][1], at);
      uint16_t *y = a.y + row * a.ldy + at.c0 * 8;
      uint4 h[CPL];
      uint32_t mx = 0;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        const bool in = at.c0 + 32 * j < at.nchunks;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[j].p[i] = f2_fma(t[j].p[i], st.rstd, st.offset);
        if (a.folded & kFoldMul) {
          const Eight m = load_fold(place(kFoldBranch | kFoldBranchAdd), j);
          if (a.folded & kFoldAdd) {
            const Eight e = load_fold(place(kFoldBranch | kFoldBranchAdd | kFoldMul), j);
#pragma unroll
            for (int i = 0; i < 4; ++i) t[j].p[i] = f2_fma(t[j].p[i], m.p[i], e.p[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[j].p[i] = f2_mul(t[j].p[i], m.p[i]);
          }
        } else if (a.folded & kFoldAdd) {
          const Eight e = load_fold(place(kFoldBranch | kFoldBranchAdd | kFoldMul), j);
#pragma unroll
          for (int i = 0; i < 4; ++i) t[j].p[i] = f2_add(t[j].p[i], e.p[i]);
        }
        h[j] = narrow8(t[j]);
        if (!in) h[j] = make_uint4(0, 0, 0, 0);
        if (in && a.y) *reinterpret_cast<uint4 *>(y + j * 256) = h[j];
        mx = absmax_chunk(mx, h[j]);
      }

      if (a.q) {  // as the int8 quantisation kernel, on the rounded row
        uint32_t m = absmax_fold(mx);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (at.W > 1) {
          if (at.lane == 0) max_lines[parity][at.w] = m;
          __syncthreads();
          m = at.lane < at.W ? max_lines[parity][at.lane] : 0u;
          m = __reduce_max_sync(0xFFFFFFFFu, m);
        }
        {
          const float amax = __uint_as_float(m << 16);
          const float s = amax == 0.0f ? 0.0f : __fdiv_rn(amax, 127.0f);
          const float inv = amax == 0.0f ? 0.0f : __frcp_rn(s);
          if (at.w == 0 && at.lane == 0) a.a_scale[row] = s;
#pragma unroll
          for (int j = 0; j < CPL; ++j) {
            const int c = at.c0 + 32 * j;
            if (c >= at.nchunks) continue;
            uint2 out = make_uint2(0, 0);
            if (amax != 0.0f) out = s >= 1e-30f ? codes8(h[j], s, inv) : codes8_ieee(h[j], s);
            *reinterpret_cast<uint2 *>(a.q + row * (int64_t)a.K + (int64_t)c * 8) = out;
          }
        }
      }

      if (a.image) {
        // a block is the four chunks of four neighbouring lanes; the image's
        // columns past K (to 256) are written too, as zeros
        const int r = (int)(row & 127);
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
          const int c = at.c0 + 32 * j;
          uint32_t m = absmax_chunk(0, h[j]);
          m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          const uint32_t code = mx4_scale_code(mx4_max_bits(m));
          if (c < a.kt * 32) {
            uint8_t *tile = a.image + ((size_t)(row >> 7) * a.kt + (c >> 5)) * kMxTileBytes;
            const int b = (c >> 2) & 7;
            *reinterpret_cast<uint32_t *>(tile + mx4_chunk_offset(r, b) + (c & 3) * 4) =
                mx4_encode8(h[j], code);
            if ((c & 3) == 0) tile[mx4_scale_offset(r, b)] = (uint8_t)code;
          }
        }
      }
    }
  }
}

FuncAttrOnce g_norm_attr[4][3];            // [shape of the instance][residual]
constexpr int kMaxFolded = 4 * 4 * 14336;  // shared memory that a launch may ask for: 224 KB

template <int CPL, int RES, int REGS>
cudaError_t run(const cudaLaunchConfig_t &cfg, const NormArgs &a) {
  auto k = block_norm_kernel<CPL, RES, REGS>;
  if (cfg.dynamicSmemBytes > 40000) {
    const cudaError_t e = g_norm_attr[REGS == 160 ? 3 : CPL - 2][RES].ensure(
        [&] { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxFolded); });
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, k, a);
}
template <int CPL, int REGS>
cudaError_t run(const cudaLaunchConfig_t &cfg, const NormArgs &a) {
  if (!a.residual) return run<CPL, kNoResidual, REGS>(cfg, a);
  if constexpr (REGS <= 128)  // (more are never chosen with an fp32 residual)
    if (a.residual_f32) return run<CPL, kResidualF32, REGS>(cfg, a);
  return run<CPL, kResidualBf16, REGS>(cfg, a);
}

constexpr int64_t kMaxNormK = 16384;

bool vector_ok(const void *p, int64_t ld, int64_t K, int64_t groups) {
  return !p || ((groups <= 1 || ld == 0 || ld >= K) && ld >= 0);
}

// Rows of K elements in memory.
struct Region {
  uintptr_t at;
  int64_t stride, width;  // bytes
  int64_t end(int64_t M) const { return (M - 1) * stride + width; }
};

Region region(const void *p, int64_t ld, int64_t K, int64_t bytes) {
  return {reinterpret_cast<uintptr_t>(p), ld * bytes, K * bytes};
}

// Whether an output may be written while the input is read: the same elements
// (each is read by the thread that writes it, before it does), or none of
// them.  Rows of different strides in one range count as overlapping.
bool apart(const Region &out, const Region &in, int64_t M) {
  if (!out.at || !in.at) return true;
  if (out.at >= in.at + in.end(M) || in.at >= out.at + out.end(M)) return true;
  if (M > 1 && out.stride != in.stride) return false;
  if (out.at == in.at && out.width == in.width) return true;
  if (M == 1) return false;
  const int64_t d = (int64_t)(in.at - out.at) % out.stride, r = d < 0 ? d + out.stride : d;
  return r >= out.width && out.stride - r >= in.width;  // columns side by side
}

}  // namespace
}  // namespace w8a8

using namespace w8a8;

extern "C" w8a8_status w8a8_block_norm(const w8a8_block_norm_args *p, w8a8_stream_t stream) {
  if (!p || !p->x) return W8A8_ERR_INVALID_ARG;
  const int64_t M = p->M, K = p->K;
  if (M < 1 || M > 0x7FFFFFFF || K < 1 || p->ldx < K) return W8A8_ERR_INVALID_ARG;
  auto kind_ok = [](const w8a8_norm &n) {
    return n.kind == W8A8_NORM_NONE ||
           ((n.kind == W8A8_NORM_RMS || n.kind == W8A8_NORM_LAYER) && n.eps > 0.0f && n.eps < 1e30f);
  };
  if (!kind_ok(p->post) || !kind_ok(p->pre)) return W8A8_ERR_INVALID_ARG;
  const bool res = p->residual != nullptr;
  if (res != (p->residual_out != nullptr)) return W8A8_ERR_INVALID_ARG;
  if (res && (p->ldr < K || p->ldro < K ||
              (p->residual_dtype != W8A8_DTYPE_BF16 && p->residual_dtype != W8A8_DTYPE_FP32)))
    return W8A8_ERR_INVALID_ARG;
  // without a residual there is no branch to gate or to norm
  if (!res && (p->gate || p->post.kind != W8A8_NORM_NONE)) return W8A8_ERR_INVALID_ARG;
  const bool out = p->y || p->q || p->image;
  if (out != (p->pre.kind != W8A8_NORM_NONE) || (!out && !res)) return W8A8_ERR_INVALID_ARG;
  if ((p->q != nullptr) != (p->a_scale != nullptr)) return W8A8_ERR_INVALID_ARG;
  if ((p->scale || p->shift) && !out) return W8A8_ERR_INVALID_ARG;
  if (p->y && p->ldy < K) return W8A8_ERR_INVALID_ARG;
  const bool mod = p->gate || p->scale || p->shift;
  if (p->group_index ? (p->groups < 1 || p->groups > 0x7FFFFFFF)
                     : (mod && (p->groups < 1 || p->rows_per_group < 1 ||
                                (M - 1) / p->rows_per_group >= p->groups)))
    return W8A8_ERR_INVALID_ARG;
  if (!vector_ok(p->gate, p->ld_gate, K, p->groups) || !vector_ok(p->scale, p->ld_scale, K, p->groups) ||
      !vector_ok(p->shift, p->ld_shift, K, p->groups))
    return W8A8_ERR_INVALID_ARG;
  if (mod && p->groups > 0x7FFFFFFF) return W8A8_ERR_INVALID_ARG;
  if (K % ((p->q || p->image) ? 16 : 8) != 0 || K > kMaxNormK) return W8A8_ERR_UNSUPPORTED_SHAPE;
  const void *ptrs[] = {p->x, p->residual, p->residual_out, p->y, p->q, p->a_scale, p->image, p->gate,
                        p->scale, p->shift};
  for (const void *q : ptrs)
    if (!aligned16(q)) return W8A8_ERR_ALIGNMENT;
  for (const w8a8_norm *n : {&p->post, &p->pre})
    if (n->kind != W8A8_NORM_NONE && (!aligned16(n->weight) || !aligned16(n->bias))) return W8A8_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(p->group_index) & 3u) return W8A8_ERR_ALIGNMENT;
  const int64_t re = p->residual_dtype == W8A8_DTYPE_FP32 ? 4 : 8;
  if (p->ldx % 8 || (res && (p->ldr % re || p->ldro % re)) || (p->y && p->ldy % 8) ||
      (p->gate && p->ld_gate % 8) || (p->scale && p->ld_scale % 8) || (p->shift && p->ld_shift % 8))
    return W8A8_ERR_ALIGNMENT;
  if (p->image && p->image_bytes < (size_t)mx4_image_bytes(M, K)) return W8A8_ERR_BUFFER_TOO_SMALL;

  NormArgs a{};
  a.x = static_cast<const uint16_t *>(p->x);
  a.residual = p->residual;
  a.residual_out = p->residual_out;
  a.y = static_cast<uint16_t *>(p->y);
  a.q = p->q;
  a.a_scale = p->a_scale;
  a.image = static_cast<uint8_t *>(p->image);
  if (p->post.kind != W8A8_NORM_NONE) {  // (without the norm its vectors are not looked at)
    a.post_w = static_cast<const uint16_t *>(p->post.weight);
    a.post_b = static_cast<const uint16_t *>(p->post.bias);
  }
  if (p->pre.kind != W8A8_NORM_NONE) {
    a.pre_w = static_cast<const uint16_t *>(p->pre.weight);
    a.pre_b = static_cast<const uint16_t *>(p->pre.bias);
  }
  a.gate = static_cast<const uint16_t *>(p->gate);
  a.scale = static_cast<const uint16_t *>(p->scale);
  a.shift = static_cast<const uint16_t *>(p->shift);
  a.group_index = p->group_index;
  a.ldx = p->ldx, a.ldr = p->ldr, a.ldro = p->ldro, a.ldy = p->ldy;
  a.ld_gate = p->ld_gate, a.ld_scale = p->ld_scale, a.ld_shift = p->ld_shift;
  a.rows_per_group = mod && !p->group_index ? p->rows_per_group : 0;
  a.groups = p->groups;
  a.M = (int)M, a.K = (int)K, a.kt = (int)mx4_ktiles(K);
  a.post_kind = p->post.kind, a.pre_kind = p->pre.kind;
  a.residual_f32 = p->residual_dtype == W8A8_DTYPE_FP32;
  a.residual_scale = p->residual_scale;
  a.post_eps = p->post.eps, a.pre_eps = p->pre.eps;
  a.inv_k = 1.0f / (float)K;

  a.folded = ((a.gate || a.post_w) ? kFoldBranch : 0) | (a.post_b ? kFoldBranchAdd : 0) |
             ((a.pre_w || a.scale) ? kFoldMul : 0) | ((a.pre_b || a.shift) ? kFoldAdd : 0);
  // Chunks per lane: two, three or four, so that a CTA has at most 16 warps.
  // Where a choice is left, by the warps that an SM then holds (a row's CTA
  // may not fit twice).  Three if that makes a quarter more warps than two:
  // both norms, 4096 x 5120 60 us with two (10 warps), 45 with three (14);
  // but 4096 x 7168 67 with two (14), 76 with three (10).  Four with 160
  // registers for many rows a CTA without an fp32 residual, if at most a
  // quarter of the warps is lost: a row takes longer, but fewer instructions
  // (8192 x 4096 59 us, with two chunks 67; 1000 x 4096 13.9 and 13.0; 4096 x
  // 4096 with an fp32 residual 44.1 and 43.1; 4096 x 8192, half the warps, 77
  // and 69).  Past 8192 three, where they suffice (4000 x 10240, fp32 residual,
  // 116 us; with four 175).  The outputs have no say: y has the same bits
  // beside codes or alone.  (An image's padding columns, to 256, are always
  // within the warps' parts, whose lanes there write them.)
  const int64_t nchunks = K / 8;
  int cpl = 2, regs = 128;
  int64_t resident = 0, smem = 0;
  auto shape = [&](int c, int r) {
    cpl = c;
    regs = r;
    a.W = (int)((nchunks + 32 * c - 1) / (32 * c));
    a.padded = a.W * 32 * c;
    smem = (int64_t)a.padded * 32 * __builtin_popcount((unsigned)a.folded);
    // CTAs that the device holds, as registers and shared memory allow
    const int64_t fit = std::min<int64_t>(65536 / r / (32 * a.W), (int64_t)226 * 1024 / (smem + 2048));
    resident = sm_count() * std::min<int64_t>(32, std::max<int64_t>(1, fit));
  };
  auto warps = [&](int c, int r) {
    shape(c, r);
    return resident * a.W;
  };
  if (nchunks > kMaxWarps * 96) {
    shape(4, 128);
  } else if (nchunks > kMaxWarps * 64) {
    shape(3, 128);
  } else {
    const int64_t three = warps(3, 128), two = warps(2, 128);
    const int c = three * 4 > two * 5 ? 3 : 2;
    const bool four = !a.residual_f32 && warps(4, 160) * 4 >= (c == 3 ? three : two) * 3 &&
                      M >= 8 * resident;
    if (!four) shape(c, 128);
  }
  if (smem > kMaxFolded) return W8A8_ERR_UNSUPPORTED_SHAPE;

  const int64_t rb = p->residual_dtype == W8A8_DTYPE_FP32 ? 4 : 2;
  const Region x = region(p->x, p->ldx, K, 2), r = region(p->residual, p->ldr, K, rb);
  const Region ro = region(p->residual_out, p->ldro, K, rb), y = region(p->y, p->ldy, K, 2);
  if (!apart(ro, x, M) || !apart(ro, r, M) || !apart(y, x, M) || !apart(y, r, M) ||
      (ro.at && y.at && (ro.at == y.at || !apart(ro, y, M))))
    return W8A8_ERR_INVALID_ARG;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(M, resident));
  cfg.blockDim = dim3((unsigned)(32 * a.W));
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cpl == 2      ? run<2, 128>(cfg, a)
                        : cpl == 3    ? run<3, 128>(cfg, a)
                        : regs == 128 ? run<4, 128>(cfg, a)
                                      : run<4, 160>(cfg, a);
  if (e == cudaSuccess) count_launch();
  return from_cuda(e);
}
