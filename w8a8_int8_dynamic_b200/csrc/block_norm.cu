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
// A row belongs to W warps, each lane holding CPL chunks of eight elements:
// x and the residual are read once, at the start, and everything until the
// stores stays in registers in fp32.  The mean is taken before the squares of
// the differences (no cancellation, whatever the mean).  The modulation and
// weight vectors are shared by many rows and come through L1.  Memory-bound:
// (2 + r) bytes read and (r + 2 | 1 | 17/32) written an element, r the bytes of
// the residual's type.
//
// A programmatic dependent that releases the next kernel at its start and
// touches memory only after its own wait.
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
  int W, R;  // warps per row, rows per CTA
};

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Eight parameters of a vector (bf16), through L1; `fill` where there is none.
__device__ __forceinline__ void params8(const uint16_t *p, int c, float fill, float (&f)[8]) {
  if (p) {
    unpack8(__ldg(reinterpret_cast<const uint4 *>(p) + c), f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fill;
  }
}

constexpr int kMaxWarps = 16;

// Sum over the row's W warps, the same in every lane.  Each call of a row has
// a shared-memory line of its own (`line`), so one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, float (*lines)[kMaxWarps], int line, int rl, int w,
                                         int W, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (W > 1) {
    float *l = lines[line] + rl * W;
    if (lane == 0) l[w] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < W; ++i) v += l[i];
  }
  return v;
}

// Normalises the lane's chunks of a row in place (without modulation).
template <int CPL>
__device__ __forceinline__ void normalise(float (&t)[CPL][8], int kind, float eps, float inv_k,
                                          const uint16_t *wp, const uint16_t *bp, int c0, int nchunks,
                                          float (*lines)[kMaxWarps], int line, int rl, int w, int W,
                                          int lane) {
  float mean = 0.0f;
  if (kind == W8A8_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < CPL; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += t[j][i];
    mean = row_sum(s, lines, line, rl, w, W, lane) * inv_k;
  }
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < CPL; ++j)
    if (c0 + 32 * j < nchunks) {  // chunks past the row hold zeros, whose difference is not zero
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[j][i] -= mean;
        s = __fmaf_rn(t[j][i], t[j][i], s);
      }
    }
  const float rstd = rsqrtf(row_sum(s, lines, line + 1, rl, w, W, lane) * inv_k + eps);
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int c = c0 + 32 * j;
    if (c < nchunks) {
      float wv[8], bv[8];
      params8(wp, c, 1.0f, wv);
      params8(bp, c, 0.0f, bv);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] = __fmaf_rn(t[j][i] * rstd, wv[i], bv[i]);
    }
  }
}

template <int CPL>
__global__ void __launch_bounds__(512) block_norm_kernel(const NormArgs a) {
  __shared__ float lines[5][kMaxWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = a.W, rl = warp / W, w = warp - rl * W;
  const int64_t row = (int64_t)blockIdx.x * a.R + rl;
  const int nchunks = a.K >> 3;
  const int c0 = w * 32 * CPL + lane;
  bool active = row < a.M;
  int64_t g = 0;
  if (active) {
    if (a.group_index) {
      g = a.group_index[row];
      active = g >= 0 && g < a.groups;  // a padding row: its outputs keep what they hold
    } else if (a.rows_per_group) {
      g = row / a.rows_per_group;
    }
  }

  // every load of the row first, so that they are in flight together
  uint4 xr[CPL], r0[CPL], r1[CPL];
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int c = c0 + 32 * j;
    const bool in = active && c < nchunks;
    xr[j] = r0[j] = r1[j] = make_uint4(0, 0, 0, 0);
    if (in) xr[j] = ld_stream_u4(a.x + row * a.ldx + (int64_t)c * 8);
    if (in && a.residual) {
      if (a.residual_f32) {
        const float *p = static_cast<const float *>(a.residual) + row * a.ldr + (int64_t)c * 8;
        r0[j] = *reinterpret_cast<const uint4 *>(p);
        r1[j] = *reinterpret_cast<const uint4 *>(p + 4);
      } else {
        r0[j] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.residual) +
                                                 row * a.ldr + (int64_t)c * 8);
      }
    }
  }
  float t[CPL][8];
#pragma unroll
  for (int j = 0; j < CPL; ++j) unpack8(xr[j], t[j]);

  if (a.post_kind != W8A8_NORM_NONE)
    normalise<CPL>(t, a.post_kind, a.post_eps, a.inv_k, a.post_w, a.post_b, c0, nchunks, lines, 0, rl, w,
                   W, lane);

  if (a.residual) {
    const uint16_t *gate = a.gate ? a.gate + g * a.ld_gate : nullptr;
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = c0 + 32 * j;
      if (!(active && c < nchunks)) continue;
      float r[8], gv[8];
      if (a.residual_f32) {
        const uint32_t b[8] = {r0[j].x, r0[j].y, r0[j].z, r0[j].w, r1[j].x, r1[j].y, r1[j].z, r1[j].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(b[i]);
      } else {
        unpack8(r0[j], r);
      }
      params8(gate, c, 1.0f, gv);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] = __fmaf_rn(gv[i], t[j][i], a.residual_scale * r[i]);
      if (a.residual_f32) {
        float *p = static_cast<float *>(a.residual_out) + row * a.ldro + (int64_t)c * 8;
        *reinterpret_cast<float4 *>(p) = make_float4(t[j][0], t[j][1], t[j][2], t[j][3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(t[j][4], t[j][5], t[j][6], t[j][7]);
      } else {
        const uint4 v = pack8(t[j]);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.residual_out) + row * a.ldro +
                                   (int64_t)c * 8) = v;
        unpack8(v, t[j]);  // the norm is of the stream as it is stored
      }
    }
  }

  if (a.pre_kind == W8A8_NORM_NONE) return;
  normalise<CPL>(t, a.pre_kind, a.pre_eps, a.inv_k, a.pre_w, a.pre_b, c0, nchunks, lines, 2, rl, w, W,
                 lane);

  const uint16_t *scale = a.scale ? a.scale + g * a.ld_scale : nullptr;
  const uint16_t *shift = a.shift ? a.shift + g * a.ld_shift : nullptr;
  uint4 h[CPL];
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int c = c0 + 32 * j;
    h[j] = make_uint4(0, 0, 0, 0);
    if (!(active && c < nchunks)) continue;
    if (scale || shift) {
      float sv[8], tv[8];
      params8(scale, c, 0.0f, sv);
      params8(shift, c, 0.0f, tv);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] = __fmaf_rn(t[j][i], 1.0f + sv[i], tv[i]);
    }
    h[j] = pack8(t[j]);
    if (a.y) *reinterpret_cast<uint4 *>(a.y + row * a.ldy + (int64_t)c * 8) = h[j];
    mx = absmax_chunk(mx, h[j]);
  }

  if (a.q) {  // as the int8 quantisation kernel, on the rounded row
    uint32_t m = absmax_fold(mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (W > 1) {
      uint32_t *l = reinterpret_cast<uint32_t *>(lines[4]) + rl * W;
      if (lane == 0) l[w] = m;
      __syncthreads();
      for (int i = 0; i < W; ++i) m = max(m, l[i]);
    }
    if (active) {
      const float amax = __uint_as_float(m << 16);
      const float s = amax == 0.0f ? 0.0f : __fdiv_rn(amax, 127.0f);
      const float inv = amax == 0.0f ? 0.0f : __frcp_rn(s);
      if (w == 0 && lane == 0) a.a_scale[row] = s;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        const int c = c0 + 32 * j;
        if (c >= nchunks) continue;
        uint2 out = make_uint2(0, 0);
        if (amax != 0.0f) out = s >= 1e-30f ? codes8(h[j], s, inv) : codes8_ieee(h[j], s);
        *reinterpret_cast<uint2 *>(a.q + row * (int64_t)a.K + (int64_t)c * 8) = out;
      }
    }
  }

  if (a.image && active) {
    // a block is the four chunks of four neighbouring lanes; the image's
    // columns past K (to 256) are written too, as zeros
    const int r = (int)(row & 127);
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const int c = c0 + 32 * j;
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

bool vector_ok(const void *p, int64_t ld, int64_t K, int64_t groups) {
  return !p || ((groups <= 1 || ld == 0 || ld >= K) && ld >= 0);
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
  if (K % ((p->q || p->image) ? 16 : 8) != 0 || K > kMaxWarps * 32 * 8 * 8) return W8A8_ERR_UNSUPPORTED_SHAPE;
  const void *ptrs[] = {p->x, p->residual, p->residual_out, p->y, p->q, p->a_scale, p->image, p->gate,
                        p->scale, p->shift, p->post.weight, p->post.bias, p->pre.weight, p->pre.bias};
  for (const void *q : ptrs)
    if (!aligned16(q)) return W8A8_ERR_ALIGNMENT;
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
  a.post_w = static_cast<const uint16_t *>(p->post.weight);
  a.post_b = static_cast<const uint16_t *>(p->post.bias);
  a.pre_w = static_cast<const uint16_t *>(p->pre.weight);
  a.pre_b = static_cast<const uint16_t *>(p->pre.bias);
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

  // Chunks per lane: 4, or 8 where a row would need more than 16 warps; an
  // image's padding columns count (the lanes that hold them write them).
  const int64_t nchunks = a.image ? (int64_t)a.kt * 32 : K / 8;
  const int64_t per_lane = (nchunks + 31) / 32;
  int cpl = 1;
  while (cpl < 4 && cpl < per_lane) cpl *= 2;
  if ((nchunks + 32 * cpl - 1) / (32 * cpl) > kMaxWarps) cpl = 8;
  a.W = (int)((nchunks + 32 * cpl - 1) / (32 * cpl));
  a.R = a.W >= 4 ? 1 : 4 / a.W;  // about 128 threads a CTA
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((M + a.R - 1) / a.R));
  cfg.blockDim = dim3((unsigned)(32 * a.W * a.R));
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cpl == 1   ? cudaLaunchKernelEx(&cfg, block_norm_kernel<1>, a)
                        : cpl == 2 ? cudaLaunchKernelEx(&cfg, block_norm_kernel<2>, a)
                        : cpl == 4 ? cudaLaunchKernelEx(&cfg, block_norm_kernel<4>, a)
                                   : cudaLaunchKernelEx(&cfg, block_norm_kernel<8>, a);
  if (e == cudaSuccess) count_launch();
  return from_cuda(e);
}
