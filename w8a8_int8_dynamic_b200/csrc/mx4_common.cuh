// mx4_common.cuh -- the microscaled 4-bit (MX: e2m1 values, one e8m0 scale to
// a block of 32) matrix image and the pieces its kernels share.
//
// Format: OCP Microscaling Formats (MX) v1.0, MXFP4.  A block is 32
// consecutive elements of a row.  Its scale is 2^(c - 127) with the byte c,
// c = 255 standing for NaN; its elements are sign, 2 exponent bits and 1
// mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.
//
// Image of a [rows, K] matrix: tiles of 128 rows x 256 elements, row slab by
// row slab (tile (s, k) at index s * ceil(K / 256) + k), each 17,408 bytes:
//   16,384 bytes of codes: the K-major 128-byte-swizzled shared-memory image
//     that tcgen05.mma reads.  Row r has 128 bytes; block b (0..7) of the row
//     is its 16-byte chunk b, stored at chunk position b ^ (r & 7).  Two codes
//     to a byte, the lower k in the low half;
//   1,024 bytes of scales: two groups of four blocks (128 elements), each the
//     32 x 16-byte source of tcgen05.cp.32x128b: the scale of block 4 g + j
//     of row r at g * 512 + (r % 32) * 16 + (r / 32) * 4 + j.
// One tile is one contiguous copy into one pipeline stage, codes and scales
// together, for either operand: activations and weights have the same image.
// K is padded to 256 with zero codes (scale byte 0); rows past the last one
// of a slab are never written: they can only reach outputs that are not stored.
#pragma once

#include <cuda_bf16.h>

#include "act.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace w8a8 {

// One lane of a converged warp (the same one on every call).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// 16 bytes that are read once, through the coherent path: for what the kernel
// ahead in the stream may have written after this one started (the read-only
// path is for memory that nothing writes while the kernel runs).
__device__ __forceinline__ uint4 ld_once_u4(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

constexpr int kMxTileRows = 128;
constexpr int kMxTileK = 256;                // elements: 128 bytes of codes a row
constexpr int kMxCodeBytes = 128 * 128;      // 16 KB
constexpr int kMxScaleBytes = 1024;
constexpr int kMxTileBytes = kMxCodeBytes + kMxScaleBytes;  // 17 KB, a multiple of 1024
constexpr int kMxGroupBytes = 512;           // scales of 128 rows x 128 elements

__host__ __device__ __forceinline__ int64_t mx4_ktiles(int64_t K) {
  return (K + kMxTileK - 1) / kMxTileK;
}
__host__ __device__ __forceinline__ int64_t mx4_slabs(int64_t rows) {
  return (rows + kMxTileRows - 1) / kMxTileRows;
}
inline int64_t mx4_image_bytes(int64_t rows, int64_t K) {
  return mx4_slabs(rows) * mx4_ktiles(K) * kMxTileBytes;
}

// Offsets inside a tile: the 16-byte chunk of block b of row r, and its scale byte.
__device__ __forceinline__ uint32_t mx4_chunk_offset(int r, int b) {
  return (uint32_t)(r * 128 + ((b ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint32_t mx4_scale_offset(int r, int b) {
  return (uint32_t)(kMxCodeBytes + (b >> 2) * kMxGroupBytes + (r & 31) * 16 + (r >> 5) * 4 + (b & 3));
}

// The scale byte of a block whose largest bf16 magnitude has the bits `m`
// (order of the 15 low bits = order of the magnitudes, Inf and NaN on top):
// floor(log2(amax)) - 2 + 127, where floor(log2) is the exponent field - 127;
// at least 0 (2^-127), which zero and subnormal maxima get; 255 (NaN) for a
// block that holds an infinity or a NaN.
__device__ __forceinline__ uint32_t mx4_scale_code(uint32_t m) {
  const uint32_t f = m >> 7;
  return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}
// 2^-(c - 127), c <= 252: the factor that brings the block's values into
// (-8, 8).  Exact: the products are bf16 values times a power of two, and one
// that underflows would have rounded to zero anyway.
__device__ __forceinline__ float mx4_inverse_scale(uint32_t c) {
  return __uint_as_float((254u - c) << 23);
}
__device__ __forceinline__ float mx4_scale_value(uint32_t c) {
  return c == 255u ? __uint_as_float(0x7FC00000u)
                   : __uint_as_float(c == 0u ? 0x00400000u : c << 23);
}

// Eight scaled values -> eight codes (round to nearest, ties to the even
// code, magnitudes past 6 to 6; zeros keep their sign), element 0 in the low
// half of the low byte.
__device__ __forceinline__ uint32_t mx4_codes8(float v0, float v1, float v2, float v3, float v4,
                                               float v5, float v6, float v7) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3), "f"(v4), "f"(v5), "f"(v6), "f"(v7));
  return r;
}

// One value of a block with scale code c -> its code.
__device__ __forceinline__ uint32_t mx4_code1(float v, uint32_t c) {
  if (c == 255u) return 0u;
  uint32_t r;
  asm("{\n\t.reg .b8 b, z;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "mov.b32 %0, {b, z, z, z};\n\t}"
      : "=r"(r)
      : "f"(v * mx4_inverse_scale(c)), "f"(0.0f));
  return r & 15u;
}

// Eight bf16 values (four packed pairs) of a block with scale code c -> codes.
__device__ __forceinline__ uint32_t mx4_encode8(const uint4 &x, uint32_t c) {
  if (c == 255u) return 0u;
  const uint64_t inv = f2_splat(mx4_inverse_scale(c));
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f2_unpack(f2_mul(f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), inv),
              v[2 * i], v[2 * i + 1]);
  return mx4_codes8(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
}

// The larger magnitude bits of a packed bf16 pair's halves, folded into m.
__device__ __forceinline__ uint32_t mx4_fold_max(uint32_t m, uint32_t pair) {
  return __vmaxu2(m, pair & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t mx4_max_bits(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

// A whole block in one thread: 16 packed bf16 pairs -> 16 bytes of codes and
// the scale byte.
__device__ __forceinline__ uint32_t mx4_encode_block(const uint4 (&x)[4], uint4 &codes) {
  uint32_t m = 0;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    m = mx4_fold_max(m, x[g].x);
    m = mx4_fold_max(m, x[g].y);
    m = mx4_fold_max(m, x[g].z);
    m = mx4_fold_max(m, x[g].w);
  }
  const uint32_t c = mx4_scale_code(mx4_max_bits(m));
  codes = make_uint4(mx4_encode8(x[0], c), mx4_encode8(x[1], c), mx4_encode8(x[2], c),
                     mx4_encode8(x[3], c));
  return c;
}

// ---- tcgen05 with block scales --------------------------------------------------
// Instruction descriptor of tcgen05.mma kind::mxf4 (dense, K = 64): B scale id
// in bits 4-5, A e2m1 (bits 7-9 = 1), B e2m1 (10-12 = 1), both K-major, N >> 3
// in bits 17-22, scales e8m0 (bit 23), M >> 4 in bits 24-28, A scale id in bits
// 29-30.  With two scales a row and instruction (scale_vec::2X) the ids are the
// byte of the 32-bit scale column at which the pair starts: 0 or 2.
__host__ __device__ constexpr uint32_t idesc_mx4(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kMxSecondPair = (2u << 29) | (2u << 4);  // both scale ids = 2

__device__ __forceinline__ void mma_mx4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
          "r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_mx4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
          "r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Shared-memory descriptor of a 512-byte scale group for tcgen05.cp.32x128b:
// no swizzle, 8 x 16-byte core matrices 128 bytes apart (stride field), one
// core matrix wide.
__device__ __forceinline__ uint64_t mx4_scale_desc(const void *smem) {
  const uint64_t addr = (smem_addr(smem) >> 4) & 0x3FFFu;
  return addr | (8ull << 16) | (8ull << 32) | (1ull << 46);
}

// 32 rows x 16 bytes of shared memory -> 4 TMEM columns, repeated in the four
// lane quarters.  Executes in order with later MMAs of the same thread.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// What every product kernel takes.  Output: y (bf16 [M, N]), or, with
// `y_image`, the image of y, which is the next product's left operand.
struct Mx4Args {
  const uint8_t *a;      // image of [M, K]
  const uint8_t *w;      // image of [N, K]
  const uint16_t *bias;  // bf16 [N], may be null
  uint16_t *y;
  uint8_t *y_image;
  int M, N;
  int kt;                // 256-element tiles of K
  int y_kt;              // tiles of the output image's K (= N)
  int tiles_m, tiles_n;
  int row_major;         // tile order (see mx4_tile_coords)
  int act;               // w8a8_act
  int *status;
};

// Few rows (mx4_stream.cu), M <= kStreamRows.  x: bf16 rows that the kernel
// quantises itself (M <= kStreamQuantRows), or null: p.a is their image.
constexpr int64_t kStreamRows = 128, kStreamQuantRows = 16;
constexpr int kMaxStreamCluster = 4;
w8a8_status launch_mx4_stream(const Mx4Args &p, const void *x, int64_t ldx, int64_t K, cudaStream_t stream);

// Many rows (mx4_pair.cu): 256 x 256 tiles on CTA pairs.
w8a8_status launch_mx4_pair(Mx4Args a, cudaStream_t stream);

// The bias, activation and rounding of 8 consecutive outputs of a row.
template <int ACT>
__device__ __forceinline__ uint4 mx4_finish8(const uint32_t *acc, const uint16_t *bias) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = __uint_as_float(acc[i]);
  const uint4 b = *reinterpret_cast<const uint4 *>(bias);
  const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    t[2 * h] = __fadd_rn(t[2 * h], __uint_as_float(bw[h] << 16));
    t[2 * h + 1] = __fadd_rn(t[2 * h + 1], __uint_as_float(bw[h] & 0xFFFF0000u));
  }
  if (ACT != W8A8_ACT_NONE) {
#pragma unroll
    for (int h = 0; h < 4; ++h) apply_act_pair(t[2 * h], t[2 * h + 1], ACT);
  }
  uint32_t r[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(t[2 * h], t[2 * h + 1]);
    r[h] = *reinterpret_cast<const uint32_t *>(&p);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace w8a8
