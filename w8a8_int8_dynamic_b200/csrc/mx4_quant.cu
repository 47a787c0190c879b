// mx4_quant.cu -- to and from the microscaled 4-bit image: quantisation of
// bf16 rows, repack of a checkpoint's codes and scales, and the way back.
//
// One warp takes two rows of a 128 x 256 tile at a time: each lane 16
// consecutive elements, so a block of 32 is two lanes.  The block maximum is a
// packed 16-bit integer maximum and one shuffle; the scale is an exponent, so
// scaling is exact and the codes are one conversion of exact values; a row's
// 16 code words of 8 bytes are one full 128-byte line of the image (permuted
// by the swizzle).  Eight rows of a warp are loaded before the first is used
// (4096 x 4096: 10.1 us; with one row of eight elements a lane 11.7).
// HBM-bound: 2 bytes read and 17/32 written an element.
//
// Quantisation and dequantisation, as the products, are programmatic
// dependents: they read and write global memory only after their own wait for
// the kernel ahead, so they may follow any kernel, and never through the
// read-only path (no __ldg, no const __restrict__ pointers), since the kernel
// ahead may still be writing when they start.  These two and the few-row
// product release the next kernel at their start; the two large products do
// not.  Repack and unpack have no wait: they have to stay ordinary launches.
#include <algorithm>

#include "mx4_common.cuh"

namespace w8a8 {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantBatch = 4;    // pairs of rows in flight per warp
constexpr int kDequantBatch = 8;  // rows in flight per warp

__device__ __forceinline__ uint8_t *tile_of(uint8_t *image, int64_t slab, int kt, int ktile) {
  return image + ((size_t)slab * kt + ktile) * kMxTileBytes;
}

// grid: (K tiles, row slabs).
__global__ void __launch_bounds__(kQuantThreads)
    mx4_quant_kernel(const uint16_t *x, int64_t ldx, int64_t rows, int K, int kt, uint8_t *image) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t slab = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  const int64_t row0 = slab * kMxTileRows;
  if (row0 >= rows) return;
  const int nrows = (int)min((int64_t)kMxTileRows, rows - row0);
  uint8_t *tile = tile_of(image, slab, kt, blockIdx.x);
  const int k = blockIdx.x * kMxTileK + (lane & 15) * 16;
  const bool in_k = k < K;  // K is a multiple of 16: all sixteen or none
  const int b = (lane & 15) >> 1, half = lane & 1;
  constexpr int kStep = kQuantThreads / 16;  // rows that the CTA takes at a time
  const uint16_t *src = x + (row0 + (threadIdx.x >> 4)) * ldx + k;
  for (int r0 = threadIdx.x >> 4; r0 - (lane >> 4) < nrows; r0 += kStep * kQuantBatch) {  // (uniform in a warp)
    uint4 v[kQuantBatch][2];
#pragma unroll
    for (int i = 0; i < kQuantBatch; ++i, src += kStep * ldx) {
      v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
      if (r0 + i * kStep < nrows && in_k) {
        v[i][0] = ld_once_u4(src);
        v[i][1] = ld_once_u4(src + 8);
      }
    }
#pragma unroll
    for (int i = 0; i < kQuantBatch; ++i) {
      const int r = r0 + i * kStep;
      uint32_t m = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m = mx4_fold_max(m, v[i][h].x);
        m = mx4_fold_max(m, v[i][h].y);
        m = mx4_fold_max(m, v[i][h].z);
        m = mx4_fold_max(m, v[i][h].w);
      }
      m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      const uint32_t c = mx4_scale_code(mx4_max_bits(m));
      if (r < nrows) {
        *reinterpret_cast<uint2 *>(tile + mx4_chunk_offset(r, b) + half * 8) =
            make_uint2(mx4_encode8(v[i][0], c), mx4_encode8(v[i][1], c));
        if (half == 0) tile[mx4_scale_offset(r, b)] = (uint8_t)c;
      }
    }
  }
}

// One thread per 16-byte chunk (block) of the image; `codes` rows are K / 2
// bytes, `scales` rows ceil(K / 32) bytes, both dense.
__global__ void __launch_bounds__(256)
    mx4_pack_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                    int64_t rows, int K, int kt, uint8_t *__restrict__ image) {
  const int64_t total = rows * kt * 8;
  const int nblk = (K + 31) / 32;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / (kt * 8);
    const int blk = (int)(i - row * (kt * 8));
    uint8_t *tile = tile_of(image, row >> 7, kt, blk >> 3);
    const int r = (int)(row & 127), b = blk & 7;
    uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
    uint8_t c = 0;
    if (blk < nblk) {  // 8-byte loads: a row of codes is a multiple of 8 bytes
      const uint8_t *src = codes + row * (K / 2) + (int64_t)blk * 16;
      lo = *reinterpret_cast<const uint2 *>(src);
      if (blk * 32 + 16 < K) hi = *reinterpret_cast<const uint2 *>(src + 8);
      c = scales[row * nblk + blk];
    }
    *reinterpret_cast<uint4 *>(tile + mx4_chunk_offset(r, b)) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    tile[mx4_scale_offset(r, b)] = c;
  }
}

__global__ void __launch_bounds__(256)
    mx4_unpack_kernel(const uint8_t *__restrict__ image, int64_t rows, int K, int kt,
                      uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const int nblk = (K + 31) / 32;
  const int64_t total = rows * nblk;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / nblk;
    const int blk = (int)(i - row * nblk);
    const uint8_t *tile = image + ((size_t)(row >> 7) * kt + (blk >> 3)) * kMxTileBytes;
    const int r = (int)(row & 127), b = blk & 7;
    const uint4 v = *reinterpret_cast<const uint4 *>(tile + mx4_chunk_offset(r, b));
    uint8_t *dst = codes + row * (K / 2) + (int64_t)blk * 16;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(v.x, v.y);
    if (blk * 32 + 16 < K) *reinterpret_cast<uint2 *>(dst + 8) = make_uint2(v.z, v.w);
    scales[i] = tile[mx4_scale_offset(r, b)];
  }
}

// Codes back to bf16: a warp takes a row of a tile, a lane eight elements (with
// sixteen, a lane's two stores fill half a sector each: 4096 x 12288 28.6 us
// against 23.5).  Every value is exact in bf16 but for scales
// near the bottom of the range, where the product may be subnormal: rounded.
__global__ void __launch_bounds__(kQuantThreads)
    mx4_dequant_kernel(const uint8_t *image, int64_t rows, int K, int kt, uint16_t *x) {
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t slab = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  const int64_t row0 = slab * kMxTileRows;
  if (row0 >= rows) return;
  const int nrows = (int)min((int64_t)kMxTileRows, rows - row0);
  const uint8_t *tile = image + ((size_t)slab * kt + blockIdx.x) * kMxTileBytes;
  const int k = blockIdx.x * kMxTileK + lane * 8;
  if (k >= K) return;
  const int b = lane >> 2;
  constexpr int kWarps = kQuantThreads / 32;
  for (int r0 = warp; r0 < nrows; r0 += kWarps * kDequantBatch) {
    uint32_t q[kDequantBatch], c[kDequantBatch];
#pragma unroll
    for (int i = 0; i < kDequantBatch; ++i) {
      const int r = r0 + i * kWarps;
      q[i] = c[i] = 0;
      if (r < nrows) {
        q[i] = *reinterpret_cast<const uint32_t *>(tile + mx4_chunk_offset(r, b) + (lane & 3) * 4);
        c[i] = tile[mx4_scale_offset(r, b)];
      }
    }
#pragma unroll
    for (int i = 0; i < kDequantBatch; ++i) {
      const int r = r0 + i * kWarps;
      if (r >= nrows) break;
      const float s = mx4_scale_value(c[i]);
      uint32_t out[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t f16x2;
        asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
            : "=r"(f16x2)
            : "r"((q[i] >> (8 * h)) & 0xFFu));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&f16x2));
        const __nv_bfloat162 p = __floats2bfloat162_rn(f.x * s, f.y * s);
        out[h] = *reinterpret_cast<const uint32_t *>(&p);
      }
      *reinterpret_cast<uint4 *>(x + (row0 + r) * K + k) = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

// (K tiles, slabs): the slab index is split over y and z, each at most 65535.
dim3 tile_grid(int64_t rows, int64_t K) {
  const int64_t slabs = mx4_slabs(rows);
  const int64_t z = (slabs + 65534) / 65535;
  return dim3((unsigned)mx4_ktiles(K), (unsigned)((slabs + z - 1) / z), (unsigned)z);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*k)(Params...), dim3 grid, bool pdl, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kQuantThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, static_cast<Params>(args)...);
  if (e == cudaSuccess) count_launch();
  return e;
}

unsigned stride_blocks(int64_t threads) {
  return (unsigned)std::min<int64_t>((threads + 255) / 256, (int64_t)sm_count() * 16);
}

w8a8_status check_shape(int64_t rows, int64_t K) {
  if (rows < 1 || rows > 0x7FFFFFFF || K < 1) return W8A8_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > kMaxK) return W8A8_ERR_UNSUPPORTED_SHAPE;
  return W8A8_OK;
}

}  // namespace

w8a8_status launch_mx4_quant(const void *x, int64_t rows, int64_t K, int64_t ldx, void *image,
                             cudaStream_t stream) {
  return from_cuda(launch(mx4_quant_kernel, tile_grid(rows, K), true, stream,
                          static_cast<const uint16_t *>(x), ldx, rows, (int)K, (int)mx4_ktiles(K),
                          static_cast<uint8_t *>(image)));
}

}  // namespace w8a8

using namespace w8a8;

extern "C" {

w8a8_status w8a8_mx4_bytes(int64_t rows, int64_t K, size_t *bytes) {
  if (!bytes) return W8A8_ERR_INVALID_ARG;
  if (const w8a8_status s = check_shape(rows, K)) return s;
  *bytes = (size_t)mx4_image_bytes(rows, K);
  return W8A8_OK;
}

w8a8_status w8a8_mx4_quant(const void *x, int64_t rows, int64_t K, int64_t ldx, void *image,
                           size_t image_bytes, w8a8_stream_t stream) {
  if (!x || !image || ldx < K) return W8A8_ERR_INVALID_ARG;
  if (const w8a8_status s = check_shape(rows, K)) return s;
  if (!aligned16(x) || !aligned16(image) || ldx % 8 != 0) return W8A8_ERR_ALIGNMENT;
  if (image_bytes < (size_t)mx4_image_bytes(rows, K)) return W8A8_ERR_BUFFER_TOO_SMALL;
  return launch_mx4_quant(x, rows, K, ldx, image, reinterpret_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_mx4_pack(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K,
                          void *image, size_t image_bytes, w8a8_stream_t stream) {
  if (!codes || !scales || !image) return W8A8_ERR_INVALID_ARG;
  if (const w8a8_status s = check_shape(rows, K)) return s;
  if (!aligned16(codes) || !aligned16(image)) return W8A8_ERR_ALIGNMENT;
  if (image_bytes < (size_t)mx4_image_bytes(rows, K)) return W8A8_ERR_BUFFER_TOO_SMALL;
  const int kt = (int)mx4_ktiles(K);
  mx4_pack_kernel<<<stride_blocks(rows * kt * 8), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      codes, scales, rows, (int)K, kt, static_cast<uint8_t *>(image));
  count_launch();
  return from_cuda(cudaGetLastError());
}

w8a8_status w8a8_mx4_unpack(const void *image, int64_t rows, int64_t K, uint8_t *codes,
                            uint8_t *scales, w8a8_stream_t stream) {
  if (!codes || !scales || !image) return W8A8_ERR_INVALID_ARG;
  if (const w8a8_status s = check_shape(rows, K)) return s;
  if (!aligned16(codes) || !aligned16(image)) return W8A8_ERR_ALIGNMENT;
  mx4_unpack_kernel<<<stride_blocks(rows * ((K + 31) / 32)), 256, 0,
                      reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t *>(image), rows, (int)K, (int)mx4_ktiles(K), codes, scales);
  count_launch();
  return from_cuda(cudaGetLastError());
}

w8a8_status w8a8_mx4_dequant(const void *image, int64_t rows, int64_t K, void *x,
                             w8a8_stream_t stream) {
  if (!x || !image) return W8A8_ERR_INVALID_ARG;
  if (const w8a8_status s = check_shape(rows, K)) return s;
  if (!aligned16(x) || !aligned16(image)) return W8A8_ERR_ALIGNMENT;
  return from_cuda(launch(mx4_dequant_kernel, tile_grid(rows, K), true,
                          reinterpret_cast<cudaStream_t>(stream),
                          static_cast<const uint8_t *>(image), rows, (int)K, (int)mx4_ktiles(K),
                          static_cast<uint16_t *>(x)));
}

}  // extern "C"
