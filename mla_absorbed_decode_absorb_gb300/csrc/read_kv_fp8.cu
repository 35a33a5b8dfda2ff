// The FP8 latent cache read back into bf16 rows: for each cached token,
// [bf16(s E4M3(code)) ; bf16(s f16(key))], 644 bytes in and 1152 out.
//
// "DeepSeek-MLA-Principle" section 7 names FP8 with scaling among the cache
// precisions; the non-absorbed path ("MLA 矩阵吸收 …" section 2.2) reads bf16
// rows, so a prefill over an FP8 cache goes through this copy.  One CTA takes
// half of a 64-token page of one sequence: the page id is looked up once, and each
// warp converts a token at a time with 8 codes per load, so that every store
// instruction of a warp covers 512 contiguous bytes.  Bound by HBM: 128 sequences of
// 1024 to 8192 tokens take 161 us, 0.98 of the measured copy bandwidth; 32 of 4096
// 39.4 us, 0.88 (a CTA per whole page: 164 and 41.3; 300 tokens 2.4 us against 3.2).
#include <cuda_fp16.h>

#include "internal.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Two E4M3 codes as floats (exact).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t scaled_pair(float2 v, float s) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * s, v.y * s);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__global__ void __launch_bounds__(kThreads)
read_kv_fp8_kernel(const uint8_t* __restrict__ c8, const float* __restrict__ scale, const uint16_t* __restrict__ kr,
                   int64_t num_pages, const int32_t* __restrict__ page_table, int pt_stride,
                   const int32_t* __restrict__ kv_lens, int max_kv_len, uint16_t* __restrict__ rows, int* status) {
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.y, slot = blockIdx.x >> 1, max_pages = gridDim.x >> 1;
  const int len = kv_lens[b];
  if (len < 0 || len > max_kv_len) {
    if (threadIdx.x == 0) record_status(status, MLA_ERR_BOUNDS);
    return;
  }
  // this CTA's tokens of the page: first .. n - 1
  const int first = (blockIdx.x & 1) * (kPage / 2), n = min(first + kPage / 2, len - slot * kPage);
  if (n <= first) return;
  const int page = page_table[static_cast<int64_t>(b) * pt_stride + slot];
  if (page < 0 || page >= num_pages) {
    if (threadIdx.x == 0) record_status(status, MLA_ERR_BOUNDS);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t src = static_cast<int64_t>(page) * kPage;
  const int64_t dst = (static_cast<int64_t>(b) * max_pages + slot) * kPage;
#pragma unroll 4
  for (int t = first + warp; t < n; t += kWarps) {
    const float s = scale[src + t];
    const uint2* code = reinterpret_cast<const uint2*>(c8 + (src + t) * kLatent);
    const uint2 lo = code[lane], hi = code[lane + 32];  // values [8 lane, +8) and [256 + 8 lane, +8)
    const uint32_t key = reinterpret_cast<const uint32_t*>(kr + (src + t) * kRope)[lane];
    uint16_t* out = rows + (dst + t) * kRow;
    uint4* out4 = reinterpret_cast<uint4*>(out);
    out4[lane] = make_uint4(scaled_pair(e4m3x2_to_f32(lo.x), s), scaled_pair(e4m3x2_to_f32(lo.x >> 16), s),
                            scaled_pair(e4m3x2_to_f32(lo.y), s), scaled_pair(e4m3x2_to_f32(lo.y >> 16), s));
    out4[lane + 32] = make_uint4(scaled_pair(e4m3x2_to_f32(hi.x), s), scaled_pair(e4m3x2_to_f32(hi.x >> 16), s),
                                 scaled_pair(e4m3x2_to_f32(hi.y), s), scaled_pair(e4m3x2_to_f32(hi.y >> 16), s));
    reinterpret_cast<uint32_t*>(out + kLatent)[lane] =
        scaled_pair(__half22float2(*reinterpret_cast<const __half2*>(&key)), s);
  }
}

}  // namespace

cudaError_t launch_read_kv_fp8(const uint8_t* c8, const float* scale, const uint16_t* kr, int64_t num_pages,
                               const int32_t* page_table, int pt_stride, const int32_t* kv_lens, int B,
                               int max_kv_len, uint16_t* rows, int* status, cudaStream_t stream) {
  const int max_pages = (max_kv_len - 1) / kPage + 1;
  return launch_kernel(read_kv_fp8_kernel, dim3(2 * max_pages, B), dim3(kThreads), 0, stream, c8, scale, kr, num_pages,
                       page_table, pt_stride, kv_lens, max_kv_len, rows, status);
}

}  // namespace mla
