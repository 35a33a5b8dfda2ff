// bf16 weights into the 4-bit format with group scales, and back.
//
//   s = bf16(max|w| / 7) over each 128 columns of a row (1 where that is zero)
//   u = clamp(round(w / s), -8, 7) + 8        w' = bf16((u - 8) s)
//
// Every step is one IEEE operation on exactly representable values (a quotient
// of two bf16 values is never so near a tie that fp32 rounds it across), so the
// codes are reproducible bit for bit.  16 lanes hold a group, 8 columns each;
// both kernels stream and are bound by HBM.
#include "w4.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
quantize_w4_kernel(const uint16_t* __restrict__ w, uint32_t* __restrict__ w4, uint16_t* __restrict__ scale,
                   uint32_t units, uint32_t groups, int K) {
  grid_dep_wait();
  grid_dep_launch();
  // unit = one group of one row; the 16 lanes of a half warp share it
  const int sub = threadIdx.x & 15;
  const uint32_t per_block = kThreads / 16;
  for (uint64_t u0 = static_cast<uint64_t>(blockIdx.x) * per_block; u0 < units;
       u0 += static_cast<uint64_t>(gridDim.x) * per_block) {
    const uint64_t u = u0 + (threadIdx.x >> 4);
    const bool here = u < units;
    const uint32_t row = here ? static_cast<uint32_t>(u) / groups : 0;
    const uint32_t g = here ? static_cast<uint32_t>(u) - row * groups : 0;
    const int col = static_cast<int>(g) * kW4Group + sub * 8;
    const bool in = here && col < K;
    const int64_t at = static_cast<int64_t>(row) * K + col;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in) v = *reinterpret_cast<const uint4*>(w + at);
    const uint32_t bits[4] = {v.x, v.y, v.z, v.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(bits[i] << 16);
      x[2 * i + 1] = __uint_as_float(bits[i] & 0xffff0000u);
    }
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    uint16_t sb = f32_to_bf16_bits(__fdiv_rn(a, 7.f));
    if (sb == 0) sb = 0x3f80;  // a group of zeros (or below bf16's smallest scale): s = 1
    const float s = bf16_bits_to_f32(sb);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -8.f), 7.f);
      word |= static_cast<uint32_t>(static_cast<int>(c) + 8) << (4 * i);
    }
    if (in) w4[at >> 3] = word;
    if (here && sub == 0) scale[u] = sb;
  }
}

__global__ void __launch_bounds__(kThreads)
dequantize_w4_kernel(const uint32_t* __restrict__ w4, const uint16_t* __restrict__ scale, uint16_t* __restrict__ w,
                     uint32_t units, uint32_t groups, int K) {
  grid_dep_wait();
  grid_dep_launch();
  const int sub = threadIdx.x & 15;
  const uint32_t per_block = kThreads / 16;
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * per_block + (threadIdx.x >> 4); u < units;
       u += static_cast<uint64_t>(gridDim.x) * per_block) {
    const uint32_t row = static_cast<uint32_t>(u) / groups;
    const int col = static_cast<int>(static_cast<uint32_t>(u) - row * groups) * kW4Group + sub * 8;
    if (col >= K) continue;
    const int64_t at = static_cast<int64_t>(row) * K + col;
    const uint32_t v = w4[at >> 3];
    const float s = bf16_bits_to_f32(scale[u]);
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lo = static_cast<int>((v >> (8 * i)) & 15u) - 8, hi = static_cast<int>((v >> (8 * i + 4)) & 15u) - 8;
      const __nv_bfloat162 b = __floats2bfloat162_rn(static_cast<float>(lo) * s, static_cast<float>(hi) * s);
      out[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(w + at) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

unsigned blocks_for(uint32_t units) {
  const uint64_t want = (static_cast<uint64_t>(units) + kThreads / 16 - 1) / (kThreads / 16);
  return static_cast<unsigned>(want < (1u << 30) ? want : (1u << 30));
}

}  // namespace

cudaError_t launch_quantize_w4(const uint16_t* w, uint8_t* w4, uint16_t* scale, int N, int K, cudaStream_t stream) {
  const uint32_t groups = w4_groups(K), units = static_cast<uint32_t>(N) * groups;
  return launch_kernel(quantize_w4_kernel, dim3(blocks_for(units)), dim3(kThreads), 0, stream, w,
                       reinterpret_cast<uint32_t*>(w4), scale, units, groups, K);
}

cudaError_t launch_dequantize_w4(const uint8_t* w4, const uint16_t* scale, uint16_t* w, int N, int K,
                                 cudaStream_t stream) {
  const uint32_t groups = w4_groups(K), units = static_cast<uint32_t>(N) * groups;
  return launch_kernel(dequantize_w4_kernel, dim3(blocks_for(units)), dim3(kThreads), 0, stream,
                       reinterpret_cast<const uint32_t*>(w4), scale, w, units, groups, K);
}

}  // namespace mla
