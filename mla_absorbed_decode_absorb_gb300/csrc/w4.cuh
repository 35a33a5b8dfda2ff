// The 4-bit weight format and its conversions to bf16 pairs.
//
// A weight row of K values is K / 2 bytes, column 2i in the low half of byte i
// and column 2i + 1 in the high half; a half byte u stands for (u - 8) * s with
// one bf16 scale s for each 128 columns.
#pragma once

#include <cuda_fp16.h>

#include "sm100.cuh"

namespace mla {

constexpr int kW4Group = MLA_W4_GROUP;
__host__ __device__ inline int w4_groups(int K) { return (K + kW4Group - 1) / kW4Group; }

// (v & mask) | bits as the one instruction it is (left to itself the compiler made two, and this conversion is most of
// what a projection of few tokens issues).
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
  return d;
}

// Integers to floats without a conversion instruction, by the published method of placing them in the low bits of a
// constant's significand and taking the constant off (Kim, Henry, Fahim, Hassan Awadalla: "Who Says Elephants Can't
// Run: Bringing Large Scale MoE Models into Cloud Scale Production", 2022); the constants follow from the formats.
//
// The eight half bytes u_0 .. u_7 of a word as four bf16 pairs (u_i - 8, u_{i+4} - 8),
// i = 0 .. 3: 0x4300 is 128, whose bf16 unit in the last place is 1, so 0x4300 | u
// is 128 + u, and the difference to 136 is exact.
__device__ __forceinline__ void w4_pairs(uint32_t v, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t biased = and_or(v >> (4 * i), 0x000f000fu, 0x43004300u);
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(biased), "r"(0x43084308u));
  }
}

// The eight half bytes in their own order, as pairs (u_{2i} - 8, u_{2i+1} - 8): two instructions more.
__device__ __forceinline__ void w4_pairs_natural(uint32_t v, uint32_t (&p)[4]) {
  const uint32_t even = v & 0x0f0f0f0fu, odd = (v >> 4) & 0x0f0f0f0fu;
  const uint32_t lo = __byte_perm(even, odd, 0x5140), hi = __byte_perm(even, odd, 0x7362);  // u_0 .. u_3, u_4 .. u_7
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t biased = __byte_perm(i < 2 ? lo : hi, 0x43434343u, i & 1 ? 0x4342 : 0x4140);
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(biased), "r"(0x43084308u));
  }
}

// The eight half bytes in their own order as E4M3 codes of (u - 8) 2^-9: E4M3's subnormals and its first binade have
// one step, 2^-9, so the code of a magnitude m <= 8 is m itself, and the sign is bit 7.
__device__ __forceinline__ void w4_e4m3(uint32_t v, uint32_t (&c)[2]) {
  const uint32_t even = v & 0x0f0f0f0fu, odd = (v >> 4) & 0x0f0f0f0fu;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = __byte_perm(even, odd, i ? 0x7362 : 0x5140);
    const uint32_t neg = ~(u >> 3) & 0x01010101u;  // 1 in the bytes with u < 8
    c[i] = ((u & 0x07070707u) ^ (neg * 7u)) + neg * 0x81u;  // u < 8: (7 - u) + 1, sign set; else u - 8
  }
}

// The pairs of w4_pairs in f16: 0x6400 is 1024, whose unit in the last place is 1, so a half byte
// in the low bits adds u and one four bits up adds 16 u; both ways back are exact.
__device__ __forceinline__ void w4_pairs_f16(uint32_t v, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = and_or(v >> (8 * i), 0x000f000fu, 0x64006400u);  // 1024 + u
    const uint32_t hi = and_or(v >> (8 * i), 0x00f000f0u, 0x64006400u);  // 1024 + 16 u
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[2 * i]) : "r"(lo), "r"(0x64086408u));                       // - 1032
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[2 * i + 1]) : "r"(hi), "r"(0x2c002c00u), "r"(0xd480d480u));  // / 16 - 72
  }
}

// ------------------------------------------------------------------ projections
constexpr int kW4MaxSplit = 8;  // CTAs of a cluster along K (the portable size)

// One projection's weight and output.
struct W4Out {
  const uint8_t* w4;    // [N, K / 2]
  const uint16_t* sw;   // [N, groups] bf16
  uint16_t* y;          // [T, N] bf16
  int N;
};

struct W4Params {
  const void* x;        // bf16 [T, K] or E4M3 [T, K]
  const float* sx;      // [T, groups] (E4M3 x)
  W4Out out[2];         // one projection of x, or two (out[1].N > 0) in one launch
  int* status;
  int T, K, groups;
  int tiles0;           // tiles of the first projection: CTA tiles from there on compute the second
  int split, per;       // CTAs of a cluster; groups per CTA (csrc/linear_w4.cu)
  int share;            // tiles of a cluster (csrc/linear_w4_tc.cu)
  int all, slices;      // tiles in all, and of the same features (slices of the tokens), there
  bool early;           // the weights may be read before the previous kernel has finished

  // Tiles of `rows` features of both projections, in order.
  __host__ int64_t tiles(int rows) const {
    return (static_cast<int64_t>(out[0].N) + rows - 1) / rows + (static_cast<int64_t>(out[1].N) + rows - 1) / rows;
  }
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// The float at shared address `at` of every CTA of the cluster, added in rank order (all loads in flight together).
__device__ __forceinline__ float sum_partials(uint32_t at, int split) {
  float v[kW4MaxSplit];
  if (split == 1) {
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(at) : "memory");
    return v[0];
  }
#pragma unroll
  for (int q = 0; q < kW4MaxSplit; ++q) v[q] = q < split ? ld_cluster_f32(sm100::mapa(at, q)) : 0.f;
  float sum = v[0];
#pragma unroll
  for (int q = 1; q < kW4MaxSplit; ++q) sum += v[q];
  return sum;
}
// The same of four floats in the CTAs lo .. hi, at `at_hi` in the last one.
__device__ __forceinline__ float4 sum_partials(uint32_t at, uint32_t at_hi, int lo, int hi) {
  float4 v[kW4MaxSplit];
#pragma unroll
  for (int q = 0; q < kW4MaxSplit; ++q) {
    v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lo + q <= hi)
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[q].x), "=f"(v[q].y), "=f"(v[q].z), "=f"(v[q].w)
                   : "r"(sm100::mapa(lo + q == hi ? at_hi : at, lo + q))
                   : "memory");
  }
  float4 sum = v[0];
#pragma unroll
  for (int q = 1; q < kW4MaxSplit; ++q) {
    sum.x += v[q].x;
    sum.y += v[q].y;
    sum.z += v[q].z;
    sum.w += v[q].w;
  }
  return sum;
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return f32_to_bf16_bits(a) | (static_cast<uint32_t>(f32_to_bf16_bits(b)) << 16);
}

// Eight values of x, as loaded, as MMA operands in the pair order (0,4) (1,5) (2,6) (3,7); E4M3 codes become f16
// (exact).  Volatile: the values are loaded a group ahead, and moved up to their load these would wait for it.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm volatile("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return h;
}
__device__ __forceinline__ uint4 pair_order(const uint4& v) {
  return make_uint4(prmt(v.x, v.z, 0x5410), prmt(v.x, v.z, 0x7632), prmt(v.y, v.w, 0x5410), prmt(v.y, v.w, 0x7632));
}
__device__ __forceinline__ uint4 pair_order(const uint2& v) {
  const uint32_t a = prmt(v.x, v.y, 0x5140), c = prmt(v.x, v.y, 0x7362);
  return make_uint4(e4m3x2_to_f16x2(a), e4m3x2_to_f16x2(a >> 16), e4m3x2_to_f16x2(c), e4m3x2_to_f16x2(c >> 16));
}

// The launch of a projection kernel: clusters of `split` CTAs along x.
struct W4Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  W4Launch(dim3 grid, int threads, size_t smem, cudaStream_t stream, int split) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = launch_overlap() > 0 ? 2 : 1;
  }
};
template <typename... KArgs, typename... Args>
cudaError_t launch_w4(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int split,
                      const Args&... args) {
  W4Launch l(grid, threads, smem, stream, split);
  return cudaLaunchKernelEx(&l.cfg, kernel, args...);
}
// Clusters of `split` CTAs that are resident on the current device at once (at least 1).
template <typename... KArgs>
cudaError_t w4_clusters(void (*kernel)(KArgs...), int threads, size_t smem, int split, int* n) {
  W4Launch l(dim3(split), threads, smem, nullptr, split);
  l.cfg.numAttrs = 1;
  *n = 0;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(n, kernel, &l.cfg);
  if (*n < 1) *n = 1;
  return e;
}

// More than a few tokens (csrc/linear_w4_tc.cu).
cudaError_t launch_linear_w4_tc(const W4Params& p, cudaStream_t stream);

}  // namespace mla
