// y[T, N] = x[T, K] W[N, K]^T with 4-bit weights and a scale for each 128
// columns, for a few tokens (T <= 256), x in bf16 or in E4M3 with a scale for
// each 128 columns of a token:
//
//   y[t, n] = sum_g sw[n, g] sx[t, g] sum_{k in g} (u[n, k] - 8) x[t, k]
//
// (sx = 1 for bf16 x.)  u - 8 and an E4M3 code are exact in bf16, so the inner
// sum is a bf16 matrix product with fp32 accumulation of exact products, and
// the scales enter in fp32 once per group: nothing is rounded below fp32 before
// the one rounding of y.
//
// A few tokens leave the work at streaming W once: half a byte per weight.
// Weights are the 16-row side of the warp MMA (m16n8k16), tokens the 8-column
// side.  A warp streams the 1 KB of one group of its 16 rows at a time through a
// cp.async ring of its own, so no barrier stands between the warps until their
// sums meet.  The K order inside an MMA is free as long as both operands agree:
// lane (g, t) = (lane / 4, lane % 4) takes word 4 j + t of rows g and g + 8, the
// columns 8 (4 j + t) + 0..7, whose half bytes i and i + 4 come out as one pair,
// and the same 8 columns of token g in the same pair order.  (The words lie in
// shared memory with the 16-byte units of row r at j ^ (r / 2 % 4), which keeps a
// warp's 32 words in 32 banks.)  8-bit x goes through f16, bf16 x through bf16.
//
// K is split over the warps of a CTA and the CTAs of a cluster; each CTA keeps its
// partials in shared memory and the cluster adds them in rank order through
// distributed shared memory, so a call needs no workspace and its result does not
// depend on timing.
#include <cuda_fp16.h>
#include <stdlib.h>

#include <type_traits>

#include "sm100.cuh"
#include "w4.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 8;         // groups a warp has in flight or in use, 1 KB each
constexpr int kMaxSplit = 8;       // CTAs of a cluster along K (the portable size)

struct W4Params {
  const void* x;        // bf16 [T, K] or E4M3 [T, K]
  const float* sx;      // [T, groups] (E4M3 x)
  const uint8_t* w4;    // [N, K / 2]
  const uint16_t* sw;   // [N, groups] bf16
  uint16_t* y;          // [T, N] bf16
  int T, K, N, groups;
  int split, per;       // CTAs along K, groups per CTA
  bool early;           // the weights may be read before the previous kernel has finished
};

template <bool kF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Two E4M3 codes (the low 16 bits) as an f16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return h;
}

// Eight values of x, as loaded, to MMA operands in the pair order (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ void pair_order(const uint4& v, uint32_t (&b)[4]) {
  b[0] = __byte_perm(v.x, v.z, 0x5410);
  b[1] = __byte_perm(v.x, v.z, 0x7632);
  b[2] = __byte_perm(v.y, v.w, 0x5410);
  b[3] = __byte_perm(v.y, v.w, 0x7632);
}
__device__ __forceinline__ void pair_order(const uint2& v, uint32_t (&b)[4]) {
  const uint32_t a = __byte_perm(v.x, v.y, 0x5140), c = __byte_perm(v.x, v.y, 0x7362);
  b[0] = e4m3x2_to_f16x2(a);
  b[1] = e4m3x2_to_f16x2(a >> 16);
  b[2] = e4m3x2_to_f16x2(c);
  b[3] = e4m3x2_to_f16x2(c >> 16);
}

// kRowWarps warps cover 16 rows each, the other kWarps / kRowWarps share their
// groups of K; kTiles tiles of 8 tokens.
template <int kRowWarps, int kTiles>
struct W4Shape {
  static constexpr int kKWarps = kWarps / kRowWarps;
  static constexpr int kRows = 16 * kRowWarps;
  static constexpr int kTok = 8 * kTiles;
  static constexpr int kLd = kRows + 4;  // floats per token of a partial: conflict-free fragment stores
  static constexpr int kRing = kStages * kWarps * 1024;
  static constexpr int kPart = kKWarps * kTok * kLd * 4;  // lies over the ring
  static constexpr int kSmem = kRing > kPart ? kRing : kPart;
};

// What one group needs besides its weights.
template <int kTiles, bool kFp8>
struct W4Operands {
  std::conditional_t<kFp8, uint2, uint4> x[kTiles][4];
  float sx[kTiles][2];
  float sw[2];
};

template <int kRowWarps, int kTiles, bool kFp8>
__global__ void __launch_bounds__(kThreads)
linear_w4_kernel(const W4Params p) {
  using S = W4Shape<kRowWarps, kTiles>;
  using Vec = std::conditional_t<kFp8, uint2, uint4>;  // 8 values of x
  extern __shared__ __align__(16) uint8_t smem[];
  float* part = reinterpret_cast<float*>(smem);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lg = lane >> 2, lt = lane & 3;
  const int rw = warp % kRowWarps, kw = warp / kRowWarps;
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const int n0 = tile * S::kRows;
  const int t0 = blockIdx.z * S::kTok;
  const int g0 = rank * p.per + kw, g1 = min(p.groups, rank * p.per + p.per);
  if (!p.early) grid_dep_wait();

  const int r0 = n0 + rw * 16 + lg;
  const int64_t row_bytes = p.K >> 1;
  const uint8_t* src0 = p.w4 + static_cast<int64_t>(r0) * row_bytes + lt * 16;
  const bool in0 = r0 < p.N, in1 = r0 + 8 < p.N;
  const uint32_t ring = smem_u32(smem) + warp * 1024;
  const uint32_t sw_off = (lg >> 1 & 3) << 4;  // the row's 16-byte unit permutation
  const uint32_t put = ring + lg * 64 + ((lt << 4) ^ sw_off);
  const uint32_t get = ring + lg * 64 + lt * 4;
  auto fetch = [&](int g, int stage) {
    // K is a multiple of 64: the last group may have only two of its four 16-byte units
    const int64_t at = static_cast<int64_t>(g) * 64;
    const bool inside = g < g1 && at + lt * 16 < row_bytes;
    const bool a = inside && in0, b = inside && in1;
    const uint32_t dst = put + stage * (kWarps * 1024);
    cp_async16_zfill(dst, a ? src0 + at : p.w4, a ? 16u : 0u);
    cp_async16_zfill(dst + 512, b ? src0 + 8 * row_bytes + at : p.w4, b ? 16u : 0u);
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(g0 + s * S::kKWarps, s);
  if (p.early) grid_dep_wait();
  grid_dep_launch();

  auto load = [&](int g, W4Operands<kTiles, kFp8>& o) {
    if (g >= g1) return;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int t = t0 + 8 * i + lg;
      const Vec* row = reinterpret_cast<const Vec*>(static_cast<const uint8_t*>(p.x) +
                                                    (static_cast<int64_t>(t) * p.K + g * kW4Group) * (kFp8 ? 1 : 2));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o.x[i][j] = t < p.T && g * kW4Group + 8 * (4 * j + lt) < p.K ? row[4 * j + lt] : Vec{};
      if (kFp8) {
        const int c = t0 + 8 * i + 2 * lt;
        o.sx[i][0] = c < p.T ? p.sx[static_cast<int64_t>(c) * p.groups + g] : 0.f;
        o.sx[i][1] = c + 1 < p.T ? p.sx[static_cast<int64_t>(c + 1) * p.groups + g] : 0.f;
      }
    }
    o.sw[0] = in0 ? bf16_bits_to_f32(p.sw[static_cast<int64_t>(r0) * p.groups + g]) : 0.f;
    o.sw[1] = in1 ? bf16_bits_to_f32(p.sw[static_cast<int64_t>(r0 + 8) * p.groups + g]) : 0.f;
  };

  float acc[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  W4Operands<kTiles, kFp8> next;
  load(g0, next);
  int stage = 0;
  for (int g = g0; g < g1; g += S::kKWarps) {
    const W4Operands<kTiles, kFp8> o = next;
    load(g + S::kKWarps, next);
    cp_async_wait_group<kStages - 2>();
    __syncwarp();  // the group has landed for every lane, and every lane has read the one before
    fetch(g + (kStages - 1) * S::kKWarps, stage == 0 ? kStages - 1 : stage - 1);
    const uint32_t at = get + stage * (kWarps * 1024);
    stage = stage + 1 == kStages ? 0 : stage + 1;

    float sum[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) sum[i][0] = sum[i][1] = sum[i][2] = sum[i][3] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t unit = (j << 4) ^ sw_off;
      const uint32_t va = ld_shared_u32(at + unit), vb = ld_shared_u32(at + 512 + unit);
      uint32_t a[4], b[4];
      if (kFp8) {
        w4_pairs_f16(va, a);
        w4_pairs_f16(vb, b);
      } else {
        w4_pairs(va, a);
        w4_pairs(vb, b);
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        uint32_t x[4];
        pair_order(o.x[i][j], x);
        mma_16816<kFp8>(sum[i], a[0], b[0], a[1], b[1], x[0], x[1]);
        mma_16816<kFp8>(sum[i], a[2], b[2], a[3], b[3], x[2], x[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = kFp8 ? sum[i][e] * o.sx[i][e & 1] : sum[i][e];
        acc[i][e] = fmaf(v, o.sw[e >> 1], acc[i][e]);
      }
  }
  cp_async_wait_all();
  __syncthreads();  // the ring is done with: the partials take its place

  // partial [K warp][token][row]
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = i * 8 + lt * 2 + (e & 1), r = rw * 16 + lg + (e >> 1) * 8;
      part[(kw * S::kTok + t) * S::kLd + r] = acc[i][e];
    }
  if (p.split > 1) cluster_sync();
  else __syncthreads();

  // the cluster's threads share the (token, row) sums, row fastest, each in rank and warp order
  const int toks = min(S::kTok, p.T - t0);
  const uint32_t base = smem_u32(part);
  for (int e = rank * kThreads + tid; e < toks * S::kRows; e += p.split * kThreads) {
    const int r = e % S::kRows, t = e / S::kRows;
    if (n0 + r >= p.N) continue;
    float v = 0.f;
    for (int q = 0; q < p.split; ++q) {
      const uint32_t at = p.split > 1 ? mapa(base, q) : base;
#pragma unroll
      for (int k = 0; k < S::kKWarps; ++k) v += ld_cluster_f32(at + ((k * S::kTok + t) * S::kLd + r) * 4);
    }
    p.y[static_cast<int64_t>(t0 + t) * p.N + n0 + r] = f32_to_bf16_bits(v);
  }
  if (p.split > 1) cluster_sync();  // peers may still be reading this CTA's partial
}

template <int kRowWarps, int kTiles, bool kFp8>
cudaError_t launch_shape(W4Params p, cudaStream_t stream) {
  using S = W4Shape<kRowWarps, kTiles>;
  static bool configured[kMaxDevicesLocal] = {};  // the attribute is per device
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  auto kernel = linear_w4_kernel<kRowWarps, kTiles, kFp8>;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const int tiles = (p.N + S::kRows - 1) / S::kRows;
  p.split = 1;
  while (p.split < kMaxSplit && tiles * p.split < 304 && p.groups >= 2 * p.split * S::kKWarps) p.split *= 2;
  if (getenv("W4_SPLIT")) p.split = atoi(getenv("W4_SPLIT"));
  p.early = launch_overlap() >= 2;
  p.per = (p.groups + p.split - 1) / p.split;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * p.split, 1, (p.T + S::kTok - 1) / S::kTok);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_overlap() > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool kFp8, int kTiles>
cudaError_t launch_rw(const W4Params& p, cudaStream_t stream) {
  const int rw = getenv("W4_RW") ? atoi(getenv("W4_RW")) : 4;
  if (rw == 1) return launch_shape<1, kTiles, kFp8>(p, stream);
  if (rw == 2) return launch_shape<2, kTiles, kFp8>(p, stream);
  if (rw == 4) return launch_shape<4, kTiles, kFp8>(p, stream);
  return launch_shape<8, kTiles, kFp8>(p, stream);
}

template <bool kFp8>
cudaError_t launch_any(const W4Params& p, cudaStream_t stream) {
  if (p.T <= 8) return launch_rw<kFp8, 1>(p, stream);
  if (p.T <= 16) return launch_rw<kFp8, 2>(p, stream);
  return launch_rw<kFp8, 4>(p, stream);
}

}  // namespace

cudaError_t launch_linear_w4(const void* x, const float* x_scale, const uint8_t* w4, const uint16_t* w_scale,
                             uint16_t* y, int T, int K, int N, cudaStream_t stream) {
  W4Params p{x, x_scale, w4, w_scale, y, T, K, N, w4_groups(K), 1, 0, false};
  return x_scale != nullptr ? launch_any<true>(p, stream) : launch_any<false>(p, stream);
}

}  // namespace mla
