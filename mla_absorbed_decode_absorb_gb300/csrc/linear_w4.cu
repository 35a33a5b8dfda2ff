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
// side.  A thread's share of one group of a 16-row tile is 16 bytes of row g and
// 16 of row g + 8 (g = lane / 4), 32 consecutive columns each, fetched by its own
// cp.async ring: no thread reads another's bytes, so the stream needs no
// barrier.  The K order inside an MMA is free as long as both operands agree:
// word j of those 16 bytes holds columns 32 (lane % 4) + 8 j + 0..7, whose half
// bytes i and i + 4 come out as one pair, and x is staged in shared memory in
// that pair order, 16 bytes per (token, 8 columns).
//
// K is split over the CTAs of a cluster; each keeps its partial in shared
// memory and the cluster adds them in rank order through distributed shared
// memory, so a call needs no workspace and its result does not depend on timing.
#include <cuda_fp16.h>

#include "sm100.cuh"
#include "w4.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 8;         // ring depth per thread, 32 bytes a stage
constexpr int kChunkGroups = 8;    // groups of x staged at a time
constexpr int kMaxSplit = 8;       // CTAs of a cluster along K (the portable size)

struct W4Params {
  const void* x;        // bf16 [T, K] or E4M3 [T, K]
  const float* sx;      // [T, groups] (E4M3 x)
  const uint8_t* w4;    // [N, K / 2]
  const uint16_t* sw;   // [N, groups] bf16
  uint16_t* y;          // [T, N] bf16
  int T, K, N, groups;
  int split, per;       // CTAs along K, groups per CTA
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
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

// Two E4M3 codes as a bf16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x, f.y);
}

// Eight bf16 values (four natural pairs) to the pair order (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ uint4 to_pair_order(uint4 v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                    __byte_perm(v.y, v.w, 0x7632));
}

// kRowWarps warps cover 16 rows each, the other kWarps / kRowWarps share their
// groups of K; kTiles tiles of 8 tokens.
template <int kRowWarps, int kTiles, bool kFp8>
struct W4Shape {
  static constexpr int kKWarps = kWarps / kRowWarps;
  static constexpr int kRows = 16 * kRowWarps;
  static constexpr int kTok = 8 * kTiles;
  static constexpr int kLd = kRows + 4;  // floats per token of a partial: conflict-free fragment stores
  static constexpr int kRing = kStages * kThreads * 32;
  static constexpr int kX = kChunkGroups * kTok * kW4Group * 2;
  static constexpr int kSx = kFp8 ? kChunkGroups * kTok * 4 : 0;
  static constexpr int kSw = kChunkGroups * kRows * 4;
  static constexpr int kPart = kKWarps * kTok * kLd * 4;
  static constexpr int kSmem = kRing + kX + kSx + kSw + kPart;
};

template <int kRowWarps, int kTiles, bool kFp8>
__global__ void __launch_bounds__(kThreads)
linear_w4_kernel(const W4Params p) {
  using S = W4Shape<kRowWarps, kTiles, kFp8>;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* xs = smem + S::kRing;
  float* sxs = reinterpret_cast<float*>(xs + S::kX);
  float* sws = reinterpret_cast<float*>(xs + S::kX + S::kSx);
  float* part = reinterpret_cast<float*>(xs + S::kX + S::kSx + S::kSw);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rw = warp % kRowWarps, kw = warp / kRowWarps;
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const int n0 = tile * S::kRows;
  const int t0 = blockIdx.z * S::kTok;
  const int g0 = rank * p.per, g1 = min(p.groups, g0 + p.per);
  grid_dep_wait();
  grid_dep_launch();

  // this thread's two rows and its 16 bytes (32 columns) of each group
  const int r0 = n0 + rw * 16 + (lane >> 2);
  const int64_t row_bytes = p.K >> 1;
  const uint8_t* src0 = p.w4 + static_cast<int64_t>(r0) * row_bytes + (lane & 3) * 16;
  const uint8_t* src1 = src0 + 8 * row_bytes;
  const bool in0 = r0 < p.N, in1 = r0 + 8 < p.N;
  const uint32_t ring = smem_u32(smem) + tid * 16;
  // K is a multiple of 64: in the last group the upper two lanes may lie past the row
  auto fetch = [&](int g, int stage) {
    const bool inside = g < g1 && static_cast<int64_t>(g) * 64 + (lane & 3) * 16 < row_bytes;
    const uint32_t dst = ring + stage * (kThreads * 32);
    const int64_t at = static_cast<int64_t>(g) * 64;
    const bool a = inside && in0, b = inside && in1;
    cp_async16_zfill(dst, a ? src0 + at : p.w4, a ? 16u : 0u);
    cp_async16_zfill(dst + kThreads * 16, b ? src1 + at : p.w4, b ? 16u : 0u);
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(g0 + kw + s * S::kKWarps, s);

  float acc[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

  int step = 0;  // this warp's groups so far
  for (int gc = g0; gc < g1; gc += kChunkGroups) {
    const int ng = min(kChunkGroups, g1 - gc);
    __syncthreads();  // the previous chunk has been read
    // x of these groups: one 16-byte unit per (token, 8 columns), zeros past T and K
    for (int u = tid; u < S::kTok * ng * 16; u += kThreads) {
      const int c = u % (ng * 16), t = u / (ng * 16);  // chunk of 8 columns, token
      const int col = gc * kW4Group + c * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (t0 + t < p.T && col < p.K) {
        const int64_t at = static_cast<int64_t>(t0 + t) * p.K + col;
        if (kFp8) {
          const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.x) + at);
          v = make_uint4(e4m3x2_to_bf16x2(q.x), e4m3x2_to_bf16x2(q.x >> 16), e4m3x2_to_bf16x2(q.y),
                         e4m3x2_to_bf16x2(q.y >> 16));
        } else {
          v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + at);
        }
      }
      const int slot = (((c >> 4) * kTiles + (t >> 3)) * 4 + (c & 3)) * 32 + (t & 7) * 4 + ((c & 15) >> 2);
      *reinterpret_cast<uint4*>(xs + slot * 16) = to_pair_order(v);
    }
    if (kFp8)
      for (int u = tid; u < S::kTok * ng; u += kThreads) {
        const int g = u % ng, t = u / ng;
        sxs[g * S::kTok + t] = t0 + t < p.T ? p.sx[static_cast<int64_t>(t0 + t) * p.groups + gc + g] : 0.f;
      }
    for (int u = tid; u < S::kRows * ng; u += kThreads) {
      const int g = u % ng, r = u / ng;
      sws[g * S::kRows + r] =
          n0 + r < p.N ? bf16_bits_to_f32(p.sw[static_cast<int64_t>(n0 + r) * p.groups + gc + g]) : 0.f;
    }
    __syncthreads();

    for (int g = g0 + kw + step * S::kKWarps; g < gc + ng; g += S::kKWarps, ++step) {
      fetch(g + (kStages - 1) * S::kKWarps, (step + kStages - 1) % kStages);
      cp_async_wait_group<kStages - 1>();
      const uint8_t* st = smem + (step % kStages) * (kThreads * 32) + tid * 16;
      const uint4 wa = *reinterpret_cast<const uint4*>(st);
      const uint4 wb = *reinterpret_cast<const uint4*>(st + kThreads * 16);
      const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
      float part_g[kTiles][4];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) part_g[i][0] = part_g[i][1] = part_g[i][2] = part_g[i][3] = 0.f;
      const int gl = g - gc;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t pa[4], pb[4];
        w4_pairs(a[j], pa);
        w4_pairs(b[j], pb);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const uint4 xv = *reinterpret_cast<const uint4*>(xs + (((gl * kTiles + i) * 4 + j) * 32 + lane) * 16);
          mma_bf16(part_g[i], pa[0], pb[0], pa[1], pb[1], xv.x, xv.y);
          mma_bf16(part_g[i], pa[2], pb[2], pa[3], pb[3], xv.z, xv.w);
        }
      }
      const float s0 = sws[gl * S::kRows + rw * 16 + (lane >> 2)];
      const float s1 = sws[gl * S::kRows + rw * 16 + (lane >> 2) + 8];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        if (kFp8) {
          const float2 q = *reinterpret_cast<const float2*>(sxs + gl * S::kTok + i * 8 + (lane & 3) * 2);
          acc[i][0] = fmaf(part_g[i][0] * q.x, s0, acc[i][0]);
          acc[i][1] = fmaf(part_g[i][1] * q.y, s0, acc[i][1]);
          acc[i][2] = fmaf(part_g[i][2] * q.x, s1, acc[i][2]);
          acc[i][3] = fmaf(part_g[i][3] * q.y, s1, acc[i][3]);
        } else {
          acc[i][0] = fmaf(part_g[i][0], s0, acc[i][0]);
          acc[i][1] = fmaf(part_g[i][1], s0, acc[i][1]);
          acc[i][2] = fmaf(part_g[i][2], s1, acc[i][2]);
          acc[i][3] = fmaf(part_g[i][3], s1, acc[i][3]);
        }
      }
    }
  }
  cp_async_wait_all();

  // partial [K warp][token][row]
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = i * 8 + (lane & 3) * 2 + (e & 1), r = rw * 16 + (lane >> 2) + (e >> 1) * 8;
      part[(kw * S::kTok + t) * S::kLd + r] = acc[i][e];
    }
  if (p.split > 1) cluster_sync();
  else __syncthreads();

  // rank q of the cluster adds and stores every split-th block of 16 rows' share:
  // element e of (token, row) with row fastest, in rank order
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
  using S = W4Shape<kRowWarps, kTiles, kFp8>;
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

template <bool kFp8>
cudaError_t launch_any(const W4Params& p, cudaStream_t stream) {
  if (p.T <= 8) return launch_shape<4, 1, kFp8>(p, stream);
  if (p.T <= 16) return launch_shape<4, 2, kFp8>(p, stream);
  return launch_shape<4, 4, kFp8>(p, stream);
}

}  // namespace

cudaError_t launch_linear_w4(const void* x, const float* x_scale, const uint8_t* w4, const uint16_t* w_scale,
                             uint16_t* y, int T, int K, int N, cudaStream_t stream) {
  W4Params p{x, x_scale, w4, w_scale, y, T, K, N, w4_groups(K), 1, 0};
  return x_scale != nullptr ? launch_any<true>(p, stream) : launch_any<false>(p, stream);
}

}  // namespace mla
