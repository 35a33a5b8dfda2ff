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
#include <type_traits>

#include "sm100.cuh"
#include "w4.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kTok = 8;        // tokens of a CTA: the columns of one MMA
constexpr int kStages = 4;     // groups a warp has in flight or in use, kM KB each
constexpr int kSms = 152;      // of the GPU this is built for: the rules below count in waves of it

// c (+)= a b; with kFirst, c = a b.
template <bool kF16, bool kFirst>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
#define MLA_MMA_16816(type)                                                                                      \
  if (kFirst)                                                                                                    \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "       \
        "{%8, %9}, {%10, %10, %10, %10};"                                                                        \
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])                                                         \
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));                                       \
  else                                                                                                           \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "       \
        "{%8, %9}, {%0, %1, %2, %3};"                                                                            \
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                         \
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if (kF16) {
    MLA_MMA_16816("f16");
  } else {
    MLA_MMA_16816("bf16");
  }
#undef MLA_MMA_16816
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// kRowWarps warps cover 16 kM rows each, the other kWarps / kRowWarps share their groups of K.
template <int kRowWarps, int kM>
struct W4Shape {
  static constexpr int kThreads = kM == 1 ? 256 : 128;
  static constexpr int kPerSm = kM == 1 ? 3 : 4;  // CTAs of an SM
  static constexpr int kWarps = kThreads / 32;
  static constexpr int kWave = kSms * kPerSm;
  static constexpr int kKWarps = kWarps / kRowWarps;
  static constexpr int kRows = 16 * kM * kRowWarps;
  static constexpr int kLd = kRows + 4;          // floats per token of a partial: conflict-free fragment stores
  static constexpr int kStage = kWarps * kM * 1024;
  static constexpr int kPart = kKWarps * kTok * kLd * 4;  // lies over the ring
  static constexpr int kRing = kStages * kStage > kPart ? kStages * kStage : kPart;
  // K over a cluster while its CTAs still fit the GPU at once and a warp keeps more than one group (7168 -> 576, one
  // token: 3.6 us in four, against 4.8 undivided and 3.7 in eight; in powers of two, because clusters of seven do not
  // all fit: 16384 -> 1024 9.0 us against 6.9 in four)
  static int split(int64_t tiles, int groups) {
    int n = 1;
    while (kRowWarps == 1 && n < kW4MaxSplit && tiles * n * 2 <= kWave && groups >= 3 * kKWarps * n) n *= 2;
    return n;
  }
};

template <int kRowWarps, int kM, bool kFp8, bool kRagged>
__global__ void __launch_bounds__(W4Shape<kRowWarps, kM>::kThreads, W4Shape<kRowWarps, kM>::kPerSm)
linear_w4_kernel(const W4Params p) {
  using S = W4Shape<kRowWarps, kM>;
  using Vec = std::conditional_t<kFp8, uint2, uint4>;  // 8 values of x
  extern __shared__ __align__(16) uint8_t smem[];
  float* part = reinterpret_cast<float*>(smem);
  constexpr int kElem = kFp8 ? 1 : 2;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lg = lane >> 2, lt = lane & 3;
  const int rw = warp % kRowWarps, kw = warp / kRowWarps;
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const bool second = tile >= p.tiles0;
  const W4Out out = second ? p.out[1] : p.out[0];
  const int n0 = (tile - (second ? p.tiles0 : 0)) * S::kRows, rw0 = rw * 16 * kM;
  const int t0 = blockIdx.z * kTok;
  const int g0 = rank * p.per + kw, g1 = min(p.groups, rank * p.per + p.per);
  const int ragged = kRagged ? p.groups - 1 : -1;  // the group with 64 columns, if any
  if (!p.early) grid_dep_wait();

  // Rows past N are read as the last one: their sums are not stored.
  const int64_t row_bytes = p.K >> 1;
  const uint8_t* src[2 * kM];
  int sw_at[2 * kM];
#pragma unroll
  for (int m = 0; m < 2 * kM; ++m) {
    const int r = min(n0 + rw0 + 8 * m + lg, out.N - 1);
    src[m] = out.w4 + r * row_bytes + g0 * 64 + lt * 16;
    sw_at[m] = r * p.groups;
  }
  const uint32_t ring = smem_u32(smem) + warp * (kM * 1024) + lg * 64;
  const uint32_t perm = (lg >> 1 & 3) << 4;  // the row's 16-byte units lie at unit ^ (row / 2 % 4)
  const uint32_t put = ring + ((lt << 4) ^ perm);
  uint32_t get[4];  // word 4 j + t of row g
#pragma unroll
  for (int j = 0; j < 4; ++j) get[j] = ring + ((j << 4) ^ perm) + lt * 4;
  auto fetch = [&](int g, int stage) {
    if (g < g1) {
      // past the 64 columns of a ragged group: its first units again, which meet zeros of x
      const int back = kRagged && g == ragged && lt >= 2 ? 32 : 0;
#pragma unroll
      for (int m = 0; m < 2 * kM; ++m) {
        cp_async16(put + stage * S::kStage + m * 512, src[m] - back);
        src[m] += S::kKWarps * 64;
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(g0 + s * S::kKWarps, s);
  // The weights' scales are two bytes here and there: lane (g, t) loads those of its rows for step t of the next
  // four, four steps ahead, and a shuffle hands them round.
  uint16_t sw[2 * kM], next_sw[2 * kM];
  auto load_sw = [&](int step) {
    const int g = min(g0 + (step + lt) * S::kKWarps, p.groups - 1);
#pragma unroll
    for (int m = 0; m < 2 * kM; ++m) next_sw[m] = out.sw[sw_at[m] + g];
  };
  load_sw(0);
  if (p.early) grid_dep_wait();
  grid_dep_launch();

  // Columns past T repeat the last token: their sums are not stored.
  const uint8_t* x_at =
      static_cast<const uint8_t*>(p.x) + (static_cast<int64_t>(min(t0 + lg, p.T - 1)) * p.K + 8 * lt) * kElem;
  const int sx_at[2] = {min(t0 + 2 * lt, p.T - 1) * p.groups, min(t0 + 2 * lt + 1, p.T - 1) * p.groups};
  Vec next_x[4];
  float next_sx[2] = {1.f, 1.f};
  auto load_x = [&](int g) {
    g = min(g, g1 - 1);  // past the last group: loaded again, not used
#pragma unroll
    for (int j = 0; j < 4; ++j)
      next_x[j] = j < 2 || g != ragged
                      ? *reinterpret_cast<const Vec*>(x_at + static_cast<int64_t>(g) * (kW4Group * kElem) + j * 32 * kElem)
                      : Vec{};
    if (kFp8) {
      next_sx[0] = p.sx[sx_at[0] + g];
      next_sx[1] = p.sx[sx_at[1] + g];
    }
  };

  float acc[kM][4];
#pragma unroll
  for (int i = 0; i < kM; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  if (g0 < g1) load_x(g0);
  static_assert(kStages == 4, "a ring slot is a step within the four of the loop");
  for (int g = g0, step = 0; g < g1; step += 4) {
#pragma unroll
    for (int m = 0; m < 2 * kM; ++m) sw[m] = next_sw[m];
    load_sw(step + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q, g += S::kKWarps) {
      if (g >= g1) break;
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = pair_order(next_x[j]);
      const float sx[2] = {next_sx[0], next_sx[1]};
      load_x(g + S::kKWarps);
      cp_async_wait_group<kStages - 2>();
      __syncwarp();  // the group has landed for every lane, and every lane has read the one before
      fetch(g + (kStages - 1) * S::kKWarps, (q + 3) & 3);
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        float sum[2][4];  // two chains of MMAs
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t at = get[j] + q * S::kStage + i * 1024;
          const uint32_t va = ld_shared_u32(at), vb = ld_shared_u32(at + 512);
          uint32_t a[4], b[4];
          if (kFp8) {
            w4_pairs_f16(va, a);
            w4_pairs_f16(vb, b);
          } else {
            w4_pairs(va, a);
            w4_pairs(vb, b);
          }
          if (j == 0) {
            mma_16816<kFp8, true>(sum[0], a[0], b[0], a[1], b[1], x[j].x, x[j].y);
            mma_16816<kFp8, true>(sum[1], a[2], b[2], a[3], b[3], x[j].z, x[j].w);
          } else {
            mma_16816<kFp8, false>(sum[0], a[0], b[0], a[1], b[1], x[j].x, x[j].y);
            mma_16816<kFp8, false>(sum[1], a[2], b[2], a[3], b[3], x[j].z, x[j].w);
          }
        }
        const float s[2] = {
            bf16_bits_to_f32(__shfl_sync(0xffffffffu, static_cast<int>(sw[2 * i]), (lane & 28) | q)),
            bf16_bits_to_f32(__shfl_sync(0xffffffffu, static_cast<int>(sw[2 * i + 1]), (lane & 28) | q))};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = sum[0][e] + sum[1][e];
          if (kFp8) v *= sx[e & 1];
          acc[i][e] = fmaf(v, s[e >> 1], acc[i][e]);
        }
      }
    }
  }
  cp_async_wait_all();
  __syncthreads();  // the ring is done with: the partials take its place

  // partial [K warp][token][row]
#pragma unroll
  for (int i = 0; i < kM; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = lt * 2 + (e & 1), r = rw0 + i * 16 + lg + (e >> 1) * 8;
      part[(kw * kTok + t) * S::kLd + r] = acc[i][e];
    }
  if (S::kKWarps > 1 || p.split == 1) __syncthreads();
  else cluster_sync();

  const int toks = min(kTok, p.T - t0);
  if (S::kKWarps > 1) {
    // this CTA's K warps in order, into the first one's place
    for (int e = tid; e < toks * S::kRows; e += S::kThreads) {
      float* at = part + (e / S::kRows) * S::kLd + e % S::kRows;
      float v = at[0];
#pragma unroll
      for (int k = 1; k < S::kKWarps; ++k) v += at[k * kTok * S::kLd];
      at[0] = v;
    }
    if (p.split > 1) cluster_sync();
    else __syncthreads();
  }

  // the cluster's threads share the (token, row) sums, row fastest, each in rank order
  const uint32_t base = smem_u32(part);
  for (int e = rank * S::kThreads + tid; e < toks * S::kRows; e += p.split * S::kThreads) {
    const int r = e % S::kRows, t = e / S::kRows;
    if (n0 + r >= out.N) continue;
    const float v = sum_partials(base + (t * S::kLd + r) * 4, p.split);
    out.y[static_cast<int64_t>(t0 + t) * out.N + n0 + r] = f32_to_bf16_bits(v);
  }
  if (p.split > 1) cluster_sync();  // peers may still be reading this CTA's partial
}

template <int kRowWarps, int kM, bool kFp8, bool kRagged>
cudaError_t launch_shape(W4Params p, cudaStream_t stream) {
  using S = W4Shape<kRowWarps, kM>;
  static bool configured[kMaxDevicesLocal] = {};  // the attribute is per device
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  auto kernel = linear_w4_kernel<kRowWarps, kM, kFp8, kRagged>;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kRing);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const int64_t tiles = p.tiles(S::kRows);
  const int slices = (p.T + kTok - 1) / kTok;
  p.tiles0 = (p.out[0].N + S::kRows - 1) / S::kRows;
  p.split = S::split(tiles * slices, p.groups);
  p.per = (p.groups + p.split - 1) / p.split;
  p.early = launch_overlap() >= 2;
  return launch_w4(kernel, dim3(static_cast<unsigned>(tiles) * p.split, 1, slices), S::kThreads, S::kRing, stream, p.split, p);
}

template <int kRowWarps, int kM>
cudaError_t launch_rows(const W4Params& p, cudaStream_t stream) {
  const bool ragged = p.K % kW4Group != 0;
  if (p.sx != nullptr)
    return ragged ? launch_shape<kRowWarps, kM, true, true>(p, stream) : launch_shape<kRowWarps, kM, true, false>(p, stream);
  return ragged ? launch_shape<kRowWarps, kM, false, true>(p, stream) : launch_shape<kRowWarps, kM, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_linear_w4(W4Params p, cudaStream_t stream) {
  const int slices = (p.T + kTok - 1) / kTok;
  const int64_t tiles = p.tiles(16) * slices;
  // Warp MMAs pass over the weights once for 8 tokens, the tensor-core kernel once for 16 to 128 but with a longer way
  // from weight to result: it wins from two passes on once they are over about 36 M weights (us, tensor cores against
  // warps: 1536 -> 16384, 16 tokens 9.0 against 11.3; 16384 -> 7168, 16 tokens 24 against 28, 64 tokens 28 against 96;
  // 7168 -> 1536, 32 tokens 8.8 against 8.9, 16 tokens 8.3 against 7.1; 512 -> 512, 256 tokens 5.2 against 3.3).
  if (slices > 1 && (static_cast<int64_t>(p.out[0].N) + p.out[1].N) * p.K * slices > 36000000) return launch_linear_w4_tc(p, stream);
  // Up to one wave of CTAs, 16 rows each and K over all eight warps: the latency of few, short streams counts; or 32 rows
  // and four warps where those, divided, fill their wave better (7168 -> 2048, one token: 512 of 608 CTAs 5.4 us, 256 of
  // 456 6.5).  Beyond, 32 rows a warp share what it unpacks of x (1536 -> 16384, one token: 6.0 us against 7.4), in CTAs
  // of four warps rather than eight (6.4), and fewer warps share K where it is short.
  using A = W4Shape<1, 1>;
  using B = W4Shape<1, 2>;
  const int64_t tiles2 = p.tiles(32) * slices;
  if (tiles <= A::kWave) {
    const int64_t a = tiles * A::split(tiles, p.groups), b = tiles2 * B::split(tiles2, p.groups);
    return b * A::kWave > a * B::kWave ? launch_rows<1, 2>(p, stream) : launch_rows<1, 1>(p, stream);
  }
  if (p.groups >= 48) return launch_rows<1, 2>(p, stream);
  if (p.groups >= 4) return launch_rows<2, 2>(p, stream);
  return launch_rows<4, 2>(p, stream);
}

}  // namespace mla
