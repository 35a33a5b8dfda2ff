// The 4-bit-weight projection of csrc/linear_w4.cu for more than a few tokens, on
// the 5th-generation tensor cores:
//
//   y[t, n] = sum_g sw[n, g] sx[t, g] sum_{k in g} (u[n, k] - 8) x[t, k]
//
// One CTA owns 128 output features (the M side) and a range of K, up to kTn tokens
// (the N side), and takes a group of 128 columns at a time.  Producer warps unpack
// the weights: thread r turns the 64 bytes of weight row r into 128 exact bf16
// values of TMEM lane r, or for 8-bit x into 128 E4M3 codes of (u - 8) 2^-9, exact too;
// x comes by TMA into 128-byte-swizzled shared memory as it is.  A thread issues the
// group's MMAs (8 of K = 16, or 4 of K = 32 on E4M3) into one of two TMEM accumulators,
// and the epilogue warps read it back and add it, scaled in fp32, to their
// registers: the accumulator holds one group's exact products only, so no scale is
// ever rounded into a weight.
//
// Up to 64 tokens two such CTAs share an SM (256 TMEM columns each), beyond one with
// twice the warps.  K is split over a cluster, whose partials meet in distributed
// shared memory in rank order.
#include "sm100.cuh"
#include "tmap.cuh"
#include "w4.cuh"

#include <type_traits>

namespace mla {
namespace {

using namespace sm100;

constexpr int kRows = 128;
constexpr int kSlot = kRows * 64;              // a group of weights
constexpr int kMaxCtas = 304;                  // two on each of 152 SMs: more never run at once
constexpr int kSxStages = 8;                   // groups of x's scales: the producers are at most six groups ahead of the sums

__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&d)[16]) { tmem_ld16(at, d); }
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&d)[8]) { tmem_ld8(at, d); }

struct Bars {
  uint64_t weights[8];  // a group of weights has landed (TMA)
  uint64_t x[4];        // a group of x has landed (TMA)
  uint64_t ready[4];    // a group's weights (and x's scales) are in place (one arrival per producer warp)
  uint64_t free[4];     // ... and have been consumed, and its x (commit)
  uint64_t full[2];     // a group's accumulator is complete (commit)
  uint64_t drained[2];  // ... and has been read (one arrival per epilogue warp)
  uint32_t tmem;
  int abort;
};

template <int kTn, bool kFp8>
struct TcShape {
  static constexpr int kPerSm = kTn <= 64 ? 2 : 1;             // CTAs of an SM
  static constexpr int kSets = kTn <= 64 ? 1 : 2;              // of four producer warps
  static constexpr int kEpilogue = 4 * kSets;                  // first epilogue warp
  static constexpr int kEpTok = kTn <= 64 ? kTn : 64;          // tokens of an epilogue thread's registers
  static constexpr int kEpWarps = 4 * (kTn / kEpTok);
  // Packed fp32 sums where the registers allow pairs (256 tokens, 16384 -> 7168: 80 us against 84; 32 tokens 25.0 against
  // 26.2); 64 sums and x's scales in pairs spill (256 tokens in 8 bits: 140 us against 95).
  static constexpr bool kPacked = kEpTok < 64 || (kTn == 128 && !kFp8);
  static constexpr int kIssuer = kEpilogue + kEpWarps;         // first of the two warps that issue MMAs
  static constexpr int kACols = kFp8 ? 32 : 64;                // TMEM columns of a group's weights
  static constexpr int kABufs = kFp8 || kTn > 64 ? 4 : 2;      // ... in place or in use, in front of two accumulators
  static constexpr uint32_t kTmemD = kABufs * kACols;
  static constexpr int kDCols = kTn <= 64 ? 64 : 128;          // TMEM columns of an accumulator
  static constexpr uint32_t kTmemCols = kTn <= 64 ? 256 : 512;
  static constexpr bool kLoader = kTn > 64;                    // x is fetched by a warp of its own
  static constexpr int kThreads = 32 * (kIssuer + 2 + (kLoader ? 1 : 0));
  static constexpr int kStages = kTn <= 64 || !kFp8 ? 4 : 8;   // groups of weights in flight or in use
  static constexpr int kRing = kStages * kSlot;
  static constexpr int kBox = kTn * 128;                       // kTn tokens x 64 columns (bf16) or 128 (E4M3)
  static constexpr int kB = kFp8 ? kBox : 2 * kBox;            // a group of x
  static constexpr int kXStages = 4;                           // groups of x in flight or in use
  static constexpr int kLd = kRows + 4;                        // floats per token of a partial
  static constexpr int kPart = kTn * kLd * 4;                  // the CTA's partial, over the operands
  static constexpr int kBody = kXStages * kB + kRing > kPart ? kXStages * kB + kRing : kPart;
  static constexpr int kSx = kFp8 ? kSxStages * kTn * 4 : 0;   // scales of x
  static constexpr int kSmem = kBody + kSx + 256 + 1024;
  static_assert(sizeof(Bars) <= 256, "barrier block");
};

template <int kTn, bool kFp8>
__global__ void __launch_bounds__(TcShape<kTn, kFp8>::kThreads, TcShape<kTn, kFp8>::kPerSm)
linear_w4_tc_kernel(const __grid_constant__ CUtensorMap tm_w0, const __grid_constant__ CUtensorMap tm_w1,
                    const __grid_constant__ CUtensorMap tm_x, const W4Params p) {
  using S = TcShape<kTn, kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + S::kXStages * S::kB;
  float* sxs = reinterpret_cast<float*>(smem + S::kBody);  // [kSxStages][kTn]
  Bars& bars = *reinterpret_cast<Bars*>(smem + S::kBody + S::kSx);
  float* part = reinterpret_cast<float*>(smem);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const bool second = tile >= p.tiles0;
  const W4Out out = second ? p.out[1] : p.out[0];
  const CUtensorMap* tm_w = second ? &tm_w1 : &tm_w0;
  const int n0 = (tile - (second ? p.tiles0 : 0)) * kRows, t0 = blockIdx.z * kTn;
  const int g0 = rank * p.per, ng = max(0, min(p.groups, g0 + p.per) - g0);
  volatile int* abort = &bars.abort;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(smem_u32(&bars.weights[i]), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bars.x[i]), 1);
      mbar_init(smem_u32(&bars.ready[i]), 4);
      mbar_init(smem_u32(&bars.free[i]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars.full[b]), 1);
      mbar_init(smem_u32(&bars.drained[b]), S::kEpWarps);
    }
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == S::kIssuer) {
    tmem_alloc(smem_u32(&bars.tmem), S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  if (!p.early || warp < S::kIssuer) grid_dep_wait();  // the issuers fetch weights
  grid_dep_launch();

  // A group of x: its place is free again once its MMAs have completed.
  auto fetch_x = [&](int i) {
    if (i >= ng) return;
    const uint32_t bar = smem_u32(&bars.x[i & 3]), at = smem_u32(smem + (i & 3) * S::kB);
    mbar_arrive_expect_tx(bar, S::kB);
    tma_load_2d(at, &tm_x, (g0 + i) * kW4Group, t0, bar);
    if (!kFp8) tma_load_2d(at + S::kBox, &tm_x, (g0 + i) * kW4Group + 64, t0, bar);
  };
  // The group has left its operands: its MMAs have completed.
  auto wait_free = [&](int i, volatile int* give_up) {
    return mbar_wait(smem_u32(&bars.free[i & 3]), (i >> 2) & 1, p.status, give_up);
  };

  if (warp < S::kEpilogue) {
    // -------------------------------------------------------------- producers
    // Rows past N and columns past K are zeros, tokens past T read as the last one (not stored).
    const int r = tid & 127, set = tid >> 7;  // a set takes every kSets-th group
    const uint8_t* wrow = ring + r * 64;
    const int perm = r >> 1 & 3;  // 64-byte swizzle: 16-byte unit q of row r lies at q ^ (r / 2 % 4)
    float sx = 0.f;  // the scale of token r's next group
    auto load_sx = [&](int i) {
      if (i < ng && r < kTn) sx = p.sx[static_cast<int64_t>(min(t0 + r, p.T - 1)) * p.groups + g0 + i];
    };
    if (kFp8) load_sx(set);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    for (int i = set; i < ng; i += S::kSets) {
      const int b = i & (S::kABufs - 1);
      ok = mbar_wait(smem_u32(&bars.weights[i % S::kStages]), (i / S::kStages) & 1, p.status, abort);
      uint32_t w[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(wrow + (i % S::kStages) * kSlot + ((q ^ perm) << 4));
        w[4 * q] = v.x;
        w[4 * q + 1] = v.y;
        w[4 * q + 2] = v.z;
        w[4 * q + 3] = v.w;
      }
      // The first kAhead parts are unpacked before the operand is free, beside the MMAs that hold it (256 tokens,
      // 16384 -> 7168: 86 us, against 99 with none, before the sums were packed; up to 64 tokens the other CTA of the SM fills that time, and the
      // registers it takes cost more).
      constexpr int kQuarters = kFp8 ? 2 : 4;  // of 16 TMEM columns
      uint32_t a[kQuarters][16];
      auto unpack = [&](int h) {
#pragma unroll
        for (int q = 0; q < 16 / kQuarters; ++q) {
          if (kFp8) {
            uint32_t c[2];
            w4_e4m3(w[8 * h + q], c);
            a[h][2 * q] = c[0];
            a[h][2 * q + 1] = c[1];
          } else {
            uint32_t c[4];
            w4_pairs_natural(w[4 * h + q], c);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[h][4 * q + e] = c[e];
          }
        }
      };
      constexpr int kAhead = kTn < 128 ? 0 : kQuarters;
#pragma unroll
      for (int h = 0; h < kAhead; ++h) unpack(h);
      if (i >= S::kABufs) ok = ok && wait_free(i - S::kABufs, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (kFp8) {
        if (r < kTn) sxs[i % kSxStages * kTn + r] = sx;
        load_sx(i + S::kSets);
      }
#pragma unroll
      for (int h = 0; h < kQuarters; ++h) {
        if (h >= kAhead) unpack(h);
        tmem_st16(tmem + lane_off + S::kACols * b + 16 * h, a[h]);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.ready[i & 3]));
    }
  } else if (S::kLoader && warp == S::kIssuer + 2) {
    // -------------------------------------------------------------- x
    if (lane == 0) {
      if (p.early) grid_dep_wait();
      int i = 0;
      for (; i < ng; ++i) {
        if (i >= 4 && !wait_free(i - 4, abort)) break;
        fetch_x(i);
      }
      // given up: wait for the copies that may still be in flight
      for (int j = max(0, i - 4); i < ng && j < i; ++j)
        mbar_wait(smem_u32(&bars.x[j & 3]), (j >> 2) & 1, p.status);
    }
    __syncwarp();
  } else if (warp >= S::kIssuer) {
    // -------------------------------------------------------------- MMA issuers
    // An MMA this narrow holds its issuing thread far longer than the tensor pipe (113 cycles for N <= 128), so
    // two warps issue: one the groups of each buffer, which share nothing.
    if (lane == 0) {
      const int b = warp - S::kIssuer;
      // the weights of this buffer's groups: a slot is free again once the producers are ready with it
      auto fetch = [&](int i) {
        if (i >= ng) return;
        const uint32_t bar = smem_u32(&bars.weights[i % S::kStages]);
        mbar_arrive_expect_tx(bar, kSlot);
        tma_load_2d(smem_u32(ring + (i % S::kStages) * kSlot), tm_w, (g0 + i) * 64, n0, bar);
      };
      int i = b;
      for (; i < S::kStages; i += 2) fetch(i);
      if (!S::kLoader) {
        if (p.early) grid_dep_wait();
        fetch_x(b);
        fetch_x(b + 2);
      }
      const uint32_t idesc = kFp8 ? idesc_f16(128, kTn, 0, 0) : idesc_bf16(128, kTn, 0, 0);
      int issued = -1;                                      // the last group whose MMAs are issued
      int w_from = b, w_to = i, x_from = b, x_to = b + 4;  // groups whose copies may be in flight
      for (i = b; i < ng; i += 2) {
        if (!S::kLoader && i >= 2) {
          if (!wait_free(i - 2, abort)) break;
          fetch_x(x_to);
          x_to += 2;
        }
        if (!mbar_wait(smem_u32(&bars.ready[i & 3]), (i >> 2) & 1, p.status, abort)) break;
        w_from = i + 2;
        fetch(w_to);
        w_to += 2;
        if (!mbar_wait(smem_u32(&bars.x[i & 3]), (i >> 2) & 1, p.status, abort)) break;
        x_from = i + 2;
        if (i >= 2 && !mbar_wait(smem_u32(&bars.drained[b]), ((i >> 1) & 1) ^ 1, p.status, abort)) break;
        tc_fence_after();
        const uint32_t b0 = smem_u32(smem + (i & 3) * S::kB);
        const uint32_t d = tmem + S::kTmemD + S::kDCols * b, a0 = tmem + S::kACols * (i & (S::kABufs - 1));
#pragma unroll
        for (int q = 0; q < (kFp8 ? 4 : 8); ++q) {
          const uint64_t bd = smem_desc(b0 + (q >> 2) * S::kBox + (q & 3) * 32, 16, 1024, kSw128);
          if (kFp8) mma_ts_f8(d, a0 + 8 * q, bd, idesc, q ? 1u : 0u);
          else mma_ts(d, a0 + 8 * q, bd, idesc, q ? 1u : 0u);
        }
        mma_commit(smem_u32(&bars.free[i & 3]));
        mma_commit(smem_u32(&bars.full[b]));
        issued = i;
      }
      if (i < ng) {
        // given up: wait for the MMAs and the copies that may still be in flight
        if (issued >= 0) wait_free(issued, nullptr);
        for (int j = w_from; j < min(ng, w_to); j += 2)
          mbar_wait(smem_u32(&bars.weights[j % S::kStages]), (j / S::kStages) & 1, p.status);
        for (int j = x_from; !S::kLoader && j < min(ng, x_to); j += 2)
          mbar_wait(smem_u32(&bars.x[j & 3]), (j >> 2) & 1, p.status);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- epilogue
    // TMEM lane = row n0 + 32 (warp % 4) + lane, column = token; a second four warps take the upper 64 tokens
    const int r = (warp & 3) * 32 + lane, c0 = (warp - S::kEpilogue) / 4 * S::kEpTok;
    float acc[S::kEpTok];
#pragma unroll
    for (int t = 0; t < S::kEpTok; ++t) acc[t] = 0.f;
    constexpr int kLoad = kTn < 64 ? 16 : 8;  // columns at a time: 64 sums leave few registers
    const uint16_t* sw = out.sw + static_cast<int64_t>(min(n0 + r, out.N - 1)) * p.groups + g0;
    uint16_t next[4];  // a thread's scales are two bytes of a row of its own: four groups ahead
#pragma unroll
    for (int q = 0; q < 4; ++q) next[q] = q < ng ? sw[q] : uint16_t(0);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    for (int i0 = 0; i0 < ng && ok; i0 += 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + q, b = q & 1;
        if (i >= ng) break;
        const float s = bf16_bits_to_f32(next[q]) * (kFp8 ? 512.f : 1.f);  // E4M3 weights carry 2^-9
        next[q] = i + 4 < ng ? sw[i + 4] : uint16_t(0);
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.full[b]), (i >> 1) & 1, p.status, abort));
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = tmem + lane_off + S::kTmemD + S::kDCols * b + c0;
        if constexpr (kFp8) {
          float s4[4];  // of the fragment's rows lane / 4 + 8 j
#pragma unroll
          for (int j = 0; j < 4; ++j) s4[j] = __shfl_sync(0xffffffffu, s, lane / 4 + 8 * j);
          const float* sx = sxs + i % kSxStages * kTn + c0 + 2 * (lane & 3);
#pragma unroll
          for (int c = 0; c < S::kEpTok; c += 16) {
            const float2 x[2] = {*reinterpret_cast<const float2*>(sx + c), *reinterpret_cast<const float2*>(sx + c + 8)};
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // the warp's rows 0 .. 15, then 16 .. 31
              uint32_t d[8];
              tmem_ld_frag16(from + c + (static_cast<uint32_t>(16 * half) << 16), d);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float2 xe = x[e >> 2];
                const float w = s4[2 * half + (e >> 1 & 1)];
                float* to = acc + c + 8 * half + e;
                const uint64_t v = mul_f32x2(f32x2(__uint_as_float(d[e]), __uint_as_float(d[e + 1])), f32x2(xe.x, xe.y));
                const float2 sum = f32x2_split(fma_f32x2(v, f32x2(w, w), f32x2(to[0], to[1])));
                to[0] = sum.x;
                to[1] = sum.y;
              }
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < S::kEpTok; c += kLoad) {
            uint32_t d[kLoad];
            tmem_load(from + c, d);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < kLoad; e += 2) {
              float* to = acc + c + e;
              const uint64_t v = f32x2(__uint_as_float(d[e]), __uint_as_float(d[e + 1]));
              if (S::kPacked) {
                const float2 sum = f32x2_split(fma_f32x2(v, f32x2(s, s), f32x2(to[0], to[1])));
                to[0] = sum.x;
                to[1] = sum.y;
              } else {
                to[0] = fmaf(__uint_as_float(d[e]), s, to[0]);
                to[1] = fmaf(__uint_as_float(d[e + 1]), s, to[1]);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.drained[b]));
      }
    }
    // every MMA has completed: the operands and the ring are free for the partial
#pragma unroll
    for (int t = 0; t < S::kEpTok; ++t) {
      if (!kFp8) {
        part[(c0 + t) * S::kLd + r] = acc[t];
      } else {
        const int e = t & 15, token = c0 + (t & ~15) + (e & 4 ? 8 : 0) + 2 * (lane & 3) + (e & 1);
        part[token * S::kLd + (warp & 3) * 32 + (e >> 3) * 16 + (e >> 1 & 1) * 8 + (lane >> 2)] = acc[t];
      }
    }
  }
  // TMEM goes back before any wait for a peer: kernels on two streams, each waiting in a cluster with TMEM that the
  // other's CTAs need to start, would wait for ever
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == S::kIssuer) tmem_dealloc(tmem, S::kTmemCols);
  if (p.split > 1) cluster_sync();

  // the cluster's threads share the (token, row) sums, row fastest, each in rank order
  const int toks = min(kTn, p.T - t0);
  const uint32_t base = smem_u32(part);
  for (int e = rank * S::kThreads + tid; e < toks * kRows; e += p.split * S::kThreads) {
    const int r = e % kRows, t = e / kRows;
    if (n0 + r >= out.N) continue;
    const float v = sum_partials(base + (t * S::kLd + r) * 4, p.split);
    out.y[static_cast<int64_t>(t0 + t) * out.N + n0 + r] = f32_to_bf16_bits(v);
  }
  if (p.split > 1) cluster_sync();  // peers may still be reading this CTA's partial
}

template <int kTn, bool kFp8>
cudaError_t launch_tn(W4Params p, cudaStream_t stream) {
  using S = TcShape<kTn, kFp8>;
  static bool configured[kMaxDevicesLocal] = {};  // the attribute is per device
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  auto kernel = linear_w4_tc_kernel<kTn, kFp8>;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  // K over the largest cluster whose CTAs still fit the GPU at once (a second, partial wave costs more: 256 tokens,
  // 7168 -> 1536 in 24 tiles: 14.0 us in clusters of 5, 24.1 in clusters of 6, which do not all fit) and that leaves a
  // CTA two groups, or seven where CTAs share an SM (32 tokens, 1536 -> 16384: 10.4 us undivided, 11.7 halved)
  const int64_t tiles = p.tiles(kRows), slices = (p.T + kTn - 1) / kTn;
  p.tiles0 = (p.out[0].N + kRows - 1) / kRows;
  static int fit[kMaxDevicesLocal][kW4MaxSplit + 1] = {};  // clusters resident at once, 0: not asked yet
  p.split = 1;
  for (int s = kW4MaxSplit; s > 1; --s) {
    const int64_t ctas = tiles * slices * s;
    if (ctas > kMaxCtas || p.groups < (ctas <= kMaxCtas / 2 ? 2 : 7) * s) continue;
    int n = fit[dev][s];
    if (n == 0) {
      const cudaError_t e = w4_clusters(kernel, S::kThreads, S::kSmem, s, &n);
      if (e != cudaSuccess) return e;
      n *= S::kPerSm;  // the query counts one CTA an SM here, measured are two (56 clusters of 5: one wave)
      fit[dev][s] = n;
    }
    if (tiles * slices <= n) {
      p.split = s;
      break;
    }
  }
  p.per = (p.groups + p.split - 1) / p.split;
  p.early = launch_overlap() >= 2;
  CUtensorMap tm_w[2], tm_x;
  for (int i = 0; i < 2; ++i) {
    const W4Out& o = p.out[i].N > 0 ? p.out[i] : p.out[0];  // (not read without a second projection)
    if (!make_tmap_u8_2d(&tm_w[i], o.w4, o.N, p.K / 2, p.K / 2, 64, kRows, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  const bool ok = kFp8 ? make_tmap_u8_2d(&tm_x, p.x, p.T, p.K, p.K, kW4Group, kTn, CU_TENSOR_MAP_SWIZZLE_128B)
                       : make_tmap_bf16_2d(&tm_x, p.x, p.T, p.K, p.K, 64, kTn, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  return launch_w4(kernel, dim3(static_cast<unsigned>(tiles) * p.split, 1, static_cast<unsigned>(slices)), S::kThreads, S::kSmem, stream, p.split,
                   tm_w[0], tm_w[1], tm_x, p);
}

template <bool kFp8>
cudaError_t launch_any(const W4Params& p, cudaStream_t stream) {
  if (p.T <= 16) return launch_tn<16, kFp8>(p, stream);
  if (p.T <= 48) return launch_tn<48, kFp8>(p, stream);
  if (p.T <= 64) return launch_tn<64, kFp8>(p, stream);
  return launch_tn<128, kFp8>(p, stream);
}

}  // namespace

cudaError_t launch_linear_w4_tc(const W4Params& p, cudaStream_t stream) {
  return p.sx != nullptr ? launch_any<true>(p, stream) : launch_any<false>(p, stream);
}

}  // namespace mla
