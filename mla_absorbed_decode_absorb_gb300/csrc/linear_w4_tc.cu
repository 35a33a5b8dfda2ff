// The 4-bit-weight projection of csrc/linear_w4.cu for more than a few tokens, on
// the 5th-generation tensor cores:
//
//   y[t, n] = sum_g sw[n, g] sx[t, g] sum_{k in g} (u[n, k] - 8) x[t, k]
//
// One CTA owns 128 output features (the M side) and a range of K, up to kTn tokens
// (the N side).  Four producer warps turn a group of 128 columns at a time into
// the MMA's operands: thread r unpacks the 64 bytes of weight row r into 128 exact
// bf16 (f16 for 8-bit x) values of TMEM lane r, and the warps place x, in the same
// pair order (0,4) (1,5) (2,6) (3,7) of each 8 columns, into 128-byte-swizzled
// shared memory.  A thread issues the group's 8 MMAs (K = 16) into one of two TMEM
// accumulators, and four epilogue warps read it back and add it, scaled in fp32,
// to their registers: the accumulator holds one group's exact products only, so no
// scale is ever rounded into a weight.  Operands and accumulators are
// double-buffered; weights arrive by TMA, eight groups deep, x through registers
// one group ahead.
//
// Two such CTAs share an SM (256 TMEM columns each).  K is split over a cluster,
// whose partials meet in distributed shared memory in rank order.
#include "sm100.cuh"
#include "tmap.cuh"
#include "w4.cuh"

#include <type_traits>

namespace mla {
namespace {

using namespace sm100;

constexpr int kRows = 128;
constexpr int kStages = 8;                     // groups of weights in flight or in use
constexpr int kSlot = kRows * 64;              // a group of weights
constexpr int kRing = kStages * kSlot;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kTmemA = 0;                 // two operands of 64 columns, then two accumulators
constexpr uint32_t kTmemD = 128;

__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&d)[16]) { tmem_ld16(at, d); }
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&d)[8]) { tmem_ld8(at, d); }

struct Bars {
  uint64_t weights[kStages];  // a group of weights has landed (TMA)
  uint64_t ready[2];    // both operands of a group are in place (one arrival per producer warp)
  uint64_t free[2];     // ... and have been consumed (commit)
  uint64_t full[2];     // a group's accumulator is complete (commit)
  uint64_t drained[2];  // ... and has been read (one arrival per epilogue warp)
  uint32_t tmem;
  int abort;
};

template <int kTn, bool kFp8>
struct TcShape {
  static constexpr int kPerSm = 2;                             // CTAs of an SM
  static constexpr int kIssuer = 8;                            // warps 0-3 produce, 4-7 add up, 8 and 9 issue MMAs
  static constexpr int kThreads = 32 * (kIssuer + 2);
  static constexpr int kBox = kTn * 128;                       // kTn tokens x 64 columns
  static constexpr int kB = 2 * kBox;                          // a group of x
  static constexpr int kLd = kRows + 4;                        // floats per token of a partial
  static constexpr int kPart = kTn * kLd * 4;                  // the CTA's partial, over the operands
  static constexpr int kBody = 2 * kB + kRing > kPart ? 2 * kB + kRing : kPart;
  static constexpr int kSx = kFp8 ? 4 * kTn * 4 : 0;           // scales of x, four groups
  static constexpr int kSmem = kBody + kSx + 256 + 1024;
  static_assert(sizeof(Bars) <= 256, "barrier block");
};

template <int kTn, bool kFp8, bool kRagged>
__global__ void __launch_bounds__(TcShape<kTn, kFp8>::kThreads, TcShape<kTn, kFp8>::kPerSm)
linear_w4_tc_kernel(const __grid_constant__ CUtensorMap tm_w, const W4Params p) {
  using S = TcShape<kTn, kFp8>;
  using Vec = std::conditional_t<kFp8, uint2, uint4>;  // 8 values of x
  constexpr int kElem = kFp8 ? 1 : 2;
  constexpr int kUnits = kTn / 8;  // of 8 values of x per producer thread and group
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * S::kB;
  float* sxs = reinterpret_cast<float*>(smem + S::kBody);  // [4][kTn]
  Bars& bars = *reinterpret_cast<Bars*>(smem + S::kBody + S::kSx);
  float* part = reinterpret_cast<float*>(smem);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const int n0 = tile * kRows, t0 = blockIdx.z * kTn;
  const int g0 = rank * p.per, ng = max(0, min(p.groups, g0 + p.per) - g0);
  const int ragged = kRagged ? p.groups - 1 - g0 : -1;  // the group with 64 columns, if any
  volatile int* abort = &bars.abort;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&bars.weights[i]), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars.ready[b]), 4);
      mbar_init(smem_u32(&bars.free[b]), 1);
      mbar_init(smem_u32(&bars.full[b]), 1);
      mbar_init(smem_u32(&bars.drained[b]), 4);
    }
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == S::kIssuer) {
    tmem_alloc(smem_u32(&bars.tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  if (!p.early || warp < S::kIssuer) grid_dep_wait();  // the issuers fetch weights
  grid_dep_launch();

  if (warp < 4) {
    // -------------------------------------------------------------- producers
    // Rows past N and columns past K are zeros, tokens past T read as the last one (not stored).
    const uint8_t* wrow = ring + tid * 64;
    const int perm = tid >> 1 & 3;  // 64-byte swizzle: 16-byte unit q of row r lies at q ^ (r / 2 % 4)
    // this thread's units of x: 8 columns of tokens xt, xt + 8, ..
    const int k = tid & 15;
    const uint32_t xt = tid >> 4;
    const uint8_t* xp = static_cast<const uint8_t*>(p.x) +
                        (static_cast<int64_t>(t0) * p.K + static_cast<int64_t>(g0) * kW4Group + k * 8) * kElem;
    const uint32_t xput = (k >> 3) * S::kBox + sw128(xt * 128 + (k & 7) * 16);
    const uint32_t x_ld = static_cast<uint32_t>(p.K) * kElem;  // T K is at most 2^30: 32-bit offsets
    const uint32_t last = p.T - 1 - t0;
    Vec xv[kUnits];
    float sx = 0.f;
    auto load_x = [&](int i) {
      if (i >= ng) return;
      const uint8_t* at = xp + static_cast<int64_t>(i) * (kW4Group * kElem);
#pragma unroll
      for (int q = 0; q < kUnits; ++q)
        xv[q] = kRagged && i == ragged && k >= 8 ? Vec{} : *reinterpret_cast<const Vec*>(at + min(xt + 8 * q, last) * x_ld);
      if (kFp8 && tid < kTn)
        sx = p.sx[static_cast<int64_t>(min(t0 + tid, p.T - 1)) * p.groups + g0 + i];
    };
    load_x(0);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    for (int i = 0; i < ng; ++i) {
      const int b = i & 1;
      ok = mbar_wait(smem_u32(&bars.weights[i % kStages]), (i / kStages) & 1, p.status, abort);
      uint32_t w[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(wrow + (i % kStages) * kSlot + ((q ^ perm) << 4));
        w[4 * q] = v.x;
        w[4 * q + 1] = v.y;
        w[4 * q + 2] = v.z;
        w[4 * q + 3] = v.w;
      }
      if (i >= 2) ok = ok && mbar_wait(smem_u32(&bars.free[b]), ((i >> 1) & 1) ^ 1, p.status, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < kUnits; ++q) *reinterpret_cast<uint4*>(smem + b * S::kB + xput + q * 1024) = pair_order(xv[q]);
      if (kFp8 && tid < kTn) sxs[(i & 3) * kTn + tid] = sx;
      load_x(i + 1);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t a[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pr[4];
          if (kFp8) w4_pairs_f16(w[4 * h + q], pr);
          else w4_pairs(w[4 * h + q], pr);
#pragma unroll
          for (int e = 0; e < 4; ++e) a[4 * q + e] = pr[e];
        }
        tmem_st16(tmem + lane_off + kTmemA + 64 * b + 16 * h, a);
      }
      tmem_wait_st();
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.ready[b]));
    }
  } else if (warp >= S::kIssuer) {
    // -------------------------------------------------------------- MMA issuers
    // An MMA this narrow holds its issuing thread far longer than the tensor pipe (113 cycles for N <= 128), so
    // two warps issue: one the groups of each buffer, which share nothing.
    if (lane == 0) {
      const int b = warp - S::kIssuer;
      // the weights of this buffer's groups: a slot is free again once its operands are ready
      auto fetch = [&](int i) {
        if (i >= ng) return;
        const uint32_t bar = smem_u32(&bars.weights[i % kStages]);
        mbar_arrive_expect_tx(bar, kSlot);
        tma_load_2d(smem_u32(ring + (i % kStages) * kSlot), &tm_w, (g0 + i) * 64, n0, bar);
      };
      int i = b;
      for (; i < kStages; i += 2) fetch(i);
      const uint32_t idesc = kFp8 ? idesc_f16(128, kTn, 0, 0) : idesc_bf16(128, kTn, 0, 0);
      int fetched = i;  // first group of this buffer not fetched yet
      for (i = b; i < ng; i += 2) {
        if (!mbar_wait(smem_u32(&bars.ready[b]), (i >> 1) & 1, p.status, abort)) break;
        fetch(fetched);
        fetched += 2;
        if (i >= 2 && !mbar_wait(smem_u32(&bars.drained[b]), ((i >> 1) & 1) ^ 1, p.status, abort)) break;
        tc_fence_after();
        const uint32_t b0 = smem_u32(smem + b * S::kB);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          mma_ts(tmem + kTmemD + 64 * b, tmem + kTmemA + 64 * b + 8 * q,
                 smem_desc(b0 + (q >> 2) * S::kBox + (q & 3) * 32, 16, 1024, kSw128), idesc, q ? 1u : 0u);
        mma_commit(smem_u32(&bars.free[b]));
        mma_commit(smem_u32(&bars.full[b]));
      }
      if (i < ng) {
        // given up: wait for the MMAs and the copies still in flight
        if (i >= 2) mbar_wait(smem_u32(&bars.free[b]), ((i >> 1) & 1) ^ 1, p.status);
        for (; i < min(ng, fetched); i += 2)
          mbar_wait(smem_u32(&bars.weights[i % kStages]), (i / kStages) & 1, p.status);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- epilogue
    // TMEM lane = row n0 + 32 (warp % 4) + lane, column = token
    const int r = (warp & 3) * 32 + lane;
    float acc[kTn];
#pragma unroll
    for (int t = 0; t < kTn; ++t) acc[t] = 0.f;
    constexpr int kLoad = kTn < 64 ? 16 : 8;  // columns at a time: 64 sums leave few registers
    const uint16_t* sw = p.sw + static_cast<int64_t>(min(n0 + r, p.N - 1)) * p.groups + g0;
    uint16_t next[4];  // a thread's scales are two bytes of a row of its own: four groups ahead
#pragma unroll
    for (int q = 0; q < 4; ++q) next[q] = q < ng ? sw[q] : uint16_t(0);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    for (int i0 = 0; i0 < ng && ok; i0 += 4) {
      uint16_t cur[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        cur[q] = next[q];
        next[q] = i0 + 4 + q < ng ? sw[i0 + 4 + q] : uint16_t(0);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + q, b = q & 1;
        if (i >= ng) break;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.full[b]), (i >> 1) & 1, p.status, abort));
        if (!ok) break;
        tc_fence_after();
        const float s = bf16_bits_to_f32(cur[q]);
#pragma unroll
        for (int c = 0; c < kTn; c += kLoad) {
          uint32_t d[kLoad];
          tmem_load(tmem + lane_off + kTmemD + 64 * b + c, d);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < kLoad; ++e) {
            const float v = __uint_as_float(d[e]);
            acc[c + e] = fmaf(kFp8 ? v * sxs[q * kTn + c + e] : v, s, acc[c + e]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.drained[b]));
      }
    }
    // every MMA has completed: the operands and the ring are free for the partial
#pragma unroll
    for (int t = 0; t < kTn; ++t) part[t * S::kLd + r] = acc[t];
  }
  tc_fence_before();
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == S::kIssuer) tmem_dealloc(tmem, kTmemCols);

  // the cluster's threads share the (token, row) sums, row fastest, each in rank order
  const int toks = min(kTn, p.T - t0);
  const uint32_t base = smem_u32(part);
  for (int e = rank * S::kThreads + tid; e < toks * kRows; e += p.split * S::kThreads) {
    const int r = e % kRows, t = e / kRows;
    if (n0 + r >= p.N) continue;
    const float v = sum_partials(base + (t * S::kLd + r) * 4, p.split);
    p.y[static_cast<int64_t>(t0 + t) * p.N + n0 + r] = f32_to_bf16_bits(v);
  }
  if (p.split > 1) cluster_sync();  // peers may still be reading this CTA's partial
}

template <int kTn, bool kFp8, bool kRagged>
cudaError_t launch_shape(W4Params p, cudaStream_t stream) {
  using S = TcShape<kTn, kFp8>;
  static bool configured[kMaxDevicesLocal] = {};  // the attribute is per device
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  auto kernel = linear_w4_tc_kernel<kTn, kFp8, kRagged>;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const int tiles = (p.N + kRows - 1) / kRows, slices = (p.T + kTn - 1) / kTn;
  p.split = 1;
  for (int s = 2; s <= kW4MaxSplit && tiles * slices * s <= 152 * S::kPerSm && p.groups >= 2 * s; ++s) p.split = s;
  p.per = (p.groups + p.split - 1) / p.split;
  p.early = launch_overlap() >= 2;
  CUtensorMap tm_w;
  if (!make_tmap_u8_2d(&tm_w, p.w4, p.N, p.K / 2, p.K / 2, 64, kRows, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  return launch_w4(kernel, dim3(tiles * p.split, 1, slices), S::kThreads, S::kSmem, stream, p.split, tm_w, p);
}

template <int kTn, bool kFp8>
cudaError_t launch_tn(const W4Params& p, cudaStream_t stream) {
  return p.K % kW4Group != 0 ? launch_shape<kTn, kFp8, true>(p, stream) : launch_shape<kTn, kFp8, false>(p, stream);
}

template <bool kFp8>
cudaError_t launch_any(const W4Params& p, cudaStream_t stream) {
  if (p.T <= 16) return launch_tn<16, kFp8>(p, stream);
  const int slices = (p.T + 63) / 64;
  if (p.T <= 48 * slices) return launch_tn<48, kFp8>(p, stream);
  return launch_tn<64, kFp8>(p, stream);
}

}  // namespace

cudaError_t launch_linear_w4_tc(const W4Params& p, cudaStream_t stream) {
  return p.sx != nullptr ? launch_any<true>(p, stream) : launch_any<false>(p, stream);
}

}  // namespace mla
