// The value up-projection for many tokens, with the merge of at most two splits:
//   O[t, h, d] = sum_m O'[t, h, m] W_UV[h, d, m],  O' = sum_s exp(lse_s - lse) O'_s
// ("MLA 矩阵吸收 …" section 2.1, V side; FlashMLA point 3 of "DeepSeek-MLA-Principle" for the merge.)
//
// What bounds it is memory: O' in float32, 2 KB a token, head and split (1024 tokens, one split: 268 MB,
// 45 us with the output).  The kernel for few tokens (out_absorb.cu) takes at most 32 tokens a CTA and
// reads the head's 128 KB of weights for each such tile from L2.  Here one CTA a head walks tiles of 128
// tokens (M) with the weights resident; pieces of 32 columns of O' come by TMA into a ring, eight warps
// merge them and round them to two bf16 parts (16 bits of O': 2^-17), which lie beside each other in a
// two-slot ring of chunks of 64 columns, one thread issues their MMAs (N = 128 output columns, both parts
// against the same columns of W_UV), and four warps store a tile while the next one accumulates in the
// other half of tensor memory.
#include "sm100.cuh"
#include "tmap.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kTile = 128;                   // tokens
constexpr int kChunk = 128 * 128;            // 128 rows x 128 bytes (SW128)
constexpr int kChunks = kLatent / 64;
constexpr int kPieces = kLatent / 32;
constexpr int kOffW = 0;                     // W_UV[h]: 8 chunks of 64 m x 128 d
constexpr int kOffRaw = kOffW + kChunks * kChunk;  // pieces: four slots of 128 rows x 128 B, or two of 256 (two splits)
constexpr int kOffA = kOffRaw + 4 * kChunk;        // two slots of merged pieces, 32 columns of either part
constexpr int kOffW2 = kOffA + 2 * kChunk;         // merge weights of a tile's tokens, double buffered
constexpr int kOffBar = kOffW2 + 2 * kTile * 8;
constexpr int kSmemBytes = kOffBar + 256;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr int kMergeThreads = 256;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kStoreWarp = 10;
constexpr int kThreads = 448;

struct Bars {
  uint64_t w_full;
  uint64_t raw_full[4];
  uint64_t raw_free[4];  // the merge warps have read the slot
  uint64_t a_full[2];
  uint64_t a_free[2];    // the MMAs have read the slot
  uint64_t d_full[2];    // a tile's output is in accumulator i & 1
  uint64_t d_free[2];    // ... and has been read
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

struct Params {
  const float* lse_part;  // [T, 2, 128] (two splits)
  uint16_t* out;
  float* lse_out;
  int T;
  int* status;
};

// kSplits 1: O'; 2: two partials.
template <int kSplits>
__global__ void __launch_bounds__(kThreads, 1)
out_absorb_many_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_o, const Params p,
                       bool weights_early) {
  extern __shared__ __align__(1024) uint8_t smem[];  // no room for slack: the launch has no static part before it
  Bars& bars = *reinterpret_cast<Bars*>(smem + kOffBar);
  volatile int* abort = &bars.abort;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int h = blockIdx.x;
  const int tiles = (p.T + kTile - 1) / kTile;
  constexpr uint32_t kRawBytes = kSplits * kChunk;
  constexpr int kRaw = 4 / kSplits;  // slots

  if (tid == 0) {
    mbar_init(smem_u32(&bars.w_full), 1);
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(smem_u32(&bars.raw_full[s]), 1);
      mbar_init(smem_u32(&bars.raw_free[s]), kMergeThreads);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&bars.a_full[s]), 8);
      mbar_init(smem_u32(&bars.a_free[s]), 1);
      mbar_init(smem_u32(&bars.d_full[s]), 1);
      mbar_init(smem_u32(&bars.d_free[s]), 4);
    }
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars.tmem_base), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  auto load_w = [&]() {
    mbar_arrive_expect_tx(smem_u32(&bars.w_full), kChunks * kChunk);
    for (int c = 0; c < kChunks; ++c)
      tma_load_2d(smem_u32(smem + kOffW + c * kChunk), &tm_w, 64 * c, h * kNope, smem_u32(&bars.w_full));
  };
  if (weights_early && tid == 32 * kLoadWarp) load_w();
  grid_dep_wait();
  grid_dep_launch();

  if (warp == kLoadWarp) {
    if (lane == 0) {
      bool ok = true;
      for (int n = 0; n < tiles * kPieces && ok; ++n) {
        const int s = n % kRaw, t0 = (n / kPieces) * kTile;
        if (n >= kRaw) ok = mbar_wait(smem_u32(&bars.raw_free[s]), (n / kRaw - 1) & 1, p.status, abort);
        if (!ok) break;
        const uint32_t bar = smem_u32(&bars.raw_full[s]);
        mbar_arrive_expect_tx(bar, kRawBytes);
        tma_load_3d(smem_u32(smem + kOffRaw + s * kRawBytes), &tm_o, 32 * (n % kPieces), h, kSplits * t0, bar);
        if (n == 0 && !weights_early) load_w();
      }
    }
  } else if (warp == kMmaWarp) {
    const uint32_t idesc = idesc_bf16(128, 128, /*a_mn=*/0, /*b_mn=*/0);
    const uint64_t d_a = smem_desc(smem_u32(smem + kOffA), 16, 1024, kSw128);
    const uint64_t d_w = smem_desc(smem_u32(smem + kOffW), 16, 1024, kSw128);
    auto wait = [&](uint64_t& bar, int phase) {
      const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), phase & 1, p.status, abort));
      tc_fence_after();
      return ok;
    };
    bool ok = wait(bars.w_full, 0);
    for (int n = 0; n < tiles * kPieces && ok; ++n) {
      const int s = n & 1, i = n / kPieces, c = n % kPieces;
      if (c == 0 && i >= 2) ok = wait(bars.d_free[i & 1], (i >> 1) - 1);
      ok = ok && wait(bars.a_full[s], n >> 1);
      if (!ok) break;
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k)  // two steps of the first part, two of the second
          mma_ss(tmem + 128 * (i & 1), d_a + s * (kChunk >> 4) + 2 * k, d_w + (c >> 1) * (kChunk >> 4) + 4 * (c & 1) + 2 * (k & 1),
                 idesc, (c > 0 || k > 0) ? 1u : 0u);
        mma_commit(smem_u32(&bars.a_free[s]));
        if (c == kPieces - 1) mma_commit(smem_u32(&bars.d_full[i & 1]));
      }
      __syncwarp();
    }
  } else if (warp >= kStoreWarp) {
    // thread = token of the tile: its 128 output columns, 256 contiguous bytes
    const int quad = warp & 3, r = quad * 32 + lane;
    for (int i = 0; i < tiles; ++i) {
      const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.d_full[i & 1]), (i >> 1) & 1, p.status, abort));
      if (!ok) break;
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 128 * (i & 1);
      const int t = i * kTile + r;
      uint16_t* dst = p.out + (static_cast<int64_t>(t) * kHeads + h) * kNope;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t v[32];
        tmem_ld32(src + 32 * k, v);
        tmem_wait_ld();
        if (k == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.d_free[i & 1]));
        }
        if (t < p.T) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t* y = v + 8 * u;
            auto two = [](uint32_t a, uint32_t b) { return pack_bf16x2(__uint_as_float(a), __uint_as_float(b)); };
            *reinterpret_cast<uint4*>(dst + 32 * k + 8 * u) =
                make_uint4(two(y[0], y[1]), two(y[2], y[3]), two(y[4], y[5]), two(y[6], y[7]));
          }
        }
      }
    }
  } else {
    // merge: thread (r, half) = 16 of a piece's columns of token r
    const int r = tid & 127, half = tid >> 7;
    float2* weights = reinterpret_cast<float2*>(smem + kOffW2);
    bool ok = true;
    for (int i = 0; i < tiles && ok; ++i) {
      float w0 = 1.f, w1 = 0.f;
      if (kSplits == 2) {
        // the tile's merge weights: exp(lse_s - lse), zero for a split (or a token) without visible tokens
        const int t = i * kTile + r;
        float2* slot = weights + (i & 1) * kTile + r;
        if (half == 0) {
          float2 w = make_float2(0.f, 0.f);
          if (t < p.T) {
            const float* ls = p.lse_part + static_cast<int64_t>(t) * 2 * kHeads + h;
            const float a = ls[0], b = ls[kHeads], m = fmaxf(a, b);
            float lse = m;
            if (a != a || b != b) lse = a + b;  // a NaN stays one (fmaxf drops it)
            if (lse != -INFINITY) {
              const float ea = expf(a - lse), eb = expf(b - lse), z = ea + eb;
              w = make_float2(ea / z, eb / z);
              lse += logf(z);
            }
            if (p.lse_out != nullptr) p.lse_out[static_cast<int64_t>(t) * kHeads + h] = lse;
          }
          *slot = w;
        }
        named_barrier_sync(1, kMergeThreads);
        w0 = slot->x;
        w1 = slot->y;
      }
      for (int c = 0; c < kPieces; ++c) {
        const int n = i * kPieces + c, s = n & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.raw_full[n % kRaw]), (n / kRaw) & 1, p.status, abort));
        if (!ok) break;
        const uint8_t* raw = smem + kOffRaw + (n % kRaw) * kRawBytes;
        uint32_t top[8], rest[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float4 f;
          if (kSplits == 1) {
            f = *reinterpret_cast<const float4*>(raw + r * 128 + (((4 * half + u) ^ (r & 7)) << 4));
          } else {  // the token's two partials in neighbouring rows
            const uint8_t* row = raw + 2 * r * 128;
            const float4 a = *reinterpret_cast<const float4*>(row + (((4 * half + u) ^ (2 * r & 7)) << 4));
            const float4 b = *reinterpret_cast<const float4*>(row + 128 + (((4 * half + u) ^ ((2 * r + 1) & 7)) << 4));
            // a split without visible tokens has zeros: its weight of zero adds nothing
            f = make_float4(w0 * a.x + w1 * b.x, w0 * a.y + w1 * b.y, w0 * a.z + w1 * b.z, w0 * a.w + w1 * b.w);
          }
          top[2 * u] = pack_bf16x2(f.x, f.y);
          top[2 * u + 1] = pack_bf16x2(f.z, f.w);
          rest[2 * u] = bf16x2_rest(f.x, f.y, top[2 * u]);
          rest[2 * u + 1] = bf16x2_rest(f.z, f.w, top[2 * u + 1]);
        }
        if (n >= 2) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.a_free[s]), ((n >> 1) - 1) & 1, p.status, abort));
        if (!ok) break;
        uint8_t* dst = smem + kOffA + s * kChunk + r * 128;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          *reinterpret_cast<uint4*>(dst + (((2 * half + u) ^ (r & 7)) << 4)) =
              make_uint4(top[4 * u], top[4 * u + 1], top[4 * u + 2], top[4 * u + 3]);
          *reinterpret_cast<uint4*>(dst + (((4 + 2 * half + u) ^ (r & 7)) << 4)) =
              make_uint4(rest[4 * u], rest[4 * u + 1], rest[4 * u + 2], rest[4 * u + 3]);
        }
        // the raw slot goes back behind the stores that depend on all its loads
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&bars.raw_free[n % kRaw]));
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.a_full[s]));
      }
      // (the weights' slot of tile i is written again for tile i + 2, behind the barrier of tile i + 1)
      if (kSplits == 2) ok = named_barrier_and(1, kMergeThreads, ok);
    }
  }
  if (*abort) let_work_land();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 256);
}

template <int kSplits>
cudaError_t launch(const float* src, const float* lse_part, const uint16_t* w_uv, uint16_t* out, float* lse_out, int T,
                   int* status, cudaStream_t stream) {
  static bool configured[kMaxDevicesLocal] = {};  // the attribute is per device
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(out_absorb_many_kernel<kSplits>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmemBytes);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const uint64_t rows = static_cast<uint64_t>(T) * kSplits;
  CUtensorMap tw, to;
  if (!make_tmap_bf16_2d(&tw, w_uv, static_cast<uint64_t>(kHeads) * kNope, kLatent, kLatent, 64, kNope,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
      // O' as [rows][128 heads][512]: boxes of 32 columns of a head
      !make_tmap_f32_3d(&to, src, kLatent, kHeads, rows, kLatent * 4ull, static_cast<uint64_t>(kHeads) * kLatent * 4, 32, 1,
                        kSplits * kTile, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const Params prm{lse_part, out, lse_out, T, status};
  return launch_kernel(out_absorb_many_kernel<kSplits>, dim3(kHeads), dim3(kThreads), kSmemBytes, stream, tw, to, prm,
                       launch_overlap() >= 2);
}

}  // namespace

cudaError_t launch_out_absorb_many(const float* src, const float* lse_part, int num_splits, const uint16_t* w_uv,
                                   uint16_t* out, float* lse_out, int T, int* status, cudaStream_t stream) {
  return num_splits == 1 ? launch<1>(src, lse_part, w_uv, out, lse_out, T, status, stream)
                         : launch<2>(src, lse_part, w_uv, out, lse_out, T, status, stream);
}

}  // namespace mla
