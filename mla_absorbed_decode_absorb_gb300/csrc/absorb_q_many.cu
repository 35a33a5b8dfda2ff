// The absorbed query and the cache rows of a tree's tokens, for many tokens:
//   q_abs[t, h, 0:512] = sum_d q_nope[t, h, d] W_UK[h, d, :],  q_abs[t, h, 512:576] = RoPE(q_rope[t, h], pos_t)
// ("MLA 矩阵吸收 …" section 2.1; "DeepSeek-MLA-Principle" key absorption and eq. (8).)
//
// What bounds it is memory: 1152 bytes written and 384 read per token and head, beside 16 MiB of
// weights (1024 tokens: 33 us).  The kernel for few tokens (absorb_q.cu) has the weights as the
// M side, so each of its threads holds one column of many tokens and stores two bytes at a time,
// and its 64-token tiles read the weights again and again: 101 us for 1024 tokens.  Here the
// tokens are M = 128 and a head's 512 latent columns N, one CTA a head that walks the token tiles:
// the head's weights (128 KB) stay in shared memory, the accumulator takes all of tensor memory,
// and rows leave as 128-byte pieces by TMA from a staging box.
//
// Warp 8 loads (the weights once, the queries of a tile as soon as the MMAs have read the last
// one's), warp 9 issues the MMAs of a tile in two halves of 256 columns, warps 0-7 write the rows
// (warp w: TMEM lanes 32 (w % 4) .., half w / 4), warps 10-17 append the cache rows and rotate, four
// of them the even tiles and four the odd ones.
#include "append_row.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kTile = 128;                  // tokens
constexpr int kChunk = 128 * 128;           // 128 rows x 64 bf16 columns (SW128)
constexpr int kOffW = 0;                    // W_UK[h]: 8 chunks of 64 m x 128 d
constexpr int kOffA = kOffW + 8 * kChunk;   // queries of a tile: 2 chunks of 64 d
constexpr int kOffO = kOffA + 2 * kChunk;   // staging: one box for each half, two for the rotated columns
constexpr int kOffPos = kOffO + 4 * kChunk;  // positions of four tiles' tokens
constexpr int kOffBar = kOffPos + 4 * 4 * kTile;
constexpr int kSmemBytes = kOffBar + 128;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr int kThreads = 576;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kRopeWarp = 10;  // warps 10-13 and 14-17

struct Bars {
  uint64_t w_full;
  uint64_t a_full;    // queries of the tile have landed
  uint64_t a_free;    // its MMAs have read them
  uint64_t d_full[2]; // columns [256 x, 256 x + 256) of the tile are in tensor memory
  uint64_t d_free[2]; // ... and have been read
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 128, "barrier block");

struct Params {
  const uint16_t* q_rope;
  const int32_t* lens;
  const int32_t* depths;
  const float* rope;
  int rope_max_pos;
  int T, n_q;
  int* status;
};

__global__ void __launch_bounds__(kThreads, 1)
absorb_q_many_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_o, const Params p, const AppendArgs ap, bool weights_early) {
  extern __shared__ __align__(1024) uint8_t smem[];  // no room for slack: the launch has no static part before it
  Bars& bars = *reinterpret_cast<Bars*>(smem + kOffBar);
  volatile int* abort = &bars.abort;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int h = blockIdx.x;
  const int last = (p.T + kTile - 1) / kTile;

  if (tid == 0) {
    mbar_init(smem_u32(&bars.w_full), 1);
    mbar_init(smem_u32(&bars.a_full), 1);
    mbar_init(smem_u32(&bars.a_free), 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&bars.d_full[x]), 1);
      mbar_init(smem_u32(&bars.d_free[x]), 4);
    }
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  auto load_w = [&]() {
    mbar_arrive_expect_tx(smem_u32(&bars.w_full), 8 * kChunk);
    for (int c = 0; c < 8; ++c) tma_load_2d(smem_u32(smem + kOffW + c * kChunk), &tm_w, 64 * c, h * kNope, smem_u32(&bars.w_full));
  };
  if (weights_early && tid == 32 * kLoadWarp) load_w();
  grid_dep_wait();
  grid_dep_launch();

  if (warp == kLoadWarp) {
    if (lane == 0) {
      if (!weights_early) load_w();
      for (int i = 0; i < last; ++i) {
        if (i > 0 && !mbar_wait(smem_u32(&bars.a_free), (i - 1) & 1, p.status, abort)) break;
        mbar_arrive_expect_tx(smem_u32(&bars.a_full), 2 * kChunk);
        for (int c = 0; c < 2; ++c)
          tma_load_3d(smem_u32(smem + kOffA + c * kChunk), &tm_q, 64 * c, h, i * kTile, smem_u32(&bars.a_full));
      }
    }
  } else if (warp == kMmaWarp) {
    const uint32_t idesc = idesc_bf16(128, 256, /*a_mn=*/0, /*b_mn=*/1);
    const uint64_t d_a = smem_desc(smem_u32(smem + kOffA), 16, 1024, kSw128);
    const uint64_t d_w = smem_desc(smem_u32(smem + kOffW), kChunk, 1024, kSw128);
    auto wait = [&](uint64_t& bar, int phase) {
      const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), phase & 1, p.status, abort));
      tc_fence_after();
      return ok;
    };
    bool ok = wait(bars.w_full, 0);
    int i = 0;
    for (; i < last && ok; ++i) {
      ok = wait(bars.a_full, i);
      for (int x = 0; x < 2 && ok; ++x) {
        if (i > 0) ok = wait(bars.d_free[x], i - 1);
        if (!ok) break;
        const uint32_t elected = static_cast<uint32_t>(lane == 0);
        if (elected) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss(tmem + 256 * x, d_a + (k >> 2) * (kChunk >> 4) + 2 * (k & 3), d_w + x * 4 * (kChunk >> 4) + 128 * k, idesc,
                   k > 0 ? 1u : 0u);
          mma_commit(smem_u32(&bars.d_full[x]));
          if (x == 1) mma_commit(smem_u32(&bars.a_free));
        }
        __syncwarp();
      }
    }
  } else if (warp >= kRopeWarp) {
    const int64_t ctas = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + warp - kRopeWarp; t < p.T; t += ctas) {
      if (ap.cache != nullptr)
        append_token_bf16<true>(ap, t, lane, p.status);
      else
        append_token_fp8<true>(ap, t, lane, p.status);
    }
    // The rotated columns, in units of eight: unit v = r + 128 i of the tile is elements 8 (v % 8) .. + 7 of row
    // v / 8, so that a warp's load covers four rows instead of pieces of 32 (1024 tokens: 44 us; a row a thread, and
    // four warps for all tiles: 51).  The same float32 steps as for few tokens, bit for bit.
    const int group = (warp - kRopeWarp) >> 2, r = tid - 32 * kRopeWarp - 128 * group, f0 = 8 * (r & 3);
    const bool second = (r & 4) != 0;  // element f < 32 pairs with f + 32, four units (lane ^ 4) away
    uint8_t* rot = smem + kOffO + (2 + group) * kChunk;
    // positions of a tile's tokens (-1: left out), a tile ahead
    int* at = reinterpret_cast<int*>(smem + kOffPos) + 2 * kTile * group;
    auto position = [&](int t) {
      if (t >= p.T) return -1;
      const int depth = p.depths[t];
      if (depth < 0) return -1;
      const int64_t pos = static_cast<int64_t>(p.lens[t / p.n_q]) + depth;
      if (pos >= 0 && pos < p.rope_max_pos) return static_cast<int>(pos);
      record_status(p.status, MLA_ERR_BOUNDS);
      return -1;
    };
    at[r] = position(group * kTile + r);
    named_barrier_sync(3 + group, 128);
    for (int i = group, n = 0; i < last; i += 2, ++n) {
      uint4 out[8];
      const int ahead = position((i + 2) * kTile + r);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint4 q[4];
        float4 cs[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = (r >> 3) + 16 * (4 * half + k), pos = at[(n & 1) * kTile + row], t = pos < 0 ? 0 : i * kTile + row;
          q[k] = __ldg(reinterpret_cast<const uint4*>(p.q_rope + (static_cast<int64_t>(t) * kHeads + h) * kRope) + (r & 7));
          const float4* tab = reinterpret_cast<const float4*>(p.rope + static_cast<int64_t>(max(pos, 0)) * kRope + f0);
          if (pos < 0) q[k] = make_uint4(0, 0, 0, 0);  // (a token left out: zeros, turned by position 0)
          cs[k][0] = __ldg(tab);
          cs[k][1] = __ldg(tab + 1);
          cs[k][2] = __ldg(tab + kHalfRope / 4);
          cs[k][3] = __ldg(tab + kHalfRope / 4 + 1);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t mine[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
          const float cc[8] = {cs[k][0].x, cs[k][0].y, cs[k][0].z, cs[k][0].w,
                               cs[k][1].x, cs[k][1].y, cs[k][1].z, cs[k][1].w};
          const float ss[8] = {cs[k][2].x, cs[k][2].y, cs[k][2].z, cs[k][2].w,
                               cs[k][3].x, cs[k][3].y, cs[k][3].z, cs[k][3].w};
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, mine[e], 4);
            float y[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float a = __uint_as_float(x ? mine[e] & 0xffff0000u : mine[e] << 16);
              const float b = __uint_as_float(x ? other & 0xffff0000u : other << 16);
              const float ac = __fmul_rn(a, cc[2 * e + x]), bs = __fmul_rn(b, ss[2 * e + x]);
              y[x] = second ? __fadd_rn(ac, bs) : __fsub_rn(ac, bs);
            }
            w[e] = pack_bf16x2(y[0], y[1]);
          }
          out[4 * half + k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      at[(~n & 1) * kTile + r] = ahead;
      if (r == 0) bulk_wait_read<0>();  // the last tile's box has been read
      named_barrier_sync(3 + group, 128);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4*>(rot + sw128(((r >> 3) + 16 * k) * 128 + (r & 7) * 16)) = out[k];
      fence_proxy_async_smem();
      named_barrier_sync(3 + group, 128);
      if (r == 0) {
        tma_store_3d(&tm_o, smem_u32(rot), kLatent, h, i * kTile);
        bulk_commit_group();
      }
    }
    if (r == 0) bulk_wait_all();
  } else {
    // Warpgroup x = warp / 4: latent columns [256 x, 256 x + 256) of row r.
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;
    const bool leader = (warp & 3) == 0 && lane == 0;
    uint8_t* box = smem + kOffO + x * kChunk;
    auto unit = [&](uint8_t* b, int u) { return reinterpret_cast<uint4*>(b + r * 128 + ((u ^ (r & 7)) << 4)); };
    bool ok = true;
    for (int i = 0; i < last; ++i) {
      ok = mbar_wait(smem_u32(&bars.d_full[x]), i & 1, p.status, abort);
      ok = named_barrier_and(1 + x, 128, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256 * x;
      // four boxes of 64 columns: the next one's columns are in registers before the staging box is free again
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t va[32], vb[32];
        tmem_ld32(src + 64 * k, va);
        tmem_ld32(src + 64 * k + 32, vb);
        tmem_wait_ld();
        if (k == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.d_free[x]));
        }
        if (leader) bulk_wait_read<0>();
        named_barrier_sync(1 + x, 128);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t* y = va + 8 * u;
          const uint32_t* z = vb + 8 * u;
          auto two = [](uint32_t m, uint32_t n) { return pack_bf16x2(__uint_as_float(m), __uint_as_float(n)); };
          *unit(box, u) = make_uint4(two(y[0], y[1]), two(y[2], y[3]), two(y[4], y[5]), two(y[6], y[7]));
          *unit(box, 4 + u) = make_uint4(two(z[0], z[1]), two(z[2], z[3]), two(z[4], z[5]), two(z[6], z[7]));
        }
        fence_proxy_async_smem();
        named_barrier_sync(1 + x, 128);
        if (leader) {
          tma_store_3d(&tm_o, smem_u32(box), 256 * x + 64 * k, h, i * kTile);
          bulk_commit_group();
        }
      }
    }
    if (leader) bulk_wait_all();
  }
  if (*abort) let_work_land();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_absorb_q_many(const uint16_t* q_nope, const uint16_t* q_rope, const int32_t* seq_lens_before,
                                 const int32_t* depths, const uint16_t* w_uk, const float* rope_table,
                                 int rope_max_pos, uint16_t* q_abs, int B, int n_q, const AppendArgs& ap, int* status,
                                 cudaStream_t stream) {
  static bool configured[kMaxDevicesLocal] = {};  // the attribute is per device
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(absorb_q_many_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const int T = B * n_q;
  const uint64_t tokens = static_cast<uint64_t>(T);
  CUtensorMap tw, tq, to;
  if (!make_tmap_bf16_2d(&tw, w_uk, static_cast<uint64_t>(kHeads) * kNope, kLatent, kLatent, 64, kNope,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_bf16_3d(&tq, q_nope, kNope, kHeads, tokens, kNope * 2ull, static_cast<uint64_t>(kHeads) * kNope * 2, 64, 1,
                         kTile, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_bf16_3d(&to, q_abs, kRow, kHeads, tokens, kRow * 2ull, static_cast<uint64_t>(kHeads) * kRow * 2, 64, 1,
                         kTile, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  Params prm;
  prm.q_rope = q_rope;
  prm.lens = seq_lens_before;
  prm.depths = depths;
  prm.rope = rope_table;
  prm.rope_max_pos = rope_max_pos;
  prm.T = T;
  prm.n_q = n_q;
  prm.status = status;
  return launch_kernel(absorb_q_many_kernel, dim3(kHeads), dim3(kThreads), kSmemBytes, stream, tw, tq, to, prm,
                       ap, launch_overlap() >= 2);
}

}  // namespace mla
