// The 4-bit-weight projection of csrc/linear_w4.cu for more than a few tokens, on
// the 5th-generation tensor cores:
//
//   y[t, n] = sum_g sw[n, g] sx[t, g] sum_{k in g} (u[n, k] - 8) x[t, k]
//
// A tile is 128 output features (the M side) by up to kTn tokens (the N side); a CTA
// takes it a group of 128 columns at a time.  Four producer warps unpack the weights:
// thread r turns the 64 bytes of weight row r into 128 exact bf16 values of TMEM lane
// r, or for 8-bit x into 128 E4M3 codes of (u - 8) 2^-9, exact too; x comes by TMA into
// 128-byte-swizzled shared memory as it is.  Two threads issue the groups' MMAs (8 of
// K = 16, or 4 of K = 32 on E4M3) into two TMEM accumulators in turn, and the epilogue
// warps read each back and add it, scaled in fp32, to their registers: an accumulator
// holds one group's exact products only, so no scale is ever rounded into a weight.
//
// The scales of 8-bit x are one for each token, i.e. for each column of the accumulator.
// Read as rows (a lane a row) every lane needs every token's, which filled the port of
// shared memory; read in the warp MMA's fragment layout a lane needs a quarter of them
// (256 tokens, 16384 -> 7168: 75 us; with rows it was 11 more).
//
// Up to 64 tokens two such CTAs share an SM (256 TMEM columns each) and hide each
// other's waits.  Beyond, one has the SM: four operand buffers in front of the
// accumulators and a warp that only fetches x (256 tokens, 16384 -> 7168: 62 us; with
// x fetched by the issuers it was 4 more, with two operand buffers as well 13).  The tile
// of 64 tokens of 8-bit x has more sums and scales than registers and spills 108 bytes.
//
// K is split over a cluster, whose partials meet in distributed shared memory in rank
// order.  Beyond 64 tokens a cluster's CTAs divide the groups of several tiles among
// them, so that the work fits the GPU in one even wave: a CTA has the tail of a tile,
// whole ones, which it stores itself, and the head of another.
//
// What bounds it (256 tokens, 16384 -> 7168: 62 us, 0.51 of the measured bf16 rate): no
// unit (issue slots 51 %, ALU 47 %, tensor pipe 45 % busy), nor the loads of x and of the
// weights, which are not waited for.  Of 66 us in undivided tiles 44 are left without the
// unpacking (58 without it alone), most MMAs (64.8) and the sums (63.8): two thirds are
// the way of a group through the waits from weights to ready, issue, commit and back,
// 0.35 us of it, whose links have not been measured apart.
#include "sm100.cuh"
#include "tmap.cuh"
#include "w4.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kRows = 128;
constexpr int kSlot = kRows * 64;              // a group of weights
constexpr int kStages = 4;                     // groups of weights in flight or in use
constexpr int kRing = kStages * kSlot;
constexpr int kMaxCtas = 304;                  // two on each of 152 SMs: more never run at once
constexpr int kSxStages = 16;                  // groups of x's scales: they are fetched at most ten ahead of the sums

__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&d)[16]) { tmem_ld16(at, d); }
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&d)[8]) { tmem_ld8(at, d); }

struct Bars {
  uint64_t weights[kStages];  // a group of weights has landed (TMA)
  uint64_t x[4];              // a group of x has landed (TMA)
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
  static constexpr int kEpilogue = 4;                          // first epilogue warp
  static constexpr int kEpTok = kTn <= 64 ? kTn : 64;          // tokens of an epilogue thread's registers
  static constexpr int kEpWarps = 4 * (kTn / kEpTok);
  static constexpr int kIssuer = kEpilogue + kEpWarps;         // first of the two warps that issue MMAs
  static constexpr int kACols = kFp8 ? 32 : 64;                // TMEM columns of a group's weights
  // ... in place or in use, in front of two accumulators: as many as fit (16 tokens, 16384 -> 7168: 23.2 us with three,
  // 24.1 with two)
  static constexpr int kABufs = kFp8 || kTn > 64 ? 4 : kTn <= 16 ? 3 : 2;
  static constexpr uint32_t kTmemD = kABufs * kACols;
  static constexpr int kDCols = kTn <= 16 ? 16 : kTn <= 64 ? 64 : 128;  // TMEM columns of an accumulator
  static constexpr uint32_t kTmemCols = kTn <= 64 ? 256 : 512;
  static constexpr bool kLoader = kTn > 64;                    // x is fetched by a warp of its own
  static constexpr int kThreads = 32 * (kIssuer + 2 + (kLoader ? 1 : 0));
  static constexpr int kBox = kTn * 128;                       // kTn tokens x 64 columns (bf16) or 128 (E4M3)
  static constexpr int kB = kFp8 ? kBox : 2 * kBox;            // a group of x
  static constexpr int kXStages = 4;                           // groups of x in flight or in use
  static constexpr int kLd = kFp8 ? kRows + 4 : kRows;         // floats per token of a partial: conflict-free stores
  static constexpr int kPart = kTn * kLd * 4;                  // the CTA's last partial, over the operands
  static constexpr bool kShare = kTn > 64;                     // a cluster may have several tiles
  static constexpr int kMid = kShare ? kPart : 0;              // ... and a CTA holds one partial more
  static constexpr int kBody = kXStages * kB + kRing > kPart ? kXStages * kB + kRing : kPart;
  static constexpr int kSx = kFp8 ? kSxStages * kTn * 4 : 0;   // scales of x
  static constexpr int kSmem = kBody + kMid + kSx + 256 + 1024;
  static_assert(sizeof(Bars) <= 256, "barrier block");
  static_assert(kTmemD + 2 * kDCols <= kTmemCols, "tensor memory");
  static_assert(kSmem * kPerSm <= 227 * 1024, "shared memory");
};

template <int kTn, bool kFp8>
__global__ void __launch_bounds__(TcShape<kTn, kFp8>::kThreads, TcShape<kTn, kFp8>::kPerSm)
linear_w4_tc_kernel(const __grid_constant__ CUtensorMap tm_w0, const __grid_constant__ CUtensorMap tm_w1,
                    const __grid_constant__ CUtensorMap tm_x, const W4Params p) {
  using S = TcShape<kTn, kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + S::kXStages * S::kB;
  float* part = reinterpret_cast<float*>(smem);
  float* mid = reinterpret_cast<float*>(smem + S::kBody);
  float* sxs = reinterpret_cast<float*>(smem + S::kBody + S::kMid);  // [kSxStages][kTn]
  Bars& bars = *reinterpret_cast<Bars*>(smem + S::kBody + S::kMid + S::kSx);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The cluster's tiles laid end to end are `total` groups, of which this CTA has ng from `begin` on.
  const int rank = blockIdx.x % p.split, first = blockIdx.x / p.split * p.share;
  const int total = S::kShare ? min(p.share, p.all - first) * p.groups : p.groups;
  const int per = (total + p.split - 1) / p.split;
  const int begin = min(total, rank * per), ng = min(total - begin, per);
  // A position in them: the group of a tile and where the tile lies.
  struct At {
    int tile, g, n0, t0;
    bool second;
  };
  auto place = [&](At& at) {
    const int q = first + at.tile, n = S::kShare ? q / p.slices : q;
    at.second = n >= p.tiles0;
    at.n0 = (n - (at.second ? p.tiles0 : 0)) * kRows;
    at.t0 = S::kShare ? (q - n * p.slices) * kTn : 0;
  };
  auto at_group = [&](int i) {
    At at;
    at.tile = S::kShare ? (begin + i) / p.groups : 0;
    at.g = begin + i - at.tile * p.groups;
    place(at);
    return at;
  };
  auto advance = [&](At& at, int groups) {
    at.g += groups;
    if (!S::kShare || at.g < p.groups) return;
    at.tile += at.g / p.groups;
    at.g %= p.groups;
    place(at);
  };
  volatile int* abort = &bars.abort;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&bars.weights[i]), 1);
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
  auto fetch_x = [&](int i, const At& at) {
    if (i >= ng) return;
    const uint32_t bar = smem_u32(&bars.x[i & 3]), to = smem_u32(smem + (i & 3) * S::kB);
    mbar_arrive_expect_tx(bar, S::kB);
    tma_load_2d(to, &tm_x, at.g * kW4Group, at.t0, bar);
    if (!kFp8) tma_load_2d(to + S::kBox, &tm_x, at.g * kW4Group + 64, at.t0, bar);
  };
  // The group has left its operands: its MMAs have completed.
  auto wait_free = [&](int i, volatile int* give_up) {
    return mbar_wait(smem_u32(&bars.free[i & 3]), (i >> 2) & 1, p.status, give_up);
  };

  if (warp < S::kEpilogue) {
    // -------------------------------------------------------------- producers
    // Rows past N and columns past K are zeros, tokens past T read as the last one (not stored).
    const int r = tid;
    const uint8_t* wrow = ring + r * 64;
    const int perm = r >> 1 & 3;  // 64-byte swizzle: 16-byte unit q of row r lies at q ^ (r / 2 % 4)
    // x's scales go to shared memory as they are, four groups ahead (a register's would be waited for one group on)
    const float* sx = p.sx;
    int sx_left = 0;  // groups from there to the end of its tile
    auto fetch_sx = [&](int i) {
      if (i < ng && r < kTn) {
        if (sx_left == 0) {
          const At at = at_group(i);
          sx = p.sx + min(at.t0 + r, p.T - 1) * p.groups + at.g;
          sx_left = S::kShare ? p.groups - at.g : ng;
        }
        cp_async4(smem_u32(sxs + i % kSxStages * kTn + r), sx++);
        --sx_left;
      }
      cp_async_commit();
    };
    if (kFp8)
      for (int i = 0; i < 4; ++i) fetch_sx(i);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    for (int i = 0; i < ng; ++i) {
      const int b = i % S::kABufs;
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
      if (i >= S::kABufs) ok = ok && wait_free(i - S::kABufs, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (kFp8) {
        fetch_sx(i + 4);
        cp_async_wait_group<4>();
      }
#pragma unroll
      for (int h = 0; h < (kFp8 ? 2 : 4); ++h) {  // 16 TMEM columns
        uint32_t a[16];
#pragma unroll
        for (int q = 0; q < (kFp8 ? 8 : 4); ++q) {
          if (kFp8) {
            uint32_t c[2];
            w4_e4m3(w[8 * h + q], c);
            a[2 * q] = c[0];
            a[2 * q + 1] = c[1];
          } else {
            uint32_t c[4];
            w4_pairs_natural(w[4 * h + q], c);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[4 * q + e] = c[e];
          }
        }
        tmem_st16(tmem + lane_off + S::kACols * b + 16 * h, a);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.ready[i & 3]));
    }
    cp_async_wait_all();
  } else if (S::kLoader && warp == S::kIssuer + 2) {
    // -------------------------------------------------------------- x
    if (lane == 0) {
      if (p.early) grid_dep_wait();
      At at = at_group(0);
      int i = 0;
      for (; i < ng; ++i) {
        if (i >= 4 && !wait_free(i - 4, abort)) break;
        fetch_x(i, at);
        advance(at, 1);
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
      At w_at = at_group(b), x_at = w_at;
      auto fetch = [&](int i) {
        if (i >= ng) return;
        const uint32_t bar = smem_u32(&bars.weights[i % kStages]);
        mbar_arrive_expect_tx(bar, kSlot);
        tma_load_2d(smem_u32(ring + (i % kStages) * kSlot), w_at.second ? &tm_w1 : &tm_w0, w_at.g * 64, w_at.n0, bar);
        advance(w_at, 2);
      };
      int i = b;
      for (; i < kStages; i += 2) fetch(i);
      auto fetch_x_here = [&](int i) {
        fetch_x(i, x_at);
        advance(x_at, 2);
      };
      // behind the early fetches, and in front of the first bounded wait: its time must not count the previous kernel's
      if (p.early) grid_dep_wait();
      if (!S::kLoader) {
        fetch_x_here(b);
        fetch_x_here(b + 2);
      }
      const uint32_t idesc = kFp8 ? idesc_f16(128, kTn, 0, 0) : idesc_bf16(128, kTn, 0, 0);
      int issued = -1;                                      // the last group whose MMAs are issued
      int w_from = b, w_to = i, x_from = b, x_to = b + 4;  // groups whose copies may be in flight
      for (i = b; i < ng; i += 2) {
        if (!S::kLoader && i >= 2) {
          if (!wait_free(i - 2, abort)) break;
          fetch_x_here(x_to);
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
        const uint32_t d = tmem + S::kTmemD + S::kDCols * b, a0 = tmem + S::kACols * (i % S::kABufs);
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
          mbar_wait(smem_u32(&bars.weights[j % kStages]), (j / kStages) & 1, p.status);
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
    constexpr int kLoad = kTn < 64 ? 16 : 8;  // columns at a time: 64 sums leave few registers
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    auto place_of = [&](int t, int& token, int& to_row) {  // of acc[t] in the tile
      token = c0 + t;
      to_row = r;
      if (kFp8) {
        token = c0 + (t & ~15) + (t & 4 ? 8 : 0) + 2 * (lane & 3) + (t & 1);
        to_row = (warp & 3) * 32 + (t >> 3 & 1) * 16 + (t >> 1 & 1) * 8 + (lane >> 2);
      }
    };
    int from_group = 0;
    if (ng > 0) do {  // the CTA's part of each of its tiles
      const uint16_t* sw;
      int n;
      {
        const At at = at_group(from_group);
        n = S::kShare ? min(ng - from_group, p.groups - at.g) : ng;
        const int last = (at.second ? p.out[1].N : p.out[0].N) - 1;
        sw = (at.second ? p.out[1].sw : p.out[0].sw) + static_cast<int64_t>(min(at.n0 + r, last)) * p.groups + at.g;
      }
      uint16_t next[4];  // a thread's scales are two bytes of a row of its own: four groups ahead
#pragma unroll
      for (int q = 0; q < 4; ++q) next[q] = q < n ? sw[q] : uint16_t(0);
#pragma unroll
      for (int t = 0; t < S::kEpTok; ++t) acc[t] = 0.f;
      bool ok = true;
      for (int j0 = 0; j0 < n && ok; j0 += 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (j0 + q >= n) break;
          const int i = (S::kShare ? from_group : 0) + j0 + q, b = i & 1;
          const float s = bf16_bits_to_f32(next[q]);
          next[q] = j0 + q + 4 < n ? sw[j0 + q + 4] : uint16_t(0);
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
                const float2 sum = f32x2_split(fma_f32x2(v, f32x2(s, s), f32x2(to[0], to[1])));
                to[0] = sum.x;
                to[1] = sum.y;
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.drained[b]));
        }
      }
      if (!ok) break;
      // E4M3 weights carry 2^-9.  It is taken off the sums here, not off the scales in front of them: those go up to
      // 2^125, and 2^9 times that is no fp32 value.
      if (kFp8) {
#pragma unroll
        for (int t = 0; t < S::kEpTok; ++t) acc[t] *= 512.f;
      }
      asm volatile("" : "+r"(from_group));  // found again rather than kept in registers: the loop has none to spare
      const At at = at_group(from_group);
      const W4Out out = at.second ? p.out[1] : p.out[0];
      from_group += n;
      if (n == p.groups) {
        // a whole tile
#pragma unroll
        for (int t = 0; t < S::kEpTok; ++t) {
          int token, to_row;
          place_of(t, token, to_row);
          if (at.t0 + token < p.T && at.n0 + to_row < out.N)
            out.y[static_cast<int64_t>(at.t0 + token) * out.N + at.n0 + to_row] = f32_to_bf16_bits(acc[t]);
        }
      } else {
        // After the CTA's last group every MMA has completed: the operands and the ring are free for the partial.
        float* to = S::kShare && from_group < ng ? mid : part;
#pragma unroll
        for (int t = 0; t < S::kEpTok; ++t) {
          int token, to_row;
          place_of(t, token, to_row);
          to[token * S::kLd + to_row] = acc[t];
        }
      }
    } while (S::kShare && from_group < ng);
  }
  // TMEM goes back before any wait for a peer: kernels on two streams, each waiting in a cluster with TMEM that the
  // other's CTAs need to start, would wait for ever
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == S::kIssuer) tmem_dealloc(tmem, S::kTmemCols);
  if (p.split == 1) return;
  cluster_sync();

  // Tiles of several CTAs: their threads share the (token, row) sums, row fastest, each in rank order, four rows at a
  // time: a round trip to a peer takes about as long whatever it brings (256 tokens, 16384 -> 7168: 3 us less than one row
  // at a time; two places at a time were no better).
  for (At at{0, 0, 0, 0, false}; at.tile * p.groups < total; ++at.tile) {
    const int lo = at.tile * p.groups / per, end = (at.tile + 1) * p.groups, hi = (end - 1) / per;
    if (lo == hi || rank < lo || rank > hi) continue;
    place(at);
    const W4Out out = at.second ? p.out[1] : p.out[0];
    // the last CTA's partial is its first one if it went on to the next tile
    const uint32_t base = smem_u32(part), base_hi = S::kShare && min(total, (hi + 1) * per) > end ? smem_u32(mid) : base;
    const int units = min(kTn, p.T - at.t0) * (kRows / 4), step = (hi - lo + 1) * S::kThreads;
    const bool four = out.N % 4 == 0 && (reinterpret_cast<uintptr_t>(out.y) & 7) == 0;
    for (int e = (rank - lo) * S::kThreads + tid; e < units; e += step) {
      const int r = e % (kRows / 4) * 4, t = e / (kRows / 4), offset = (t * S::kLd + r) * 4;
      if (at.n0 + r >= out.N) continue;
      const float4 sum = sum_partials(base + offset, base_hi + offset, lo, hi);
      uint16_t* y = out.y + static_cast<int64_t>(at.t0 + t) * out.N + at.n0 + r;
      const uint32_t y01 = bf16_pair(sum.x, sum.y), y23 = bf16_pair(sum.z, sum.w);
      if (four) {
        *reinterpret_cast<uint2*>(y) = make_uint2(y01, y23);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at.n0 + r + k < out.N) y[k] = static_cast<uint16_t>((k < 2 ? y01 : y23) >> (k & 1) * 16);
      }
    }
  }
  cluster_sync();  // peers may still be reading this CTA's partials
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
  const int64_t tiles = p.tiles(kRows);
  p.tiles0 = (p.out[0].N + kRows - 1) / kRows;
  p.slices = (p.T + kTn - 1) / kTn;
  p.all = static_cast<int>(tiles * p.slices);
  static int fit[kMaxDevicesLocal][kW4MaxSplit + 1] = {};  // clusters resident at once, 0: not asked yet
  for (int s = 1; s <= kW4MaxSplit; ++s) {
    if (fit[dev][s] != 0) continue;
    int n = 0;
    const cudaError_t e = w4_clusters(kernel, S::kThreads, S::kSmem, s, &n);
    if (e != cudaSuccess) return e;
    fit[dev][s] = n * S::kPerSm;  // the query counts one CTA an SM here, measured are two (56 clusters of 5: one wave)
  }
  p.split = p.share = 1;
  if (S::kShare) {
    // One wave of clusters of `split` CTAs that divide the groups of `share` tiles evenly, whichever leaves a CTA the
    // fewest groups; adding partials up costs about four groups' time (256 tokens, 16384 -> 7168, 112 tiles of 128
    // groups: 66 us in a CTA each, 62 in clusters of five for four tiles).
    int64_t best = -1;
    for (int s = 1; s <= kW4MaxSplit; ++s) {
      const int64_t share = (p.all + fit[dev][s] - 1) / fit[dev][s];
      const int64_t groups = (share * p.groups + s - 1) / s + (s > 1 ? 4 : 0);
      if (best >= 0 && groups >= best) continue;
      best = groups;
      p.split = s;
      p.share = static_cast<int>(share);
    }
  } else {
    // K over the largest cluster whose CTAs still fit the GPU at once (a second, partial wave costs more) and that leaves
    // a CTA two groups, or seven where CTAs share an SM (32 tokens, 1536 -> 16384: 9.6 us undivided, halved 1.3 more)
    for (int s = kW4MaxSplit; s > 1; --s) {
      const int64_t ctas = tiles * s;
      if (ctas > kMaxCtas || p.groups < (ctas <= kMaxCtas / 2 ? 2 : 7) * s || tiles > fit[dev][s]) continue;
      p.split = s;
      break;
    }
  }
  p.early = launch_overlap() >= 2;
  CUtensorMap tm_w[2], tm_x;
  for (int i = 0; i < 2; ++i) {
    const W4Out& o = p.out[i];
    if (o.N == 0) tm_w[i] = tm_w[0];  // no second projection: not read
    else if (!make_tmap_u8_2d(&tm_w[i], o.w4, o.N, p.K / 2, p.K / 2, 64, kRows, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  const bool ok = kFp8 ? make_tmap_u8_2d(&tm_x, p.x, p.T, p.K, p.K, kW4Group, kTn, CU_TENSOR_MAP_SWIZZLE_128B)
                       : make_tmap_bf16_2d(&tm_x, p.x, p.T, p.K, p.K, 64, kTn, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  const unsigned clusters = (static_cast<unsigned>(p.all) + p.share - 1) / p.share;
  return launch_w4(kernel, dim3(clusters * p.split), S::kThreads, S::kSmem, stream, p.split, tm_w[0], tm_w[1], tm_x, p);
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
