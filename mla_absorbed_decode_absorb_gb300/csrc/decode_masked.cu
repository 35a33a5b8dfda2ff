// Attention over the paged latent cache for queries that see only part of it: a
// tree of drafted tokens, a sliding window with first tokens that stay visible.
//
// Per (sequence b, query j, split s) and head h, over the visible tokens t of the split:
//   score_t = (q_abs[h, 0:512] . c_t + q_abs[h, 512:576] . kR_t) / sqrt(192)
//   O'_s[h] = sum_t softmax(score)_t c_t,   lse_s[h] = log sum_t exp(score_t)
// ("MLA 矩阵吸收 …" section 4.1 and "DeepSeek-MLA-Principle" section 2 and FlashMLA
//  points 3 and 4, as the causal kernel; the pages name no trees and no windows.)
//
// What is visible is a set of pages and, within a page, a 64-bit word (view.cuh): the
// same for all heads of a query, so masking costs nothing on whole pages.
//
// The 128 heads of a query are the M = 128 rows of one tcgen05 tile spread over a pair
// of CTAs (cta_group::2): CTA r holds heads [64r, 64r + 64) of the query, of the
// scores and of O'.  At M = 128 a pair's tile puts its 64 rows into all 128 TMEM lanes
// of each CTA: lanes 0-63 hold the first half of the N columns, lanes 64-127 the
// second.  O' of 64 heads is then 256 TMEM columns, which leaves room for two score
// buffers, and the pair needs no exchange of partial scores.  Measured, MMAs back to
// back: this shape takes 34 cycles at N = 128 and 66 at N = 256, the full rate, where
// its operands sit in shared memory and one elected thread of a converged warp issues
// it (52 cycles at least from a divergent thread).
//
// A tile is two pages, e and o.  For S = Q K^T (N = 128 tokens) CTA 0 holds the keys of
// page e and CTA 1 those of page o.  For O' += P V (N = 256 latent columns at a time)
// CTA 0 holds columns [0, 256) of both pages and CTA 1 [256, 512).  An MMA finds its
// operand at the same offset in both CTAs, so a buffer has two halves of 32 KB, X0 and
// X1, and one of them changes its contents between the two products:
//             X0                                   X1
//   CTA 0   e columns 0-255 (keys and values)    e columns 256-511, then o columns 0-255
//   CTA 1   o columns 0-255, then e 256-511      o columns 256-511 (keys and values)
// 104 KB of a tile's 144 KB go to each CTA.  Two such buffers, the RoPE keys (8 KB, one
// buffer, needed last), the query (72 KB) and P (16 KB) fill the shared memory.
//
// The FP8 cache keeps this shape and multiplies the E4M3 codes as they are (kind::f8f6f4,
// K = 32 at the same time as K = 16 of 16 bits), with the other operand in two 8-bit parts.
// The query: x1 = E4M3(x) and x2 = E4M3(x - x1), which holds a bf16 value without loss (its
// rows scaled by a power of two, down to 2^-10 of the row's largest value; E5M2 first would take
// the range further, and a bit from every value).  P, whose small
// weights count where there are many: x1 = E5M2(x) and x2 = E4M3(x - x1), with 2^9 at the row's
// reference, the largest product of a weight and its token's scale.  That is bf16's half a step,
// 2^-8 of a product, down to 2^-11 of the largest, and 2^-3 of it, to nearest, down to 2^-23 (0
// below 2^-26).  With both parts in E4M3 and 64 at the reference a product was within 2^-9, but 0
// below 2^-16: of 8191 tokens 12 nats below a first one a quarter of the result was missing.
// Codes take half the bytes of bf16 rows on the way and in shared memory, so three buffers fit
// instead of two.  Widening them to f16 in front of the MMAs instead, by eight warps of each CTA,
// took 6,700 cycles a tile: they waited for their own loads.
//
// What bounds it: a tile's products take 2,284 cycles by themselves, a tile 2,680 (2,650 to 2,770 over
// the units of 32 x 32 queries; FP8: 2,570 for a unit by itself, 2,780 on a full GPU), so the tensor cores
// work 85% of the time.  What the other 15% wait for is not known: operands, loads and P move 360 KB
// through each CTA's shared memory (240 + 104 + 16; 2,880 cycles if all of it went at 128 bytes a cycle,
// which the measured tile shows it need not).  32 sequences of 8192 tokens, 32 queries each: 1420 us, 1.64
// PFLOP/s; 16 of 2000-6000 with 24 over the FP8 cache: 339 us.  A pair's fixed cost (launch, query, first
// tile, the way out) is some six tiles, and where units do not fill their last wave of pairs the GPU
// waits for it: 96 queries of 2060 tokens 64 us, of which the products are 31.  Sharing out all tiles
// evenly instead (pairs that go on from one unit to the next) filled the waves, but its bookkeeping in
// every role cost 5-25% a tile, more than it gained on all but a few sizes.
//
// P is rounded to bf16, the type of the rows that it weighs (a second bf16 part would be 16 more products of 66
// cycles a tile, and 16 KB of shared memory that the tiles fill); O' leaves in float32, as a split's partial too.
//
// Roles: warps 0-7 softmax (thread = one head and half a page of the tile); warp 8 loads keys,
// warp 9 the RoPE keys, the values that replace keys, and scales; in CTA 0 warp 10 issues the
// products S and warp 11 the products O', each waiting for its own barriers, so that neither
// waits behind the other's.
#include "sm100.cuh"
#include "tmap.cuh"
#include "view.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kRows = 64;             // heads of a CTA
constexpr int kSoftThreads = 256;     // warps 0-7
constexpr int kKeysWarp = 8;
constexpr int kValuesWarp = 9;
constexpr int kScoresMmaWarp = 10;
constexpr int kOutMmaWarp = 11;
constexpr int kThreads = 384;
constexpr int kChunk = 64 * 128;      // 64 rows x 128 bytes (SW128): 64 columns of 16 bits, 128 of 8
template <bool kFp8>
constexpr int kHalf = kFp8 ? 2 * kChunk : 4 * kChunk;  // X0 or X1: 256 columns of 64 tokens
template <bool kFp8>
constexpr int kBufs = kFp8 ? 3 : 2;   // tiles in shared memory
constexpr int kOffQ = 0;              // 64 heads: 9 chunks of bf16, or 4 + 4 of the two E4M3 parts and one of f16
constexpr int kOffX = kOffQ + 9 * kChunk;
constexpr int kOffR = kOffX + 16 * kChunk;  // RoPE keys of the tile
constexpr int kOffP = kOffR + kChunk;       // P: a chunk for each page, or for each E4M3 part
constexpr int kOffBar = kOffP + 2 * kChunk;
constexpr int kOffHx = kOffBar + 320;  // a row's four maxima, then its four sums; double buffered
constexpr int kOffScale = kOffX + 2 * kBufs<true> * kHalf<true>;  // FP8: scales of a tile's tokens, double buffered
constexpr int kOffLog2 = kOffScale + 2 * 4 * 2 * kPage;  // and, of each softmax warp's 32, their exponents
constexpr int kSmemBytes = kOffHx + 2 * 4 * 4 * kRows;
static_assert(2 * kBufs<false> * kHalf<false> == 16 * kChunk && kOffLog2 + 4 * kSoftThreads <= kOffR, "buffers");
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemO = 0;    // O': column 128 h + c of lane l is latent column 256 (l / 64) + 128 h + c
constexpr uint32_t kTmemS = 256;  // two score buffers of 64 columns
constexpr uint32_t kTmemR = 384;  // FP8: the RoPE part of the scores, two buffers as well
// O' is rescaled where a row's maximum grows by more than this.  The FP8 form's P is 2^kPUpLog2 at the
// reference and must stay below 2^12, from where on what E5M2 leaves over passes E4M3's 448.
template <bool kFp8>
constexpr float kPUpLog2 = kFp8 ? 9.f : 0.f;
template <bool kFp8>
constexpr float kRescaleLog2 = kFp8 ? 2.8f : 8.f;
static_assert(kPUpLog2<true> + kRescaleLog2<true> < 12.f, "P in two parts");
constexpr int kOutPitch = 4 * kLatent + 16;  // a row of O' on its way out
static_assert(kOffX + kRows * kOutPitch <= kOffP, "rows of O' in the tiles' place");
constexpr uint16_t kBoth = 0x3;
constexpr int kMostSorted = 256;  // splits that are sorted by length

struct Bars {
  uint64_t sc_full[2];  // FP8: the scales of tile i have landed
  uint64_t q_land;      // FP8: the query of this CTA has landed (it is split before it counts as full)
  uint64_t q_full;      // (CTA 0) the query of both CTAs is in place
  uint64_t k_full[8];   // (CTA 0) keys of tile i in buffer i mod kBufs, half h: 2 (i mod kBufs) + h
  uint64_t r_full;      // (CTA 0) RoPE keys of the tile
  uint64_t v_full[4];   // the half that changes holds the other page's values (this CTA)
  uint64_t q0_done[2];  // the first product of S of tile i has read the keys in X0
  uint64_t s_full[2];   // S of tile i in score buffer i & 1; all its keys have been read
  uint64_t s_free[2];   // (CTA 0) both CTAs have read it
  uint64_t p_full[2];   // (CTA 0) P of page e (o) of the tile and its values are in place in both (and O' rescaled)
  uint64_t x_empty[8];  // O' of tile i has read X0 (X1) of its buffer
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int chosen;           // the place of this unit's split
};
static_assert(sizeof(Bars) <= 320, "barrier block");

struct Params {
  const uint8_t* c8;  // FP8 cache
  const float* scale;
  const int32_t* page_table;
  const int32_t* kv_lens;
  const uint64_t* words;  // [B, n_q] visible drafts, or nullptr: causal
  const int32_t* depths;  // [B, n_q] a draft's position past the context, or nullptr: its index
  float* o_out;
  float* lse_out;
  int* status;
  int64_t num_pages;
  int pt_stride;
  int n_q;
  int max_kv_len;
  int window;
  int sinks;
  int split_pages;
  int num_splits;
  int max_pages;
  int longest_first;  // splits to sort by length (0: as they come)
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma2_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same of E4M3 operands (K = 32); idesc_f16's formats (0) are E4M3 here.
__device__ __forceinline__ void mma2_ss_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the pair's MMAs issued so far have completed.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(bar), "h"(kBoth)
               : "memory");
}
// Arrive on a barrier of CTA 0, releasing at the scope of this CTA: what it orders are this
// CTA's own tensor memory and shared memory, where the pair's MMAs read them.  (Released at
// cluster scope, an arrive held its warp for 1,100 cycles and a tile took 4,130 instead of 3,300.)
__device__ __forceinline__ void arrive_pair(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// 3-D tiled load into this CTA's shared memory that completes on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load2_3d(uint32_t dst, const void* tmap, int32_t x, int32_t y, int32_t z,
                                             uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
      : "memory");
}

// An f16 pair in two E4M3 parts: x1 = E4M3(x) and x2 = E4M3(x - x1) (the difference is exact).
__device__ __forceinline__ void split_e4m3(uint32_t x, uint16_t& x1, uint16_t& x2) {
  uint32_t back, rest;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(x1) : "r"(x));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(x1));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(x), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(x2) : "r"(rest));
}
// The same of a weight's pair (not negative): E5M2 is an f16's upper byte, rounded.
__device__ __forceinline__ void split_e5m2(uint32_t x, uint16_t& x1, uint16_t& x2) {
  uint32_t rest;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(x1) : "r"(x));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(x), "r"(__byte_perm(x1, 0, 0x1404)));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(x2) : "r"(rest));
}
// A bf16 pair times k as f16.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t u, float k) {
  return pack_f16x2(__uint_as_float(u << 16) * k, __uint_as_float(u & 0xffff0000u) * k);
}

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
decode_masked_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c,
                     const __grid_constant__ CUtensorMap tm_r, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];  // no room for slack: the launch has no static part before it
  Bars& bars = *reinterpret_cast<Bars*>(smem + kOffBar);
  volatile int* abort = &bars.abort;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  // the queries of one sequence and split are neighbours: they read the same pages
  const int unit = blockIdx.x >> 1;
  const int j = unit % p.n_q;
  int bs = unit / p.n_q;

  if (tid == 0) {
    mbar_init(smem_u32(&bars.q_land), 1);
    mbar_init(smem_u32(&bars.q_full), kFp8 ? 16 : 1);  // the softmax warps of both CTAs
    for (int k = 0; k < 8; ++k) {
      mbar_init(smem_u32(&bars.k_full[k]), 1);
      mbar_init(smem_u32(&bars.x_empty[k]), 1);
    }
    mbar_init(smem_u32(&bars.r_full), 1);
    for (int k = 0; k < 4; ++k) mbar_init(smem_u32(&bars.v_full[k]), 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&bars.q0_done[k]), 1);
      mbar_init(smem_u32(&bars.s_full[k]), 1);
      mbar_init(smem_u32(&bars.sc_full[k]), 1);
      mbar_init(smem_u32(&bars.s_free[k]), 16);              // the softmax warps of both CTAs
      mbar_init(smem_u32(&bars.p_full[k]), k == 0 ? 16 : 8);  // all of them; those of page o
    }
    mbar_init(smem_u32(&bars.drain), 2);  // both issuers
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kScoresMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bars.tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and tensor memory exist
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  grid_dep_wait();
  grid_dep_launch();

  if (p.longest_first > 0) {
    // The bs-th of the splits in the order of their length: the last ones to start are then short, and no pair is
    // left with a long one while the others have nothing to do.  (8 sequences of 1000-5000 tokens with 13 queries
    // each: 104 us as they come, 82 longest first; equal lengths, where it decides nothing: 66 and 67.)
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem + kOffP);  // length, then place
    if (tid < kMostSorted) {
      const int pages = tid < p.longest_first
                            ? min(pages_of(max(p.kv_lens[tid / p.num_splits], 0)), p.max_pages) -
                                  (tid % p.num_splits) * p.split_pages
                            : 0;
      const int length = min(max(pages, 0), min(p.split_pages, 1 << 20));
      keys[tid] = tid < p.longest_first ? static_cast<uint32_t>(length + 1) * kMostSorted - tid : 0u;
    }
    __syncthreads();
    if (tid < p.longest_first) {
      const uint32_t mine = keys[tid];
      int before = 0;
      for (int e = 0; e < p.longest_first; e += 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + e);
        before += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
      }
      if (before == bs) bars.chosen = tid;
    }
    __syncthreads();
    bs = bars.chosen;
  }
  const int split = bs % p.num_splits, b = bs / p.num_splits;
  const int64_t bj = static_cast<int64_t>(b) * p.n_q + j;

  // what the query sees of this split: pages [k0, k0 + n) of its view, the same in both CTAs
  const int kv = p.kv_lens[b];
  uint64_t word = p.words != nullptr ? p.words[bj] & low_bits(p.n_q) : low_bits(j + 1);
  const int depth = p.depths != nullptr ? p.depths[bj] : j;
  const bool used = word != 0;  // a node that sees nothing is not part of the tree
  const bool bad = used && (kv > p.max_kv_len || kv < p.n_q || pages_of(kv) > p.pt_stride || depth < 0 || depth >= p.n_q);
  QueryView v{};
  if (used && !bad) v = make_view(kv - p.n_q, kv - p.n_q + depth, word, p.words == nullptr, p.window, p.sinks);
  const int k0 = split * p.split_pages;
  const int n = max(0, min(p.split_pages, v.n_pages - k0));
  const int tiles = (n + 1) / 2;
  if (tid == 0 && bad && rank == 0) record_status(p.status, MLA_ERR_BOUNDS);

  constexpr int kNB = kBufs<kFp8>, kH = kHalf<kFp8>;
  auto passed = [&](uint64_t& bar, int phase) {
    return mbar_wait_cluster(smem_u32(&bar), phase & 1, p.status, abort);
  };

  if (warp == kKeysWarp || warp == kValuesWarp) {
    // ------------------------------------------------------------ TMA
    auto load = [&]() {
      const int32_t* pt = p.page_table + static_cast<int64_t>(b) * p.pt_stride;
      const uint32_t x0 = smem_u32(smem + kOffX);
      const int me = static_cast<int>(rank), it = me ^ 1;  // pages 2 i + me and 2 i + it of tile i
      auto lead = [&](uint64_t& bar) { return mapa(smem_u32(&bar), 0); };
      // the page id of the split's k-th page (0 past its end), read well before it is used
      auto page_id = [&](int k) { return k < n ? pt[view_page(v, k0 + k)] : 0; };
      auto page_row = [&](int id) {  // its first cache row
        if (id >= 0 && id < p.num_pages) return id * kPage;
        record_status(p.status, MLA_ERR_BOUNDS);
        return 0;  // stay in bounds; the result of this unit is not meaningful
      };
      // keys of tile i, half h: this CTA's page of it
      auto load_keys = [&](int i, int h, int id) {
        const int s = 2 * (i % kNB) + h;
        const bool odd = 2 * i + 1 < n;  // the tile has a page o
        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&bars.k_full[s]), odd ? 2 * kH : kH);
        if (rank == 0 || odd) tma_load2_3d(x0 + s * kH, &tm_c, 0, page_row(id), (kFp8 ? 2 : 4) * h, lead(bars.k_full[s]));
      };
      auto load_rope = [&](int i, int id) {
        const bool odd = 2 * i + 1 < n;
        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&bars.r_full), odd ? 2 * kChunk : kChunk);
        if (rank == 0 || odd)
          tma_load2_3d(smem_u32(smem + kOffR), &tm_r, 0, page_row(id), kFp8 ? 0 : 8, lead(bars.r_full));
      };
      // values of the other page of tile i into the half that its keys have left: CTA 0 X1, CTA 1 X0
      auto load_values = [&](int i, int id) {
        const uint32_t vb = smem_u32(&bars.v_full[i % kNB]);
        if (2 * i + it < n) {
          mbar_arrive_expect_tx(vb, kH);
          tma_load_3d(x0 + (2 * (i % kNB) + it) * kH, &tm_c, 0, page_row(id), (kFp8 ? 2 : 4) * me, vb);
        } else {
          mbar_arrive(vb);
        }
      };
      // FP8: scales of both pages of tile i
      auto load_scales = [&](int i, int id_mine, int id_other) {
        const uint32_t sb = smem_u32(&bars.sc_full[i & 1]);
        const uint32_t dst = smem_u32(smem + kOffScale + (i & 1) * 8 * kPage);
        const bool mine = 2 * i + me < n, other = 2 * i + it < n;
        mbar_arrive_expect_tx(sb, 4 * kPage * (static_cast<int>(mine) + static_cast<int>(other)));
        if (mine) bulk_load(dst + me * 4 * kPage, p.scale + page_row(id_mine), 4 * kPage, sb);
        if (other) bulk_load(dst + it * 4 * kPage, p.scale + page_row(id_other), 4 * kPage, sb);
      };
      auto prefetch = [&](int k, int id) {  // a page of this CTA into L2
        if (k >= n || id < 0 || id >= p.num_pages) return;
        tma_prefetch_l2_3d(&tm_c, 0, id * kPage, 0);
        tma_prefetch_l2_3d(&tm_c, 0, id * kPage, kFp8 ? 2 : 4);
        tma_prefetch_l2_3d(&tm_r, 0, id * kPage, kFp8 ? 0 : 8);
      };
      if (warp == kKeysWarp) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_c);
        const uint32_t qb = kFp8 ? smem_u32(&bars.q_land) : lead(bars.q_full);
        if (kFp8)
          mbar_arrive_expect_tx(qb, 9 * kChunk);
        else if (rank == 0)
          mbar_arrive_expect_tx(smem_u32(&bars.q_full), 18 * kChunk);
        int first[kNB];
#pragma unroll
        for (int i = 0; i < kNB; ++i) first[i] = page_id(2 * i + me);
        // each page id is read an iteration ahead
        int id = page_id(2 * kNB + me), id1 = page_id(2 * (kNB + 1) + me);
        for (int c = 0; c < 9; c += 3)
          tma_load2_3d(smem_u32(smem + kOffQ + c * kChunk), &tm_q, 0, static_cast<int32_t>(bj * kHeads + kRows * rank), c,
                       qb);
#pragma unroll
        for (int i = 0; i < kNB; ++i) {
          if (i < tiles) {
            load_keys(i, 0, first[i]);
            load_keys(i, 1, first[i]);
          }
        }
        // tile i takes the place of tile i - kNB once O' of that has read its values
        for (int i = kNB; i < tiles; ++i) {
          const int id2 = page_id(2 * (i + 2) + me);
          for (int h = 0; h < 2; ++h) {
            if (!passed(bars.x_empty[2 * (i % kNB) + h], i / kNB - 1)) return;
            load_keys(i, h, id);
            if (h == 0) prefetch(2 * (i + 1) + me, id1);
          }
          id = id1;
          id1 = id2;
        }
      } else {
        tma_prefetch_desc(&tm_r);
        int mine0 = page_id(me), mine1 = page_id(2 + me), other0 = page_id(it), other1 = page_id(2 + it);
        load_rope(0, mine0);
        if (kFp8) load_scales(0, mine0, other0);
        if (kFp8 && tiles > 1) load_scales(1, mine1, other1);
        for (int i = 0; i < tiles; ++i) {
          const int mine2 = page_id(2 * (i + 2) + me), other2 = page_id(2 * (i + 2) + it);
          const bool more = i + 1 < tiles;
          if (rank == 1) {
            if (!passed(bars.q0_done[i & 1], i >> 1)) return;
            load_values(i, other0);  // X0
          }
          if (!passed(bars.s_full[i & 1], i >> 1)) return;
          if (more) load_rope(i + 1, mine1);
          if (rank == 0) load_values(i, other0);  // X1
          if (kFp8 && i >= 1 && more) {
            // O'(i - 1) is complete, so P of tile i - 1 is, which holds its scales.  (An arrive behind the
            // loads of the scales alone would not do: it may pass loads that are still on their way.)
            if (!passed(bars.x_empty[2 * ((i - 1) % kNB) + 1], (i - 1) / kNB)) return;
            load_scales(i + 1, mine1, other1);
          }
          mine1 = mine2;
          other0 = other1;
          other1 = other2;
        }
      }
    };
    if (tiles > 0 && lane == 0) load();
    __syncwarp();
  } else if (warp == kScoresMmaWarp || warp == kOutMmaWarp) {
    // ------------------------------------------------------------ the pair's MMAs
    if (rank == 0 && tiles > 0) {
      // 16-bit operands of the RoPE product (FP8: f16) and, of a bf16 cache, of all the others
      const uint32_t idesc_s = kFp8 ? idesc_f16(128, 128, /*a_mn=*/0, /*b_mn=*/0) : idesc_bf16(128, 128, 0, 0);
      const uint32_t idesc_o = kFp8 ? idesc_f16(128, 256, /*a_mn=*/0, /*b_mn=*/1) : idesc_bf16(128, 256, 0, 1);
      constexpr uint32_t kE5m2A = 1u << 7;  // (FP8) P's first part
      const uint64_t d_q = smem_desc(smem_u32(smem + kOffQ), 16, 1024, kSw128);
      const uint64_t d_k = smem_desc(smem_u32(smem + kOffX), 16, 1024, kSw128);      // keys (K-major)
      const uint64_t d_r = smem_desc(smem_u32(smem + kOffR), 16, 1024, kSw128);
      const uint64_t d_v = smem_desc(smem_u32(smem + kOffX), kChunk, 1024, kSw128);  // values (MN-major)
      const uint64_t d_p = smem_desc(smem_u32(smem + kOffP), 16, 1024, kSw128);
      constexpr uint64_t kC = kChunk >> 4;  // descriptors count 16 bytes
      auto wait = [&](uint64_t& bar, int phase) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&bar), phase & 1, p.status, abort));
        tc_fence_after();
        return ok;
      };
      bool ok = warp == kOutMmaWarp || wait(bars.q_full, 0);
      // S of tile i from the keys in X0 (h = 0), or from X1 and the RoPE keys (h = 1)
      auto scores = [&](int i, int h) {
        const int buf = i & 1, half = 2 * (i % kNB) + h;
        const uint32_t d = tmem + kTmemS + 64 * buf;
        if (h == 0 && i >= 2) ok = ok && wait(bars.s_free[buf], (i >> 1) - 1);
        ok = ok && wait(bars.k_full[half], i / kNB);
        if (!ok) return;
        const uint64_t kb = d_k + half * static_cast<uint64_t>(kH >> 4);
        if (elect_one()) {
          if (kFp8) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {  // two chunks of 128 columns, four steps of 32, the query's two parts
              const int c = k >> 3, step = (k >> 1) & 3, part = k & 1;
              mma2_ss_f8(d, d_q + (4 * part + 2 * h + c) * kC + 2 * step, kb + c * kC + 2 * step, idesc_s,
                         (h > 0 || k > 0) ? 1u : 0u);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)  // four chunks of 64 columns, four steps of 16
              mma2_ss(d, d_q + (4 * h + (k >> 2)) * kC + (k & 3) * 2, kb + (k >> 2) * kC + (k & 3) * 2, idesc_s,
                      (h > 0 || k > 0) ? 1u : 0u);
          }
          if (h == 0) commit2(smem_u32(&bars.q0_done[buf]));
        }
        __syncwarp();
        if (h == 0) return;
        ok = wait(bars.r_full, i);
        if (!ok) return;
        if (elect_one()) {
          // Products of two kinds into one accumulator are not kept in order (their shapes differ): the FP8
          // form adds its f16 part in the softmax.
          const uint32_t dr = kFp8 ? tmem + kTmemR + 64 * buf : d;
#pragma unroll
          for (int k = 0; k < 4; ++k) mma2_ss(dr, d_q + 8 * kC + 2 * k, d_r + 2 * k, idesc_s, (!kFp8 || k > 0) ? 1u : 0u);
          commit2(smem_u32(&bars.s_full[buf]));
        }
        __syncwarp();
      };
      // O' += P V of page e (pg = 0: X0) or o of tile i
      auto values = [&](int i, int pg) {
        ok = ok && wait(bars.p_full[pg], i);
        if (!ok) return;
        const int half = 2 * (i % kNB) + pg;
        if (elect_one()) {
          if (2 * i + pg < n) {
            const uint64_t vb = d_v + half * static_cast<uint64_t>(kH >> 4);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t acc = (i > 0 || pg > 0 || k > 0) ? 1u : 0u;
                if (kFp8) {  // two steps of 32 tokens, P's two parts
                  const int step = k >> 1, part = k & 1;
                  mma2_ss_f8(tmem + kTmemO + 128 * h, d_p + part * kC + 2 * (2 * pg + step), vb + h * kC + 256 * step,
                             idesc_o | (part == 0 ? kE5m2A : 0u), acc);
                } else {  // four steps of 16 tokens
                  mma2_ss(tmem + kTmemO + 128 * h, d_p + pg * kC + 2 * k, vb + h * 2 * kC + 128 * k, idesc_o, acc);
                }
              }
          }
          commit2(smem_u32(&bars.x_empty[half]));
        }
        __syncwarp();
      };
      if (warp == kScoresMmaWarp) {
        for (int i = 0; i < tiles && ok; ++i)
          for (int h = 0; h < 2; ++h) scores(i, h);
      } else {
        for (int i = 0; i < tiles && ok; ++i)
          for (int pg = 0; pg < 2; ++pg) values(i, pg);
      }
      // no MMA of the pair may still be running when tensor memory is released
      if (elect_one())
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(smem_u32(&bars.drain))
                     : "memory");
      __syncwarp();
      mbar_wait(smem_u32(&bars.drain), 0, p.status, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // Thread (r, hf, ch): head 64 rank + r; tokens [32 ch, 32 ch + 32) of page e (hf = 0) or o of
    // every tile; latent columns [256 hf + 128 ch, + 128) of O'.  Four threads share a row.
    const int hf = (warp & 3) >> 1, ch = warp >> 2, r = (warp & 1) * 32 + lane, quarter = 2 * hf + ch;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lane_off + kTmemO + 128 * ch;
    float* hx = reinterpret_cast<float*>(smem + kOffHx) + r;  // the row's slots, 64 apart
    const int slot = quarter * kRows;
    const float4* sc = reinterpret_cast<const float4*>(smem + kOffScale) + 8 * quarter;
    float* logs = reinterpret_cast<float*>(smem + kOffLog2) + 32 * warp;  // (the warp's 32 tokens are the same in all its rows)
    const uint32_t s_free = mapa(smem_u32(&bars.s_free[0]), 0), p_full = mapa(smem_u32(&bars.p_full[0]), 0);
    float score_log2 = kScaleLog2;  // a score's factor, in exponents of 2
    float rot_factor = 1.f;         // FP8: and that of its RoPE part, to the latent part's units
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (kFp8 && tiles > 0) {
      // The query in place: the latent columns times 2^a as two E4M3 parts, the RoPE columns times 2^ar as
      // f16, with the row's a bringing its largest latent value into [128, 256) and its ar the largest RoPE
      // value into [2^14, 2^15).  Their scores meet in the softmax.  (Latent values 2^60 below the RoPE ones are
      // given up, so that the factor between the two stays in range.)  This thread takes bf16 chunks 2 quarter
      // and 2 quarter + 1 and 16 RoPE columns.
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.q_land), 0, p.status, abort));
      uint8_t* q = smem + kOffQ + r * 128;
      auto unit = [&](int chunk, int u) { return reinterpret_cast<uint4*>(q + chunk * kChunk + ((u ^ (r & 7)) << 4)); };
      uint4 lat[16], rot[2];
      uint32_t top_lat = 0, top_rot = 0;  // largest |x| as bf16 bits, both halves of a word
      auto top = [](uint32_t t, const uint4& x) {
        t = __vmaxu2(__vmaxu2(t, x.x & 0x7fff7fffu), __vmaxu2(x.y & 0x7fff7fffu, x.z & 0x7fff7fffu));
        return __vmaxu2(t, x.w & 0x7fff7fffu);
      };
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        lat[u] = *unit(2 * quarter + (u >> 3), u & 7);
        top_lat = top(top_lat, lat[u]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        rot[u] = *unit(8, 2 * quarter + u);
        top_rot = top(top_rot, rot[u]);
      }
      top_lat = max(top_lat & 0xffffu, top_lat >> 16);
      top_rot = max(top_rot & 0xffffu, top_rot >> 16);
      hx[slot] = __uint_as_float(top_lat << 16 | top_rot);
      named_barrier_sync(1, kSoftThreads);  // every thread holds its part, too
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t t = __float_as_uint(hx[k * kRows]);
        top_lat = max(top_lat, t >> 16);
        top_rot = max(top_rot, t & 0xffffu);
      }
      const int e_lat = static_cast<int>(top_lat >> 7) - 127, e_rot = static_cast<int>(top_rot >> 7) - 127;
      const int ar = min(100, 14 - e_rot), a = min(min(100, 7 - e_lat), ar + 60);
      auto power = [](int e) { return __uint_as_float(static_cast<uint32_t>(127 + max(-126, e)) << 23); };
      const float up = power(a), up_rot = power(ar);
      score_log2 *= power(-a);
      rot_factor = power(a - ar);
      if (e_lat == 128 || e_rot == 128) score_log2 = NAN;  // an infinity or a NaN (E4M3 would saturate)
#pragma unroll
      for (int u = 0; u < 8; ++u) {  // 16 columns: two units of bf16 in, one of each part out
        const uint32_t w[8] = {lat[2 * u].x,     lat[2 * u].y,     lat[2 * u].z,     lat[2 * u].w,
                               lat[2 * u + 1].x, lat[2 * u + 1].y, lat[2 * u + 1].z, lat[2 * u + 1].w};
        uint32_t o1[4], o2[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint16_t a1, a2, b1, b2;
          split_e4m3(bf16x2_to_f16x2(w[2 * k], up), a1, a2);
          split_e4m3(bf16x2_to_f16x2(w[2 * k + 1], up), b1, b2);
          o1[k] = a1 | static_cast<uint32_t>(b1) << 16;
          o2[k] = a2 | static_cast<uint32_t>(b2) << 16;
        }
        *unit(quarter, u) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
        *unit(4 + quarter, u) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        *unit(8, 2 * quarter + u) = make_uint4(bf16x2_to_f16x2(rot[u].x, up_rot), bf16x2_to_f16x2(rot[u].y, up_rot),
                                               bf16x2_to_f16x2(rot[u].z, up_rot), bf16x2_to_f16x2(rot[u].w, up_rot));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_pair(mapa(smem_u32(&bars.q_full), 0));
      named_barrier_sync(1, kSoftThreads);  // hx has been read
    }
    const uint64_t scale2 = f32x2(score_log2, score_log2), rot2 = f32x2(rot_factor, rot_factor);
    for (int i = 0; i < tiles; ++i) {
      const int buf = i & 1;
      const bool there = 2 * i + hf < n;  // the tile has this thread's page
      const uint64_t word = there ? view_bits(v, view_page(v, k0 + 2 * i + hf)) : 0ull;
      const uint32_t w = static_cast<uint32_t>(word >> (32 * ch));
      float2 st[16];  // FP8: the tokens' scales
      if (kFp8) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.sc_full[buf]), (i >> 1) & 1, p.status, abort)) && ok;
        // log2 of the scales, a lane's token each (one nobody sees: its score is -inf, whatever its scale).  They set
        // the reference alone, so the hardware's 2^-22 will do; log2f took a tile 200 cycles (this 40 to 140).  A scale
        // of 0 leaves a token its part of the sum, and the reference finite: 2^-96 keeps that sum in range.
        const float s = reinterpret_cast<const float*>(sc)[buf * 2 * kPage + lane];
        logs[lane] = (w >> lane & 1u) != 0 ? fmaxf(__log2f(s), -96.f) : 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 f = sc[buf * 2 * kPage / 4 + c];
          st[2 * c] = make_float2(f.x, f.y);
          st[2 * c + 1] = make_float2(f.z, f.w);
        }
        if (w != ~0u) {  // the scale of a token nobody sees may be anything
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (!(w >> (2 * c) & 1u)) st[c].x = 0.f;
            if (!(w >> (2 * c + 1) & 1u)) st[c].y = 0.f;
          }
        }
        __syncwarp();
      }
      ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&bars.s_full[buf]), (i >> 1) & 1, p.status, abort)) && ok;
      tc_fence_after();
      float sv[32];
      {
        uint32_t a[32];
        tmem_ld32(tmem + lane_off + kTmemS + 64 * buf + 32 * ch, a);
        if (kFp8) {
          uint32_t rot[32];
          tmem_ld32(tmem + lane_off + kTmemR + 64 * buf + 32 * ch, rot);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 f = f32x2_split(fma_f32x2(f32x2(__uint_as_float(rot[c]), __uint_as_float(rot[c + 1])), rot2,
                                                   f32x2(__uint_as_float(a[c]), __uint_as_float(a[c + 1]))));
            sv[c] = f.x;
            sv[c + 1] = f.y;
          }
        } else {
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) sv[c] = __uint_as_float(a[c]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_pair(s_free + 8 * buf);
      if (kFp8) {  // the MMAs ran on codes: the scores carry 1 / s_t
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 f = f32x2_split(mul_f32x2(f32x2(sv[2 * c], sv[2 * c + 1]), f32x2(st[c].x, st[c].y)));
          sv[2 * c] = f.x;
          sv[2 * c + 1] = f.y;
        }
      }
      if (w != ~0u) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (!(w >> c & 1u)) sv[c] = -INFINITY;
      }
      float m8[8];
      if (kFp8) {
        // of weight times scale, token by token: a large scale under a low score must not lift it (a bound of
        // the largest score plus the largest scale did, and pushed every real weight out of E4M3's range)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 f = reinterpret_cast<const float4*>(logs)[c];
          const float2 x = f32x2_split(fma_f32x2(f32x2(sv[4 * c], sv[4 * c + 1]), scale2, f32x2(f.x, f.y)));
          const float2 y = f32x2_split(fma_f32x2(f32x2(sv[4 * c + 2], sv[4 * c + 3]), scale2, f32x2(f.z, f.w)));
          m8[c] = fmaxf(fmaxf(x.x, x.y), fmaxf(y.x, y.y));
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) m8[c] = fmaxf(fmaxf(sv[c], sv[c + 8]), fmaxf(sv[c + 16], sv[c + 24]));
      }
      const float top = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                              fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
      // The row's maximum over its four threads, in exponents of 2; FP8: of weight times scale, which is
      // what P holds.  The slots are written again behind the next tile's barrier.
      float* hb = hx + buf * 4 * kRows;
      hb[slot] = kFp8 ? top : top * score_log2;
      ok = named_barrier_and(1, kSoftThreads, ok);  // the warps leave together
      if (!ok) break;
      const float mx = fmaxf(fmaxf(hb[0], hb[kRows]), fmaxf(hb[2 * kRows], hb[3 * kRows]));
      float factor = 1.f;
      bool rescale = false;
      if (m == -INFINITY) {
        m = mx;
      } else if (mx > m + kRescaleLog2<kFp8>) {
        factor = ex2_approx(m - mx);
        m = mx;
        rescale = true;
      }
      const float neg_m = kPUpLog2<kFp8> - (m == -INFINITY ? 0.f : m);
      const uint64_t neg2 = f32x2(neg_m, neg_m);
      uint32_t pk[16];
      uint64_t s2[2] = {0ull, 0ull};
      uint16_t half1 = 0, half2 = 0;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float2 e = f32x2_split(fma_f32x2(f32x2(sv[2 * c], sv[2 * c + 1]), scale2, neg2));
        const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
        s2[c & 1] = add_f32x2(s2[c & 1], f32x2(p0, p1));
        if (kFp8) {  // words c / 2 of both parts; P carries s_t, the row sum does not
          uint16_t x1, x2;
          const float2 y = f32x2_split(mul_f32x2(f32x2(p0, p1), f32x2(st[c].x, st[c].y)));
          split_e5m2(pack_f16x2(y.x, y.y), x1, x2);
          if (c & 1) {
            pk[c >> 1] = half1 | static_cast<uint32_t>(x1) << 16;
            pk[8 + (c >> 1)] = half2 | static_cast<uint32_t>(x2) << 16;
          } else {
            half1 = x1;
            half2 = x2;
          }
        } else {
          pk[c] = pack_bf16x2(p0, p1);
        }
      }
      const float2 s1 = f32x2_split(add_f32x2(s2[0], s2[1]));
      l = l * factor + (s1.x + s1.y);
      // O'(i - 1) has read this page's P; to be rescaled it has to be complete
      const bool any = __any_sync(0xffffffffu, rescale);
      if (i > 0) {
        ok = __all_sync(0xffffffffu, passed(bars.x_empty[2 * ((i - 1) % kNB) + (any ? 1 : hf)], (i - 1) / kNB));
        tc_fence_after();
      }
      if (any && ok) {
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t x[32];
          tmem_ld32(o_addr + c0, x);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * factor);
          tmem_st32(o_addr + c0, x);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      if (hf == 1) {
        __syncwarp();
        if (lane == 0) arrive_pair(p_full);
      }
      // four units of 8 tokens in page hf's chunk, or two units of 16 in each part's
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int chunk = kFp8 ? c >> 1 : hf, u = kFp8 ? 2 * quarter + (c & 1) : 4 * ch + c;
        *reinterpret_cast<uint4*>(smem + kOffP + chunk * kChunk + r * 128 + ((u ^ (r & 7)) << 4)) =
            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
      }
      // this page's values are in place (in the other half of the pair's buffer they came as its keys)
      if (hf != static_cast<int>(rank))
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.v_full[i % kNB]), (i / kNB) & 1, p.status, abort)) && ok;
      // a value row nobody sees may hold anything (NaN in slots never written): 0 * NaN would reach O'
      if (there && word != ~0ull) {
        uint8_t* half = smem + kOffX + (2 * (i % kNB) + hf) * kH;
#pragma unroll 1
        for (int u = ch * kRows + r; u < kH / 16; u += 2 * kRows)
          if (!(word >> ((u >> 3) & 63) & 1ull)) *reinterpret_cast<uint4*>(half + u * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_pair(p_full + 8 * hf);
    }
    // the row's sum, then O' / l
    const int64_t out_row = (bj * p.num_splits + split) * kHeads + kRows * rank + r;
    if (tiles > 0) {
      ok = ok && passed(bars.x_empty[2 * ((tiles - 1) % kNB) + 1], (tiles - 1) / kNB);
      ok = named_barrier_and(1, kSoftThreads, ok);
      tc_fence_after();
      float* hb = hx + (tiles & 1) * 4 * kRows;
      hb[slot] = l;
      named_barrier_sync(1, kSoftThreads);
      l = (hb[0] + hb[kRows]) + (hb[2 * kRows] + hb[3 * kRows]);
    }
    const bool some = ok && tiles > 0 && l != 0.f;
    const float inv = some ? 1.f / l : 0.f;
    if (slot == 0 && p.lse_out != nullptr) {
      float lse = some ? (m - kPUpLog2<kFp8> + log2f(l)) * kLn2 : -INFINITY;
      // a visible NaN: the merge leaves out a split whose weight is NaN, but not one that makes all of them 0 / 0
      if (p.num_splits > 1 && lse != lse) lse = INFINITY;
      p.lse_out[out_row] = lse;
    }
    // Each thread's columns leave by way of shared memory, where no tile is any more, in copies of 256 bytes: 5,750
    // cycles a CTA, of which 4,300 are the 128 KB on their way out (stores of sectors from registers: 7,900).  The
    // pitch spreads a warp's rows over the banks.
    float* mine = reinterpret_cast<float*>(smem + kOffX + r * kOutPitch) + 256 * hf + 128 * ch;
    if (ok) {
#pragma unroll 1
      for (int c0 = 0; c0 < 128; c0 += 32) {
        uint32_t x[32];
        if (tiles > 0) {
          tmem_ld32(o_addr + c0, x);
          tmem_wait_ld();
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = some ? __float_as_uint(__uint_as_float(x[c]) * inv) : 0u;
#pragma unroll
        for (int c = 0; c < 32; c += 4)
          *reinterpret_cast<uint4*>(mine + c0 + c) = make_uint4(x[c], x[c + 1], x[c + 2], x[c + 3]);
        if (c0 & 32) {
          fence_proxy_async_smem();
          bulk_store(p.o_out + out_row * kLatent + 256 * hf + 128 * ch + c0 - 32, smem_u32(mine + c0 - 32), 256);
          bulk_commit_group();
        }
      }
      bulk_wait_read<0>();  // (the writes themselves are complete at the kernel's end)
    }
  }
  if (*abort) let_work_land();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's MMAs have finished, and nobody addresses the other CTA any more
  if (warp == kScoresMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  cluster_sync();
}

bool g_configured[kMaxDevicesLocal];
int g_slots[kMaxDevicesLocal];

bool configure(int dev) {
  if (dev < 0) return false;
  if (!g_configured[dev]) {
    if (cudaFuncSetAttribute(decode_masked_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(decode_masked_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
            cudaSuccess)
      return false;
    g_configured[dev] = true;
  }
  return true;
}

}  // namespace

int masked_cluster_slots() {
  const int dev = current_device_index();
  if (dev < 0) return 74;
  if (g_slots[dev] > 0) return g_slots[dev];
  int n = 0;
  if (configure(dev)) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, decode_masked_kernel<false>, &cfg) != cudaSuccess) n = 0;
  }
  if (n <= 0) {
    cudaGetLastError();
    int sms = 148;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    n = sms / 2;
  }
  g_slots[dev] = n;
  return n;
}

cudaError_t launch_decode_masked(const MaskedArgs& a, const SplitPlan& plan, float* o_out, float* lse_out, int* status,
                                 cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.B) * a.n_q * plan.num_splits;
  if (units == 0) return cudaSuccess;
  if (!configure(current_device_index())) return cudaErrorInvalidDevice;
  const bool fp8 = a.cache == nullptr;
  const uint64_t rows = static_cast<uint64_t>(a.num_pages) * kPage;
  CUtensorMap tq, tc, tr;
  if (!make_tmap_bf16_chunks(&tq, a.q_abs, static_cast<uint64_t>(a.B) * a.n_q * kHeads, kRow, kRows, 3) ||
      // an FP8 cache's f16 keys move as 16-bit values: the bytes alone count
      !make_tmap_bf16_chunks(&tr, fp8 ? a.kr : a.cache, rows, fp8 ? kRope : kRow, kPage, 1) ||
      !(fp8 ? make_tmap_u8_chunks(&tc, a.c8, rows, kLatent, kPage, 2) : make_tmap_bf16_chunks(&tc, a.cache, rows, kRow, kPage, 4)))
    return cudaErrorInvalidValue;
  Params prm;
  prm.c8 = a.c8;
  prm.scale = a.scale;
  prm.page_table = a.page_table;
  prm.kv_lens = a.kv_lens;
  prm.words = a.words;
  prm.depths = a.depths;
  prm.o_out = o_out;
  prm.lse_out = lse_out;
  prm.status = status;
  prm.num_pages = a.num_pages;
  prm.pt_stride = a.pt_stride;
  prm.n_q = a.n_q;
  prm.max_kv_len = a.max_kv_len;
  prm.window = a.window;
  prm.sinks = a.sinks;
  prm.split_pages = plan.split_pages;
  prm.num_splits = plan.num_splits;
  prm.max_pages = plan.max_pages;
  const int64_t splits = static_cast<int64_t>(a.B) * plan.num_splits;
  prm.longest_first = a.B > 1 && splits <= kMostSorted && units > masked_cluster_slots() ? static_cast<int>(splits) : 0;
  const dim3 grid(static_cast<unsigned>(2 * units));
  return fp8 ? launch_kernel(decode_masked_kernel<true>, grid, dim3(kThreads), kSmemBytes, stream, tq, tc, tr, prm)
             : launch_kernel(decode_masked_kernel<false>, grid, dim3(kThreads), kSmemBytes, stream, tq, tc, tr, prm);
}

}  // namespace mla
