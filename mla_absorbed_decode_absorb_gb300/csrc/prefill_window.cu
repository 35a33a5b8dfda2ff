// Non-absorbed attention of a chunk of new tokens whose queries see a window and the
// first tokens (sinks): softmax([q^C ; RoPE(q^R)] . [k^C ; k^R] / sqrt(192)) V over the
// decompressed keys and values, query j at position p = seq_lens_before + j over the
// tokens i <= p with i > p - window or i < sinks.
//
// What bounds it.  A tile of 128 queries and 128 keys is 128 x 128 x (192 + 128)
// multiply-adds, 1,280 cycles of the tensor cores, and its softmax about 1,550.  So the
// products have to run while a softmax does: a CTA works on two query tiles at once,
// neighbours of one head that share the key tiles, each with its own softmax warps and its
// own issuing warp.  The two take turns at the tensor cores: without turns both sets of
// products end at the same time, then both softmaxes run, and neither product does (5,500
// cycles for a pair of tiles instead of 4,600).  Both take a key tile from L2 once.
// Prompts of 4 x 4096 tokens over a window of 1024 take 1210 us here; one query tile at a
// time (the causal kernel's form with the window's mask) took 1781 us, 2 x 512 tokens behind
// 16384 over 2048 take 171 and 191 us.  A pair of tiles takes 4,200 cycles now, of which the
// products are 2,560: the loads of a key tile wait for places in the ring.
//
// One CTA per SM walks units (sequence, head, 256 queries) in head order, so that the
// heads in flight keep their keys and values in L2; every other head is walked backwards,
// so that a CTA's units are not all early or all late ones.  Warps 0-3 and 4-7: softmax of
// the first and second query tile, one thread a row, which holds the row's maximum and sum
// by itself.  Warp 8 loads, warp 9 works out the units for all the others, warps 10 and 11
// issue the two tiles' products, and warps 12-15 bring in RoPE(q^R) of the next unit and
// take O out, so that the softmax goes on with the next unit.  Keys and values go through
// one ring of eight 16 KB chunks in the order in which they are needed: of a key tile three
// chunks of 64 columns (the third the cache's RoPE keys), then two chunks of 64 values'
// rows.  A chunk is free again once both query tiles are done with it, so a key tile that
// only one of them sees is passed by the other without a product.
//
// Code size counts: the roles run side by side, and with every wait and each role's unit
// arithmetic inlined (186 KB) a product took 260 cycles to issue instead of 64.  So the
// units are worked out once, waits are short, and the softmax reads S in rolled loops.
//
// TMEM: two O (128 columns each) and two S (128 each).  P (bf16, 64 columns) takes the place
// of its S, in halves of 64 keys; one thread issues P V of a tile and then Q K^T of the
// next, which may overwrite P behind it.
#include "sm100.cuh"
#include "tmap.cuh"
#include "view.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kTile = 128;                 // queries and keys of a tile
constexpr int kThreads = 512;
constexpr int kLoadWarp = 8;
constexpr int kUnitWarp = 9;
constexpr int kMmaWarp = 10;               // and 11
constexpr int kEndsWarp = 12;              // to 15
constexpr int kGroup = 128;                // softmax threads of a query tile
constexpr int kChunk = 128 * 128;          // 128 rows x 64 bf16 columns, or two of 64 rows
constexpr int kRing = 8;
constexpr int kOffQ = 0;                   // two query tiles of three chunks (q^C, q^C, RoPE(q^R))
constexpr int kOffRing = 6 * kChunk;
constexpr int kOffBar = kOffRing + kRing * kChunk;
constexpr int kOffSum = kOffBar + 512;     // row sums [2 query tiles][128]
constexpr int kOffUnit = kOffSum + 1024;   // the next units
constexpr int kSmemBytes = kOffUnit + 256 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemO = 0, kTmemS = 256;  // of query tile g: O at 128 g, S at 256 + 128 g
constexpr int kUnits = 4;                  // units known ahead
constexpr int kReaders = 15;               // warps that read them
constexpr float kRescaleLog2 = 8.f;

struct Bars {
  uint64_t full[kRing];
  uint64_t empty[kRing];   // both issuers are done with the chunk
  // per query tile
  uint64_t q_full[2];      // q^C has landed
  uint64_t q_ready[2];     // RoPE(q^R) is in shared memory
  uint64_t q_free[2];      // the unit's last Q K^T has read the query
  uint64_t s_full[2];
  uint64_t p_full[2][2];   // halves of P (and S has been read)
  uint64_t o_full[2];
  uint64_t sum_full[2];    // the rows' sums are in shared memory
  uint64_t o_free[2];      // the epilogue has read O
  uint64_t turn[2];        // the query tile's turn at the tensor cores
  uint64_t unit_full[kUnits];
  uint64_t unit_empty[kUnits];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

struct Params {
  const uint16_t* q_nope;
  const uint16_t* q_rope;
  const int32_t* seq_lens_before;
  const float* rope;
  const int32_t* page_table;
  const int32_t* kv_lens;
  uint16_t* out;
  float* lse;
  int* status;
  int64_t num_pages;
  int n_units;      // B heads n_pair
  int n_pair;       // units of a head
  int pt_stride;
  int rope_max_pos;
  int max_kv_len;
  int n_q;
  int B;
  int window;
  int sinks;
};

// Two query tiles of a head and the key tiles that they see: the g-th one's are [0, ns[g]) and [w0[g], end[g])
// (end 0: no such query tile).  The unit's are the first one's from its oldest on, up to the last one's end, n in
// all (sinks that only the second sees are in the first's window); n 0: there are no more units.
struct Unit {
  int b, h, L, kv, j0;
  int n;
  int ns[2], w0[2], end[2];
  __device__ __forceinline__ int tile(int k) const { return k < ns[0] ? k : k - ns[0] + w0[0]; }
  __device__ __forceinline__ bool sees(int g, int x) const { return x < ns[g] || (x >= w0[g] && x < end[g]); }
};
static_assert(kUnits * sizeof(Unit) <= 256, "units");

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void prefetch_l2(const void* ptr) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(ptr)));
}

__global__ void __launch_bounds__(kThreads, 1)
prefill_window_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_q,
                      const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + kOffBar);
  float* sums = reinterpret_cast<float*>(smem + kOffSum);
  Unit* units = reinterpret_cast<Unit*>(smem + kOffUnit);
  volatile int* abort = &bars.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int c = 0; c < kRing; ++c) {
      mbar_init(smem_u32(&bars.full[c]), 1);
      mbar_init(smem_u32(&bars.empty[c]), 2);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_u32(&bars.q_full[g]), 1);
      mbar_init(smem_u32(&bars.q_ready[g]), kGroup);
      mbar_init(smem_u32(&bars.q_free[g]), 1);
      mbar_init(smem_u32(&bars.s_full[g]), 1);
      for (int h = 0; h < 2; ++h) mbar_init(smem_u32(&bars.p_full[g][h]), kGroup);
      mbar_init(smem_u32(&bars.o_full[g]), 1);
      mbar_init(smem_u32(&bars.sum_full[g]), kGroup);
      mbar_init(smem_u32(&bars.o_free[g]), kGroup);
      mbar_init(smem_u32(&bars.turn[g]), 1);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_u32(&bars.unit_full[i]), 1);
      mbar_init(smem_u32(&bars.unit_empty[i]), kReaders);
    }
    mbar_init(smem_u32(&bars.drain), 2);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kLoadWarp) {
    tmem_alloc(smem_u32(&bars.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  grid_dep_wait();
  grid_dep_launch();

  auto warp_wait = [&](uint64_t& bar, int phase) {
    return __all_sync(0xffffffffu, mbar_wait_short(smem_u32(&bar), phase & 1, p.status, abort)) != 0;
  };
  // the CTA's i-th unit, and (every reader's lane 0) done with it
  auto unit_there = [&](int i) { return warp_wait(bars.unit_full[i % kUnits], i / kUnits); };
  auto unit_done = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.unit_empty[i % kUnits]));
  };

  if (warp == kUnitWarp) {
    // ------------------------------------------------------------ units
    int i = 0;
    bool ok = true;
    // Units of a last round that at most half the CTAs have are cut in two, a query tile each.  (2 x 512 tokens behind
    // 16384: 512 units on 152 SMs, 169 us whole, 166 so.)
    const int rest = p.n_units % static_cast<int>(gridDim.x);
    const int whole = 2 * rest <= static_cast<int>(gridDim.x) ? p.n_units - rest : p.n_units;
    const int64_t end = whole + 2 * static_cast<int64_t>(p.n_units - whole);
#pragma unroll 1
    for (int64_t wide = blockIdx.x; ok; wide += gridDim.x) {
      Unit u{};
      if (wide < end) {
        const bool cut = wide >= whole;
        const int w = static_cast<int>(cut ? whole + (wide - whole) / 2 : wide), bh = w / p.n_pair, x = w - bh * p.n_pair;
        u.b = bh / kHeads;
        u.h = bh % kHeads;
        u.j0 = (bh & 1 ? p.n_pair - 1 - x : x) * 2 * kTile + (cut && ((wide - whole) & 1) ? kTile : 0);
        if (u.j0 >= p.n_q) continue;
        const int j1 = min(p.n_q, u.j0 + (cut ? 1 : 2) * kTile);  // behind its last query
        u.L = p.seq_lens_before[u.b];
        u.kv = p.kv_lens[u.b];
        if (u.kv < p.n_q || u.kv - p.n_q != u.L || u.kv > p.max_kv_len || pages_of(u.kv) > p.pt_stride ||
            u.kv > p.rope_max_pos) {
          // an invalid sequence: O = 0 and lse = -inf.  (L + n_q may wrap, onto a kv that did; kv - n_q may not here.)
          if (lane == 0) record_status(p.status, MLA_ERR_BOUNDS);
#pragma unroll 1
          for (int j = u.j0; j < j1; ++j) {
            const int64_t row = (static_cast<int64_t>(u.b) * p.n_q + j) * kHeads + u.h;
            if (lane < kNope / 8) *reinterpret_cast<uint4*>(p.out + row * kNope + 8 * lane) = make_uint4(0, 0, 0, 0);
            if (lane == 0 && p.lse != nullptr) p.lse[row] = -INFINITY;
          }
          continue;
        }
        for (int g = 0; g < 2; ++g) {
          const int j0 = u.j0 + kTile * g, lo = max(0, u.L + j0 - p.window + 1);
          if (j0 >= j1) break;
          u.w0[g] = lo / kTile;
          u.ns[g] = min((min(p.sinks, lo) + kTile - 1) / kTile, u.w0[g]);
          u.end[g] = (u.L + min(p.n_q, j0 + kTile) - 1) / kTile + 1;
        }
        u.n = u.ns[0] + max(u.end[0], u.end[1]) - u.w0[0];
      }
      ok = warp_wait(bars.unit_empty[i % kUnits], i / kUnits + 1);
      if (!ok) break;
      if (lane == 0) {
        units[i % kUnits] = u;
        mbar_arrive(smem_u32(&bars.unit_full[i % kUnits]));
      }
      __syncwarp();
      ++i;
      if (u.n == 0) break;
    }
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loads
    int c = 0;  // chunks so far
    bool ok = true;
#pragma unroll 1
    for (int i = 0; ok && unit_there(i); ++i) {
      const Unit& u = units[i % kUnits];
      const int n = u.n;
      if (n == 0) break;
      const int32_t* pt = p.page_table + static_cast<int64_t>(u.b) * p.pt_stride;
      const int n_pg = (u.kv + kPage - 1) / kPage;  // pages that hold the sequence (<= pt_stride)
      const int bh = u.b * kHeads + u.h, lo = max(0, u.L + u.j0 - p.window + 1);
      int ids = 0;
#pragma unroll 1
      for (int kt = 0; kt < n && ok; ++kt) {
        if ((kt & 15) == 0) {  // the page ids of 16 key tiles, one a lane
          const int q = 2 * u.tile(kt + (lane >> 1)) + (lane & 1);
          ids = q < n_pg ? pt[q] : 0;
        }
        const int t0 = u.tile(kt) * kTile;
#pragma unroll 1
        for (int x = 0; x < 5; ++x, ++c) {
          const int s = c % kRing;
          ok = warp_wait(bars.empty[s], c / kRing + 1);
          const uint32_t dst = smem_u32(smem + kOffRing + s * kChunk), bar = smem_u32(&bars.full[s]);
          int page = __shfl_sync(0xffffffffu, ids, (2 * kt + (lane & 1)) & 31);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar, kChunk);
          __syncwarp();
          if (x < 2) {
            if (lane == 0) tma_load_3d(dst, &tm_k, 64 * x, t0, bh, bar);
          } else if (lane < 2) {  // halves, a lane each
            if (x == 2) {
              const int tok = t0 + lane * kPage;
              if (tok >= u.kv || (tok + kPage <= lo && tok >= p.sinks)) {
                page = 0;  // past the sequence, or no token visible: masked, any page will do
              } else if (page < 0 || page >= p.num_pages) {
                record_status(p.status, MLA_ERR_BOUNDS);
                page = 0;  // stay in bounds; the result is not meaningful
              }
              tma_load_2d(dst + lane * (kChunk / 2), &tm_kr, kLatent, page * kPage, bar);
            } else {
              tma_load_3d(dst + lane * (kChunk / 2), &tm_v, 64 * lane, t0 + 64 * (x - 3), bh, bar);
            }
          }
          __syncwarp();
        }
      }
      unit_done(i);
    }
    // no copy may still be under way when the CTA ends
    for (int x = max(0, c - kRing); x < c; ++x)
      mbar_wait_short(smem_u32(&bars.full[x % kRing]), (x / kRing) & 1, p.status, nullptr);
  } else if (warp >= kMmaWarp && warp < kEndsWarp) {
    // ------------------------------------------------------------ products of query tile g
    const int g = warp - kMmaWarp;
    const uint32_t idesc_qk = idesc_bf16(128, 128, /*a_mn=*/0, /*b_mn=*/0);
    const uint32_t idesc_pv = idesc_bf16(128, 128, /*a_mn=*/0, /*b_mn=*/1);
    const uint64_t d_q = smem_desc(smem_u32(smem + kOffQ + 3 * g * kChunk), 16, 1024, kSw128);
    const uint64_t d_k = smem_desc(smem_u32(smem + kOffRing), 16, 1024, kSw128);
    const uint64_t d_v = smem_desc(smem_u32(smem + kOffRing), kChunk / 2, 1024, kSw128);
    const uint32_t tm_o = tmem + kTmemO + kTile * g, tm_s = tmem + kTmemS + kTile * g;
    bool ok = true;
    int c = 0;            // chunks done with
    int t = 0, done = 0;  // key tiles and units of this query tile's so far
    int step = 0;         // steps of the units so far
    int queries = 0;      // loads of q^C so far
    auto load_q = [&](int i) {  // q^C of the i-th unit, if it has this query tile
      ok = ok && unit_there(i);
      const Unit& u = units[i % kUnits];
      if (!ok || u.end[g] == 0) return;
      ++queries;
      if (elect_one()) {
        const uint32_t bar = smem_u32(&bars.q_full[g]);
        mbar_arrive_expect_tx(bar, 2 * kChunk);
        for (int x = 0; x < 2; ++x)
          tma_load_3d(smem_u32(smem + kOffQ + (3 * g + x) * kChunk), &tm_q, 64 * x, u.h, u.b * p.n_q + u.j0 + kTile * g, bar);
      }
      __syncwarp();
    };
    auto chunk_there = [&](int x) { ok = ok && warp_wait(bars.full[x % kRing], x / kRing); };
    load_q(0);
#pragma unroll 1
    for (int i = 0; ok; ++i) {
      const Unit& u = units[i % kUnits];  // load_q has waited for it
      const int n = u.n;
      if (n == 0) break;
      const int last = u.end[g] - 1;
      bool first = true;
      if (last >= 0) ok = warp_wait(bars.q_full[g], done) && warp_wait(bars.q_ready[g], done);
      // Steps of the unit: k = -1 (no values), then its key tiles; P V of tile k goes out with Q K^T of the next,
      // whose keys may arrive meanwhile (their places are free: those of tiles before this step's turn).  A tile that
      // the other query tile alone sees is passed by: its keys only behind P V, since their places may be those of
      // values that wait for it.
      auto pass = [&](int x) {
        if (lane == 0) mbar_arrive(smem_u32(&bars.empty[x % kRing]));
      };
#pragma unroll 1
      for (int k = -1; k < n && ok; ++k) {
        const bool pv = k >= 0 && u.sees(g, u.tile(k)), qk = k + 1 < n && u.sees(g, u.tile(k + 1));
        const bool end = pv && u.tile(k) == last, qk_end = qk && u.tile(k + 1) == last;
        const int v = k < 0 ? 0 : 2, keys = k + 1 < n ? 3 : 0;  // chunks of the step
#pragma unroll 1
        for (int x = 0; x < v; ++x) {
          chunk_there(c + x);
          if (ok && !pv) pass(c + x);
        }
        if (pv && first && done > 0) ok = ok && warp_wait(bars.o_free[g], done - 1);  // P V overwrites O
        if (pv) ok = ok && warp_wait(bars.p_full[g][0], t);
        // The two query tiles take turns, step by step: products of both at once would end at the same time, and
        // then both softmaxes run at the same time, and neither product does.  (A unit's last step out of turn, so
        // that the other query tile can begin with the next unit: 1235 us instead of 1210 at 4 x 4096 tokens.)
        ok = ok && warp_wait(bars.turn[g], step + 1 - g);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = __reduce_max_sync(0xffffffffu, static_cast<unsigned>(c));  // in a uniform register
        auto slot = [&](int x) { return (at + x) % kRing; };
        if (pv) {
          if (elect_one()) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              mma_ts(tm_o, tm_s + 8 * y, d_v + slot(0) * (kChunk >> 4) + 128 * y, idesc_pv, (!first || y > 0) ? 1u : 0u);
          }
          __syncwarp();
          ok = warp_wait(bars.p_full[g][1], t);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              mma_ts(tm_o, tm_s + 32 + 8 * y, d_v + slot(1) * (kChunk >> 4) + 128 * y, idesc_pv, 1u);
            mma_commit(smem_u32(&bars.empty[slot(0)]));
            mma_commit(smem_u32(&bars.empty[slot(1)]));
            if (end) mma_commit(smem_u32(&bars.o_full[g]));
          }
          __syncwarp();
          first = false;
          ++t;
        }
        if (qk) {
#pragma unroll
          for (int x = 0; x < 3; ++x) {
            chunk_there(c + v + x);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t a = d_q + x * (kChunk >> 4), b = d_k + slot(v + x) * (kChunk >> 4);
#pragma unroll
              for (int y = 0; y < 4; ++y) mma_ss(tm_s, a + 2 * y, b + 2 * y, idesc_qk, (x > 0 || y > 0) ? 1u : 0u);
              if (x == 2) {
                mma_commit(smem_u32(&bars.s_full[g]));
#pragma unroll
                for (int y = 0; y < 3; ++y) mma_commit(smem_u32(&bars.empty[slot(v + y)]));
              }
              if (x == 2 && qk_end) mma_commit(smem_u32(&bars.q_free[g]));
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        if (elect_one()) mbar_arrive(smem_u32(&bars.turn[g ^ 1]));
        __syncwarp();
        ++step;
        if (!qk) {
#pragma unroll 1
          for (int x = v; x < v + keys; ++x) {
            chunk_there(c + x);
            if (ok) pass(c + x);
          }
        }
        c += v + keys;
        // the unit's last scores have been read: Q K^T is done with the query
        if (end || (last < 0 && k + 1 == n)) load_q(i + 1);
      }
      if (last >= 0) ++done;
      unit_done(i);
    }
    // no copy may still be under way, and no product when TMEM is released
    if (queries > 0) mbar_wait_short(smem_u32(&bars.q_full[g]), (queries - 1) & 1, p.status, nullptr);
    if (elect_one()) mma_commit(smem_u32(&bars.drain));
    __syncwarp();
    mbar_wait(smem_u32(&bars.drain), 0, p.status, nullptr);
  } else if (warp >= kEndsWarp) {
    // ------------------------------------------------------------ both ends of a unit: RoPE(q^R) and O / l
    const int r = tid - 32 * kEndsWarp;  // row (TMEM lane)
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    int queries = 0, outs = 0;  // parities of the query tiles' counts (bit g), and
    int begun = 0;              // whether they have had one
    // RoPE(q^R) of a unit's query tile, in 16-byte units: unit v = r + 128 i is elements 8 (v % 8) .. + 7 of row v / 8
    auto rotate = [&](const Unit& u, int g) {
      const int j0 = u.j0 + kTile * g, f0 = 8 * (r & 3);
      // element f < 32 pairs with f + 32, four units (lane ^ 4) away: a cos - b sin, and a cos + b sin behind
      const uint32_t sign = (r & 4) != 0 ? 0u : 0x80000000u;
      const uint16_t* src = p.q_rope + ((static_cast<int64_t>(u.b) * p.n_q + j0) * kHeads + u.h) * kRope + 8 * (r & 7);
      const float* tab = p.rope + static_cast<int64_t>(u.L + j0) * kRope + f0;
      uint4 rot[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = min((r >> 3) + 16 * i, p.n_q - 1 - j0);  // behind the last query: its own again
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(src + rr * (kHeads * kRope)));
        const float4* row = reinterpret_cast<const float4*>(tab + rr * kRope);  // cos, then sin
        const float4 cs[4] = {__ldg(row), __ldg(row + 1), __ldg(row + kHalfRope / 4), __ldg(row + kHalfRope / 4 + 1)};
        const uint32_t mine[4] = {q.x, q.y, q.z, q.w};
        const float cc[8] = {cs[0].x, cs[0].y, cs[0].z, cs[0].w, cs[1].x, cs[1].y, cs[1].z, cs[1].w};
        const float sn[8] = {cs[2].x, cs[2].y, cs[2].z, cs[2].w, cs[3].x, cs[3].y, cs[3].z, cs[3].w};
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, mine[e], 4);
          float o[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // products rounded by themselves, as everywhere the rotation is taken
            const float a = __uint_as_float(y ? mine[e] & 0xffff0000u : mine[e] << 16);
            const float b = __uint_as_float((y ? other & 0xffff0000u : other << 16) ^ sign);
            o[y] = __fadd_rn(__fmul_rn(a, cc[2 * e + y]), __fmul_rn(b, sn[2 * e + y]));
          }
          w[e] = pack_bf16x2(o[0], o[1]);
        }
        rot[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (begun >> g & 1) ok = warp_wait(bars.q_free[g], (queries >> g) ^ 1);
      uint8_t* qs = smem + kOffQ + (3 * g + 2) * kChunk + sw128((r >> 3) * 128 + (r & 7) * 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(qs + 2048 * i) = rot[i];
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&bars.q_ready[g]));
      queries ^= 1 << g;
      begun |= 1 << g;
    };
    // rows of a query tile and their cos / sin pulled into L2 ahead
    auto prefetch = [&](const Unit& u, int g) {
      const int j = u.j0 + kTile * g + r;
      if (j >= p.n_q) return;
      const int64_t row = (static_cast<int64_t>(u.b) * p.n_q + j) * kHeads + u.h;
      prefetch_l2(p.q_nope + row * kNope);
      prefetch_l2(p.q_nope + row * kNope + 64);
      prefetch_l2(p.q_rope + row * kRope);
      prefetch_l2(p.rope + static_cast<int64_t>(u.L + j) * kRope);
      prefetch_l2(p.rope + static_cast<int64_t>(u.L + j) * kRope + 32);
    };
    // Queries of unit i + 1 go in while unit i runs, then its O comes out.
#pragma unroll 1
    for (int i = -1; ok; ++i) {
      if (!unit_there(i + 1)) break;
      const Unit& next = units[(i + 1) % kUnits];
#pragma unroll 1
      for (int g = 0; g < 2; ++g)
        if (next.end[g] > 0) prefetch(next, g);
#pragma unroll 1
      for (int g = 0; g < 2 && ok; ++g)
        if (next.end[g] > 0) rotate(next, g);
      if (i < 0) {
        if (next.n == 0) break;
        continue;
      }
      const Unit& u = units[i % kUnits];
#pragma unroll 1
      for (int g = 0; g < 2 && ok; ++g) {
        if (u.end[g] == 0) continue;
        ok = warp_wait(bars.sum_full[g], outs >> g) && warp_wait(bars.o_full[g], outs >> g);
        if (!ok) break;
        outs ^= 1 << g;
        tc_fence_after();
        const int j = u.j0 + kTile * g + r;
        const bool live = j < p.n_q;
        const float inv = live ? 1.f / sums[g * kGroup + r] : 0.f;
        uint16_t* row = p.out + ((static_cast<int64_t>(u.b) * p.n_q + (live ? j : 0)) * kHeads + u.h) * kNope;
#pragma unroll 1
        for (int x = 0; x < kNope; x += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + lane_off + kTmemO + kTile * g + x, v);
          tmem_wait_ld();
          uint32_t w[16];
#pragma unroll
          for (int y = 0; y < 16; ++y)
            w[y] = pack_bf16x2(__uint_as_float(v[2 * y]) * inv, __uint_as_float(v[2 * y + 1]) * inv);
          if (live) {
#pragma unroll
            for (int y = 0; y < 16; y += 4)
              *reinterpret_cast<uint4*>(row + x + 2 * y) = make_uint4(w[y], w[y + 1], w[y + 2], w[y + 3]);
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&bars.o_free[g]));  // the next unit's first product may overwrite O
      }
      const bool over = next.n == 0;
      unit_done(i);
      if (over) break;
    }
  } else {
    // ------------------------------------------------------------ softmax of query tile g, one thread a row
    const int g = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;  // its row (TMEM lane)
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tm_o = tmem + lane_off + kTmemO + kTile * g, tm_s = tmem + lane_off + kTmemS + kTile * g;
    const uint64_t scale2 = f32x2(kScaleLog2, kScaleLog2);
    bool ok = true;
    int t = 0, done = 0;  // key tiles and units so far
#pragma unroll 1
    for (int i = 0; ok && unit_there(i); ++i) {
      const Unit& u = units[i % kUnits];
      const int n = u.n;
      if (n == 0) break;
      if (u.end[g] == 0) {
        unit_done(i);
        continue;
      }
      const int j = u.j0 + kTile * g + r;                            // its query
      const int pos = j < p.n_q ? u.L + j : -1 - p.window - kTile;   // and that one's position (no query: sees nothing)
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int k = 0; k < n && ok; ++k) {
        const int tile = u.tile(k);
        if (!u.sees(g, tile)) continue;
        ok = warp_wait(bars.s_full[g], t);
        if (!ok) break;
        tc_fence_after();
        // Visible columns: up to the query, of those in the window or among the first tokens.  Where a row of the
        // warp has others, their scores become -inf first (whatever was there; the weight is then 2^-inf = 0).
        const int t0 = tile * kTile, hi = pos + 1 - t0, lo = hi - p.window, sk = min(p.sinks - t0, hi);
        if (!__all_sync(0xffffffffu, hi >= kTile && (lo <= 0 || sk >= kTile))) {
#pragma unroll 1
          for (int x = 0; x < kTile; x += 32) {
            uint32_t v[32];
            tmem_ld32(tm_s + x, v);
            tmem_wait_ld();
            const uint32_t bits = static_cast<uint32_t>(low_bits(min(hi - x, 32)) & ~low_bits(min(lo - x, 32)) |
                                                        low_bits(min(sk - x, 32)));
#pragma unroll
            for (int y = 0; y < 32; ++y) v[y] = (bits >> y & 1u) != 0 ? v[y] : 0xff800000u;
            tmem_st32(tm_s + x, v);
          }
          tmem_wait_st();
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int x = 0; x < kTile; x += 64) {
          uint32_t v[2][32];
          tmem_ld32(tm_s + x, v[0]);
          tmem_ld32(tm_s + x + 32, v[1]);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 64; ++y) m4[y & 3] = fmaxf(m4[y & 3], __uint_as_float(v[y >> 5][y & 31]));
        }
        const float mx = kScaleLog2 * fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        // the weights' reference: the running maximum, taken over where it has grown by more than 2^8
        float factor = 1.f;
        if (m == -INFINITY) {
          m = mx;
        } else if (mx > m + kRescaleLog2) {
          factor = ex2_approx(m - mx);
          m = mx;
        }
        if (__any_sync(0xffffffffu, factor != 1.f)) {  // O is complete up to the last tile: its products are before this S
#pragma unroll 1
          for (int x = 0; x < kNope; x += 32) {
            uint32_t v[32];
            tmem_ld32(tm_o + x, v);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) v[y] = __float_as_uint(__uint_as_float(v[y]) * factor);
            tmem_st32(tm_o + x, v);
          }
        }
        // P = 2^(S scale - m) in bf16 (to nearest even, unbiased), the type of the decompressed keys and values,
        // whose own rounding is as large: P in two bf16 parts took the result's error from 3.0e-3 to 2.6e-3 (the
        // output's rounding alone is 1.7e-3) and 1570 us instead of 1210.  The sum adds the weights in float32.  P
        // of a half takes the place of scores that have been read.
        const float neg_m = m == -INFINITY ? 0.f : -m;
        const uint64_t neg2 = f32x2(neg_m, neg_m);
        uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t v[2][32], pk[32];
          tmem_ld32(tm_s + 64 * h, v[0]);
          tmem_ld32(tm_s + 64 * h + 32, v[1]);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 32; ++y) {
            const uint32_t* s2 = &v[y >> 4][2 * (y & 15)];
            const float2 e = f32x2_split(fma_f32x2(f32x2(__uint_as_float(s2[0]), __uint_as_float(s2[1])), scale2, neg2));
            const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
            pk[y] = pack_bf16x2(p0, p1);
            sum[y & 3] = add_f32x2(sum[y & 3], f32x2(p0, p1));
          }
          tmem_st32(tm_s + 32 * h, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(smem_u32(&bars.p_full[g][h]));
        }
        const float2 s2 = f32x2_split(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])));
        l = l * factor + (s2.x + s2.y);
        ++t;
      }
      // the sums take the place of the last unit's once O's reader has read those
      if (done > 0) ok = ok && warp_wait(bars.o_free[g], done - 1);
      if (!ok) break;
      sums[g * kGroup + r] = l;
      mbar_arrive(smem_u32(&bars.sum_full[g]));
      if (j < p.n_q && p.lse != nullptr)
        p.lse[(static_cast<int64_t>(u.b) * p.n_q + j) * kHeads + u.h] = (m + log2f(l)) * kLn2;
      ++done;
      unit_done(i);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kLoadWarp) tmem_dealloc(tmem, 512);
}

bool g_configured[64];
int g_sms[64];

}  // namespace

cudaError_t launch_prefill_attn_window(const uint16_t* q_nope, const uint16_t* q_rope, const int32_t* seq_lens_before,
                                       const float* rope_table, int rope_max_pos, const uint16_t* k_nope,
                                       const uint16_t* v, int max_kv_len, const uint16_t* cache, int64_t num_pages,
                                       const int32_t* page_table, int pt_stride, const int32_t* kv_lens, int B, int n_q,
                                       int window, int sinks, uint16_t* out, float* lse, int* status,
                                       cudaStream_t stream) {
  if (B == 0 || n_q == 0) return cudaSuccess;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!g_configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(prefill_window_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    g_configured[dev] = true;
  }
  CUtensorMap tk, tv, tkr, tq;
  const uint64_t bh = static_cast<uint64_t>(B) * kHeads, row = kNope * 2;
  // keys and values [sequence and head][token][128]: rows past max_kv_len read as zeros
  if (!make_tmap_bf16_3d(&tk, k_nope, kNope, max_kv_len, bh, row, row * max_kv_len, 64, kTile, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_bf16_3d(&tv, v, kNope, max_kv_len, bh, row, row * max_kv_len, 64, 64, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_bf16_2d(&tkr, cache, static_cast<uint64_t>(num_pages) * kPage, kRow, kRow, 64, 64,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
      // q^C [B n_q tokens][heads][128]: box of 64 columns x 1 head x 128 tokens
      !make_tmap_bf16_3d(&tq, q_nope, kNope, kHeads, static_cast<uint64_t>(B) * n_q, row,
                         static_cast<uint64_t>(kHeads) * kNope * 2, 64, 1, kTile, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  Params prm;
  prm.q_nope = q_nope;
  prm.q_rope = q_rope;
  prm.seq_lens_before = seq_lens_before;
  prm.rope = rope_table;
  prm.page_table = page_table;
  prm.kv_lens = kv_lens;
  prm.out = out;
  prm.lse = lse;
  prm.status = status;
  prm.num_pages = num_pages;
  prm.n_pair = (n_q + 2 * kTile - 1) / (2 * kTile);
  if (static_cast<int64_t>(B) * kHeads * prm.n_pair > 0x7fffffff) return cudaErrorInvalidValue;
  prm.n_units = B * kHeads * prm.n_pair;
  prm.pt_stride = pt_stride;
  prm.rope_max_pos = rope_max_pos;
  prm.max_kv_len = max_kv_len;
  prm.n_q = n_q;
  prm.B = B;
  prm.window = window < max_kv_len ? window : max_kv_len;  // (sums with positions stay in range)
  prm.sinks = sinks < max_kv_len ? sinks : max_kv_len;
  const int grid = prm.n_units < g_sms[dev] ? prm.n_units : g_sms[dev];
  return launch_kernel(prefill_window_kernel, dim3(grid), dim3(kThreads), kSmemBytes, stream, tk, tv, tkr, tq, prm);
}

}  // namespace mla
