// Which cached tokens a query sees: the window, the first tokens that stay visible
// (sinks), and the drafted tokens of a tree.  Shared by the masked attention, its
// split plan and the windowed prefill.
#pragma once

#include "internal.cuh"

namespace mla {

// Query j of a sequence with L tokens before the step's n_q new ones.  It sees
// context tokens [0, sink_hi) and [lo, L), and the new token L + k where bit k of
// `word` is set.  Its pages, in order: [0, ns), then from w0 on, n_pages in all
// (0: it sees nothing).
struct QueryView {
  int L, lo, sink_hi, ns, w0, n_pages;
  uint64_t word;
};

__host__ __device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// pos: the query's position; `word` as given (a tree) or the causal one, which the
// window then cuts as well.  window 0: everything.
__device__ __forceinline__ QueryView make_view(int L, int pos, uint64_t word, bool causal, int window, int sinks) {
  QueryView v;
  v.L = L;
  const int first = window > 0 ? max(0, pos - window + 1) : 0;  // the window's oldest token
  if (causal && first > L) word &= ~(low_bits(first - L) & ~low_bits(min(sinks, first) - L));
  v.word = word;
  v.lo = min(first, L);
  v.sink_hi = min(sinks, v.lo);
  const int end = word != 0 ? L + 64 - __clzll(static_cast<long long>(word)) : L;
  if (end <= 0) {
    v.ns = v.w0 = v.n_pages = 0;
    return v;
  }
  v.w0 = min(v.lo, end - 1) / kPage;
  v.ns = min(pages_of(v.sink_hi), v.w0);  // the sinks' last page may be the window's first
  v.n_pages = v.ns + (end - 1) / kPage - v.w0 + 1;
  return v;
}

// The page of the sequence that is the view's k-th.
__device__ __forceinline__ int view_page(const QueryView& v, int k) { return k < v.ns ? k : k - v.ns + v.w0; }

// Its visible tokens, one bit a slot.
__device__ __forceinline__ uint64_t view_bits(const QueryView& v, int page) {
  const int t0 = page * kPage, sh = v.L - t0;
  uint64_t bits = low_bits(v.sink_hi - t0) | (low_bits(sh) & ~low_bits(v.lo - t0));
  if (sh >= 0 && sh < 64) bits |= v.word << sh;
  if (sh < 0 && sh > -64) bits |= v.word >> -sh;
  return bits;
}

// The most pages a view holds, over every query of a sequence of at most max_kv_len
// tokens: all of them, or the sinks' and a window's that starts anywhere in a page.
inline int max_view_pages(int n_q, int max_kv_len, int window, int sinks) {
  const int all = pages_of(max_kv_len);
  if (window <= 0) return all;
  const int64_t span = static_cast<int64_t>(window) + n_q - 1;  // oldest token of the first query .. the last new one
  const int64_t pages = (sinks + static_cast<int64_t>(kPage) - 1) / kPage + (span + kPage - 2) / kPage + 1;
  return pages < all ? static_cast<int>(pages) : all;
}

}  // namespace mla
