// The plan of a call over a shared prefix (shared_prefix.cuh): checks the shared pages and every
// sequence's length and own pages, gives each sequence its own part, and lists the tiles of all items
// for the pairs of the tensor-core kernel (decode_tc.cuh).
#pragma once

#include "common.cuh"

namespace mla {
namespace shared {
constexpr int kScanSeqs = 4096;  // sequences whose tile counts the plan kernel keeps in shared memory
constexpr int kPlanTile = 128;   // tokens of a tile
constexpr int kMaxPairs = 128;   // pairs at most
// A pair spends on an item, beside its tiles, the time of about kItemUnits more: its queries'
// load, the pipeline's fill and the epilogue (a one-tile item took 6.7 us where a tile of a long
// one takes 2.6). With items counted by tiles alone, 256 one-token sequences behind 32768 shared
// tokens fell to the last pairs and the call took 1520 us (580 so).
constexpr int kItemUnits = 2;

struct PlanArgs {
  const int* seq_lens;  // [B]
  const int* bt;        // [B, max_pages]
  int B, max_pages, num_pages, max_seq_len, page_size;
  const int* shared_pages;
  int n_given;       // pages of the prefix: a bad one rejects every sequence that has them
  int n_shared;      // n_given where rows are packed over the prefix, 0: no sequence has a shared part
  int lanes;         // threads that check one sequence's pages (a power of two <= 32)
  int prefix_items;  // packed row tiles
  int* first;        // [B] first token of the sequence's own part, -1 for a rejected sequence
  int* len;          // [B] its length, 0 for a rejected sequence
  int* tile_prefix;  // [prefix_items + B + 1] places before each item in the list of the items'
                     // tiles, kItemUnits places and then its tiles to an item that has any; or null
  int* pairs;        // [prefix_items + B] first and last pair of an item's tiles, c0 | c1 << 16, -1: none
  int4* start;       // [C] item that each pair begins in, its places [y, z), all places
  int C;             // pairs
};

// Places [T c / C, T (c+1) / C) of T are pair c's; the pair that has place g:
__device__ __forceinline__ int pair_of(int g, int T, int C) {
  if (T < INT32_MAX / kMaxPairs) return (int)(((unsigned)(g + 1) * (unsigned)C - 1u) / (unsigned)T);
  return (int)(((long)(g + 1) * C - 1) / T);
}

template <int kThreads, int kCounts>
struct PlanScratch {
  int count[kCounts];  // places of each sequence (in tile_prefix where there are more)
  int run[kThreads];
  int warp_total[32];
};

// By all kThreads threads of the block. A sequence shorter than the prefix (an idle row of a padded
// batch) attends to its own tokens alone. Rejected sequences have no tiles; their output becomes
// zeros. The host keeps the places of the list within int32. `report`: this block records errors.
template <int kThreads, int kCounts>
__device__ void make_plan(const PlanArgs& a, PlanScratch<kThreads, kCounts>& sc, bool report) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = a.page_size, shared_len = a.n_shared * P;
  // the first sequence's length, and the page it then most likely asks for first, are requested
  // beside the shared pages
  const int per_pass = kThreads / a.lanes, sub = tid & (a.lanes - 1);
  const int b_first = tid / a.lanes, t_first = a.n_shared + sub;
  const int L_first = b_first < a.B ? a.seq_lens[b_first] : 0;
  const int pg_first = b_first < a.B && t_first < a.max_pages ? a.bt[(long)b_first * a.max_pages + t_first] : 0;
  if (tid < 32) sc.warp_total[tid] = 0;
  bool bad = false;
  for (int t = tid; t < a.n_given; t += kThreads) {
    const int pg = a.shared_pages[t];
    bad |= pg < 0 || pg >= a.num_pages;
  }
  const bool bad_prefix = __syncthreads_or(bad);
  const bool in_scratch = a.B <= kCounts;
  for (int b0 = 0; b0 < a.B; b0 += per_pass) {
    const int b = b0 + b_first;
    int L = 0, n = 0, f = 0;
    bool len_ok = false;
    if (b < a.B) {
      L = b0 == 0 ? L_first : a.seq_lens[b];
      len_ok = L >= 1 && L <= a.max_seq_len;
      n = len_ok ? (L - 1) / P + 1 : 0;
      len_ok = len_ok && n <= a.max_pages;
      f = len_ok && shared_len > 0 && L >= shared_len ? shared_len : 0;
    }
    bad = false;
    if (len_ok) {
      const int* row = a.bt + (long)b * a.max_pages;
      int t = f / P + sub;
      if (b0 == 0 && t == t_first && t < n) {
        bad |= pg_first < 0 || pg_first >= a.num_pages;
        t += a.lanes;
      }
#pragma unroll 4
      for (; t < n; t += a.lanes) {
        const int pg = row[t];
        bad |= pg < 0 || pg >= a.num_pages;
      }
    }
    for (int o = 1; o < a.lanes; o <<= 1) bad |= __shfl_xor_sync(0xffffffffu, (int)bad, o) != 0;
    bad |= bad_prefix && L >= a.n_given * P;
    if (b < a.B && sub == 0) {
      if (report && !len_ok) record_error(MLA_ERR_BAD_SEQ_LEN);
      else if (report && bad) record_error(MLA_ERR_BAD_PAGE);
      const bool ok = len_ok && !bad;
      a.first[b] = ok ? f : -1;
      a.len[b] = ok ? L : 0;
      if (a.tile_prefix != nullptr) {
        const int places = ok && L > f ? kItemUnits + (L - f + kPlanTile - 1) / kPlanTile : 0;
        if (in_scratch) sc.count[b] = places;
        else a.tile_prefix[a.prefix_items + b] = places;
      }
    }
  }
  if (a.tile_prefix == nullptr) return;
  const int nt = bad_prefix || shared_len == 0 ? 0 : kItemUnits + (shared_len + kPlanTile - 1) / kPlanTile;
  int* const mine = a.tile_prefix + a.prefix_items;
  for (int i = tid; i < a.prefix_items; i += kThreads) a.tile_prefix[i] = i * nt;
  __syncthreads();
  const int* const count = in_scratch ? sc.count : mine;
  // exclusive scan: thread tid sums `per` sequences, then a two-level shuffle scan of the sums
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += count[b];
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sc.warp_total[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = sc.warp_total[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += v;
    }
    sc.warp_total[lane] = w;
  }
  __syncthreads();
  const int T = a.prefix_items * nt + sc.warp_total[31];
  auto pairs_of = [&](int begin, int n) {
    return n == 0 ? -1 : pair_of(begin + kItemUnits, T, a.C) | (pair_of(begin + n - 1, T, a.C) << 16);
  };
  for (int i = tid; i < a.prefix_items; i += kThreads) a.pairs[i] = pairs_of(i * nt, nt);
  int run = a.prefix_items * nt + incl - sum + (warp > 0 ? sc.warp_total[warp - 1] : 0);
  sc.run[tid] = run;
  for (int b = b0; b < b1; ++b) {
    const int n = count[b];  // read before the same place may be overwritten
    mine[b] = run;
    a.pairs[a.prefix_items + b] = pairs_of(run, n);
    run += n;
  }
  if (tid == kThreads - 1) mine[a.B] = T;
  __syncthreads();
  if (tid < a.C) {  // the item that pair tid begins in
    const int g = (int)((long)T * tid / a.C);
    int item, base, next;
    if (g < a.prefix_items * nt) {
      item = g / nt;
      base = item * nt;
      next = base + nt;
    } else {
      int lo = 0, hi = kThreads - 1;  // the last thread whose sequences begin at or before g
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sc.run[mid] <= g) lo = mid; else hi = mid - 1;
      }
      // (threads past the last sequence hold the total, which only a list without places reaches)
      int b = min(lo * per, a.B - 1);
      base = sc.run[lo];
      if (per == 1) {
        next = b + 1 < a.B ? sc.run[b + 1] : T;
      } else {
        for (next = mine[b + 1]; b + 1 < a.B && next <= g; next = mine[b + 1]) {
          ++b;
          base = next;
        }
      }
      item = a.prefix_items + b;
    }
    a.start[tid] = make_int4(item, base, next, T);
  }
}

}  // namespace shared
}  // namespace mla
