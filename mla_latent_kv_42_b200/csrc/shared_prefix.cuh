// Latent attention of a batch whose sequences begin with the same cached pages (a system prompt,
// one document asked many questions). Softmax attention over a sequence is the join of its parts
// by log-sum-exp,
//   o = (e^{lse_1} o_1 + e^{lse_2} o_2) / (e^{lse_1} + e^{lse_2}),
// so the part over the shared pages is computed once for the whole batch: every head of every
// sequence is one more query row against the same keys. The B n_h rows of q are packed into tiles
// of 128 (the tensor-core kernel of decode_tc.cuh) or 64 rows (k_shared_mma below), so a tile of
// shared tokens is loaded and multiplied ceil(B n_h / 128) times instead of B times. Each
// sequence's own tokens are an item of their own, and k_shared_merge (or k_lse_merge_warp) joins
// the parts in a fixed order. All partials are fp32.
#pragma once

#include "decode_mma.cuh"
#include "decode_tc.cuh"

namespace mla {

namespace shared {
constexpr int kScanSeqs = 4096;  // sequences whose tile counts the plan keeps in shared memory

struct PlanArgs {
  const int* seq_lens;  // [B]
  const int* bt;        // [B, max_pages]
  int B, max_pages, num_pages, max_seq_len, page_size;
  const int* shared_pages;
  int n_shared;      // pages of the prefix; 0: no sequence has a shared part
  int lanes;         // threads that check one sequence's pages (a power of two <= 32)
  int prefix_items;  // packed row tiles
  int* first;        // [B] first token of the sequence's own part, -1 for a rejected sequence
  int* len;          // [B] its length, 0 for a rejected sequence
  int* tile_prefix;  // [prefix_items + B + 1] 128-token tiles before each item, or null
};
}  // namespace shared

// One block of 1024 threads: checks the shared pages and every sequence's length and own pages,
// gives each sequence its own part, and (tile_prefix) lists the tiles of all items: the packed row
// tiles first, each over the whole prefix, then the sequences. A sequence shorter than the prefix
// (an idle row of a padded batch) attends to its own tokens alone. Rejected sequences have no
// tiles; their output becomes zeros. The host keeps the tile total within int32.
__global__ void __launch_bounds__(1024) k_shared_plan(const shared::PlanArgs a) {
  __shared__ int s_count[shared::kScanSeqs];
  __shared__ int warp_total[32];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = a.page_size, shared_len = a.n_shared * P;
  bool bad = false;
  for (int t = tid; t < a.n_shared; t += 1024) {
    const int pg = a.shared_pages[t];
    bad |= pg < 0 || pg >= a.num_pages;
  }
  const bool bad_prefix = __syncthreads_or(bad);
  const int per_pass = 1024 / a.lanes, sub = tid & (a.lanes - 1);
  for (int b0 = 0; b0 < a.B; b0 += per_pass) {
    const int b = b0 + tid / a.lanes;
    int L = 0, n = 0, f = 0;
    bool len_ok = false;
    if (b < a.B) {
      L = a.seq_lens[b];
      len_ok = L >= 1 && L <= a.max_seq_len;
      n = len_ok ? (L + P - 1) / P : 0;
      len_ok = len_ok && n <= a.max_pages;
      f = len_ok && shared_len > 0 && L >= shared_len ? shared_len : 0;
    }
    bad = false;
    if (len_ok) {
      const int* row = a.bt + (long)b * a.max_pages;
#pragma unroll 4
      for (int t = f / P + sub; t < n; t += a.lanes) {
        const int pg = row[t];
        bad |= pg < 0 || pg >= a.num_pages;
      }
    }
    for (int o = 1; o < a.lanes; o <<= 1) bad |= __shfl_xor_sync(0xffffffffu, (int)bad, o) != 0;
    bad |= f > 0 && bad_prefix;
    if (b < a.B && sub == 0) {
      if (!len_ok) record_error(MLA_ERR_BAD_SEQ_LEN);
      else if (bad) record_error(MLA_ERR_BAD_PAGE);
      const bool ok = len_ok && !bad;
      a.first[b] = ok ? f : -1;
      a.len[b] = ok ? L : 0;
      if (a.tile_prefix != nullptr) {
        const int tiles = ok ? (int)(((long)(L - f) + tc::dec::kTile - 1) / tc::dec::kTile) : 0;
        if (a.B <= shared::kScanSeqs) s_count[b] = tiles;
        else a.tile_prefix[a.prefix_items + b] = tiles;
      }
    }
  }
  if (a.tile_prefix == nullptr) return;
  const int nt = bad_prefix ? 0 : (shared_len + tc::dec::kTile - 1) / tc::dec::kTile;
  int* const mine = a.tile_prefix + a.prefix_items;
  for (int i = tid; i < a.prefix_items; i += 1024) a.tile_prefix[i] = i * nt;
  __syncthreads();
  const int* const count = a.B <= shared::kScanSeqs ? s_count : mine;
  // exclusive scan: thread tid sums `per` sequences, then a two-level shuffle scan of the sums
  const int per = (a.B + 1023) / 1024;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += count[b];
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = warp_total[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += v;
    }
    warp_total[lane] = w;
  }
  __syncthreads();
  int run = a.prefix_items * nt + incl - sum + (warp > 0 ? warp_total[warp - 1] : 0);
  for (int b = b0; b < b1; ++b) {
    const int n = count[b];  // read before the same place may be overwritten
    mine[b] = run;
    run += n;
  }
  if (tid == 1023) mine[a.B] = a.prefix_items * nt + warp_total[31];
}

namespace shared {
struct MergeArgs {
  const float *o_pre, *lse_pre;    // prefix partials: slots of 128 packed rows
  const float *o_part, *lse_part;  // own partials: slots of n_h rows
  const int* tile_prefix;
  const int* first;
  int B, n_h, prefix_items, C;
  void* o_lat;
  float* lse_out;
};
// Partial slots of an item whose tiles start at g0: part k is in slot item + pair, the pair being
// c0 + k when every pair has tiles (T >= C), else the one that owns tile g0 + k (no two tiles
// share a pair then).
struct Parts {
  long T;
  int C, item, g0, c0, n;
  __device__ __forceinline__ Parts(long T_, int C_, int item_, int g0_, int g1) : T(T_), C(C_), item(item_), g0(g0_) {
    c0 = 0;
    n = 0;
    if (g1 <= g0) return;
    c0 = tc::cluster_of(g0, T, C);
    n = T >= C ? tc::cluster_of(g1 - 1, T, C) - c0 + 1 : g1 - g0;
  }
  __device__ __forceinline__ int slot(int k) const {
    return item + (T >= C ? c0 + k : tc::cluster_of(g0 + k, T, C));
  }
};
}  // namespace shared

// Joins each query row's partials, those over the prefix and those over its own tokens, in pair
// order. A warp per row, each lane 16 of the 512 latent values; two parts' loads in flight. A
// rejected sequence gets zeros and an lse of -inf. Without prefix items a row that one pair
// finished is already in o_lat. Bound by the 2 KB of a partial row: R rows with n parts move
// 2048 R n bytes.
template <typename T>
__global__ void __launch_bounds__(256) k_shared_merge(const shared::MergeArgs a) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  const int lane = threadIdx.x & 31;
  const int r = (int)(blockIdx.x * 8 + (threadIdx.x >> 5));
  if (r >= a.B * a.n_h) return;
  const int b = r / a.n_h, h = r - b * a.n_h;
  const int f = a.first[b];
  const long T_ = a.tile_prefix[a.prefix_items + a.B];
  T* const out = static_cast<T*>(a.o_lat) + (long)r * tc::dec::kDc;
  if (f < 0) {
    for (int e = lane; e < tc::dec::kDc / 8; e += 32) *reinterpret_cast<uint4*>(out + 8 * e) = make_uint4(0, 0, 0, 0);
    if (a.lse_out != nullptr && lane == 0) a.lse_out[r] = -INFINITY;
    return;
  }
  const int it = r >> 7;  // the packed tile of this row
  const bool pre = a.prefix_items > 0 && f > 0;
  const shared::Parts pp(T_, a.C, it, pre ? a.tile_prefix[it] : 0, pre ? a.tile_prefix[it + 1] : 0);
  const shared::Parts po(T_, a.C, b, a.tile_prefix[a.prefix_items + b], a.tile_prefix[a.prefix_items + b + 1]);
  if (a.prefix_items == 0 && po.n == 1) return;
  const int n = pp.n + po.n;
  auto row_of = [&](int k) -> long {  // row of part k among the rows of its buffer
    return k < pp.n ? (long)pp.slot(k) * 128 + (r & 127) : (long)po.slot(k - pp.n) * a.n_h + h;
  };
  auto lse_of = [&](int k) { return k < pp.n ? a.lse_pre[row_of(k)] : a.lse_part[row_of(k)]; };
  auto load = [&](int k, float4 (&v)[4]) {
    const float4* src = reinterpret_cast<const float4*>((k < pp.n ? a.o_pre : a.o_part) + row_of(k) * tc::dec::kDc);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = src[lane + 32 * j];
  };
  // the first two parts are requested before the weights are formed
  float4 v0[4], v1[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v0[j] = v1[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n > 0) load(0, v0);
  if (n > 1) load(1, v1);
  const float mine = lane < n ? lse_of(lane) : -INFINITY;
  float mx = mine;
  for (int k = lane + 32; k < n; k += 32) mx = fmaxf(mx, lse_of(k));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  auto weight_of = [&](float l) { return l > -INFINITY ? exp2f((l - mx) * kLog2e) : 0.f; };
  float z = weight_of(mine);
  for (int k = lane + 32; k < n; k += 32) z += weight_of(lse_of(k));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  float4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int k, const float4 (&v)[4]) {
    const float l = k < 32 ? __shfl_sync(0xffffffffu, mine, k) : lse_of(k);
    const float w = weight_of(l);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[j].x = fmaf(w, v[j].x, acc[j].x);
      acc[j].y = fmaf(w, v[j].y, acc[j].y);
      acc[j].z = fmaf(w, v[j].z, acc[j].z);
      acc[j].w = fmaf(w, v[j].w, acc[j].w);
    }
  };
  for (int k = 0; k < n; k += 2) {
    float4 n0[4], n1[4];
    if (k + 2 < n) load(k + 2, n0);
    if (k + 3 < n) load(k + 3, n1);
    add(k, v0);
    if (k + 1 < n) add(k + 1, v1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v0[j] = n0[j];
      v1[j] = n1[j];
    }
  }
  const float inv = z > 0.f ? 1.f / z : 0.f;
  typename Pack<T>::T2* dst = reinterpret_cast<typename Pack<T>::T2*>(out);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 2 * (lane + 32 * j);
    dst[e] = Pack<T>::make(acc[j].x * inv, acc[j].y * inv);
    dst[e + 1] = Pack<T>::make(acc[j].z * inv, acc[j].w * inv);
  }
  if (a.lse_out != nullptr && lane == 0) a.lse_out[r] = z > 0.f ? mx + logf(z) : -INFINITY;
}

// ---------------------------------------------------------------- narrow rows, few heads
namespace shared {
constexpr int kRowTile = 64;  // query rows of a CTA: 16 per warp
struct MmaArgs {
  MmaAttnArgs own;          // a sequence's own tokens (bt, lengths and partials of the call)
  const int* shared_pages;  // prefix
  int prefix_len, row_tiles, pre_splits, pre_split_len, own_splits;
};
}  // namespace shared

// Tokens [t0, t1) of the prefix for query rows [row0, row0 + 64): each warp holds 16 rows (A
// fragments of Q, fp32 O) and runs over all 64 tokens of a stage, so a stage that one sequence's
// heads would use once serves 64 rows. The arithmetic is attn_mma_item's: P stays in registers as
// the A fragment of the value product.
template <typename T>
__device__ void prefix_mma_item(const shared::MmaArgs& a, int tile, int split, uint8_t* sm) {
  using namespace dmma;
  using P2 = typename Pack<T>::T2;
  const MmaAttnArgs& g0 = a.own;
  const int D = g0.D, d_c = g0.d_c, KD = D / 16, ND = d_c / 8;
  const int R = g0.B * g0.n_h;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int stride = row_stride(D);
  const uint32_t sm_u32 = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
  const T* __restrict__ q = static_cast<const T*>(g0.q);
  const T* __restrict__ pool = static_cast<const T*>(g0.pool);
  const int t0 = split * a.pre_split_len, t1 = min(a.prefix_len, t0 + a.pre_split_len);
  const int n_stages = t1 > t0 ? (t1 - t0 + kStageTokens - 1) / kStageTokens : 0;
  const int row_base = tile * shared::kRowTile + 16 * warp;
  const int rows[2] = {row_base + g, row_base + g + 8};
  bool live[2];  // the row exists and its sequence has this prefix
#pragma unroll
  for (int e = 0; e < 2; ++e) live[e] = rows[e] < R && g0.first[rows[e] / g0.n_h] > 0;
  const bool warp_live = __any_sync(0xffffffffu, live[0] || live[1]);

  uint32_t qa[kMaxKD][4];
#pragma unroll
  for (int ks = 0; ks < kMaxKD; ++ks)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = rows[e & 1], col = 16 * ks + 2 * tq + ((e & 2) ? 8 : 0);
      qa[ks][e] = ks < KD && row < R ? __ldg(reinterpret_cast<const unsigned*>(q + (long)row * D + col)) : 0u;
    }

  // pages are looked up by each 16-token group's threads (page_size % 16 == 0) and were checked by
  // the plan; an id outside the pool reads as zeros
  const int chunks = D / 8;
  auto issue_stage = [&](int st) {
    const uint32_t base = sm_u32 + (st % kStages) * kStageTokens * stride;
    const int s0 = t0 + st * kStageTokens;
    for (int c = tid; c < kStageTokens * chunks; c += 128) {
      const int row = c / chunks, col = c - row * chunks;
      const int tok = s0 + row;
      int pg = -1;
      if (tok < t1) pg = __ldg(a.shared_pages + tok / g0.page_size);
      const bool valid = pg >= 0 && pg < g0.num_pages;
      const T* src = valid ? pool + ((long)pg * g0.page_size + tok % g0.page_size) * D + col * 8 : pool;
      cp_async16(base + row * stride + col * 16, src, valid ? 16u : 0u);
    }
  };

  float oacc[kMaxND][4];
#pragma unroll
  for (int j = 0; j < kMaxND; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) oacc[j][e] = 0.f;
  float m_ref[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
  for (int st = 0; st < kStages - 1; ++st) {
    if (st < n_stages) issue_stage(st);
    cp_async_commit();
  }
  const int mi = lane >> 3, ri = lane & 7;
  for (int st = 0; st < n_stages; ++st) {
    if (st + kStages - 1 < n_stages) issue_stage(st + kStages - 1);
    cp_async_commit();
    cp_async_wait<kStages - 1>();
    __syncthreads();
    const uint32_t tile_u32 = sm_u32 + (st % kStages) * kStageTokens * stride;
    const int s0 = t0 + st * kStageTokens;
    if (warp_live) {
      float s[8][4];
#pragma unroll
      for (int n8 = 0; n8 < 8; ++n8)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n8][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < kMaxKD; ++ks) {
        if (ks < KD) {
#pragma unroll
          for (int n16 = 0; n16 < 4; ++n16) {
            uint32_t bfr[4];
            ldsm_x4(tile_u32 + (16 * n16 + ri + 8 * (mi >> 1)) * stride + (16 * ks + 8 * (mi & 1)) * 2, bfr);
            mma16816<T>(s[2 * n16], qa[ks], bfr[0], bfr[1]);
            mma16816<T>(s[2 * n16 + 1], qa[ks], bfr[2], bfr[3]);
          }
        }
      }
      const int left = t1 - s0;  // tokens of the stage that count
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        float mx = -INFINITY;
#pragma unroll
        for (int n8 = 0; n8 < 8; ++n8)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& v = s[n8][2 * h2 + e];
            v = 8 * n8 + 2 * tq + e < left ? v * g0.scale_log2 : -INFINITY;
            mx = fmaxf(mx, v);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (mx > m_ref[h2] + kLazy) {  // the quad agrees
          const float alpha = exp2f(m_ref[h2] - mx);
          lsum[h2] *= alpha;
#pragma unroll
          for (int j = 0; j < kMaxND; ++j) {
            oacc[j][2 * h2] *= alpha;
            oacc[j][2 * h2 + 1] *= alpha;
          }
          m_ref[h2] = mx;
        }
#pragma unroll
        for (int n8 = 0; n8 < 8; ++n8) {
          // the denominator sums the weights before they are rounded to 16 bits
          const float p0 = exp2f(s[n8][2 * h2] - m_ref[h2]), p1 = exp2f(s[n8][2 * h2 + 1] - m_ref[h2]);
          lsum[h2] += p0 + p1;
          const P2 two = Pack<T>::make(p0, p1);
          s[n8][2 * h2] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&two));
        }
      }
#pragma unroll
      for (int k16 = 0; k16 < 4; ++k16) {
        const uint32_t pa[4] = {__float_as_uint(s[2 * k16][0]), __float_as_uint(s[2 * k16][2]),
                                __float_as_uint(s[2 * k16 + 1][0]), __float_as_uint(s[2 * k16 + 1][2])};
#pragma unroll
        for (int jp = 0; jp < kMaxND / 2; ++jp) {
          if (2 * jp < ND) {
            uint32_t bfr[4];
            ldsm_x4_t(tile_u32 + (16 * k16 + ri + 8 * (mi & 1)) * stride + (16 * jp + 8 * (mi >> 1)) * 2, bfr);
            mma16816<T>(oacc[2 * jp], pa, bfr[0], bfr[1]);
            mma16816<T>(oacc[2 * jp + 1], pa, bfr[2], bfr[3]);
          }
        }
      }
    }
    __syncthreads();  // every warp is done with this buffer before it is refilled
  }
  cp_async_wait<0>();
#pragma unroll
  for (int h2 = 0; h2 < 2; ++h2) {
    float l = lsum[h2];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (rows[h2] >= R) continue;
    const bool some = live[h2] && l > 0.f;
    const float inv = some ? 1.f / l : 0.f;
    const long part = (long)rows[h2] * g0.n_splits + split;
#pragma unroll
    for (int j = 0; j < kMaxND; ++j)
      if (j < ND)
        *reinterpret_cast<float2*>(g0.o_part + part * d_c + 8 * j + 2 * tq) =
            some ? make_float2(oacc[j][2 * h2] * inv, oacc[j][2 * h2 + 1] * inv) : make_float2(0.f, 0.f);
    if (tq == 0) g0.lse_part[part] = some ? (m_ref[h2] + log2f(l)) * kLn2 : -INFINITY;
  }
}

// Blocks [0, row_tiles * pre_splits): prefix items; the rest: (sequence, split) items over own
// tokens. 128 threads.
template <typename T>
__global__ void __launch_bounds__(128) k_shared_mma(const shared::MmaArgs a) {
  extern __shared__ __align__(16) uint8_t sm[];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  const int n_pre = a.row_tiles * a.pre_splits, i = blockIdx.x;
  if (i < n_pre) {
    prefix_mma_item<T>(a, i / a.pre_splits, i % a.pre_splits, sm);
  } else {
    const int j = i - n_pre;
    attn_mma_item<T, true>(a.own, j / a.own_splits, j % a.own_splits, sm);
  }
}

}  // namespace mla
