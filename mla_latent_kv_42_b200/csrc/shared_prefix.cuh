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

// The plan as a kernel of its own: one block. Calls with few sequences run it in every CTA of the
// attention kernel instead (see shared_folds in libmla.cu).
__global__ void __launch_bounds__(1024) k_shared_plan(const shared::PlanArgs a) {
  __shared__ shared::PlanScratch<1024, shared::kScanSeqs> scratch;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  shared::make_plan<1024>(a, scratch, true);
}

namespace shared {
struct MergeArgs {
  const float *o_pre, *lse_pre;    // prefix partials: slots of 128 packed rows
  const float *o_part, *lse_part;  // own partials: slots of n_h rows
  const int* tile_prefix;
  const int* pairs;
  const int* first;
  int B, n_h, prefix_items, C;
  void* o_lat;
  float* lse_out;
};
// Partial slots of an item: part k is in slot `item` + its pair. When every pair has places in the
// list (T >= C) the pairs between the first and the last one of the item's tiles lie within them, so
// the slots are consecutive; else part k is tile k, alone on the pair that has its place.
struct Parts {
  int first, n, item, g0;
  __device__ __forceinline__ Parts(bool dense, int item_, const int* prefix, int pairs)
      : first(item_ + (pairs & 0xffff)), n(0), item(item_), g0(0) {
    if (pairs < 0) return;
    n = (pairs >> 16) - (pairs & 0xffff) + 1;
    if (!dense) {
      g0 = prefix[0] + kItemUnits;
      n = prefix[1] - g0;
    }
  }
  template <bool kDense>
  __device__ __forceinline__ int slot(int k, int T, int C) const {
    return kDense ? first + k : item + ((g0 + k + 1) * C - 1) / T;
  }
};
constexpr int kMergeAhead = 8;  // vectors of parts that a thread has in flight
}  // namespace shared

// Joins each query row's partials, those over the prefix and those over its own tokens, in a fixed
// order. kGroups groups of kLanes threads share a row and take its parts in turn, a thread 512 /
// kLanes of the latent values and kMergeAhead vectors of parts in flight: four groups where the
// rows are few and so are cut into many parts, one of fewer threads where they are many (at 8192
// rows of two parts the instructions of 128 threads a row took longer than the partials' bytes).
// Every warp forms the weights of up to 32 parts for itself; more go through shared memory where a
// block has one row. A rejected sequence gets zeros and an lse of -inf. Without prefix items a row
// that one pair finished is already in o_lat. A block of four groups has one row, else its 128
// threads have 128 / kLanes.
template <typename T, int kLanes, int kGroups, bool kDense>
__device__ __forceinline__ void merge_row(const shared::MergeArgs& a, const shared::Parts& pp, const shared::Parts& po,
                                          int r, int b, int T_) {
  constexpr int kVec = 128 / kLanes, kThreads = kLanes * kGroups, kWarps = kThreads / 32;
  constexpr int kMergeAhead = shared::kMergeAhead / kVec;
  __shared__ float s_w[2 * tc::kMaxDecodeClusters];
  __shared__ float s_red[kWarps];
  __shared__ float4 s_acc[kGroups > 1 ? kGroups - 1 : 1][kGroups > 1 ? 128 : 1];
  const int tid = threadIdx.x % kThreads, lane = tid & 31, warp = tid >> 5, group = tid / kLanes;
  const int col = 4 * (tid % kLanes);
  const int n = pp.n + po.n, h = r - b * a.n_h;
  auto row_of = [&](int k) -> long {  // row of part k among the rows of its buffer
    return k < pp.n ? (long)pp.template slot<kDense>(k, T_, a.C) * 128 + (r & 127)
                    : (long)po.template slot<kDense>(k - pp.n, T_, a.C) * a.n_h + h;
  };
  auto lse_of = [&](int k) { return (k < pp.n ? a.lse_pre : a.lse_part)[row_of(k)]; };
  float4 v[kMergeAhead][kVec];
  auto load = [&](int k, float4 (&x)[kVec]) {
    if (k >= n) return;
    const float* src = (k < pp.n ? a.o_pre : a.o_part) + row_of(k) * tc::dec::kDc + col;
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = *reinterpret_cast<const float4*>(src + 4 * kLanes * j);
  };
#pragma unroll
  for (int u = 0; u < kMergeAhead; ++u) load(group + kGroups * u, v[u]);  // requested before the weights are formed
  auto warp_max = [](float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  };
  const bool many = kGroups > 1 && n > 32;  // the same in the whole block
  float mx = -INFINITY;
  const float mine = lane < n ? lse_of(lane) : -INFINITY;
  if (!many) {
    mx = mine;
    for (int k = lane + 32; k < n; k += 32) mx = fmaxf(mx, lse_of(k));
    mx = warp_max(mx);
  } else {
    for (int k = tid; k < n; k += kThreads) mx = fmaxf(mx, s_w[k] = lse_of(k));
    mx = warp_max(mx);
    if (lane == 0) s_red[warp] = mx;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_red[w]);
  }
  auto weight_of = [&](float l) { return l == -INFINITY ? 0.f : exp2f((l - mx) * kLog2e); };  // a NaN stays
  const float w_lane = weight_of(mine);
  float z = 0.f;
  if (!many) {
    z = w_lane;
    for (int k = lane + 32; k < n; k += 32) z += weight_of(lse_of(k));
    z = warp_sum(z);
  } else {
    __syncthreads();  // s_red has been read
    for (int k = tid; k < n; k += kThreads) z += s_w[k] = weight_of(s_w[k]);
    z = warp_sum(z);
    if (lane == 0) s_red[warp] = z;
    __syncthreads();
    z = 0.f;
    for (int w = 0; w < kWarps; ++w) z += s_red[w];
  }
  float4 acc[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = group; k0 < n; k0 += kGroups * kMergeAhead) {
#pragma unroll
    for (int u = 0; u < kMergeAhead; ++u) {
      const int k = k0 + kGroups * u;
      if (k >= n) break;  // the same in the whole warp
      const float w = many ? s_w[k] : k < 32 ? __shfl_sync(0xffffffffu, w_lane, k) : weight_of(lse_of(k));
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        acc[j].x = fmaf(w, v[u][j].x, acc[j].x);
        acc[j].y = fmaf(w, v[u][j].y, acc[j].y);
        acc[j].z = fmaf(w, v[u][j].z, acc[j].z);
        acc[j].w = fmaf(w, v[u][j].w, acc[j].w);
      }
      load(k + kGroups * kMergeAhead, v[u]);
    }
  }
  if constexpr (kGroups > 1) {
    static_assert(kVec == 1, "one vector per thread where groups are joined");
    if (group > 0) s_acc[group - 1][tid % kLanes] = acc[0];
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < kGroups - 1; ++g) {
      const float4 o = s_acc[g][tid];
      acc[0].x += o.x;
      acc[0].y += o.y;
      acc[0].z += o.z;
      acc[0].w += o.w;
    }
  }
  const float inv = z != 0.f ? 1.f / z : 0.f;
  T* const out = static_cast<T*>(a.o_lat) + (long)r * tc::dec::kDc + col;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const typename Pack<T>::T2 two[2] = {Pack<T>::make(acc[j].x * inv, acc[j].y * inv),
                                         Pack<T>::make(acc[j].z * inv, acc[j].w * inv)};
    *reinterpret_cast<uint2*>(out + 4 * kLanes * j) = *reinterpret_cast<const uint2*>(two);
  }
  if (a.lse_out != nullptr && tid == 0) a.lse_out[r] = z != 0.f ? mx + logf(z) : -INFINITY;
}

template <typename T, int kLanes, int kGroups>
__global__ void __launch_bounds__(kGroups > 1 ? kLanes * kGroups : 128) k_shared_merge(const shared::MergeArgs a) {
  constexpr int kThreads = kLanes * kGroups, kRows = kGroups > 1 ? 1 : 128 / kLanes;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  const int r = (int)blockIdx.x * kRows + (int)threadIdx.x / kThreads, tid = threadIdx.x % kThreads;
  if (r >= a.B * a.n_h) return;
  const int b = r / a.n_h;
  const int it = r >> 7;  // the packed tile of this row
  const int f = a.first[b], T_ = a.tile_prefix[a.prefix_items + a.B];
  const int po_pairs = a.pairs[a.prefix_items + b];
  const int pp_pairs = a.prefix_items > 0 && f > 0 ? a.pairs[it] : -1;
  if (f < 0) {
    T* const out = static_cast<T*>(a.o_lat) + (long)r * tc::dec::kDc;
    for (int e = tid; e < tc::dec::kDc / 8; e += kThreads)
      *reinterpret_cast<uint4*>(out + 8 * e) = make_uint4(0, 0, 0, 0);
    if (a.lse_out != nullptr && tid == 0) a.lse_out[r] = -INFINITY;
    return;
  }
  const bool dense = T_ >= a.C;
  const shared::Parts pp(dense, it, a.tile_prefix + it, pp_pairs);
  const shared::Parts po(dense, b, a.tile_prefix + a.prefix_items + b, po_pairs);
  if (a.prefix_items == 0 && po.n == 1) return;
  if (dense) merge_row<T, kLanes, kGroups, true>(a, pp, po, r, b, T_);
  else merge_row<T, kLanes, kGroups, false>(a, pp, po, r, b, T_);
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
// the A fragment of the value product. KDC: k steps of the score product, the row's rounded up to 32
// columns. With the shared-memory row stride a constant every ldmatrix address is a base and an
// immediate, and a step past the row's end multiplies by zeros of Q (columns read again there).
template <typename T, int KDC>
__device__ void prefix_mma_item(const shared::MmaArgs& a, int tile, int split, uint8_t* sm) {
  using namespace dmma;
  using P2 = typename Pack<T>::T2;
  const MmaAttnArgs& g0 = a.own;
  const int D = g0.D, d_c = g0.d_c, KD = D / 16, ND = d_c / 8;
  const int R = g0.B * g0.n_h;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, tq = lane & 3;
  constexpr int stride = row_stride(16 * KDC);
  const uint32_t sm_u32 = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
  const T* __restrict__ q = static_cast<const T*>(g0.q);
  const T* __restrict__ pool = static_cast<const T*>(g0.pool);
  const int t0 = split * a.pre_split_len, t1 = min(a.prefix_len, t0 + a.pre_split_len);
  const int n_stages = t1 > t0 ? (t1 - t0 + kStageTokens - 1) / kStageTokens : 0;
  const int row_base = tile * shared::kRowTile + 16 * warp;
  const int rows[2] = {row_base + g, row_base + g + 8};
  bool live[2];    // the row exists and its sequence has this prefix
  bool theirs[2];  // another item writes the row's partial
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = rows[e] / g0.n_h;
    live[e] = rows[e] < R && g0.first[b] > 0;
    theirs[e] = rows[e] >= R || short_has(g0, b, split);
  }
  const bool warp_live = __any_sync(0xffffffffu, live[0] || live[1]);

  uint32_t qa[KDC][4];
#pragma unroll
  for (int ks = 0; ks < KDC; ++ks)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = rows[e & 1], col = 16 * ks + 2 * tq + ((e & 2) ? 8 : 0);
      qa[ks][e] = ks < KD && row < R ? __ldg(reinterpret_cast<const unsigned*>(q + (long)row * D + col)) : 0u;
    }

  // two threads to a row, each every other 16-byte chunk of it. The pages were checked by the plan;
  // an id outside the pool reads as zeros. A stage's page id is requested a stage ahead.
  const int chunks = D / 8, my_row = tid >> 1;
  auto page_of = [&](int st) {
    const int tok = t0 + st * kStageTokens + my_row;
    return tok < t1 ? __ldg(a.shared_pages + tok / g0.page_size) : -1;
  };
  int pg_next = page_of(0);
  auto issue_stage = [&](int st) {
    const int tok = t0 + st * kStageTokens + my_row, pg = pg_next;
    pg_next = page_of(st + 1);
    const bool valid = pg >= 0 && pg < g0.num_pages;
    const T* const src = valid ? pool + ((long)pg * g0.page_size + tok % g0.page_size) * D : pool;
    const uint32_t dst = sm_u32 + ((st % kStages) * kStageTokens + my_row) * stride;
    for (int col = tid & 1; col < chunks; col += 2)
      cp_async16(dst + col * 16, valid ? src + col * 8 : pool, valid ? 16u : 0u);
  };

  float oacc[kMaxND][4];
#pragma unroll
  for (int j = 0; j < kMaxND; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) oacc[j][e] = 0.f;
  float m_ref[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
  float rsum[2] = {0.f, 0.f};  // lsum of the rounded weights
  for (int st = 0; st < kStages - 1; ++st) {
    if (st < n_stages) issue_stage(st);
    cp_async_commit();
  }
  const int mi = lane >> 3, ri = lane & 7;
  // ldmatrix rows of this lane: keys of the score product, values of the other (transposed)
  const uint32_t k_lane = sm_u32 + (ri + 8 * (mi >> 1)) * stride + 16 * (mi & 1);
  const uint32_t v_lane = sm_u32 + (ri + 8 * (mi & 1)) * stride + 16 * (mi >> 1);
  const int last_k = 32 * (KD - 1);  // byte offset of the row's last k step
  for (int st = 0; st < n_stages; ++st) {
    if (st + kStages - 1 < n_stages) issue_stage(st + kStages - 1);
    cp_async_commit();
    cp_async_wait<kStages - 1>();
    __syncthreads();
    const uint32_t buf = (st % kStages) * kStageTokens * stride;
    const uint32_t kb = k_lane + buf, vb = v_lane + buf;
    const int s0 = t0 + st * kStageTokens;
    if (warp_live) {
      float s[8][4];
#pragma unroll
      for (int n8 = 0; n8 < 8; ++n8)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n8][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KDC; ++ks) {
        const uint32_t at = kb + (ks < KDC - 1 ? 32 * ks : last_k);  // D > 32 (KDC / 2 - 1)
#pragma unroll
        for (int n16 = 0; n16 < 4; ++n16) {
          uint32_t bfr[4];
          ldsm_x4(at + 16 * n16 * stride, bfr);
          mma16816<T>(s[2 * n16], qa[ks], bfr[0], bfr[1]);
          mma16816<T>(s[2 * n16 + 1], qa[ks], bfr[2], bfr[3]);
        }
      }
      if (t1 - s0 < kStageTokens) {  // the prefix's last stage
#pragma unroll
        for (int n8 = 0; n8 < 8; ++n8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * n8 + 2 * tq + (e & 1) >= t1 - s0) s[n8][e] = -INFINITY;
      }
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        float mx = -INFINITY;
#pragma unroll
        for (int n8 = 0; n8 < 8; ++n8) mx = fmaxf(mx, fmaxf(s[n8][2 * h2], s[n8][2 * h2 + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * g0.scale_log2;
        if (mx > m_ref[h2] + kLazy) {  // the quad agrees
          const float alpha = exp2f(m_ref[h2] - mx);
          lsum[h2] *= alpha;
          rsum[h2] *= alpha;
#pragma unroll
          for (int j = 0; j < kMaxND; ++j) {
            oacc[j][2 * h2] *= alpha;
            oacc[j][2 * h2 + 1] *= alpha;
          }
          m_ref[h2] = mx;
        }
#pragma unroll
        for (int n8 = 0; n8 < 8; ++n8) {
          const float p0 = tc::ex2_approx(fmaf(s[n8][2 * h2], g0.scale_log2, -m_ref[h2]));
          const float p1 = tc::ex2_approx(fmaf(s[n8][2 * h2 + 1], g0.scale_log2, -m_ref[h2]));
          const P2 two = Pack<T>::make(p0, p1);
          const float2 back = Pack<T>::f2(two);
          lsum[h2] += p0 + p1;
          rsum[h2] += back.x + back.y;
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
            ldsm_x4_t(vb + 16 * k16 * stride + 32 * jp, bfr);
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
    // the lse from the weights before rounding (good to fp32), o over the sum of the rounded ones
    float l = lsum[h2], rounded = rsum[h2];
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      rounded += __shfl_xor_sync(0xffffffffu, rounded, o);
    }
    if (theirs[h2]) continue;
    const bool some = live[h2] && l != 0.f;  // a NaN goes through
    const float inv = some ? 1.f / rounded : 0.f;
    const long part = (long)rows[h2] * g0.n_splits + split;
#pragma unroll
    for (int j = 0; j < kMaxND; ++j)
      if (j < ND)
        *reinterpret_cast<float2*>(g0.o_part + part * d_c + 8 * j + 2 * tq) =
            some ? make_float2(oacc[j][2 * h2] * inv, oacc[j][2 * h2 + 1] * inv) : make_float2(0.f, 0.f);
    if (tq == 0) g0.lse_part[part] = some ? (m_ref[h2] + log2f(l)) * kLn2 : -INFINITY;
  }
}

// Blocks [0, row_tiles * pre_splits): prefix items, and then what sequences shorter than the prefix
// whose first row is the tile's have in the same partial; the rest: (sequence, split) items over
// own tokens. 128 threads. Three CTAs to an SM, at the price of spilling 12 to 76 bytes a
// thread: with two none spill, and 232 sequences of 8 heads behind 8192 tokens take 63.0 us instead of 59.7, 100 of 16
// behind 16384 103.1 instead of 99.5, 64 behind 4096 29.3 either way, but 16 behind 32768 49.5
// instead of 61.3 (whole rounds of stages, by the count of CTAs that the splits aim at).
template <typename T, int KDC>
__global__ void __launch_bounds__(128, 3) k_shared_mma(const shared::MmaArgs a) {
  extern __shared__ __align__(16) uint8_t sm[];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  const int n_pre = a.row_tiles * a.pre_splits, i = blockIdx.x;
  int b, b_end, split;
  if (i < n_pre) {
    const int tile = i / a.pre_splits, s = i % a.pre_splits, n_h = a.own.n_h;
    b = (tile * shared::kRowTile + n_h - 1) / n_h;  // (at most 64 sequences)
    b_end = min(a.own.B, ((tile + 1) * shared::kRowTile + n_h - 1) / n_h);
    split = a.own_splits + s;
    const int mine = b + (int)threadIdx.x;
    const bool has = mine < b_end && short_has(a.own, mine, s);
    prefix_mma_item<T, KDC>(a, tile, s, sm);
    if (!__syncthreads_or(has)) return;
  } else {
    const int j = i - n_pre;
    b = j / a.own_splits;
    b_end = b + 1;
    split = j % a.own_splits;
  }
  for (; b < b_end; ++b) {
    if (i < n_pre) {
      if (!short_has(a.own, b, split - a.own_splits)) continue;  // the same in the whole block
      __syncthreads();  // shared memory of the item before
    }
    attn_mma_item<T, true>(a.own, b, split, sm);
  }
}

}  // namespace mla
