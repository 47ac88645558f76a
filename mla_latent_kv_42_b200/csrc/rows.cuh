// Rows of the paged latent cache written from given projections, and read back.
//
// k_norm_append: x_t = [c ‖ k^] of token t (the output of [W^DKV; W^KR], or a slice of a wider fused
// projection). Each part is optionally RMS-normalised, k^ is rotated ("DeepSeek-V2 from Scratch",
// §4.2), and the row goes to the token's slot of a 16-bit or an e4m3 cache (the page format of
// fp8.cuh):
//   c' = c / sqrt(mean(c^2) + eps) * g_c,  k' likewise with g_r,  k^R = RoPE(k', pos).
// k_read_rows: the rows of given (sequence, position) pairs as 16-bit rows.
//
// Both are bound by memory (and by latency when there are few tokens): a warp per token, 8 elements
// per lane and step, everything between the load and the store in fp32 registers and rounded once.
#pragma once

#include "fp8.cuh"

namespace mla {
namespace rows {
constexpr int kGroups = 3;    // 8-element groups per lane: D <= 768
constexpr int kMaxPairs = 284;  // d_rope / 2
constexpr int kPowers = 9;      // kMaxPairs < 2^9
constexpr int kWarps = 8;     // per CTA
constexpr int kReadTokens = 4;  // tokens a warp of k_read_rows has in flight

// Slot (row of the pool) of position p of sequence s, or -1 if it is outside the table or the pool.
struct SlotMap {
  const int* bt;  // [num_seqs, max_pages]
  int num_seqs, max_pages, num_pages, page_size;
  __device__ __forceinline__ long operator()(int s, int p) const {
    if (s < 0 || s >= num_seqs || p < 0) return -1;
    const int lp = p / page_size;
    if (lp >= max_pages) return -1;
    const int page = bt[(long)s * max_pages + lp];
    if (page < 0 || page >= num_pages) return -1;
    return (long)page * page_size + (p - lp * page_size);
  }
};

// RoPE frequencies in turns per position, theta_k / 2 pi. theta_k = r^k with r = base^(-2/d_rope)
// is multiplied together from the powers r^(2^j) in double (a relative error of at most
// 9 + k units in the 54th bit, so an angle is off by less than 1e-15 pos radians); a table of
// theta_k takes their place.
struct Turns {
  double pw[kPowers];
  const double* table;
  __device__ __forceinline__ double operator()(int k) const {
    constexpr double kInv2Pi = 0.15915494309189533577;
    if (table != nullptr) return table[k] * kInv2Pi;
    double f = kInv2Pi;
#pragma unroll
    for (int j = 0; j < kPowers; ++j)
      if ((k >> j) & 1) f *= pw[j];
    return f;
  }
};

// cos and sin of pos * theta from turns = theta / 2 pi: whole turns are taken off in double, so the
// rest, at most half a turn, loses nothing that fp32 holds.
__device__ __forceinline__ void turn_cos_sin(int pos, double turns, float& c, float& s) {
  const double t = (double)pos * turns;
  sincospif(2.f * (float)(t - rint(t)), &s, &c);
}

// v / s for a normal s with a normal reciprocal, given inv = 1 / s rounded: the quotient's remainder is
// exact in an fma, and one step with it gives the correctly rounded quotient (Markstein 1990,
// theorem on division from a correctly rounded reciprocal). Three instructions to the value.
__device__ __forceinline__ float quotient(float v, float s, float inv) {
  const float q = v * inv;
  return fmaf(fmaf(-q, s, v), inv, q);
}

struct AppendArgs {
  const void* x;  // [T] rows of D elements, x_stride apart
  long x_stride;
  const void* g_c;  // [d_c] or null
  const void* g_r;  // [d_rope] or null
  float eps;
  const int* seq_idx;
  const int* pos;
  SlotMap slot;
  int d_c, D, T;
  void* pool;
  Turns turns;
};
}  // namespace rows

// A warp per token, the next token's row, position and sequence requested before this one's
// arithmetic. The frequencies are formed once per CTA in shared memory (they are doubles), and the
// warp's lanes share a token's cosines and sines, one pair each, through it.
template <typename T, bool kFp8>
__global__ void __launch_bounds__(32 * rows::kWarps) k_norm_append(const rows::AppendArgs a) {
  using namespace rows;
  using P2 = typename Pack<T>::T2;
  __shared__ double s_turns[kMaxPairs];
  __shared__ float2 s_cs[kWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.D / 8, Gc = a.d_c / 8;  // groups of the row, of its latent part
  const int pairs = (a.D - a.d_c) / 2;
  if (a.turns.table == nullptr)  // from the arguments alone: ahead of the wait
    for (int k = threadIdx.x; k < pairs; k += 32 * kWarps) s_turns[k] = a.turns(k);
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  if (a.turns.table != nullptr)
    for (int k = threadIdx.x; k < pairs; k += 32 * kWarps) s_turns[k] = a.turns(k);
  __syncthreads();
  float2* const cs = s_cs[warp];
  const int n_warps = gridDim.x * kWarps;
  int t = blockIdx.x * kWarps + warp;
  uint4 raw[kGroups];
  int p = 0, seq = 0;
  auto request = [&](int tt) {
    if (tt >= a.T) return;
    const T* src = static_cast<const T*>(a.x) + (long)tt * a.x_stride;
    p = a.pos[tt];
    seq = a.seq_idx[tt];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int g = lane + 32 * i;
      raw[i] = g < G ? *reinterpret_cast<const uint4*>(src + 8 * g) : make_uint4(0, 0, 0, 0);
    }
  };
  request(t);
  for (; t < a.T; t += n_warps) {
    const int pos = p;
    const long slot = a.slot(seq, pos);
    float v[kGroups][8];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) unpack8<T>(raw[i], v[i]);
    request(t + n_warps);
    if (slot < 0) {
      if (lane == 0) record_error(MLA_ERR_BAD_PAGE);
      continue;
    }
    for (int k = lane; k < pairs; k += 32) turn_cos_sin(pos, s_turns[k], cs[k].x, cs[k].y);
    float ss_c = 0.f, ss_r = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
      if (lane + 32 * i < Gc) ss_c += ss;
      else ss_r += ss;
    }
    if (a.g_c != nullptr) ss_c = rsqrtf(warp_sum(ss_c) / (float)a.d_c + a.eps);
    if (a.g_r != nullptr) ss_r = rsqrtf(warp_sum(ss_r) / (float)(a.D - a.d_c) + a.eps);
    __syncwarp();  // cs is written
    float mc = 0.f, mr = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int g = lane + 32 * i;
      const bool lat = g < Gc;
      const void* gain = lat ? a.g_c : a.g_r;
      if (gain != nullptr && g < G) {
        float gf[8];
        unpack8<T>(ldg16(static_cast<const T*>(gain) + 8 * (lat ? g : g - Gc)), gf);
        const float rs = lat ? ss_c : ss_r;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * rs * gf[e];
      }
      if (!lat && g < G) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 c = cs[4 * (g - Gc) + e];
          const float x0 = v[i][2 * e], x1 = v[i][2 * e + 1];
          v[i][2 * e] = x0 * c.x - x1 * c.y;
          v[i][2 * e + 1] = x0 * c.y + x1 * c.x;
        }
      }
      if constexpr (kFp8) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[i][e]));
        if (lat) mc = fmaxf(mc, m);
        else mr = fmaxf(mr, m);
      }
    }
    __syncwarp();  // cs has been read
    if constexpr (!kFp8) {
      T* dst = static_cast<T*>(a.pool) + slot * a.D;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int g = lane + 32 * i;
        if (g < G) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const P2 two = Pack<T>::make(v[i][2 * e], v[i][2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&two);
          }
          *reinterpret_cast<uint4*>(dst + 8 * g) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    } else {
      // non-negative floats order as their bit patterns
      mc = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mc)));
      mr = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mr)));
      const float sc = mc > 0.f ? mc / fp8::kE4m3Max : 1.f;
      const float sr = mr > 0.f ? mr / fp8::kE4m3Max : 1.f;
      const float ic = 1.f / sc, ir = 1.f / sr;
      // scales whose reciprocal or whose products with values are not normal divide as they are
      const bool plain = !(fminf(sc, sr) > 0x1p-100f && fmaxf(sc, sr) < 0x1p100f);
      const int ps = a.slot.page_size;
      const long page = slot / ps;
      const int row = (int)(slot - page * ps);
      uint8_t* const pg = static_cast<uint8_t*>(a.pool) + page * fp8::page_bytes(ps, a.D);
      auto store = [&](auto divide) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const int g = lane + 32 * i;
          if (g < G) {
            const float s = g < Gc ? sc : sr, inv = g < Gc ? ic : ir;
            uint32_t q[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float* x = v[i] + 4 * h;
              const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
                  make_float2(divide(x[0], s, inv), divide(x[1], s, inv)), __NV_SATFINITE, __NV_E4M3);
              const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
                  make_float2(divide(x[2], s, inv), divide(x[3], s, inv)), __NV_SATFINITE, __NV_E4M3);
              q[h] = (uint32_t)lo | ((uint32_t)hi << 16);
            }
            *reinterpret_cast<uint2*>(pg + (long)row * a.D + 8 * g) = make_uint2(q[0], q[1]);
          }
        }
      };
      if (plain) store([](float x, float s, float) { return x / s; });
      else store([](float x, float s, float inv) { return quotient(x, s, inv); });
      if (lane == 0) *reinterpret_cast<float2*>(pg + (long)ps * a.D + 8 * row) = make_float2(sc, sr);
    }
  }
}

namespace rows {
struct ReadArgs {
  const void* pool;
  const int* seq_idx;
  const int* pos;
  SlotMap slot;
  int d_c, D, T;
  void* out;  // [T] rows of D elements, out_stride apart
  long out_stride;
};
}  // namespace rows

// A warp takes kReadTokens consecutive tokens at a time: lanes 0 .. kReadTokens - 1 look up their
// slots (three dependent reads, once for the group), then every lane has the loads of all of them
// in flight. A token without a valid slot becomes a zero row and records MLA_ERR_BAD_PAGE.
template <typename T, bool kFp8>
__global__ void __launch_bounds__(32 * rows::kWarps) k_read_rows(const rows::ReadArgs a) {
  using namespace rows;
  using P2 = typename Pack<T>::T2;
  using Raw = std::conditional_t<kFp8, uint2, uint4>;  // 8 elements
  const int lane = threadIdx.x & 31;
  const int G = a.D / 8, Gc = a.d_c / 8;
  const int ps = a.slot.page_size;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  const long n_warps = (long)gridDim.x * kWarps;
  for (long t0 = ((long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kReadTokens; t0 < a.T;
       t0 += n_warps * kReadTokens) {
    long mine = -1;
    if (lane < kReadTokens && t0 + lane < a.T) {
      mine = a.slot(a.seq_idx[t0 + lane], a.pos[t0 + lane]);
      if (mine < 0) record_error(MLA_ERR_BAD_PAGE);
    }
    Raw raw[kReadTokens][kGroups];
    float2 sc[kReadTokens];
#pragma unroll
    for (int u = 0; u < kReadTokens; ++u) {
      const long slot = __shfl_sync(0xffffffffu, mine, u);
      const uint8_t* src;
      if constexpr (kFp8) {
        const long page = slot / ps;
        const int row = (int)(slot - page * ps);
        const uint8_t* pg = static_cast<const uint8_t*>(a.pool) + page * fp8::page_bytes(ps, a.D);
        src = pg + (long)row * a.D;
        sc[u] = slot >= 0 ? *reinterpret_cast<const float2*>(pg + (long)ps * a.D + 8 * row) : make_float2(0.f, 0.f);
      } else {
        src = static_cast<const uint8_t*>(a.pool) + slot * a.D * (long)sizeof(T);
      }
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int g = lane + 32 * i;
        raw[u][i] = slot >= 0 && g < G ? *reinterpret_cast<const Raw*>(src + sizeof(Raw) * g) : Raw{};
      }
    }
#pragma unroll
    for (int u = 0; u < kReadTokens; ++u) {
      if (t0 + u >= a.T) break;
      T* dst = static_cast<T*>(a.out) + (t0 + u) * a.out_stride;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int g = lane + 32 * i;
        if (g >= G) continue;
        uint4 o;
        if constexpr (kFp8) {
          // value = scale * e4m3 in fp32 (the e4m3 value is exact in fp16), rounded once
          const float s = g < Gc ? sc[u].x : sc[u].y;
          const uint32_t in[2] = {raw[u][i].x, raw[u][i].y};
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2_raw hr =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(in[e >> 1] >> (16 * (e & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
            const P2 two = Pack<T>::make(f.x * s, f.y * s);
            w[e] = *reinterpret_cast<const uint32_t*>(&two);
          }
          o = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          o = raw[u][i];
        }
        *reinterpret_cast<uint4*>(dst + 8 * g) = o;
      }
    }
  }
}

}  // namespace mla
