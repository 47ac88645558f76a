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
constexpr int kLatGroups = 2; // 8-element groups of the latent part per lane: d_c <= 512
constexpr int kMaxR = 9;      // pairs of the rotated part per lane: d_rope / 2 <= 284 <= 32 kMaxR
constexpr int kPowers = 9;    // 32 kMaxR < 2^9
constexpr int kWarps = 8;     // per CTA
// CTAs per SM at most; warps then loop over tokens. A writer keeps what is the same for every token
// in registers and requests a token ahead: as many CTAs as fit (8192 tokens to e4m3: 6.9 us with
// three, 7.5 with four, 10.2 with five at 48 registers a thread, 7.5 with eight of which three fit).
// A reader has nothing to keep (131072 tokens: 41.9 us).
constexpr int kAppendPerSm = 3, kReadPerSm = 32;

// Page and row in it of position p of sequence s; page -1 if it is outside the table or the pool.
struct Slot {
  int page, row;
};
struct SlotMap {
  const int* bt;  // [num_seqs, max_pages]
  int num_seqs, max_pages, num_pages, page_size;
  __device__ __forceinline__ Slot operator()(int s, int p) const {
    if (s < 0 || s >= num_seqs || p < 0) return {-1, 0};
    const int lp = p / page_size;
    if (lp >= max_pages) return {-1, 0};
    const int page = bt[(long)s * max_pages + lp];
    return {page < num_pages ? page : -1, p - lp * page_size};  // (a negative entry stays negative)
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
// arithmetic. A lane holds kC groups of 8 latent values and kR pairs of the rotated part: one pair
// to a lane at d_rope <= 64, so that a token's cosines and sines are formed by 32 lanes at once.
// What a lane needs of the gains and the frequencies (doubles) is the same for every token and
// stays in its registers.
template <typename T, bool kFp8, int kR>
__global__ void __launch_bounds__(32 * rows::kWarps, kR == 1 ? rows::kAppendPerSm : 1) k_norm_append(const rows::AppendArgs a) {
  using namespace rows;
  using P2 = typename Pack<T>::T2;
  constexpr int kC = kLatGroups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Gc = a.d_c / 8, pairs = (a.D - a.d_c) / 2;
  double turns[kR];
#pragma unroll
  for (int j = 0; j < kR; ++j)  // from the arguments alone: ahead of the wait
    turns[j] = a.turns.table == nullptr ? a.turns(lane + 32 * j) : 0.0;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  uint4 gc[kC];
  uint32_t gr[kR];
#pragma unroll
  for (int i = 0; i < kC; ++i)
    gc[i] = a.g_c != nullptr && lane + 32 * i < Gc ? ldg16(static_cast<const T*>(a.g_c) + 8 * (lane + 32 * i))
                                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < kR; ++j) {
    const int k = lane + 32 * j;
    gr[j] = a.g_r != nullptr && k < pairs ? __ldg(static_cast<const uint32_t*>(a.g_r) + k) : 0u;
    if (a.turns.table != nullptr && k < pairs) turns[j] = a.turns(k);
  }
  auto two = [](uint32_t w) { return Pack<T>::f2(*reinterpret_cast<const P2*>(&w)); };
  const int n_warps = gridDim.x * kWarps;
  int t = blockIdx.x * kWarps + warp;
  uint4 raw_c[kC];
  uint32_t raw_r[kR];
  int p = 0, seq = 0;
  auto request = [&](int tt) {
    if (tt >= a.T) return;
    const T* src = static_cast<const T*>(a.x) + (long)tt * a.x_stride;
    p = a.pos[tt];
    seq = a.seq_idx[tt];
#pragma unroll
    for (int i = 0; i < kC; ++i)
      raw_c[i] = lane + 32 * i < Gc ? *reinterpret_cast<const uint4*>(src + 8 * (lane + 32 * i)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < kR; ++j)
      raw_r[j] = lane + 32 * j < pairs ? *reinterpret_cast<const uint32_t*>(src + a.d_c + 2 * (lane + 32 * j)) : 0u;
  };
  request(t);
  for (; t < a.T; t += n_warps) {
    const int pos = p;
    const Slot at = a.slot(seq, pos);  // used at the end: the table's read overlaps the arithmetic
    float v[kC][8];
    float2 r[kR];
#pragma unroll
    for (int i = 0; i < kC; ++i) unpack8<T>(raw_c[i], v[i]);
#pragma unroll
    for (int j = 0; j < kR; ++j) r[j] = two(raw_r[j]);
    request(t + n_warps);
    if (a.g_c != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
      const float rs = rsqrtf(warp_sum(ss) / (float)a.d_c + a.eps);
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        float gf[8];
        unpack8<T>(gc[i], gf);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * rs * gf[e];
      }
    }
    if (a.g_r != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < kR; ++j) ss = fmaf(r[j].x, r[j].x, fmaf(r[j].y, r[j].y, ss));
      const float rs = rsqrtf(warp_sum(ss) / (float)(a.D - a.d_c) + a.eps);
#pragma unroll
      for (int j = 0; j < kR; ++j) {
        const float2 g = two(gr[j]);
        r[j] = make_float2(r[j].x * rs * g.x, r[j].y * rs * g.y);
      }
    }
#pragma unroll
    for (int j = 0; j < kR; ++j) {
      float c, s;
      turn_cos_sin(pos, turns[j], c, s);
      r[j] = make_float2(r[j].x * c - r[j].y * s, r[j].x * s + r[j].y * c);
    }
    float mc = 0.f, mr = 0.f;
    if constexpr (kFp8) {  // non-negative floats order as their bit patterns
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) mc = fmaxf(mc, fabsf(v[i][e]));
#pragma unroll
      for (int j = 0; j < kR; ++j) mr = fmaxf(mr, fmaxf(fabsf(r[j].x), fabsf(r[j].y)));
      mc = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mc)));
      mr = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mr)));
    }
    if (at.page < 0) {
      if (lane == 0) record_error(MLA_ERR_BAD_PAGE);
      continue;
    }
    if constexpr (!kFp8) {
      T* dst = static_cast<T*>(a.pool) + ((long)at.page * a.slot.page_size + at.row) * a.D;
#pragma unroll
      for (int i = 0; i < kC; ++i)
        if (lane + 32 * i < Gc) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const P2 pk = Pack<T>::make(v[i][2 * e], v[i][2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&pk);
          }
          *reinterpret_cast<uint4*>(dst + 8 * (lane + 32 * i)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
      for (int j = 0; j < kR; ++j)
        if (lane + 32 * j < pairs)
          *reinterpret_cast<P2*>(dst + a.d_c + 2 * (lane + 32 * j)) = Pack<T>::make(r[j].x, r[j].y);
    } else {
      // 1 for an all-zero part, and for one so small (below 2^-141) that fp32 holds its scale as zero
      const float qc = mc / fp8::kE4m3Max, qr = mr / fp8::kE4m3Max;
      const float sc = qc > 0.f ? qc : 1.f, sr = qr > 0.f ? qr : 1.f;
      const float ic = 1.f / sc, ir = 1.f / sr;
      // scales whose reciprocal or whose products with values are not normal divide as they are
      const bool plain = !(fminf(sc, sr) > 0x1p-100f && fmaxf(sc, sr) < 0x1p100f);
      const int ps = a.slot.page_size;
      uint8_t* const pg = static_cast<uint8_t*>(a.pool) + at.page * fp8::page_bytes(ps, a.D);
      uint8_t* const dst = pg + (long)at.row * a.D;
      auto store = [&](auto divide) {
        auto e4m3x2 = [&](float x, float y, float s, float inv) {
          return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(divide(x, s, inv), divide(y, s, inv)), __NV_SATFINITE,
                                                    __NV_E4M3);
        };
#pragma unroll
        for (int i = 0; i < kC; ++i)
          if (lane + 32 * i < Gc) {
            const float* x = v[i];
            *reinterpret_cast<uint2*>(dst + 8 * (lane + 32 * i)) =
                make_uint2(e4m3x2(x[0], x[1], sc, ic) | (e4m3x2(x[2], x[3], sc, ic) << 16),
                           e4m3x2(x[4], x[5], sc, ic) | (e4m3x2(x[6], x[7], sc, ic) << 16));
          }
#pragma unroll
        for (int j = 0; j < kR; ++j)
          if (lane + 32 * j < pairs)
            *reinterpret_cast<uint16_t*>(dst + a.d_c + 2 * (lane + 32 * j)) = (uint16_t)e4m3x2(r[j].x, r[j].y, sr, ir);
      };
      if (plain) store([](float x, float s, float) { return x / s; });
      else store([](float x, float s, float inv) { return quotient(x, s, inv); });
      if (lane == 0) *reinterpret_cast<float2*>(pg + (long)ps * a.D + 8L * at.row) = make_float2(sc, sr);
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

// A warp per token. Bound by the writes: 151 MB of rows out of 76 MB of e4m3 pages take 41.9 us, and
// setting 151 MB to zero takes 41.5 (3.6 TB/s; the reads run beside it). Two, four or eight tokens to
// a warp at a time, or stores that do not stay in L2, were no faster; 1021 tokens then took 2.6, 3.2
// and 4.6 us against 2.0. A token without a valid slot becomes a zero row and records MLA_ERR_BAD_PAGE.
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
  const int n_warps = gridDim.x * kWarps;
  for (int t = blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += n_warps) {
    const Slot at = a.slot(a.seq_idx[t], a.pos[t]);
    const bool there = at.page >= 0;
    if (!there && lane == 0) record_error(MLA_ERR_BAD_PAGE);
    Raw raw[kGroups];
    float2 sc = make_float2(0.f, 0.f);
    const uint8_t* src;
    if constexpr (kFp8) {
      const uint8_t* pg = static_cast<const uint8_t*>(a.pool) + at.page * fp8::page_bytes(ps, a.D);
      src = pg + (long)at.row * a.D;
      if (there) sc = *reinterpret_cast<const float2*>(pg + (long)ps * a.D + 8L * at.row);
    } else {
      src = static_cast<const uint8_t*>(a.pool) + ((long)at.page * ps + at.row) * a.D * (long)sizeof(T);
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int g = lane + 32 * i;
      raw[i] = there && g < G ? *reinterpret_cast<const Raw*>(src + sizeof(Raw) * g) : Raw{};
    }
    T* dst = static_cast<T*>(a.out) + (long)t * a.out_stride;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int g = lane + 32 * i;
      if (g >= G) continue;
      uint4 o;
      if constexpr (kFp8) {
        // value = scale * e4m3 in fp32 (the e4m3 value is exact in fp16), rounded once
        const float s = g < Gc ? sc.x : sc.y;
        const uint32_t in[2] = {raw[i].x, raw[i].y};
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
        o = raw[i];
      }
      *reinterpret_cast<uint4*>(dst + 8 * g) = o;
    }
  }
}

}  // namespace mla
