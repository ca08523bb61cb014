// The single-token step of the softmax attention on a paged cache.
//
// A row's keys and values are read once, 2 D bytes of 8 bits or twice that of bf16 for
// each token and key head, and serve the HQ / HKV query heads of the group: the bound is
// HBM. The heads of a group (up to 16) are the rows of a warp-level tensor-core product
// of m16n8k16, whose 16 tokens a step lie in one page: a warp loads them (4 KB of keys,
// 4 KB of values at D = 128 in bf16) with 16-byte asynchronous copies, several steps
// ahead, into shared memory of its own, keeps its own running maximum and sum, and no
// barrier stands in its loop. The warps of a CTA, and the CTAs of a cluster that split
// a row's tokens between them, join their results at the end, in a fixed order. So are, in
// a workspace, the results of several clusters on a row and of the prefix that all rows
// share, which the prompt kernel computes beside the rows' own tokens.
//
// 8-bit keys and values become f16, exactly; a token's key scale multiplies its scores in
// fp32, and the logarithm of its value scale is added to the score that its weight for the
// product with the values comes from. These weights are rounded to f16, and to bf16 with a
// bf16 cache; the sum takes unrounded ones. f16 holds the largest weight times scale at 2^15;
// tokens more than 2^32 below it have products of their own (a head of zeros has the scale 1,
// far above others', and sets that maximum though it adds nothing). 256 rows of about 2000
// tokens: 191 us, as without the look for such tokens; cold caches: 205 us, and 278 where a head
// of zeros is 40 nats above all others of every row.
#include "kda_attn.cuh"
#include "kda_attn_fwd.h"
#include "kda_cluster.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kGroup = 16;       // tokens that the products take at once; divides every page
constexpr int kMaxSplits = 8;    // CTAs of a cluster
// The f16 weights of 8-bit values: 2^kTopWeight is the largest, and down to kWeightBits below it,
// 2^-17, a rounding is at most 2^-8 (half of f16's smallest step, 2^-24). Smaller ones are taken in
// kParts - 1 further parts, each kWeightBits wide: to 2^-128 of the largest.
constexpr float kTopWeight = 15.f;
constexpr int kWeightBits = 32, kParts = 4;

struct Params {
  kda_attn_step_args a;
  int G, head_tiles;
  int page_bits;          // page_size = 2^page_bits
  int splits, chunks;     // CTAs of a cluster and clusters on each row and key head (and tile of its heads)
  const float* part_o;    // [parts, B, HQ, D]: results to join, normalised: the clusters' where a
  const float* part_lse;  // row has several, and the prefix's; [parts, B, HQ], in powers of two
  int parts;
  float* own_o;           // the clusters' part of them; nullptr: the one cluster of a row writes o
  float* own_lse;
};

template <int D, bool E4, int WARPS, bool MANY>
struct Shape {
  static constexpr int kRow = D * (E4 ? 1 : 2);                        // bytes of a token
  // Groups of a warp's step: two of 8-bit tokens (the same bytes as one of bf16; with one,
  // what a step costs besides its products kept 256 rows of 2000 tokens at 262 us). MANY: one,
  // so that three CTAs fit an SM (plan_of).
  static constexpr int kSub = E4 && !MANY ? 2 : 1;
  static constexpr int kTokens = kSub * kGroup;
  static constexpr int kStage = 2 * kTokens * kRow + (E4 ? 8 * kTokens : 0);  // keys, values, scales of both
  static constexpr int kStages = D == 128 ? (MANY ? 4 : 3) : 6;
  static constexpr int kResult = (D + 4) * 64 + 16 / WARPS * D * 4;  // a warp's result, and rows of the CTA's
  static constexpr int kWarpBytes = kStages * kStage > kResult ? kStages * kStage : kResult;
  static constexpr int kSmem = WARPS * kWarpBytes;
};

// 16-byte piece c of token row r: the pieces of 8 rows that an access takes together lie
// in different banks.
template <int ROW>
__device__ __forceinline__ int piece(int r, int c) {
  return r * ROW + ((ROW >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void copy16(unsigned char* dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(dst)), "l"(src), "r"(real ? 16 : 0));
}

// Two e4m3 values (the low or the high half of w) as f16, exactly; NaN stays NaN.
__device__ __forceinline__ uint32_t low_f16(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t high_f16(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// One partial result (sum l and weighted values o, relative to 2^m) joined to another. A part
// without keys has m = -inf and l = 0 and changes nothing.
struct Joined {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float pm, float pl, float4 po) {
    if (pm == -INFINITY && pl == 0.f) return;
    const float top = pm > m ? pm : m;
    const float a = m == -INFINITY ? 0.f : exp2f(m - top);
    const float b = pm == -INFINITY ? 0.f : pm == top ? 1.f : exp2f(pm - top);
    m = top;
    l = l * a + pl * b;
    o.x = weighed(o.x, a) + weighed(po.x, b), o.y = weighed(o.y, a) + weighed(po.y, b);
    o.z = weighed(o.z, a) + weighed(po.z, b), o.w = weighed(o.w, a) + weighed(po.w, b);
  }
};

// Two weights as an operand.
template <bool E4>
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  if (!E4) return Bf16::pack(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What results under the maximum `was` are worth under `now`.
__device__ __forceinline__ float factor(float was, float now) { return was == now ? 1.f : was == -INFINITY ? 0.f : ex2_approx(was - now); }

// Adds the results in the workspace for a row and head, 4 channels from d. A logarithm of -inf
// is a part without keys, or with keys that weigh nothing, which has NaN as its values: where
// no other part has a weight the row is NaN (0 / 0), otherwise they change nothing.
template <int D>
__device__ __forceinline__ void join_parts(const Params& p, long long b, int head, int d, Joined& j, int& any) {
  constexpr int kAtOnce = 4;  // loads in flight together
  for (int s0 = 0; s0 < p.parts; s0 += kAtOnce) {
    float lse[kAtOnce];
    float4 o[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const long long at = (static_cast<long long>(min(s0 + i, p.parts - 1)) * p.a.B + b) * p.a.HQ + head;
      lse[i] = s0 + i < p.parts ? __ldcg(p.part_lse + at) : -INFINITY;
      o[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + d));
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (lse[i] == -INFINITY) {
        any |= o[i].x != o[i].x;
        continue;
      }
      any = 1;
      // (2^-8 each: with up to 70 parts, sums of weighted values stay below the largest)
      j.add(lse[i] + 8.f, 0x1p-8f, make_float4(o[i].x * 0x1p-8f, o[i].y * 0x1p-8f, o[i].z * 0x1p-8f, o[i].w * 0x1p-8f));
    }
  }
}

template <int D>
__device__ __forceinline__ void store_row(const kda_attn_step_args& a, long long b, int head, int d, const Joined& j, int any) {
  // (keys whose scores are all -inf: 0 / 0, as the definition has it)
  const float inv = 1.f / j.l;
  uint2 w = make_uint2(0u, 0u);
  if (any) w = make_uint2(Bf16::pack(j.o.x * inv, j.o.y * inv), Bf16::pack(j.o.z * inv, j.o.w * inv));
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + b * a.o_stride + static_cast<long long>(head) * D + d) = w;
  if (a.lse && d == 0) a.lse[b * a.HQ + head] = any ? (j.m + log2f(j.l)) * kLn2 : -INFINITY;
}

// Rows that several clusters, or the prefix and several clusters, worked on.
template <int D>
__global__ void __launch_bounds__(128) kda_attn_join_kernel(const __grid_constant__ Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long u = static_cast<long long>(blockIdx.x) * 128 + threadIdx.x, r = u / (D / 4);
  if (r >= static_cast<long long>(p.a.B) * p.a.HQ) return;
  const long long b = r / p.a.HQ;
  const int head = static_cast<int>(r % p.a.HQ), d = static_cast<int>(u % (D / 4)) * 4, len = p.a.seq_lens[b];
  Joined j;
  int any = 0;
  if (len >= 0 && len <= p.a.table_width * p.a.page_size) join_parts<D>(p, b, head, d, j, any);
  store_row<D>(p.a, b, head, d, j, any);
}

// (Where there are many CTAs, as many fit an SM as the registers can be held to without spills: with
// 64 channels and up to 8 heads four, 256 rows of about 2000 tokens 134 us, cold; 148 with three.)
template <int D, bool E4, int WARPS, bool MANY, int ROWS>
__global__ void __launch_bounds__(32 * WARPS, MANY ? (D == 64 && ROWS == 1 ? 4 : 3) : 1) kda_attn_step_kernel(const __grid_constant__ Params p) {
  using Sh = Shape<D, E4, WARPS, MANY>;
  constexpr int kThreads = 32 * WARPS;
  extern __shared__ __align__(128) unsigned char raw[];
  __shared__ float cta_m[16], cta_l[16];
  __shared__ float warp_m[WARPS][16], warp_l[WARPS][16];
  __shared__ int cta_used;

  const kda_attn_step_args& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x % (p.splits * p.chunks)), in_cluster = rank % p.splits;  // of the row's CTAs
  long long unit = blockIdx.x / (p.splits * p.chunks);
  const int tile = static_cast<int>(unit % p.head_tiles);
  unit /= p.head_tiles;
  const int h = static_cast<int>(unit % a.HKV);
  const int b = static_cast<int>(unit / a.HKV);
  const int head0 = h * p.G + tile * 16, heads = min(16, p.G - tile * 16);

  // pages of this warp's next 32 groups, one a lane; the first ones are asked for before the
  // row's length is there (entries behind its last page are not used)
  constexpr int T = Sh::kTokens;
  const int first = rank * WARPS + warp, step = p.chunks * p.splits * WARPS;  // of the row's steps of T tokens
  const int32_t* table = a.block_table + static_cast<long long>(b) * a.table_width;
  int pages = 0;
  {
    const long long tok = static_cast<long long>(first + lane / Sh::kSub * step) * T + lane % Sh::kSub * kGroup;
    if (tok < static_cast<long long>(a.table_width) << p.page_bits) pages = table[tok >> p.page_bits];
  }

  int len = a.seq_lens[b];
  const bool row = len >= 0 && len <= a.table_width * a.page_size;
  if (!row) {
    if (len >= 0 && tid == 0) set_err(a.err, KDA_ERR_INVALID_ARG);
    len = 0;
  }
  if (tid == 0) cta_used = 0;
  const float below = below_one(len);

  // queries as the products' A operand: heads g and g + 8; channels 16 k + 2 t, + 1 and
  // + 8, + 9 for bf16 keys, the 4 from 16 k + 4 t for 8-bit ones (an order of the sum
  // that gives a lane four consecutive bytes of a key). With 8-bit keys they are f16, as
  // the keys are (e4m3 fits it), after a power of two of the head's own that brings the
  // largest to 2^10 .. 2^11: what falls below f16's range is 2^-34 of that.
  uint32_t q[D / 16][4];
  float c2[2] = {a.scale * kLog2e, a.scale * kLog2e};  // of the two heads: to scores in powers of two
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int head = g + 8 * r;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_stride + static_cast<long long>(head0 + head) * D;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint2 w = make_uint2(0u, 0u);
      if (head < heads) {
        if (E4) w = *reinterpret_cast<const uint2*>(x + 16 * k + 4 * t);
        else w = make_uint2(*reinterpret_cast<const uint32_t*>(x + 16 * k + 2 * t), *reinterpret_cast<const uint32_t*>(x + 16 * k + 2 * t + 8));
      }
      q[k][r] = w.x;
      q[k][2 + r] = w.y;
    }
    if (E4) {
      float most = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int u = r; u < 4; u += 2) {
          most = max_nan(most, fabsf(__uint_as_float(q[k][u] << 16)));
          most = max_nan(most, fabsf(__uint_as_float(q[k][u] & 0xffff0000u)));
        }
      }
      most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // 2^(10 - e) of the largest's exponent e (as two factors: one may leave the range)
      const int e = static_cast<int>(__float_as_uint(most) >> 23);
      const int by = e == 0 || e == 255 ? 0 : 137 - e, b1 = by / 2, b2 = by - b1;
      const float f1 = __uint_as_float(static_cast<uint32_t>(127 + b1) << 23), f2 = __uint_as_float(static_cast<uint32_t>(127 + b2) << 23);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int u = r; u < 4; u += 2) {
          const __half2 h = __floats2half2_rn(__uint_as_float(q[k][u] << 16) * f1 * f2, __uint_as_float(q[k][u] & 0xffff0000u) * f1 * f2);
          q[k][u] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      c2[r] = c2[r] * (1.f / f1) * (1.f / f2);
    }
  }

  unsigned char* ring = raw + warp * Sh::kWarpBytes;
  const int all = (len + T - 1) / T;  // the row's steps; this warp has every (CTAs of the row x WARPS)-th
  const int steps = all > first ? (all - first + step - 1) / step : 0;
  uint32_t bad = 0;  // by stage and group: its page is out of range
  bool any_bad = false;
  auto load = [&](int i) {
    const int s = i % Sh::kStages;
    unsigned char* dst = ring + s * Sh::kStage;
#pragma unroll
    for (int u = 0; u < Sh::kSub; ++u) {
      const int at0 = i * Sh::kSub + u;
      if (at0 % 32 == 0 && at0 > 0) {
        const int at = at0 + lane, tok = (first + at / Sh::kSub * step) * T + at % Sh::kSub * kGroup;
        pages = at < steps * Sh::kSub && tok < len ? table[tok >> p.page_bits] : 0;
      }
      const int page = __shfl_sync(0xffffffffu, pages, at0 % 32), bit = s * Sh::kSub + u;
      const int tok = (first + i * step) * T + u * kGroup;
      const bool there = tok < len, good = there && page >= 0 && page < a.pages;
      bad = good || !there ? bad & ~(1u << bit) : bad | 1u << bit;
      any_bad |= there && !good;
      const long long at = good ? ((static_cast<long long>(page) * a.HKV + h) << p.page_bits) + (tok & (a.page_size - 1)) : 0;
      const int real = good ? min(kGroup, len - tok) : 0;
      constexpr int C = Sh::kRow / 16;
      const unsigned char* ks = static_cast<const unsigned char*>(a.k_cache) + at * Sh::kRow + 16 * lane;
      const unsigned char* vs = static_cast<const unsigned char*>(a.v_cache) + at * Sh::kRow + 16 * lane;
      unsigned char* to = dst + u * kGroup * Sh::kRow;
      if (real == kGroup) {
#pragma unroll
        for (int j = 0; j < kGroup * C / 32; ++j) {
          const int n = 32 * j + lane, at_piece = piece<Sh::kRow>(n / C, n % C);
          cp_async16(to + at_piece, ks + 512 * j);
          cp_async16(to + T * Sh::kRow + at_piece, vs + 512 * j);
        }
      } else {  // tokens that are not there become zeros
#pragma unroll
        for (int j = 0; j < kGroup * C / 32; ++j) {
          const int n = 32 * j + lane, r = n / C, at_piece = piece<Sh::kRow>(r, n % C);
          copy16(to + at_piece, r < real ? static_cast<const void*>(ks + 512 * j) : a.q, r < real);
          copy16(to + T * Sh::kRow + at_piece, r < real ? static_cast<const void*>(vs + 512 * j) : a.q, r < real);
        }
      }
      if (E4 && lane < 8)
        copy16(dst + 2 * T * Sh::kRow + (lane / 4) * 4 * T + u * 4 * kGroup + 16 * (lane & 3),
               good ? static_cast<const void*>((lane < 4 ? a.k_scale : a.v_scale) + at + 4 * (lane & 3)) : a.q, good);
    }
  };

  // running maximum of the scores, sum of the weights, and, with 8-bit values, the maximum of the
  // weights times their values' scales, of which o is relative to 2^-kTopWeight (its own otherwise)
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, mv[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  bool used = false;

#pragma unroll
  for (int i = 0; i < Sh::kStages - 1; ++i) {
    if (i < steps) load(i);
    cp_async_commit();
  }
  for (int i = 0; i < steps; ++i) {
    cp_async_wait<Sh::kStages - 2>();
    __syncwarp();
    const int s = i % Sh::kStages;
    const unsigned char* ks = ring + s * Sh::kStage;
    const unsigned char* vs = ks + T * Sh::kRow;
    constexpr int U = Sh::kSub, N = 2 * U;  // groups; products' 8 tokens
    int real[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      real[u] = (bad >> (s * U + u) & 1u) ? 0 : min(kGroup, len - (first + i * step) * T - u * kGroup);
      used |= real[u] > 0;
    }

    float sc[N][4], sd[N][4];  // (two sums each: a product waits for the one before it)
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[n][e] = sd[n][e] = 0.f;
    }
    if (E4) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(ks + piece<Sh::kRow>(8 * n + g, k) + 4 * t);
          mma16816<F16>(k % 2 ? sd[n] : sc[n], q[k], low_f16(w), high_f16(w));
        }
      }
    } else {
      const int r = (lane & 7) + (lane >> 4) * 8, c = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t w[4];
        ldsm_x4(w, ks + piece<Sh::kRow>(r, 2 * k + c));
        mma16816<Bf16>(k % 2 ? sd[0] : sc[0], q[k], w[0], w[1]);
        mma16816<Bf16>(k % 2 ? sd[1] : sc[1], q[k], w[2], w[3]);
      }
    }
    // scores in powers of two; tokens that are not there weigh nothing
    const float* scales = reinterpret_cast<const float*>(vs + T * Sh::kRow);
    float top[2] = {m[0], m[1]}, topv[2] = {mv[0], mv[1]};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float lv[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) lv[e] = E4 ? lg2_approx(scales[T + 8 * n + 2 * t + e]) : 0.f;
#pragma unroll
      for (int e = 0; e < 2 * ROWS; ++e) {
        const int tok = 8 * n + 2 * t + (e & 1);
        const float x = (sc[n][e] + sd[n][e]) * (E4 ? scales[tok] * c2[e >> 1] : c2[e >> 1]);
        sc[n][e] = tok % kGroup < real[n / 2] ? x : -INFINITY;
        top[e >> 1] = fmaxf(top[e >> 1], sc[n][e]);
        if (E4) {
          sd[n][e] = tok % kGroup < real[n / 2] ? x + lv[e & 1] : -INFINITY;
          topv[e >> 1] = fmaxf(topv[e >> 1], sd[n][e]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      if (E4) topv[r] = fmaxf(topv[r], __shfl_xor_sync(0xffffffffu, topv[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      if (E4) topv[r] = fmaxf(topv[r], __shfl_xor_sync(0xffffffffu, topv[r], 2));
    }
    if (__any_sync(0xffffffffu, top[0] > m[0] || topv[0] > mv[0] || (ROWS > 1 && (top[1] > m[1] || topv[1] > mv[1])))) {
      float keep[2];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        keep[r] = factor(m[r], top[r]);
        m[r] = top[r];
        l[r] *= keep[r];
        if (E4) {
          keep[r] = factor(mv[r], topv[r]);
          mv[r] = topv[r];
        }
      }
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][0] *= keep[0], o[j][1] *= keep[0];
        if (ROWS > 1) o[j][2] *= keep[1], o[j][3] *= keep[1];
      }
    }
    const float mz[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
    const float mvz[2] = {mv[0] == -INFINITY ? 0.f : mv[0] - kTopWeight, mv[1] == -INFINITY ? 0.f : mv[1] - kTopWeight};
    // by their bits, exponents of weights below the limit and above -inf: from the limit's own
    // bits (0) up to those of -inf; all other values, NaN among them, come out larger
    constexpr float kLimit = kTopWeight - kWeightBits;
    const uint32_t limit = __float_as_uint(kLimit), past = __float_as_uint(-INFINITY) - limit;
    uint32_t small = past;
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int e = 0; e < 2 * ROWS; ++e) {
        float w = ex2_approx(sc[n][e] - mz[e >> 1]);
        l[e >> 1] += w;
        if (E4) {
          const float y = sd[n][e] - mvz[e >> 1];
          small = min(small, __float_as_uint(y) - limit);
          w = ex2_approx(y);
        }
        sc[n][e] = w;
      }
    }
    // With weights below the limit: those in f16's reach first, then the next kWeightBits as if they
    // were and what is summed so far lifted with them, and so on while the sums have room: they are
    // up to 2^53 (2^15 * 448 for 2^29 tokens), which two lifts leave below 2^117. Heads that are all
    // but zeros, whose small weights count, have room for the third. In one loop: a second copy
    // of the products took 40 registers more.
    const int parts = E4 && __any_sync(0xffffffffu, small < past) ? kParts : 1;
    float most = 0.f;  // of the sums
#pragma unroll 1
    for (int part = 0;;) {
      if (E4 && parts > 1) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
          for (int e = 0; e < 2 * ROWS; ++e) {
            const float y = sd[n][e] - mvz[e >> 1] + static_cast<float>(kWeightBits * part);
            const bool here = part == 0 ? !(y < kLimit) : y < kTopWeight && y >= kLimit;
            sc[n][e] = here ? ex2_approx(y) : 0.f;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t pa[4] = {pack_weights<E4>(sc[2 * u][0], sc[2 * u][1]), ROWS == 1 ? 0u : pack_weights<E4>(sc[2 * u][2], sc[2 * u][3]),
                                pack_weights<E4>(sc[2 * u + 1][0], sc[2 * u + 1][1]),
                                ROWS == 1 ? 0u : pack_weights<E4>(sc[2 * u + 1][2], sc[2 * u + 1][3])};
        const int r = u * kGroup + (lane & 7) + ((lane >> 3) & 1) * 8, c = lane >> 4;
        if (E4) {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {  // 32 channels: even and odd ones of each 16 in tiles of their own
            uint32_t w[4];
            ldsm_x4_trans(w, vs + piece<Sh::kRow>(r, 2 * j + c));
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = __byte_perm(w[x], 0u, 0x3120);
            mma16816<F16>(o[4 * j], pa, low_f16(w[0]), low_f16(w[1]));
            mma16816<F16>(o[4 * j + 1], pa, high_f16(w[0]), high_f16(w[1]));
            mma16816<F16>(o[4 * j + 2], pa, low_f16(w[2]), low_f16(w[3]));
            mma16816<F16>(o[4 * j + 3], pa, high_f16(w[2]), high_f16(w[3]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t w[4];
            ldsm_x4_trans(w, vs + piece<Sh::kRow>(r, 2 * j + c));
            mma16816<Bf16>(o[2 * j], pa, w[0], w[1]);
            mma16816<Bf16>(o[2 * j + 1], pa, w[2], w[3]);
          }
        }
      }
      if (!E4 || parts == 1) break;
      ++part;
      const bool more = part < kParts && __all_sync(0xffffffffu, most < 0x1p89f);  // (and this part's products below 2^54)
      const float by = __uint_as_float(static_cast<uint32_t>(127 + (more ? 1 : 1 - part) * kWeightBits) << 23);
      most = 0.f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
#pragma unroll
        for (int e = 0; e < 2 * ROWS; ++e) o[j][e] *= by, most = fmaxf(most, fabsf(o[j][e]));
      }
      if (!more) break;
    }
    __syncwarp();
    if (i + Sh::kStages - 1 < steps) load(i + Sh::kStages - 1);
    cp_async_commit();
  }
  cp_async_wait<0>();
  // Results relative to 2^below times the maximum's weight: what the joins add up over the row stays
  // below the largest value. (8 bits: o is relative to the maximum of its own so far. In two factors:
  // one might leave the range.)
  const float down = exp2f(-below);
  bool redo[2] = {false, false};
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const float by = !E4 || mv[r] == m[r] ? 1.f : mv[r] == -INFINITY ? 0.f : exp2f(mv[r] - m[r]), f = E4 ? down * exp2f(-kTopWeight) : down;
    float finite = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
#pragma unroll
      for (int e = 2 * r; e < 2 * r + 2; ++e) {
        finite = fmaf(o[j][e], 0.f, finite);
        o[j][e] = o[j][e] * f * by;
      }
    }
    redo[r] = !E4 && finite != finite;
    l[r] *= down;
  }
  if (any_bad && lane == 0) set_err(a.err, KDA_ERR_INVALID_ARG);

  // this warp's result: its ring now holds the weighted values [16][D + 4]
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  __syncwarp();
  float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = E4 ? 16 * (j / 2) + 4 * t + 2 * (e & 1) + (j & 1) : 8 * j + 2 * t + (e & 1);
      mine[(g + 8 * (e >> 1)) * (D + 4) + d] = o[j][e];
    }
  }
  if (t == 0) {
    warp_m[warp][g] = m[0] + below, warp_m[warp][g + 8] = m[1] + below;
    warp_l[warp][g] = l[0], warp_l[warp][g + 8] = l[1];
  }
  if (!E4) {
    // Heads that an infinity, or a sum past fp32, is in, again, one by one: a weight that rounds to 0
    // made NaN of an infinite value. (Weights held above 0 instead gave values of 1e38 weights that
    // they do not have.) Where the sum of the weights is NaN the results are.
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      uint32_t again = __ballot_sync(0xffffffffu, redo[r] && l[r] == l[r] && g + 8 * r < heads);
      while (again != 0) {
        const int head = (__ffs(again) - 1) / 4;
        again &= ~(0xfu << (4 * head));
        const int row = head + 8 * r;
        const Keys keys = {a.k_cache, a.v_cache, table, a.pages, a.page_size, a.HKV, 0, 0, 0};
        const int last = (first + (steps - 1) * step) * T, count = (steps - 1) * T + min(T, len - last);  // of this warp's tokens
        float x[D / 32], y[D / 32], rm, rl;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          x[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[b * a.q_stride + static_cast<long long>(head0 + row) * D + lane + 32 * c]);
        attend_row<D>(x, keys, h, count, [first, step](int j) { return (first + j / T * step) * T + j % T; }, below, a.scale * kLog2e, lane, a.err, rm, rl, y);
        __syncwarp();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) mine[row * (D + 4) + lane + 32 * c] = y[c];
        if (lane == 0) warp_m[warp][row] = rm, warp_l[warp][row] = rl;
      }
    }
  }
  __syncthreads();
  if (used && lane == 0) cta_used = 1;
  constexpr int Q = D / 4;  // 4 channels at a time
  // the CTA's result lies behind its warps', some rows behind each
  constexpr int kEach = 16 / WARPS;
  const auto cta_o = [&](int r, int d) {
    return reinterpret_cast<float*>(raw + r / kEach * Sh::kWarpBytes + (D + 4) * 64) + r % kEach * D + d;
  };
  for (int u = tid; u < heads * Q; u += kThreads) {
    const int r = u / Q, d = 4 * (u % Q);
    Joined j;
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      j.add(warp_m[w][r], warp_l[w][r], *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(raw + w * Sh::kWarpBytes) + r * (D + 4) + d));
    *reinterpret_cast<float4*>(cta_o(r, d)) = j.o;
    if (d == 0) cta_m[r] = j.m, cta_l[r] = j.l;
  }
  if (p.splits > 1) cluster_sync_all();
  else __syncthreads();

  // the splits' results and the prefix's, in order (the prefix's kernel may still be running;
  // where another launch joins the results, one CTA waits for it and the others make room)
  if (p.own_o == nullptr || blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int u = in_cluster * kThreads + tid; u < heads * Q; u += p.splits * kThreads) {
    const int r = u / Q, d = 4 * (u % Q), head = head0 + r;
    Joined j;
    int any = 0;
    if (p.splits > 1) {
      for (int s = 0; s < p.splits; ++s) {
        any |= ld_shared_cluster_s32(mapa_shared(smem_u32(&cta_used), s));
        j.add(ld_cluster(mapa_shared(smem_u32(&cta_m[r]), s)), ld_cluster(mapa_shared(smem_u32(&cta_l[r]), s)),
              ld_cluster4(mapa_shared(smem_u32(cta_o(r, d)), s)));
      }
    } else {
      any = cta_used;
      j.add(cta_m[r], cta_l[r], *reinterpret_cast<const float4*>(cta_o(r, d)));
    }
    if (p.own_o != nullptr) {  // kda_attn_join_kernel takes the results together (keys without weight: 0 / 0, and -inf)
      const long long at = (static_cast<long long>(rank / p.splits) * a.B + b) * a.HQ + head;
      const float inv = any ? 1.f / j.l : 0.f;
      *reinterpret_cast<float4*>(p.own_o + at * D + d) = make_float4(j.o.x * inv, j.o.y * inv, j.o.z * inv, j.o.w * inv);
      if (d == 0) p.own_lse[at] = any && j.l != 0.f ? j.m + log2f(j.l) : -INFINITY;
      continue;
    }
    if (row) join_parts<D>(p, b, head, d, j, any);
    store_row<D>(a, b, head, d, j, any);
  }
  if (p.splits > 1) cluster_sync_all();  // no CTA ends while another may read its results
}

template <int D, bool E4, int WARPS, bool MANY, int ROWS>
cudaError_t launch(const Params& p, bool after_prefix, cudaStream_t s) {
  using Sh = Shape<D, E4, WARPS, MANY>;
  static std::atomic<uint64_t> smem_set{0};
  auto kernel = kda_attn_step_kernel<D, E4, WARPS, MANY, ROWS>;
  cudaError_t e = set_smem_limit_once(kernel, Sh::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.a.B) * p.a.HKV * p.head_tiles * p.splits * p.chunks;
  if (grid > INT32_MAX) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  int n = 0;
  if (p.splits > 1) {
    attrs[n].id = cudaLaunchAttributeClusterDimension;
    attrs[n].val.clusterDim.x = static_cast<unsigned>(p.splits);
    attrs[n].val.clusterDim.y = attrs[n].val.clusterDim.z = 1;
    ++n;
  }
  if (after_prefix) {  // its CTAs start where the prefix's leave SMs free
    attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attrs;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// How a call's work is laid out, and where its parts' results lie in the workspace.
struct Plan {
  int splits = 1, chunks = 1, parts = 0;  // of the rows' own tokens; all results to join
  int prefix_splits = 0, prefix_pages = 0;
  int warps = 4;                          // to a CTA: 2, 4 or 8
  bool many = false;                      // CTAs: more of them on an SM
  bool join = false;                      // a launch of its own joins the results
  size_t lse = 0, o = 0, table = 0, k = 0, v = 0, bytes = 0;
};

template <int D, bool E4, int ROWS>
cudaError_t launch_rows(const Params& p, const Plan& x, cudaStream_t s) {
  const bool after = x.prefix_splits > 0;
  if (x.warps == 8) return launch<D, E4, 8, false, ROWS>(p, after, s);
  if constexpr (E4) {
    if (x.many) return launch<D, E4, 4, true, ROWS>(p, after, s);
  } else {
    if (x.many) return launch<D, E4, 2, false, ROWS>(p, after, s);
  }
  return launch<D, E4, 4, false, ROWS>(p, after, s);
}

// (A lane's scores are of heads g and g + 8: with up to 8 heads the second half is nothing.)
template <int D, bool E4>
cudaError_t launch_warps(const Params& p, const Plan& x, cudaStream_t s) {
  return p.G <= 8 ? launch_rows<D, E4, 1>(p, x, s) : launch_rows<D, E4, 2>(p, x, s);
}

// ---- the prefix ----
// Its keys meet the queries of all rows: products of 128 rows, which the prompt kernel
// computes as one sequence of B queries that sees every key, split over its blocks.

// bf16's largest value, which an 8-bit prefix's copies are held to (a head of bf16's last values
// may hold 256 times 2^120, 2^-8 above it).
constexpr float kMost = 3.3895313892515355e38f;

// An 8-bit prefix in bf16 (exact with scales that are powers of two), as pages 0, 1, ...
// of a cache of its own; table[i] is i, or -1 where the prefix's page is out of range.
template <int D>
__global__ void __launch_bounds__(256) kda_attn_prefix_bf16_kernel(const kda_attn_step_args a, __nv_bfloat16* k, __nv_bfloat16* vals, int32_t* table) {
  const int page = a.prefix_table[blockIdx.x], h = blockIdx.y;
  const bool good = page >= 0 && page < a.pages;
  if (h == 0 && threadIdx.x == 0) table[blockIdx.x] = good ? static_cast<int>(blockIdx.x) : -1;
  if (!good) return;
  const long long from = (static_cast<long long>(page) * a.HKV + h) * a.page_size, to = (static_cast<long long>(blockIdx.x) * a.HKV + h) * a.page_size;
  for (int u = threadIdx.x; u < 2 * a.page_size * (D / 8); u += 256) {
    const bool of_v = u >= a.page_size * (D / 8);
    const int w = of_v ? u - a.page_size * (D / 8) : u, t = w / (D / 8), c = w % (D / 8) * 8;
    const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(of_v ? a.v_cache : a.k_cache) + (from + t) * D + c);
    const float s = (of_v ? a.v_scale : a.k_scale)[from + t];
    const uint32_t in[2] = {x.x, x.y};
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = low_f16(in[i]), hi = high_f16(in[i]);
      const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&lo)), v = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      float x[4] = {u.x * s, u.y * s, v.x * s, v.y * s};
      if (s > kMost / 448.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = x[e] > kMost ? kMost : x[e] < -kMost ? -kMost : x[e];
      }
      out[2 * i] = Bf16::pack(x[0], x[1]);
      out[2 * i + 1] = Bf16::pack(x[2], x[3]);
    }
    *reinterpret_cast<uint4*>((of_v ? vals : k) + (to + t) * D + c) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

Plan plan_of(const kda_attn_step_args& a) {
  Plan x;
  const int G = a.HQ / a.HKV;
  // A cluster for each row and key head (and 16 heads of its group): CTAs for two on each
  // of the 152 SMs as far as their share stays at 64 tokens of what the table has room
  // for, and enough that a CTA's share is no more than 1 MB (rows of unequal lengths leave
  // SMs idle behind the longest: 64 rows of up to 8192 tokens took 223 us with one CTA
  // each, 178 with four).
  const long long units = static_cast<long long>(a.B) * a.HKV * ((G + 15) / 16), room = static_cast<long long>(a.table_width) * a.page_size;
  const bool e4 = a.cache_dtype == KDA_DTYPE_E4M3;
  const long long share = (1 << 20) / (2 * a.D * (e4 ? 1 : 2));
  while (x.splits < kMaxSplits && (units * x.splits < 2 * 152 || room > share * x.splits) && room > 64ll * x.splits) x.splits *= 2;
  // Few long rows: several clusters each, with a launch of its own to join their results.
  // (Clusters of 16 leave SMs idle: one row of 131072 tokens took 140 us with them.)
  if (units * x.splits <= 152 && room >= KDA_ATTN_LONG_TOKENS) {
    const long long fill = 2 * 152 / (units * x.splits), each = room / (512 * x.splits);
    x.chunks = static_cast<int>(fill < each ? fill : each);
    x.join = x.chunks > 1;
  }
  // Many CTAs: more and smaller ones on an SM, so that one's start and end pass under the
  // others' loads. bf16: four of two warps (256 rows of up to 500 tokens with a prefix: 94 ->
  // 89 us). 8 bits, whose products take longer: three of four warps, one group a step (256 rows
  // of about 2000: 198 -> 192; of 64 channels 147 -> 125; two warps each 208). Not where they
  // are few (16 rows of 2000 to 4000, 512 CTAs: 33 -> 37; 4 of 32768 to 65536: 94 -> 113).
  // Few: eight warps.
  const long long ctas = units * x.splits * x.chunks;
  x.many = ctas >= 4 * 152;
  if (x.many && !e4) x.warps = 2;
  if (ctas <= 152 && room >= 128ll * x.splits * x.chunks) x.warps = 8;
  if (a.prefix_len > 0) {
    // The prefix's splits, by what they leave to the rows' own tokens, in units of a block's
    // time on an SM (1.17 us): rounds of CTAs, each with its share of the blocks and 5 blocks'
    // time for what a CTA does besides; own CTAs run on the SMs that these leave free, for half
    // of the tokens that the table has room for and 6 units besides. Unless all fit at once,
    // own CTAs must not wait for the prefix, which would keep the next ones out, and a
    // launch joins the results. (256 rows, 32 heads on 8, prefix 8192, up to 500 own tokens: 2
    // splits on 64 SMs 73 us, 4 splits on 128 SMs 87, and 89 with CTAs that wait; 32 rows 27
    // and 38; 8 rows of up to 64 tokens, prefix 512, which fit, 10.8, and 12.4 with a join.)
    const AttnTiles t = attn_tiles(G);
    const long long tiles = (static_cast<long long>(a.B) + t.tokens - 1) / t.tokens * a.HKV * (G / t.heads);
    const int blocks = (a.prefix_len - 1) / 128 + 1;
    const double own = static_cast<double>(units) * room / 2 * (2 * a.D * (e4 ? 1 : 2)) / 7e6 + 6;
    const long long own_sms = (ctas * x.warps + 7) / 8;
    double best = 0;
    for (int s = 1; s <= 32 && s <= blocks; ++s) {
      const long long n = tiles * s;
      const double prefix = static_cast<double>((n + 151) / 152) * ((blocks + s - 1) / s + 5);
      const bool fits = n + own_sms <= 152;
      const double beside = n < 152 ? prefix * (152 - n) / 152 * 1.2 : 0;
      const double cost = fits ? prefix : prefix + (own > beside ? own - beside : 0) + 2;
      if (x.prefix_splits == 0 || cost < best) {
        x.prefix_splits = s;
        x.join = x.chunks > 1 || !fits;
        best = cost;
      }
    }
    x.prefix_pages = (a.prefix_len - 1) / a.page_size + 1;
  }
  x.parts = (x.join ? x.chunks : 0) + x.prefix_splits;
  const size_t rows = static_cast<size_t>(a.B) * a.HQ * x.parts;
  const auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  x.o = up(rows * sizeof(float));
  x.table = x.o + up(rows * a.D * sizeof(float));
  x.bytes = x.table;
  if (x.prefix_splits > 0 && a.cache_dtype == KDA_DTYPE_E4M3) {
    const size_t cache = static_cast<size_t>(x.prefix_pages) * a.HKV * a.page_size * a.D * 2;
    x.k = x.table + up(x.prefix_pages * sizeof(int32_t));
    x.v = x.k + cache;
    x.bytes = x.v + cache;
  }
  return x;
}

cudaError_t launch_prefix(const kda_attn_step_args& a, const Plan& x, unsigned char* w, const AttnParts& parts, cudaStream_t s) {
  kda_attn_fwd_args f = {};
  f.B = f.N = 1;
  f.T = a.B, f.HQ = a.HQ, f.HKV = a.HKV, f.D = a.D;
  f.page_size = a.page_size, f.table_width = x.prefix_pages;
  f.scale = a.scale;
  f.q = a.q, f.q_stride = a.q_stride, f.err = a.err;
  f.pages = a.pages, f.k = a.k_cache, f.v = a.v_cache, f.block_table = a.prefix_table;
  if (a.cache_dtype == KDA_DTYPE_E4M3) {
    __nv_bfloat16 *k = reinterpret_cast<__nv_bfloat16*>(w + x.k), *v = reinterpret_cast<__nv_bfloat16*>(w + x.v);
    int32_t* table = reinterpret_cast<int32_t*>(w + x.table);
    const dim3 grid(static_cast<unsigned>(x.prefix_pages), static_cast<unsigned>(a.HKV));
    if (a.D == 64) kda_attn_prefix_bf16_kernel<64><<<grid, 256, 0, s>>>(a, k, v, table);
    else kda_attn_prefix_bf16_kernel<128><<<grid, 256, 0, s>>>(a, k, v, table);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    f.pages = x.prefix_pages, f.k = k, f.v = v, f.block_table = table;
  }
  return launch_attn_prompts(f, parts, s);
}

}  // namespace

size_t attn_step_workspace_bytes(const kda_attn_step_args& a) { return plan_of(a).bytes; }

cudaError_t launch_attn_step(const kda_attn_step_args& a, void* workspace, cudaStream_t s) {
  const Plan x = plan_of(a);
  unsigned char* w = static_cast<unsigned char*>(workspace);
  float *o = reinterpret_cast<float*>(w + x.o), *lse = reinterpret_cast<float*>(w + x.lse);
  const Params p = {a, a.HQ / a.HKV, (a.HQ / a.HKV + 15) / 16, __builtin_ctz(a.page_size), x.splits, x.chunks, o, lse, x.parts, x.join ? o : nullptr, lse};
  const size_t own = x.join ? static_cast<size_t>(x.chunks) * a.B * a.HQ : 0;  // the prefix's results come behind these
  if (x.prefix_splits > 0) {
    const cudaError_t e = launch_prefix(a, x, w, AttnParts{o + own * a.D, lse + own, x.prefix_splits, a.prefix_len}, s);
    if (e != cudaSuccess) return e;
  }
  const bool e4 = a.cache_dtype == KDA_DTYPE_E4M3;
  const cudaError_t e = a.D == 64 ? (e4 ? launch_warps<64, true>(p, x, s) : launch_warps<64, false>(p, x, s))
                                  : (e4 ? launch_warps<128, true>(p, x, s) : launch_warps<128, false>(p, x, s));
  if (e != cudaSuccess || !x.join) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(a.B) * a.HQ * (a.D / 4) + 127) / 128));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr;  // (launched while the step's last CTAs run; it waits for them)
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return a.D == 64 ? cudaLaunchKernelEx(&cfg, kda_attn_join_kernel<64>, p) : cudaLaunchKernelEx(&cfg, kda_attn_join_kernel<128>, p);
}

}  // namespace kda
