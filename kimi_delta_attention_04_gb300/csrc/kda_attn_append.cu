// Rotary positions and the append of keys and values to the paged cache.
//
// Bound by memory: each value is read once and written once (twice for the keys where
// k_out is asked for). Lanes of D / 8 take a head with 8 channels (16 bytes) each; a
// group of them keeps its channels' cosines and sines in registers and goes through
// several heads of its token, all loads first. The pairs that a rotation turns are in
// one lane (neighbours), or in two lanes of the group (halves, exchanged by shuffles)
// where rot allows whole 8-channel pieces; other rot go through a per-channel path.
#include "kda_elem.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsAtOnce = 3;  // heads of a group whose loads are in flight together

__device__ __forceinline__ void unpack8(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3]), Bf16::pack(v[4], v[5]), Bf16::pack(v[6], v[7]));
}

// The smallest power of two s with m <= 448 s (448 = 1.75 * 2^8), at least 2^-110; 1
// for 0, NaN for infinities and NaN. Division by it, and the product that gives a
// stored value back, are exact.
__device__ __forceinline__ float power_scale(float m) {
  const uint32_t b = __float_as_uint(m);
  if (b >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  if (b == 0) return 1.f;
  const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(e > 17 ? e : 17) << 23);  // (17: 2^-110)
}

// How a lane's 8 channels are turned.
enum { kPlain = 0, kHalves = 1, kNeighbours = 2, kAny = 3 };

template <int D, int MODE, bool E4>
__global__ void __launch_bounds__(kThreads, MODE == kAny ? 2 : 4) kda_kv_append_kernel(const __grid_constant__ kda_kv_append_args p, int group_bits, int page_bits, int heads) {
  constexpr int L = D / 8;  // lanes of a head
  const int lane = threadIdx.x % L, c = 8 * lane;
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
  const int groups = 1 << group_bits;
  const long long token = unit >> group_bits;
  const int group = static_cast<int>(unit) & (groups - 1);
  const bool live = token < p.tokens;
  const long long t = live ? token : 0;
  const int HQ = p.q ? p.HQ : 0;
  const int rot = MODE == kPlain ? 0 : p.rot, half = rot / 2;
  const bool pairs = MODE == kNeighbours || (MODE == kAny && (p.flags & KDA_KV_FLAG_INTERLEAVED));

  const __nv_bfloat16* xq = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride + c;
  const __nv_bfloat16* xk = static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride + c;
  const __nv_bfloat16* xv = static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride + c;
  int slot = live ? p.slots[t] : -1;
  int pos = MODE != kPlain && live ? p.positions[t] : 0;
  bool turn = true, looked = false;
  float cs[8], sn[8];  // value of channel c + i: x cs[i] + partner sn[i]
  int page = 0, off = 0;
  const int other = MODE == kHalves ? (c >= rot ? lane : c < half ? lane + half / 8 : lane - half / 8) : lane;

  for (int base = 0; base < heads; base += groups * kHeadsAtOnce) {  // (the same for a warp's lanes: they shuffle)
    const int h0 = base + group;
    uint4 raw[kHeadsAtOnce];
    float partner[MODE == kAny ? kHeadsAtOnce : 1][8];
    // all of a group's loads come before its stores (q_out may be q, and k_out k), and before
    // what depends on the token's place and position
#pragma unroll
    for (int u = 0; u < kHeadsAtOnce; ++u) {
      const int h = h0 + u * groups;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (live && h < heads) {
        const __nv_bfloat16* x = h < HQ ? xq + h * D : h < HQ + p.HKV ? xk + (h - HQ) * D : xv + (h - HQ - p.HKV) * D;
        raw[u] = *reinterpret_cast<const uint4*>(x);
        if (MODE == kAny) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int d = c + i;
            const int q = d >= rot ? d : pairs ? (d ^ 1) : d < half ? d + half : d - half;
            partner[u][i] = __bfloat162float(x[q - c]);
          }
        }
      }
    }
    if (!looked) {
      looked = true;
      if (MODE != kPlain && live) {
        turn = pos >= 0 && pos < p.max_positions;
        if (!turn) {
          if (slot >= 0 && lane == 0 && group == 0) set_err(p.err, KDA_ERR_INVALID_ARG);
          slot = -1;
        }
      }
      if (slot >= p.pages * p.page_size) {
        if (lane == 0 && group == 0) set_err(p.err, KDA_ERR_INVALID_ARG);
        slot = -1;
      }
      if (slot >= 0) page = slot >> page_bits, off = slot & (p.page_size - 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
      if (MODE != kPlain && live && turn && c < rot) {
        const float* row = p.cos_sin + static_cast<long long>(pos) * rot;
        if (MODE == kHalves) {
          const int at = c < half ? c : c - half;
          const float sign = c < half ? -1.f : 1.f;
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(row + at + i), b = *reinterpret_cast<const float4*>(row + half + at + i);
            cs[i] = a.x, cs[i + 1] = a.y, cs[i + 2] = a.z, cs[i + 3] = a.w;
            sn[i] = sign * b.x, sn[i + 1] = sign * b.y, sn[i + 2] = sign * b.z, sn[i + 3] = sign * b.w;
          }
        } else if (MODE == kNeighbours) {
          const float4 a = *reinterpret_cast<const float4*>(row + c / 2), b = *reinterpret_cast<const float4*>(row + half + c / 2);
          cs[0] = cs[1] = a.x, cs[2] = cs[3] = a.y, cs[4] = cs[5] = a.z, cs[6] = cs[7] = a.w;
          sn[0] = -b.x, sn[1] = b.x, sn[2] = -b.y, sn[3] = b.y, sn[4] = -b.z, sn[5] = b.z, sn[6] = -b.w, sn[7] = b.w;
        } else if (MODE == kAny) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int d = c + i;
            if (d >= rot) continue;
            const int at = pairs ? d / 2 : d < half ? d : d - half;
            cs[i] = row[at];
            sn[i] = (pairs ? d % 2 == 0 : d < half) ? -row[half + at] : row[half + at];
          }
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kHeadsAtOnce; ++u) {
      const int h = h0 + u * groups;
      if (base + u * groups >= heads) break;  // (no lane of the warp has a head here)
      const bool valid = live && h < heads, is_v = h >= HQ + p.HKV;
      float x[8], y[8];
      unpack8(raw[u], x);
      if (MODE == kHalves) {
        uint4 r;
        r.x = __shfl_sync(0xffffffffu, raw[u].x, other, L);
        r.y = __shfl_sync(0xffffffffu, raw[u].y, other, L);
        r.z = __shfl_sync(0xffffffffu, raw[u].z, other, L);
        r.w = __shfl_sync(0xffffffffu, raw[u].w, other, L);
        unpack8(r, y);
      } else if (MODE == kNeighbours) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
      } else if (MODE == kAny) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = partner[u][i];
      }
      // channels that are not turned keep their bits (infinities too: no 0 * partner)
      if (MODE != kPlain && !is_v && (c < rot || !turn)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!turn) x[i] = 0.f;
          else if (MODE != kAny || c + i < rot) x[i] = x[i] * cs[i] + y[i] * sn[i];
        }
      }
      if (valid && h < HQ) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) + t * p.q_out_stride + h * D + c) = pack8(x);
      } else if (valid && !is_v && p.k_out) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_out) + t * p.k_out_stride + (h - HQ) * D + c) = pack8(x);
      }
      if (E4) {
        if (base + (u + 1) * groups <= HQ) continue;  // (queries only in the whole warp)
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (valid && h >= HQ && slot >= 0) {
          const float s = power_scale(m), inv = s == s ? __uint_as_float((254u << 23) - __float_as_uint(s)) : s;
          const long long at = ((static_cast<long long>(page) * p.HKV + (is_v ? h - HQ - p.HKV : h - HQ)) << page_bits) + off;
          uint2 b;
          b.x = pack_e4m3x2(x[0] * inv, x[1] * inv) | pack_e4m3x2(x[2] * inv, x[3] * inv) << 16;
          b.y = pack_e4m3x2(x[4] * inv, x[5] * inv) | pack_e4m3x2(x[6] * inv, x[7] * inv) << 16;
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + at * D + c) = b;
          if (lane == 0) (is_v ? p.v_scale : p.k_scale)[at] = s;
        }
      } else if (valid && h >= HQ && slot >= 0) {
        const long long at = ((static_cast<long long>(page) * p.HKV + (is_v ? h - HQ - p.HKV : h - HQ)) << page_bits) + off;
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache) + at * D + c) = pack8(x);
      }
    }
  }
}

template <int D, int MODE>
cudaError_t launch(const kda_kv_append_args& a, cudaStream_t s) {
  const int heads = (a.q ? a.HQ : 0) + 2 * a.HKV;
  // Groups of a token: each has up to kHeadsAtOnce heads, unless that is more groups than a
  // CTA holds. With tokens enough for two rounds of 4 CTAs on each of the 152 SMs, down to 4
  // groups: what a lane works out for its channels serves more heads (8192 tokens, 32 + 8
  // heads of 128, 8-bit cache: 16 groups 45 us, 8 groups 40, 4 groups 39.5).
  constexpr long long per = kThreads / (D / 8);
  int bits = 0;
  while ((1 << bits) < per && (kHeadsAtOnce << bits) < heads) ++bits;
  while (bits > 2 && (static_cast<long long>(a.tokens) << (bits - 1)) / per >= 2 * 4 * 152) --bits;
  const int page_bits = __builtin_ctz(a.page_size);
  const long long units = static_cast<long long>(a.tokens) << bits;
  const long long grid = (units + per - 1) / per;
  if (grid > INT32_MAX) return cudaErrorNotSupported;
  if (a.cache_dtype == KDA_DTYPE_E4M3) kda_kv_append_kernel<D, MODE, true><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, bits, page_bits, heads);
  else kda_kv_append_kernel<D, MODE, false><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, bits, page_bits, heads);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_mode(const kda_kv_append_args& a, cudaStream_t s) {
  if (a.rot == 0) return launch<D, kPlain>(a, s);
  const bool pairs = a.flags & KDA_KV_FLAG_INTERLEAVED;
  if (pairs && a.rot % 8 == 0) return launch<D, kNeighbours>(a, s);
  if (!pairs && a.rot % 16 == 0) return launch<D, kHalves>(a, s);
  return launch<D, kAny>(a, s);
}

}  // namespace

cudaError_t launch_kv_append(const kda_kv_append_args& a, cudaStream_t s) {
  return a.D == 64 ? launch_mode<64>(a, s) : launch_mode<128>(a, s);
}

}  // namespace kda
