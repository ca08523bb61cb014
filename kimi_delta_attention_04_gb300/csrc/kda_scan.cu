// Gated linear recurrence, one fp32 state per sequence and channel:
//   h_t = a_t h_{t-1} + u_t,  u_t = x_t or (1 - a_t) x_t,  a_t = exp(g) or sigmoid(f),
// its gradients, and the single-token step on a pool of states.
//
// Split. A warp holds one chunk of 16 tokens x 64 channels (two a lane) in
// registers; the kWarps warps of a CTA and the S CTAs of a cluster hold
// consecutive chunks, so a cluster advances S * kWarps * 16 tokens at a time and
// no token is read twice. Each warp reduces its chunk to the pair (A, B) of
// h_out = A h_in + B (A the product of the decays, B the state from zero); the
// pairs meet in shared memory, the CTAs' totals in every CTA of the cluster
// (remote asynchronous stores, counted on a barrier), and each warp composes the
// pairs before it with the carried state and runs its chunk again from the state
// that enters it. The next advances' tiles are on their way meanwhile (asynchronous
// copies, a ring of two or three tiles a warp). Sums have one fixed order, so results
// do not vary from run to run. Batches of short equal sequences have kernels of their
// own, with no more warps than a sequence has chunks and no ring.
//
// HBM traffic is the bound to come to: 8192 x 4096 bf16 runs at 4.6 TB/s forward (44
// us; the rest is the latency of the exchange and 23 instructions an element) and 5.1
// TB/s backward, 4 x 4096 x 2048 with fp32 gates at 5.7 and 6.3 TB/s.
#include <algorithm>

#include "kda_cluster.cuh"
#include "kda_device_counts.h"
#include "kda_elem.cuh"

namespace kda {
namespace {

constexpr int kScanChunk = 16;    // tokens between the states of h_chunks, and of a warp's tile
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kShortWarps = 4;    // most warps of a CTA of the kernels for short sequences
constexpr int kBlockCh = 64;      // channels of a CTA
constexpr int kMaxCluster = 8;
constexpr int kStepThreads = 128;
constexpr int kKeysAt = kThreads + 4;  // ints before the keys that order packed sequences: a multiple of 4
constexpr uint64_t kWaitNs = 2000000000ull;

// A CTA's sequences, one after another.
struct Sequences {
  int n, last;           // the present one, and the last that this CTA takes
  int start, end;        // its tokens
  long long chunk_base;  // its first chunk in h_chunks
};

// Chunks of a sequence of a packed batch, and whether its two ends are in order.
__device__ __forceinline__ unsigned chunks_of(int s, int e, int T, bool& bad) {
  const bool wrong = e < s || s < 0 || e > T;
  bad |= wrong;
  return wrong ? 0u : static_cast<unsigned>(e - s + kScanChunk - 1) / kScanChunk;
}

// The first sequence of a CTA, checking the whole of cu_seqlens on the way (all
// threads of the CTA call it; scratch: kKeysAt + kThreads ints of shared memory
// that nothing else uses meanwhile). Up to kThreads packed sequences take a CTA (or
// cluster) each, longest first, so that no long one starts when the others are done
// (16 sequences of 512 to 8192 tokens: 133 -> 116 us forward); more of them are
// shared out in runs of neighbours, so that the check of all N is made once a CTA.
// Returns false, after reporting, where the array is bad.
template <int W>
__device__ __forceinline__ bool first_sequence(const kda_scan_args& p, Sequences& q, int* scratch) {
  const int y = blockIdx.y, rows = gridDim.y, tid = threadIdx.x;
  if (W != kWarps || p.cu_seqlens == nullptr) {
    q.n = y;
    q.last = p.N - 1;
    q.start = y * p.T;
    q.end = q.start + p.T;
    q.chunk_base = static_cast<long long>(y) * ((p.T + kScanChunk - 1) / kScanChunk);
    return true;
  }
  // chunks before the sequence, of all (ends in order give at most T / 16 + N; the
  // sums of others may wrap, but those are refused whatever they come to)
  __shared__ unsigned base, total;
  __shared__ int chosen;
  if (tid == 0) base = total = 0;
  bool bad = false;
  unsigned mine = 0, all = 0;
  int n;
  if (p.N <= kThreads) {
    // one key orders by length (up to 2^24 chunks) and then by place, so that a
    // sequence's rank is the number of larger keys: 256 sequences of 16 tokens,
    // 1024 channels, 4096 CTAs: 65 us forward instead of 93 with lengths and places
    // compared by themselves
    unsigned* keys = reinterpret_cast<unsigned*>(scratch + kKeysAt);
    unsigned key = 0;
    if (tid < p.N) {
      const int s = p.cu_seqlens[tid], e = p.cu_seqlens[tid + 1];
      scratch[tid] = s;
      if (tid == p.N - 1) scratch[p.N] = e;
      all = chunks_of(s, e, p.T, bad);
      bad |= (tid == 0 && s != 0) || (tid == p.N - 1 && e != p.T);
      key = (all < 0xffffffu ? all : 0xffffffu) << 8 | (kThreads - 1 - tid);
    }
    keys[tid] = key;
    __syncthreads();
    if (tid < p.N) {
      int rank = 0;
      for (int i = 0; i < p.N; i += 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
        rank += (k.x > key) + (k.y > key) + (k.z > key) + (k.w > key);
      }
      if (rank == y) chosen = tid;
    }
    __syncthreads();
    n = chosen;
    if (tid < n) mine = all;
    q.start = scratch[n];
    q.end = scratch[n + 1];
    q.last = n;
  } else {
    n = static_cast<int>(static_cast<long long>(p.N) * y / rows);
    q.last = static_cast<int>(static_cast<long long>(p.N) * (y + 1) / rows) - 1;
    q.start = p.cu_seqlens[n];
    q.end = p.cu_seqlens[n + 1];
    for (unsigned i = tid; i < static_cast<unsigned>(p.N); i += kThreads) {  // (N + kThreads may pass 2^31)
      const unsigned chunks = chunks_of(p.cu_seqlens[i], p.cu_seqlens[i + 1], p.T, bad);
      all += chunks;
      if (i < static_cast<unsigned>(n)) mine += chunks;
    }
    bad |= tid == 0 && (p.cu_seqlens[0] != 0 || p.cu_seqlens[p.N] != p.T);
    __syncthreads();  // base and total are 0
  }
  if (p.h_chunks != nullptr) {
    mine = __reduce_add_sync(0xffffffffu, mine);
    all = __reduce_add_sync(0xffffffffu, all);
    if (tid % 32 == 0 && all != 0) {
      atomicAdd(&base, mine);
      atomicAdd(&total, all);
    }
    __syncthreads();
    bad |= total > p.h_chunks_rows;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_err(p.err, KDA_ERR_INVALID_ARG);
    return false;
  }
  q.n = n;
  q.chunk_base = static_cast<long long>(base);
  return true;
}

// Moves to the CTA's next sequence; false when there is none.
__device__ __forceinline__ bool next_sequence(const kda_scan_args& p, Sequences& q) {
  const int step = p.cu_seqlens == nullptr ? static_cast<int>(gridDim.y) : 1;
  if (q.n > q.last - step) return false;
  q.chunk_base += static_cast<long long>(step) * ((q.end - q.start + kScanChunk - 1) / kScanChunk);
  q.n += step;
  q.start = p.cu_seqlens == nullptr ? q.n * p.T : q.end;
  q.end = p.cu_seqlens == nullptr ? q.start + p.T : p.cu_seqlens[q.n + 1];
  return true;
}

// How a tile's rows are read and written, by their alignment: 16 bytes at a time,
// a pair of channels at a time, or one.
enum { kWide = 2, kPair = 1, kSingle = 0 };

// Two channels of one token: 2 lane and 2 lane + 1 of the block, or with kSingle
// lane and lane + 32.
template <typename T>
struct Raw2;
template <>
struct Raw2<__nv_bfloat16> {
  uint32_t v;
  __device__ __forceinline__ float2 get() const {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
    v = *reinterpret_cast<const uint16_t*>(p) | (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(q)) << 16);
  }
};
template <>
struct Raw2<float> {
  float2 v;
  __device__ __forceinline__ float2 get() const { return v; }
  __device__ __forceinline__ void load(const float* p, const float* q) { v = make_float2(*p, *q); }
};

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 r = *reinterpret_cast<const float4*>(p);
  v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xffff0000u);
  v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* v) { *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3]));
}
__device__ __forceinline__ void store2(__nv_bfloat16* p, float2 v) { *reinterpret_cast<uint32_t*>(p) = Bf16::pack(v.x, v.y); }
__device__ __forceinline__ void store2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }

template <int BYTES>
__device__ __forceinline__ void cp_async_bytes(void* smem, const void* gmem) {
  if (BYTES == 16) cp_async16(smem, gmem);
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(smem)), "l"(gmem), "n"(BYTES) : "memory");
}

// A lane's two channels, and which of them exist.
struct Lane {
  int block_ch, c0, c1;
  bool p0, p1;
};

template <int ACC>
__device__ __forceinline__ Lane lane_channels(int block_ch, int D) {
  const int lane = threadIdx.x & 31;
  Lane l;
  l.block_ch = block_ch;
  l.c0 = block_ch + (ACC == kSingle ? lane : 2 * lane);
  l.c1 = block_ch + (ACC == kSingle ? lane + 32 : 2 * lane + 1);
  l.p0 = l.c0 < D;
  l.p1 = l.c1 < D;
  return l;
}

// One tensor's share of a warp's tile on its way in: 16 tokens x 64 channels,
// token by token, in shared memory that only this warp touches. fetch() starts the
// copies (kSingle loads and stores); once they have landed and the warp has
// synchronised, get() reads a lane's pair. Tokens past m and channels past D are
// not copied: what their slots held is read, and the results are not used.
template <typename T, int ACC>
struct Tile {
  Raw2<T>* pairs;  // this warp's
  __device__ __forceinline__ void fetch(const T* rows, long long stride, int m, const Lane& l, int D) const {
    const int lane = threadIdx.x & 31;
    if (ACC == kWide) {
      constexpr int PER = 16 / sizeof(T), LANES = kBlockCh / PER, TOK = 32 / LANES;  // lanes of a token, tokens a step
      const int i0 = lane / LANES, c = lane % LANES * PER;
      if (l.block_ch + c >= D) return;
      const T* src = rows + i0 * stride + l.block_ch + c;
      unsigned char* dst = reinterpret_cast<unsigned char*>(pairs) + (i0 * kBlockCh + c) * sizeof(T);
#pragma unroll
      for (int i = 0; i < kScanChunk / TOK; ++i, src += TOK * stride)
        if (i * TOK + i0 < m) cp_async_bytes<16>(dst + i * TOK * kBlockCh * sizeof(T), src);
    } else if (ACC == kPair) {
      if (!l.p0) return;
      const T* src = rows + l.c0;
#pragma unroll
      for (int i = 0; i < kScanChunk; ++i, src += stride)
        if (i < m) cp_async_bytes<2 * sizeof(T)>(pairs + i * 32 + lane, src);
    } else {
      // tokens and channels that do not exist read the last that do: 32 loads without
      // a condition stay in flight together
      const T *p0 = rows + min(l.c0, D - 1), *p1 = rows + min(l.c1, D - 1);
      Raw2<T> r[kScanChunk];
#pragma unroll
      for (int i = 0; i < kScanChunk; ++i) {
        const long long at = min(i, m - 1) * stride;
        r[i].load(p0 + at, p1 + at);
      }
#pragma unroll
      for (int i = 0; i < kScanChunk; ++i) pairs[i * 32 + lane] = r[i];
    }
  }
  __device__ __forceinline__ float2 get(int i) const { return pairs[i * 32 + (threadIdx.x & 31)].get(); }
};
template <typename T>
constexpr size_t tile_bytes() { return sizeof(Raw2<T>) * 32 * kScanChunk; }  // of one warp

template <int ACC, typename T>
__device__ __forceinline__ void store_pair(T* row, const Lane& l, float2 v) {
  if (ACC != kSingle) {
    if (l.p0) store2(row + l.c0, v);
  } else {
    if (l.p0) store_f(row + l.c0, v.x);
    if (l.p1) store_f(row + l.c1, v.y);
  }
}

// States are [.., D] fp32 rows: no alignment is assumed of them.
__device__ __forceinline__ float2 load_state(const float* base, long long row, int D, const Lane& l) {
  if (base == nullptr) return make_float2(0.f, 0.f);
  base += row * D;
  return make_float2(l.p0 ? base[l.c0] : 0.f, l.p1 ? base[l.c1] : 0.f);
}
__device__ __forceinline__ void store_state(float* base, long long row, int D, const Lane& l, float2 v) {
  base += row * D;
  if (l.p0) base[l.c0] = v.x;
  if (l.p1) base[l.c1] = v.y;
}

// The decays: expf(g), or the sigmoid. e^v is 2^z (1 + d) with z = v / ln 2 rounded and d =
// v - z ln 2 what that lost. fp32 gates take d with it, and e = e^-|f| <= 1 (1 / (1 + e)
// for f >= 0, e / (1 + e) below), so that a decay is good to a few fp32 steps of itself over
// the whole range. Without them a small decay is off by |f| / 2 steps; bf16 gates, whose
// gradients are rounded at 2^-9, do without (with both, 8192 x 4096 forward took 8 %
// longer).
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// e^-f of bf16 gates, e^-|f| of fp32 ones.
template <typename G>
__device__ __forceinline__ float2 exp_neg(float2 f) {
  constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
  if (sizeof(G) == 2) {
    const float2 z = mul2(f, make_float2(-kLog2e, -kLog2e));
    return make_float2(ex2_approx(z.x), ex2_approx(z.y));
  }
  // (e is 0 from |f| = 88 on; an infinite v would make d NaN)
  const float2 v = make_float2(max_nan(-fabsf(f.x), -128.f), max_nan(-fabsf(f.y), -128.f));
  const float2 z = mul2(v, make_float2(kLog2e, kLog2e)), d = fma2(z, make_float2(-kLn2, -kLn2), v);
  const float2 e = make_float2(ex2_approx(z.x), ex2_approx(z.y));
  return fma2(e, d, e);
}
template <int MODE, typename G>
__device__ __forceinline__ float2 decay_of(float2 f) {
  if (MODE == KDA_SCAN_LOG_DECAY) return make_float2(expf(f.x), expf(f.y));
  const float2 e = exp_neg<G>(f), q = add2(e, make_float2(1.f, 1.f)), r = make_float2(rcp_approx(q.x), rcp_approx(q.y));
  if (sizeof(G) == 2) return r;  // (e = inf gives 0)
  const float2 s = mul2(e, r);
  return make_float2(f.x < 0.f ? s.x : r.x, f.y < 0.f ? s.y : r.y);
}
// 1 - a to a few steps of itself: from f = 17 on a rounds to 1, and at f = 10 the
// difference has three digits, with one sign for a given gate. e a is 1 - a exactly; below
// f = 0 the difference is good, and e may be infinite. With log decays it is 1 - e^g, near 0
// by a polynomial in g (fitted to (e^g - 1) / g for the least relative error on [-0.7,
// 0.7]: 3e-8).
template <int MODE, typename G>
__device__ __forceinline__ float2 rest_of(float2 f, float2 a) {
  float2 near;
  bool x, y;
  if (MODE == KDA_SCAN_LOG_DECAY) {
    auto both = [](float c) { return make_float2(c, c); };
    near = fma2(both(1.98409674e-04f), f, both(1.41012878e-03f));
    near = fma2(near, f, both(8.33449047e-03f));
    near = fma2(near, f, both(4.16615158e-02f));
    near = fma2(near, f, both(1.66666389e-01f));
    near = fma2(near, f, both(5.00000298e-01f));
    near = mul2(fma2(near, f, both(1.f)), make_float2(-f.x, -f.y));
    x = fabsf(f.x) > 0.7f, y = fabsf(f.y) > 0.7f;
  } else {
    near = mul2(exp_neg<G>(f), a);
    x = f.x < 0.f, y = f.y < 0.f;
  }
  return make_float2(x ? 1.f - a.x : near.x, y ? 1.f - a.y : near.y);
}

// A tile's gates and inputs, all read before anything is written to its slots.
template <typename X, typename G, int ACC>
__device__ __forceinline__ void read_tiles(float2 (&f)[kScanChunk], float2 (&u)[kScanChunk], const Tile<G, ACC>& gate,
                                           const Tile<X, ACC>& x) {
#pragma unroll
  for (int i = 0; i < kScanChunk; ++i) f[i] = gate.get(i);
#pragma unroll
  for (int i = 0; i < kScanChunk; ++i) u[i] = x.get(i);
}
// Decays in the place of the gates, and inputs as they enter the states.
template <int MODE, bool COMP, typename G>
__device__ __forceinline__ void weigh(float2 (&a)[kScanChunk], float2 (&u)[kScanChunk]) {
#pragma unroll
  for (int i = 0; i < kScanChunk; ++i) {
    const float2 f = a[i];
    a[i] = decay_of<MODE, G>(f);
    if (COMP) u[i] = mul2(rest_of<MODE, G>(f, a[i]), u[i]);
  }
}
// Four bytes a value in the slots of tiles that have been read: the gate's, or with bf16
// the gate's and the input's, a half each.
template <int ACC>
__device__ __forceinline__ void put_pair(const Tile<float, ACC>& gate, const Tile<float, ACC>&, int i, float2 b) {
  gate.pairs[i * 32 + (threadIdx.x & 31)].v = b;
}
template <int ACC>
__device__ __forceinline__ void put_pair(const Tile<float, ACC>& gate, const Tile<__nv_bfloat16, ACC>&, int i, float2 b) {
  gate.pairs[i * 32 + (threadIdx.x & 31)].v = b;
}
template <int ACC>
__device__ __forceinline__ void put_pair(const Tile<__nv_bfloat16, ACC>& gate, const Tile<__nv_bfloat16, ACC>& x, int i, float2 b) {
  const int at = i * 32 + (threadIdx.x & 31);
  gate.pairs[at].v = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x7632);
  x.pairs[at].v = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x5410);
}
template <typename X, int ACC>
__device__ __forceinline__ float2 get_pair(const Tile<float, ACC>& gate, const Tile<X, ACC>&, int i) {
  return gate.get(i);
}
template <int ACC>
__device__ __forceinline__ float2 get_pair(const Tile<__nv_bfloat16, ACC>& gate, const Tile<__nv_bfloat16, ACC>& x, int i) {
  const int at = i * 32 + (threadIdx.x & 31);
  const uint32_t hi = gate.pairs[at].v, lo = x.pairs[at].v;
  return make_float2(__uint_as_float(__byte_perm(lo, hi, 0x5410)), __uint_as_float(__byte_perm(lo, hi, 0x7632)));
}

// Decays in the place of the gates, and in the place of the inputs what each decay's
// gradient is a multiple of: the state before the token (h before the first), less the input
// where that has the weight 1 - a. 1 - a itself, where it is needed, is left in the tiles'
// slots for the gradients (64 registers hold the other two, and forming it again there
// made every backward pass a third longer).
template <int MODE, bool COMP, typename X, typename G, int ACC>
__device__ __forceinline__ void run_through(float2 (&a)[kScanChunk], float2 (&w)[kScanChunk], float2 h, const Tile<G, ACC>& gate,
                                            const Tile<X, ACC>& x) {
#pragma unroll
  for (int i = 0; i < kScanChunk; ++i) {
    const float2 f = a[i];
    float2 u = w[i];
    a[i] = decay_of<MODE, G>(f);
    w[i] = COMP ? make_float2(h.x - u.x, h.y - u.y) : h;
    if (COMP || MODE == KDA_SCAN_LOGITS) {
      const float2 b = rest_of<MODE, G>(f, a[i]);
      put_pair(gate, x, i, b);
      if (COMP) u = mul2(b, u);
    }
    h = fma2(a[i], h, u);
  }
}

// The map h -> A h + B of some consecutive tokens, for a lane's two channels.
struct Map {
  float2 A, B;
};
__device__ __forceinline__ Map then(const Map& first, const Map& second) {
  return Map{mul2(first.A, second.A), fma2(second.A, first.B, second.B)};
}
__device__ __forceinline__ Map identity_map() { return Map{make_float2(1.f, 1.f), make_float2(0.f, 0.f)}; }

// A state may be infinite, and then a product of decays that has rounded to 0 makes it
// NaN where one token after the other leaves it infinite. So maps that are handed on
// have A = 0 only where one of their decays is 0: other products are held at the
// smallest fp32 (which adds 2^-149 of a state at most, as much as rounding there does).
// The factors are looked at again only where it matters, so the cost is a comparison.
constexpr float kSmallest = 1.40129846e-45f;
__device__ __forceinline__ void keep_nonzero(Map& map, const float2 (&a)[kScanChunk], int m) {
  if (map.A.x != 0.f && map.A.y != 0.f) return;
  float2 least = make_float2(kSmallest, kSmallest);
#pragma unroll
  for (int i = 0; i < kScanChunk; ++i)
    if (i < m) least = make_float2(fminf(least.x, a[i].x), fminf(least.y, a[i].y));
  map.A = make_float2(fmaxf(map.A.x, least.x), fmaxf(map.A.y, least.y));
}
// The same for the product of the first n warps' maps.
__device__ __forceinline__ float2 nonzero_product(float2 A, const Map (*maps)[32], int n) {
  float2 least = make_float2(kSmallest, kSmallest);
  const int lane = threadIdx.x & 31;
  for (int w = 0; w < n; ++w) least = make_float2(fminf(least.x, maps[w][lane].A.x), fminf(least.y, maps[w][lane].A.y));
  return make_float2(fmaxf(A.x, least.x), fmaxf(A.y, least.y));
}
__device__ __forceinline__ bool any_infinite(float2 h) { return fmaxf(fabsf(h.x), fabsf(h.y)) > 3.40282347e+38f; }  // (beside a NaN too)
// Warps of a CTA of a kernel made for up to W of them: kWarps always, or those launched.
template <int W>
__device__ __forceinline__ int cta_warps() {
  return W == kWarps ? kWarps : blockDim.x >> 5;
}

template <int W>
struct __align__(128) ScanSmem {  // a map travels between CTAs as one word of 16 bytes
  Map warp[2][W][32];           // the warps' maps of an advance, by parity of the advance
  Map cta[2][W == kWarps ? kMaxCluster : 1][32];  // the CTAs' maps
  uint64_t bar[2];              // all CTAs' maps of the advance have arrived
};

static_assert(sizeof(ScanSmem<kWarps>::warp) >= (kKeysAt + kThreads) * sizeof(int) && kThreads <= 256 && kKeysAt % 4 == 0, "");
static_assert(sizeof(Map) == 16 && alignof(ScanSmem<kWarps>) % 16 == 0 && offsetof(ScanSmem<kWarps>, cta) % 16 == 0, "");

// A lane's map into another CTA's shared memory, counted in bytes on its barrier.
__device__ __forceinline__ void st_async_map(uint32_t addr, const Map& m, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "r"(__float_as_uint(m.A.x)), "r"(__float_as_uint(m.A.y)), "r"(__float_as_uint(m.B.x)),
               "r"(__float_as_uint(m.B.y)), "r"(bar)
               : "memory");
}

// From this warp's map of advance number `it` and the state `carry` that enters the
// advance (the same in every warp of the cluster): the state that enters this
// warp's chunk; carry becomes the state after the advance. All threads of the
// cluster call it. The buffers alternate: a CTA sends its map of advance it + 2 only
// after every CTA's map of it + 1, which each sent after all its warps had read
// those of it. A wait for the other CTAs that runs out clears `ok`; the thread then
// goes on through the same barriers without waiting for them again, so that all
// threads still reach the end (with results that the error word disowns).
template <int W>
__device__ __forceinline__ float2 enter_state(ScanSmem<W>& sm, const Map& mine, float2& carry, bool& ok, int it, int S, int rank) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, parity = it & 1, warps = cta_warps<W>();
  sm.warp[parity][warp][lane] = mine;
  __syncthreads();
  Map before = identity_map();
#pragma unroll
  for (int w = 0; w < W - 1; ++w)
    if (w < warp) before = then(before, sm.warp[parity][w][lane]);
  if (W != kWarps || S == 1) {
    Map total = then(before, mine);
    for (int w = warp + 1; w < warps; ++w) total = then(total, sm.warp[parity][w][lane]);
    if (any_infinite(carry)) {
      before.A = nonzero_product(before.A, sm.warp[parity], warp);
      total.A = nonzero_product(total.A, sm.warp[parity], warps);
    }
    const float2 in = fma2(before.A, carry, before.B);
    carry = fma2(total.A, carry, total.B);
    return in;
  }
  const uint32_t bar = smem_u32(&sm.bar[parity]);
  if (warp == warps - 1) {
    Map total = then(before, mine);
    if (total.A.x == 0.f || total.A.y == 0.f) total.A = nonzero_product(total.A, sm.warp[parity], warps);
    if (lane == 0) mbar_arrive_expect_tx_local(&sm.bar[parity], S * 32 * sizeof(Map));
    const uint32_t at = smem_u32(&sm.cta[parity][rank][lane]);
    for (int r = 0; r < S; ++r) st_async_map(mapa_shared(at, r), total, mapa_shared(bar, r));
  }
  if (ok) ok = mbar_wait_bounded(bar, (it >> 1) & 1, kWaitNs);
  float2 h = carry, start = carry;
  for (int r = 0; r < S; ++r) {
    if (r == rank) start = h;
    const Map& m = sm.cta[parity][r][lane];
    h = fma2(m.A, h, m.B);
  }
  carry = h;
  if (any_infinite(start)) before.A = nonzero_product(before.A, sm.warp[parity], warp);
  return fma2(before.A, start, before.B);
}

// Stages of the ring of tiles: what leaves two CTAs on an SM (about 100 KB each),
// at least two; one for short sequences, which are one advance.
constexpr int stages_for(size_t stage, int W) { return W != kWarps ? 1 : 100 * 1024 / (kWarps * stage) >= 3 ? 3 : 2; }

template <int W>
__device__ __forceinline__ void scan_prologue(ScanSmem<W>& sm, int S) {
  if (W != kWarps || S == 1) return;
  if (threadIdx.x == 0) {
    mbar_init(&sm.bar[0], 1);
    mbar_init(&sm.bar[1], 1);
    fence_mbarrier_init_cluster();
  }
  cluster_sync_all();  // every CTA of the cluster runs before its shared memory is written
}

// Forward. Grid (S * channel blocks, sequences), cluster (S, 1, 1). W is kWarps, or
// kShortWarps for batches of equal sequences of up to that many chunks, with as many
// warps as they have chunks and S = 1.
template <typename X, typename G, int ACC, int W>
__global__ void __launch_bounds__(32 * W, 2 * kWarps / W) kda_scan_fwd_kernel(const kda_scan_args p, int S) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ ScanSmem<W> sm;
  constexpr size_t kStage = tile_bytes<X>() + tile_bytes<G>();  // of one warp
  constexpr int kStages = stages_for(kStage, W);
  const int warp = threadIdx.x >> 5, rank = blockIdx.x % S, warps = cta_warps<W>(), advance = S * warps * kScanChunk;
  const Lane l = lane_channels<ACC>(blockIdx.x / S * kBlockCh, p.D);
  const bool comp = p.flags & KDA_SCAN_FLAG_COMPLEMENT;
  unsigned char* mine_ring = ring + warp * kStages * kStage;
  scan_prologue(sm, S);
  int it = 0;
  bool ok = true;
  Sequences pos;
  bool more = first_sequence<W>(p, pos, reinterpret_cast<int*>(sm.warp));  // (the same answer in every CTA)
  for (; more; more = next_sequence(p, pos)) {
    const int len = pos.end - pos.start;
    // the tiles of advance j, whose first token for this warp is first(j)
    auto tile_x = [&](int slot) { return Tile<X, ACC>{reinterpret_cast<Raw2<X>*>(mine_ring + slot * kStage)}; };
    auto tile_g = [&](int slot) { return Tile<G, ACC>{reinterpret_cast<Raw2<G>*>(mine_ring + slot * kStage + tile_bytes<X>())}; };
    auto first = [&](int j) { return j * advance + (rank * warps + warp) * kScanChunk; };
    auto fetch = [&](int j, int slot) {
      const int i0 = first(j);
      if (i0 < len) {
        const long long t0 = pos.start + static_cast<long long>(i0);
        tile_x(slot).fetch(static_cast<const X*>(p.x) + t0 * p.x_stride, p.x_stride, len - i0, l, p.D);
        tile_g(slot).fetch(static_cast<const G*>(p.gate) + t0 * p.gate_stride, p.gate_stride, len - i0, l, p.D);
      }
      cp_async_commit();
    };
    float2 carry = load_state(p.h0, pos.n, p.D, l);
    for (int j = 0; j < kStages - 1; ++j) fetch(j, j);
    int slot = 0;  // of advance j; its stage before is the one to fill
    for (int j = 0; j * static_cast<long long>(advance) < len; ++j, ++it, slot = slot + 1 == kStages ? 0 : slot + 1) {
      fetch(j + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const int i0 = first(j), m = len - i0;
      float2 a[kScanChunk], u[kScanChunk];
      const Tile<X, ACC> tx = tile_x(slot);
      const Tile<G, ACC> tg = tile_g(slot);
      read_tiles(a, u, tg, tx);
      if (p.gate_mode == KDA_SCAN_LOG_DECAY) {
        if (comp) weigh<KDA_SCAN_LOG_DECAY, true, G>(a, u);
        else weigh<KDA_SCAN_LOG_DECAY, false, G>(a, u);
      } else {
        if (comp) weigh<KDA_SCAN_LOGITS, true, G>(a, u);
        else weigh<KDA_SCAN_LOGITS, false, G>(a, u);
      }
      __syncwarp();  // the slots are free for the fetch of the next iteration
      Map mine = identity_map();
      if (m >= kScanChunk) {
#pragma unroll
        for (int i = 0; i < kScanChunk; ++i) mine = then(mine, Map{a[i], u[i]});
      } else {
#pragma unroll
        for (int i = 0; i < kScanChunk; ++i)
          if (i < m) mine = then(mine, Map{a[i], u[i]});
      }
      keep_nonzero(mine, a, m);
      float2 h = enter_state(sm, mine, carry, ok, it, S, rank);
      if (m > 0 && p.h_chunks) store_state(p.h_chunks, pos.chunk_base + i0 / kScanChunk, p.D, l, h);
      X* y = static_cast<X*>(p.y) + (pos.start + static_cast<long long>(i0)) * p.y_stride;
      if (m >= kScanChunk) {
#pragma unroll
        for (int i = 0; i < kScanChunk; ++i, y += p.y_stride) {
          h = fma2(a[i], h, u[i]);
          store_pair<ACC>(y, l, h);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kScanChunk; ++i, y += p.y_stride) {
          if (i < m) {
            h = fma2(a[i], h, u[i]);
            store_pair<ACC>(y, l, h);
          }
        }
      }
    }
    if (p.hT && rank == 0 && warp == 0) store_state(p.hT, pos.n, p.D, l, carry);
  }
  cp_async_wait<0>();
  if (!ok) set_err(p.err, KDA_ERR_TIMEOUT);
  __syncwarp();
  if (S > 1) cluster_sync_all();  // no CTA ends while another may still write to it
}

// Backward: the same over the chunks from the last to the first, with the map of
// d (the gradient of a state) over a chunk; the states within a chunk come from
// h_chunks, so the forward direction needs no exchange.
template <typename X, typename G, int ACC, int W>
__global__ void __launch_bounds__(32 * W, 2 * kWarps / W) kda_scan_bwd_kernel(const kda_scan_bwd_args q, int S) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ ScanSmem<W> sm;
  constexpr size_t kStage = 2 * tile_bytes<X>() + tile_bytes<G>();
  constexpr int kStages = stages_for(kStage, W);
  const kda_scan_args& p = q.fwd;
  const int warp = threadIdx.x >> 5, rank = blockIdx.x % S, warps = cta_warps<W>();
  const Lane l = lane_channels<ACC>(blockIdx.x / S * kBlockCh, p.D);
  const bool comp = p.flags & KDA_SCAN_FLAG_COMPLEMENT, logits = p.gate_mode == KDA_SCAN_LOGITS;
  unsigned char* mine_ring = ring + warp * kStages * kStage;
  scan_prologue(sm, S);
  int it = 0;
  bool ok = true;
  Sequences pos;
  bool more = first_sequence<W>(p, pos, reinterpret_cast<int*>(sm.warp));
  for (; more; more = next_sequence(p, pos)) {
    const int len = pos.end - pos.start, chunks = (len + kScanChunk - 1) / kScanChunk;
    auto tile_x = [&](int slot) { return Tile<X, ACC>{reinterpret_cast<Raw2<X>*>(mine_ring + slot * kStage)}; };
    auto tile_d = [&](int slot) { return Tile<X, ACC>{reinterpret_cast<Raw2<X>*>(mine_ring + slot * kStage + tile_bytes<X>())}; };
    auto tile_g = [&](int slot) { return Tile<G, ACC>{reinterpret_cast<Raw2<G>*>(mine_ring + slot * kStage + 2 * tile_bytes<X>())}; };
    // this warp's chunk of advance j (negative: none left)
    auto chunk_of = [&](int j) { return chunks - 1 - ((j * S + rank) * warps + warp); };
    auto fetch = [&](int j, int slot) {
      const int k = chunk_of(j);
      if (k >= 0) {
        const int m = len - k * kScanChunk;
        const long long t0 = pos.start + static_cast<long long>(k) * kScanChunk;
        tile_x(slot).fetch(static_cast<const X*>(p.x) + t0 * p.x_stride, p.x_stride, m, l, p.D);
        tile_g(slot).fetch(static_cast<const G*>(p.gate) + t0 * p.gate_stride, p.gate_stride, m, l, p.D);
        tile_d(slot).fetch(static_cast<const X*>(q.dy) + t0 * q.dy_stride, q.dy_stride, m, l, p.D);
      }
      cp_async_commit();
    };
    auto chunk_state = [&](int j) {
      const int k = chunk_of(j);
      return k >= 0 ? load_state(p.h_chunks, pos.chunk_base + k, p.D, l) : make_float2(0.f, 0.f);
    };
    float2 carry = load_state(q.dhT, pos.n, p.D, l), next_h = chunk_state(0);
    for (int j = 0; j < kStages - 1; ++j) fetch(j, j);
    int slot = 0;  // of advance j; its stage before is the one to fill
    for (int j = 0; j * S * warps < chunks; ++j, ++it, slot = slot + 1 == kStages ? 0 : slot + 1) {
      const int k = chunk_of(j), m = k < 0 ? 0 : len - k * kScanChunk;
      const float2 h = next_h;
      next_h = chunk_state(j + 1);
      fetch(j + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const Tile<X, ACC> tx = tile_x(slot), td = tile_d(slot);
      float2 a[kScanChunk], w[kScanChunk];  // decay; what d multiplies in the decay's gradient
      const Tile<G, ACC> tg = tile_g(slot);
      read_tiles(a, w, tg, tx);
      if (logits) {
        if (comp) run_through<KDA_SCAN_LOGITS, true>(a, w, h, tg, tx);
        else run_through<KDA_SCAN_LOGITS, false>(a, w, h, tg, tx);
      } else {
        if (comp) run_through<KDA_SCAN_LOG_DECAY, true>(a, w, h, tg, tx);
        else run_through<KDA_SCAN_LOG_DECAY, false>(a, w, h, tg, tx);
      }
      Map mine = identity_map();  // d -> a (d + dy), last token first
      if (m >= kScanChunk) {
#pragma unroll
        for (int i = kScanChunk - 1; i >= 0; --i) mine = then(mine, Map{a[i], mul2(a[i], td.get(i))});
      } else {
#pragma unroll
        for (int i = kScanChunk - 1; i >= 0; --i)
          if (i < m) mine = then(mine, Map{a[i], mul2(a[i], td.get(i))});
      }
      keep_nonzero(mine, a, m);
      float2 d = enter_state(sm, mine, carry, ok, it, S, rank);
      const long long last = pos.start + static_cast<long long>(k) * kScanChunk + kScanChunk - 1;
      X* dx = static_cast<X*>(q.dx) + last * q.dx_stride;
      G* dg = static_cast<G*>(q.dgate) + last * q.dgate_stride;
      auto token = [&](int i) {
        float2 b = make_float2(1.f, 1.f);  // 1 - a, where it is needed
        if (logits || comp) b = get_pair(tg, tx, i);
        d = add2(d, td.get(i));
        store_pair<ACC>(dx, l, comp ? mul2(b, d) : d);
        d = mul2(a[i], d);
        const float2 g = mul2(d, w[i]);
        store_pair<ACC>(dg, l, logits ? mul2(b, g) : g);
      };
      if (m >= kScanChunk) {
#pragma unroll
        for (int i = kScanChunk - 1; i >= 0; --i, dx -= q.dx_stride, dg -= q.dgate_stride) token(i);
      } else {
#pragma unroll
        for (int i = kScanChunk - 1; i >= 0; --i, dx -= q.dx_stride, dg -= q.dgate_stride)
          if (i < m) token(i);
      }
      __syncwarp();  // the slots are free for the fetch of the next iteration
    }
    if (q.dh0 && rank == 0 && warp == 0) store_state(q.dh0, pos.n, p.D, l, carry);
  }
  cp_async_wait<0>();
  if (!ok) set_err(p.err, KDA_ERR_TIMEOUT);
  __syncwarp();
  if (S > 1) cluster_sync_all();  // no CTA ends while another may still write to it
}

// One token: C channels a thread (4 where the rows allow their accesses), rows of
// the batch strided over the grid.
template <typename X, typename G, int C>
__global__ void __launch_bounds__(kStepThreads) kda_scan_step_kernel(const kda_scan_step_args p) {
  const unsigned c = (blockIdx.x * kStepThreads + threadIdx.x) * C;  // (may pass 2^31)
  if (c >= static_cast<unsigned>(p.D)) return;
  for (long long b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int slot = p.indices[b];
    const bool live = slot >= 0 && slot < p.num_slots;
    if (!live && slot >= 0 && c == 0) set_err(p.err, KDA_ERR_INVALID_ARG);
    const G* gate = static_cast<const G*>(p.gate) + b * p.gate_stride + c;
    const X* x = static_cast<const X*>(p.x) + b * p.x_stride + c;
    X* y = static_cast<X*>(p.y) + b * p.y_stride + c;
    float f[C], u[C], h[C];
    if (C == 4) {
      load4(gate, f);
      load4(x, u);
    } else {
      f[0] = load_f(gate);
      u[0] = load_f(x);
    }
    const long long at = static_cast<long long>(live ? slot : 0) * p.D + c;
#pragma unroll
    for (int j = 0; j < C; ++j) h[j] = 0.f;
    if (live) {
      if (C == 4) load4(p.state_in + at, h);
      else h[0] = p.state_in[at];
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const float2 pair = make_float2(f[j], f[j]);
        const bool log = p.gate_mode == KDA_SCAN_LOG_DECAY;
        const float2 a = log ? decay_of<KDA_SCAN_LOG_DECAY, G>(pair) : decay_of<KDA_SCAN_LOGITS, G>(pair);
        if (p.flags & KDA_SCAN_FLAG_COMPLEMENT)
          u[j] *= (log ? rest_of<KDA_SCAN_LOG_DECAY, G>(pair, a) : rest_of<KDA_SCAN_LOGITS, G>(pair, a)).x;
        h[j] = fmaf(a.x, h[j], u[j]);
      }
      if (C == 4) store4(p.state_out + at, h);
      else p.state_out[at] = h[0];
    }
    if (C == 4) store4(y, h);
    else store_f(y, h[0]);
  }
}

size_t elem_bytes(int32_t dt) { return dt == KDA_DTYPE_FP32 ? 4 : 2; }

// How rows of D channels at p can be accessed: the widest of 16 bytes, a pair, one
// channel that D, the stride and the address are all multiples of.
int access_of(const void* p, int64_t stride, int D, int32_t dt) {
  const int64_t e = static_cast<int64_t>(elem_bytes(dt));
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  if (D * e % 16 == 0 && stride * e % 16 == 0 && at % 16 == 0) return kWide;
  return D % 2 == 0 && stride % 2 == 0 && at % (2 * e) == 0 ? kPair : kSingle;
}

// What one instance of a kernel remembers of each device: whether its shared-memory
// limit has been raised, and how many of its clusters of each size are resident at once.
struct Instance {
  std::atomic<uint64_t> smem_set{0};
  DeviceCounts<kMaxCluster + 1> resident;
};

template <int W, typename Args>
cudaError_t launch_clusters(void (*kernel)(Args, int), Instance& inst, size_t warp_smem, const Args& a, const kda_scan_args& f,
                            cudaStream_t s) {
  cudaError_t e = set_smem_limit_once(kernel, W * warp_smem, inst.smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int warps = W == kWarps ? kWarps : std::max(1, (f.T + kScanChunk - 1) / kScanChunk);
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = warps * warp_smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  // The most CTAs a cluster that leave the whole grid resident at once, no more than
  // the sequences (their mean length, where they are packed) have chunks for: with
  // clusters of 7, which the GPU's groups of SMs hold 38 of, 40 channel blocks of
  // 8192 tokens take two rounds and 54 us, with clusters of 5 one. Packed sequences
  // differ in length, so they get up to two rounds, which, longest first, even the
  // lengths out (16 of 512 to 8192 tokens, 1000 channels: 250 us forward and backward
  // with clusters of 2, 260 with 4, 290 with 1).
  const long long blocks = (f.D + kBlockCh - 1) / kBlockCh, work = blocks * f.N;
  const long long mean = f.cu_seqlens ? (static_cast<long long>(f.T) + f.N - 1) / f.N : f.T;
  const int rounds = f.cu_seqlens && f.N > 1 ? 2 : 1;
  int device = 0;
  e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  int S = kMaxCluster;
  for (; S > 1; --S) {
    if (mean <= static_cast<long long>(S - 1) * kWarps * kScanChunk) continue;
    int fit = 0;
    e = static_cast<cudaError_t>(inst.resident.get(device, S, &fit, [&](int* count) {
      attr.val.clusterDim.x = S;
      cfg.gridDim = dim3(S);
      return static_cast<int>(cudaOccupancyMaxActiveClusters(count, kernel, &cfg));
    }));
    if (e != cudaSuccess) return e;
    if (work <= static_cast<long long>(fit) * rounds) break;
  }
  attr.val.clusterDim.x = S;
  long long rows = f.N < 65535 ? f.N : 65535;
  // (many packed sequences: runs of them, eight rounds of CTAs in all)
  if (f.cu_seqlens && f.N > kThreads) rows = std::min(rows, std::max<long long>(kThreads, 8 * 2 * 152 / blocks));
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * S), static_cast<unsigned>(rows));
  return cudaLaunchKernelEx(&cfg, kernel, a, S);
}

// Equal sequences of up to kShortWarps chunks get a warp for each and one stage of
// tiles, so that an SM holds many of them: 256 of 16 tokens, 1024 channels: 10 us
// forward and 15 backward, three to six times that with the eight warps and the ring that
// long ones need. How short the sequences of a packed batch are only the GPU knows.
inline bool short_sequences(const kda_scan_args& a) { return !a.cu_seqlens && a.T <= kShortWarps * kScanChunk; }

template <typename X, typename G, int ACC, int W>
cudaError_t launch_warps(const kda_scan_args& a, cudaStream_t s) {
  static Instance inst;
  constexpr size_t stage = tile_bytes<X>() + tile_bytes<G>();
  return launch_clusters<W>(kda_scan_fwd_kernel<X, G, ACC, W>, inst, stages_for(stage, W) * stage, a, a, s);
}

template <typename X, typename G, int ACC, int W>
cudaError_t launch_warps(const kda_scan_bwd_args& a, cudaStream_t s) {
  static Instance inst;
  constexpr size_t stage = 2 * tile_bytes<X>() + tile_bytes<G>();
  return launch_clusters<W>(kda_scan_bwd_kernel<X, G, ACC, W>, inst, stages_for(stage, W) * stage, a, a.fwd, s);
}

inline const kda_scan_args& fwd_of(const kda_scan_args& a) { return a; }
inline const kda_scan_args& fwd_of(const kda_scan_bwd_args& a) { return a.fwd; }

template <typename X, typename G, int ACC, typename Args>
cudaError_t launch_acc(const Args& a, cudaStream_t s) {
  return short_sequences(fwd_of(a)) ? launch_warps<X, G, ACC, kShortWarps>(a, s) : launch_warps<X, G, ACC, kWarps>(a, s);
}
template <typename X, typename G, typename Args>
cudaError_t launch_any(const Args& a, int acc, cudaStream_t s) {
  return acc == kWide   ? launch_acc<X, G, kWide>(a, s)
         : acc == kPair ? launch_acc<X, G, kPair>(a, s)
                        : launch_acc<X, G, kSingle>(a, s);
}

// The instance for a call's types: x bf16 with a bf16 or fp32 gate, or both fp32.
template <typename Args>
cudaError_t launch_types(const Args& a, const kda_scan_args& f, int acc, cudaStream_t s) {
  if (f.dtype == KDA_DTYPE_FP32) return launch_any<float, float>(a, acc, s);
  if (f.gate_dtype == KDA_DTYPE_FP32) return launch_any<__nv_bfloat16, float>(a, acc, s);
  return launch_any<__nv_bfloat16, __nv_bfloat16>(a, acc, s);
}

}  // namespace

cudaError_t launch_scan_fwd(const kda_scan_args& a, cudaStream_t s) {
  int acc = kWide;
  for (const int v : {access_of(a.x, a.x_stride, a.D, a.dtype), access_of(a.gate, a.gate_stride, a.D, a.gate_dtype),
                      access_of(a.y, a.y_stride, a.D, a.dtype)})
    acc = v < acc ? v : acc;
  return launch_types(a, a, acc, s);
}

cudaError_t launch_scan_bwd(const kda_scan_bwd_args& a, cudaStream_t s) {
  const kda_scan_args& f = a.fwd;
  int acc = kWide;
  for (const int v : {access_of(f.x, f.x_stride, f.D, f.dtype), access_of(f.gate, f.gate_stride, f.D, f.gate_dtype),
                      access_of(a.dy, a.dy_stride, f.D, f.dtype), access_of(a.dx, a.dx_stride, f.D, f.dtype),
                      access_of(a.dgate, a.dgate_stride, f.D, f.gate_dtype)})
    acc = v < acc ? v : acc;
  return launch_types(a, f, acc, s);
}

namespace {

template <typename X, typename G>
cudaError_t launch_step(const kda_scan_step_args& a, cudaStream_t s) {
  // four channels an access: 16 bytes of fp32, 8 of bf16
  auto fours = [&](const void* p, int64_t stride, size_t elem) {
    return reinterpret_cast<uintptr_t>(p) % (4 * elem) == 0 && stride % 4 == 0;
  };
  const bool four = a.D % 4 == 0 && fours(a.x, a.x_stride, sizeof(X)) && fours(a.gate, a.gate_stride, sizeof(G)) &&
                    fours(a.y, a.y_stride, sizeof(X)) && fours(a.state_in, 0, 4) && fours(a.state_out, 0, 4);
  const int per = kStepThreads * (four ? 4 : 1);
  const dim3 grid(static_cast<unsigned>((a.D - 1) / per + 1), static_cast<unsigned>(std::min(a.B, 65535)));
  if (four) kda_scan_step_kernel<X, G, 4><<<grid, kStepThreads, 0, s>>>(a);
  else kda_scan_step_kernel<X, G, 1><<<grid, kStepThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_step(const kda_scan_step_args& a, cudaStream_t s) {
  if (a.dtype == KDA_DTYPE_FP32) return launch_step<float, float>(a, s);
  if (a.gate_dtype == KDA_DTYPE_FP32) return launch_step<__nv_bfloat16, float>(a, s);
  return launch_step<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace kda
