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
// (distributed shared memory), and each warp composes the pairs before it with
// the carried state and runs its chunk again from the state that enters it.
// Nothing waits on memory flags: two barriers per advance, in a fixed order, so
// results do not vary from run to run.
#include "kda_cluster.cuh"
#include "kda_elem.cuh"

namespace kda {
namespace {

constexpr int kScanChunk = 16;    // tokens between the states of h_chunks, and of a warp's tile
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlockCh = 64;      // channels of a CTA
constexpr int kMaxCluster = 8;
constexpr int kStepThreads = 128;

// The decay, to about an fp32 step. Long memories multiply hundreds of decays near
// 1, so exp keeps expf's accuracy; in the sigmoid the error of e^-f is scaled by
// 1 - a, and the special-function unit's ex2 and rcp do. (e^-f = inf gives 0.)
__device__ __forceinline__ float decay_of(float f, int mode) {
  if (mode == KDA_SCAN_LOG_DECAY) return expf(f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_approx(-1.44269504f * f)));
  return r;
}

struct SeqPos {
  int start, end;        // tokens of the sequence
  long long chunk_base;  // its first chunk in h_chunks
};

// Finds sequence n, checking the whole of cu_seqlens on the way (all threads of
// the CTA call it). Returns false, after reporting, where the array is bad.
__device__ __forceinline__ bool find_sequence(const kda_scan_args& p, int n, SeqPos& pos) {
  if (p.cu_seqlens == nullptr) {
    pos.start = n * p.T;
    pos.end = pos.start + p.T;
    pos.chunk_base = static_cast<long long>(n) * ((p.T + kScanChunk - 1) / kScanChunk);
    return true;
  }
  __shared__ unsigned long long base, total;  // chunks before sequence n, of all
  __syncthreads();  // the previous sequence's have been read
  if (threadIdx.x == 0) base = total = 0;
  bool bad = threadIdx.x == 0 && (p.cu_seqlens[0] != 0 || p.cu_seqlens[p.N] != p.T);
  unsigned long long mine = 0, all = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.N; i += blockDim.x) {
    const int s = p.cu_seqlens[i], e = p.cu_seqlens[i + 1];
    bad |= e < s || s < 0 || e > p.T;
    const unsigned chunks = bad ? 0u : static_cast<unsigned>(e - s + kScanChunk - 1) / kScanChunk;
    all += chunks;
    if (i < n) mine += chunks;
  }
  if (mine != 0) atomicAdd(&base, mine);
  if (all != 0) atomicAdd(&total, all);
  __syncthreads();
  bad |= p.h_chunks != nullptr && total > static_cast<unsigned long long>(p.h_chunks_rows);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_err(p.err, KDA_ERR_INVALID_ARG);
    return false;
  }
  pos.start = p.cu_seqlens[n];
  pos.end = p.cu_seqlens[n + 1];
  pos.chunk_base = static_cast<long long>(base);
  return true;
}

// Two channels of one token. VEC: a lane's channels are 2 lane and 2 lane + 1
// (even D and strides, aligned pointers), one access; otherwise lane and
// lane + 32, two accesses, whatever the alignment.
template <typename T>
struct Raw2;
template <>
struct Raw2<__nv_bfloat16> {
  uint32_t v;
  __device__ __forceinline__ void zero() { v = 0; }
  __device__ __forceinline__ float2 get() const {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
    const uint32_t lo = p ? *reinterpret_cast<const uint16_t*>(p) : 0u;
    const uint32_t hi = q ? *reinterpret_cast<const uint16_t*>(q) : 0u;
    v = lo | (hi << 16);
  }
};
template <>
struct Raw2<float> {
  float2 v;
  __device__ __forceinline__ void zero() { v = make_float2(0.f, 0.f); }
  __device__ __forceinline__ float2 get() const { return v; }
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ void load(const float* p, const float* q) { v = make_float2(p ? *p : 0.f, q ? *q : 0.f); }
};

__device__ __forceinline__ void store2(__nv_bfloat16* p, float2 v) { *reinterpret_cast<uint32_t*>(p) = Bf16::pack(v.x, v.y); }
__device__ __forceinline__ void store2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }

// 4- or 8-byte asynchronous copy into shared memory.
template <int BYTES>
__device__ __forceinline__ void cp_async_small(void* smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(smem)), "l"(gmem), "n"(BYTES) : "memory");
}

// A lane's two channels and which of them exist.
struct Lane {
  int c0, c1;
  bool p0, p1;
};

template <bool VEC>
__device__ __forceinline__ Lane lane_channels(int block_ch, int D) {
  const int lane = threadIdx.x & 31;
  Lane l;
  l.c0 = block_ch + (VEC ? 2 * lane : lane);
  l.c1 = block_ch + (VEC ? 2 * lane + 1 : lane + 32);
  l.p0 = l.c0 < D;
  l.p1 = l.c1 < D;
  return l;
}

template <bool VEC, typename T>
__device__ __forceinline__ Raw2<T> load_pair(const T* row, const Lane& l) {
  Raw2<T> r;
  if (VEC) {
    if (l.p0) r.load(row + l.c0);
    else r.zero();
  } else {
    r.load(l.p0 ? row + l.c0 : nullptr, l.p1 ? row + l.c1 : nullptr);
  }
  return r;
}

// One tensor's share of a warp's tile on its way in: the 16 tokens of this thread's
// two channels, in slots of shared memory that only this thread touches, so a
// thread waits for its own copies alone. fetch() starts the copies (where pairs
// cannot be copied as one word it loads and stores them); get() reads a slot.
template <typename T, bool VEC>
struct Tile {
  using Slot = Raw2<T>;
  Slot* slots;  // [token][thread]
  __device__ __forceinline__ void fetch(const T* rows, long long stride, int m, const Lane& l) const {
    if (VEC) {
      if (l.p0) {
#pragma unroll
        for (int i = 0; i < kScanChunk; ++i)
          if (i < m) cp_async_small<sizeof(Slot)>(slots + i * kThreads + threadIdx.x, rows + i * stride + l.c0);
      }
    } else {
      Slot r[kScanChunk];
#pragma unroll
      for (int i = 0; i < kScanChunk; ++i) {
        r[i].zero();
        if (i < m) r[i] = load_pair<VEC>(rows + i * stride, l);
      }
#pragma unroll
      for (int i = 0; i < kScanChunk; ++i) slots[i * kThreads + threadIdx.x] = r[i];
    }
  }
  // (a token or channel that does not exist reads what the slot held: its result is not used)
  __device__ __forceinline__ float2 get(int i) const { return slots[i * kThreads + threadIdx.x].get(); }
};
template <typename T>
constexpr size_t tile_bytes() { return sizeof(Raw2<T>) * kScanChunk * kThreads; }

template <bool VEC, typename T>
__device__ __forceinline__ void store_pair(T* row, const Lane& l, float2 v) {
  if (VEC) {
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

__device__ __forceinline__ float2 decay2(float2 f, int mode) { return make_float2(decay_of(f.x, mode), decay_of(f.y, mode)); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }

// The map h -> A h + B of some consecutive tokens, for a lane's two channels.
struct Map {
  float2 A, B;
};
__device__ __forceinline__ Map then(const Map& first, const Map& second) {
  return Map{mul2(first.A, second.A), fma2(second.A, first.B, second.B)};
}

struct ScanSmem {
  Map warp[kWarps][32];                  // this advance's maps, by warp
  Map cta[2][kMaxCluster][32];           // the CTAs' maps, by parity of the advance
};

__device__ __forceinline__ void st_cluster_map(uint32_t addr, const Map& m) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(m.A.x), "f"(m.A.y), "f"(m.B.x),
               "f"(m.B.y)
               : "memory");
}

// From this warp's map of the advance and the state `carry` that enters the
// advance (the same in every warp of the cluster): the state that enters this
// warp's chunk; carry becomes the state after the advance. All threads of the
// cluster call it.
__device__ __forceinline__ float2 enter_state(ScanSmem& sm, const Map& mine, float2& carry, int parity, int S, int rank) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  sm.warp[warp][lane] = mine;
  __syncthreads();
  Map before{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
  for (int w = 0; w < warp; ++w) before = then(before, sm.warp[w][lane]);
  if (warp == kWarps - 1) {
    const Map total = then(before, mine);
    const uint32_t at = smem_u32(&sm.cta[parity][rank][lane]);
    for (int r = 0; r < S; ++r) st_cluster_map(mapa_shared(at, r), total);
  }
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  float2 h = carry, in = carry;
  for (int r = 0; r < S; ++r) {
    if (r == rank) in = h;
    const Map& m = sm.cta[parity][r][lane];
    h = fma2(m.A, h, m.B);
  }
  carry = h;
  return fma2(before.A, in, before.B);
}

// Stages of the ring of tiles: what leaves two CTAs on an SM (about 100 KB each),
// at least two.
constexpr int stages_for(size_t stage) { return 100 * 1024 / stage >= 3 ? 3 : 2; }

// Forward. Grid (S * channel blocks, sequences), cluster (S, 1, 1).
template <typename X, typename G, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) kda_scan_fwd_kernel(const kda_scan_args p, int S) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ ScanSmem sm;
  constexpr size_t kStage = tile_bytes<X>() + tile_bytes<G>();
  constexpr int kStages = stages_for(kStage);
  const int warp = threadIdx.x >> 5, rank = blockIdx.x % S, advance = S * kWarps * kScanChunk;
  const Lane l = lane_channels<VEC>(blockIdx.x / S * kBlockCh, p.D);
  const bool comp = p.flags & KDA_SCAN_FLAG_COMPLEMENT;
  if (S > 1) cluster_sync_all();  // every CTA of the cluster runs before its shared memory is written
  int parity = 0;
  for (int n = blockIdx.y; n < p.N; n += gridDim.y) {
    SeqPos pos;
    if (!find_sequence(p, n, pos)) return;  // (the same answer in every CTA)
    const int len = pos.end - pos.start;
    // the tiles of advance j, whose first token for this warp is i0
    auto tile_x = [&](int j) { return Tile<X, VEC>{reinterpret_cast<Raw2<X>*>(ring + (j % kStages) * kStage)}; };
    auto tile_g = [&](int j) { return Tile<G, VEC>{reinterpret_cast<Raw2<G>*>(ring + (j % kStages) * kStage + tile_bytes<X>())}; };
    auto first = [&](int j) { return j * advance + (rank * kWarps + warp) * kScanChunk; };
    auto fetch = [&](int j) {
      const int i0 = first(j);
      if (i0 < len) {
        const long long t0 = pos.start + static_cast<long long>(i0);
        tile_x(j).fetch(static_cast<const X*>(p.x) + t0 * p.x_stride, p.x_stride, len - i0, l);
        tile_g(j).fetch(static_cast<const G*>(p.gate) + t0 * p.gate_stride, p.gate_stride, len - i0, l);
      }
      cp_async_commit();
    };
    float2 carry = load_state(p.h0, n, p.D, l);
    for (int j = 0; j < kStages - 1; ++j) fetch(j);
    for (int j = 0; j * static_cast<long long>(advance) < len; ++j, parity ^= 1) {
      fetch(j + kStages - 1);
      cp_async_wait<kStages - 1>();
      const int i0 = first(j), m = min(kScanChunk, len - i0);
      const Tile<X, VEC> tx = tile_x(j);
      const Tile<G, VEC> tg = tile_g(j);
      float2 a[kScanChunk], u[kScanChunk];
      Map mine{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < kScanChunk; ++i) {
        a[i] = decay2(tg.get(i), p.gate_mode);
        u[i] = tx.get(i);
        if (comp) u[i] = make_float2((1.f - a[i].x) * u[i].x, (1.f - a[i].y) * u[i].y);
        if (i < m) mine = then(mine, Map{a[i], u[i]});
      }
      float2 h = enter_state(sm, mine, carry, parity, S, rank);
      if (m > 0) {
        if (p.h_chunks) store_state(p.h_chunks, pos.chunk_base + i0 / kScanChunk, p.D, l, h);
        X* y = static_cast<X*>(p.y) + (pos.start + static_cast<long long>(i0)) * p.y_stride;
#pragma unroll
        for (int i = 0; i < kScanChunk; ++i) {
          if (i < m) {
            h = fma2(a[i], h, u[i]);
            store_pair<VEC>(y + i * p.y_stride, l, h);
          }
        }
      }
    }
    if (p.hT && rank == 0 && warp == 0) store_state(p.hT, n, p.D, l, carry);
  }
}

// Backward: the same over the chunks from the last to the first, with the map of
// d (the gradient of a state) over a chunk; the states within a chunk come from
// h_chunks, so the forward direction needs no exchange.
template <typename X, typename G, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) kda_scan_bwd_kernel(const kda_scan_bwd_args q, int S) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ ScanSmem sm;
  constexpr size_t kStage = 2 * tile_bytes<X>() + tile_bytes<G>();
  constexpr int kStages = stages_for(kStage);
  const kda_scan_args& p = q.fwd;
  const int warp = threadIdx.x >> 5, rank = blockIdx.x % S;
  const Lane l = lane_channels<VEC>(blockIdx.x / S * kBlockCh, p.D);
  const bool comp = p.flags & KDA_SCAN_FLAG_COMPLEMENT, logits = p.gate_mode == KDA_SCAN_LOGITS;
  if (S > 1) cluster_sync_all();  // every CTA of the cluster runs before its shared memory is written
  int parity = 0;
  for (int n = blockIdx.y; n < p.N; n += gridDim.y) {
    SeqPos pos;
    if (!find_sequence(p, n, pos)) return;
    const int len = pos.end - pos.start, chunks = (len + kScanChunk - 1) / kScanChunk;
    auto tile_x = [&](int j) { return Tile<X, VEC>{reinterpret_cast<Raw2<X>*>(ring + (j % kStages) * kStage)}; };
    auto tile_d = [&](int j) { return Tile<X, VEC>{reinterpret_cast<Raw2<X>*>(ring + (j % kStages) * kStage + tile_bytes<X>())}; };
    auto tile_g = [&](int j) { return Tile<G, VEC>{reinterpret_cast<Raw2<G>*>(ring + (j % kStages) * kStage + 2 * tile_bytes<X>())}; };
    // this warp's chunk of advance j (negative: none left)
    auto chunk_of = [&](int j) { return chunks - 1 - ((j * S + rank) * kWarps + warp); };
    auto fetch = [&](int j) {
      const int k = chunk_of(j);
      if (k >= 0) {
        const int m = len - k * kScanChunk;
        const long long t0 = pos.start + static_cast<long long>(k) * kScanChunk;
        tile_x(j).fetch(static_cast<const X*>(p.x) + t0 * p.x_stride, p.x_stride, m, l);
        tile_g(j).fetch(static_cast<const G*>(p.gate) + t0 * p.gate_stride, p.gate_stride, m, l);
        tile_d(j).fetch(static_cast<const X*>(q.dy) + t0 * q.dy_stride, q.dy_stride, m, l);
      }
      cp_async_commit();
    };
    float2 carry = load_state(q.dhT, n, p.D, l);
    for (int j = 0; j < kStages - 1; ++j) fetch(j);
    for (int j = 0; j * S * kWarps < chunks; ++j, parity ^= 1) {
      const int k = chunk_of(j), m = k < 0 ? 0 : min(kScanChunk, len - k * kScanChunk);
      const long long t0 = pos.start + static_cast<long long>(k) * kScanChunk;
      float2 h = m > 0 ? load_state(p.h_chunks, pos.chunk_base + k, p.D, l) : make_float2(0.f, 0.f);
      fetch(j + kStages - 1);
      cp_async_wait<kStages - 1>();
      const Tile<X, VEC> tx = tile_x(j), td = tile_d(j);
      const Tile<G, VEC> tg = tile_g(j);
      float2 a[kScanChunk], w[kScanChunk];  // decay; what d multiplies in the decay's gradient
#pragma unroll
      for (int i = 0; i < kScanChunk; ++i) {
        a[i] = decay2(tg.get(i), p.gate_mode);
        const float2 xv = tx.get(i);
        w[i] = comp ? make_float2(h.x - xv.x, h.y - xv.y) : h;
        h = comp ? fma2(a[i], w[i], xv) : fma2(a[i], h, xv);  // a h + (1 - a) x = x + a (h - x)
      }
      Map mine{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};  // d -> a (d + dy), last token first
#pragma unroll
      for (int i = kScanChunk - 1; i >= 0; --i)
        if (i < m) mine = then(mine, Map{a[i], mul2(a[i], td.get(i))});
      float2 d = enter_state(sm, mine, carry, parity, S, rank);
      X* dx = static_cast<X*>(q.dx) + t0 * q.dx_stride;
      G* dg = static_cast<G*>(q.dgate) + t0 * q.dgate_stride;
#pragma unroll
      for (int i = kScanChunk - 1; i >= 0; --i) {
        if (i < m) {
          const float2 dyv = td.get(i), b = make_float2(1.f - a[i].x, 1.f - a[i].y);
          d = make_float2(d.x + dyv.x, d.y + dyv.y);
          store_pair<VEC>(dx + i * q.dx_stride, l, comp ? mul2(b, d) : d);
          d = mul2(a[i], d);
          float2 g = mul2(d, w[i]);
          if (logits) g = mul2(b, g);
          store_pair<VEC>(dg + i * q.dgate_stride, l, g);
        }
      }
    }
    if (q.dh0 && rank == 0 && warp == 0) store_state(q.dh0, n, p.D, l, carry);
  }
}

template <typename X, typename G>
__global__ void __launch_bounds__(kStepThreads) kda_scan_step_kernel(const kda_scan_step_args p) {
  const int c = blockIdx.x * kStepThreads + threadIdx.x;
  const long long b = blockIdx.y;
  if (c >= p.D) return;
  const int slot = p.indices[b];
  X* y = static_cast<X*>(p.y) + b * p.y_stride + c;
  if (slot < 0 || slot >= p.num_slots) {
    if (slot >= 0 && c == 0) set_err(p.err, KDA_ERR_INVALID_ARG);
    store_f(y, 0.f);
    return;
  }
  const float a = decay_of(load_f(static_cast<const G*>(p.gate) + b * p.gate_stride + c), p.gate_mode);
  const float x = load_f(static_cast<const X*>(p.x) + b * p.x_stride + c);
  const long long at = static_cast<long long>(slot) * p.D + c;
  const float h = a * p.state_in[at] + (p.flags & KDA_SCAN_FLAG_COMPLEMENT ? (1.f - a) * x : x);
  p.state_out[at] = h;
  store_f(y, h);
}

// CTAs of a cluster: as many as leave the whole grid resident at once (two CTAs on
// each of 152 SMs), no more than the sequences (their mean length, where they are
// packed) have advances for. Packed sequences differ in length, so they get up to
// four times as many, whose order of execution evens the lengths out.
int cluster_size(const kda_scan_args& a) {
  const long long blocks = (a.D + kBlockCh - 1) / kBlockCh * static_cast<long long>(a.N);
  const long long mean = a.cu_seqlens ? (a.T + a.N - 1) / a.N : a.T;
  const long long room = 2 * 152 * (a.cu_seqlens && a.N > 1 ? 4 : 1);
  int S = 1;
  while (S < kMaxCluster && blocks * S * 2 <= room && mean > S * kWarps * kScanChunk) S *= 2;
  return S;
}

// Whether pairs of channels can be read as one access of 2 * elem bytes.
bool pairs_ok(const void* p, int64_t stride, size_t elem) {
  return reinterpret_cast<uintptr_t>(p) % (2 * elem) == 0 && stride % 2 == 0;
}
size_t elem_bytes(int32_t dt) { return dt == KDA_DTYPE_FP32 ? 4 : 2; }

// One instance's launch. `done` is the instance's record of devices whose
// shared-memory limit has been raised.
template <typename Args>
cudaError_t launch_clusters(void (*kernel)(Args, int), std::atomic<uint64_t>& done, size_t smem, const Args& a,
                            const kda_scan_args& f, cudaStream_t s) {
  const cudaError_t e = set_smem_limit_once(kernel, smem, done);
  if (e != cudaSuccess) return e;
  const int S = cluster_size(f);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((f.D + kBlockCh - 1) / kBlockCh * S), static_cast<unsigned>(f.N < 65535 ? f.N : 65535));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = S;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, S);
}

template <typename X, typename G, bool VEC>
cudaError_t launch_fwd(const kda_scan_args& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t stage = tile_bytes<X>() + tile_bytes<G>();
  return launch_clusters(kda_scan_fwd_kernel<X, G, VEC>, done, stages_for(stage) * stage, a, a, s);
}

template <typename X, typename G, bool VEC>
cudaError_t launch_bwd(const kda_scan_bwd_args& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t stage = 2 * tile_bytes<X>() + tile_bytes<G>();
  return launch_clusters(kda_scan_bwd_kernel<X, G, VEC>, done, stages_for(stage) * stage, a, a.fwd, s);
}

}  // namespace

// The instances by tensor types: x bf16 with a bf16 or fp32 gate, or both fp32.
#define KDA_SCAN_LAUNCH(launch, vec, xt, gt, ...)                                                        \
  ((xt) == KDA_DTYPE_FP32   ? ((vec) ? launch<float, float, true>(__VA_ARGS__) : launch<float, float, false>(__VA_ARGS__)) \
   : (gt) == KDA_DTYPE_FP32 ? ((vec) ? launch<__nv_bfloat16, float, true>(__VA_ARGS__)                   \
                                     : launch<__nv_bfloat16, float, false>(__VA_ARGS__))                 \
                            : ((vec) ? launch<__nv_bfloat16, __nv_bfloat16, true>(__VA_ARGS__)           \
                                     : launch<__nv_bfloat16, __nv_bfloat16, false>(__VA_ARGS__)))

cudaError_t launch_scan_fwd(const kda_scan_args& a, cudaStream_t s) {
  const size_t xe = elem_bytes(a.dtype), ge = elem_bytes(a.gate_dtype);
  const bool vec = a.D % 2 == 0 && pairs_ok(a.x, a.x_stride, xe) && pairs_ok(a.gate, a.gate_stride, ge) &&
                   pairs_ok(a.y, a.y_stride, xe);
  return KDA_SCAN_LAUNCH(launch_fwd, vec, a.dtype, a.gate_dtype, a, s);
}

cudaError_t launch_scan_bwd(const kda_scan_bwd_args& a, cudaStream_t s) {
  const kda_scan_args& f = a.fwd;
  const size_t xe = elem_bytes(f.dtype), ge = elem_bytes(f.gate_dtype);
  const bool vec = f.D % 2 == 0 && pairs_ok(f.x, f.x_stride, xe) && pairs_ok(f.gate, f.gate_stride, ge) &&
                   pairs_ok(a.dy, a.dy_stride, xe) && pairs_ok(a.dx, a.dx_stride, xe) &&
                   pairs_ok(a.dgate, a.dgate_stride, ge);
  return KDA_SCAN_LAUNCH(launch_bwd, vec, f.dtype, f.gate_dtype, a, s);
}

cudaError_t launch_scan_step(const kda_scan_step_args& a, cudaStream_t s) {
  if (a.B > 65535) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>((a.D + kStepThreads - 1) / kStepThreads), static_cast<unsigned>(a.B));
  if (a.dtype == KDA_DTYPE_FP32) kda_scan_step_kernel<float, float><<<grid, kStepThreads, 0, s>>>(a);
  else if (a.gate_dtype == KDA_DTYPE_FP32) kda_scan_step_kernel<__nv_bfloat16, float><<<grid, kStepThreads, 0, s>>>(a);
  else kda_scan_step_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kStepThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
