// Projection with its epilogue: y = act((x w^T) xs[m] ws[n] + bias[n]) + residual.
//
// One CTA computes a tile of 128 outputs (rows of w, the M side of the tensor
// core's product) x TOK tokens (rows of x, its N side): thread i of the four
// epilogue warps then holds output i of the tile in tensor-memory lane i, so bias
// and weight scale are one value per thread, and a warp's stores of one token are
// 32 consecutive outputs. Operands go through shared memory in blocks of 128
// bytes along K (64 bf16 or 128 e4m3 values), in the 128-byte swizzle.
//
// Roles: warps 0-3 the epilogue, warp 4 issues the MMAs, warp 5 the TMA loads
// through a ring of stages. Rows that TMA cannot describe (an address or a row
// pitch that is no multiple of 16 bytes) are copied by sixteen loader warps
// instead.
//
// Few tiles (small M) leave most SMs without work, so a cluster of S CTAs splits
// K of one tile: each sums its share, puts it into its own shared memory, and
// finishes 1/S of the tokens from all S (distributed shared memory), in the
// order of the ranks, so results do not vary from run to run.
#include "kda_linear.cuh"

namespace kda {
namespace {

using namespace linear;

constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;
constexpr int kEpiThreads = 128;
constexpr int kTmaThreads = kEpiThreads + 64;       // + MMA warp, TMA warp
constexpr int kLoaders = 16;
constexpr int kRawStages = 4;
constexpr int kCopyThreads = kEpiThreads + 32 + 32 * kLoaders;  // + MMA warp, loader warps

struct LinearHead {
  uint64_t full[kMaxStages], empty[kMaxStages], acc;
  uint32_t tmem_base;
  int failed;
};

// The operand rows of a tile for rows that start at any byte: warp `warp` of the 16
// loaders brings rows warp, warp + 16, .. of the 128 + TOK (first w's, then x's).
// fetch() starts copies of the aligned 4-byte words that hold a row's 128 bytes (33
// of them; bytes past the row and rows past the end are zero-filled) into raw
// shared memory that only this warp uses; place() shifts them into the swizzled
// tile (16-byte chunk c of row r at chunk c ^ (r % 8)). What bounds it is the
// instructions per row and block: 12 here, 96 in a first form that formed every
// word's address and length anew (777 x 1001 -> 1111: 55 us, now 26).
template <typename E, int TOK>
struct RowLoader {
  static constexpr int kPer = (kOut + TOK) / kLoaders;   // rows of a warp
  static constexpr int kPitch = 33;                      // words of a raw row
  static constexpr uint32_t kRawWords = kLoaders * kPer * kPitch;
  const unsigned char* w;
  const unsigned char* x;
  long long w_pitch, x_pitch, row_bytes;
  int n, m, n_end, m_end, warp;  // this warp's first rows
  __device__ __forceinline__ RowLoader(const kda_linear_args& p, int n0, int m0, int loader)
      : w_pitch(p.ldw * static_cast<long long>(sizeof(E))), x_pitch(p.ldx * static_cast<long long>(sizeof(E))),
        row_bytes(p.K * static_cast<long long>(sizeof(E))), n(n0 + loader), m(m0 + loader), n_end(p.N), m_end(p.M), warp(loader) {
    w = static_cast<const unsigned char*>(p.w) + n * w_pitch;
    x = static_cast<const unsigned char*>(p.x) + m * x_pitch;
  }
  // Row j of the warp: where it starts, and whether it exists. Rows that do not are
  // left alone: what they put into the tile reaches outputs that are not stored.
  __device__ __forceinline__ const unsigned char* row(int j) const {
    return j < kOut / kLoaders ? w + j * kLoaders * w_pitch : x + (j - kOut / kLoaders) * kLoaders * x_pitch;
  }
  __device__ __forceinline__ bool live(int j) const {
    return j < kOut / kLoaders ? n + j * kLoaders < n_end : m + (j - kOut / kLoaders) * kLoaders < m_end;
  }
  __device__ __forceinline__ bool first_of_matrix(int j) const {
    return j < kOut / kLoaders ? n + j * kLoaders == 0 : m + (j - kOut / kLoaders) * kLoaders == 0;
  }
  __device__ __forceinline__ static uint32_t shift_of(const unsigned char* p) { return reinterpret_cast<uintptr_t>(p) & 3; }
  // Word `word` of row j at byte `at`, where the row may end inside it or start
  // after it. (The word that the first row of a matrix starts inside of would begin
  // before the matrix; place() reads the row's first bytes by themselves.)
  __device__ __forceinline__ void copy_edge_word(uint32_t* dst, int j, long long at, int word) const {
    const unsigned char* p = row(j);
    const long long off = at + 4 * word - shift_of(p), left = row_bytes - off;
    if (!live(j) || (off < 0 && first_of_matrix(j))) return;
    if (left <= 0) {
      *dst = 0u;
      return;
    }
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(p + off),
                 "r"(left < 4 ? static_cast<uint32_t>(left) : 4u)
                 : "memory");
  }
  __device__ __forceinline__ static void copy_word(uint32_t* dst, const unsigned char* p) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uintptr_t>(p) & ~uintptr_t{3})
                 : "memory");
  }
  __device__ __forceinline__ void fetch(uint32_t* raw, int block) const {
    const int lane = threadIdx.x & 31;
    const long long at = static_cast<long long>(block) * kKBytes;
    raw += warp * kPer * kPitch;
    if (block > 0 && at + 4 * kPitch <= row_bytes) {  // every word of the block lies inside its row
      const unsigned char* p = w + at + 4 * lane;
#pragma unroll
      for (int j = 0; j < kOut / kLoaders; ++j, p += kLoaders * w_pitch)
        if (live(j)) copy_word(raw + j * kPitch + lane, p);
      p = x + at + 4 * lane;
#pragma unroll
      for (int j = kOut / kLoaders; j < kPer; ++j, p += kLoaders * x_pitch)
        if (live(j)) copy_word(raw + j * kPitch + lane, p);
      if (lane < kPer && live(lane)) copy_word(raw + lane * kPitch + 32, row(lane) + at + 4 * 32);
    } else {
#pragma unroll 1
      for (int j = 0; j < kPer; ++j) copy_edge_word(raw + j * kPitch + lane, j, at, lane);
      if (lane < kPer) copy_edge_word(raw + lane * kPitch + 32, lane, at, 32);
    }
  }
  __device__ __forceinline__ void place(uint32_t* raw, unsigned char* tile, int block) const {
    const int lane = threadIdx.x & 31;
    raw += warp * kPer * kPitch;
    if (block == 0) {  // the word a row starts inside of, element by element: lane j does row j
      if (lane < kPer && live(lane)) {
        const unsigned char* p = row(lane);
        const int shift = static_cast<int>(shift_of(p)), E_ = static_cast<int>(sizeof(E));
        uint32_t first = 0;
        for (int i = 0; i * E_ + shift < 4 && i * E_ < row_bytes; ++i)
          first |= static_cast<uint32_t>(reinterpret_cast<const E*>(p)[i]) << (8 * (shift + E_ * i));
        raw[lane * kPitch] = first;
      }
      __syncwarp();
    }
    unsigned char* dst = tile + warp * kKBytes + (((lane >> 2) ^ (warp & 7)) << 4) + 4 * (lane & 3);
    const uint32_t w_low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(w)), w_step = static_cast<uint32_t>(kLoaders * w_pitch);
    const uint32_t x_low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x)), x_step = static_cast<uint32_t>(kLoaders * x_pitch);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t low = j < kOut / kLoaders ? w_low + j * w_step : x_low + (j - kOut / kLoaders) * x_step;
      // (the funnel shift takes the distance modulo 32: 8 * (address % 4))
      *reinterpret_cast<uint32_t*>(dst + j * kLoaders * kKBytes) =
          __funnelshift_r(raw[j * kPitch + lane], raw[j * kPitch + lane + 1], 8 * low);
    }
  }
};

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Tokens c .. c_end - 1 of the tile from the sums of all S CTAs (part: [token][output]
// in each one's shared memory), C tokens at a time so that their reads overlap.
template <int C, typename Y>
__device__ __forceinline__ void finish_shared(const Epilogue<Y>& finish, const float* part, int c, int c_end, int m0, int M,
                                              int S, int out) {
  for (; c < c_end && m0 + c < M; c += C) {
    float v[C];
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = 0.f;
    const uint32_t at = smem_u32(part + c * kOut + out);
#pragma unroll 2
    for (int r = 0; r < S; ++r) {
      const uint32_t peer = mapa_shared(at, r);
      float u[C];
#pragma unroll
      for (int j = 0; j < C; ++j) u[j] = ld_shared_cluster_f32(peer + j * kOut * 4);
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] += u[j];
    }
    finish(v, static_cast<long long>(m0) + c);
  }
}

// Grid (S * output tiles, token tiles), cluster (S, 1, 1).
// E: bits of an operand element (uint16_t bf16, uint8_t e4m3).
template <typename E, typename Y, int TOK, bool TMA>
__global__ void __launch_bounds__(TMA ? kTmaThreads : kCopyThreads)
    kda_linear_kernel(const kda_linear_args p, const __grid_constant__ CUtensorMap wmap,
                      const __grid_constant__ CUtensorMap xmap, int S, int stages) {
  extern __shared__ unsigned char raw[];
  __shared__ LinearHead sm;
  constexpr uint32_t kWBytes = kOut * kKBytes, kXBytes = TOK * kKBytes, kStage = kWBytes + kXBytes;
  constexpr int EPB = kKBytes / sizeof(E);
  constexpr uint32_t kCols = TOK < 32 ? 32 : TOK;
  unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % S;
  const int n0 = blockIdx.x / S * kOut, m0 = blockIdx.y * TOK;
  const int blocks = (p.K + EPB - 1) / EPB;
  const int kb0 = static_cast<int>(static_cast<long long>(blocks) * rank / S);
  const int nkb = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / S) - kb0;

  if (TMA && warp == 5 && lane == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
  }
  if (warp == 0) {
    tc05::tmem_alloc(&sm.tmem_base, kCols);
    tc05::tmem_relinquish();
  }
  if (tid == kEpiThreads) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sm.full[i], TMA ? 1 : kLoaders);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.acc, 1);
    sm.failed = 0;
    fence_mbarrier_init_cluster();
  }
  tc05::fence_before_sync();
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;

  if (warp == 4) {
    if (lane == 0) {
      constexpr uint32_t idesc = tc05::idesc_f16kind(kOut, TOK, sizeof(E) == 2);
      bool ok = true;
      for (int i = 0; i < nkb && ok; ++i) {
        const int s = i % stages;
        ok = mbar_wait_bounded(smem_u32(&sm.full[s]), (i / stages) & 1, kLinearWaitNs);
        if (!ok) break;
        tc05::fence_after_sync();
        const uint32_t w = smem_u32(ring + s * kStage), x = w + kWBytes;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t wd = tc05::smem_desc(w + 32 * k, 16, 1024, tc05::kSwizzle128B);
          const uint64_t xd = tc05::smem_desc(x + 32 * k, 16, 1024, tc05::kSwizzle128B);
          if (sizeof(E) == 2) tc05::mma_ss(tmem, wd, xd, idesc, i > 0 || k > 0);
          else mma_ss_f8(tmem, wd, xd, idesc, i > 0 || k > 0);
        }
        tc05::commit(&sm.empty[s]);
      }
      if (ok) tc05::commit(&sm.acc);
      else sm.failed = 1;
    }
  } else if (TMA && warp == 5) {
    if (lane == 0) {
      bool ok = true;
      int i = 0;
      for (; i < nkb; ++i) {
        const int s = i % stages;
        if (i >= stages) ok = mbar_wait_bounded(smem_u32(&sm.empty[s]), (i / stages - 1) & 1, kLinearWaitNs);
        if (!ok) break;
        const uint32_t w = smem_u32(ring + s * kStage), bar = smem_u32(&sm.full[s]);
        mbar_arrive_expect_tx_local(&sm.full[s], kStage);
        tma_load_2d(w, &wmap, (kb0 + i) * EPB, n0, bar);
        tma_load_2d(w + kWBytes, &xmap, (kb0 + i) * EPB, m0, bar);
      }
      if (!ok) sm.failed = 1;
      // no copy is left in flight when the CTA ends
      for (int j = i > stages ? i - stages : 0; j < i; ++j)
        mbar_wait_bounded(smem_u32(&sm.full[j % stages]), (j / stages) & 1, kLinearWaitNs);
    }
  } else if (!TMA && warp >= 5) {
    const RowLoader<E, TOK> rows(p, n0, m0, warp - 5);
    uint32_t* raws = reinterpret_cast<uint32_t*>(ring + stages * kStage);
    auto raw = [&](int i) { return raws + (i % kRawStages) * RowLoader<E, TOK>::kRawWords; };
    bool ok = true;
    for (int i = 0; i < kRawStages - 1; ++i) {
      if (i < nkb) rows.fetch(raw(i), kb0 + i);
      cp_async_commit();
    }
    for (int i = 0; i < nkb; ++i) {
      if (i + kRawStages - 1 < nkb) rows.fetch(raw(i + kRawStages - 1), kb0 + i + kRawStages - 1);
      cp_async_commit();
      cp_async_wait<kRawStages - 1>();
      __syncwarp();
      const int s = i % stages;
      if (i >= stages) ok = mbar_wait_bounded(smem_u32(&sm.empty[s]), (i / stages - 1) & 1, kLinearWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      rows.place(raw(i), ring + s * kStage, kb0 + i);
      fence_proxy_async_smem();
      __syncwarp();  // (also: the raw words have been read before their next copies start)
      if (lane == 0) mbar_arrive_local(&sm.full[s]);
    }
    cp_async_wait<0>();
    if (!ok) sm.failed = 1;
  }
  __syncwarp();

  bool ok = true;
  if (warp < 4) ok = mbar_wait_bounded(smem_u32(&sm.acc), 0, kLinearWaitNs);
  if (!ok) sm.failed = 1;
  tc05::fence_after_sync();
  const uint32_t tlane = tmem + (static_cast<uint32_t>(32 * warp) << 16);
  if (S == 1) {
    if (warp < 4 && __all_sync(0xffffffffu, ok)) {
      const Epilogue<Y> finish(p, n0 + tid);
      for (int c0 = 0; c0 < TOK && m0 + c0 < p.M; c0 += 16) {
        float v[16];
        tmem_load(tlane + c0, v);
        finish(v, static_cast<long long>(m0) + c0);
      }
    }
  } else {
    // this CTA's sums, token by token, over the ring (every copy and MMA is done)
    float* part = reinterpret_cast<float*>(ring);
    if (warp < 4 && __all_sync(0xffffffffu, ok)) {
      for (int c0 = 0; c0 < TOK; c0 += 16) {
        float v[16];
        tmem_load(tlane + c0, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c0 + j) * kOut + tid] = v[j];
      }
    }
    cluster_sync_all();
    if (warp < 4) {
      const Epilogue<Y> finish(p, n0 + tid);
      const int per = TOK / S;
      if (per % 8 == 0) finish_shared<8>(finish, part, rank * per, (rank + 1) * per, m0, p.M, S, tid);
      else finish_shared<2>(finish, part, rank * per, (rank + 1) * per, m0, p.M, S, tid);
    }
    cluster_sync_all();  // nobody reads this CTA's shared memory any more
  }
  tc05::fence_before_sync();
  __syncthreads();
  if (tid == 0 && sm.failed) set_err(p.err, KDA_ERR_TIMEOUT);
  if (warp == 0) {
    tc05::fence_after_sync();
    tc05::tmem_dealloc(tmem, kCols);
  }
}

template <typename E, typename Y, int TOK, bool TMA>
cudaError_t launch_tile(const kda_linear_args& a, cudaStream_t s) {
  constexpr size_t stage = (kOut + TOK) * kKBytes;
  constexpr int EPB = kKBytes / sizeof(E);
  const long long gx = (static_cast<long long>(a.N) + kOut - 1) / kOut, gy = (static_cast<long long>(a.M) + TOK - 1) / TOK;
  if (gy > 65535 || gx * kMaxSplit > INT32_MAX) return cudaErrorNotSupported;
  // With TMA two CTAs share an SM's 227 KB: a ring of about 100 KB. The loaders' raw
  // words leave one CTA an SM, and one stage to fill while another is read.
  constexpr int kCtas = TMA ? 2 : 1;
  constexpr size_t kRaw = TMA ? 0 : kRawStages * RowLoader<E, TOK>::kRawWords * sizeof(uint32_t);
  constexpr int kFit = static_cast<int>(100 * 1024 / stage);
  constexpr int stages = !TMA ? 2 : kFit < kMaxStages ? kFit : kMaxStages;
  static_assert(stages * stage >= TOK * kOut * sizeof(float), "the ring holds a CTA's sums");
  // split K while the CTAs still fit the SMs and each keeps four blocks of K
  const long long blocks = (a.K + EPB - 1) / EPB;
  int S = 1;
  while (S < kMaxSplit && 2 * S <= TOK && gx * gy * S * 2 <= kCtas * 152 && blocks >= 2 * S * 4) S *= 2;
  CUtensorMap wmap = {}, xmap = {};
  if (TMA && !(encode_rows(&wmap, a.w, sizeof(E), a.K, a.N, a.ldw, kOut) && encode_rows(&xmap, a.x, sizeof(E), a.K, a.M, a.ldx, TOK)))
    return cudaErrorInvalidValue;
  constexpr size_t smem = stages * stage + kRaw + 1024;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit_once(kda_linear_kernel<E, Y, TOK, TMA>, smem, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gx * S), static_cast<unsigned>(gy));
  cfg.blockDim = dim3(TMA ? kTmaThreads : kCopyThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = S;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kda_linear_kernel<E, Y, TOK, TMA>, a, wmap, xmap, S, stages);
}

// Whether TMA can describe the rows: address and pitch on 16-byte boundaries
// (one row has no pitch).
bool tma_ok(const void* p, long long rows, long long ld, size_t elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows == 1 || ld * static_cast<long long>(elem) % 16 == 0);
}

template <typename E, typename Y>
cudaError_t launch(const kda_linear_args& a, cudaStream_t s) {
  if (!tma_ok(a.x, a.M, a.ldx, sizeof(E)) || !tma_ok(a.w, a.N, a.ldw, sizeof(E)))
    return a.M <= 16   ? launch_tile<E, Y, 16, false>(a, s)
           : a.M <= 64 ? launch_tile<E, Y, 64, false>(a, s)
                       : launch_tile<E, Y, 128, false>(a, s);
  if (a.M <= 16) return launch_tile<E, Y, 16, true>(a, s);
  if (a.M <= 32) return launch_tile<E, Y, 32, true>(a, s);
  if (a.M <= 64) return launch_tile<E, Y, 64, true>(a, s);
  return launch_linear_wide(a, s);
}

}  // namespace

cudaError_t launch_linear(const kda_linear_args& a, cudaStream_t s) {
  if (a.dtype == KDA_DTYPE_BF16)
    return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint16_t, __nv_bfloat16>(a, s) : launch<uint16_t, float>(a, s);
  return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint8_t, __nv_bfloat16>(a, s) : launch<uint8_t, float>(a, s);
}

}  // namespace kda
