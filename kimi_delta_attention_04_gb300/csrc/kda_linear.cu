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
// pitch that is no multiple of 16 bytes) are copied by eight loader warps
// instead, two groups of four taking alternate blocks.
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
constexpr int kCopyThreads = kEpiThreads + 32 + 256;  // + MMA warp, two groups of loaders

struct LinearHead {
  uint64_t full[kMaxStages], empty[kMaxStages], acc;
  uint32_t tmem_base;
  int failed;
};

// 16 bytes of a row at byte offset `off` of [0, row_bytes): bytes past the row are
// zero. `lo` and `hi` bound the matrix's memory: where the two aligned 16-byte
// words that hold the bytes lie inside, they are read and shifted; at the
// matrix's very ends the bytes are read one element at a time.
template <typename E>
__device__ __forceinline__ uint4 load_unaligned16(const unsigned char* row, long long off, long long row_bytes,
                                                  const unsigned char* lo, const unsigned char* hi) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  const long long left = row_bytes - off;
  if (left <= 0) return make_uint4(0u, 0u, 0u, 0u);
  const unsigned char* p = row + off;
  const unsigned char* base = reinterpret_cast<const unsigned char*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t{15});
  if (base >= lo && base + 32 <= hi) {
    const uint4 a = *reinterpret_cast<const uint4*>(base), b = *reinterpret_cast<const uint4*>(base + 16);
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const int sh = static_cast<int>(p - base), words = sh >> 2;
    const uint32_t bits = (sh & 3) * 8;
    // word i + words of v for a run-time `words`: selects, no local memory
    uint32_t u[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint32_t a0 = v[i], a1 = v[i + 1 < 8 ? i + 1 : 7], a2 = v[i + 2 < 8 ? i + 2 : 7], a3 = v[i + 3 < 8 ? i + 3 : 7];
      u[i] = words == 0 ? a0 : words == 1 ? a1 : words == 2 ? a2 : a3;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(u[i], u[i + 1], bits);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // zero what lies past the row
      const long long keep = left - 4 * i;
      if (keep < 4) w[i] = keep <= 0 ? 0u : w[i] & (0xffffffffu >> (8 * (4 - keep)));
    }
  } else {
    constexpr int PER = 4 / sizeof(E);
#pragma unroll
    for (int i = 0; i < 16 / static_cast<int>(sizeof(E)); ++i)
      if (i * static_cast<int>(sizeof(E)) < left)
        w[i / PER] |= static_cast<uint32_t>(reinterpret_cast<const E*>(p)[i]) << (8 * sizeof(E) * (i % PER));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Copies rows row0 .. row0 + ROWS - 1 of one K block into a swizzled tile (16-byte
// chunk c of row r at chunk c ^ (r % 8)) with 128 threads; rows past row_end are zero.
template <typename E, int ROWS>
__device__ __forceinline__ void copy_tile(unsigned char* tile, const void* src, long long ld, int row0, int row_end,
                                          int block, int K, int tid) {
  const unsigned char* lo = static_cast<const unsigned char*>(src);
  const long long pitch = ld * static_cast<long long>(sizeof(E)), bytes = static_cast<long long>(K) * sizeof(E);
  const unsigned char* hi = lo + (row_end - 1) * pitch + bytes;
  constexpr int STEP = 4;  // chunks in flight per thread
  constexpr int CHUNKS = ROWS * 8;
  static_assert(CHUNKS % 128 == 0, "");
#pragma unroll 1
  for (int i0 = tid; i0 < CHUNKS; i0 += 128 * STEP) {
    uint4 v[STEP];
#pragma unroll
    for (int j = 0; j < STEP; ++j) {
      const int i = i0 + 128 * j, r = i >> 3, c = i & 7;
      v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (i < CHUNKS && row0 + r < row_end)
        v[j] = load_unaligned16<E>(lo + (row0 + r) * pitch, static_cast<long long>(block) * kKBytes + 16 * c, bytes, lo, hi);
    }
#pragma unroll
    for (int j = 0; j < STEP; ++j) {
      const int i = i0 + 128 * j, r = i >> 3, c = i & 7;
      if (i < CHUNKS) *reinterpret_cast<uint4*>(tile + r * kKBytes + (((c ^ r) & 7) << 4)) = v[j];
    }
  }
}

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

  if (warp == 0) {
    tc05::tmem_alloc(&sm.tmem_base, kCols);
    tc05::tmem_relinquish();
  }
  if (tid == kEpiThreads) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sm.full[i], TMA ? 1 : 128);
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
    const int group = (warp - 5) >> 2, t = tid - kEpiThreads - 32 - 128 * group;
    bool ok = true;
    for (int i = group; i < nkb && ok; i += 2) {
      const int s = i % stages;
      if (i >= stages) ok = mbar_wait_bounded(smem_u32(&sm.empty[s]), (i / stages - 1) & 1, kLinearWaitNs);
      if (!ok) break;
      unsigned char* w = ring + s * kStage;
      copy_tile<E, kOut>(w, p.w, p.ldw, n0, p.N, kb0 + i, p.K, t);
      copy_tile<E, TOK>(w + kWBytes, p.x, p.ldx, m0, p.M, kb0 + i, p.K, t);
      fence_proxy_async_smem();
      mbar_arrive_local(&sm.full[s]);
    }
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
  // two CTAs share an SM's 227 KB: ring of about 100 KB
  const int stages = static_cast<int>(100 * 1024 / stage) < kMaxStages ? static_cast<int>(100 * 1024 / stage) : kMaxStages;
  // split K while the CTAs still fit the SMs (two on each) and each keeps four blocks of K
  const long long blocks = (a.K + EPB - 1) / EPB;
  int S = 1;
  while (S < kMaxSplit && 2 * S <= TOK && gx * gy * S * 2 <= 2 * 152 && blocks >= 2 * S * 4) S *= 2;
  CUtensorMap wmap = {}, xmap = {};
  if (TMA && !(encode_rows(&wmap, a.w, sizeof(E), a.K, a.N, a.ldw, kOut) && encode_rows(&xmap, a.x, sizeof(E), a.K, a.M, a.ldx, TOK)))
    return cudaErrorInvalidValue;
  const size_t smem = stages * stage + 1024;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit_once(kda_linear_kernel<E, Y, TOK, TMA>, 104 * 1024, smem_set);
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
    return a.M <= 16 ? launch_tile<E, Y, 16, false>(a, s) : launch_tile<E, Y, 64, false>(a, s);
  if (a.M <= 16) return launch_tile<E, Y, 16, true>(a, s);
  if (a.M <= 32) return launch_tile<E, Y, 32, true>(a, s);
  if (a.M <= 64) return launch_tile<E, Y, 64, true>(a, s);
  if (a.M <= 128) return launch_tile<E, Y, 128, true>(a, s);
  return launch_linear_pair(a, s);
}

}  // namespace

cudaError_t launch_linear(const kda_linear_args& a, cudaStream_t s) {
  if (a.dtype == KDA_DTYPE_BF16)
    return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint16_t, __nv_bfloat16>(a, s) : launch<uint16_t, float>(a, s);
  return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint8_t, __nv_bfloat16>(a, s) : launch<uint8_t, float>(a, s);
}

}  // namespace kda
