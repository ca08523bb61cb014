// The projection for many tokens: pairs of SMs (cta_group::2) on one tile of 256
// outputs x 256 tokens, persistent.
//
// Each CTA of a pair stages 128 rows of w and 128 of x per block of K (32 KB, six
// stages), so an operand byte that reaches shared memory feeds twice the products
// of a tile that one SM works on alone; the leader CTA issues the MMAs for both.
// CTA c's tensor memory holds outputs 128 c .. 128 c + 127 (lanes) of all 256
// tokens (columns), twice: while the epilogue warps read one accumulator the next
// tile's products fill the other.
//
// Roles: warps 0-7 the epilogue (lane quarter w % 4, token half w / 4), warp 8
// issues the MMAs (leader only), warp 9 the TMA loads of its own CTA, counted on
// the leader's barrier.
#include "kda_linear.cuh"

namespace kda {
namespace {

using namespace linear;

constexpr int kTok = 256;        // tokens per tile
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 32 * (kEpiWarps + 2);
constexpr uint32_t kHalfBytes = 128 * kKBytes;    // 128 rows of one operand
constexpr uint32_t kStageBytes = 2 * kHalfBytes;  // per CTA
constexpr uint32_t kCols = 512;                   // two accumulators of 256 columns
constexpr int kBand = 8;                          // token tiles that are worked on together

struct PairHead {
  uint64_t full[kStages];   // leader: both CTAs' copies of a stage have landed
  uint64_t empty[kStages];  // each CTA: the MMAs that read the stage are done
  uint64_t acc_full[2];     // each CTA: an accumulator is complete
  uint64_t acc_empty[2];    // leader: the epilogue warps of both CTAs have read it
  uint32_t tmem_base;
  int failed;
};
constexpr size_t kPairSmem = kStages * kStageBytes + 1024;

// TMA load into this CTA's shared memory, counted on a barrier of the pair's
// leader (an address of the cluster's shared memory).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t smem, const CUtensorMap* map, int x, int y, uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem),
      "l"(map), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}

template <int EBYTES>
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  if (EBYTES == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
}

// Arrives on the barrier at the same offset in both CTAs when every MMA that this
// thread issued before has completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Tile t of the grid: bands of kBand token tiles, output tiles within a band, so
// that the tiles in work at one time share few rows of w and of x.
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int& m, int& n) {
  const int band = t / (kBand * nt), first = band * kBand, width = min(kBand, mt - first), r = t - band * kBand * nt;
  n = r / width;
  m = first + r % width;
}

template <typename E, typename Y>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    kda_linear_pair_kernel(const kda_linear_args p, const __grid_constant__ CUtensorMap wmap,
                           const __grid_constant__ CUtensorMap xmap, int mt, int nt) {
  extern __shared__ unsigned char raw[];
  __shared__ PairHead sm;
  constexpr int EPB = kKBytes / sizeof(E);
  unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = mt * nt;
  const int blocks = (p.K + EPB - 1) / EPB;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 32 * kEpiWarps) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.acc_empty[i], 2 * kEpiWarps);
    }
    sm.failed = 0;
    fence_mbarrier_init_cluster();
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  cluster_sync_all();
  tc05::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;

  if (warp == kEpiWarps + 1) {
    if (lane == 0) {
      bool ok = true;
      int i = 0;  // blocks loaded so far
      for (int t = pair; t < tiles && ok; t += pairs) {
        int m, n;
        tile_of(t, mt, nt, m, n);
        const int n0 = n * 2 * kOut + rank * kOut, m0 = m * kTok + rank * (kTok / 2);
        for (int b = 0; b < blocks; ++b, ++i) {
          const int s = i % kStages;
          if (i >= kStages) ok = mbar_wait_bounded(smem_u32(&sm.empty[s]), (i / kStages - 1) & 1, kLinearWaitNs);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx_local(&sm.full[s], 2 * kStageBytes);
          const uint32_t w = smem_u32(ring + s * kStageBytes), bar = mapa_shared(smem_u32(&sm.full[s]), 0);
          tma_load_2d_pair(w, &wmap, b * EPB, n0, bar);
          tma_load_2d_pair(w + kHalfBytes, &xmap, b * EPB, m0, bar);
        }
      }
      // every stage's last use has been consumed: no copy and no arrival is left
      // in flight when the CTA ends
      for (int j = i > kStages ? i - kStages : 0; j < i; ++j)
        ok &= mbar_wait_bounded(smem_u32(&sm.empty[j % kStages]), (j / kStages) & 1, kLinearWaitNs);
      if (!ok) sm.failed = 1;
    }
  } else if (warp == kEpiWarps) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = tc05::idesc_f16kind(256, kTok, sizeof(E) == 2);
      bool ok = true;
      int i = 0, k = 0;  // blocks, tiles so far
      for (int t = pair; t < tiles && ok; t += pairs, ++k) {
        const int buf = k & 1;
        if (k >= 2) ok = mbar_wait_bounded(smem_u32(&sm.acc_empty[buf]), (k / 2 - 1) & 1, kLinearWaitNs);
        tc05::fence_after_sync();
        for (int b = 0; b < blocks && ok; ++b, ++i) {
          const int s = i % kStages;
          ok = mbar_wait_bounded(smem_u32(&sm.full[s]), (i / kStages) & 1, kLinearWaitNs);
          if (!ok) break;
          tc05::fence_after_sync();
          const uint32_t w = smem_u32(ring + s * kStageBytes), x = w + kHalfBytes;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_pair<sizeof(E)>(tmem + buf * kTok, tc05::smem_desc(w + 32 * j, 16, 1024, tc05::kSwizzle128B),
                                tc05::smem_desc(x + 32 * j, 16, 1024, tc05::kSwizzle128B), idesc, b > 0 || j > 0);
          commit_pair(&sm.empty[s]);
        }
        if (ok) commit_pair(&sm.acc_full[buf]);
      }
      if (!ok) sm.failed = 1;
    }
  } else {
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + half * (kTok / 2);
    bool ok = true;
    int k = 0;
    for (int t = pair; t < tiles; t += pairs, ++k) {
      int m, n;
      tile_of(t, mt, nt, m, n);
      const int buf = k & 1;
      ok = mbar_wait_bounded(smem_u32(&sm.acc_full[buf]), (k / 2) & 1, kLinearWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc05::fence_after_sync();
      const Epilogue<Y> finish(p, n * 2 * kOut + rank * kOut + 32 * quarter + lane);
      const long long m0 = static_cast<long long>(m) * kTok + half * (kTok / 2);
#pragma unroll 1
      for (int c0 = 0; c0 < kTok / 2; c0 += 32) {
        float v[32];
        tmem_load(lane_base + buf * kTok + c0, v);
        if (c0 == kTok / 2 - 32) {  // the accumulator has been read: the next but one tile may start
          tc05::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sm.acc_empty[buf]), 0));
        }
        finish(v, m0 + c0);
      }
    }
    if (!ok) sm.failed = 1;
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  if (tid == 0 && sm.failed) set_err(p.err, KDA_ERR_TIMEOUT);
  cluster_sync_all();  // neither CTA ends while the other may still signal it
  tc05::fence_after_sync();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
}

template <typename E, typename Y>
cudaError_t launch(const kda_linear_args& a, cudaStream_t s) {
  const long long mt = (static_cast<long long>(a.M) + kTok - 1) / kTok, nt = (static_cast<long long>(a.N) + 2 * kOut - 1) / (2 * kOut);
  if (mt * nt > INT32_MAX / 2) return cudaErrorNotSupported;
  CUtensorMap wmap, xmap;
  if (!encode_rows(&wmap, a.w, sizeof(E), a.K, a.N, a.ldw, kOut) || !encode_rows(&xmap, a.x, sizeof(E), a.K, a.M, a.ldx, kTok / 2))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit_once(kda_linear_pair_kernel<E, Y>, kPairSmem, smem_set);
  if (e != cudaSuccess) return e;
  const long long pairs = mt * nt < 152 / 2 ? mt * nt : 152 / 2;
  kda_linear_pair_kernel<E, Y><<<static_cast<unsigned>(2 * pairs), kPairThreads, kPairSmem, s>>>(
      a, wmap, xmap, static_cast<int>(mt), static_cast<int>(nt));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_pair(const kda_linear_args& a, cudaStream_t s) {
  if (a.dtype == KDA_DTYPE_BF16)
    return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint16_t, __nv_bfloat16>(a, s) : launch<uint16_t, float>(a, s);
  return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint8_t, __nv_bfloat16>(a, s) : launch<uint8_t, float>(a, s);
}

}  // namespace kda
