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
// through a ring of stages.
//
// Rows that TMA cannot describe (an address or a row pitch that is no multiple of 16
// bytes) are first copied to a pitch that is one, in the caller's workspace: a pass
// over the operand costs less than loads that shift every row on its way into every
// tile (777 x 1001 -> 1111: 27 us in the best such form).
//
// Few tiles (few tokens, or few outputs and a long K) leave most SMs without work, so a cluster of S CTAs splits
// K of one tile: each sums its share, puts it into its own shared memory, and
// finishes 1/S of the tokens from all S (distributed shared memory), in the
// order of the ranks, so results do not vary from run to run. 16 x 4096 -> 4096 e4m3
// takes 7.8 us (its weights alone 2.5 at the copy rate: what is left is the chain of
// launch, first load, products and exchange), 16 x 4096 -> 12288 bf16 22 us, 4.6 TB/s.
#include "kda_linear.cuh"

namespace kda {
namespace {

using namespace linear;

constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;
constexpr int kEpiThreads = 128;
constexpr int kThreads = kEpiThreads + 64;  // + MMA warp, TMA warp

struct LinearHead {
  uint64_t full[kMaxStages], empty[kMaxStages], acc;
  uint32_t tmem_base;
  int failed;
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
template <typename E, typename Y, int TOK>
__global__ void __launch_bounds__(kThreads)
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
  const int blocks = (p.K - 1) / EPB + 1;  // (K + EPB may pass 2^31)
  const int kb0 = static_cast<int>(static_cast<long long>(blocks) * rank / S);
  const int nkb = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / S) - kb0;

  if (warp == 5 && lane == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
  }
  if (warp == 0) {
    tc05::tmem_alloc(&sm.tmem_base, kCols);
    tc05::tmem_relinquish();
  }
  if (tid == kEpiThreads) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sm.full[i], 1);
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
  } else if (warp == 5) {
    if (lane == 0) {
      wait_for_copy();
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
  }
  __syncwarp();

  bool ok = true;
  if (warp < 4) ok = mbar_wait_bounded(smem_u32(&sm.acc), 0, tile_wait_ns(nkb));
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

// CTAs that share a tile's K: as many as still fit the SMs (two on each), with four
// blocks of K or more for each.
int split_of(long long tiles, long long blocks, int tokens) {
  int S = 1;
  while (S < kMaxSplit && 2 * S <= tokens && tiles * S * 2 <= 2 * 152 && blocks >= 2 * S * 4) S *= 2;
  return S;
}

template <typename E, typename Y, int TOK>
cudaError_t launch_tile(const kda_linear_args& a, bool after_copy, cudaStream_t s) {
  constexpr size_t stage = (kOut + TOK) * kKBytes;
  constexpr int EPB = kKBytes / sizeof(E);
  const long long gx = (static_cast<long long>(a.N) + kOut - 1) / kOut, gy = (static_cast<long long>(a.M) + TOK - 1) / TOK;
  if (gy > 65535 || gx * kMaxSplit > INT32_MAX) return cudaErrorNotSupported;
  // two CTAs share an SM's 227 KB: a ring of about 100 KB
  constexpr int kFit = static_cast<int>(100 * 1024 / stage);
  constexpr int stages = kFit < kMaxStages ? kFit : kMaxStages;
  static_assert(stages * stage >= TOK * kOut * sizeof(float), "the ring holds a CTA's sums");
  const int S = split_of(gx * gy, (a.K - 1) / EPB + 1, TOK);
  CUtensorMap wmap, xmap;
  if (!encode_rows(&wmap, a.w, sizeof(E), a.K, a.N, a.ldw, kOut) || !encode_rows(&xmap, a.x, sizeof(E), a.K, a.M, a.ldx, TOK))
    return cudaErrorInvalidValue;
  constexpr size_t smem = stages * stage + 1024;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit_once(kda_linear_kernel<E, Y, TOK>, smem, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gx * S), static_cast<unsigned>(gy));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  set_attributes(cfg, attrs, S, after_copy);
  return cudaLaunchKernelEx(&cfg, kda_linear_kernel<E, Y, TOK>, a, wmap, xmap, S, stages);
}

template <typename E, typename Y>
cudaError_t launch(const kda_linear_args& a, bool after_copy, cudaStream_t s) {
  if (a.M <= 16) return launch_tile<E, Y, 16>(a, after_copy, s);
  if (a.M <= 32) return launch_tile<E, Y, 32>(a, after_copy, s);
  if (a.M <= 64) return launch_tile<E, Y, 64>(a, after_copy, s);
  // More tokens: whole K on tiles that share it between few SMs' loads, or, where a
  // long K meets few tiles, K split over clusters. In units of one block of K on the
  // wide kernel (0.23 us): a round there costs its blocks and 17, here a CTA's share
  // of the blocks, 1.5 each and slowed by its neighbours, and 40 for the cluster's
  // sums. 128 x 4096 -> 4096 bf16: 18.6 us wide, 14.6 split; 256 x 4096 -> 512: 19.5
  // and 10.7; e4m3 (half the blocks) 128 x 4096 -> 4096: 11.8 and 13.5.
  const long long blocks = (static_cast<long long>(a.K) * sizeof(E) + kKBytes - 1) / kKBytes;
  const long long tiles = (static_cast<long long>(a.N) + kOut - 1) / kOut * ((static_cast<long long>(a.M) + 127) / 128);
  const int S = split_of(tiles, blocks, 128);
  const double crowd = static_cast<double>(tiles * S) / 152;
  if (S > 1 && 40 + 1.5 * (crowd > 1 ? crowd : 1) * blocks / S < 17 + blocks) return launch_tile<E, Y, 128>(a, after_copy, s);
  return launch_linear_wide(a, after_copy, s);
}

// ---- rows to a pitch that TMA describes ----

struct Repitch {
  const unsigned char* src;
  unsigned char* dst;
  long long src_pitch, dst_pitch, row_bytes;
  int rows;
};

// A warp a row, 16 bytes a lane and step, from the aligned 4-byte words around them;
// where those words may lie outside the row (its first and last bytes), element by
// element. Bytes of the new pitch past the row are not written: no map reaches them.
template <typename E>
__global__ void __launch_bounds__(256) kda_linear_repitch_kernel(const Repitch x, const Repitch w) {
  asm volatile("griddepcontrol.launch_dependents;");  // the product's CTAs set themselves up meanwhile
  const int lane = threadIdx.x & 31;
  const long long total = static_cast<long long>(x.rows) + w.rows;
  for (long long r = (blockIdx.x * 256LL + threadIdx.x) >> 5; r < total; r += gridDim.x * 8LL) {
    const bool of_x = r < x.rows;
    const Repitch& m = of_x ? x : w;
    const long long row = of_x ? r : r - x.rows;
    const unsigned char* src = m.src + row * m.src_pitch;
    unsigned char* dst = m.dst + row * m.dst_pitch;
    for (long long b = 16 * lane; b < m.row_bytes; b += 512) {
      const unsigned char* p = src + b;
      if (b >= 4 && b + 20 <= m.row_bytes) {
        const uint32_t shift = reinterpret_cast<uintptr_t>(p) & 3;
        const uint32_t* at = reinterpret_cast<const uint32_t*>(p - shift);
        uint32_t v[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) v[i] = at[i];
        uint4 out;
        out.x = __funnelshift_r(v[0], v[1], 8 * shift);
        out.y = __funnelshift_r(v[1], v[2], 8 * shift);
        out.z = __funnelshift_r(v[2], v[3], 8 * shift);
        out.w = __funnelshift_r(v[3], v[4], 8 * shift);
        *reinterpret_cast<uint4*>(dst + b) = out;
      } else {
        for (int i = 0; i < 16 && b + i < m.row_bytes; i += sizeof(E))
          *reinterpret_cast<E*>(dst + b + i) = *reinterpret_cast<const E*>(p + i);
      }
    }
  }
}

// Whether TMA can describe the rows: address and pitch on 16-byte boundaries
// (one row has no pitch).
bool tma_ok(const void* p, long long rows, long long ld, size_t elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows == 1 || ld * static_cast<long long>(elem) % 16 == 0);
}

size_t elem_of(const kda_linear_args& a) { return a.dtype == KDA_DTYPE_BF16 ? 2 : 1; }
size_t pitch_of(const kda_linear_args& a) { return (a.K * elem_of(a) + 15) / 16 * 16; }
size_t copy_bytes(const kda_linear_args& a, const void* p, long long rows, long long ld) {
  return tma_ok(p, rows, ld, elem_of(a)) ? 0 : (rows * pitch_of(a) + 255) / 256 * 256;
}

// Operands that need it into the workspace; `a` then refers to the copies.
cudaError_t repitch(kda_linear_args& a, void* workspace, cudaStream_t s) {
  const size_t e = elem_of(a), pitch = pitch_of(a), xb = copy_bytes(a, a.x, a.M, a.ldx), wb = copy_bytes(a, a.w, a.N, a.ldw);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const long long bytes = static_cast<long long>(a.K) * e, dst_pitch = static_cast<long long>(pitch);
  const Repitch x = {static_cast<const unsigned char*>(a.x), ws, a.ldx * static_cast<long long>(e), dst_pitch, bytes, xb ? a.M : 0};
  const Repitch w = {static_cast<const unsigned char*>(a.w), ws + xb, a.ldw * static_cast<long long>(e), dst_pitch, bytes, wb ? a.N : 0};
  const long long rows = static_cast<long long>(x.rows) + w.rows, grid = (rows + 7) / 8;
  const unsigned ctas = static_cast<unsigned>(grid < 8 * 152 ? grid : 8 * 152);
  if (e == 2) kda_linear_repitch_kernel<uint16_t><<<ctas, 256, 0, s>>>(x, w);
  else kda_linear_repitch_kernel<uint8_t><<<ctas, 256, 0, s>>>(x, w);
  if (xb) {
    a.x = x.dst;
    a.ldx = static_cast<int64_t>(pitch / e);
  }
  if (wb) {
    a.w = w.dst;
    a.ldw = static_cast<int64_t>(pitch / e);
  }
  return cudaGetLastError();
}

}  // namespace

size_t linear_workspace_bytes(const kda_linear_args& a) { return copy_bytes(a, a.x, a.M, a.ldx) + copy_bytes(a, a.w, a.N, a.ldw); }

cudaError_t launch_linear(kda_linear_args a, void* workspace, cudaStream_t s) {
  const bool copied = linear_workspace_bytes(a) != 0;
  const cudaError_t e = copied ? repitch(a, workspace, s) : cudaSuccess;
  if (e != cudaSuccess) return e;
  if (a.dtype == KDA_DTYPE_BF16)
    return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint16_t, __nv_bfloat16>(a, copied, s) : launch<uint16_t, float>(a, copied, s);
  return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint8_t, __nv_bfloat16>(a, copied, s) : launch<uint8_t, float>(a, copied, s);
}

}  // namespace kda
