// The projection for many tokens, persistent: a pair of SMs (cta_group::2) works on
// one tile of 256 tokens x NT outputs, or, up to 128 tokens, each SM on a tile of
// 128 tokens.
//
// Here tokens are the M side of the tensor core's product (tensor-memory lanes) and
// outputs the N side, whose width NT is any multiple of 16 up to 256: the launcher
// takes the one that spreads the outputs most evenly over the SMs (12288 outputs of
// 256 tokens: 70 tiles of 176 on the 76 pairs instead of 48 of 256).
//
// Each CTA stages 128 rows of x and NT / CTAS rows of w per 128-byte block of K, as
// many stages as 200 KB hold (6 at NT = 256, up to 12: a load takes 3000 cycles under
// way, and narrow tiles use a stage up in a fraction of the 512 of a wide one); in a
// pair an operand byte that reaches shared memory feeds twice the products of a tile
// that one SM works on alone, and the leader CTA issues the MMAs for both. CTA c's tensor memory holds tokens 128 c .. 128 c + 127 (lanes) of all NT
// outputs (columns), twice: while the epilogue warps read one accumulator the next
// tile's products fill the other.
//
// 8192 x 4096 -> 12288 bf16 runs at 1.95 PFLOP/s (424 us, tensor pipe 95 % busy), 8192 x
// 4096 -> 4096 e4m3 with bias, silu and residual at 3.1 (88 us), 256 x 4096 -> 12288 in
// 25 us, in which loads bring each SM 1.77 MB, 36 bytes a cycle from launch to end.
//
// Roles: warps 0-11 the epilogue (lane quarter w % 4, every third block of 32 columns;
// with eight warps gelu on 4691 x 312 -> 8608 took 57 us instead of 54), warp 12 issues
// the MMAs (leader only), warps 13 and 14 the TMA loads of x and of w for their own
// CTA, counted on the leader's barrier.
#include "kda_linear.cuh"

namespace kda {
namespace {

using namespace linear;

constexpr int kRows = 128;       // tokens of a CTA
constexpr int kMaxN = 256;       // outputs of a tile, at most
constexpr int kMaxStages = 12;
constexpr size_t kRingBytes = 6 * 32768;
constexpr int kEpiWarps = 12;
constexpr int kParts = kEpiWarps / 4;  // warps that share a lane quarter
constexpr int kWideThreads = 32 * (kEpiWarps + 3);
constexpr uint32_t kXBytes = kRows * kKBytes;
constexpr uint32_t kCols = 512;  // two accumulators of 256 columns
constexpr int kBand = 8;         // token tiles that are worked on together
constexpr int kStageCols = 33;   // floats of a staged row (an odd pitch: no bank conflicts)

struct WideHead {
  uint64_t full[kMaxStages];   // leader: all copies of a stage have landed
  uint64_t empty[kMaxStages];  // each CTA: the MMAs that read the stage are done
  uint64_t acc_full[2];     // each CTA: an accumulator is complete
  uint64_t acc_empty[2];    // leader: the epilogue warps of all CTAs have read it
  uint32_t tmem_base;
  int failed;
  alignas(16) float col[2][2][kMaxN];  // by accumulator: weight scales and biases of its outputs
};

template <int CTAS>
__device__ __forceinline__ void tma_load(uint32_t smem, const CUtensorMap* map, int x, int y, uint32_t leader_bar) {
  if (CTAS == 1) {
    tma_load_2d(smem, map, x, y, leader_bar);
  } else {  // into this CTA's shared memory, counted on a barrier of the leader
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem),
        "l"(map), "r"(x), "r"(y), "r"(leader_bar)
        : "memory");
  }
}

template <int CTAS, int EBYTES>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  if (CTAS == 1) {
    if (EBYTES == 2) tc05::mma_ss(d_tmem, a_desc, b_desc, idesc, acc);
    else mma_ss_f8(d_tmem, a_desc, b_desc, idesc, acc);
  } else if (EBYTES == 2) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
  }
}

// Arrives on the barrier at the same offset in every CTA of the tile when every MMA
// that this thread issued before has completed.
template <int CTAS>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (CTAS == 1) {
    tc05::commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  }
}

// Tile t of the grid: bands of kBand token tiles, output tiles within a band, so
// that the tiles in work at one time share few rows of w and of x.
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int& m, int& n) {
  const int band = t / (kBand * nt), first = band * kBand, width = min(kBand, mt - first), r = t - band * kBand * nt;
  n = r / width;
  m = first + r % width;
}

// 32 bytes at once (sm_100 and later).
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// 16 consecutive values of a row, 32 bytes an access.
__device__ __forceinline__ void store16(__nv_bfloat16* y, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = Bf16::pack(v[2 * i], v[2 * i + 1]);
  store32(y, w);
}
__device__ __forceinline__ void store16(float* y, const float* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
    store32(y + 8 * h, w);
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* v) {
  uint32_t w[8];
  load32(p, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load16(const float* p, float* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
    load32(p + 8 * h, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * h + i] = __uint_as_float(w[i]);
  }
}

// 8 consecutive values of a row, 16 bytes an access.
__device__ __forceinline__ void store8(__nv_bfloat16* y, const float* v) {
  *reinterpret_cast<uint4*>(y) =
      make_uint4(Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3]), Bf16::pack(v[4], v[5]), Bf16::pack(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* y, const float* v) {
  reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// How rows of y and of the residual can be accessed: 32 or 16 bytes at a time by one
// thread, or (any alignment) through shared memory. A lane's rows are a pitch apart,
// so each access of a warp is 32 separate pieces whatever its width: 32 bytes instead
// of 16 took 5536 x 800 -> 5216 e4m3 from 37 to 29 us.
// (An instance of the kernel each: with all three in one, its instructions no longer
// fit the caches near the SM's schedulers, and every path took a third longer.)
enum { kRows32 = 2, kRows16 = 1, kRowsAny = 0 };

// Finishes 32 consecutive outputs n .. of one token: those below `end` (a multiple
// of the access's values).
template <typename Y, int ACCESS, bool SCALED>
__device__ __forceinline__ void finish_row(const kda_linear_args& p, float (&v)[32], const float* ws, const float* bias, float xs,
                                           long long m, int n, int end) {
  if (m >= p.M) return;
  float res[32];
  if (p.residual) {
    const Y* r = static_cast<const Y*>(p.residual) + m * p.ld_residual + n;
#pragma unroll
    for (int b = 0; b < 32; b += 8 * ACCESS) {
      if (n + b < end) {
        if (ACCESS == kRows32) load16(r + b, res + b);
        else load8(r + b, res + b);
      }
    }
  }
  if (SCALED) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 s = *reinterpret_cast<const float4*>(ws + j);
      v[j] *= xs * s.x, v[j + 1] *= xs * s.y, v[j + 2] *= xs * s.z, v[j + 3] *= xs * s.w;
    }
  }
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 b = *reinterpret_cast<const float4*>(bias + j);
      v[j] += b.x, v[j + 1] += b.y, v[j + 2] += b.z, v[j + 3] += b.w;
    }
  }
  switch (p.activation) {
    case KDA_ACT_SILU: activate_all<KDA_ACT_SILU>(v); break;
    case KDA_ACT_GELU: activate_all<KDA_ACT_GELU>(v); break;
    case KDA_ACT_SIGMOID: activate_all<KDA_ACT_SIGMOID>(v); break;
    case KDA_ACT_RELU: activate_all<KDA_ACT_RELU>(v); break;
    default: break;
  }
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += res[j];
  }
  Y* y = static_cast<Y*>(p.y) + m * p.ldy + n;
#pragma unroll
  for (int b = 0; b < 32; b += 8 * ACCESS) {
    if (n + b < end) {
      if (ACCESS == kRows32) store16(y + b, v + b);
      else store8(y + b, v + b);
    }
  }
}

template <typename E, typename Y, int CTAS, int ACCESS>
__global__ void __launch_bounds__(kWideThreads, 1)
    kda_linear_wide_kernel(const kda_linear_args p, const __grid_constant__ CUtensorMap wmap,
                           const __grid_constant__ CUtensorMap xmap, int mt, int nt, int NT, int stages) {
  extern __shared__ unsigned char raw[];
  __shared__ WideHead sm;
  constexpr int EPB = kKBytes / sizeof(E);
  unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  const uint32_t w_bytes = static_cast<uint32_t>(NT / CTAS) * kKBytes;
  const uint32_t stage = kXBytes + ((w_bytes + 1023) & ~1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CTAS == 1 ? 0 : static_cast<int>(cluster_ctarank());
  const int unit = blockIdx.x / CTAS, units = gridDim.x / CTAS, tiles = mt * nt;
  const int blocks = (p.K - 1) / EPB + 1;  // (K + EPB may pass 2^31)

  if (warp == kEpiWarps + 1 && lane == 0) {
    prefetch_map(&xmap);
    prefetch_map(&wmap);
  }
  if (warp == 0) {
    if (CTAS == 1) {
      tc05::tmem_alloc(&sm.tmem_base, kCols);
      tc05::tmem_relinquish();
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                   "r"(kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  if (tid == 32 * kEpiWarps) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.acc_empty[i], CTAS * kEpiWarps);
    }
    sm.failed = 0;
    fence_mbarrier_init_cluster();
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  if (CTAS > 1) cluster_sync_all();
  tc05::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;

  if (warp > kEpiWarps) {
    // One warp loads x, one w: a single thread's pace (wait, count, two copies) is 600
    // cycles a block, more than a narrow tile's products take.
    const bool of_x = warp == kEpiWarps + 1;
    if (lane == 0) {
      wait_for_copy();
      bool ok = true;
      int loaded = 0, s = 0;  // blocks so far, stage
      uint32_t phase = 1;     // of the stage's previous use
      const CUtensorMap* map = of_x ? &xmap : &wmap;
      const uint32_t base = smem_u32(ring) + (of_x ? 0 : kXBytes);
      const uint32_t bars = CTAS == 1 ? smem_u32(sm.full) : mapa_shared(smem_u32(sm.full), 0);
      for (int t = unit; t < tiles && ok; t += units) {
        int m, n;
        tile_of(t, mt, nt, m, n);
        const int row = of_x ? (m * CTAS + rank) * kRows : n * NT + rank * (NT / CTAS);
        for (int b = 0; b < blocks; ++b) {
          if (loaded >= stages) ok = mbar_wait_bounded(smem_u32(&sm.empty[s]), phase, kLinearWaitNs);
          if (!ok) break;
          if (of_x && rank == 0) mbar_arrive_expect_tx_local(&sm.full[s], CTAS * (kXBytes + w_bytes));
          tma_load<CTAS>(base + s * stage, map, b * EPB, row, bars + 8 * s);
          ++loaded;
          if (++s == stages) s = 0, phase ^= 1;
        }
      }
      // every stage's last use has been consumed: no copy and no arrival is left
      // in flight when the CTA ends (each wait is bounded)
      for (int j = loaded > stages ? loaded - stages : 0; j < loaded; ++j)
        ok &= mbar_wait_bounded(smem_u32(&sm.empty[j % stages]), (j / stages) & 1, kLinearWaitNs);
      if (!ok) sm.failed = 1;
    }
  } else if (warp == kEpiWarps) {
    if (rank == 0 && lane == 0) {
      const uint32_t idesc = tc05::idesc_f16kind(CTAS * kRows, NT, sizeof(E) == 2);
      bool ok = true;
      int k = 0, s = 0;  // tiles so far, stage
      uint32_t phase = 0;
      for (int t = unit; t < tiles && ok; t += units, ++k) {
        const int buf = k & 1;
        if (k >= 2) ok = mbar_wait_bounded(smem_u32(&sm.acc_empty[buf]), (k / 2 - 1) & 1, kLinearWaitNs);
        tc05::fence_after_sync();
        for (int b = 0; b < blocks && ok; ++b) {
          ok = mbar_wait_bounded(smem_u32(&sm.full[s]), phase, kLinearWaitNs);
          if (!ok) break;
          tc05::fence_after_sync();
          const uint32_t x = smem_u32(ring) + s * stage;
          const uint64_t xd = tc05::smem_desc(x, 16, 1024, tc05::kSwizzle128B);
          const uint64_t wd = tc05::smem_desc(x + kXBytes, 16, 1024, tc05::kSwizzle128B);
#pragma unroll
          for (int j = 0; j < 4; ++j)  // 32 bytes of K each: 2 in the descriptor's units of 16
            mma<CTAS, sizeof(E)>(tmem + buf * kMaxN, xd + 2 * j, wd + 2 * j, idesc, b > 0 || j > 0);
          commit<CTAS>(&sm.empty[s]);
          if (++s == stages) s = 0, phase ^= 1;
        }
        if (ok) commit<CTAS>(&sm.acc_full[buf]);
      }
      if (!ok) sm.failed = 1;
    }
  } else {
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    float* staged = reinterpret_cast<float*>(ring + stages * stage) + warp * 16 * kStageCols;
    const int chunks = (NT + 31) / 32;  // blocks of 32 columns (the last may be half)
    bool ok = true;
    int k = 0;
    for (int t = unit; t < tiles; t += units, ++k) {
      int mi, ni;
      tile_of(t, mt, nt, mi, ni);
      const int buf = k & 1, n0 = ni * NT, end = min(n0 + NT, p.N);
      const long long m0 = (static_cast<long long>(mi) * CTAS + rank) * kRows + 32 * quarter;
      float* ws = sm.col[buf][0];
      float* bias = sm.col[buf][1];
      if (ACCESS != kRowsAny) {
        // (the tile before the last that used these has been finished by every warp:
        // each passed the named barrier of the tile in between afterwards)
        const int n = n0 + tid;
        if (tid < kMaxN) {
          ws[tid] = p.w_scale && n < end ? p.w_scale[n] : 1.f;
          bias[tid] = p.bias && n < end ? p.bias[n] : 0.f;
        }
        named_bar_sync(1, 32 * kEpiWarps);
      }
      const float xs = p.x_scale && m0 + lane < p.M ? p.x_scale[m0 + lane] : 1.f;
      // the residual into L2 while the products run: from HBM each of a warp's blocks
      // would wait 1.2 us for it after they are done
      if (p.residual && m0 + lane < p.M) {
        for (int c = part; c < chunks; c += kParts) {
          const Y* r = static_cast<const Y*>(p.residual) + (m0 + lane) * p.ld_residual + n0 + 32 * c;
          if (n0 + 32 * c < end) asm volatile("prefetch.global.L2 [%0];" ::"l"(r));
        }
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&sm.acc_full[buf]), (k / 2) & 1, tile_wait_ns(blocks)));
      tc05::fence_after_sync();
      for (int c = part; c < chunks; c += kParts) {
        float v[32];
        tc05::ld32_wait(lane_base + buf * kMaxN + 32 * c, v);
        if (c + kParts >= chunks) {  // this warp has read its share: the next but one tile may start
          tc05::fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if (CTAS == 1) mbar_arrive_local(&sm.acc_empty[buf]);
            else mbar_arrive_cluster(mapa_shared(smem_u32(&sm.acc_empty[buf]), 0));
          }
        }
        if (!ok) continue;
        if constexpr (ACCESS != kRowsAny) {
          finish_row<Y, ACCESS, sizeof(E) == 1>(p, v, ws + 32 * c, bias + 32 * c, xs, m0 + lane, n0 + 32 * c, end);
        } else {
          // rows of any alignment: 16 tokens x 32 outputs at a time through shared
          // memory, so that a warp's accesses are 32 consecutive outputs of a token
          const int n = n0 + 32 * c + lane;
          const Epilogue<Y> finish(p, n < end ? n : p.N);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __syncwarp();
            if (lane / 16 == h) {
#pragma unroll
              for (int j = 0; j < 32; ++j) staged[(lane % 16) * kStageCols + j] = sizeof(E) == 1 ? v[j] * xs : v[j];
            }
            __syncwarp();
            float u[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) u[j] = staged[j * kStageCols + lane];
            finish.template operator()<sizeof(E) == 1>(u, m0 + 16 * h);
          }
        }
      }
      if (part >= chunks && lane == 0) {  // a tile of one block of columns: no share to read
        if (CTAS == 1) mbar_arrive_local(&sm.acc_empty[buf]);
        else mbar_arrive_cluster(mapa_shared(smem_u32(&sm.acc_empty[buf]), 0));
      }
    }
    if (!ok) sm.failed = 1;
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  if (tid == 0 && sm.failed) set_err(p.err, KDA_ERR_TIMEOUT);
  if (CTAS > 1) cluster_sync_all();  // neither CTA ends while the other may still signal it
  tc05::fence_after_sync();
  if (warp == 0) {
    if (CTAS == 1) tc05::tmem_dealloc(tmem, kCols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

// Whether rows of N values at p can be accessed `bytes` at a time.
bool rows_allow(const void* p, int64_t ld, int N, size_t elem, int64_t bytes) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * static_cast<int64_t>(elem) % bytes == 0 &&
                          N % (bytes / 2) == 0);  // (16 or 8 values at a time, of either type)
}

template <typename E, typename Y, int CTAS, int ACCESS>
cudaError_t launch(const kda_linear_args& a, bool after_copy, cudaStream_t s) {
  constexpr int kUnits = 152 / CTAS;
  const long long mt = (static_cast<long long>(a.M) + CTAS * kRows - 1) / (CTAS * kRows);
  // (One CTA on a tile stages all of its outputs' rows: at most 128 of them.)
  // The width whose rounds over the SMs cost least: rounds * (NT + 24), 24 columns
  // standing for what a tile costs besides its products (first loads, last stores).
  int NT = 0;
  long long best = 0;
  for (int w = CTAS == 1 ? kMaxN / 2 : kMaxN; w >= 32; w -= 16) {
    const long long tiles = mt * ((a.N - 1) / w + 1), cost = (tiles + kUnits - 1) / kUnits * (w + 24);
    if (NT == 0 || cost < best) {
      NT = w;
      best = cost;
    }
  }
  const long long nt = (a.N - 1) / NT + 1;
  if (mt * nt > INT32_MAX / 2) return cudaErrorNotSupported;
  CUtensorMap wmap, xmap;
  if (!encode_rows(&wmap, a.w, sizeof(E), a.K, a.N, a.ldw, NT / CTAS) || !encode_rows(&xmap, a.x, sizeof(E), a.K, a.M, a.ldx, kRows))
    return cudaErrorInvalidValue;
  const size_t stage = kXBytes + ((static_cast<size_t>(NT / CTAS) * kKBytes + 1023) & ~size_t{1023});
  constexpr size_t kStaged = kEpiWarps * 16 * kStageCols * sizeof(float);
  constexpr size_t kMost = kRingBytes + kStaged + 1024;
  const int stages = static_cast<int>(kRingBytes / stage) < kMaxStages ? static_cast<int>(kRingBytes / stage) : kMaxStages;
  const size_t smem = stages * stage + (ACCESS == kRowsAny ? kStaged : 0) + 1024;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit_once(kda_linear_wide_kernel<E, Y, CTAS, ACCESS>, kMost, smem_set);
  if (e != cudaSuccess) return e;
  const long long units = mt * nt < kUnits ? mt * nt : kUnits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(CTAS * units));
  cfg.blockDim = dim3(kWideThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  set_attributes(cfg, attrs, CTAS, after_copy);
  return cudaLaunchKernelEx(&cfg, kda_linear_wide_kernel<E, Y, CTAS, ACCESS>, a, wmap, xmap, static_cast<int>(mt), static_cast<int>(nt),
                            NT, stages);
}

template <typename E, typename Y, int CTAS>
cudaError_t launch_access(const kda_linear_args& a, bool after_copy, cudaStream_t s) {
  auto allow = [&](int64_t bytes) {
    return rows_allow(a.y, a.ldy, a.N, sizeof(Y), bytes) && rows_allow(a.residual, a.ld_residual, a.N, sizeof(Y), bytes);
  };
  if (allow(32)) return launch<E, Y, CTAS, kRows32>(a, after_copy, s);
  return allow(16) ? launch<E, Y, CTAS, kRows16>(a, after_copy, s) : launch<E, Y, CTAS, kRowsAny>(a, after_copy, s);
}

template <typename E, typename Y>
cudaError_t launch_ctas(const kda_linear_args& a, bool after_copy, cudaStream_t s) {
  return a.M <= kRows ? launch_access<E, Y, 1>(a, after_copy, s) : launch_access<E, Y, 2>(a, after_copy, s);
}

}  // namespace

cudaError_t launch_linear_wide(const kda_linear_args& a, bool after_copy, cudaStream_t s) {
  if (a.dtype == KDA_DTYPE_BF16)
    return a.y_dtype == KDA_DTYPE_BF16 ? launch_ctas<uint16_t, __nv_bfloat16>(a, after_copy, s) : launch_ctas<uint16_t, float>(a, after_copy, s);
  return a.y_dtype == KDA_DTYPE_BF16 ? launch_ctas<uint8_t, __nv_bfloat16>(a, after_copy, s) : launch_ctas<uint8_t, float>(a, after_copy, s);
}

}  // namespace kda
