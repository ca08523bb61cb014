// Softmax attention over whole prompts on the 5th-generation tensor cores, and the
// shared prefix of the single-token step.
//
// A CTA takes 256 rows of queries, as two tiles of 128 that share every block of 128 keys
// it loads. The rows of a tile are tokens x query heads of one key head, so that a causal
// tile covers few tokens and a group's heads share their keys' loads. For each tile and block
//   S = Q K^T     128 x 128 into tensor memory (tcgen05.mma, both operands in shared memory)
//   P = 2^(S c - m c)   a thread for each row: running maximum m and sum l in registers
//   O += P V      P from tensor memory, where it takes S's place; V as it lies, MN-major
// While one tile's rows are in the exponentials, the other's products run. O stays in
// tensor memory and is scaled again only when a row's maximum has grown by more than
// 2^8 (the weights stay below that, in bf16 and in the sums' fp32), which after the first
// blocks is rare. P is rounded to bf16, as V is (at most 2^-8 of a weight; outputs are 2.1e-3 to 2.3e-3
// off in the mean square, 1.7e-3 by their own rounding); l adds the unrounded weights. (Two tiles in
// turn, and scaling O again only for large growth, are published methods for fused attention on
// these tensor cores, not this file's own.)
//
// Bound: the products, 1024 cycles of the tensor core for a tile and block of 128 channels.
// Alone, a CTA's ring of five keys' or values' tiles (160 KB beside 64 KB of queries) is
// short for what a load takes; a pair of CTAs (cta_group::2) makes each product 256 rows
// wide, each CTA holds half of the keys (rows) and of the values (channels), and the ring
// lasts twice as long. One 8192-token prompt, 32 heads of 128 on 8: 311 to 315 us, 1.75 PFLOP/s,
// 92 % of the rate of a large matrix product; single CTAs 335.
//
// Roles: warps 0-3 and 4-7 the rows of the two tiles (200 registers a thread: a row's 128
// scores are held at once), warp 8 issues the products (in a pair the first CTA's, for
// both), warp 9 the TMA loads, warp 10 writes zeros behind the last key, warp 11 finds
// what comes next. A CTA goes on with the places of CTAs that have not started (launch
// control answers which), so that its start and the ends of its items overlap.
//
// What a row does not see must not reach it: its scores are replaced before the maximum,
// and the places behind a sequence's last key in the last block of V are zeroed in shared
// memory (they may hold anything). A NaN or an infinity in the values of a key that some
// rows of a tile see and others do not still meets a weight of 0 in the product; rows
// whose result is not finite are therefore computed again by attend_row, which reads only
// what the row sees (0.3 to 0.5 us a key for a row and warp, about 1000 times the cost).
#include "kda_attn.cuh"
#include "kda_attn_fwd.h"
#include "kda_cluster.cuh"
#include "kda_tcgen05.cuh"
#include "kda_tma.h"

namespace kda {
namespace {

using namespace attn;

constexpr int kThreads = 384;
constexpr int kRows = 128;            // rows of a tile; keys of a block
constexpr int kHalf = kRows * 128;    // bytes of a block's 64 channels
constexpr float kGrow = 8.f;          // how far, in powers of two, a row's maximum may pass the one in use
// The tensor core truncates what it adds to O, by half an ulp of O on the average for each 16 keys:
// values of one sign came out 0.08 % low at 131072 keys, 0.66 % at 2^20, 10 % at 2^24. After every
// kHold blocks a row's O is therefore rounded to bf16 into the row's place of the output, and
// the tensor memory keeps the rest.
constexpr int kHold = 256;

template <int D, int CTAS>
struct Shape {
  static constexpr int kQTile = kRows * D * 2;
  static constexpr int kTile = kQTile / CTAS;       // this CTA's part of a block's keys, or of its values
  static constexpr int kKeys = kRows / CTAS;        // of its keys
  static constexpr int kStages = D == 128 ? 5 * CTAS : 8;
  static constexpr int kSmem = 2 * kQTile + kStages * kTile + 1024;
  static constexpr uint32_t kO = 256;  // columns: S and P of the tiles at 0 and 128, O at 256 and 256 + D
};

struct Params {
  kda_attn_fwd_args a;
  AttnParts parts;
  int G, Gp, sub, heads;      // Gp query heads to a tile, sub such sets a key head, heads sets in all
  int tile_tokens, per_token; // tokens to a tile; 65536 / Gp rounded up: row r is of token r per_token >> 16
  int slots;                  // places for query tiles
  long long keys;             // that a sequence may have
  unsigned long long limit;   // how long a wait may last, in ns, in the kernels for long rows
};

// What a CTA works on next.
struct Item {
  int n, hk, h0;         // sequence (-1: there is nothing left), key head, first query head
  int q0, k0;            // its first query and key
  int T, S, shift;       // queries and keys; query i sees keys up to i + shift
  int t0;                // first query token of the CTA
  int split, first;      // of the key blocks: which part of them, the first of these,
  int count[2];          // and how many each tile has
};

struct Head {
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], tail_there, tail_zero, drain;  // p_full: of each half of a block's keys
  uint64_t full[10], empty[10];
  uint64_t item_full[2], item_empty[2], item_near, ready, next_there;  // item_near: the loads of an item are almost all under way
  alignas(16) uint32_t next[4];  // the answer to the request for another CTA's place
  Item items[2];
  uint32_t bad[8];            // by block, of the last 8: keys on pages that are out of range, a bit for each 16
  float held_top[2 * kRows];  // by row: the maximum in use when its O was last held (not in a register: it is rarely looked at)
  uint32_t tmem_base;
  int failed;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 32 bytes at once, on a 32-byte boundary.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// One lane of the warp, which all enter.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}

// How long a wait may last where a sequence may have so many keys: ten seconds, and what 32 rows
// that a warp computes again may take beside others that do, 2 us a key and row (four times what
// one warp alone needs: 0.3 us with 64 channels, 0.46 with 128). (A limit that starts again while
// such rows go on cost every wait some instructions, and prompt tiles of two blocks 4 %: 32.3 ->
// 33.4 us for 64 prompts of up to 333 tokens; one that is not a constant 0.6 %.)
__host__ __device__ constexpr unsigned long long wait_limit(long long keys) { return 10000000000ull + 64000ull * static_cast<unsigned long long>(keys); }

// Waits for a phase, for a limited time; whether it came. (One statement, and callers that look
// at the results seldom: with the loop and its exits in the compiler's hands each wait of the
// thread that issues products left the tensor core idle for 140 cycles instead of 40. No hint that
// lets the thread sleep: 395 us instead of 407 for 8192 tokens and 32 heads of 128.)
template <bool LONG>
__device__ __forceinline__ bool wait(const Params& p, uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 t0, t1;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE;\n mov.u64 t0, %globaltimer;\n"
      "AGAIN:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE;\n mov.u64 t1, %globaltimer;\n"
      " sub.u64 t1, t1, t0;\n setp.lt.u64 q, t1, %3;\n @q bra AGAIN;\n mov.u32 %0, 0;\n bra END;\n"
      "DONE:\n mov.u32 %0, 1;\nEND:\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "l"(LONG ? p.limit : wait_limit(kHold * kRows))
      : "memory");
  return ok != 0;
}

// ---- what differs where a pair of CTAs works on tiles of 256 rows ----

// An arrival on the barrier at the same place in the pair's first CTA, whose thread issues
// the products of both.
template <int CTAS>
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  if (CTAS == 1) mbar_arrive_local(bar);
  else mbar_arrive_cluster(mapa_shared(smem_u32(bar), 0));
}

// An arrival on the barrier at the same place in every CTA when the products issued before are done.
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

template <int CTAS>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if (CTAS == 1) {
    tc05::mma_ss(d, a, b, idesc, add);
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  }
}
template <int CTAS>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if (CTAS == 1) {
    tc05::mma_ts(d, a, b, idesc, add);
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  }
}

// A load into this CTA's shared memory, counted on a barrier of the pair's first CTA.
template <int CTAS>
__device__ __forceinline__ void load_tile(void* smem, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  if (CTAS == 1) {
    tma_load_3d(smem, map, x, y, z, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(mapa_shared(smem_u32(bar), 0))
        : "memory");
  }
}

// The products of both tiles, issued by one thread. (It is elected: operands are then as
// the tensor core's instructions want them and an issue takes the products' own time, 64
// cycles each, where a thread chosen by its lane took 140. A warp for each tile's products
// interleaves them, and each waits longer for its own: 444 us instead of 395 for 8192
// tokens and 32 heads of 128.)
template <int D, int CTAS, bool LONG>
__device__ __forceinline__ bool issue_products(const Params& p, Head& sm, const unsigned char* tiles) {
  using Sh = Shape<D, CTAS>;
  constexpr uint32_t qk = tc05::idesc_f16kind(CTAS * kRows, kRows, true), pv = tc05::idesc_f16kind(CTAS * kRows, D, true) | tc05::kIdescBMnMajor;
  const uint64_t desc = tc05::smem_desc(0, 16, 1024, tc05::kSwizzle128B), desc_mn = tc05::smem_desc(0, kHalf, 1024, tc05::kSwizzle128B);
  const uint32_t q_base = smem_u32(tiles) >> 4, r_base = q_base + (2 * Sh::kQTile >> 4);
  auto scores = [&](int m, int s) {  // S = Q K^T
    const uint64_t q = desc + (q_base + m * (Sh::kQTile >> 4)), k = desc + (r_base + s * (Sh::kTile >> 4));
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      mma_ss<CTAS>(m * kRows, q + ((c / 4 * kHalf + c % 4 * 32) >> 4), k + ((c / 4 * (Sh::kKeys * 128) + c % 4 * 32) >> 4), qk, c > 0);
    }
    commit<CTAS>(&sm.s_full[m]);
  };
  auto values = [&](int m, int s, int from, int to, bool add) {  // O (+)= P V over keys 16 from .. 16 to - 1
    const uint64_t v = desc_mn + (r_base + s * (Sh::kTile >> 4));
#pragma unroll
    for (int c = from; c < to; ++c) mma_ts<CTAS>(Sh::kO + m * D, m * kRows + 8 * c, v + ((c * 16 * 128) >> 4), pv, add || c > 0);
  };
  bool going = true;
  int s = 0, phase = 0;              // stage of the ring that comes next
  int done[2] = {0, 0}, tiles_done[2] = {0, 0}, tails = 0;  // blocks and tiles so far, whose parities their barriers have
  auto advance = [&]() {
    if (++s == Sh::kStages) s = 0, phase ^= 1;
  };
  for (int k = 0; going; ++k) {
    going = wait<LONG>(p, &sm.item_full[k & 1], (k >> 1) & 1);
    if (!going) break;
    const Item& it = sm.items[k & 1];
    if (it.n < 0) break;
    const int count0 = it.count[0], count1 = it.count[1], blocks = max(count0, count1), keys = it.S - it.first * kRows;
    if (blocks > 0) {
      going = wait<LONG>(p, &sm.full[s], phase);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int count = m == 0 ? count0 : count1;
        if (count == 0) continue;
        going = going && wait<LONG>(p, &sm.q_full[m], tiles_done[m]++ & 1);
        tc05::fence_after_sync();
        if (going) scores(m, s);
        if (count == 1) commit<CTAS>(&sm.q_empty[m]);
      }
      commit<CTAS>(&sm.empty[s]);
      advance();
    }
    int i = 0;
    // blocks that both tiles use and that others follow: no conditions between the products
    for (const int both = min(count0, count1) - 1; i < both && going; ++i) {
      const int vs = s;
      bool there = wait<LONG>(p, &sm.full[vs], phase);
      advance();
      there &= wait<LONG>(p, &sm.full[s], phase);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int parity = done[m]++ & 1;
        there &= wait<LONG>(p, &sm.p_full[m][0], parity);
        tc05::fence_after_sync();
        values(m, vs, 0, 4, i > 0);
        there &= wait<LONG>(p, &sm.p_full[m][1], parity);
        tc05::fence_after_sync();
        values(m, vs, 4, kRows / 16, true);
        scores(m, s);
        if (i + 2 == (m == 0 ? count0 : count1)) commit<CTAS>(&sm.q_empty[m]);
      }
      commit<CTAS>(&sm.empty[s]);
      commit<CTAS>(&sm.empty[vs]);
      advance();
      going = there;
    }
    for (; i < blocks && going; ++i) {
      const int vs = s, v_phase = phase;  // the block's values; the next block's keys come after them
      advance();
      going = wait<LONG>(p, &sm.full[vs], v_phase);
      if (i + 1 < blocks) going = going && wait<LONG>(p, &sm.full[s], phase);
      const bool tail = keys < (i + 1) * kRows;  // the sequence's last block is not full: zeros behind its last key
      if (tail && going) {
        mbar_arrive_local(&sm.tail_there);
        if (CTAS == 2) mbar_arrive_cluster(mapa_shared(smem_u32(&sm.tail_there), 1));
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int count = m == 0 ? count0 : count1;
        if (i >= count || !going) continue;
        const bool last_v = m == 1 || i >= count1, last_k = m == 1 || i + 1 >= count1;  // no other tile needs the block
        const int parity = done[m]++ & 1;
        going = wait<LONG>(p, &sm.p_full[m][0], parity);
        if (tail) going = going && wait<LONG>(p, &sm.tail_zero, tails & 1);
        tc05::fence_after_sync();
        if (going) values(m, vs, 0, 4, i > 0);
        going = going && wait<LONG>(p, &sm.p_full[m][1], parity);
        tc05::fence_after_sync();
        if (going) values(m, vs, 4, kRows / 16, true);
        if (i + 1 < count) {
          if (going) scores(m, s);
          if (i + 2 == count) commit<CTAS>(&sm.q_empty[m]);
          if (last_k) commit<CTAS>(&sm.empty[s]);
        } else {
          commit<CTAS>(&sm.o_full[m]);
        }
        if (last_v) commit<CTAS>(&sm.empty[vs]);
      }
      if (tail) ++tails;
      if (i + 1 < blocks) advance();
    }
    mbar_arrive_local(&sm.item_empty[k & 1]);
  }
  if (!going) {  // products in flight end before their tensor memory is given back
    commit<CTAS>(&sm.drain);
    wait<LONG>(p, &sm.drain, 0);
  }
  return going;
}

// The item of a place in the grid: false where no tile has it. One warp.
// Places in falling order, so that a causal prompt's long tiles start first. Sequence n's
// tiles have the places from cu_seqlens[n] / (tokens of a CTA) + n on, of which there are
// enough for it before the next sequence's.
template <bool PAGED, int CTAS>
__device__ __forceinline__ bool item_of(const Params& p, long long index, int lane, Item& it) {
  const kda_attn_fwd_args& a = p.a;
  const int tile_tokens = CTAS * p.tile_tokens, cta_tokens = 2 * tile_tokens;
  it.split = static_cast<int>(index % p.parts.splits);
  index /= p.parts.splits;
  const int set = static_cast<int>(index % p.heads);
  const int slot = p.slots - 1 - static_cast<int>(index / p.heads);
  it.hk = set / p.sub;
  it.h0 = it.hk * p.G + set % p.sub * p.Gp;
  int tile;
  if (a.cu_seqlens) {
    int lo = 0, n = a.N;  // the last sequence whose places start at this one or before it
    while (n > 1) {
      const int step = (n + 31) / 32, at = lane * step;
      const bool before = at < n && a.cu_seqlens[lo + at] / cta_tokens + lo + at <= slot;
      const int which = __popc(__ballot_sync(0xffffffffu, before)) - 1;
      lo += which * step;
      n = min(step, n - which * step);
    }
    it.n = lo;
    it.q0 = a.cu_seqlens[lo];
    it.T = a.cu_seqlens[lo + 1] - it.q0;
    tile = slot - (it.q0 / cta_tokens + lo);
    const int32_t* ck = a.cu_seqlens_k ? a.cu_seqlens_k : a.cu_seqlens;
    it.k0 = ck[lo];
    it.S = ck[lo + 1] - it.k0;
  } else {
    it.n = slot % a.N;
    tile = slot / a.N;
    it.T = a.T;
    it.S = a.S;
    it.q0 = it.n * it.T;
    it.k0 = it.n * it.S;
  }
  if (PAGED) it.S = a.seq_lens_k ? a.seq_lens_k[it.n] : p.parts.keys;
  if (static_cast<long long>(tile) * cta_tokens >= it.T) return false;
  it.t0 = tile * cta_tokens;
  it.shift = it.S - it.T;
  const int blocks = (it.S + kRows - 1) / kRows, per = (blocks + p.parts.splits - 1) / p.parts.splits;
  it.first = min(blocks, it.split * per);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int t = it.t0 + m * tile_tokens, last = min(t + tile_tokens, it.T) - 1;
    const int seen = t >= it.T ? 0 : a.flags & KDA_ATTN_FLAG_CAUSAL ? min(it.S, last + it.shift + 1) : it.S;
    it.count[m] = max(0, min((max(seen, 0) + kRows - 1) / kRows, it.first + per) - it.first);
  }
  return true;
}

// Asks for the place of a CTA (or pair) of this grid that has not started yet; the answer
// comes to sm.next of every CTA of the pair and counts 16 bytes on its sm.next_there.
template <int CTAS>
__device__ __forceinline__ void ask_for_place(Head& sm) {
  if (CTAS == 1) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_u32(sm.next)),
                 "r"(smem_u32(&sm.next_there))
                 : "memory");
  } else {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], [%1];" ::"r"(
            smem_u32(sm.next)),
        "r"(smem_u32(&sm.next_there))
        : "memory");
  }
}
// Whether the answer gives a place, and which.
__device__ __forceinline__ bool place_given(const Head& sm, uint32_t& place) {
  uint32_t given;
  asm volatile(
      "{\n .reg .b128 answer;\n .reg .pred p;\n .reg .b64 lo, hi;\n"
      " ld.shared.v2.b64 {lo, hi}, [%2];\n mov.b128 answer, {lo, hi};\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, answer;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, answer;\n}\n"
      : "=r"(given), "=r"(place)
      : "r"(smem_u32(sm.next))
      : "memory");
  return given != 0;
}

// Where a row's rounded part of O is held: its place of the output, or the second half of its
// (fp32) place among the results to join, which the results are written to from the front.
template <int D>
__device__ __forceinline__ __nv_bfloat16* held_row(const Params& p, const Item& it, int ti, int row_head) {
  const kda_attn_fwd_args& a = p.a;
  const long long tok = it.q0 + ti;
  if (p.parts.o == nullptr) return static_cast<__nv_bfloat16*>(a.o) + tok * a.o_stride + static_cast<long long>(it.h0 + row_head) * D;
  const long long row = static_cast<long long>(it.split) * a.B * a.T * a.HQ + tok * a.HQ + it.h0 + row_head;
  return reinterpret_cast<__nv_bfloat16*>(p.parts.o + row * D + D / 2);
}

// What values held under the maximum `was` are worth under `now`.
__device__ __forceinline__ float held_keep(float was, float now, float c2) { return was == now ? 1.f : ex2_approx((was - now) * c2); }

// Adds what is held, times `keep` (0: there is nothing yet), to a row of O in tensor memory, and, with
// `out`, holds the sum's bf16 part instead. `held`: nullptr for rows that are not there. A warp.
// (Rolled up and apart: beside the loop's other instructions it took prompt tiles of two blocks
// from 32.3 to 34.3 us.)
template <int D>
__device__ __forceinline__ void hold(uint32_t o_at, __nv_bfloat16* held, float keep, bool out) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tc05::ld32_wait(o_at + c, o);
    if (held != nullptr) {
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        uint4* at = reinterpret_cast<uint4*>(held + c + j);
        uint4 r = keep != 0.f ? *at : make_uint4(0u, 0u, 0u, 0u);
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float &x = o[j + 2 * e], &y = o[j + 2 * e + 1];
          x += keep * __uint_as_float(w[e] << 16);
          y += keep * __uint_as_float(w[e] & 0xffff0000u);
          if (!out) continue;
          w[e] = Bf16::pack(x, y);
          x -= __uint_as_float(w[e] << 16);
          y -= __uint_as_float(w[e] & 0xffff0000u);
        }
        if (out) *at = r;
      }
    }
    __syncwarp();
    tc05::st32_wait(o_at + c, o);
  }
}

// LONG: rows may have more than kHold blocks. Shorter ones have kernels without what these need (64
// prompts of up to 333 tokens, heads of 64: 32.4 us instead of 34.3; 128 prompts of 256, heads of
// 128: 179 instead of 181).
template <int D, bool PAGED, int CTAS, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
    kda_attn_fwd_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using Sh = Shape<D, CTAS>;
  extern __shared__ unsigned char raw[];
  __shared__ Head sm;
  const kda_attn_fwd_args& a = p.a;
  // (a step that joins these results has work of its own to do before it)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  unsigned char* ring = tiles + 2 * Sh::kQTile;
  const int rank = CTAS == 1 ? 0 : static_cast<int>(cluster_ctarank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool causal = a.flags & KDA_ATTN_FLAG_CAUSAL;

  // The arrays of lengths: checked whole by every CTA, so that a call with bad ones does nothing.
  bool ok = true;
  if (a.cu_seqlens || a.seq_lens_k) {
    for (int i = tid; i <= a.N; i += kThreads) {
      if (a.cu_seqlens) ok &= i == 0 ? a.cu_seqlens[0] == 0 : a.cu_seqlens[i] >= a.cu_seqlens[i - 1] && a.cu_seqlens[i] <= a.T;
      if (a.cu_seqlens_k) ok &= i == 0 ? a.cu_seqlens_k[0] == 0 : a.cu_seqlens_k[i] >= a.cu_seqlens_k[i - 1] && a.cu_seqlens_k[i] <= a.S;
      if (a.seq_lens_k && i < a.N) ok &= a.seq_lens_k[i] >= 0 && a.seq_lens_k[i] <= a.table_width * a.page_size;
    }
    if (!__syncthreads_and(ok)) {
      if (blockIdx.x == 0 && tid == 0) set_err(a.err, KDA_ERR_INVALID_ARG);
      return;
    }
  }

  if (warp == 0) {
    if (CTAS == 1) {
      tc05::tmem_alloc(&sm.tmem_base, 512);
      tc05::tmem_relinquish();
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)), "r"(512) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  if (tid == 8 * 32) {
    for (int m = 0; m < 2; ++m) {
      mbar_init(&sm.q_full[m], 1);
      mbar_init(&sm.q_empty[m], 1);
      mbar_init(&sm.item_full[m], 1);
      mbar_init(&sm.item_empty[m], rank == 0 ? 11 : 10);
      mbar_init(&sm.s_full[m], 1);
      mbar_init(&sm.p_full[m][0], 4 * CTAS);
      mbar_init(&sm.p_full[m][1], 4 * CTAS);
      mbar_init(&sm.o_full[m], 1);
    }
    for (int s = 0; s < Sh::kStages; ++s) {
      mbar_init(&sm.full[s], PAGED ? CTAS : 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.tail_there, 1);
    mbar_init(&sm.tail_zero, CTAS);
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.item_near, 1);
    mbar_init(&sm.ready, CTAS);
    mbar_init(&sm.next_there, 1);
    sm.failed = 0;
    fence_mbarrier_init_cluster();
  }
  if (warp == 9 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&qmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  if (CTAS > 1) cluster_sync_all();
  tc05::fence_after_sync();
  // (all 512 columns: the allocation starts at 0)
  const uint32_t tmem = 0;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 9) {
      // ---- loads: the tiles' queries, then keys and values block by block ----
      // a block's keys and values in boxes of so many keys and 64 channels, one a lane
      constexpr int kParts = D / 64;
      const int box_keys = PAGED ? min(a.page_size, Sh::kKeys) : Sh::kKeys, v_box_keys = PAGED ? box_keys : kRows;
      const uint32_t q_bytes = static_cast<uint32_t>(p.Gp * p.tile_tokens) * D * 2;
      bool going = true;
      int loaded = 0, blocks_done = 0, tiles_done[2] = {0, 0};
      for (int k = 0; going; ++k) {
        going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.item_full[k & 1], (k >> 1) & 1));
        if (!going) break;
        const Item it = sm.items[k & 1];
        if (it.n < 0) break;
        const int most = max(it.count[0], it.count[1]);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (it.count[m] == 0 || !going) continue;
          if (tiles_done[m] > 0) going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.q_empty[m], (tiles_done[m] - 1) & 1));
          if (!going) continue;
          ++tiles_done[m];
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx_local(&sm.q_full[m], CTAS * q_bytes);
            for (int c = 0; c < D / 64; ++c)
              load_tile<CTAS>(tiles + m * Sh::kQTile + c * kHalf, &qmap, 64 * c, it.h0, it.q0 + it.t0 + (m * CTAS + rank) * p.tile_tokens, &sm.q_full[m]);
          }
        }
        if (lane == 0 && most <= 1) mbar_arrive_local(&sm.item_near);
        for (int j = it.first; j < it.first + most && going; ++j) {
          if (lane == 0 && most > 1 && j == it.first + most - 2) mbar_arrive_local(&sm.item_near);
          for (int kv = 0; kv < 2 && going; ++kv, ++loaded) {
            // keys: this CTA's share of them, all channels; values: all keys, its share of the channels
            const int parts = kv == 0 ? kParts : kParts / CTAS, keys = kv == 0 ? box_keys : v_box_keys;
            const int boxes = (kv == 0 ? Sh::kKeys : kRows) / keys * parts, part = lane / parts, half = lane % parts;
            const int tok = j * kRows + part * keys + (kv == 0 ? rank * Sh::kKeys : 0);
            int y = it.hk, z = it.k0 + tok;
            uint32_t bad = 0;
            if (PAGED) {
              // a page that is out of range, or behind the last key, reads as zeros
              const int32_t* table = a.block_table + static_cast<long long>(it.n) * a.table_width;
              int page = -1;
              if (lane < boxes && tok < it.S) {
                page = table[tok / a.page_size];
                if (page >= a.pages) page = -1;
              }
              y = tok % a.page_size;
              z = page < 0 ? -1 : page * a.HKV + it.hk;
              if (kv == 0) {  // a bit for each 16 of the block's keys, those of the pair's other CTA among them
                if (CTAS == 1) {
                  bad = __ballot_sync(0xffffffffu, lane < boxes && tok < it.S && page < 0);
                  if (bad != 0) bad = __ballot_sync(0xffffffffu, lane < 8 && (bad >> (lane * 16 / keys * parts) & 1u));
                } else {
                  const int at = j * kRows + 16 * lane;
                  const bool there = lane < 8 && at < it.S;
                  if (there) page = table[at / a.page_size];
                  bad = __ballot_sync(0xffffffffu, there && (page < 0 || page >= a.pages));
                }
                if (bad != 0 && lane == 0) set_err(a.err, KDA_ERR_INVALID_ARG);
              }
            }
            const int s = loaded % Sh::kStages;
            if (loaded >= Sh::kStages) going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.empty[s], (loaded / Sh::kStages - 1) & 1));
            if (!going) break;
            if (lane == 0) {
              // (before the keys' arrival, and so before their scores; the loads are at most 5
              // blocks ahead of the weights, which read this)
              if (PAGED && kv == 0) sm.bad[(blocks_done + j - it.first) & 7] = bad;
              if (rank == 0) mbar_arrive_expect_tx_local(&sm.full[s], CTAS * Sh::kTile);
              else if (PAGED) arrive_first<CTAS>(&sm.full[s]);
            }
            __syncwarp();
            if (lane < boxes)
              load_tile<CTAS>(ring + s * Sh::kTile + half * (kv == 0 ? Sh::kKeys * 128 : kHalf) + part * keys * 128, kv == 0 ? &kmap : &vmap,
                              64 * (half + (kv == 0 ? 0 : rank * parts)), y, z, &sm.full[s]);
          }
        }
        blocks_done += most;
        __syncwarp();
        if (lane == 0) mbar_arrive_local(&sm.item_empty[k & 1]);
      }
      // every tile and stage has been used up: no copy and no arrival is left under way when
      // the CTA ends (after a wait that ran out: the copies have come, those of a pair both
      // counted in its first CTA, and neither CTA ends before the other)
      bool idle = going;
      for (int m = 0; m < 2; ++m)
        if (idle && tiles_done[m] > 0) idle = wait<LONG>(p, &sm.q_empty[m], (tiles_done[m] - 1) & 1);
      for (int i = max(0, loaded - Sh::kStages); i < loaded && idle; ++i) idle = wait<LONG>(p, &sm.empty[i % Sh::kStages], (i / Sh::kStages) & 1);
      if (!idle && rank == 0) {
        bool there = true;
        for (int m = 0; m < 2; ++m)
          if (there && tiles_done[m] > 0) there = wait<LONG>(p, &sm.q_full[m], (tiles_done[m] - 1) & 1);
        for (int i = max(0, loaded - Sh::kStages); i < loaded && there; ++i) there = wait<LONG>(p, &sm.full[i % Sh::kStages], (i / Sh::kStages) & 1);
      }
      going = idle;
      if (!going) sm.failed = 1;
    } else if (warp == 8) {
      if (rank == 0 && elect_one() && !issue_products<D, CTAS, LONG>(p, sm, tiles)) sm.failed = 1;
    } else if (warp == 10) {
      // ---- what stands behind the last key may be anything: zeros in its place ----
      bool going = true;
      int loaded = 0, tails = 0;
      for (int k = 0; going; ++k) {
        going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.item_full[k & 1], (k >> 1) & 1));
        if (!going) break;
        const Item it = sm.items[k & 1];
        if (it.n < 0) break;
        const int most = max(it.count[0], it.count[1]), live = it.S - (it.first + most - 1) * kRows;
        if (most > 0 && live < kRows) {
          const int s = (loaded + 2 * most - 1) % Sh::kStages;
          going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.tail_there, tails++ & 1));
          if (!going) break;
          unsigned char* v = ring + s * Sh::kTile;
          for (int c = 0; c < D / 64 / CTAS; ++c)
            for (int u = live * 8 + lane; u < kRows * 8; u += 32) *reinterpret_cast<uint4*>(v + c * kHalf + u * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_first<CTAS>(&sm.tail_zero);
        }
        loaded += 2 * most;
        __syncwarp();
        if (lane == 0) mbar_arrive_local(&sm.item_empty[k & 1]);
      }
      if (!going) sm.failed = 1;
    } else {
      // ---- places: this CTA's own, then those of CTAs that have not started. One is asked
      // for when the loads are two blocks from the end of the item before: earlier, the
      // first CTAs of a grid of few would take the others' places from idle SMs. ----
      bool going = true, more = true;
      uint32_t place = blockIdx.x;
      int k = 0, asked = 0;
      while (going) {
        Item it;
        if (!more) it.n = -1;
        if (!more || item_of<PAGED, CTAS>(p, place / CTAS, lane, it)) {
          if (k >= 2) going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.item_empty[k & 1], ((k >> 1) - 1) & 1));
          if (going && lane == 0) {
            sm.items[k & 1] = it;
            mbar_arrive_local(&sm.item_full[k & 1]);
          }
          if (more && going) going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.item_near, k & 1));
          ++k;
        }
        if (!more || !going) break;
        // (every CTA of a pair has read the last answer, and expects the next, before it is asked for)
        if (lane == 0) {
          mbar_arrive_expect_tx_local(&sm.next_there, 16);
          arrive_first<CTAS>(&sm.ready);
        }
        if (rank == 0) going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.ready, asked & 1));
        if (going && rank == 0 && lane == 0) ask_for_place<CTAS>(sm);
        ++asked;
        if (!going) break;
        going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.next_there, (asked - 1) & 1));
        if (!going) break;
        more = place_given(sm, place);
        fence_proxy_async_smem();  // (the next answer is written after this one has been read)
        __syncwarp();
      }
      if (!going) sm.failed = 1;
    }
  } else {
    // ---- rows ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int m = warp >> 2, r = tid & (kRows - 1);
    const int row_token = r * p.per_token >> 16, row_head = r - row_token * p.Gp;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t s_at = lanes + m * kRows, o_at = lanes + Sh::kO + m * D;
    const float c2 = a.scale * kLog2e;
    bool going = true;
    int done = 0, tiles_done = 0, blocks_done = 0;
    for (int k = 0; going; ++k) {
    going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.item_full[k & 1], (k >> 1) & 1));
    if (!going) break;
    const Item& it = sm.items[k & 1];
    if (it.n < 0) break;
    const int first = it.first, count = it.count[m];
    const int own = it.t0 + (m * CTAS + rank) * p.tile_tokens;  // the first token of this CTA's rows
    const int ti = own + row_token;
    const bool valid = row_token < p.tile_tokens && ti < it.T;
    const int limit = !valid ? 0 : causal ? max(0, min(it.S, ti + it.shift + 1)) : it.S;  // keys this row sees
    // blocks below this end need no mask (the tile's first row sees all of them)
    const int open = causal ? min(it.S, own + it.shift + 1) : it.S;
    float top = -INFINITY, sum = 0.f;
    for (int i = 0;;) {
    for (const int end = LONG ? min(count, i + kHold) : count; i < end && going; ++i, ++done) {
      const bool there = wait<LONG>(p, &sm.s_full[m], done & 1);  // (looked at below, when nothing waits for it)
      __syncwarp();
      tc05::fence_after_sync();
      const int k0 = (first + i) * kRows;
      const uint32_t bad = PAGED ? sm.bad[(blocks_done + i) & 7] : 0;
      float s[128];
      auto load = [&]() {
        tc05::ld128_wait(s_at, s);
        if (k0 + kRows > open || (PAGED && bad != 0)) {
#pragma unroll
          for (int j = 0; j < 128; ++j) s[j] = k0 + j < limit ? s[j] : -INFINITY;
          if (PAGED && bad != 0) {
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (bad >> (j / 16) & 1u) s[j] = -INFINITY;
          }
        }
      };
      load();
      const float2 c22 = make_float2(c2, c2);
      float2 base2, sum2[2];
      float w[32];  // weights of half of the block's keys, in bf16 pairs
      auto weigh = [&](int h) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float2 x = fma2(make_float2(s[h + 2 * j], s[h + 2 * j + 1]), c22, base2);
          x.x = ex2_approx(x.x);
          x.y = ex2_approx(x.y);
          sum2[j & 1] = add2(sum2[j & 1], x);
          w[j] = __uint_as_float(Bf16::pack(x.x, x.y));
        }
      };
      auto restart = [&]() {
        const float base = top == -INFINITY ? 0.f : -top * c2;
        base2 = make_float2(base, base);
        sum2[0] = sum2[1] = make_float2(0.f, 0.f);
        weigh(0);
      };
      // With 128 channels, the first half's weights under the maximum in use, while this
      // block's is found: it rarely changes after the first blocks (in pairs, 8192 tokens and
      // 32 heads: 314 us instead of 337). With 64, where a block's products are half as long
      // and short prompts are nothing but first blocks, after it (64 prompts of up to 333
      // tokens: 33 us instead of 36; 64 of 512: 184 and 200; 8192 tokens, 32 heads: 279 and
      // 278), but in the kernels for long rows (40000 tokens, 8 heads: 1560 and 1420).
      constexpr bool kAhead = D == 128 || LONG;
      if (kAhead) restart();
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int j = 4; j < 124; j += 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[j + 2 * e], s[j + 2 * e + 1]);
      }
      const float high = fmaxf(max3(max3(mx[0], s[124], s[125]), max3(mx[1], s[126], s[127]), mx[2]), mx[3]);
      const bool grew = (high - top) * c2 > kGrow || (top == -INFINITY && high > top);
      if (__any_sync(0xffffffffu, grew)) {
        // (S of this block is there, so the product that last changed O is done)
        const float now = grew ? high : top;
        const float keep = grew ? ex2_approx((top - now) * c2) : 1.f;
        top = now;
        sum *= keep;
        if (i > 0) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tc05::ld32_wait(o_at + c, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= keep;
            tc05::st32_wait(o_at + c, o);
          }
        }
        if (kAhead) {
          load();
          restart();
        }
      }
      if (!kAhead) restart();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1) weigh(64);
        tc05::st32(s_at + 32 * h, w);
        tc05::wait_st();
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_first<CTAS>(&sm.p_full[m][h]);  // the products of these keys may start
      }
      going = __all_sync(0xffffffffu, there);
      sum += (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
    }
    if (!LONG || i == count || !going) break;
    // (S of the next block is there when the product that last changed O is done)
    going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.s_full[m], done & 1));
    if (!going) break;
    tc05::fence_after_sync();
    hold<D>(o_at, valid ? held_row<D>(p, it, ti, row_head) : nullptr, i > kHold ? held_keep(sm.held_top[m * kRows + r], top, c2) : 0.f, true);
    sm.held_top[m * kRows + r] = top;
    }
    if (going && count > 0) {
      going = __all_sync(0xffffffffu, wait<LONG>(p, &sm.o_full[m], tiles_done++ & 1));
      tc05::fence_after_sync();
      if (LONG && count > kHold) hold<D>(o_at, valid ? held_row<D>(p, it, ti, row_head) : nullptr, held_keep(sm.held_top[m * kRows + r], top, c2), false);
    }
    if (going) {
      const long long tok = it.q0 + ti, row = tok * a.HQ + it.h0 + row_head;
      const bool part = p.parts.o != nullptr;
      const long long part_row = static_cast<long long>(it.split) * a.B * a.T * a.HQ + row;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + tok * a.o_stride + static_cast<long long>(it.h0 + row_head) * D;
      const bool some = count > 0 && limit > first * kRows;  // this row has keys here
      const float inv = 1.f / sum;
      float2 total = make_float2(0.f, 0.f);  // not finite where a value is not (or where the values are next to that)
      const bool wide = part || ((reinterpret_cast<uintptr_t>(a.o) | static_cast<uintptr_t>(a.o_stride * 2)) & 31) == 0;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (count > 0) tc05::ld32_wait(o_at + c, o);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          o[j] = some ? o[j] * inv : 0.f;
          o[j + 1] = some ? o[j + 1] * inv : 0.f;
          total = add2(total, make_float2(o[j], o[j + 1]));
        }
        if (!valid) continue;
        // (32 bytes a store: a lane's rows are apart, and each store of a warp is 32 pieces
        // whatever their width; in 16 bytes the two tiles' took 5000 cycles)
        if (part) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[j + e]);
            store32(p.parts.o + part_row * D + c + j, w);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; j += 16) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = Bf16::pack(o[j + 2 * e], o[j + 2 * e + 1]);
            if (wide) {
              store32(out + c + j, w);
            } else {
              *reinterpret_cast<uint4*>(out + c + j) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(out + c + j + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      const bool finite = fabsf(total.x + total.y) < INFINITY;
      const float lse2 = some ? top * c2 + log2f(sum) : -INFINITY;
      if (valid && part) p.parts.lse[part_row] = lse2;
      if (valid && !part && a.lse) a.lse[row] = lse2 * kLn2;
      // rows that infinities or NaN took part in, one by one
      uint32_t again = __ballot_sync(0xffffffffu, valid && some && !finite);
      while (again != 0) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        __syncwarp();  // (the row's own lane has stored what all lanes store again)
        const long long stok = __shfl_sync(0xffffffffu, tok, src);
        const int shead = __shfl_sync(0xffffffffu, it.h0 + row_head, src);
        const int end = min(__shfl_sync(0xffffffffu, limit, src), (first + count) * kRows);
        const Keys keys = {a.k, a.v, PAGED ? a.block_table + static_cast<long long>(it.n) * a.table_width : nullptr,
                           a.pages, a.page_size, a.HKV, a.k_stride, a.v_stride, it.k0};
        float q[D / 32], o[D / 32], rm, rl;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          q[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[stok * a.q_stride + static_cast<long long>(shead) * D + lane + 32 * c]);
        const int begin = first * kRows, seen = max(end - begin, 0);
        const int used = attend_row<D>(q, keys, it.hk, seen, [begin](int j) { return begin + j; }, below_one(seen), c2, lane, a.err, rm, rl, o);
        const long long srow = stok * a.HQ + shead;
        const long long spart = static_cast<long long>(it.split) * a.B * a.T * a.HQ + srow;
        const float l2 = used == 0 || rl == 0.f ? -INFINITY : rm + log2f(rl);  // (keys that all score -inf: o is 0 / 0)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const float x = used == 0 ? 0.f : o[c] / rl;
          if (part) p.parts.o[spart * D + lane + 32 * c] = x;
          else static_cast<__nv_bfloat16*>(a.o)[stok * a.o_stride + static_cast<long long>(shead) * D + lane + 32 * c] = __float2bfloat16_rn(x);
        }
        if (lane == 0 && part) p.parts.lse[spart] = l2;
        if (lane == 0 && !part && a.lse) a.lse[srow] = l2 * kLn2;
      }
    }
    blocks_done += max(it.count[0], it.count[1]);
    // (O has been read: the next item's weights, and with them its products into O, come after this)
    tc05::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive_local(&sm.item_empty[k & 1]);
    }
    if (!going) sm.failed = 1;
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  tc05::fence_after_sync();
  if (tid == 0 && sm.failed) set_err(a.err, KDA_ERR_TIMEOUT);
  if (CTAS > 1) cluster_sync_all();  // neither CTA ends while the other may still signal it or read its memory
  if (warp == 0) {
    if (CTAS == 1) tc05::tmem_dealloc(tmem, 512);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Query heads of a tile's tokens: the largest divisor of the group that leaves no more
// than 8 of the 128 rows without a token (14 heads on 2: 18 tokens of 7 heads).
int heads_of_tile(int group) {
  for (int h = group < kRows ? group : kRows; h > 1; --h)
    if (group % h == 0 && kRows / h * h >= kRows - 8) return h;
  return 1;
}

template <int D, bool PAGED, int CTAS, bool LONG>
cudaError_t launch(Params p, cudaStream_t s) {
  using Sh = Shape<D, CTAS>;
  const kda_attn_fwd_args& a = p.a;
  const int tokens = 2 * CTAS * p.tile_tokens;
  const long long slots = a.cu_seqlens ? static_cast<long long>(a.T) / tokens + a.N : (static_cast<long long>(a.T) + tokens - 1) / tokens * a.N;
  if (slots > INT32_MAX) return cudaErrorNotSupported;
  p.slots = static_cast<int>(slots);
  CUtensorMap qmap, kmap, vmap;
  const long long queries = static_cast<long long>(a.B) * a.T;
  bool ok = encode_heads(&qmap, a.q, D, a.HQ, D, queries, a.q_stride, static_cast<unsigned>(p.Gp), static_cast<unsigned>(p.tile_tokens));
  if (PAGED) {
    // a cache without pages is never read (every page is out of range): any map will do
    const long long rows = static_cast<long long>(a.pages) * a.HKV, page = static_cast<long long>(a.page_size) * D;
    const unsigned box = static_cast<unsigned>(a.page_size < Sh::kKeys ? a.page_size : Sh::kKeys);
    const bool none = a.pages == 0;
    ok = ok && encode_heads(&kmap, none ? a.q : a.k, D, a.page_size, D, none ? 1 : rows, page, box, 1) &&
         encode_heads(&vmap, none ? a.q : a.v, D, a.page_size, D, none ? 1 : rows, page, box, 1);
  } else {
    const long long keys = static_cast<long long>(a.B) * a.S;
    const bool none = keys == 0;
    ok = ok && encode_heads(&kmap, none ? a.q : a.k, D, a.HKV, D, none ? 1 : keys, a.k_stride, 1, Sh::kKeys) &&
         encode_heads(&vmap, none ? a.q : a.v, D, a.HKV, D, none ? 1 : keys, a.v_stride, 1, kRows);
  }
  if (!ok) return cudaErrorInvalidValue;
  const long long grid = slots * p.heads * p.parts.splits * CTAS;
  if (grid > INT32_MAX) return cudaErrorNotSupported;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_limit_once(kda_attn_fwd_kernel<D, PAGED, CTAS, LONG>, Sh::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = CTAS;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = CTAS > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kda_attn_fwd_kernel<D, PAGED, CTAS, LONG>, p, qmap, kmap, vmap);
}

template <bool PAGED, bool LONG>
cudaError_t launch_width(const Params& p, cudaStream_t s) {
  const kda_attn_fwd_args& a = p.a;
  if (a.D == 64) return launch<64, PAGED, 1, LONG>(p, s);
  // Pairs of CTAs, each of which holds half of the keys and values, where there are two
  // rounds of them on the 76 pairs of SMs and sequences fill a tile on the average (32 heads
  // of 128 on 8: 64 prompts of up to 512 tokens 116 us with pairs, 130 without; 128 of 256
  // 177 and 207; 512 of 64 312 and 195; 4 x 512 tokens on 6512 keys, 128 pairs' work, 158
  // and 149).
  const int tokens = 4 * p.tile_tokens;
  const long long each = a.cu_seqlens ? static_cast<long long>(a.T) / a.N : a.T, items = static_cast<long long>(a.B) * a.T / tokens * p.heads;
  if (p.parts.o == nullptr && each >= tokens && items >= 2 * 76) return launch<128, PAGED, 2, LONG>(p, s);
  return launch<128, PAGED, 1, LONG>(p, s);
}

}  // namespace

AttnTiles attn_tiles(int group) {
  const int h = heads_of_tile(group);
  return {2 * (kRows / h), h};
}

cudaError_t launch_attn_prompts(const kda_attn_fwd_args& a, const AttnParts& parts, cudaStream_t s) {
  Params p = {};
  p.a = a, p.parts = parts;
  p.G = a.HQ / a.HKV;
  p.Gp = heads_of_tile(p.G);
  p.sub = p.G / p.Gp;
  p.heads = a.HKV * p.sub;
  p.tile_tokens = kRows / p.Gp;
  p.per_token = (65536 + p.Gp - 1) / p.Gp;
  p.keys = a.block_table == nullptr ? a.S : a.seq_lens_k ? static_cast<long long>(a.table_width) * a.page_size : parts.keys;
  p.limit = wait_limit(p.keys);
  if (p.keys > kHold * kRows) return a.block_table ? launch_width<true, true>(p, s) : launch_width<false, true>(p, s);
  return a.block_table ? launch_width<true, false>(p, s) : launch_width<false, false>(p, s);
}

cudaError_t launch_attn_fwd(const kda_attn_fwd_args& a, cudaStream_t s) { return launch_attn_prompts(a, AttnParts{nullptr, nullptr, 1, 0}, s); }

}  // namespace kda
