// What the softmax attention kernels share: where keys and values lie, partial
// results of a row and how they are joined, and a row's attention computed directly.
#pragma once

#include "kda_elem.cuh"

namespace kda {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Keys and values of one sequence. Paged: token t at place t % page_size of page
// table[t / page_size] of a cache [pages, HKV, page_size, D]; otherwise rows of a
// [tokens, HKV, D] tensor with a stride of their own, `first` being token 0.
struct Keys {
  const void* k;
  const void* v;
  const int32_t* table;  // nullptr: rows
  int pages, page_size, HKV;
  long long k_stride, v_stride, first;
};

// How far, in powers of two, the weights of n keys are held below 1: their sum stays below
// 1 / 2, and with it a sum of weighted values below the largest value (four times 1e38 is
// infinite, its mean is not).
__device__ __forceinline__ float below_one(int n) { return static_cast<float>(33 - __clz(n)); }

// A value times a weight that may have left fp32's range downwards: infinities stay.
__device__ __forceinline__ float weighed(float v, float w) { return fabsf(v) == INFINITY ? v : v * w; }

// Attention of one row of queries over `count` keys, the tokens token(0), token(1), ..; one
// warp, each key in turn with a running maximum: lane l holds channels l + 32 i. Reads only
// what the row sees, and follows the definition where infinities and NaN take part: a score of
// -inf weighs 0, a finite one always more than that, so that an infinite value stays one (and
// a finite one adds what fp32 has of its weight, which may be nothing). The sum l and the
// values o are relative to 2^m, which is 2^below above the largest score; 1024 keys are added
// up at a time (one sum would stop growing at 2^24 equal weights). q is the row already in
// fp32; scale2 = scale * log2(e). Returns how many keys there were (those on pages out of range
// are left out).
template <int D, typename Token>
__device__ __forceinline__ int attend_row(const float (&q)[D / 32], const Keys& s, int h, int count, const Token& token, float below, float scale2,
                                           int lane, int32_t* err, float& m, float& l, float (&o)[D / 32]) {
  m = -INFINITY, l = 0.f;
  float best = -INFINITY;  // the largest score; m is `below` above it
  float sum = 0.f, total[D / 32] = {};  // of the 1024s before
  int used = 0;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f, nan |= q[i] != q[i];
  const bool nan_row = __any_sync(0xffffffffu, nan);  // (padding that nothing has written, say)
  constexpr int N = 4;  // keys whose loads and sums are under way together
  const auto add = [&]() {
    sum += l, l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) total[i] += o[i], o[i] = 0.f;
  };
  for (int j0 = 0; j0 < count; j0 += N) {
    if (j0 % 1024 == 0) add();
    float x[N], v[N][D / 32];
    bool there[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      there[u] = j0 + u < count;
      x[u] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[u][i] = 0.f;
      if (!there[u]) continue;
      const int j = token(j0 + u);
      long long ka, va;
      if (s.table != nullptr) {
        const int page = s.table[j / s.page_size];
        there[u] = page >= 0 && page < s.pages;
        if (!there[u]) {
          if (lane == 0) set_err(err, KDA_ERR_INVALID_ARG);
          continue;
        }
        ka = va = ((static_cast<long long>(page) * s.HKV + h) * s.page_size + j % s.page_size) * D;
      } else {
        ka = (s.first + j) * s.k_stride + static_cast<long long>(h) * D;
        va = (s.first + j) * s.v_stride + static_cast<long long>(h) * D;
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int d = lane + 32 * i;
        x[u] += q[i] * __bfloat162float(static_cast<const __nv_bfloat16*>(s.k)[ka + d]);
        v[u][i] = __bfloat162float(static_cast<const __nv_bfloat16*>(s.v)[va + d]);
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) x[u] = warp_sum(x[u]) * scale2;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (!there[u]) continue;
      ++used;
      const float top = x[u] > best ? x[u] : best;  // (a NaN leaves it and makes p and l NaN)
      if (top != best) {  // (in all lanes)
        const float keep = best == -INFINITY ? 0.f : exp2f(best - top);
        best = top;
        l *= keep, sum *= keep;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = weighed(o[i], keep), total[i] = weighed(total[i], keep);
      }
      m = top + below;
      const float p = exp2f(x[u] - (top == -INFINITY ? 0.f : m));
      l += p;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] += x[u] == -INFINITY ? 0.f * v[u][i] : weighed(v[u][i], p);
    }
    if (l != l || (nan_row && used > 0)) {  // every output is NaN from here on
      l = __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = l;
      return used;
    }
  }
  add();
  l = sum;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = total[i];
  return used;
}

}  // namespace attn
}  // namespace kda
