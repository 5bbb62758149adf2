// attn.cuh - attention of a ragged batch's new tokens over a paged cache.
//
//   s_j = scale q . k_j  for the keys j <= p (and j > p - window),
//   o = sum_j softmax(s)_j v_j,  lse = ln sum_j exp(s_j),
// p the position of the new token, kv_len - q_len + its place among the new
// tokens. One pass over the keys with the running maximum and sum; scores,
// statistics and o in fp32, o rounded once to bf16.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "rope.cuh"

namespace fp8k {

struct AttnArgs {
  const uint16_t* q;
  int64_t ldq;
  uint16_t* o;
  int64_t ldo;
  float* lse;  // null: not wanted
  int T, Hq, G, max_q;
  int window;  // keys a token sees at most
  float scale;
};

// One warp per (row, head); lane l holds elements l D/32 .. of q and o.
template <int D>
__global__ void __launch_bounds__(128) attn_simple_kernel(AttnArgs a, PagedArgs c) {
  constexpr int E = D / 32;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<int64_t>(a.T) * a.Hq) return;
  const int t = static_cast<int>(w / a.Hq), h = static_cast<int>(w % a.Hq);
  int b = 0;
  for (int i0 = 0; i0 < c.batch; i0 += 32)
    b += __popc(__ballot_sync(0xFFFFFFFFu, i0 + lane < c.batch && c.cu_q[min(i0 + lane, c.batch - 1) + 1] <= t));
  if (b >= c.batch) return;
  const int q0 = c.cu_q[b], q1 = c.cu_q[b + 1], len = c.kv_lens[b];
  if (!seq_ok(c, q0, q1, len, a.T) || q0 > t || t >= q1 || q1 - q0 > a.max_q) {
    if (lane == 0) report(FP8_DEV_BAD_INDEX);
    return;
  }
  const int p = len - q1 + t;
  float q[E], o[E], m = -INFINITY, l = 0.0f;
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.ldq + h * D + lane * E + e]) << 16) * a.scale;
    o[e] = 0.0f;
  }
  for (int j = max(0, p - a.window + 1); j <= p; ++j) {
    const int32_t page = c.table[static_cast<int64_t>(b) * c.max_pages + j / c.page_size];
    if (page < 0 || page >= c.num_pages) {
      if (lane == 0) report(FP8_DEV_BAD_INDEX);
      continue;
    }
    const int64_t at = page * c.page_stride + (j % c.page_size) * c.token_stride + h / a.G * c.head_stride + lane * E;
    float s = 0.0f;
    for (int e = 0; e < E; ++e) s += q[e] * __uint_as_float(static_cast<uint32_t>(c.k[at + e]) << 16);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    const float mn = fmaxf(m, s);
    const float f = expf(m - mn), pr = expf(s - mn);
    l = l * f + pr;
    m = mn;
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + pr * __uint_as_float(static_cast<uint32_t>(c.v[at + e]) << 16);
  }
  for (int e = 0; e < E; ++e)
    a.o[t * a.ldo + h * D + lane * E + e] = f32_to_bf16_rn(l > 0.0f ? o[e] / l : 0.0f);
  if (a.lse && lane == 0) a.lse[static_cast<int64_t>(t) * a.Hq + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace fp8k
