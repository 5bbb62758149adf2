// rope.cuh - rotary positions, and appending keys and values to a paged cache
// with the rotation applied on the way.
//
// A pair (x1, x2) of a head at position p turns by the angle p * f_j:
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s,  c = a cos(p f_j), s = a sin(p f_j),
// pair j = elements (j, j + R/2) (half layout) or (2j, 2j + 1) (interleaved)
// of the head's first R elements; the elements from R on are copied. fp32
// products and sums, one rounding to bf16.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "gemm.cuh"
#include "ptx.cuh"

namespace fp8k {

constexpr int kRopeThreads = 256;  // of a block, at most
constexpr int kRopeMaxRotary = 512;

struct RopeArgs {
  const float* inv_freq;  // [R / 2] radians per position
  int R;                  // rotated elements of a head (multiple of 16; 0 = none)
  int interleaved;
  float amplitude;
};

// c and s of the pairs of one position, into cs[R / 2]. The angle of a far
// position loses its low bits in fp32 (p = 131072: 8e-3 radians), so the
// turn is formed in fp64: p * f has at most 55 significant bits, and what
// is left of it after whole turns goes to fp32 in units of pi.
__device__ __forceinline__ void rope_angles(const RopeArgs& r, int p, float2* cs, int tid,
                                            int threads) {
  for (int j = tid; j < r.R / 2; j += threads) {
    const double t = static_cast<double>(p) * static_cast<double>(r.inv_freq[j]) *
                     0.31830988618379067154;  // 1 / pi
    const float u = static_cast<float>(t - 2.0 * rint(0.5 * t));
    float s, c;
    sincospif(u, &s, &c);
    cs[j] = make_float2(r.amplitude * c, r.amplitude * s);
  }
}

// A head's work comes in units of two 16-byte vectors: R / 16 rotating ones
// (eight pairs each), then copying ones for the other D - R elements (the
// last with one vector only when D - R is no multiple of 16). The first
// vectors of neighbouring units lie side by side, and so do the second ones,
// so that a warp's accesses are contiguous.
__host__ __device__ __forceinline__ int rope_units(int D) { return (D + 15) / 16; }  // R is a multiple of 16

struct RopeUnit {
  uint4 a, b;
  int ia, ib;  // element offsets in the head; ib < 0: no second vector
  bool rot;    // a rotating unit
};

__device__ __forceinline__ void rope_unit_load(RopeUnit& u, const uint16_t* head, int unit, int D,
                                               const RopeArgs& r, bool rotate) {
  const int rot = rotate ? r.R / 16 : 0;
  if (unit < rot) {
    u.rot = true;
    u.ia = 8 * unit;
    u.ib = u.ia + r.R / 2;
  } else {
    const int base = 16 * rot, second = (D - base + 15) / 16 * 8;  // elements the first vectors take
    u.rot = false;
    u.ia = base + 8 * (unit - rot);
    u.ib = u.ia + second < D ? u.ia + second : -1;
  }
  u.a = *reinterpret_cast<const uint4*>(head + u.ia);
  if (u.ib >= 0) u.b = *reinterpret_cast<const uint4*>(head + u.ib);
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void rope_unit_store(RopeUnit& u, uint16_t* head, const float2* cs,
                                                const RopeArgs& r) {
  if (u.rot) {
    float a[8], b[8];
    bf16x8_to_f32(u.a, a);
    bf16x8_to_f32(u.b, b);
    // eight pairs: from ia on, or when interleaved four from ia / 2 and four from ib / 2 on
    const float4* c4 = reinterpret_cast<const float4*>(cs + (r.interleaved ? u.ia / 2 : u.ia));
    const float4* d4 = reinterpret_cast<const float4*>(cs + (r.interleaved ? u.ib / 2 : u.ia + 4));
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = i < 2 ? c4[i] : d4[i - 2];
      c[2 * i] = v.x, s[2 * i] = v.y, c[2 * i + 1] = v.z, s[2 * i + 1] = v.w;
    }
    if (r.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a1 = a[2 * i], a2 = a[2 * i + 1], b1 = b[2 * i], b2 = b[2 * i + 1];
        a[2 * i] = a1 * c[i] - a2 * s[i];
        a[2 * i + 1] = a2 * c[i] + a1 * s[i];
        b[2 * i] = b1 * c[4 + i] - b2 * s[4 + i];
        b[2 * i + 1] = b2 * c[4 + i] + b1 * s[4 + i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x1 = a[i], x2 = b[i];
        a[i] = x1 * c[i] - x2 * s[i];
        b[i] = x2 * c[i] + x1 * s[i];
      }
    }
    u.a = f32_to_bf16x8(a);
    u.b = f32_to_bf16x8(b);
  }
  *reinterpret_cast<uint4*>(head + u.ia) = u.a;
  if (u.ib >= 0) *reinterpret_cast<uint4*>(head + u.ib) = u.b;
}

// Both kernels: a block takes a few tokens, whose rows (heads of one token
// after the other) are dealt to groups of rope_units(D) threads; a thread has
// the same unit in all of its rows, so it divides only once, and has
// kRopeFlight rows in flight. The positions and angles of the block's tokens
// are worked out once, under the first rows' loads. Bound by the bytes (one read,
// one write): 8191 tokens of 32 heads of 128 22.6 us, 5.9 TB/s, 0.92 of the copy
// rate; with their 8 + 8 heads of keys and values appended (8650 tokens) 39.6
// us, 5.4 TB/s. Two rows in flight: with one 27 us, with three 28 (fewer blocks
// on an SM).
constexpr int kRopeFlight = 2;
constexpr int kRopeTokens = 4;  // a block's, at most

struct RopeRow {
  int tok, row;  // row of the token
  int by_tok, by_row, per;
  __device__ __forceinline__ RopeRow(int first, int by, int per_) : per(per_) {
    tok = first / per, row = first - tok * per;
    by_tok = by / per, by_row = by - by_tok * per;
  }
  __device__ __forceinline__ void step() {
    tok += by_tok;
    row += by_row;
    if (row >= per) row -= per, ++tok;
  }
};

// y[t, h] = x[t, h] rotated by positions[t]. In place (y == x) is sound: a
// unit is read whole by the thread that writes it.
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const uint16_t* x, int64_t ldx,
                                                            const int32_t* __restrict__ positions, int T,
                                                            int tokens, int H, int D, RopeArgs r,
                                                            uint16_t* y, int64_t ldy) {
  extern __shared__ __align__(16) float2 rope_cs[];  // [tokens][R / 2]
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * tokens, nt = min(tokens, T - t0);
  const int units = rope_units(D), groups = blockDim.x / units, group = threadIdx.x / units;
  const int unit = threadIdx.x - group * units;
  RopeRow w(group, groups, H);
  if (group >= groups) w.tok = nt;  // a thread left over
  bool first = true;
  while (first || w.tok < nt) {
    RopeUnit u[kRopeFlight];
    int64_t at[kRopeFlight];
    int tk[kRopeFlight];
#pragma unroll
    for (int f = 0; f < kRopeFlight; ++f) {
      tk[f] = w.tok;
      if (w.tok < nt) {
        at[f] = static_cast<int64_t>(w.row) * D;
        rope_unit_load(u[f], x + (t0 + w.tok) * ldx + at[f], unit, D, r, true);
        w.step();
      }
    }
    if (first) {
      for (int k = 0; k < nt; ++k) rope_angles(r, positions[t0 + k], rope_cs + k * (r.R / 2), threadIdx.x, blockDim.x);
      __syncthreads();
      first = false;
    }
#pragma unroll
    for (int f = 0; f < kRopeFlight; ++f)
      if (tk[f] < nt) rope_unit_store(u[f], y + (t0 + tk[f]) * ldy + at[f], rope_cs + tk[f] * (r.R / 2), r);
  }
}

// ------------------------------------------------------------------ append
// The paged cache and the ragged batch, as the kernels see them (strides in
// elements; see bf16_paged_kv).
struct PagedArgs {
  uint16_t* k;
  uint16_t* v;
  int64_t num_pages, page_stride, token_stride, head_stride;
  int page_size, heads, D;
  const int32_t* table;
  int batch, max_pages;
  const int32_t* cu_q;
  const int32_t* kv_lens;
};

// Whether a sequence's offsets and length describe one (see the header).
__device__ __forceinline__ bool seq_ok(const PagedArgs& c, int q0, int q1, int len, int T) {
  return q0 >= 0 && q0 <= q1 && q1 <= T && len >= 0 &&
         len <= static_cast<int64_t>(c.max_pages) * c.page_size;
}

struct AppendArgs {
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  int64_t ldk, ldv, ldq, ldq_out;
  int Hq;  // 0: no queries
  int T;
};

// The new tokens' keys (rotated) and values go to their places in the cache,
// their queries (rotated) to q_out. The sequence of a block's first token is
// the number of offsets at or below it, counted by the block (one look for up
// to as many sequences as threads, two for their square); those of its other
// tokens follow from there.
__global__ void __launch_bounds__(kRopeThreads) kv_append_kernel(AppendArgs a, PagedArgs c, int tokens,
                                                                 RopeArgs r) {
  extern __shared__ __align__(16) float2 rope_cs[];  // [tokens][R / 2]
  __shared__ int64_t place[kRopeTokens];  // a token's offset in the cache; -1: it has none
  __shared__ int where[kRopeTokens];      // its position
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * tokens, nt = min(tokens, a.T - t0);
  int b0 = 0;
  int end = c.batch;  // it is in [b0, end]
#pragma unroll 1
  while (end - b0 > static_cast<int>(blockDim.x)) {  // thread i looks past the i-th `step` sequences
    const int step = (end - b0 + blockDim.x - 1) / blockDim.x, i = b0 + (threadIdx.x + 1) * step;
    b0 += step * __syncthreads_count(i <= end && c.cu_q[min(i, end)] <= t0);
    end = min(end, b0 + step);
  }
  const int next = b0 + threadIdx.x + 1;
  b0 += __syncthreads_count(next <= end && c.cu_q[min(next, end)] <= t0);
  if (threadIdx.x < nt) {
    const int t = t0 + threadIdx.x;
    int b = b0;
    while (b < c.batch && c.cu_q[b + 1] <= t) ++b;
    int64_t at = -1;
    int p = 0;
    if (b < c.batch && (b > 0 || t >= c.cu_q[0])) {  // (else a row behind the last sequence or in front of the first)
      const int q0 = c.cu_q[b], q1 = c.cu_q[b + 1], len = c.kv_lens[b];
      const int64_t p64 = static_cast<int64_t>(len) - q1 + t;  // len - q_len + (t - q0)
      int32_t page = -1;
      if (seq_ok(c, q0, q1, len, a.T) && q0 <= t && t < q1 && p64 >= 0) {
        p = static_cast<int>(p64);
        page = c.table[static_cast<int64_t>(b) * c.max_pages + p / c.page_size];
      }
      if (page >= 0 && page < c.num_pages)
        at = page * c.page_stride + (p % c.page_size) * c.token_stride;
      else
        report(FP8_DEV_BAD_INDEX);
    }
    place[threadIdx.x] = at;
    where[threadIdx.x] = p;
  }
  // a token's rows: its keys, its queries, its values
  const int units = rope_units(c.D), groups = blockDim.x / units, group = threadIdx.x / units;
  const int unit = threadIdx.x - group * units, nk = c.heads, nkq = c.heads + a.Hq;
  RopeRow w(group, groups, nkq + c.heads);
  if (group >= groups) w.tok = nt;  // a thread left over
  bool first = true;
  while (first || w.tok < nt) {
    RopeUnit u[kRopeFlight];
    int tk[kRopeFlight], row[kRopeFlight];
#pragma unroll
    for (int f = 0; f < kRopeFlight; ++f) {
      tk[f] = w.tok;
      row[f] = w.row;
      if (w.tok < nt) {
        const int64_t t = t0 + w.tok;
        const uint16_t* src = w.row < nk    ? a.k + t * a.ldk + static_cast<int64_t>(w.row) * c.D
                              : w.row < nkq ? a.q + t * a.ldq + static_cast<int64_t>(w.row - nk) * c.D
                                            : a.v + t * a.ldv + static_cast<int64_t>(w.row - nkq) * c.D;
        rope_unit_load(u[f], src, unit, c.D, r, w.row < nkq);
        w.step();
      }
    }
    if (first) {
      __syncthreads();  // place, where
      for (int k = 0; k < nt; ++k) rope_angles(r, where[k], rope_cs + k * (r.R / 2), threadIdx.x, blockDim.x);
      __syncthreads();
      first = false;
    }
#pragma unroll
    for (int f = 0; f < kRopeFlight; ++f) {
      if (tk[f] >= nt || place[tk[f]] < 0) continue;
      uint16_t* dst = row[f] < nk    ? c.k + place[tk[f]] + row[f] * c.head_stride
                      : row[f] < nkq ? a.q_out + (t0 + tk[f]) * a.ldq_out + static_cast<int64_t>(row[f] - nk) * c.D
                                     : c.v + place[tk[f]] + (row[f] - nkq) * c.head_stride;
      rope_unit_store(u[f], dst, rope_cs + tk[f] * (r.R / 2), r);
    }
  }
}

}  // namespace fp8k
