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

constexpr int kRopeThreads = 256;
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

// A head's work comes in units: R / 16 rotating ones (eight pairs: two
// 16-byte vectors) and (D - R) / 8 copying ones (one vector).
__device__ __forceinline__ int rope_units(int D, int R) { return R / 16 + (D - R) / 8; }

struct RopeUnit {
  uint4 a, b;
  int ia, ib;  // element offsets in the head; ib < 0: a copying unit
  int pair;    // first pair of a rotating unit
};

__device__ __forceinline__ void rope_unit_load(RopeUnit& u, const uint16_t* head, int unit,
                                               const RopeArgs& r) {
  const int rot = r.R / 16;
  if (unit < rot) {
    u.pair = 8 * unit;
    u.ia = r.interleaved ? 16 * unit : 8 * unit;
    u.ib = r.interleaved ? u.ia + 8 : u.ia + r.R / 2;
    u.b = *reinterpret_cast<const uint4*>(head + u.ib);
  } else {
    u.ia = r.R + 8 * (unit - rot);
    u.ib = -1;
  }
  u.a = *reinterpret_cast<const uint4*>(head + u.ia);
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
  if (u.ib >= 0) {
    float a[8], b[8];
    bf16x8_to_f32(u.a, a);
    bf16x8_to_f32(u.b, b);
    const float4* c4 = reinterpret_cast<const float4*>(cs + u.pair);
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = c4[i];
      c[2 * i] = v.x, s[2 * i] = v.y, c[2 * i + 1] = v.z, s[2 * i + 1] = v.w;
    }
    if (r.interleaved) {  // a: pairs 0..3 of the unit, b: pairs 4..7
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
    *reinterpret_cast<uint4*>(head + u.ib) = u.b;
  }
  *reinterpret_cast<uint4*>(head + u.ia) = u.a;
}

// y[t, h] = x[t, h] rotated by positions[t]; one block per token. In place
// (y == x) is sound: a unit is read whole by the thread that writes it.
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const uint16_t* x, int64_t ldx,
                                                            const int32_t* __restrict__ positions,
                                                            int H, int D, RopeArgs r, uint16_t* y,
                                                            int64_t ldy) {
  __shared__ __align__(16) float2 cs[kRopeMaxRotary / 2];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int units = rope_units(D, r.R), n = H * units;
  rope_angles(r, positions[t], cs, threadIdx.x, kRopeThreads);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kRopeThreads) {
    const int h = i / units;
    RopeUnit u;
    rope_unit_load(u, x + t * ldx + static_cast<int64_t>(h) * D, i - h * units, r);
    rope_unit_store(u, y + t * ldy + static_cast<int64_t>(h) * D, cs, r);
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

// New token t of the batch: its keys (rotated) and values go to its place in
// the cache, its queries (rotated) to q_out; one block per token. The
// sequence is the number of offsets at or below t, counted by the block.
__global__ void __launch_bounds__(kRopeThreads) kv_append_kernel(AppendArgs a, PagedArgs c,
                                                                 RopeArgs r) {
  __shared__ __align__(16) float2 cs[kRopeMaxRotary / 2];
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.x;
  int b = 0;
  for (int i0 = 0; i0 < c.batch; i0 += kRopeThreads) {
    const int i = i0 + threadIdx.x;
    b += __syncthreads_count(i < c.batch && c.cu_q[min(i, c.batch - 1) + 1] <= t);
  }
  if (b >= c.batch) return;  // a row behind the last sequence
  const int q0 = c.cu_q[b], q1 = c.cu_q[b + 1], len = c.kv_lens[b];
  const int64_t p64 = static_cast<int64_t>(len) - q1 + t;  // len - q_len + (t - q0)
  const bool ok = seq_ok(c, q0, q1, len, a.T) && q0 <= t && t < q1 && p64 >= 0;
  const int p = ok ? static_cast<int>(p64) : 0;
  const int32_t page = ok ? c.table[static_cast<int64_t>(b) * c.max_pages + p / c.page_size] : -1;
  if (page < 0 || page >= c.num_pages) {
    if (threadIdx.x == 0) report(FP8_DEV_BAD_INDEX);
    return;
  }
  rope_angles(r, p, cs, threadIdx.x, kRopeThreads);
  __syncthreads();
  const int64_t slot = page * c.page_stride + (p % c.page_size) * c.token_stride;
  const int units = rope_units(c.D, r.R), vecs = c.D / 8;
  const int nk = c.heads * units, nq = a.Hq * units, nv = c.heads * vecs;
  for (int i = threadIdx.x; i < nk + nq + nv; i += kRopeThreads) {
    if (i < nk + nq) {
      const bool key = i < nk;
      const int j = key ? i : i - nk;
      const int h = j / units;
      const uint16_t* src = key ? a.k + t * a.ldk : a.q + t * a.ldq;
      uint16_t* dst = key ? c.k + slot + h * c.head_stride
                          : a.q_out + t * a.ldq_out + static_cast<int64_t>(h) * c.D;
      RopeUnit u;
      rope_unit_load(u, src + static_cast<int64_t>(h) * c.D, j - h * units, r);
      rope_unit_store(u, dst, cs, r);
    } else {
      const int j = i - nk - nq;
      const int h = j / vecs, e = 8 * (j - h * vecs);
      *reinterpret_cast<uint4*>(c.v + slot + h * c.head_stride + e) =
          *reinterpret_cast<const uint4*>(a.v + t * a.ldv + static_cast<int64_t>(h) * c.D + e);
    }
  }
}

}  // namespace fp8k
