// attn.cuh - attention of a ragged batch's new tokens over a paged cache.
//
//   s_j = scale q . k_j  for the keys j <= p (and j > p - window),
//   o = sum_j softmax(s)_j v_j,  lse = ln sum_j exp(s_j),
// p the position of the new token, kv_len - q_len + its place among the new
// tokens. One pass over the keys with the running maximum and sum of the
// softmax, in base 2 (the scale times log2 e is folded into the exponent's
// argument); scores, statistics and o in fp32. The probabilities go to bf16
// for their product with v, as the tensor core takes them: each is off by 2^-8
// of itself at most, while their sum adds the unrounded ones (lse stays an
// fp32 value). o is rounded once to bf16. Against 64 bits the relative error of
// o, root mean square, is 1.8e-3 to 2.3e-3; that last rounding alone is 1.7e-3.
//
// Work. The query heads that share a key/value head are taken together: row
// r of an item is new token r / G, head r % G of the group, so keys and
// values are read once for the group. The items' key tiles, laid end to end
// (sequence, head, block of tokens, tile), are cut into equal runs, one per
// CTA: a ragged batch, a single long context and a full batch all load the
// device evenly. An item cut between CTAs leaves an unnormalised o with its
// maximum and sum for each part in the workspace, and a join kernel adds the
// parts in order. The cut depends on the lengths, the heads, the window, max_q
// (which picks the kernel) and the grid alone, so results are
// bit-reproducible. Every warp finds its CTA's run by itself from
// the lengths, so a captured graph follows lengths that change.
//
// Two kernels: attn_rows_kernel for items of at most 16 rows (max_q * G <= 16,
// one mma.sync row tile), attn_chunk_kernel for more, on tcgen05. The first is
// the one whose items cost little, and its cost grows with the rows; the
// second's does not. Measured, first / second, us, batches of 64 requests:
//              up to 300 keys                up to 4096 keys
//   rows       4           8           16           4          8          16
//   D 64   16.4/41.1   18.3/41.2   22.5/41.2    85/98      88/98      92/99
//   D 128  21.8/45.4   24.6/45.3   30.0/45.5   117/122    121/123    127/125
//   D 256  25.6/44.6   27.2/43.8   31.8/44.0   115/125    120/126    131/128
// At exactly 16 rows over long contexts of wide heads the second is ahead by
// some 2 % (single runs 8 %), over short ones the first by a third, so the rule
// takes the first.
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
  int window;        // keys a token sees at most
  float scale_log2;  // scale * log2(e)
  int box_rows;      // tokens of a page that one TMA box brings
  int drop;          // test hook: the load that CTA 0 skips (no arrive, no copies); -1: none
  // workspace: parts' o [2 per CTA][rows][D], their (maximum, sum)
  // [2 per CTA][rows], and per CTA what to join
  float* part_o;
  float2* part_ml;
  int4* part_desc;
};

// ------------------------------------------------------------------ work
// A sequence's new tokens and the key tiles they see: tiles tile0 ..
// tile0 + tiles - 1 of BN keys, of which the keys lo .. len - 1 count. A
// sequence without keys has one tile (of which none count), so that its
// zeros are written; one without new tokens, or an invalid one, none.
struct SeqSpan {
  int q0, ql, len;
  int lo, tile0, tiles;
  bool ok;
};

__device__ __forceinline__ SeqSpan seq_span(const AttnArgs& a, const PagedArgs& c, int b, int BN) {
  SeqSpan s;
  s.q0 = c.cu_q[b];
  const int q1 = c.cu_q[b + 1];
  s.len = c.kv_lens[b];
  s.ok = seq_ok(c, s.q0, q1, s.len, a.T) && q1 - s.q0 <= a.max_q;
  s.ql = s.ok ? q1 - s.q0 : 0;
  s.lo = max(0, s.len - s.ql - a.window + 1);  // lengths and window are at most 2^30
  s.tile0 = s.lo / BN;
  s.tiles = s.ql == 0 ? 0 : max(1, (s.len + BN - 1) / BN - s.tile0);
  return s;
}

// A CTA's run: the key tiles that start in `units` units from one of sequence
// `seq`'s on; `per` is the length of a full run. A tile is one unit long, or
// two, and an item's first one `extra` units more (what an item costs besides
// its tiles).
struct AttnRun {
  int seq;
  int units;
  int per;
  int extra;
  int head;       // the head it starts in,
  long long off;  // and the head's units before it
};

// Quotients of numbers that nearly always fit 32 bits (a 64-bit division
// takes some hundred cycles).
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// Sum, and sum of the lanes up to one's own, over a warp of numbers that nearly
// always fit 32 bits together.
__device__ __forceinline__ long long warp_sum(long long v) {
  if (!__any_sync(0xFFFFFFFFu, v >> 26)) return __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(v));
#pragma unroll 1
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {
  const int lane = lane_id();
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}
__device__ __forceinline__ long long warp_scan(long long v) {
  if (!__any_sync(0xFFFFFFFFu, v >> 26)) return warp_scan(static_cast<uint32_t>(v));
  const int lane = lane_id();
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// Units of a run from which on items count their own cost (an 8K prompt, runs
// of some 470 units: 541 us if they never do, 486 if they do; a draft check,
// runs of 14: 36.5 and 35.1); below, a run is about as short as the cost, and
// whole tiles decide.
constexpr int kExtraRun = 8;

// A head's key tiles, in units, and its items.
struct HeadUnits {
  long long units;
  int items;
  bool wide;  // some tiles are two units long
};

// Finds CTA `cta`'s run of `ctas`; whole warps call it, each for itself (that
// needs no barrier: for up to 32 sequences one round of loads and a scan).
// per_head(b), called by whole warps: one of sequence b's heads; none for b >=
// batch. A run is never shorter than the distance of two tiles' starts, so
// that every run inside an item holds a tile of it.
template <typename PerHead>
__device__ __forceinline__ AttnRun find_run(int batch, int heads, int cta, int ctas, int extra, PerHead per_head) {
  const int lane = lane_id();
  HeadUnits u = per_head(lane);
  long long sum = u.units, items = u.items;
  bool wide = u.wide;
#pragma unroll 1
  for (int b0 = 32; b0 < batch; b0 += 32) {
    const HeadUnits v = per_head(b0 + lane);
    sum += v.units, items += v.items, wide |= v.wide;
  }
  sum = warp_sum(sum) * heads, items = warp_sum(items) * heads;
  if (sum < static_cast<long long>(kExtraRun) * ctas) extra = 0;
  sum += items * extra;
  AttnRun r;
  r.seq = 0, r.units = 0, r.head = 0, r.off = 0, r.extra = extra;
  const long long per = max(__any_sync(0xFFFFFFFFu, wide) ? 2ll : 1ll, div_ll(sum + ctas - 1, ctas)), start = per * cta;
  r.per = static_cast<int>(per);
  if (start >= sum) return r;
  long long base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < batch; b0 += 32) {
    if (b0 > 0) u = per_head(b0 + lane);
    const long long units = u.units + static_cast<long long>(u.items) * extra, incl = warp_scan(units);
    const long long lo = base + (incl - units) * heads;
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, lo <= start && start < lo + units * heads);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const long long off = start - __shfl_sync(0xFFFFFFFFu, lo, src), n = __shfl_sync(0xFFFFFFFFu, units, src);
      r.seq = b0 + src;
      r.units = static_cast<int>(min(per, sum - start));
      r.head = static_cast<int>(div_ll(off, n));
      r.off = off - r.head * n;
      return r;
    }
    base += __shfl_sync(0xFFFFFFFFu, incl, 31) * heads;
  }
  return r;
}

// Base-2 exponential, flushing to zero (2 ulp).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr int kRowsMax = 16;  // rows of an attn_rows_kernel item
constexpr float kLn2 = 0.69314718055994531f;

// 1 / l for a sum of probabilities: 0 where no key was seen, so that o is 0;
// a NaN stays, so that it reaches o even where that was finite.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

// lse from a row's maximum and sum (base 2): -inf where no key was seen, and
// only there.
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2; }

// ------------------------------------------------------------------ join
// The parts of one cut item, in order: the first in slot `slot`, then slot
// 2 (cta + i) of the `more` following CTAs. Rows of the item: token t0 + r /
// G, head h0 + r % G.
__device__ __forceinline__ int4 join_desc(int more, int slot, int t0, int h0, int rows) {
  return make_int4(more | (rows << 16), slot, t0, h0);
}

// Parts of attn_rows_kernel, [slot][row][D]. One block per row of an item:
// warp w adds the parts w, w + 8, ... (a single long context has hundreds),
// then the warps' sums are added in order.
template <int D>
__global__ void __launch_bounds__(256) attn_join_rows_kernel(AttnArgs a) {
  constexpr int E = D / 32;  // values per lane
  __shared__ float so[8][D];
  pdl_launch_dependents();
  pdl_wait();
  const int4 d = a.part_desc[blockIdx.x];
  const int more = d.x & 0xFFFF, rows = d.x >> 16, r = blockIdx.y;
  if (more == 0 || r >= rows) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto slot = [&](int i) { return i == 0 ? d.y : 2 * (static_cast<int>(blockIdx.x) + i); };
  // every part's maximum and sum, by all lanes (each warp alike)
  float m = -INFINITY;
  for (int i = lane; i <= more; i += 32) m = fmaxf(m, a.part_ml[static_cast<int64_t>(slot(i)) * kRowsMax + r].x);
#pragma unroll
  for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
  const float mb = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int i0 = 0; i0 <= more; i0 += 32) {
    float f_l = 0.0f;
    if (i0 + lane <= more) {
      const float2 ml = a.part_ml[static_cast<int64_t>(slot(i0 + lane)) * kRowsMax + r];
      f_l = ex2(ml.x - mb);
      l += f_l * ml.y;
    }
    const int n = min(32, more + 1 - i0);
#pragma unroll 4
    for (int i = warp; i < n; i += 8) {
      const float f = __shfl_sync(0xFFFFFFFFu, f_l, i);
      const float* p = a.part_o + (static_cast<int64_t>(slot(i0 + i)) * kRowsMax + r) * D + lane * (E < 4 ? E : 4);
      if constexpr (E == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        acc[0] += f * v.x, acc[1] += f * v.y;
      } else {
#pragma unroll
        for (int q = 0; q < E / 4; ++q) {
          const float4 v = *reinterpret_cast<const float4*>(p + 128 * q);
          acc[4 * q] += f * v.x, acc[4 * q + 1] += f * v.y, acc[4 * q + 2] += f * v.z, acc[4 * q + 3] += f * v.w;
        }
      }
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, s);
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
  __syncthreads();
  if (warp != 0) return;
  for (int i = 1; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += so[i][lane * E + e];
  const int t = d.z + r / a.G, h = d.w + r % a.G;
  const float inv = inverse_sum(l);
  uint16_t* o = a.o + t * a.ldo + static_cast<int64_t>(h) * D + lane * (E < 4 ? E : 4);
  if constexpr (E == 2) {
    *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  } else {
#pragma unroll
    for (int q = 0; q < E / 4; ++q)
      *reinterpret_cast<uint2*>(o + 128 * q) =
          make_uint2(pack_bf16x2(acc[4 * q] * inv, acc[4 * q + 1] * inv),
                     pack_bf16x2(acc[4 * q + 2] * inv, acc[4 * q + 3] * inv));
  }
  if (a.lse && lane == 0)
    a.lse[static_cast<int64_t>(t) * a.Hq + h] = lse_of(m, l);
}

// Parts of attn_chunk_kernel, [slot][D / 4][row][4]: written by one thread
// per row, so that a warp's store is 512 bytes in a row. One block per 32
// rows of an item: a lane per row, the columns dealt to the eight warps; the
// rows leave through shared memory, 16 bytes a lane.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) attn_join_chunk_kernel(AttnArgs a) {
  constexpr int Q = D / 32;  // groups of four columns per warp
  __shared__ __align__(16) uint16_t so[32][D + 8];
  pdl_launch_dependents();
  pdl_wait();
  const int4 d = a.part_desc[blockIdx.x];
  const int more = d.x & 0xFFFF, rows = d.x >> 16;
  if (more == 0 || static_cast<int>(blockIdx.y) * 32 >= rows) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * 32 + lane;
  const bool live = r < rows;
  const auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? d.y : 2 * (static_cast<int>(blockIdx.x) + i)); };
  float m = -INFINITY, l = 0.0f;
  float4 acc[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) acc[q] = make_float4(0, 0, 0, 0);
  // Two parts at a time, all their loads at once.
  for (int i = 0; live && i <= more; i += 2) {
    float2 ml[2];
    float4 v[2][Q];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t at = slot(min(i + k, more));
      ml[k] = a.part_ml[at * ROWS + r];
      const float4* p = reinterpret_cast<const float4*>(a.part_o) + at * (D / 4) * ROWS + r;
#pragma unroll
      for (int q = 0; q < Q; ++q) v[k][q] = p[(warp + 8 * q) * ROWS];
    }
    if (i == more) ml[1] = make_float2(-INFINITY, 0.0f);
    const float mn = fmaxf(m, fmaxf(ml[0].x, ml[1].x)), mb = mn == -INFINITY ? 0.0f : mn;
    const float f = ex2(m - mb);
    m = mn;
    l *= f;
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[q].x *= f, acc[q].y *= f, acc[q].z *= f, acc[q].w *= f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float fk = ex2(ml[k].x - mb);
      l += fk * ml[k].y;
      // A part in which the row saw no key has no o. The factor does not tell
      // (maxima pass over NaN, so it may be 0 where l and o hold one).
      if (ml[k].x == -INFINITY && ml[k].y == 0.0f) continue;
#pragma unroll
      for (int q = 0; q < Q; ++q)
        acc[q].x += fk * v[k][q].x, acc[q].y += fk * v[k][q].y, acc[q].z += fk * v[k][q].z, acc[q].w += fk * v[k][q].w;
    }
  }
  const float inv = inverse_sum(l);
#pragma unroll
  for (int q = 0; q < Q; ++q)
    *reinterpret_cast<uint2*>(&so[lane][4 * (warp + 8 * q)]) =
        make_uint2(pack_bf16x2(acc[q].x * inv, acc[q].y * inv), pack_bf16x2(acc[q].z * inv, acc[q].w * inv));
  if (a.lse && live && warp == 0)
    a.lse[static_cast<int64_t>(d.z + r / a.G) * a.Hq + d.w + r % a.G] = lse_of(m, l);
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * (D / 8); i += 256) {
    const int rr = i / (D / 8), c8 = i % (D / 8), ro = blockIdx.y * 32 + rr;
    if (ro < rows)
      *reinterpret_cast<uint4*>(a.o + (d.z + ro / a.G) * a.ldo + static_cast<int64_t>(d.w + ro % a.G) * D + 8 * c8) =
          *reinterpret_cast<const uint4*>(&so[rr][8 * c8]);
  }
}

// ------------------------------------------------------------------ few rows
// attn_rows_kernel: items of at most 16 rows (one or a few new tokens times
// the heads of a group). Bound by the cache's bytes: 16 rows are 16 flops a
// byte, far below what mma.sync gives, and with 16 rows the warp-level
// instruction wastes nothing that a 128-row tcgen05 one would not waste
// eight times. A producer warp streams key and value tiles of 64 keys into a
// ring of shared-memory slots by TMA (one box per page piece); each of four
// warps takes 16 keys of every tile, with a maximum, sum and o of its own, so
// the main loop has no exchange between warps; they join through shared
// memory at an item's end. 64 requests of up to 8K keys (8 key/value heads of
// 128) take 212 us, 6.1 TB/s, 0.95 of the copy rate; one request's 120K keys (4
// of 256) 87 us, 5.7 TB/s; one of 1000 keys 8.5 us, which is latency: two
// launches, a look at the lengths, two tiles and the join.
constexpr int kRowsBN = 64;
constexpr int kRowsThreads = 160;

template <int D, int SLOTS>
struct RowsCfg {
  static constexpr int kSlotBytes = kRowsBN * D * 2;
  static constexpr int kXStride = 40;  // floats per row of the exchange: 32 columns, conflict-free
  static constexpr int kXBytes = 4 * kRowsMax * kXStride * 4;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(SLOTS) * kSlotBytes + kXBytes +
                                  2 * 4 * kRowsMax * 4 + 16 * SLOTS + 16;
};

// 5-D tiled load (see make_tmap_paged): coordinates (0, token, 0, head, page).
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int32_t token, int32_t head, int32_t page,
                                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %3, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(token), "r"(head), "r"(page),
      "l"(policy)
      : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Walks a run's segments: (sequence, head, tiles t0 .. t1 - 1 of the
// sequence's span). All roles walk alike.
struct RowsWalk {
  int b, h, t, left;
  SeqSpan s;
  __device__ __forceinline__ RowsWalk(const AttnArgs& a, const PagedArgs& c, const AttnRun& r) {
    b = r.seq;
    left = r.units;
    h = 0, t = 0;
    if (left > 0) {
      s = seq_span(a, c, b, kRowsBN);
      h = r.head;
      t = static_cast<int>(r.off);
    }
  }
  __device__ __forceinline__ int seg() const { return min(left, s.tiles - t); }
  __device__ __forceinline__ void next(const AttnArgs& a, const PagedArgs& c, int n) {
    left -= n;
    t = 0;
    if (++h == c.heads && left > 0) {
      h = 0;
      do {  // left > 0: a sequence with tiles follows
        if (++b >= c.batch) {
          left = 0;
          break;
        }
        s = seq_span(a, c, b, kRowsBN);
      } while (s.tiles == 0);
    }
  }
};

template <int D, int SLOTS>
__global__ void __launch_bounds__(kRowsThreads)
    attn_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const AttnArgs a, const PagedArgs c) {
  using C = RowsCfg<D, SLOTS>;
  static_assert(SLOTS % 2 == 0 && SLOTS <= 32, "slots: keys and values in turn");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  float* xch = reinterpret_cast<float*>(smem + SLOTS * C::kSlotBytes);
  float2* xml = reinterpret_cast<float2*>(xch + 4 * kRowsMax * C::kXStride);  // [4][16]
  uint64_t* bars = reinterpret_cast<uint64_t*>(xml + 4 * kRowsMax);
  uint32_t* abort_p = reinterpret_cast<uint32_t*>(bars + 2 * SLOTS);
  const uint32_t slot0 = smem_u32(smem), full0 = smem_u32(bars), empty0 = smem_u32(bars + SLOTS);
  const uint32_t abort_w = smem_u32(abort_p);
  const int warp = warp_id(), lane = lane_id(), cta = blockIdx.x;
  if (threadIdx.x == 0) {
    st_shared_volatile_u32(abort_w, 0u);
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 4);
    }
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  const AttnRun run = find_run(c.batch, c.heads, cta, gridDim.x, 0, [&](int b) -> HeadUnits {
    if (b >= c.batch) return {0, 0, false};
    const SeqSpan s = seq_span(a, c, b, kRowsBN);
    if (!s.ok && cta == 0) report(FP8_DEV_BAD_INDEX);
    return {s.tiles, 0, false};
  });
  RowsWalk w(a, c, run);

  if (warp == 4) {
    // ---------------------------------------------------------- producer
    const uint64_t policy = l2_policy_evict_first();
    const int rows = a.box_rows, boxes = kRowsBN / rows;
    const uint32_t box_bytes = static_cast<uint32_t>(rows) * D * 2;
    const int drop = cta == 0 ? a.drop : -1;
    int slot = 0, filled = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (w.left > 0 && ok) {
      const int n = w.seg();
      const int32_t* row = c.table + static_cast<int64_t>(w.b) * c.max_pages;
      // lane l holds the page of box l % boxes of tile l / boxes of a batch of 32 / boxes tiles
      int page = -1;
      for (int i = 0; i < n && ok; ++i) {
        const int batch_i = i % (32 / boxes);
        const int tile = w.s.tile0 + w.t + i;
        if (batch_i == 0) {
          const uint32_t tok = (static_cast<uint32_t>(tile) * boxes + lane) * rows;
          page = -2;  // not needed
          if (tok < static_cast<uint32_t>(w.s.len) && tok + rows > static_cast<uint32_t>(w.s.lo)) {
            page = row[tok / c.page_size];
            if (page < 0 || page >= c.num_pages) {
              report(FP8_DEV_BAD_INDEX);
              page = -1;
            }
          }
        }
        const int pg = __shfl_sync(0xFFFFFFFFu, page, (batch_i * boxes + lane) & 31);
        const bool mine = lane < boxes && pg >= 0;
        const int in_page = static_cast<int>((static_cast<uint32_t>(tile) * kRowsBN + lane * rows) % c.page_size);
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, mine)) * box_bytes;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (filled >= SLOTS && !mbar_wait_ab(empty0 + 8 * slot, phase ^ 1, abort_w)) ok = false;
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          const bool load = filled != drop;
          if (lane == 0 && load) mbar_arrive_expect_tx(full0 + 8 * slot, bytes);
          __syncwarp();
          if (mine && load)
            tma_load_page(slot0 + slot * C::kSlotBytes + lane * box_bytes, kv ? &tmV : &tmK,
                          full0 + 8 * slot, in_page, w.h, pg, policy);
          ++filled;
          if (++slot == SLOTS) slot = 0, phase ^= 1;
        }
      }
      w.next(a, c, n);
    }
    // Every copy started is waited for (bounded) before the CTA can exit, also
    // where the consumers give up after the last of them is on its way.
    if (lane == 0)
      for (int i = max(0, filled - SLOTS); i < filled; ++i)
        if (i != drop) mbar_wait(full0 + 8 * (i % SLOTS), (i / SLOTS) & 1);
    return;
  }

  // ------------------------------------------------------------ consumers
  const int g = lane >> 2, tq = lane & 3;
  // byte offsets of this lane's ldmatrix rows inside a slot: keys are
  // matrices 0,1 / 2,3 by eight rows and 16-byte columns 0 / 1 alternating,
  // values the other way round
  const int box = a.box_rows;
  auto key_row = [&](int key, uint32_t& off, uint32_t& sw) {
    const int r = key & (box - 1);
    off = static_cast<uint32_t>((key - r) * D * 2 + r * 128);  // box_rows is a power of two
    sw = static_cast<uint32_t>(r & 7) << 4;
  };
  uint32_t koff, ksw, voff, vsw;
  key_row(16 * warp + ((lane >> 4) << 3) + (lane & 7), koff, ksw);
  key_row(16 * warp + (((lane >> 3) & 1) << 3) + (lane & 7), voff, vsw);
  const uint32_t kcol = ((lane >> 3) & 1) << 4, vcol = (lane >> 4) << 4;
  const uint32_t half = static_cast<uint32_t>(box) * 128;  // bytes between 64-wide column groups
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true, desc_written = false;
  for (bool first = true; w.left > 0; first = false) {
    const int n = w.seg();
    const int rows = w.s.ql * a.G, h0 = w.h * a.G;
    const int p_first = w.s.len - w.s.ql;
    // positions of this lane's two rows
    const int pos0 = p_first + g / a.G, pos1 = p_first + (g + 8) / a.G;
    uint32_t qf[D / 16][4];
    {
      const bool v0 = g < rows, v1 = g + 8 < rows;
      const uint32_t* q0 = reinterpret_cast<const uint32_t*>(
          a.q + (w.s.q0 + (v0 ? g / a.G : 0)) * a.ldq + static_cast<int64_t>(h0 + (v0 ? g % a.G : 0)) * D);
      const uint32_t* q1 = reinterpret_cast<const uint32_t*>(
          a.q + (w.s.q0 + (v1 ? (g + 8) / a.G : 0)) * a.ldq + static_cast<int64_t>(h0 + (v1 ? (g + 8) % a.G : 0)) * D);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][0] = v0 ? q0[8 * k + tq] : 0u;
        qf[k][1] = v1 ? q1[8 * k + tq] : 0u;
        qf[k][2] = v0 ? q0[8 * k + 4 + tq] : 0u;
        qf[k][3] = v1 ? q1[8 * k + 4 + tq] : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;

    for (int i = 0; i < n && ok; ++i) {
      const int key0 = (w.s.tile0 + w.t + i) * kRowsBN + 16 * warp;
      // ---- scores of 16 keys
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_ab(full0 + 8 * slot, phase, abort_w));
      if (!ok) break;
      float s[2][4] = {};
      const uint32_t kb = slot0 + slot * C::kSlotBytes + koff;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t r[4];
        ldsm4(r, kb + (k >> 2) * half + ((((k & 3) << 5) + kcol) ^ ksw));
        mma16816(s[0], qf[k], r[0], r[1]);
        mma16816(s[1], qf[k], r[2], r[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * slot);
      if (++slot == SLOTS) slot = 0, phase ^= 1;
      // ---- running maximum, probabilities
      uint32_t vmask[2];  // values that count, of key pairs tq of each eight
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        vmask[nt] = 0u;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = key0 + 8 * nt + 2 * tq + e;
          if (j >= w.s.lo && j < w.s.len) vmask[nt] |= e ? 0xFFFF0000u : 0xFFFFu;
          const bool in0 = j <= pos0 && pos0 - j < a.window && j < w.s.len;
          const bool in1 = j <= pos1 && pos1 - j < a.window && j < w.s.len;
          s[nt][e] = in0 ? s[nt][e] * a.scale_log2 : -INFINITY;
          s[nt][2 + e] = in1 ? s[nt][2 + e] * a.scale_log2 : -INFINITY;
        }
      }
      float n0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float n1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      n0 = fmaxf(n0, __shfl_xor_sync(0xFFFFFFFFu, n0, 1));
      n1 = fmaxf(n1, __shfl_xor_sync(0xFFFFFFFFu, n1, 1));
      n0 = fmaxf(m0, fmaxf(n0, __shfl_xor_sync(0xFFFFFFFFu, n0, 2)));
      n1 = fmaxf(m1, fmaxf(n1, __shfl_xor_sync(0xFFFFFFFFu, n1, 2)));
      if (__any_sync(0xFFFFFFFFu, n0 > m0 || n1 > m1)) {
        const float f0 = n0 == -INFINITY ? 1.0f : ex2(m0 - n0), f1 = n1 == -INFINITY ? 1.0f : ex2(m1 - n1);
        l0 *= f0, l1 *= f1;
#pragma unroll
        for (int t = 0; t < D / 8; ++t) {
          o[t][0] *= f0, o[t][1] *= f0;
          o[t][2] *= f1, o[t][3] *= f1;
        }
        m0 = n0, m1 = n1;
      }
      const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[nt][e] = ex2(s[nt][e] - b0);
          s[nt][2 + e] = ex2(s[nt][2 + e] - b1);
        }
      l0 += (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]);
      l1 += (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
      const uint32_t pf[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                              pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
      // ---- o += p v
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_ab(full0 + 8 * slot, phase, abort_w));
      if (!ok) break;
      const uint32_t vb = slot0 + slot * C::kSlotBytes + voff;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        uint32_t r[4];
        ldsm4_t(r, vb + (t >> 2) * half + ((((t & 3) << 5) + vcol) ^ vsw));
        // values that do not count are taken as zeros: 0 times whatever they hold
        mma16816(o[2 * t], pf, r[0] & vmask[0], r[1] & vmask[1]);
        mma16816(o[2 * t + 1], pf, r[2] & vmask[0], r[3] & vmask[1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * slot);
      if (++slot == SLOTS) slot = 0, phase ^= 1;
    }

    // ---- the four warps' parts, in warp order
    l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 1);
    l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 1);
    l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 2);
    l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 2);
    if (tq == 0) {
      xml[warp * kRowsMax + g] = make_float2(m0, l0);
      xml[warp * kRowsMax + g + 8] = make_float2(m1, l1);
    }
    if (named_bar_or(1, 128, !ok)) {  // a wait gave up: the outputs are undefined
      if (threadIdx.x == 0) a.part_desc[cta] = make_int4(0, 0, 0, 0);
      return;
    }
    // this lane's factors, and the row it writes out
    auto joint = [&](int r, float& mm) {
      mm = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) mm = fmaxf(mm, xml[i * kRowsMax + r].x);
    };
    float j0, j1;
    joint(g, j0);
    joint(g + 8, j1);
    const float f0 = j0 == -INFINITY ? 0.0f : ex2(m0 - j0), f1 = j1 == -INFINITY ? 0.0f : ex2(m1 - j1);
    const int r = threadIdx.x >> 3, cg = (threadIdx.x & 7) * 4;
    float jm, jl = 0.0f;
    joint(r, jm);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = xml[i * kRowsMax + r];
      jl += (jm == -INFINITY ? 0.0f : ex2(v.x - jm)) * v.y;
    }
    const bool whole = w.t == 0 && n == w.s.tiles;
    const int part = 2 * cta + (first ? 0 : 1);
    const float inv = inverse_sum(jl);
    const int tok = w.s.q0 + r / a.G, head = h0 + r % a.G;
#pragma unroll
    for (int cb = 0; cb < D / 32; ++cb) {
      float* x = xch + warp * kRowsMax * C::kXStride;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        *reinterpret_cast<float2*>(x + g * C::kXStride + 8 * t + 2 * tq) =
            make_float2(o[4 * cb + t][0] * f0, o[4 * cb + t][1] * f0);
        *reinterpret_cast<float2*>(x + (g + 8) * C::kXStride + 8 * t + 2 * tq) =
            make_float2(o[4 * cb + t][2] * f1, o[4 * cb + t][3] * f1);
      }
      named_bar_sync(1, 128);
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 u = *reinterpret_cast<const float4*>(xch + (i * kRowsMax + r) * C::kXStride + cg);
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      if (r < rows) {
        if (whole)
          *reinterpret_cast<uint2*>(a.o + tok * a.ldo + static_cast<int64_t>(head) * D + 32 * cb + cg) =
              make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        else
          *reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(part) * kRowsMax + r) * D + 32 * cb + cg) = v;
      }
      named_bar_sync(1, 128);
    }
    if (r < rows && cg == 0) {
      if (!whole)
        a.part_ml[static_cast<int64_t>(part) * kRowsMax + r] = make_float2(jm, jl);
      else if (a.lse)
        a.lse[static_cast<int64_t>(tok) * a.Hq + head] = lse_of(jm, jl);
    }
    if (w.t == 0 && !whole) {  // the item's first part: what follows joins it
      desc_written = true;
      if (threadIdx.x == 0)
        a.part_desc[cta] = join_desc((w.s.tiles - n + run.per - 1) / run.per, part, w.s.q0, h0, rows);
    }
    w.next(a, c, n);
  }
  if (!desc_written && threadIdx.x == 0) a.part_desc[cta] = make_int4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ many rows
// attn_chunk_kernel: items of up to NT x 128 rows on the tensor cores. Per
// tile of 128 rows (128 / G tokens times the G heads of a group) and unit of
// keys:
//   S = Q K^T        tcgen05, both operands in shared memory, S in TMEM;
//   softmax          one thread per row: the unit's scores from TMEM to
//                    registers, P (bf16) back to TMEM over S;
//   O += P V         tcgen05, P from TMEM, V (keys x D) as a transposed
//                    operand, O in TMEM.
// Warps: four per row tile for the softmax, one that issues the MMAs, two that
// load (queries and keys; values). The softmax of 128 keys and the round trip
// P -> O += P V -> next S -> softmax are about as long (some 1700 and 1950
// cycles), so two are kept going: head_dim <= 128 with two row tiles, or, where
// an item has only one, with its key tiles in turn (each group of softmax
// warps with an o of its own, joined at the end: a draft check 42.5 -> 37.6
// us); head_dim 256 (whose O takes half of TMEM) with two buffers for S of its
// one row tile, the next scores being formed under this softmax. P is handed
// over in two halves, so that the product starts under the second half's
// exponentials.
// O is rescaled only when a row's maximum has grown by more than 2^8 since
// the last time (the factor cancels in the end, and 2^8 times a probability is
// as exact in bf16 and far from overflow in the sums): after the first tiles
// hardly ever, so the softmax threads do it themselves.
// Bound: 8192 tokens of 32 heads (head_dim 128, 8 key/value heads) take 500 us,
// 1.10 PFLOP/s, in short bursts at 1965 MHz, and 573 us call after call, where
// the 1000 W limit holds the clock at 1660 MHz. Per key tile of two row tiles that is some
// 3500 cycles, of which the tensor core works 2048 and the exponentials (4 a
// cycle and scheduler) 2048: what is left is the chain above, which with the
// two row tiles that TMEM holds (S, P and O of a third do not fit) is not quite
// covered. Slower: S and P apart in units of 64 keys (583 against 530 us),
// two threads per row (562), an issuing warp per row tile (613).
constexpr int kChunkBN = 128;  // keys of a loaded tile

template <int D>
struct ChunkCfg {
  static constexpr int kNT = D == 256 ? 1 : 2;       // row tiles of an item
  static constexpr int kParts = D == 256 ? 2 : 1;    // slots per key tile and per value tile
  static constexpr int kBufs = D == 256 ? 2 : 1;     // buffers for S per row tile
  static constexpr int kSlots = D == 64 ? 10 : 5;
  static constexpr int kSlotBytes = 128 * (D < 128 ? D : 128) * 2;
  static constexpr int kKCols = D < 128 ? D : 128;   // head elements of a key slot
  static constexpr int kVKeys = kChunkBN / kParts;   // keys of a value slot
  static constexpr int kQBytes = kNT * 128 * D * 2;
  static constexpr int kThreads = kNT * 128 + 128;
  static constexpr int kRows = kNT * 128;            // rows of a part in the workspace
  static constexpr int kBars = 2 * kSlots + 2 + 2 + 4 + 2 + 2 + 2;  // see ChunkBars
  static constexpr int kItemUnits = D == 256 ? 2 : 3;  // what an item costs besides its tiles, in units
  static constexpr int kWalkInts = 16;
  static constexpr size_t kSmem = 1024 + kQBytes + static_cast<size_t>(kSlots) * kSlotBytes + 8 * kBars + 16 +
                                  (kThreads / 32) * kWalkInts * 4 + (kNT == 2 ? 128 * 8 : 0);
};

// Key tiles that block j (tt tokens from tok0 on, the first at position
// first + tok0) of a sequence sees: from max(0, p - window + 1) to its last
// token, in tiles of 128; one where it sees none.
__device__ __forceinline__ int block_tiles(int first, int window, int tok0, int ntok, int& tile0) {
  const int p0 = first + tok0;
  tile0 = max(0, p0 < window ? 0 : p0 - window + 1) / kChunkBN;
  return max(1, (max(0, p0 + ntok) + kChunkBN - 1) / kChunkBN - tile0);
}

// How a key or value tile lies in shared memory: groups of 64 elements one
// after the other, each with all rows; or, where pages come in pieces of eight
// rows, the groups of a piece side by side, so that one box brings the piece
// whole: half as many boxes at head_dim 128, of which a warp starts one in some
// 60 cycles (pages of 8: a chunk beside decoding requests 147 -> 109 us). Longer
// pieces cannot lie like that: their rows' distances would not be even.
// (Both ways in one kernel cost the issuing thread 4 % of a prompt.)
constexpr int kPackedRows = 8;

// Units that a key tile of ntok tokens' rows counts for: CTAs' times in a
// mixed batch fit 1.1 us per key tile of one row tile, 1.9 us of two, and 3.4 us
// an item (ChunkCfg::kItemUnits; head_dim 256: 2.2 and 3.9 us). A chunk beside
// decoding requests took 127 us with all tiles alike and takes 110; an 8K
// prompt, whose early blocks are short items, 547 us without the items' cost
// and 495 with it.
__device__ __forceinline__ int tile_units(int ntok, int tt1) { return ntok > tt1 ? 2 : 1; }

// Block j's units in a head of ql new tokens; none behind the last.
__device__ __forceinline__ int block_units(const AttnArgs& a, int first, int ql, int j, int tt, int tt1) {
  const int tok0 = j * tt, ntok = min(tt, ql - tok0);
  int tile0;
  return ntok > 0 ? block_tiles(first, a.window, tok0, ntok, tile0) * tile_units(ntok, tt1) : 0;
}

// find_run's per_head: a lane per sequence of one block; the blocks of longer
// ones are added up by the whole warp, a block per lane.
__device__ __forceinline__ HeadUnits chunk_heads(const AttnArgs& a, const PagedArgs& c, int b, int tt, int tt1) {
  int first = 0, ql = 0;
  if (b < c.batch) {
    const SeqSpan s = seq_span(a, c, b, kChunkBN);
    if (!s.ok && blockIdx.x == 0) report(FP8_DEV_BAD_INDEX);
    first = s.len - s.ql, ql = s.ql;
  }
  HeadUnits u = {0, (ql + tt - 1) / tt, ql > tt1 && tt > tt1};
  if (ql <= tt) u.units = block_units(a, first, ql, 0, tt, tt1);
  for (uint32_t rest = __ballot_sync(0xFFFFFFFFu, ql > tt); rest; rest &= rest - 1) {
    const int src = __ffs(rest) - 1;
    const int f = __shfl_sync(0xFFFFFFFFu, first, src), q = __shfl_sync(0xFFFFFFFFu, ql, src);
    long long sum = 0;
#pragma unroll 1
    for (int j0 = 0; j0 * tt < q; j0 += 32)
      sum += __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(block_units(a, f, q, j0 + lane_id(), tt, tt1)));
    if (lane_id() == src) u.units = sum;
  }
  return u;
}

// The block of tt tokens at which a run starts in its head, and how far into
// it (whole warps).
__device__ __forceinline__ void find_block(const AttnRun& r, const AttnArgs& a, const PagedArgs& c, int tt, int tt1,
                                           int& block, int& unit) {
  block = unit = 0;
  if (r.units <= 0) return;
  const int lane = lane_id();
  const SeqSpan s = seq_span(a, c, r.seq, kChunkBN);
  const int first = s.len - s.ql;
  long long base = 0;
#pragma unroll 1
  for (int j0 = 0; j0 * tt < s.ql; j0 += 32) {
    const uint32_t units = block_units(a, first, s.ql, j0 + lane, tt, tt1);
    const uint32_t mine = units ? units + r.extra : 0, incl = warp_scan(mine);
    const long long lo = base + incl - mine;
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, lo <= r.off && r.off < lo + mine);
    if (hit) {
      const int src = __ffs(hit) - 1;
      block = j0 + src;
      unit = static_cast<int>(r.off - __shfl_sync(0xFFFFFFFFu, lo, src));
      return;
    }
    base += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
}

// A run's segments: tiles t .. of item (sequence b, head h, block j). Each
// warp has one in shared memory (the fields are needed once a segment and
// would cost the inner loops their registers); lane 0 moves it on.
struct ChunkWalk {
  int b, h, j, t, left;
  int q0, ql, len, first;  // the sequence
  int lo_seq;              // keys below it no new token sees
  int tok0, ntok, tile0, n;  // the item: tokens tok0 .. of the sequence, key tiles tile0 .. + n
  uint32_t g;                // key tiles walked so far
  int extra;

  __device__ __forceinline__ bool seq(const AttnArgs& a, const PagedArgs& c) {
    const SeqSpan s = seq_span(a, c, b, kChunkBN);
    q0 = s.q0, ql = s.ql, len = s.len;
    first = len - ql;
    lo_seq = s.lo;
    return ql > 0;
  }
  __device__ __forceinline__ void item(const AttnArgs& a, int tt) {
    tok0 = j * tt;
    ntok = min(ql - tok0, tt);
    n = block_tiles(first, a.window, tok0, ntok, tile0);
  }
  __device__ __forceinline__ void start(const AttnArgs& a, const PagedArgs& c, const AttnRun& r, int block, int unit,
                                        int tt, int tt1) {
    if (lane_id() == 0) {
      b = r.seq, left = r.units, h = r.head, j = block, t = 0, g = 0, extra = r.extra;
      if (left > 0) {
        seq(a, c);
        item(a, tt);
        if (unit > 0) {  // the first tile that starts in the run
          const int wt = tile_units(ntok, tt1);
          t = max(1, (unit - extra + wt - 1) / wt);
          left -= extra + t * wt - unit;
          if (t == n) advance(a, c, 0, tt, tt1);
        }
      }
    }
    __syncwarp();
  }
  __device__ __forceinline__ int seg(int tt1) const {
    const int x = t == 0 ? max(1, left - extra) : left;
    return min(ntok > tt1 ? (x + 1) >> 1 : x, n - t);
  }
  // The runs after this one that hold a part of the item, whose first tile is next.
  __device__ __forceinline__ int more(int per, int tt1) const {
    return n == 1 ? 0 : (per - left + extra + (n - 1) * tile_units(ntok, tt1)) / per;
  }
  // Past m tiles (one thread).
  __device__ __forceinline__ void advance(const AttnArgs& a, const PagedArgs& c, int m, int tt, int tt1) {
    left -= m * tile_units(ntok, tt1) + (t == 0 ? extra : 0);
    g += m;
    t = 0;
    if (left <= 0) return;
    ++j;
    if (j * tt >= ql) {
      j = 0;
      if (++h == c.heads) {
        h = 0;
        do {  // left > 0: a sequence with new tokens follows
          if (++b >= c.batch) {
            left = 0;
            return;
          }
        } while (!seq(a, c));
      }
    }
    item(a, tt);
  }
  __device__ __forceinline__ void next(const AttnArgs& a, const PagedArgs& c, int m, int tt, int tt1) {
    __syncwarp();
    if (lane_id() == 0) advance(a, c, m, tt, tt1);
    __syncwarp();
  }
  // Row tile i (tt1 tokens each): its tokens, and those of the segment's m key
  // tiles, [from, to), in which it sees keys.
  __device__ __forceinline__ int tile_tokens(int i, int tt1) const { return max(0, min(tt1, ntok - i * tt1)); }
  __device__ __forceinline__ void tile_range(const AttnArgs& a, int i, int tt1, int m, int& from, int& to) const {
    const int nt = tile_tokens(i, tt1);
    from = to = 0;
    if (nt == 0) return;
    const int p0 = first + tok0 + i * tt1;
    const int lo = (p0 < a.window ? 0 : p0 - a.window + 1) / kChunkBN;
    const int hi = max(lo + 1, (max(0, p0 + nt) + kChunkBN - 1) / kChunkBN);
    from = max(0, lo - tile0 - t);
    to = max(from, min(m, hi - tile0 - t));
  }
};

// tcgen05.mma with A in TMEM, issued by one thread.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory descriptors by halves: the upper one has the bytes from eight
// rows (or eight of K) to the next, 1024 unless said, version 1 and the
// 128-byte swizzle, the lower one the address in 16-byte units, to which
// offsets are simply added, and the lead offset: unused where K is contiguous,
// and where M/N is (the values: 64 elements of N by eight keys make a
// 1024-byte atom) the bytes from one group of 64 to the next.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr, uint32_t lead_bytes) {
  return (smem_addr >> 4) | (lead_bytes >> 4 << 16);
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi = kDescHi) {
  return (static_cast<uint64_t>(hi) << 32) | lo;
}
constexpr uint32_t kIdescBMnMajor = 1u << 16;  // operand B's contiguous dimension is N

// 5-D tiled load, coordinates (0, token, group of 64, head, page).
__device__ __forceinline__ void tma_load_page_cols(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                   int32_t token, int32_t group, int32_t head,
                                                   int32_t page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(token), "r"(group), "r"(head),
      "r"(page)
      : "memory");
}
// 4-D tiled load of queries, coordinates (0, head, token, group of 64).
__device__ __forceinline__ void tma_load_q(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                           int32_t head, int32_t token, int32_t group) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(head), "r"(token), "r"(group)
      : "memory");
}

// The largest of three (one instruction).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two sums, packed.
__device__ __forceinline__ void fadd2(float2& s, float a, float b) {
  asm("{\n\t.reg .b64 ps, pa;\n\t"
      "mov.b64 ps, {%0, %1};\n\tmov.b64 pa, {%2, %3};\n\t"
      "add.rn.f32x2 ps, ps, pa;\n\tmov.b64 {%0, %1}, ps;\n\t}"
      : "+f"(s.x), "+f"(s.y)
      : "f"(a), "f"(b));
}

// Two products plus a shared pair: d = a * b + c per lane.
__device__ __forceinline__ void ffma2(float& d0, float& d1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 pa, pb, pc, pd;\n\t"
      "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %4};\n\tmov.b64 pc, {%5, %5};\n\t"
      "fma.rn.f32x2 pd, pa, pb, pc;\n\tmov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}

// u[j] of lane q of four becomes u[q] of lane j: 4 x 4 pieces of 16 bytes.
__device__ __forceinline__ void quad_transpose(uint32_t (&u)[4][4], int lane) {
#pragma unroll
  for (int s = 1; s <= 2; s <<= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & s) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t r = __shfl_xor_sync(0xFFFFFFFFu, up ? u[j][e] : u[j + s][e], s);
        u[j][e] = up ? r : u[j][e];
        u[j + s][e] = up ? u[j + s][e] : r;
      }
    }
  }
}

// The probabilities of 64 keys from their scores (pairs of bf16, to TMEM),
// added up in sum.
__device__ __forceinline__ void chunk_probs(const uint32_t (&s)[64], float scale, float shift, uint32_t p_addr, float2 (&sum)[2]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float x0, x1;
      ffma2(x0, x1, __uint_as_float(s[32 * q + e]), __uint_as_float(s[32 * q + e + 1]), scale, shift);
      x0 = ex2(x0);
      x1 = ex2(x1);
      fadd2(sum[(e / 2) & 1], x0, x1);
      pk[e / 2] = pack_bf16x2(x0, x1);
    }
    tmem_st16(p_addr + 16 * q, pk);
  }
}

// The softmax of one row tile's rows, one thread per row. s_full, p_full: the
// tile's barriers, one and two (halves) per buffer.
template <int D>
__device__ __forceinline__ void chunk_softmax(const AttnArgs& a, const PagedArgs& c, ChunkWalk& w, int tile,
                                              int tt1, uint32_t tmem, uint32_t s_full, uint32_t p_full,
                                              uint32_t o_done, uint32_t ml_full, float2* ml, uint32_t abort_w,
                                              int per) {
  using C = ChunkCfg<D>;
  const int lane = lane_id(), quad = warp_id() & 3;
  const int rr = 32 * quad + lane;  // row of the tile
  const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
  const uint32_t s_addr0 = tmem + lanes + tile * C::kBufs * kChunkBN, o_addr = tmem + lanes + 256 + tile * D;
  const int cta = blockIdx.x;
  uint32_t done = 0;  // key tiles so far: products with V asked for
  bool ok = true;
  int4 desc = make_int4(0, 0, 0, 0);
  uint32_t segs = 0, joins = 0;
  for (bool first_seg = true; w.left > 0 && ok; first_seg = false) {
    const int m = w.seg(tt1);
    const bool turns = C::kNT == 2 && w.ntok <= tt1;  // both groups on row tile 0
    const bool join = turns && m > 1;
    const int rt = turns ? 0 : tile, step = turns ? 2 : 1;
    int from, to;
    w.tile_range(a, rt, tt1, m, from, to);
    if (turns) from += tile;
    const int ntok = w.tile_tokens(rt, tt1);
    const bool idle = 32 * quad >= ntok * a.G;     // this warp has no row
    const int p0 = w.first + w.tok0 + rt * tt1;    // positions p0 .. p0 + ntok - 1
    const int key_seg = (w.tile0 + w.t) * kChunkBN;
    const int rel0 = p0 + rr / a.G - key_seg;      // this row's position, from the segment's first key
    float mu = -INFINITY, l = 0.0f;
    for (int u = from; u < to; u += step) {
      const uint32_t buf = C::kBufs == 2 ? done & 1 : 0;
      const uint32_t s_addr = s_addr0 + buf * kChunkBN;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_ab(s_full + 8 * buf, (C::kBufs == 2 ? done >> 1 : done) & 1, abort_w));
      if (!ok) break;
      tc_fence_after();
      if (C::kBufs == 1 && idle) {  // P keeps what it holds: nothing reads those rows of o
        if (lane == 0) mbar_arrive(p_full), mbar_arrive(p_full + 8);
        ++done;
        continue;
      }
      const int key0 = key_seg + kChunkBN * u;
      const bool edge = key0 + kChunkBN - 1 > p0 || p0 + ntok - 1 - key0 >= a.window;
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t x[64];
        tmem_ld32(s_addr + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(x));
        tmem_ld32(s_addr + 64 * half + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
        tmem_ld_wait();
        if (edge) {
          const int rel = rel0 - kChunkBN * u - 64 * half;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (static_cast<uint32_t>(rel - e) >= static_cast<uint32_t>(a.window)) x[e] = 0xFF800000u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 16; e += 2) mx[q] = max3(mx[q], __uint_as_float(x[16 * q + e]), __uint_as_float(x[16 * q + e + 1]));
      }
      const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * a.scale_log2;
      const bool grow = top > mu + 8.0f;
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float nm = grow ? top : mu;
        const float f = grow ? ex2(mu - nm) : 1.0f;  // mu = -inf: 0 (l and o are 0)
        l *= f;
        mu = nm;
        if (u > from) {  // o holds the earlier keys: wait for their product
          if (C::kBufs == 2) ok = __all_sync(0xFFFFFFFFu, mbar_wait_ab(o_done, (done - 1) & 1, abort_w));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int cb = 0; cb < D; cb += 16) {
            uint32_t o[16];
            tmem_ld16(o_addr + cb, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(o_addr + cb, o);
          }
        }
      }
      const float shift = mu == -INFINITY ? 0.0f : -mu;
      float2 sum[2] = {};
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t x[64];
        tmem_ld32(s_addr + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(x));
        tmem_ld32(s_addr + 64 * half + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
        tmem_ld_wait();
        if (edge) {
          const int rel = rel0 - kChunkBN * u - 64 * half;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (static_cast<uint32_t>(rel - e) >= static_cast<uint32_t>(a.window)) x[e] = 0xFF800000u;
        }
        chunk_probs(x, a.scale_log2, shift, s_addr + 32 * half, sum);
        if (C::kBufs == 2 && half == 0 && u + 1 == to && u > from)
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_ab(o_done, (done - 1) & 1, abort_w));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 16 * buf + 8 * half);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      ++done;
    }
    if (!ok) break;
    // ---- the segment's o
    if (to > from) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_ab(o_done, (C::kBufs == 2 ? done - 1 : segs) & 1, abort_w));
      ++segs;
      if (!ok) break;
      tc_fence_after();
    }
    // A finite score that the scale takes past fp32 gives the maximum +inf,
    // from which the fused product and sum sees it as -inf: the sum says NaN.
    if (mu == INFINITY) l = __int_as_float(0x7FFFFFFF);
    // Two groups on one row tile: the second leaves its rows' statistics in
    // shared memory, the first reads them and both groups' o (its lanes of
    // TMEM are the same) and goes on alone.
    float f0 = 1.0f, f1 = 0.0f;
    if (join) {
      if (tile == 1) {
        ml[rr] = make_float2(mu, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_ab(ml_full + 8, joins & 1, abort_w));  // read
        tc_fence_after();
      } else {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_ab(ml_full, joins & 1, abort_w));
        tc_fence_after();
        const float2 x = ml[rr];
        const float mm = fmaxf(mu, x.x), mb = mm == -INFINITY ? 0.0f : mm;
        f0 = ex2(mu - mb);
        f1 = ex2(x.x - mb);
        mu = mm;
        l = l * f0 + x.y * f1;
      }
      ++joins;
      if (!ok) break;
    }
    const bool whole = w.t == 0 && m == w.n;
    const int part = 2 * cta + (first_seg ? 0 : 1);
    const bool live = rr < ntok * a.G && !(turns && tile == 1);  // ntok <= tt1
    const int row = rt * tt1 * a.G + rr;
    const int64_t tok = w.q0 + w.tok0 + rt * tt1 + rr / a.G;
    const int head = w.h * a.G + rr % a.G;
    const auto load_o = [&](int cb, uint32_t (&o)[32]) {
      tmem_ld32(o_addr + cb, o);
      tmem_ld_wait();
      if (C::kNT == 2 && join) {
        uint32_t o1[32];
        tmem_ld32(o_addr + D + cb, o1);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + __uint_as_float(o1[e]) * f1);
      }
    };
    if (to > from && !idle && !(turns && tile == 1)) {
      const float inv = inverse_sum(l);
      if (whole) {
        // Four lanes turn their rows' 16-byte pieces among themselves, so that
        // a store covers 8 rows x 64 bytes instead of 32 x 16.
        const int64_t mine = live ? tok * a.ldo + static_cast<int64_t>(head) * D : -1;
        int64_t at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) at[j] = __shfl_sync(0xFFFFFFFFu, mine, (lane & ~3) + j);
#pragma unroll 1
        for (int cb = 0; cb < D; cb += 32) {
          uint32_t o[32], u[4][4];
          load_o(cb, o);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              u[q][e] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * e]) * inv, __uint_as_float(o[8 * q + 2 * e + 1]) * inv);
          quad_transpose(u, lane);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (at[j] >= 0)
              *reinterpret_cast<uint4*>(a.o + at[j] + cb + 8 * (lane & 3)) = make_uint4(u[j][0], u[j][1], u[j][2], u[j][3]);
        }
      } else {
        float4* dst = reinterpret_cast<float4*>(a.part_o) + static_cast<int64_t>(part) * (D / 4) * C::kRows + row;
#pragma unroll 1
        for (int cb = 0; cb < D; cb += 32) {
          uint32_t o[32];
          load_o(cb, o);
          if (live)
#pragma unroll
            for (int q = 0; q < 8; ++q)
              dst[(cb / 4 + q) * C::kRows] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                                         __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
        }
      }
    }
    tc_fence_before();
    if (join && tile == 0) {
      __syncwarp();
      if (lane == 0) mbar_arrive(ml_full + 8);
    }
    if (live) {
      if (!whole)
        a.part_ml[static_cast<int64_t>(part) * C::kRows + row] = make_float2(mu, l);
      else if (a.lse)
        a.lse[tok * a.Hq + head] = lse_of(mu, l);
    }
    if (w.t == 0 && !whole)
      desc = join_desc(w.more(per, tt1), part, w.q0 + w.tok0, w.h * a.G, w.ntok * a.G);
    w.next(a, c, m, C::kNT * tt1, tt1);
  }
  if (tile == 0 && rr == 0) a.part_desc[cta] = ok ? desc : make_int4(0, 0, 0, 0);
}

// Barriers of the chunk kernel, by their addresses' offsets: full[kSlots],
// empty[kSlots], queries full and empty, S full (per buffer), P full (two
// halves per buffer), O done (per row tile), the V loader's own, drained, the
// second softmax group's statistics there and read.
template <int D>
struct ChunkBars {
  using C = ChunkCfg<D>;
  static constexpr uint32_t kEmpty = 8 * C::kSlots, kQFull = 16 * C::kSlots, kQEmpty = kQFull + 8, kSFull = kQFull + 16,
                            kPFull = kSFull + 16, kODone = kPFull + 32, kVTmp = kODone + 16, kDrained = kVTmp + 8, kMlFull = kDrained + 8, kMlEmpty = kMlFull + 8;
  static_assert(kMlEmpty + 8 == 8 * C::kBars, "barriers");
};

// The MMAs, issued by one thread. It shares its scheduler and instruction
// cache with two softmax warps, so what it does between two products counts:
// the slots' waits come before the probabilities' and the releases last.
template <int D, bool PACKED>
__device__ __forceinline__ bool chunk_issue_all(const AttnArgs& a, const PagedArgs& c, ChunkWalk& w, int tt1,
                                                uint32_t tmem, uint32_t q_smem, uint32_t slot0, uint32_t bars,
                                                uint32_t abort_w, bool& issued) {
  using C = ChunkCfg<D>;
  using B = ChunkBars<D>;
  constexpr int NT = C::kNT, NS = C::kSlots, PARTS = C::kParts;
  constexpr uint32_t kIdescS = idesc_kind<kKindBF16>(128, kChunkBN);
  constexpr uint32_t kIdescO = idesc_kind<kKindBF16>(128, D) | kIdescBMnMajor;
  // keys and values as the loads leave them (see kPackedRows)
  const uint32_t q_lo = desc_lo(q_smem, 16), k_lo = desc_lo(slot0, 16),
                 v_lo = desc_lo(slot0, PACKED ? 1024 : C::kVKeys * 128);
  constexpr uint32_t k_hi = PACKED ? kDescHi + (C::kKCols / 64 - 1) * 64 : kDescHi,
                     v_hi = PACKED ? kDescHi + (D / 64 - 1) * 64 : kDescHi;
  constexpr uint32_t k_group = PACKED ? 64 : 1024, v_step = PACKED ? D * 2 : 128;
  int slot = 0;  // next slot in load order
  uint32_t phase = 0, q_par = 0, p_par = 0;
  const auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait_ab(bars + bar, parity, abort_w); };
  // Waits for the next PARTS slots; they are used in load order.
  const auto take = [&](int (&at)[PARTS]) {
    bool ok = true;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      at[p] = slot;
      ok = ok && wait(8 * slot, phase);
      if (++slot == NS) slot = 0, phase ^= 1;
    }
    return ok;
  };
  const auto release = [&](const int (&at)[PARTS]) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) umma_commit(bars + B::kEmpty + 8 * at[p]);
  };
  // S of a key tile for row tile `tile` into its buffer `buf`.
  const auto scores = [&](int tile, int q_tile, uint32_t buf, const int (&at)[PARTS]) {
    const uint32_t b = tile * C::kBufs + buf;
    uint32_t kb[PARTS];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) kb[p] = k_lo + at[p] * (C::kSlotBytes / 16);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int p = k * 16 / C::kKCols, kk = k - p * (C::kKCols / 16);
      umma_kind<kKindBF16>(tmem + b * kChunkBN,
                           desc_of(q_lo + (q_tile * (128 * D * 2) + (k >> 2) * 16384 + (k & 3) * 32) / 16),
                           desc_of(kb[p] + (kk >> 2) * k_group + (kk & 3) * 2, k_hi), kIdescS, k > 0);
    }
    umma_commit(bars + B::kSFull + 8 * b);
    issued = true;
  };
  // Adds the product of P, as its halves come, with V.
  const auto product = [&](int tile, uint32_t buf, const int (&at)[PARTS], bool add, bool lastp) {
    const uint32_t b = tile * C::kBufs + buf, par = p_par >> b & 1;
    p_par ^= 1u << b;
    uint32_t vb[PARTS];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) vb[p] = v_lo + at[p] * (C::kSlotBytes / 16);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (!wait(B::kPFull + 16 * b + 8 * half, par)) return false;
      tc_fence_after();
#pragma unroll
      for (int k = 4 * half; k < 4 * half + 4; ++k) {
        const int p = k * 16 / C::kVKeys, kk = k - p * (C::kVKeys / 16);
        umma_bf16_ts(tmem + 256 + tile * D, tmem + b * kChunkBN + 8 * k, desc_of(vb[p] + kk * v_step, v_hi), kIdescO,
                     k > 0 ? 1u : static_cast<uint32_t>(add));
      }
    }
    if (C::kBufs == 2 || lastp) umma_commit(bars + B::kODone + 8 * tile);
    return true;
  };
  while (w.left > 0) {
    const int m = w.seg(tt1);
    int from[NT], to[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) w.tile_range(a, i, tt1, m, from[i], to[i]);
    int kat[PARTS], vat[PARTS];
    if (!wait(B::kQFull, q_par)) return false;
    q_par ^= 1;
    if (!take(kat)) return false;
    tc_fence_after();
    if (NT == 2 && w.ntok <= tt1) {
      // one row tile: the two softmax groups take the key tiles in turn
      for (int n = -2; n < m; ++n) {
        const int i = n & 1;
        if (n >= 0) {
          if (!take(vat) || !product(i, 0, vat, n > 1, n + 2 >= m)) return false;
          release(vat);
        }
        if (n + 2 < m) {
          if (n > -2 && !take(kat)) return false;
          tc_fence_after();
          scores(i, 0, 0, kat);
          release(kat);
        }
        if (n + 3 == m) umma_commit(bars + B::kQEmpty);
      }
    } else if constexpr (NT == 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (from[i] == 0 && to[i] > 0) scores(i, i, 0, kat);
      release(kat);
      if (m == 1) umma_commit(bars + B::kQEmpty);
      for (int n = 0; n < m; ++n) {
        const bool next = n + 1 < m;
        if (!take(vat) || (next && !take(kat))) return false;
        // per row tile: O += P V of this key tile, then S of the next over P
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (n >= from[i] && n < to[i] && !product(i, 0, vat, n > from[i], n + 1 == to[i])) return false;
          if (next && n + 1 >= from[i] && n + 1 < to[i]) scores(i, i, 0, kat);
        }
        release(vat);
        if (next) release(kat);
        if (n + 2 == m) umma_commit(bars + B::kQEmpty);
      }
    } else {
      scores(0, 0, w.g & 1, kat);
      release(kat);
      if (m == 1) umma_commit(bars + B::kQEmpty);
      for (int n = 0; n < m; ++n) {
        const uint32_t buf = (w.g + n) & 1;
        if (n + 1 < m) {
          if (!take(kat)) return false;
          tc_fence_after();
          scores(0, 0, buf ^ 1, kat);
          release(kat);
          if (n + 2 == m) umma_commit(bars + B::kQEmpty);
        }
        if (!take(vat) || !product(0, buf, vat, n > 0, false)) return false;
        release(vat);
      }
    }
    w.advance(a, c, m, NT * tt1, tt1);
  }
  return true;
}

template <int D, bool PACKED>
__device__ __forceinline__ void chunk_issue(const AttnArgs& a, const PagedArgs& c, ChunkWalk& w, int tt1, uint32_t tmem,
                                            uint32_t q_smem, uint32_t slot0, uint32_t bars, uint32_t abort_w) {
  bool issued = false;
  chunk_issue_all<D, PACKED>(a, c, w, tt1, tmem, q_smem, slot0, bars, abort_w, issued);
  if (issued) {
    // Everything issued is done before TMEM is given back and the CTA's shared
    // memory goes (bounded), also where a softmax warp gave up on the last
    // product. In a sound run the softmax's own end is later.
    umma_commit(bars + ChunkBars<D>::kDrained);
    mbar_wait(bars + ChunkBars<D>::kDrained, 0);
  }
}

template <int D, bool PACKED>
__global__ void __launch_bounds__(ChunkCfg<D>::kThreads, 1)
    attn_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const AttnArgs a, const PagedArgs c) {
  using C = ChunkCfg<D>;
  constexpr int NT = C::kNT, NS = C::kSlots, PARTS = C::kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* slots = smem + C::kQBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(slots + NS * C::kSlotBytes);
  using B = ChunkBars<D>;
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + B::kEmpty, q_full = full0 + B::kQFull,
                 q_empty = full0 + B::kQEmpty, s_full = full0 + B::kSFull, p_full = full0 + B::kPFull,
                 o_done = full0 + B::kODone, v_tmp = full0 + B::kVTmp;
  uint32_t* words = reinterpret_cast<uint32_t*>(bars + C::kBars);
  const uint32_t abort_w = smem_u32(words);
  uint32_t* tmem_holder = words + 1;
  static_assert(sizeof(ChunkWalk) <= C::kWalkInts * 4, "walks");
  auto& w = *reinterpret_cast<ChunkWalk*>(words + 4 + C::kWalkInts * warp_id());
  auto* ml = reinterpret_cast<float2*>(words + 4 + C::kWalkInts * (C::kThreads / 32));
  const uint32_t q_smem = smem_u32(smem), slot0 = smem_u32(slots);
  const int warp = warp_id(), lane = lane_id();
  constexpr int kMmaWarp = NT * 4, kLoadWarp = NT * 4 + 1;  // and kLoadWarp + 1

  if (threadIdx.x == 0) {
    st_shared_volatile_u32(abort_w, 0u);
    for (int s = 0; s < NS; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(v_tmp, 1);
    mbar_init(full0 + B::kDrained, 1);
    mbar_init(full0 + B::kMlFull, 4);
    mbar_init(full0 + B::kMlEmpty, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(o_done + 8 * i, 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(p_full + 8 * i, 4);
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_launch_dependents();  // this CTA holds its TMEM
  pdl_wait();
  const int tt1 = 128 / a.G, tt = NT * tt1;
  const AttnRun run = find_run(c.batch, c.heads, blockIdx.x, gridDim.x, C::kItemUnits,
                               [&](int b) { return chunk_heads(a, c, b, tt, tt1); });
  int block, unit;
  find_block(run, a, c, tt, tt1, block, unit);
  w.start(a, c, run, block, unit, tt, tt1);

  if (warp < kMmaWarp) {
    const int tile = warp >> 2;
    chunk_softmax<D>(a, c, w, tile, tt1, tmem, s_full + 8 * tile, p_full + 16 * tile, o_done + 8 * tile,
                     full0 + B::kMlFull, ml, abort_w, run.per);
  } else if (warp == kMmaWarp) {
    if (lane == 0) chunk_issue<D, PACKED>(a, c, w, tt1, tmem, q_smem, slot0, full0, abort_w);
  } else if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    // ------------------------------------------------------------- loads
    // One warp for queries and keys, one for values; they share the ring,
    // whose order both know, and each passes over the other's slots.
    const bool keys = warp == kLoadWarp;
    const CUtensorMap* map = keys ? &tmK : &tmV;
    const int rows = a.box_rows;
    constexpr int kColGroups = C::kKCols / 64, kAllGroups = D / 64;
    // a slot's boxes, one per lane: piece `piece` (rows keys), column group grp
    // (packed: all groups)
    const int all = keys ? kColGroups : kAllGroups, groups = PACKED ? 1 : all;
    const uint32_t box_bytes = static_cast<uint32_t>(rows) * (PACKED ? all * 128 : 128);
    const int pieces = (keys ? kChunkBN : C::kVKeys) / rows;  // per slot
    const int piece = lane / groups, grp = lane % groups;
    const uint32_t dst0 = slot0 + grp * (pieces * box_bytes) + piece * box_bytes;
    const bool has_box = lane < pieces * groups;
    const int drop = blockIdx.x == 0 ? a.drop : -1;
    int slot = 0, filled = 0;
    uint32_t phase = 0, q_count = 0;
    uint32_t armed = 0, armed_phase = 0;  // this warp's slots and the phases that its last loads fill
    bool ok = true;
    const auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait_ab(bar, parity, abort_w));
      return ok;
    };
    const auto pass = [&] {
      ++filled;
      if (++slot == NS) slot = 0, phase ^= 1;
    };
    // lane l: page and place in it of piece l of a tile; page < 0: not loaded
    const auto pages_of = [&](int tile) {
      const uint32_t tok = static_cast<uint32_t>(tile) * kChunkBN + lane * rows;
      int2 pg = make_int2(-2, 0);
      if (lane * rows < kChunkBN && tok < static_cast<uint32_t>(w.len) &&
          tok + rows > static_cast<uint32_t>(w.lo_seq)) {
        const uint32_t i = tok / static_cast<uint32_t>(c.page_size);
        pg.x = c.table[static_cast<int64_t>(w.b) * c.max_pages + i];
        pg.y = tok - i * c.page_size;
        if (pg.x < 0 || pg.x >= c.num_pages) {
          report(FP8_DEV_BAD_INDEX);
          pg.x = -1;
        }
      }
      return pg;
    };
    uint32_t v_par = 0;
    bool v_tmp_armed = false;
    const auto load = [&](const int2& pg, int key0) {
      // Value rows that are not keys of the sequence's new tokens hold anything
      // (or are not loaded): zeros, which the zero probabilities leave alone.
      // Such a tile comes in on a barrier of the loader's own, is cleared, and
      // then handed on.
      const int lo = w.lo_seq - key0, hi = w.len - key0;  // rows [lo, hi) count
      const bool edge = !keys && (lo > 0 || hi < kChunkBN);
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        // key slots split the columns, value slots the keys
        const int from = (keys ? 0 : p * pieces) + piece;
        const int page = __shfl_sync(0xFFFFFFFFu, pg.x, from & 31);
        const int token = __shfl_sync(0xFFFFFFFFu, pg.y, from & 31);
        const bool mine = has_box && page >= 0;
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, mine)) * box_bytes;
        if (filled >= NS && !wait(empty0 + 8 * slot, phase ^ 1)) return;
        if (filled == drop) {
          pass();
          continue;
        }
        const uint32_t bar = edge ? v_tmp : full0 + 8 * slot;
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (mine)
          tma_load_page_cols(dst0 + slot * C::kSlotBytes, map, bar, token, (keys ? p * kColGroups : 0) + grp, w.h,
                             page);
        if (edge) {
          v_tmp_armed = true;
          if (!wait(v_tmp, v_par)) return;
          v_tmp_armed = false;
          v_par ^= 1;
          for (int r = 0; r < C::kVKeys; ++r) {
            const int key = p * C::kVKeys + r;
            if ((key < lo || key >= hi) && lane < D / 8)
              *reinterpret_cast<uint4*>(slots + slot * C::kSlotBytes + (lane & 7) * 16 +
                                        (PACKED ? (r >> 3) * (D * 16) + (lane >> 3) * 1024 + (r & 7) * 128
                                                : (lane >> 3) * (C::kVKeys * 128) + r * 128)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(full0 + 8 * slot);
        } else {
          armed |= 1u << slot;
          armed_phase = (armed_phase & ~(1u << slot)) | (phase << slot);
        }
        pass();
      }
    };
    const auto skip = [&] {
#pragma unroll
      for (int p = 0; p < PARTS; ++p) pass();
    };
    while (w.left > 0 && ok) {
      const int m = w.seg(tt1);
      const int tile = w.tile0 + w.t;
      int2 pg;
      if (keys) {
        if (q_count > 0) {  // the first keys come in under the last segment's end; the first queries come first
          load(pages_of(tile), 0);
          wait(q_empty, (q_count - 1) & 1);
        }
        if (ok) {
          ++q_count;
          const int nq = w.tile_tokens(1, tt1) > 0 && NT == 2 ? 2 : 1;
          if (lane == 0)
            mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(nq) * kAllGroups * tt1 * a.G * 128);
          __syncwarp();
          if (lane < nq * kAllGroups) {
            const int i = lane / kAllGroups, qg = lane % kAllGroups;
            tma_load_q(q_smem + i * (128 * D * 2) + qg * 16384, &tmQ, q_full, w.h * a.G,
                       w.q0 + w.tok0 + i * tt1, qg);
          }
          if (q_count == 1) load(pages_of(tile), 0);
        }
        // order: K0 V0 K1 V1 ..., with one row tile K0 K1 V0 K2 V1 ...
        const bool ahead = NT == 1 || w.ntok <= tt1;
        int2 pg_next = m > 1 ? pages_of(tile + 1) : make_int2(-2, 0);
        for (int n = 0; n < m && ok; ++n) {
          pg = pg_next;
          if (n + 2 < m) pg_next = pages_of(tile + n + 2);
          if (!ahead) skip();
          if (n + 1 < m) load(pg, 0);
          if (ahead) skip();
        }
      } else {
        const bool ahead = NT == 1 || w.ntok <= tt1;
        pg = pages_of(tile);
        skip();
        for (int n = 0; n < m && ok; ++n) {
          const int2 pg_next = n + 1 < m ? pages_of(tile + n + 1) : make_int2(-2, 0);
          if (ahead && n + 1 < m) skip();
          load(pg, (tile + n) * kChunkBN);
          if (!ahead && n + 1 < m) skip();
          pg = pg_next;
        }
      }
      w.next(a, c, m, tt, tt1);
    }
    // Every copy started is waited for (bounded) before the CTA can exit. The
    // ring's last slots are given back when the products have read them (both
    // warps end with the same count, so no later load moves their barriers
    // on); if a consumer gives up before, the copies themselves are waited for.
    for (int i = max(0, filled - NS); i < filled; ++i) wait(empty0 + 8 * (i % NS), (i / NS) & 1);
    if (!ok && lane == 0) {
      for (int i = 0; i < NS; ++i)
        if (armed >> i & 1) mbar_wait(full0 + 8 * i, armed_phase >> i & 1);
      if (q_count > 0) mbar_wait(q_full, (q_count - 1) & 1);
      if (v_tmp_armed) mbar_wait(v_tmp, v_par);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace fp8k
