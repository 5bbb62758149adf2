// attn.cuh - attention of a ragged batch's new tokens over a paged cache.
//
//   s_j = scale q . k_j  for the keys j <= p (and j > p - window),
//   o = sum_j softmax(s)_j v_j,  lse = ln sum_j exp(s_j),
// p the position of the new token, kv_len - q_len + its place among the new
// tokens. One pass over the keys with the running maximum and sum of the
// softmax, in base 2 (the scale times log2 e is folded into the exponent's
// argument); scores, statistics and o in fp32; the probabilities go to bf16
// for their product with v (|p| <= 1 relative to the row's maximum, so each
// is off by 2^-8 of itself at most), o is rounded once to bf16.
//
// Work. The query heads that share a key/value head are taken together: row
// r of an item is new token r / G, head r % G of the group, so keys and
// values are read once for the group. The items' key tiles, laid end to end
// (sequence, head, tile), are cut into equal runs, one per CTA: a ragged
// batch, a single long context and a full batch all load the device evenly.
// An item cut between CTAs leaves an unnormalised o with its maximum and sum
// for each part in the workspace, and attn_join_kernel adds the parts in
// order. The cut depends on the lengths and the grid alone, so results are
// bit-reproducible. Every CTA finds its run by itself from the lengths (a
// scan over the batch), so a captured graph follows lengths that change.
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
  s.lo = static_cast<int>(max(0ll, static_cast<long long>(s.len) - s.ql - a.window + 1));
  s.tile0 = s.lo / BN;
  s.tiles = s.ql == 0 ? 0 : max(1, (s.len + BN - 1) / BN - s.tile0);
  return s;
}

// A CTA's run: `units` key tiles from tile `tile` of the item (seq, sub) on
// (sub numbers a sequence's items); `per` is the length of a full run.
struct AttnRun {
  int seq;
  int units;
  int per;
  long long sub_off;  // units of the sequence before the run
};

template <int THREADS>
struct PlanSmem {
  long long wsum[THREADS / 32];
  AttnRun run;
};

// Finds CTA `cta`'s run of `ctas`; every thread of the block calls it. The
// weight of a sequence is weight(b) units.
template <int THREADS, typename Weight>
__device__ __forceinline__ AttnRun find_run(PlanSmem<THREADS>& sm, int batch, int cta, int ctas,
                                            Weight weight) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  // all units, and this thread's first weight (the only one when batch <= THREADS)
  long long first = tid < batch ? weight(tid) : 0, sum = first;
  for (int b = tid + THREADS; b < batch; b += THREADS) sum += weight(b);
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if (lane == 0) sm.wsum[w] = sum;
  if (tid == 0) sm.run.units = 0;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) total += sm.wsum[i];
  const long long per = max(1ll, (total + ctas - 1) / ctas);
  const long long start = per * cta;
  if (start < total) {  // block-uniform
    long long base = 0;
    for (int b0 = 0; b0 < batch && base <= start; b0 += THREADS) {
      const int b = b0 + tid;
      const long long mine = b0 == 0 ? first : b < batch ? weight(b) : 0;
      long long incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += v;
      }
      __syncthreads();  // wsum is free
      if (lane == 31) sm.wsum[w] = incl;
      __syncthreads();
      long long before = base, all = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        before += i < w ? sm.wsum[i] : 0;
        all += sm.wsum[i];
      }
      const long long hi = before + incl, lo = hi - mine;
      if (lo <= start && start < hi) {
        sm.run.seq = b;
        sm.run.sub_off = start - lo;
        sm.run.units = static_cast<int>(min(per, total - start));
      }
      base += all;
    }
  }
  __syncthreads();
  AttnRun r = sm.run;
  r.per = static_cast<int>(per);
  return r;
}

// Base-2 exponential, flushing to zero (2 ulp).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLn2 = 0.69314718055994531f;

// ------------------------------------------------------------------ join
// The parts of one cut item, in order: the first in slot `slot`, then slot
// 2 (cta + i) of the `more` following CTAs. Rows of the item: token t0 + r /
// G, head h0 + r % G.
__device__ __forceinline__ int4 join_desc(int more, int slot, int t0, int h0, int rows) {
  return make_int4(more | (rows << 16), slot, t0, h0);
}

// One block per (CTA that holds an item's first part, row group): a row by
// WPR warps, each adding the parts w, w + WPR, ..., joined in warp order.
template <int D, int ROWS, int WPR>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs a) {
  constexpr int E = D / 32;  // values per lane
  constexpr int RPB = 8 / WPR;
  __shared__ float so[WPR > 1 ? 8 : 1][D];
  pdl_launch_dependents();
  pdl_wait();
  const int4 d = a.part_desc[blockIdx.x];
  const int more = d.x & 0xFFFF, rows = d.x >> 16;
  if (more == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * RPB + warp / WPR, w = warp % WPR;
  if (WPR == 1 ? r >= rows : blockIdx.y * RPB >= rows) return;
  auto slot = [&](int i) { return i == 0 ? d.y : 2 * (static_cast<int>(blockIdx.x) + i); };
  const bool live = r < rows;
  // every part's maximum and sum, by all lanes (each warp of the row alike)
  float m = -INFINITY;
  for (int i = lane; live && i <= more; i += 32)
    m = fmaxf(m, a.part_ml[static_cast<int64_t>(slot(i)) * ROWS + r].x);
#pragma unroll
  for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
  const float mb = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int i0 = 0; live && i0 <= more; i0 += 32) {
    float f_l = 0.0f;
    if (i0 + lane <= more) {
      const float2 ml = a.part_ml[static_cast<int64_t>(slot(i0 + lane)) * ROWS + r];
      f_l = ex2(ml.x - mb);
      l += f_l * ml.y;
    }
    const int n = min(32, more + 1 - i0);
    const int first = (w - i0 % WPR + WPR) % WPR;
#pragma unroll 4
    for (int i = first; i < n; i += WPR) {
      const float f = __shfl_sync(0xFFFFFFFFu, f_l, i);
      const float* p = a.part_o + (static_cast<int64_t>(slot(i0 + i)) * ROWS + r) * D + lane * (E < 4 ? E : 4);
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
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (w != 0 || !live) return;
    for (int i = 1; i < WPR; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += so[warp + i][lane * E + e];
  }
  const int t = d.z + r / a.G, h = d.w + r % a.G;
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
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
    a.lse[static_cast<int64_t>(t) * a.Hq + h] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
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
// memory at an item's end.
constexpr int kRowsBN = 64;
constexpr int kRowsMax = 16;
constexpr int kRowsThreads = 160;

template <int D, int SLOTS>
struct RowsCfg {
  static constexpr int kSlotBytes = kRowsBN * D * 2;
  static constexpr int kXStride = 40;  // floats per row of the exchange: 32 columns, conflict-free
  static constexpr int kXBytes = 4 * kRowsMax * kXStride * 4;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(SLOTS) * kSlotBytes + kXBytes +
                                  2 * 4 * kRowsMax * 4 + 16 * SLOTS + 16 + sizeof(PlanSmem<kRowsThreads>);
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
      h = static_cast<int>(r.sub_off / s.tiles);
      t = static_cast<int>(r.sub_off % s.tiles);
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
  auto* plan = reinterpret_cast<PlanSmem<kRowsThreads>*>(abort_p + 4);
  const uint32_t slot0 = smem_u32(smem), full0 = smem_u32(bars), empty0 = smem_u32(bars + SLOTS);
  const uint32_t abort_w = smem_u32(abort_p);
  const int warp = warp_id(), lane = lane_id();
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
  pdl_launch_dependents();
  pdl_wait();
  const int cta = blockIdx.x;
  const AttnRun run = find_run<kRowsThreads>(*plan, c.batch, cta, gridDim.x, [&](int b) -> long long {
    const SeqSpan s = seq_span(a, c, b, kRowsBN);
    if (!s.ok && cta == 0) report(FP8_DEV_BAD_INDEX);
    return static_cast<long long>(s.tiles) * c.heads;
  });
  RowsWalk w(a, c, run);

  if (warp == 4) {
    // ---------------------------------------------------------- producer
    const uint64_t policy = l2_policy_evict_first();
    const int rows = a.box_rows, boxes = kRowsBN / rows;
    const uint32_t box_bytes = static_cast<uint32_t>(rows) * D * 2;
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
          if (lane == 0) mbar_arrive_expect_tx(full0 + 8 * slot, bytes);
          __syncwarp();
          if (mine)
            tma_load_page(slot0 + slot * C::kSlotBytes + lane * box_bytes, kv ? &tmV : &tmK,
                          full0 + 8 * slot, in_page, w.h, pg, policy);
          ++filled;
          if (++slot == SLOTS) slot = 0, phase ^= 1;
        }
      }
      w.next(a, c, n);
    }
    if (!ok && lane == 0) {
      // every copy started is waited for (bounded) before the CTA can exit
      for (int i = max(0, filled - SLOTS); i < filled; ++i)
        mbar_wait(full0 + 8 * (i % SLOTS), (i / SLOTS) & 1);
    }
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
    const float inv = jl > 0.0f ? 1.0f / jl : 0.0f;
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
        a.lse[static_cast<int64_t>(tok) * a.Hq + head] = jl > 0.0f ? (jm + log2f(jl)) * kLn2 : -INFINITY;
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
    q[e] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.ldq + h * D + lane * E + e]) << 16) * a.scale_log2;
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
    const float f = exp2f(m - mn), pr = exp2f(s - mn);
    l = l * f + pr;
    m = mn;
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + pr * __uint_as_float(static_cast<uint32_t>(c.v[at + e]) << 16);
  }
  for (int e = 0; e < E; ++e)
    a.o[t * a.ldo + h * D + lane * E + e] = f32_to_bf16_rn(l > 0.0f ? o[e] / l : 0.0f);
  if (a.lse && lane == 0) a.lse[static_cast<int64_t>(t) * a.Hq + h] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace fp8k
