// Attention of drafted rows over a cache and over each other (rf_tree_attention).
//
// out = sum_j w_j v_j / sum_j w_j, w_j = exp(scale q.k_j - m): one pass over the keys with
// a running maximum m and sum per query row. The G query heads of a KV head share its
// keys, so the rows of an item are (node, head) pairs, node-major, up to 128 to a tile
// (one TMEM lane each).
//
// Bound: with R rows to a KV head a key costs 4 R hd flops against 4 hd bytes, so below
// about R = 275 (the ratio of the measured rates) the cache's bytes are the floor, above
// it the two matrix products.
//
// Work split. The 128-key tiles of all items (sequence, KV head, row tiles) are laid end to
// end and cut into equal shares, one per CTA and one CTA per SM, whatever the lengths are
// (they are known on the device only). An item weighs four tiles more than it has: its
// queries, first scores and epilogue take about that long, and a share of many short items
// would finish last (16 trees over 913 to 16,384 rows: 156 us without, 134 with). The rows
// of an item that was cut leave unnormalised sums, maxima and totals in the workspace, and
// k_attn_combine joins them in the order of the cuts.
//
// Two streams per CTA, each with its own score tile S_s and accumulator O_s in TMEM and
// its own four softmax warps, so that one stream's matrix products run while the other's
// weights are formed:
//   up to 128 rows   one row tile; the streams take alternate key tiles, and their
//                    accumulators are joined when a segment ends;
//   more rows        two row tiles; every key tile serves both.
//
//   warps 0-3, 4-7   softmax of stream 0 / 1: a thread is a row. S_s -> weights in bf16,
//                    written back over S_s as the A operand of the second product. The
//                    accumulator is rescaled only when the maximum has grown by more than
//                    a factor 2^8 (weights stay below 2^8 of the reference, which fp32
//                    sums and bf16 weights hold without loss), so rarely after the first
//                    tiles.
//   warp 8           TMA: query tiles, then K and V tiles through one ring
//   warp 9           MMA: S_s = Q K^T, O_s += P_s V (P_s from TMEM); with two row tiles warp 10
//                    issues the second one's, in turns with it. It also clears what
//                    the second product must not see: V rows beyond a sequence's length
//                    (any bits; their weights are 0, but 0 x NaN is NaN), and elements of
//                    drafted V rows that are not finite. Rows that do see such an element
//                    get it in the epilogue.
//   warp 11          fills the third warpgroup, which gives registers to the first two
//
// Measured (128 channels): one token, 40 query heads on 8, over 32,767 rows: 33 us, 4.1 TB/s of
// the cache's bytes (22 us of it in the tiles). 16 trees of 64 nodes, 32 heads on 8, over 913 to
// 16,384 rows: 138 us, 4.5 TB/s and 1,100 TFLOP/s. 4,096 rows in order over 28,672, 40 heads on
// 8: 2.03 ms in long runs, at the power limit (1,270 TFLOP/s, 0.68 of the measured burst rate and
// 0.75 of the sustained), 1.84 ms from rest. 64 channels: 22 us, 105 us and 1.55 ms; the bytes
// and products are half, the exponentials (32 a clock and SM: 0.54 ms of the last) the same.
// A stream's turn at the tensor
// cores, for 16 products that take 1,030 cycles back to back, lasts about 1,400: the wait between
// the two parts of the weights, the issue beside eight busy warps, and the hand-over to the other
// stream. A shorter softmax does not change that (weights formed against the last maximum while
// the tile's own is taken: 1.87 ms), nor do sums behind the hand-over (1.89 ms) or streams
// without turns (2.33 ms).
#include <algorithm>
#include <cmath>

#include "rf_device.cuh"
#include "rf_host.h"

namespace rf {

constexpr int kAtTile = 128;      // keys of a tile, rows of a row tile
constexpr int kAtThreads = 384;
// Registers a thread: 168 at the launch, then 208 for the softmax warps, which hold a row's 128
// scores and 64 packed weights, and 88 for the others: 256 x 208 + 128 x 88 = 384 x 168.
constexpr int kAtRegsSoftmax = 208, kAtRegsOther = 88;
static_assert(256 * kAtRegsSoftmax + 128 * kAtRegsOther <= kAtThreads * 168, "more registers than the launch has");
constexpr int kAtFirst = 96;      // keys of the first part in which a tile's weights are handed over
constexpr int kAtItemCost = 4;    // tiles that an item weighs beyond its own
constexpr int kAtMaxCtas = 160;   // bounds the workspace
constexpr int kAtMaxStages = 8;
constexpr float kAtLog2e = 1.4426950408889634f;
constexpr float kAtRescale = 8.0f;  // log2 of the growth of the maximum that is let pass

// The first tiles of a CTA's share, for k_attn_combine.
struct AttnPlan {
  long long item;  // linear index, -1: no tiles
  int b, h, mt, t0;
};
// Where a share starts: `at` in the weight of item (b, h, mt), whose tiles come behind
// kAtItemCost of it.
struct AttnShare {
  long long weight;  // of the share
  int b, h, mt, at;
  int len, n_tiles;  // rows in use of sequence b, tiles of the item
};

struct AttnArgs {
  CUtensorMap tm_q, tm_k, tm_v, tm_kd, tm_vd;
  const int32_t* lens;
  const unsigned long long* mask;
  const __nv_bfloat16* v_draft;
  __nv_bfloat16* out;
  float* lse;
  float4* part_o;    // [2 * ctas][head_dim / 4][rows of an item]
  float2* part_ml;   // [2 * ctas][rows of an item]
  AttnPlan* plan;    // [ctas]
  int32_t* dev_status;
  uint64_t timeout_ns;
  long long out_row, out_seq, draft_row, draft_seq;
  int n_seqs, heads, group, n, capacity, words;
  int npt;        // nodes of a row tile
  int m_items;    // items (groups of row tiles) of a sequence and head
  int draft_sum;  // draft tiles summed over those items
  float scale;
};

struct AttnShared {
  uint64_t full[kAtMaxStages], empty[kAtMaxStages];
  uint64_t q_full, q_empty, s_full[2], p_full[2][2], o_final, o_empty, ml_full, turn[2], v_clean[2], mma_done[2];
  AttnShare share;
  int bad[2];                // a drafted V row of the segment is not finite
  uint32_t tmem;
  int abort;
};

// With one row tile the streams exchange maxima and totals: [segment parity][stream][row].
using AttnExchange = float2[2][2][kAtTile];

template <int kHD, bool kDual>
struct AttnCfg {
  static constexpr int kTileBytes = kAtTile * kHD * 2;
  static constexpr int kQBytes = (kDual ? 2 : 1) * kTileBytes;
  static constexpr int kStages = kHD == 128 ? 5 : 8;
  static constexpr size_t kSmem =
      1024 + kQBytes + static_cast<size_t>(kStages) * kTileBytes + sizeof(AttnShared) + (kDual ? 0 : sizeof(AttnExchange));
  static constexpr int kRows = (kDual ? 2 : 1) * kAtTile;  // of an item
};

// Cache and draft tiles of one item.
struct ItemShape {
  int len, cached, tiles;  // rows in use, cache tiles, all tiles
};
template <bool kDual>
__device__ __forceinline__ int draft_tiles(const AttnArgs& a, int mt) {
  const int seen = a.mask != nullptr ? a.n : min(a.n, (mt + 1) * a.npt * (kDual ? 2 : 1));
  return (seen + kAtTile - 1) / kAtTile;
}
__device__ __forceinline__ int length_of(const AttnArgs& a, int b) {  // -1: out of range
  const int len = a.lens[b];
  return len < 0 || len > a.capacity ? -1 : len;
}
template <bool kDual>
__device__ __forceinline__ ItemShape item_shape(const AttnArgs& a, int b, int mt) {
  ItemShape s;
  s.len = length_of(a, b);
  s.cached = (max(s.len, 0) + kAtTile - 1) / kAtTile;
  s.tiles = s.len < 0 ? 0 : s.cached + draft_tiles<kDual>(a, mt);
  return s;
}

// A CTA's share, segment by segment; every role walks it alike, a converged warp at a time.
template <bool kDual>
struct Walk {
  int b, h, mt, t0, t1;  // an item and the tiles of it that are the share's
  int at;                // where the share stands in the item's weight
  long long left;        // weight
  ItemShape shape;
  __device__ __forceinline__ Walk(const AttnArgs& a, const AttnShared* sh) {
    b = uniform(sh->share.b);
    h = uniform(sh->share.h);
    mt = uniform(sh->share.mt);
    at = uniform(sh->share.at);
    left = uniform(sh->share.weight);
    shape.len = uniform(sh->share.len);
    shape.cached = (shape.len + kAtTile - 1) / kAtTile;
    shape.tiles = uniform(sh->share.n_tiles);
    t0 = t1 = 0;
    if (left > 0) settle(a);
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ int end() const {
    return static_cast<int>(min(static_cast<long long>(shape.tiles + kAtItemCost), at + left));
  }
  // The first tiles from here on (a share may end within an item's extra weight).
  __device__ __forceinline__ void settle(const AttnArgs& a) {
    while (true) {
      t0 = max(at - kAtItemCost, 0);
      t1 = max(end() - kAtItemCost, 0);
      if (t1 > t0) return;
      next_item(a);
      if (left <= 0) return;
    }
  }
  __device__ __forceinline__ void next(const AttnArgs& a) {
    next_item(a);
    if (left > 0) settle(a);
  }
  __device__ __forceinline__ void next_item(const AttnArgs& a) {
    left -= end() - at;
    if (left <= 0) return;
    at = 0;
    do {
      if (++mt == a.m_items) {
        mt = 0;
        if (++h == a.heads) {
          h = 0;
          if (++b >= a.n_seqs) {  // lengths that changed under the kernel: no sequence is left
            left = 0;
            return;
          }
        }
      }
      shape = item_shape<kDual>(a, b, mt);
      shape.len = uniform(shape.len);
      shape.cached = uniform(shape.cached);
      shape.tiles = uniform(shape.tiles);
    } while (shape.tiles == 0);
  }
};

// The start of share `cta` of `ctas`: one warp sums the sequences' weights, then finds the
// sequence, head, item and place of its first one. Writes the share to shared memory, and
// to `plan` what k_attn_combine needs.
template <bool kDual>
__device__ void find_share(const AttnArgs& a, AttnShared* sh, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  auto weight_of = [&](int len) -> long long {
    return len < 0 ? 0ll
                   : static_cast<long long>(a.heads) *
                         (static_cast<long long>(a.m_items) * ((len + kAtTile - 1) / kAtTile + kAtItemCost) + a.draft_sum);
  };
  long long total = 0;
  int len = -1;  // of sequence `lane`, then of later ones
  for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
    len = b0 + lane < a.n_seqs ? length_of(a, b0 + lane) : -1;
    if (len < 0 && b0 + lane < a.n_seqs) record_status(a.dev_status, RF_ERR_INVALID_ARG);
    total += weight_of(len);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const long long shares = min(static_cast<long long>(ctas), total);
  AttnShare p{};
  if (cta < shares) {
    const long long first = share_start(total, cta, static_cast<int>(shares));
    p.weight = share_start(total, cta + 1, static_cast<int>(shares)) - first;
    long long base = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
      if (a.n_seqs > 32) len = b0 + lane < a.n_seqs ? length_of(a, b0 + lane) : -1;
      const long long own = weight_of(len);
      long long x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, first < base + x);
      if (hit) {
        const int at = __ffs(hit) - 1;
        p.b = b0 + at;
        p.len = __shfl_sync(0xffffffffu, len, at);
        const int cached = (p.len + kAtTile - 1) / kAtTile;
        long long r = first - base - __shfl_sync(0xffffffffu, x - own, at);
        const long long per_head = quick_div(__shfl_sync(0xffffffffu, own, at), a.heads);
        p.h = static_cast<int>(quick_div(r, per_head));
        r -= p.h * per_head;
        p.mt = 0;
        p.n_tiles = cached + draft_tiles<kDual>(a, 0);
        if (a.mask != nullptr) {
          p.mt = static_cast<int>(quick_div(r, p.n_tiles + kAtItemCost));
          r -= static_cast<long long>(p.mt) * (p.n_tiles + kAtItemCost);
        } else {
          while (r >= p.n_tiles + kAtItemCost) {
            r -= p.n_tiles + kAtItemCost;
            p.n_tiles = cached + draft_tiles<kDual>(a, ++p.mt);
          }
        }
        p.at = static_cast<int>(r);
        break;
      }
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  if (lane == 0) sh->share = p;
  __syncwarp();
  const Walk<kDual> w(a, sh);
  if (lane == 0)
    a.plan[cta] = AttnPlan{w.more() ? (static_cast<long long>(w.b) * a.heads + w.h) * a.m_items + w.mt : -1ll, w.b, w.h, w.mt, w.t0};
}

// A row's 128 scores, from `ts`, and their maximum; keys that are not seen (kMasked) become
// -inf. The second half is on its way while the first half's maximum is taken.
template <bool kMasked>
__device__ __forceinline__ float row_scores(uint32_t ts, const uint32_t (&keep)[4], uint32_t (&r)[4][32]) {
  float m[4];
  auto take = [&](int c) {
    if (kMasked) {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[c][i] = (keep[c] >> i) & 1u ? r[c][i] : 0xff800000u;
    }
    m[c] = fmaxf(u2f(r[c][0]), u2f(r[c][1]));
#pragma unroll
    for (int i = 2; i < 32; i += 2) m[c] = fmaxf(fmaxf(m[c], u2f(r[c][i])), u2f(r[c][i + 1]));
  };
  tmem_ld32(ts, r[0]);
  tmem_ld32(ts + 32, r[1]);
  tmem_wait_ld32(r[0]);
  tmem_wait_ld32(r[1]);
  tmem_ld32(ts + 64, r[2]);
  tmem_ld32(ts + 96, r[3]);
  take(0);
  take(1);
  tmem_wait_ld32(r[2]);
  tmem_wait_ld32(r[3]);
  take(2);
  take(3);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// The weights 2^(s sc + off) of 32-key groups c0 .. c1 - 1, written over the scores in bf16;
// adds to their sums.
__device__ __forceinline__ void row_weights(uint32_t ts, uint32_t (&r)[4][32], int c0, int c1, float sc, float off,
                                            float2& t0, float2& t1) {
  const float2 sc2 = make_float2(sc, sc), off2 = make_float2(off, off);
#pragma unroll
  for (int c = c0; c < c1; ++c) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      float2 x = fma_x2(make_float2(u2f(r[c][i]), u2f(r[c][i + 1])), sc2, off2);
      float2 y = fma_x2(make_float2(u2f(r[c][i + 2]), u2f(r[c][i + 3])), sc2, off2);
      x = make_float2(exp2f_ftz(x.x), exp2f_ftz(x.y));
      y = make_float2(exp2f_ftz(y.x), exp2f_ftz(y.y));
      t0 = add_x2(t0, x);
      t1 = add_x2(t1, y);
      w[i / 2] = pack_bf16x2(x.x, x.y);
      w[i / 2 + 1] = pack_bf16x2(y.x, y.y);
    }
    tmem_st16(ts + c * 16, w);
  }
  tmem_wait_st();
}

// Bits of the keys of tile `t` that query node `node` sees.
__device__ __forceinline__ void visible(const AttnArgs& a, const ItemShape& s, int b, int node, int t, uint32_t (&keep)[4]) {
  int limit;  // keys of the tile that exist for this row
  if (t < s.cached) {
    limit = s.len - t * kAtTile;
  } else {
    const int j0 = (t - s.cached) * kAtTile;
    limit = (a.mask != nullptr ? a.n : min(a.n, node + 1)) - j0;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int k = limit - c * 32;
    keep[c] = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
  }
  if (t >= s.cached && a.mask != nullptr) {
    const int w0 = (t - s.cached) * 2;
    const unsigned long long* words = a.mask + (static_cast<long long>(b) * a.n + node) * a.words;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const unsigned long long m = w0 + c < a.words ? words[w0 + c] : 0ull;
      keep[2 * c] &= static_cast<uint32_t>(m);
      keep[2 * c + 1] &= static_cast<uint32_t>(m >> 32);
    }
  }
}

template <int kHD, bool kDual>
__global__ void __launch_bounds__(kAtThreads, 1) k_attn(const __grid_constant__ AttnArgs a) {
  using Cfg = AttnCfg<kHD, kDual>;
  constexpr int kChunks = kHD / 64;                 // 64-channel slabs of a tile, 16 KB each
  constexpr int kSlab = kAtTile * 128;
  constexpr int kMmaWarps = kDual ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  AttnShared* sh = reinterpret_cast<AttnShared*>(smem + Cfg::kQBytes + Cfg::kStages * Cfg::kTileBytes);
  AttnExchange& ml = *reinterpret_cast<AttnExchange*>(sh + 1);  // (one row tile)
  const uint32_t s_q = smem_u32(smem), s_ring = s_q + Cfg::kQBytes;
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh->abort;
  const uint64_t timeout = a.timeout_ns;

  pdl_launch_dependents();  // the next kernel's CTAs may take their places as this one's leave
  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg::kStages; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], kMmaWarps);
    }
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, kMmaWarps);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh->s_full[s], 1);
      for (int i = 0; i < 2; ++i) mbar_init(&sh->p_full[s][i], 4);
    }
    mbar_init(&sh->o_final, kMmaWarps + 1);
    mbar_init(&sh->o_empty, 8);
    mbar_init(&sh->ml_full, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->v_clean[i], 1);
      mbar_init(&sh->turn[i], 1);
      mbar_init(&sh->mma_done[i], 1);
    }
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
    tma_prefetch_desc(&a.tm_kd);
    tma_prefetch_desc(&a.tm_vd);
  }
  if (warp == 9) {
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  // All above is this kernel's own; from here on it reads what earlier ones wrote, and writes.
  pdl_wait();
  if (warp == 0) find_share<kDual>(a, sh, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sh->tmem);

  if (warp == 8) {
    regs_dec<kAtRegsOther>();
    {  // the whole warp waits, one lane issues: a lane's wait by itself takes twice as long
      const auto wait = [&](uint64_t* bar, uint32_t par) { return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, timeout)) != 0; };
      int stage = 0;
      uint32_t phase = 0, q_phase = 0;
      long long issued = 0;
      bool ok = true, q_inflight = false;
      auto load = [&](const Walk<kDual>& w, int t, bool v) {
        if (!wait(&sh->empty[stage], phase ^ 1u)) return false;
        const bool draft = t >= w.shape.cached;
        const CUtensorMap* tm = draft ? (v ? &a.tm_vd : &a.tm_kd) : (v ? &a.tm_v : &a.tm_k);
        const int row = (draft ? t - w.shape.cached : t) * kAtTile;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh->full[stage], Cfg::kTileBytes);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            tma_load_4d(s_ring + stage * Cfg::kTileBytes + c * kSlab, tm, smem_u32(&sh->full[stage]), c * 64, w.h, row, w.b);
        }
        __syncwarp();
        ++issued;
        if (++stage == Cfg::kStages) {
          stage = 0;
          phase ^= 1u;
        }
        return true;
      };
      for (Walk<kDual> w(a, sh); w.more() && ok; w.next(a)) {
        if (!wait(&sh->q_empty, q_phase ^ 1u)) break;
        q_inflight = true;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh->q_full, (kDual ? 2 : 1) * kChunks * 64 * 2 * a.group * a.npt);
          for (int s = 0; s < (kDual ? 2 : 1); ++s)
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              tma_load_4d(s_q + s * Cfg::kTileBytes + c * kSlab, &a.tm_q, smem_u32(&sh->q_full), c * 64, w.h * a.group,
                          (w.mt * (kDual ? 2 : 1) + s) * a.npt, w.b);
        }
        __syncwarp();
        q_phase ^= 1u;
        // the order in which warp 9 takes them
        if (kDual) {
          for (int t = w.t0; t < w.t1 && ok; ++t) ok = load(w, t, false) && load(w, t, true);
        } else {
          ok = load(w, w.t0, false);
          for (int t = w.t0 + 1; t < w.t1 && ok; ++t) ok = load(w, t, false) && load(w, t - 1, true);
          ok = ok && load(w, w.t1 - 1, true);
        }
      }
      // Drain: every issued copy lands before the CTA may exit.
      int dummy = 0;
      if (q_inflight) mbar_wait(&sh->q_full, q_phase ^ 1u, &dummy, timeout);
      for (long long i = (issued > Cfg::kStages ? issued - Cfg::kStages : 0); i < issued; ++i)
        mbar_wait(&sh->full[i % Cfg::kStages], static_cast<uint32_t>((i / Cfg::kStages) & 1), &dummy, timeout);
    }
  } else if (warp == 9 || (kDual && warp == 10)) {
    regs_dec<kAtRegsOther>();
    constexpr uint32_t idesc_s = make_idesc_bf16(kAtTile, kAtTile, 0, 0);
    constexpr uint32_t idesc_o = make_idesc_bf16(kAtTile, kHD, 0, 1);
    const uint32_t issue = lane == 0;
    int stage = 0;
    uint32_t phase = 0, q_phase = 0, o_phase = 0, cleaned = 0, turn_phase = warp == 9 ? 1 : 0, p_phase[2] = {0, 0};
    int seg = 0;
    auto advance = [&] {
      if (++stage == Cfg::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    auto wait = [&](uint64_t* bar, uint32_t par) {  // whole warp
      const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, timeout));
      if (ok) tc_fence_after();
      return ok;
    };
    // Products are issued back to back behind all of their waits: the pipe takes one as the
    // last ends, so whatever stands between two of them is lost time.
    auto qk = [&](int s, int q, int k_stage) {  // S_s = Q_q K^T
      const uint32_t k0 = s_ring + k_stage * Cfg::kTileBytes, q0 = s_q + q * Cfg::kTileBytes;
#pragma unroll
      for (int k = 0; k < kHD / 16; ++k) {
        const uint32_t off = (k / 4) * kSlab + (k % 4) * 32;
        tc_mma_bf16_warp(tmem + s * kAtTile, make_sdesc_sw128(q0 + off, 16, 1024), make_sdesc_sw128(k0 + off, 16, 1024),
                         idesc_s, k > 0 ? 1u : 0u, issue);
      }
    };
    // O_s (+)= P_s V, the first part of whose weights is there; the second comes while the
    // first's products run.
    auto pv = [&](int s, int v_stage, bool fresh) {
      const uint32_t v0 = s_ring + v_stage * Cfg::kTileBytes;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (part == 1 && !wait(&sh->p_full[s][1], p_phase[s])) return false;
#pragma unroll
        for (int k = part * kAtFirst / 16; k < (part == 0 ? kAtFirst : kAtTile) / 16; ++k)
          tc_mma_bf16_ts_warp(tmem + 256 + s * 128, tmem + s * kAtTile + k * 8,
                              make_sdesc_sw128(v0 + k * 2048, kSlab, 1024), idesc_o, fresh && k == 0 ? 0u : 1u, issue);
      }
      p_phase[s] ^= 1u;
      return true;
    };
    // Two row tiles: the two issuing warps take turns.
    auto my_turn = [&] {
      const bool ok = wait(&sh->turn[warp - 9], turn_phase);
      turn_phase ^= 1u;
      return ok;
    };
    auto your_turn = [&] {
      if (lane == 0) mbar_arrive(&sh->turn[10 - warp]);
    };
    // The next tile of the ring: its stage, or -1 after an abort.
    auto take = [&] {
      const int st = stage;
      if (!wait(&sh->full[st], phase)) return -1;
      advance();
      return st;
    };
    auto to_clean = [&](const Walk<kDual>& w, int t) { return t >= w.shape.cached || (t + 1) * kAtTile > w.shape.len; };
    // Clears V elements of stage `st` that no product may see (whole warp).
    auto clean = [&](const Walk<kDual>& w, int t, int st) {
      const uint32_t v0 = s_ring + st * Cfg::kTileBytes;
      if (t < w.shape.cached) {
        const int rows = w.shape.len - t * kAtTile;
        for (int i = rows * 8 + lane; i < kAtTile * 8; i += 32)
#pragma unroll
          for (int c = 0; c < kChunks; ++c) st_shared_v4(v0 + c * kSlab + i * 16, 0, 0, 0, 0);
      } else {
        // 0 times a number is 0, 0 times an infinity or NaN is NaN: one multiply-add finds
        // out about two elements. What it finds is rare and looked for one by one.
        const int rows = min(kAtTile, a.n - (t - w.shape.cached) * kAtTile);
        const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
        __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll 8
          for (int i = lane; i < rows * 8; i += 32) {
            const uint4 v = *reinterpret_cast<const uint4*>(smem + Cfg::kQBytes + st * Cfg::kTileBytes + c * kSlab + i * 16);
            const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = __hfma2(x[e], zero, acc[e]);
          }
        const __nv_bfloat162 sum = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
        if (__any_sync(0xffffffffu, __hisnan(sum.x) || __hisnan(sum.y))) {
          for (int i = lane; i < rows * 8 * kChunks; i += 32) {
            const uint32_t at = v0 + (i / (rows * 8)) * kSlab + (i % (rows * 8)) * 16;
            uint4 v = ld_shared_v4(at);
            uint32_t* x = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((x[e] & 0x7f80u) == 0x7f80u) x[e] &= 0xffff0000u;
              if ((x[e] & 0x7f800000u) == 0x7f800000u) x[e] &= 0xffffu;
            }
            st_shared_v4(at, x[0], x[1], x[2], x[3]);
          }
          sh->bad[seg & 1] = 1;
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
    };
    for (Walk<kDual> w(a, sh); w.more(); w.next(a)) {
      const int n_tiles = w.t1 - w.t0;
      if (warp == 9 && lane == 0) sh->bad[seg & 1] = 0;
      __syncwarp();
      if (!wait(&sh->q_full, q_phase)) goto mma_done;
      q_phase ^= 1u;
      if (kDual) {
        // Warp 9 issues stream 0's products, warp 10 stream 1's, a tile's second product and the
        // next tile's first in one go, in turn: so one stream's products run while the other's
        // weights are formed, and a warp's own waits and commits fall into the other's turn.
        const int s = warp - 9;
        int k = take();
        if (k < 0 || !my_turn()) goto mma_done;
        qk(s, s, k);
        tc_commit_warp(&sh->s_full[s], issue);  // before the other's products, not behind them
        your_turn();
        tc_commit_warp(&sh->empty[k], issue);
        if (n_tiles == 1) tc_commit_warp(&sh->q_empty, issue);
        if (!wait(&sh->o_empty, o_phase ^ 1u)) goto mma_done;
        for (int i = 0; i < n_tiles; ++i) {
          const bool more = i + 1 < n_tiles;
          const int v = take();
          if (v < 0) goto mma_done;
          if (to_clean(w, w.t0 + i)) {
            // Two barriers in turns: warp 9 may clean the next tile before warp 10 has looked at this
            // one's barrier, but not the one after that, which lies behind a turn that warp 10 gives
            // back after its wait. With one barrier the phase could wrap under that wait.
            if (s == 0) {
              clean(w, w.t0 + i, v);
              if (lane == 0) mbar_arrive(&sh->v_clean[cleaned & 1u]);
            } else {
              if (!wait(&sh->v_clean[cleaned & 1u], (cleaned >> 1) & 1u)) goto mma_done;
            }
            ++cleaned;
          }
          k = more ? take() : 0;
          if (k < 0) goto mma_done;
          if (!wait(&sh->p_full[s][0], p_phase[s])) goto mma_done;
          if (!my_turn() || !pv(s, v, i == 0)) goto mma_done;
          if (more) {
            qk(s, s, k);
            tc_commit_warp(&sh->s_full[s], issue);
          }
          your_turn();
          tc_commit_warp(&sh->empty[v], issue);
          if (more) tc_commit_warp(&sh->empty[k], issue);
          if (i + 2 == n_tiles) tc_commit_warp(&sh->q_empty, issue);
        }
      } else {
        for (int i = 0; i < 2 && i < n_tiles; ++i) {
          const int k = take();
          if (k < 0) goto mma_done;
          qk(i, 0, k);
          tc_commit_warp(&sh->s_full[i], issue);
          tc_commit_warp(&sh->empty[k], issue);
          if (i + 1 == n_tiles) tc_commit_warp(&sh->q_empty, issue);
        }
        if (!wait(&sh->o_empty, o_phase ^ 1u)) goto mma_done;
        for (int i = 0; i < n_tiles; ++i) {
          const int s = i & 1;
          const bool more = i + 2 < n_tiles;
          const int v = take();
          if (v < 0) goto mma_done;
          if (to_clean(w, w.t0 + i)) clean(w, w.t0 + i, v);
          const int k = more ? take() : 0;
          if (k < 0) goto mma_done;
          if (!wait(&sh->p_full[s][0], p_phase[s]) || !pv(s, v, i < 2)) goto mma_done;
          tc_commit_warp(&sh->empty[v], issue);
          if (more) {
            qk(s, 0, k);
            tc_commit_warp(&sh->s_full[s], issue);
          }
          if (more) tc_commit_warp(&sh->empty[k], issue);
          if (i + 3 == n_tiles) tc_commit_warp(&sh->q_empty, issue);
        }
      }
      tc_commit_warp(&sh->o_final, issue);
      if (warp == 9 && lane == 0) mbar_arrive(&sh->o_final);  // and what it found in V
      o_phase ^= 1u;
      ++seg;
    }
  mma_done:
    tc_commit_warp(&sh->mma_done[warp - 9], issue);
    if (lane == 0) {
      int dummy = 0;
      mbar_wait(&sh->mma_done[warp - 9], 0, &dummy, timeout);
    }
    __syncwarp();
  } else if (warp >= 10) {
    regs_dec<kAtRegsOther>();
  } else {
    regs_inc<kAtRegsSoftmax>();
    const int s = warp >> 2;             // stream
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + s * kAtTile;
    const float sc = a.scale * kAtLog2e;
    uint32_t s_phase = 0, f_phase = 0;
    int seg = 0;
    for (Walk<kDual> w(a, sh); w.more(); w.next(a)) {
      const int n_tiles = w.t1 - w.t0;
      const int node0 = (w.mt * (kDual ? 2 : 1) + (kDual ? s : 0)) * a.npt;
      const int rows = max(0, min(a.npt, a.n - node0)) * a.group;  // of this tile
      const bool idle = (warp & 3) * 32 >= rows;                   // a warp without rows
      const int node = min(node0 + row / a.group, a.n - 1);
      float m = -INFINITY, l = 0.0f;
      bool first = true;
      for (int i = kDual ? 0 : s; i < n_tiles; i += kDual ? 1 : 2) {
        bool ok = mbar_wait(&sh->s_full[s], s_phase, abort_flag, timeout);
        if (!__all_sync(0xffffffffu, ok)) goto softmax_done;
        s_phase ^= 1u;
        tc_fence_after();
        if (!idle) {
          const int t = w.t0 + i;
          const bool masked = t >= w.shape.cached || (t + 1) * kAtTile > w.shape.len;
          uint32_t keep[4] = {}, r[4][32];
          float mx;
          if (masked) {
            visible(a, w.shape, w.b, node, t, keep);
            mx = row_scores<true>(ts, keep, r);
          } else {
            mx = row_scores<false>(ts, keep, r);
          }
          mx = fmaxf(mx, m);
          const bool grown = m == -INFINITY ? mx > -INFINITY : (mx - m) * sc > kAtRescale;
          if (__any_sync(0xffffffffu, grown)) {
            // With nothing seen so far l and the accumulator's row are 0 (or not written yet).
            const float f = grown ? (m == -INFINITY ? 0.0f : exp2f_ftz((m - mx) * sc)) : 1.0f;
            if (!first) {  // the previous product is done: this tile's scores were issued behind it
#pragma unroll 1
              for (int c = 0; c < kHD; c += 16) {
                uint32_t o[16];
                tmem_ld16(tmem + lanes + 256 + s * 128 + c, o);
                tmem_wait_ld16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(u2f(o[e]) * f);
                tmem_st16(tmem + lanes + 256 + s * 128 + c, o);
              }
            }
            l *= f;
            if (grown) m = mx;
          }
          const float off = m == -INFINITY ? 0.0f : -m * sc;
          float2 l0 = make_float2(l, 0.0f), l1 = make_float2(0.0f, 0.0f);
          row_weights(ts, r, 0, kAtFirst / 32, sc, off, l0, l1);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->p_full[s][0]);
          row_weights(ts, r, kAtFirst / 32, 4, sc, off, l0, l1);
          l = (l0.x + l0.y) + (l1.x + l1.y);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->p_full[s][1]);
        } else if (lane == 0) {
          mbar_arrive(&sh->p_full[s][0]);
          mbar_arrive(&sh->p_full[s][1]);
        }
        first = false;
      }
      // Epilogue.
      if (!kDual) {
        ml[seg & 1][s][row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->ml_full);
        if (!__all_sync(0xffffffffu, mbar_wait(&sh->ml_full, f_phase, abort_flag, timeout))) goto softmax_done;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&sh->o_final, f_phase, abort_flag, timeout))) goto softmax_done;
      f_phase ^= 1u;
      tc_fence_after();
      {
        // stream sums to join (one row tile): this warp takes half of the channels of both
        float f0 = 1.0f, f1 = 0.0f;
        if (!kDual) {
          const float2 u = ml[seg & 1][0][row], v = ml[seg & 1][1][row];
          m = fmaxf(u.x, v.x);
          f0 = u.x == -INFINITY ? 0.0f : exp2f_ftz((u.x - m) * sc);
          f1 = v.x == -INFINITY ? 0.0f : exp2f_ftz((v.x - m) * sc);
          l = u.y * f0 + v.y * f1;
          if (m == INFINITY) l = NAN;  // inf - inf above
        }
        const bool whole = w.t0 == 0 && w.t1 == w.shape.tiles;
        const bool bad = *reinterpret_cast<volatile int*>(&sh->bad[seg & 1]) != 0;
        const bool write = row < rows;
        const int head = w.h * a.group + row % a.group;
        const long long slot = 2LL * blockIdx.x + (w.t0 > 0 ? 0 : 1);
        const int prow = (kDual ? s * kAtTile : 0) + row;
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        if (!idle) {
          constexpr int kCols = kDual ? kHD : kHD / 2;
          const int col0 = kDual ? 0 : s * kCols;
          const uint32_t to = tmem + lanes + 256 + (kDual ? s * 128 : 0) + col0;
#pragma unroll 1
          for (int c = 0; c < kCols; c += 16) {
            uint32_t o[16];
            tmem_ld16(to + c, o);
            tmem_wait_ld16(o);
            float x[16];
            if (!kDual) {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = f0 != 0.0f ? u2f(o[e]) * f0 : 0.0f;
              if (n_tiles > 1) {
                tmem_ld16(to + 128 + c, o);
                tmem_wait_ld16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] += f1 != 0.0f ? u2f(o[e]) * f1 : 0.0f;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = u2f(o[e]);
            }
            if (bad) {  // elements that the product did not see: an infinity or NaN swallows any sum
              const int d1 = min(a.n, (w.t1 - w.shape.cached) * kAtTile);
              for (int j = max(0, w.t0 - w.shape.cached) * kAtTile; j < d1; ++j) {
                const bool sees = a.mask != nullptr
                                      ? (a.mask[(static_cast<long long>(w.b) * a.n + node) * a.words + (j >> 6)] >> (j & 63)) & 1u
                                      : j <= node;
                if (!sees) continue;
                const __nv_bfloat16* v = a.v_draft + w.b * a.draft_seq + j * a.draft_row + w.h * kHD + col0 + c;
                for (int e = 0; e < 16; ++e) {
                  const float y = __bfloat162float(v[e]);
                  if (!isfinite(y)) x[e] += y;
                }
              }
            }
            if (write) {
              if (whole) {
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(x[2 * e] * inv, x[2 * e + 1] * inv);
                __nv_bfloat16* dst = a.out + w.b * a.out_seq + node * a.out_row + static_cast<long long>(head) * kHD + col0 + c;
                st_global_v4(dst, pk[0], pk[1], pk[2], pk[3]);
                st_global_v4(dst + 8, pk[4], pk[5], pk[6], pk[7]);
              } else {  // rows side by side: a warp's store is 512 bytes in a row
                float4* dst = a.part_o + (slot * (kHD / 4) + (col0 + c) / 4) * Cfg::kRows + prow;
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[e * Cfg::kRows] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
              }
            }
          }
          if (write && (kDual || s == 0)) {
            if (!whole) a.part_ml[slot * Cfg::kRows + prow] = make_float2(m, l);
            else if (a.lse != nullptr)
              a.lse[(static_cast<long long>(w.b) * a.n + node) * (static_cast<long long>(a.heads) * a.group) + head] =
                  l == 0.0f ? -INFINITY : m * a.scale + logf(l);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->o_empty);
      ++seg;
    }
  softmax_done:;
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sh->abort) record_status(a.dev_status, RF_ERR_TIMEOUT);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the rows of items that were cut. Block (x, y): the cut before share x + 1, rows
// 32 y .. 32 y + 31 of its item; the first cut inside an item answers for it. A lane is a
// row (or part of one), a warp 16 channels of it. Launched as a dependent of k_attn: its CTAs
// wait in place for that one's end.
struct CombineArgs {
  const AttnPlan* plan;
  const float4* part_o;
  const float2* part_ml;
  __nv_bfloat16* out;
  float* lse;
  long long out_row, out_seq;
  int n, heads, group, npt, tiles, ctas;  // tiles: row tiles of an item
  float scale;
};

// kBatch: parts in flight together; kSplit: lanes that share a row, each joining every kSplit-th
// part. Few rows of few items, cut into 8 parts or more: 8 and 4, so that one round of loads
// holds up to 32 parts. Else 4 and 1: more rows a CTA, more CTAs an SM. The whole call, one way
// and the other: 25 rows in 19 parts 34.6 and 38.4 us, 20 rows in 2.4 parts 40.4 and 39.3,
// 125 rows in 19 parts 24.0 and 21.8.
template <int kHD, int kBatch, int kSplit>
__global__ void __launch_bounds__(kHD * 2) k_attn_combine(const __grid_constant__ CombineArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // lane i: the share c - 1 + i
  const AttnPlan q = a.plan[min(c - 1 + lane, a.ctas - 1)];
  const long long item = __shfl_sync(0xffffffffu, q.item, 1);
  if (item < 0 || __shfl_sync(0xffffffffu, q.t0, 1) == 0) return;
  if (__shfl_sync(0xffffffffu, q.item, 0) == item && __shfl_sync(0xffffffffu, q.t0, 0) > 0) return;
  const int b = __shfl_sync(0xffffffffu, q.b, 1), h = __shfl_sync(0xffffffffu, q.h, 1), mt = __shfl_sync(0xffffffffu, q.mt, 1);
  // parts of the item: from share c - 1, and from every share from c on that starts inside it
  const unsigned inside = __ballot_sync(0xffffffffu, lane == 0 || (c - 1 + lane < a.ctas && q.item == item && q.t0 > 0));
  int parts = inside == 0xffffffffu ? 32 : __ffs(~inside) - 1;
  while (parts % 32 == 0) {
    const int i = c - 1 + parts + lane;
    const bool in = i < a.ctas && a.plan[i].item == item && a.plan[i].t0 > 0;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (m == 0u) break;
    parts += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
  }
  const int item_rows = a.tiles * kAtTile;
  constexpr int kLanes = 32 / kSplit;
  const int r = blockIdx.y * kLanes + lane % kLanes, in_tile = r % kAtTile;
  const int node = (mt * a.tiles + r / kAtTile) * a.npt + in_tile / a.group;
  const bool live = r < item_rows && in_tile < a.npt * a.group && node < a.n;
  if (kSplit == 1 && !live) return;
  const int head = h * a.group + in_tile % a.group;
  const float sc = a.scale * kAtLog2e;
  auto slot_of = [&](int i) { return i == 0 ? 2LL * (c - 1) + 1 : 2LL * (c - 1 + i); };
  float m = -INFINITY, l = 0.0f;
  float4 x[4] = {};
  for (int i0 = live ? lane / kLanes : parts; i0 < parts; i0 += kBatch * kSplit) {
    float2 ml[kBatch];
    float4 v[kBatch][4];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (i0 + j * kSplit >= parts) break;
      const long long slot = slot_of(i0 + j * kSplit);
      ml[j] = a.part_ml[slot * item_rows + r];
      const float4* src = a.part_o + (slot * (kHD / 4) + warp * 4) * item_rows + r;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = src[e * item_rows];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (i0 + j * kSplit >= parts) break;
      // a running maximum: one pass over the parts
      const float mx = fmaxf(m, ml[j].x);
      const float f = m == -INFINITY ? 0.0f : exp2f_ftz((m - mx) * sc);
      const float g = ml[j].x == -INFINITY ? 0.0f : exp2f_ftz((ml[j].x - mx) * sc);
      m = mx;
      l = l * f + ml[j].y * g;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e].x = x[e].x * f + v[j][e].x * g;
        x[e].y = x[e].y * f + v[j][e].y * g;
        x[e].z = x[e].z * f + v[j][e].z * g;
        x[e].w = x[e].w * f + v[j][e].w * g;
      }
    }
  }
  if constexpr (kSplit > 1) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) {
      const float m1 = __shfl_xor_sync(0xffffffffu, m, o), l1 = __shfl_xor_sync(0xffffffffu, l, o);
      const float mx = fmaxf(m, m1);
      const float f = m == -INFINITY ? 0.0f : exp2f_ftz((m - mx) * sc);
      const float g = m1 == -INFINITY ? 0.0f : exp2f_ftz((m1 - mx) * sc);
      m = mx;
      l = l * f + l1 * g;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e].x = x[e].x * f + __shfl_xor_sync(0xffffffffu, x[e].x, o) * g;
        x[e].y = x[e].y * f + __shfl_xor_sync(0xffffffffu, x[e].y, o) * g;
        x[e].z = x[e].z * f + __shfl_xor_sync(0xffffffffu, x[e].z, o) * g;
        x[e].w = x[e].w * f + __shfl_xor_sync(0xffffffffu, x[e].w, o) * g;
      }
    }
    if (!live || lane >= kLanes) return;
  }
  if (m == INFINITY) l = NAN;  // inf - inf
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  uint32_t pk[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    pk[2 * e] = pack_bf16x2(x[e].x * inv, x[e].y * inv);
    pk[2 * e + 1] = pack_bf16x2(x[e].z * inv, x[e].w * inv);
  }
  __nv_bfloat16* dst = a.out + b * a.out_seq + node * a.out_row + static_cast<long long>(head) * kHD + warp * 16;
  st_global_v4(dst, pk[0], pk[1], pk[2], pk[3]);
  st_global_v4(dst + 8, pk[4], pk[5], pk[6], pk[7]);
  if (warp == 0 && a.lse != nullptr)
    a.lse[(static_cast<long long>(b) * a.n + node) * (static_cast<long long>(a.heads) * a.group) + head] =
        l == 0.0f ? -INFINITY : m * a.scale + logf(l);
}

rf_status check_attn_desc(const rf_attn_desc* d) {
  if (d == nullptr) return fail(RF_ERR_INVALID_ARG, "desc is NULL");
  if (d->n_seqs < 0 || d->n_q_heads <= 0 || d->n_kv_heads <= 0 || d->n_nodes <= 0 || d->capacity <= 0)
    return fail(RF_ERR_INVALID_ARG, "need n_seqs >= 0, n_q_heads, n_kv_heads, n_nodes, capacity > 0");
  // (exponents are formed in base 2)
  const float scale = static_cast<float>(d->scale);
  if (!(d->scale > 0.0) || !(scale > 0.0f) || !std::isfinite(scale * kAtLog2e))
    return fail(RF_ERR_INVALID_ARG, "scale must be > 0 and scale / ln 2 finite in fp32");
  if (d->flags != 0) return fail(RF_ERR_INVALID_ARG, "flags must be 0");
  if (d->head_dim != 64 && d->head_dim != 128) return fail(RF_ERR_SHAPE, "head_dim must be 64 or 128");
  if (d->n_q_heads % d->n_kv_heads != 0 || d->n_q_heads / d->n_kv_heads > 128)
    return fail(RF_ERR_SHAPE, "n_q_heads must be a multiple of n_kv_heads, at most 128 times it");
  if (d->n_nodes > (int64_t(1) << 20) || d->capacity > (int64_t(1) << 30) || d->n_seqs > (int64_t(1) << 20) ||
      d->n_q_heads > (int64_t(1) << 20))
    return fail(RF_ERR_SHAPE, "need n_nodes, n_seqs, n_q_heads <= 2^20, capacity <= 2^30");
  const int64_t qw = d->n_q_heads * d->head_dim, kw = d->n_kv_heads * d->head_dim;
  const int64_t rows[4] = {d->q_row_stride, d->draft_row_stride, d->cache_row_stride, d->out_row_stride};
  const int64_t seqs[4] = {d->q_seq_stride, d->draft_seq_stride, d->cache_seq_stride, d->out_seq_stride};
  const int64_t least[4] = {qw, kw, kw, qw};
  for (int i = 0; i < 4; ++i) {
    if (rows[i] < least[i] || rows[i] % 8 || seqs[i] % 8 || (d->n_seqs > 1 && seqs[i] <= 0))
      return fail(RF_ERR_ALIGN, "strides must be multiples of 8, row strides >= heads*head_dim, sequence strides > 0");
    if (rows[i] >= (int64_t(1) << 39) || seqs[i] >= (int64_t(1) << 39)) return fail(RF_ERR_SHAPE, "strides must be < 2^39");
  }
  return RF_OK;
}

struct AttnLayout {
  float4* part_o;
  float2* part_ml;
  AttnPlan* plan;
  int tiles;  // row tiles of an item
  size_t bytes;
};

static AttnLayout attn_layout(const rf_attn_desc* d, void* ws) {
  AttnLayout l;
  l.tiles = d->n_nodes * (d->n_q_heads / d->n_kv_heads) > kAtTile ? 2 : 1;
  const size_t rows = static_cast<size_t>(2 * kAtMaxCtas) * l.tiles * kAtTile;
  Carve c(ws);
  l.part_o = c.take<float4>(rows * d->head_dim / 4);
  l.part_ml = c.take<float2>(rows);
  l.plan = c.take<AttnPlan>(kAtMaxCtas);
  l.bytes = c.bytes();
  return l;
}

template <int kHD, bool kDual>
static rf_status launch_attn(const AttnArgs& a, int ctas, cudaStream_t s) {
  static uint64_t done = 0;
  using Cfg = AttnCfg<kHD, kDual>;
  static_assert(Cfg::kSmem <= 227 * 1024, "shared memory beyond the 227 KB a CTA may hold");
  rf_status st = set_smem_attr(reinterpret_cast<const void*>(&k_attn<kHD, kDual>), Cfg::kSmem, &done);
  if (st != RF_OK) return st;
  ProfScope prof(s, RF_STAGE_ATTENTION);
  return cuda_check(launch_dependent(k_attn<kHD, kDual>, dim3(static_cast<unsigned>(ctas)), dim3(kAtThreads), Cfg::kSmem, s, 1, a),
                    "k_attn launch");
}

}  // namespace rf

using namespace rf;

extern "C" size_t rf_attn_workspace_bytes(const rf_attn_desc* desc) {
  if (check_attn_desc(desc) != RF_OK) return 0;
  return attn_layout(desc, nullptr).bytes;
}

extern "C" rf_status rf_tree_attention(const rf_attn_desc* d, const rf_bf16* q, const rf_bf16* k_cache,
                                       const rf_bf16* v_cache, const int32_t* lens, const rf_bf16* k_draft,
                                       const rf_bf16* v_draft, const uint64_t* tree_mask, rf_bf16* out, float* lse,
                                       int32_t* dev_status, void* workspace, size_t workspace_bytes,
                                       rf_stream_t stream) {
  clear_error();
  rf_status st = check_attn_desc(d);
  if (st != RF_OK) return st;
  if (tree_mask != nullptr && d->n_nodes > RF_TREE_MAX_NODES)
    return fail(RF_ERR_SHAPE, "n_nodes must be <= %d with a mask", RF_TREE_MAX_NODES);
  if (d->n_seqs == 0) return RF_OK;
  if (!q || !k_cache || !v_cache || !lens || !k_draft || !v_draft || !out)
    return fail(RF_ERR_INVALID_ARG, "tensor pointers must be non-NULL");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_draft) || !aligned16(v_draft) ||
      !aligned16(out))
    return fail(RF_ERR_ALIGN, "row buffers must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(lens) & 3u) || (reinterpret_cast<uintptr_t>(tree_mask) & 7u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(RF_ERR_ALIGN, "arrays must be aligned to their elements");
  const AttnLayout lay = attn_layout(d, workspace);
  if (workspace == nullptr || workspace_bytes < lay.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(RF_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", lay.bytes, workspace_bytes);
  int sms = 0;
  if ((st = current_device(&sms)) != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint64_t hd = d->head_dim, H = d->n_kv_heads, Hq = d->n_q_heads, n = d->n_nodes, B = d->n_seqs;
  const int group = static_cast<int>(Hq / H);
  AttnArgs a{};
  a.npt = kAtTile / group;
  const uint64_t cap = d->capacity;
  // a box of a row tile: every head of the group, npt nodes
  if ((st = make_tmap_bf16_4d(&a.tm_q, q, {hd, Hq, n, B}, {hd, (uint64_t)d->q_row_stride, (uint64_t)d->q_seq_stride},
                              {64, (uint32_t)group, (uint32_t)a.npt, 1})) != RF_OK)
    return st;
  const uint64_t cs[3] = {hd, (uint64_t)d->cache_row_stride, (uint64_t)d->cache_seq_stride};
  const uint64_t ds[3] = {hd, (uint64_t)d->draft_row_stride, (uint64_t)d->draft_seq_stride};
  const uint64_t cd[4] = {hd, H, cap, B}, dd[4] = {hd, H, n, B};
  const uint32_t box[4] = {64, 1, kAtTile, 1};
  if ((st = make_tmap_bf16_4d(&a.tm_k, k_cache, cd, cs, box)) != RF_OK) return st;
  if ((st = make_tmap_bf16_4d(&a.tm_v, v_cache, cd, cs, box)) != RF_OK) return st;
  if ((st = make_tmap_bf16_4d(&a.tm_kd, k_draft, dd, ds, box)) != RF_OK) return st;
  if ((st = make_tmap_bf16_4d(&a.tm_vd, v_draft, dd, ds, box)) != RF_OK) return st;
  a.lens = lens;
  a.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  a.v_draft = reinterpret_cast<const __nv_bfloat16*>(v_draft);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.part_o = lay.part_o;
  a.part_ml = lay.part_ml;
  a.plan = lay.plan;
  a.dev_status = dev_status;
  a.timeout_ns = wait_timeout_ns();
  a.out_row = d->out_row_stride;
  a.out_seq = d->out_seq_stride;
  a.draft_row = d->draft_row_stride;
  a.draft_seq = d->draft_seq_stride;
  a.n_seqs = static_cast<int>(B);
  a.heads = static_cast<int>(H);
  a.group = group;
  a.n = static_cast<int>(n);
  a.capacity = static_cast<int>(cap);
  a.words = static_cast<int>(RF_TREE_WORDS(n));
  a.scale = static_cast<float>(d->scale);
  const int64_t per = static_cast<int64_t>(a.npt) * lay.tiles;  // nodes of an item
  a.m_items = static_cast<int>((n + per - 1) / per);
  int64_t draft_sum = 0;
  for (int64_t mt = 0; mt < a.m_items; ++mt) {
    const int64_t seen = tree_mask != nullptr ? static_cast<int64_t>(n) : std::min<int64_t>(n, (mt + 1) * per);
    draft_sum += (seen + kAtTile - 1) / kAtTile;
  }
  if (draft_sum >= (int64_t(1) << 31)) return fail(RF_ERR_SHAPE, "n_nodes is too large");
  a.draft_sum = static_cast<int>(draft_sum);
  // no more CTAs than weight, which is at least the tiles
  const int64_t most = static_cast<int64_t>(B * H) * (a.m_items * static_cast<int64_t>((cap + kAtTile - 1) / kAtTile + kAtItemCost) + draft_sum);
  const int ctas = static_cast<int>(std::min<int64_t>(most, std::min(sms, kAtMaxCtas)));
  if (hd == 128) st = lay.tiles == 2 ? launch_attn<128, true>(a, ctas, s) : launch_attn<128, false>(a, ctas, s);
  else st = lay.tiles == 2 ? launch_attn<64, true>(a, ctas, s) : launch_attn<64, false>(a, ctas, s);
  if (st != RF_OK || ctas < 2) return st;
  CombineArgs c{};
  c.plan = lay.plan;
  c.part_o = lay.part_o;
  c.part_ml = lay.part_ml;
  c.out = a.out;
  c.lse = lse;
  c.out_row = a.out_row;
  c.out_seq = a.out_seq;
  c.n = a.n;
  c.heads = a.heads;
  c.group = group;
  c.npt = a.npt;
  c.tiles = lay.tiles;
  c.ctas = ctas;
  c.scale = a.scale;
  // rows of an item that exist, in a tile's numbering (the first tile's are followed by a gap)
  const int tile_rows = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(n) * group, a.npt * group));
  const int rows = lay.tiles == 2 ? 2 * kAtTile : tile_rows;
  const bool few = rows <= 32 && B * H * a.m_items * 8 <= ctas;
  const dim3 grid(static_cast<unsigned>(ctas - 1), static_cast<unsigned>((rows + (few ? 7 : 31)) / (few ? 8 : 32)));
  ProfScope prof(s, RF_STAGE_ATTN_COMBINE);
  void (*combine)(CombineArgs) = hd == 128 ? (few ? k_attn_combine<128, 8, 4> : k_attn_combine<128, 4, 1>)
                                           : (few ? k_attn_combine<64, 8, 4> : k_attn_combine<64, 4, 1>);
  return cuda_check(launch_dependent(combine, grid, dim3(static_cast<unsigned>(2 * hd)), 0, s, 1, c),
                    "k_attn_combine launch");
}
