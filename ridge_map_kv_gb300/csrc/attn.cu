// Attention of drafted rows over a cache and over each other (rf_tree_attention), and over a prefix that
// all sequences share besides (rf_prefix_attention).
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
//
// With a shared prefix, softmax sums are joined over two sets of keys: the prefix, as one more sequence whose
// rows are those of all sequences, so that its keys are read once and serve one matrix product; and each
// sequence's own. Bound: the bytes of the prefix and of all own rows up to some 275 query rows per KV head (all
// sequences together), the products over the prefix beyond. See PrefixArgs, and k_attn where it forms pairs of heads
// and copies of few rows. Measured (128 channels, 8 KV heads): 4 sequences of one token, 5 query heads on one, over
// 32,767 shared rows and up to 200 of their own: 35 us (3.9 TB/s; 20 would be the bytes). 64 of one token, 4 on
// one, over 16,384 and up to 1,024: 63 us (3.2 TB/s, 30). 16 trees of 64 nodes, 4 on one, over 28,672 and up to
// 300: 352 us from rest and 368 in long runs (1,370 and 1,310 TFLOP/s, 249 at the burst rate). 100 times three rows, 10 on one of 2
// heads of 64 channels, over 4,099 and up to 4,000: 57 us (1.9 TB/s, 16). One sequence's cache at a time, the prefix in
// each, would read the prefix 64 times in the second case. With two row tiles and 128 channels the kernel's four kinds of
// items leave 60 bytes of a thread without a register; those without a prefix, and of 64 channels, have room.
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
constexpr int kPfRows = 256;      // rows that a part may have
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
  static constexpr bool kPrefix = false;
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

// With a prefix that all sequences share (rf_prefix_attention), it is one more sequence, b = -1, before
// the others: its rows are those of all sequences, so its keys are read once for all. Every row then has
// parts in two items, its own sequence's and the prefix's, which k_prefix_join adds up. Items that were
// not cut leave their parts in places of their own.
struct PrefixArgs : AttnArgs {
  static constexpr bool kPrefix = true;
  CUtensorMap tm_qp, tm_kp, tm_vp;
  const int32_t* prefix_len;
  int prefix_capacity;
  // A row tile of the prefix: p_nodes nodes of each of p_seqs sequences. Few nodes: whole sequences, as many
  // as fit; else p_split tiles a sequence, which is the last of them not full.
  int p_nodes, p_seqs, p_split;
  int p_items;       // items of a head
  // Where the prefix takes two row tiles and a sequence's rows of a head fit into one, a sequence's items are pairs of
  // heads, one to a stream; rows that are at most 32 are there four times (see k_attn).
  int pairs;         // 1 or 0
  int own_heads;     // items of a sequence (heads, or pairs of them) at a time of its rows
  int copies;        // 4 or 1
  int in_step;           // tiles of a prefix beyond which its items go in step (see Walk)
  // What an item, a tile of the prefix and a tile of a sequence's own weigh in the shares.
  int w_item, w_prefix, w_own;
  int rows, p_rows;      // rows of an item's stored part, of a sequence and of the prefix
  float4* whole_o;   // [items][head_dim / 4][rows of the item], the prefix's items first
  float2* whole_ml;
  int2* item_ctas;   // [items] the CTAs of an item's first and last tile
};

struct AttnShared {
  uint64_t full[kAtMaxStages], empty[kAtMaxStages];
  uint64_t q_full, q_empty, s_full[2], p_full[2][2], o_final, o_empty, ml_full, turn[2], v_clean[2], mma_done[2];
  AttnShare share, beginning;  // beginning: what of the share comes last (see Walk), of weight 0 where nothing does
  int bad[2][2];             // [segment parity][stream]: a drafted V row of the segment is not finite
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
__device__ __forceinline__ int prefix_of(const PrefixArgs& a) {
  const int len = *a.prefix_len;
  return len < 0 || len > a.prefix_capacity ? -1 : len;
}
template <class Args>
__device__ __forceinline__ int heads_of(const Args& a, int b) {  // or pairs of heads
  if constexpr (Args::kPrefix) return b < 0 ? a.heads : a.own_heads;
  else return a.heads;
}
template <class Args>
__device__ __forceinline__ int items_of(const Args& a, int b) {  // of a head
  if constexpr (Args::kPrefix) return b < 0 ? a.p_items : a.m_items;
  else return a.m_items;
}
// An item weighs item_weight and tile_weight for each of its tiles. With one row tile all tiles weigh alike, with a prefix
// or without: a tile is its bytes. (Weights that are known at run time only cost a call of 37 us one.)
template <bool kDual, class Args>
__device__ __forceinline__ int item_weight(const Args& a) {
  if constexpr (kDual && Args::kPrefix) return a.w_item;
  else return kAtItemCost;
}
template <bool kDual, class Args>
__device__ __forceinline__ int tile_weight(const Args& a, int b) {
  if constexpr (kDual && Args::kPrefix) return b < 0 ? a.w_prefix : a.w_own;
  else return 1;
}
// The first tile that lies behind `at` in the weight of an item of sequence b.
template <bool kDual, class Args>
__device__ __forceinline__ int tile_behind(const Args& a, int at, int b) {
  const int x = max(at - item_weight<kDual>(a), 0);
  if constexpr (kDual && Args::kPrefix) return x / tile_weight<kDual>(a, b);
  else return x;
}
template <bool kDual, class Args>
__device__ __forceinline__ ItemShape item_shape(const Args& a, int b, int mt) {
  ItemShape s;
  if constexpr (Args::kPrefix) {
    if (b < 0) {
      s.len = prefix_of(a);
      s.cached = s.tiles = (max(s.len, 0) + kAtTile - 1) / kAtTile;
      return s;
    }
  }
  s.len = length_of(a, b);
  s.cached = (max(s.len, 0) + kAtTile - 1) / kAtTile;
  s.tiles = s.len < 0 ? 0 : s.cached + draft_tiles<kDual>(a, mt);
  return s;
}

// A CTA's share, segment by segment; every role walks it alike, a converged warp at a time.
template <bool kDual, class Args>
struct Walk {
  int b, h, mt, t0, t1;  // an item and the tiles of it that are the share's
  int at;                // where the share stands in the item's weight
  long long left;        // weight
  ItemShape shape;
  // Where the prefix has several items a head, its keys are read from memory about once if their CTAs go through them in
  // step. So a share that begins within one of them and goes on into the next does that beginning last: every CTA is
  // then near the tile whose number is the time. (16 trees of 64 nodes over 28,672 rows: 395 us in the order of the
  // shares, 1.4 GB read for 0.12, and 366 so. It takes a prefix that L2 does not hold beside the rest: 133 us either way
  // over 8,192 rows, 33 MB; 91 and 96 over 4,096.)
  static constexpr bool kInStep = kDual && Args::kPrefix;
  __device__ __forceinline__ Walk(const Args& a, const AttnShared* sh) {
    begin(a, sh->share);
    if constexpr (kInStep) {
      if (left <= 0) begin(a, sh->beginning);
    }
  }
  __device__ __forceinline__ void begin(const Args& a, const AttnShare& share) {
    b = uniform(share.b);
    h = uniform(share.h);
    mt = uniform(share.mt);
    at = uniform(share.at);
    left = uniform(share.weight);
    shape.len = uniform(share.len);
    shape.cached = (shape.len + kAtTile - 1) / kAtTile;
    shape.tiles = uniform(share.n_tiles);
    t0 = t1 = 0;
    if (left > 0) settle(a);
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ int end(const Args& a) const {
    return static_cast<int>(min(static_cast<long long>(shape.tiles) * tile_weight<kDual>(a, b) + item_weight<kDual>(a), at + left));
  }
  // The first tiles from here on (a share may end within an item's extra weight).
  __device__ __forceinline__ void settle(const Args& a) {
    while (true) {
      if constexpr (Args::kPrefix) {  // (most items are whole ones)
        const int whole = shape.tiles * tile_weight<kDual>(a, b) + item_weight<kDual>(a);
        t0 = at == 0 ? 0 : tile_behind<kDual>(a, at, b);
        t1 = at + left >= whole ? shape.tiles : tile_behind<kDual>(a, end(a), b);
      } else {
        t0 = tile_behind<kDual>(a, at, b);
        t1 = tile_behind<kDual>(a, end(a), b);
      }
      if (t1 > t0) return;
      next_item(a);
      if (left <= 0) return;
    }
  }
  __device__ __forceinline__ void next(const Args& a, const AttnShared* sh) {
    const bool ahead = t0 == 0;  // (not the beginning: what comes before that begins at its item's first tile)
    next_item(a);
    if (left > 0) settle(a);
    if constexpr (kInStep) {
      if (left <= 0 && ahead) begin(a, sh->beginning);
    }
  }
  __device__ __forceinline__ void next_item(const Args& a) {
    left -= end(a) - at;
    if (left <= 0) return;
    at = 0;
    do {
      if (++mt == items_of(a, b)) {
        mt = 0;
        if (++h == heads_of(a, b)) {
          h = 0;
          if (++b >= a.n_seqs) {  // lengths that changed under the kernel: no sequence is left
            left = 0;
            return;
          }
        } else if (Args::kPrefix && items_of(a, b) == 1) {
          continue;  // another head of the same sequence: the same shape
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
template <bool kDual, class Args>
__device__ void find_share(const Args& a, AttnShared* sh, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  int prefix = 0, prefix_tiles = 0;
  long long prefix_weight = 0;
  const int len_0 = lane < a.n_seqs ? length_of(a, lane) : -1;
  if constexpr (Args::kPrefix) {
    prefix = prefix_of(a);
    if (prefix < 0) record_status(a.dev_status, RF_ERR_INVALID_ARG);
    prefix_tiles = (max(prefix, 0) + kAtTile - 1) / kAtTile;
    if (prefix_tiles > 0)
      prefix_weight = static_cast<long long>(a.heads) * a.p_items * (static_cast<long long>(prefix_tiles) * tile_weight<kDual>(a, -1) + item_weight<kDual>(a));
  }
  auto weight_of = [&](int len) -> long long {
    return len < 0 ? 0ll
                   : static_cast<long long>(heads_of(a, 0)) *
                         (static_cast<long long>(a.m_items) *
                              (static_cast<long long>((len + kAtTile - 1) / kAtTile) * tile_weight<kDual>(a, 0) + item_weight<kDual>(a)) +
                          static_cast<long long>(a.draft_sum) * tile_weight<kDual>(a, 0));
  };
  long long total = 0;
  int len = -1;  // of sequence `lane`, then of later ones
  for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
    len = b0 == 0 ? len_0 : b0 + lane < a.n_seqs ? length_of(a, b0 + lane) : -1;
    if (len < 0 && b0 + lane < a.n_seqs) record_status(a.dev_status, RF_ERR_INVALID_ARG);
    total += weight_of(len);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total = prefix < 0 ? 0 : total + prefix_weight;  // (a prefix that is out of range: no sequence can be answered)
  // (no share is less than a tile: every CTA between an item's first and last one has a part of it)
  long long most = total;
  if constexpr (kDual && Args::kPrefix) most = total / max(a.w_prefix, a.w_own);
  const long long shares = min(static_cast<long long>(ctas), most);
  AttnShare p{};
  if (cta < shares) {
    const long long first = share_start(total, cta, static_cast<int>(shares));
    p.weight = share_start(total, cta + 1, static_cast<int>(shares)) - first;
    long long base = prefix_weight;
    if constexpr (Args::kPrefix) {
      if (first < prefix_weight) {
        p.b = -1;
        p.len = prefix;
        p.n_tiles = prefix_tiles;
        const long long per_item = static_cast<long long>(prefix_tiles) * tile_weight<kDual>(a, -1) + item_weight<kDual>(a), per_head = a.p_items * per_item;
        p.h = static_cast<int>(quick_div(first, per_head));
        const long long at = first - p.h * per_head;
        p.mt = static_cast<int>(quick_div(at, per_item));
        p.at = static_cast<int>(at - p.mt * per_item);
      }
    }
    for (int b0 = 0; b0 < a.n_seqs && first >= prefix_weight; b0 += 32) {
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
        const long long per_head = quick_div(__shfl_sync(0xffffffffu, own, at), heads_of(a, 0));
        p.h = static_cast<int>(quick_div(r, per_head));
        r -= p.h * per_head;
        p.mt = 0;
        p.n_tiles = cached + draft_tiles<kDual>(a, 0);
        const auto weight = [&] { return static_cast<long long>(p.n_tiles) * tile_weight<kDual>(a, 0) + item_weight<kDual>(a); };
        if (a.mask != nullptr) {
          p.mt = static_cast<int>(quick_div(r, weight()));
          r -= p.mt * weight();
        } else {
          while (r >= weight()) {
            r -= weight();
            p.n_tiles = cached + draft_tiles<kDual>(a, ++p.mt);
          }
        }
        p.at = static_cast<int>(r);
        break;
      }
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  if constexpr (Walk<kDual, Args>::kInStep) {
    AttnShare first{};
    const int whole = prefix_tiles * a.w_prefix + a.w_item;
    if (p.weight > whole - p.at && p.b < 0 && prefix_tiles > a.in_step && a.p_items > 1 && tile_behind<kDual>(a, p.at, -1) > 0 &&
        (p.h + 1 < a.heads || p.mt + 1 < a.p_items)) {
      first = p;
      first.weight = whole - p.at;
      p.weight -= first.weight;
      p.at = 0;
      if (++p.mt == a.p_items) {
        p.mt = 0;
        ++p.h;
      }
    }
    if (lane == 0) sh->beginning = first;
  }
  if (lane == 0) sh->share = p;
  __syncwarp();
  if constexpr (Args::kPrefix) return;
  const Walk<kDual, Args> w(a, sh);
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

// Multiplies a row of the accumulator.
template <int kHD>
__device__ __forceinline__ void rescale_row(uint32_t to, float f) {
#pragma unroll 1
  for (int c = 0; c < kHD; c += 16) {
    uint32_t o[16];
    tmem_ld16(to + c, o);
    tmem_wait_ld16(o);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(u2f(o[e]) * f);
    tmem_st16(to + c, o);
  }
}

// The same as row_weights for 32 keys.
__device__ __forceinline__ void quarter_weights(uint32_t to, uint32_t (&r)[32], float sc, float off, float2& t0, float2& t1) {
  const float2 sc2 = make_float2(sc, sc), off2 = make_float2(off, off);
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    float2 x = fma_x2(make_float2(u2f(r[i]), u2f(r[i + 1])), sc2, off2);
    float2 y = fma_x2(make_float2(u2f(r[i + 2]), u2f(r[i + 3])), sc2, off2);
    x = make_float2(exp2f_ftz(x.x), exp2f_ftz(x.y));
    y = make_float2(exp2f_ftz(y.x), exp2f_ftz(y.y));
    t0 = add_x2(t0, x);
    t1 = add_x2(t1, y);
    w[i / 2] = pack_bf16x2(x.x, x.y);
    w[i / 2 + 1] = pack_bf16x2(y.x, y.y);
  }
  tmem_st16(to, w);
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

// Those of its keys 32 c .. 32 c + 31.
__device__ __forceinline__ uint32_t visible_quarter(const AttnArgs& a, const ItemShape& s, int b, int node, int t, int c) {
  const bool draft = t >= s.cached;
  const int j0 = (t - s.cached) * kAtTile;
  const int k = (!draft ? s.len - t * kAtTile : (a.mask != nullptr ? a.n : min(a.n, node + 1)) - j0) - c * 32;
  uint32_t keep = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
  if (draft && a.mask != nullptr) {
    const int w = (t - s.cached) * 2 + (c >> 1);
    const unsigned long long m = w < a.words ? a.mask[(static_cast<long long>(b) * a.n + node) * a.words + w] : 0ull;
    keep &= static_cast<uint32_t>(m >> ((c & 1) * 32));
  }
  return keep;
}

template <int kHD, bool kDual, class Args>
__global__ void __launch_bounds__(kAtThreads, 1) k_attn(const __grid_constant__ Args a) {
  using Cfg = AttnCfg<kHD, kDual>;
  constexpr int kChunks = kHD / 64;                 // 64-channel slabs of a tile, 16 KB each
  constexpr int kSlab = kAtTile * 128;
  constexpr int kMmaWarps = kDual ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  AttnShared* sh = reinterpret_cast<AttnShared*>(smem + Cfg::kQBytes + Cfg::kStages * Cfg::kTileBytes);
  // Items of one row tile, whose streams take alternate key tiles, exchange maxima and totals.
  AttnExchange& ml = *reinterpret_cast<AttnExchange*>(sh + 1);
  // With a prefix: two heads of a sequence, each of whose rows fit into one row tile, are an item, a head to a
  // stream with key tiles of its own. (One head at a time, its key tiles in turns on both streams, an item of
  // one to five tiles took 5 us beside them for its first and last steps; two go side by side.)
  const auto paired = [&](int b) {
    if constexpr (kDual && Args::kPrefix) return b >= 0 && a.pairs != 0;
    else return false;
  };
  const auto heads_in = [&](int h) { return min(2, a.heads - 2 * h); };  // of a pair
  // Of those, heads of at most 32 rows: a row tile's four warps read 32 TMEM lanes each, so one of them would take
  // all exponentials. Instead the rows are there four times, 32 rows apart, and each copy's warp sees a quarter of
  // every tile's keys: four parts with their own maxima and totals, which the join adds up. (64 sequences of one token,
  // 4 query heads on one, over 484 rows: a tile's weights took 1.0 us of one warp.)
  const auto copied = [&](int b) {
    if constexpr (kDual && Args::kPrefix) return b >= 0 && a.copies > 1;
    else return false;
  };
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
    mbar_init(&sh->o_final, 2 * kMmaWarps);
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
    if constexpr (Args::kPrefix) {
      tma_prefetch_desc(&a.tm_qp);
      tma_prefetch_desc(&a.tm_kp);
      tma_prefetch_desc(&a.tm_vp);
    }
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
      auto load = [&](const Walk<kDual, Args>& w, int t, bool v, int h) {
        if (!wait(&sh->empty[stage], phase ^ 1u)) return false;
        const bool draft = t >= w.shape.cached;
        const CUtensorMap* tm = draft ? (v ? &a.tm_vd : &a.tm_kd) : (v ? &a.tm_v : &a.tm_k);
        if constexpr (Args::kPrefix) {
          if (w.b < 0) tm = v ? &a.tm_vp : &a.tm_kp;
        }
        const int row = (draft ? t - w.shape.cached : t) * kAtTile;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh->full[stage], Cfg::kTileBytes);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            tma_load_4d(s_ring + stage * Cfg::kTileBytes + c * kSlab, tm, smem_u32(&sh->full[stage]), c * 64, h, row, max(w.b, 0));
        }
        __syncwarp();
        ++issued;
        if (++stage == Cfg::kStages) {
          stage = 0;
          phase ^= 1u;
        }
        return true;
      };
      for (Walk<kDual, Args> w(a, sh); w.more() && ok; w.next(a, sh)) {
        const bool pair = paired(w.b);
        const int heads = pair ? heads_in(w.h) : 1, h0 = pair ? 2 * w.h : w.h;
        // With a prefix there are many short items, so the first K tiles are loaded before the queries, which wait
        // until the last item's are done with.
        int ahead = 0;
        if constexpr (Args::kPrefix) {
          ok = load(w, w.t0, false, h0);
          if (ok && heads > 1) ok = load(w, w.t0, false, h0 + 1);
          ahead = 1;
          if (!ok) break;
        }
        if (!wait(&sh->q_empty, q_phase ^ 1u)) break;
        q_inflight = true;
        if (lane == 0) {
          const CUtensorMap* tm = &a.tm_q;
          const int tiles = pair ? heads : kDual ? 2 : 1;
          int rows = a.group * a.npt, copies = 1;
          if constexpr (Args::kPrefix) {
            if (w.b < 0) tm = &a.tm_qp;
            rows = a.group * a.p_nodes * (w.b < 0 ? a.p_seqs : 1);
            if (pair) copies = a.copies;
          }
          mbar_arrive_expect_tx(&sh->q_full, tiles * copies * kChunks * 64 * 2 * rows);
          for (int s = 0; s < tiles; ++s) {
            const int tile = pair ? 0 : w.mt * (kDual ? 2 : 1) + s;
            int node = tile * a.npt, seq = w.b;
            if constexpr (Args::kPrefix) {
              if (w.b < 0) {
                seq = a.p_split > 1 ? tile / a.p_split : tile * a.p_seqs;
                node = a.p_split > 1 ? (tile - seq * a.p_split) * a.p_nodes : 0;
              }
            }
            for (int copy = 0; copy < copies; ++copy)
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
                tma_load_4d(s_q + s * Cfg::kTileBytes + c * kSlab + copy * 32 * 128, tm, smem_u32(&sh->q_full), c * 64,
                            (pair ? h0 + s : h0) * a.group, node, seq);
          }
        }
        __syncwarp();
        q_phase ^= 1u;
        // the order in which warp 9 takes them
        if (pair) {
          for (int t = w.t0; t < w.t1 && ok; ++t)
            for (int x = t == w.t0 ? heads : 0; x < 2 * heads && ok; ++x) ok = load(w, t, x >= heads, h0 + x % heads);
        } else if (kDual) {
          for (int t = w.t0; t < w.t1 && ok; ++t) ok = (t - w.t0 < ahead || load(w, t, false, h0)) && load(w, t, true, h0);
        } else {
          ok = ahead > 0 || load(w, w.t0, false, h0);
          for (int t = w.t0 + 1; t < w.t1 && ok; ++t) ok = load(w, t, false, h0) && load(w, t - 1, true, h0);
          ok = ok && load(w, w.t1 - 1, true, h0);
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
    auto to_clean = [&](const Walk<kDual, Args>& w, int t) { return t >= w.shape.cached || (t + 1) * kAtTile > w.shape.len; };
    // Clears V elements of stage `st` that no product may see (whole warp).
    auto clean = [&](const Walk<kDual, Args>& w, int t, int st) {
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
          sh->bad[seg & 1][warp - 9] = 1;
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
    };
    for (Walk<kDual, Args> w(a, sh); w.more(); w.next(a, sh)) {
      const int n_tiles = w.t1 - w.t0;
      if (lane == 0) sh->bad[seg & 1][warp - 9] = 0;
      __syncwarp();
      if (!wait(&sh->q_full, q_phase)) goto mma_done;
      q_phase ^= 1u;
      if (paired(w.b)) {
        // Warp 9 + s issues the products of the pair's head s. Both warps walk the whole ring, and give back at once what
        // is the other's.
        const int s = warp - 9, heads = heads_in(w.h);
        auto next = [&](bool own) {  // the next tile: its stage where it is this warp's, else given back
          const int st = take();
          if (st >= 0 && !own && lane == 0) mbar_arrive(&sh->empty[st]);
          return st;
        };
        for (int i = 0; i < n_tiles; ++i) {
          for (int x = 0; x < heads; ++x) {
            const int k = next(x == s);
            if (k < 0) goto mma_done;
            if (x != s) continue;
            qk(s, s, k);
            tc_commit_warp(&sh->s_full[s], issue);
            tc_commit_warp(&sh->empty[k], issue);
          }
          if (i + 1 == n_tiles) tc_commit_warp(&sh->q_empty, issue);
          if (i == 0 && !wait(&sh->o_empty, o_phase ^ 1u)) goto mma_done;
          for (int x = 0; x < heads; ++x) {
            const int v = next(x == s);
            if (v < 0) goto mma_done;
            if (x != s) continue;
            if (to_clean(w, w.t0 + i)) clean(w, w.t0 + i, v);
            if (!wait(&sh->p_full[s][0], p_phase[s]) || !pv(s, v, i == 0)) goto mma_done;
            tc_commit_warp(&sh->empty[v], issue);
          }
        }
      } else if (kDual) {
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
      if (lane == 0) mbar_arrive(&sh->o_final);  // and what it found in V
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
    uint32_t s_phase = 0, f_phase = 0, ml_phase = 0;
    int seg = 0;
    for (Walk<kDual, Args> w(a, sh); w.more(); w.next(a, sh)) {
      const int n_tiles = w.t1 - w.t0;
      const bool quarter = copied(w.b);                       // the warp sees a quarter of a tile's keys
      const bool pair = paired(w.b);                           // each stream has a head of its own
      constexpr bool joint = !kDual;                          // the streams share one row tile and join their sums
      const int tile = pair ? 0 : w.mt * (kDual ? 2 : 1) + (joint ? 0 : s);
      const bool none = pair && s >= heads_in(w.h);           // no head for this stream
      const int node0 = tile * a.npt;
      int rows = max(0, min(a.npt, a.n - node0)) * a.group;  // of this tile
      if constexpr (Args::kPrefix) {
        if (w.b < 0) {
          const int seq = a.p_split > 1 ? tile / a.p_split : tile * a.p_seqs;
          const int nodes = a.p_split > 1 ? min(a.p_nodes, a.n - (tile - seq * a.p_split) * a.p_nodes)
                                          : min(a.p_seqs, a.n_seqs - seq) * a.n;
          rows = seq < a.n_seqs ? nodes * a.group : 0;
        }
      }
      const bool idle = !quarter && (warp & 3) * 32 >= rows;       // a warp without rows
      const int in_item = quarter ? lane : row;
      const int node = min(node0 + in_item / a.group, a.n - 1);
      float m = -INFINITY, l = 0.0f;
      bool first = true;
      if constexpr (Args::kPrefix) {
        for (int i = 0; quarter && !none && i < n_tiles; ++i) {
          if (!__all_sync(0xffffffffu, mbar_wait(&sh->s_full[s], s_phase, abort_flag, timeout))) goto softmax_done;
          s_phase ^= 1u;
          tc_fence_after();
          const int t = w.t0 + i;
          uint32_t r[32];
          tmem_ld32(ts + (warp & 3) * 32, r);
          uint32_t keep = 0xffffffffu;
          if (t >= w.shape.cached || (t + 1) * kAtTile > w.shape.len) keep = visible_quarter(a, w.shape, w.b, node, t, warp & 3);
          tmem_wait_ld32(r);
          if (keep != 0xffffffffu) {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = (keep >> e) & 1u ? r[e] : 0xff800000u;
          }
          float mx = fmaxf(u2f(r[0]), u2f(r[1]));
#pragma unroll
          for (int e = 2; e < 32; e += 2) mx = fmaxf(fmaxf(mx, u2f(r[e])), u2f(r[e + 1]));
          mx = fmaxf(mx, m);
          const bool grown = m == -INFINITY ? mx > -INFINITY : (mx - m) * sc > kAtRescale;
          if (__any_sync(0xffffffffu, grown)) {
            const float f = grown ? (m == -INFINITY ? 0.0f : exp2f_ftz((m - mx) * sc)) : 1.0f;
            if (!first) rescale_row<kHD>(tmem + lanes + 256 + s * 128, f);
            l *= f;
            if (grown) m = mx;
          }
          const float off = m == -INFINITY ? 0.0f : -m * sc;
          // the other copies' keys have no weight in this one
          const uint32_t none[16] = {};
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c != (warp & 3)) tmem_st16(ts + c * 16, none);
          float2 l0 = make_float2(l, 0.0f), l1 = make_float2(0.0f, 0.0f);
          quarter_weights(ts + (warp & 3) * 16, r, sc, off, l0, l1);
          l = (l0.x + l0.y) + (l1.x + l1.y);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh->p_full[s][0]);
            mbar_arrive(&sh->p_full[s][1]);
          }
          first = false;
        }
      }
      for (int i = joint ? s : 0; !quarter && !none && i < n_tiles; i += joint ? 2 : 1) {
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
            if (!first) rescale_row<kHD>(tmem + lanes + 256 + s * 128, f);  // (the previous product is done:
                                                                          // this tile's scores were issued behind it)
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
      if (joint) {
        ml[seg & 1][s][row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->ml_full);
        if (!__all_sync(0xffffffffu, mbar_wait(&sh->ml_full, ml_phase, abort_flag, timeout))) goto softmax_done;
        ml_phase ^= 1u;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&sh->o_final, f_phase, abort_flag, timeout))) goto softmax_done;
      f_phase ^= 1u;
      tc_fence_after();
      {
        // stream sums to join (one row tile): this warp takes half of the channels of both
        float f0 = 1.0f, f1 = 0.0f;
        if (joint) {
          const float2 u = ml[seg & 1][0][row], v = ml[seg & 1][1][row];
          m = fmaxf(u.x, v.x);
          f0 = u.x == -INFINITY ? 0.0f : exp2f_ftz((u.x - m) * sc);
          f1 = v.x == -INFINITY ? 0.0f : exp2f_ftz((v.x - m) * sc);
          l = u.y * f0 + v.y * f1;
          if (m == INFINITY) l = NAN;  // inf - inf above
        }
        const bool whole = w.t0 == 0 && w.t1 == w.shape.tiles;
        const bool bad = *reinterpret_cast<volatile int*>(&sh->bad[seg & 1][pair ? s : 0]) != 0;
        const bool write = in_item < rows && !none;
        const int kv = pair ? 2 * w.h + s : w.h;
        const int head = kv * a.group + in_item % a.group;
        const long long slot = 2LL * blockIdx.x + (w.t0 > 0 ? 0 : 1);
        int prow = (joint ? 0 : s * kAtTile) + row;
        if constexpr (Args::kPrefix) {
          if (pair) prow = (s * a.copies + (quarter ? warp & 3 : 0)) * rows + in_item;
        }
        // where the rows' parts go, one after another
        constexpr int kRows = Args::kPrefix ? kPfRows : Cfg::kRows;
        float4* part_o = a.part_o + slot * (kHD / 4) * kRows + prow;
        float2* part_ml = a.part_ml + slot * kRows + prow;
        int part_rows = kRows;
        if constexpr (Args::kPrefix) {
          const long long prefix_items = static_cast<long long>(a.heads) * a.p_items;
          const long long item = w.b < 0 ? static_cast<long long>(w.h) * a.p_items + w.mt
                                         : (static_cast<long long>(w.b) * a.own_heads + w.h) * a.m_items + w.mt;
          if (whole) {
            part_rows = w.b < 0 ? a.p_rows : a.rows;
            const int at = pair ? prow : (joint ? 0 : s * (part_rows / 2)) + row;
            const long long before = w.b < 0 ? item * a.p_rows : prefix_items * a.p_rows + item * a.rows;
            part_o = a.whole_o + before * (kHD / 4) + at;
            part_ml = a.whole_ml + before + at;
          }
          if (threadIdx.x == 0) {
            int2* at = a.item_ctas + (w.b < 0 ? 0 : prefix_items) + item;
            if (w.t0 == 0) at->x = static_cast<int>(blockIdx.x);
            if (w.t1 == w.shape.tiles) at->y = static_cast<int>(blockIdx.x);
          }
        }
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        if (!idle) {
          if constexpr (Args::kPrefix) {
            if (quarter && !bad) {
              const uint32_t from = tmem + lanes + 256 + s * 128;
#pragma unroll 1
              for (int c = 0; c < kHD; c += 64) {
                uint32_t o[2][32];
                tmem_ld32(from + c, o[0]);
                tmem_ld32(from + c + 32, o[1]);
                tmem_wait_ld32(o[0]);
                tmem_wait_ld32(o[1]);
                if (write) {
                  float4* dst = part_o + static_cast<long long>(c / 4) * part_rows;
#pragma unroll
                  for (int e = 0; e < 64; e += 4)
                    dst[e / 4 * part_rows] = make_float4(u2f(o[e / 32][e % 32]), u2f(o[e / 32][e % 32 + 1]), u2f(o[e / 32][e % 32 + 2]),
                                                         u2f(o[e / 32][e % 32 + 3]));
                }
              }
            }
          }
          const int cols = quarter && !bad ? 0 : joint ? kHD / 2 : kHD;
          const int col0 = joint ? s * (kHD / 2) : 0;
          const uint32_t to = tmem + lanes + 256 + (joint ? 0 : s * 128) + col0;
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            uint32_t o[16];
            tmem_ld16(to + c, o);
            tmem_wait_ld16(o);
            float x[16];
            if (joint) {
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
                if (quarter && ((j >> 5) & 3) != (warp & 3)) continue;  // (of four parts, the one that has the key)
                const __nv_bfloat16* v = a.v_draft + static_cast<long long>(w.b) * a.draft_seq + j * a.draft_row + kv * kHD + col0 + c;
                for (int e = 0; e < 16; ++e) {
                  const float y = __bfloat162float(v[e]);
                  if (!isfinite(y)) x[e] += y;
                }
              }
            }
            if (write) {
              if (!Args::kPrefix && whole) {
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(x[2 * e] * inv, x[2 * e + 1] * inv);
                __nv_bfloat16* dst = a.out + w.b * a.out_seq + node * a.out_row + static_cast<long long>(head) * kHD + col0 + c;
                st_global_v4(dst, pk[0], pk[1], pk[2], pk[3]);
                st_global_v4(dst + 8, pk[4], pk[5], pk[6], pk[7]);
              } else {  // rows side by side: a warp's store is 512 bytes in a row
                float4* dst = part_o + static_cast<long long>((col0 + c) / 4) * part_rows;
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[e * part_rows] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
              }
            }
          }
          if (write && (!joint || s == 0)) {
            if (Args::kPrefix || !whole) *part_ml = make_float2(m, l);
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

// Adds up each row's parts of a call with a prefix: those of the prefix's item, then those of its own
// sequence's. Block (x, y): rows 32 x .. 32 x + 31 (or 8, see below) of KV head y, counted over the
// sequences' nodes and the head's queries; a warp takes 16 channels. (With more heads than a grid has places
// along y: rows 32 y .., head x.)
struct JoinArgs {
  const float4* part_o;
  const float2* part_ml;
  const float4* whole_o;
  const float2* whole_ml;
  const int2* item_ctas;
  const int32_t* lens;
  const int32_t* prefix_len;
  __nv_bfloat16* out;
  float* lse;
  long long out_row, out_seq;
  int n_seqs, n, heads, group, npt, tiles, m_items, p_nodes, p_seqs, p_split, p_items, rows, p_rows, ctas;
  int pairs, own_heads, copies;
  int capacity, prefix_capacity;
  float scale;
};

// kBatch, kSplit as for k_attn_combine: lanes share a row where there are fewer blocks than SMs otherwise, and more parts
// are in flight where an item has many (one row tile).
template <int kHD, int kBatch, int kSplit, bool kHeadsAlongX = false>
__global__ void __launch_bounds__(kHD * 2) k_prefix_join(const __grid_constant__ JoinArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kLanes = 32 / kSplit;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = kHeadsAlongX ? blockIdx.x : blockIdx.y;
  const int r = (kHeadsAlongX ? blockIdx.y : blockIdx.x) * kLanes + lane % kLanes;
  const int per_seq = a.n * a.group;
  const int b = r / per_seq, in_seq = r - b * per_seq, node = in_seq / a.group, g = in_seq - node * a.group;
  const bool there = b < a.n_seqs;
  // The row's place in the prefix's items and in its own sequence's.
  struct Place {
    const float4* whole_o;
    const float2* whole_ml;
    int whole_rows, at;  // at: within the rows of a part that was cut
    int first, parts;    // CTAs
    int of, apart;       // parts of a CTA's (4 of copied rows) and the rows between them
  } at[2] = {};
  bool live = false;
  if (there) {
    const int tile_rows = a.tiles == 2 ? kAtTile : 0;
    const long long prefix_items = static_cast<long long>(a.heads) * a.p_items;
    // `in`: the row's place among those of its item's stored part
    auto place = [&](int i, int in, int in_cut, long long before, int rows, int copies, int apart) {
      at[i].whole_rows = rows;
      at[i].whole_o = a.whole_o + before * (kHD / 4) + in;
      at[i].whole_ml = a.whole_ml + before + in;
      at[i].at = in_cut;
      at[i].of = copies;
      at[i].apart = apart;
    };
    const int p_tile = a.p_split > 1 ? b * a.p_split + node / a.p_nodes : b / a.p_seqs;
    const int p_row = a.p_split > 1 ? (node % a.p_nodes) * a.group + g : (b % a.p_seqs) * per_seq + in_seq;
    const long long p_item = static_cast<long long>(h) * a.p_items + p_tile / a.tiles;
    const int tile = node / a.npt, own_row = (node - tile * a.npt) * a.group + g;
    const long long item = (static_cast<long long>(b) * a.own_heads + (a.pairs ? h >> 1 : h)) * a.m_items + tile / a.tiles;
    // (loads that do not wait for one another; without prefix rows what lies there is not used)
    const int prefix = *a.prefix_len, len = a.lens[b];
    const int2 c[2] = {a.item_ctas[p_item], a.item_ctas[prefix_items + item]};
    const int p_s = p_tile % a.tiles, s = tile % a.tiles, in_pair = (h & 1) * a.copies * per_seq + in_seq;
    place(0, p_s * (a.p_rows / 2) + p_row, p_s * tile_rows + p_row, p_item * a.p_rows, a.p_rows, 1, 0);
    place(1, a.pairs ? in_pair : s * (a.rows / 2) + own_row, a.pairs ? in_pair : s * tile_rows + own_row,
          prefix_items * a.p_rows + item * a.rows, a.rows, a.copies, per_seq);
    live = len >= 0 && len <= a.capacity && prefix >= 0 && prefix <= a.prefix_capacity;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      at[i].first = min(max(c[i].x, 0), a.ctas - 1);
      at[i].parts = i == 0 && prefix <= 0 ? 0 : min(max(c[i].y, at[i].first), a.ctas - 1) - at[i].first + 1;
    }
  }
  if (kSplit == 1 && !live) return;
  const int parts_0 = at[0].parts * at[0].of, parts = parts_0 + at[1].parts * at[1].of;
  const float sc = a.scale * kAtLog2e;
  float m = -INFINITY, l = 0.0f;
  float4 x[4] = {};
  for (int i0 = live ? lane / kLanes : parts; i0 < parts; i0 += kBatch * kSplit) {
    float2 ml[kBatch];
    float4 v[kBatch][4];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      int i = i0 + j * kSplit;
      if (i >= parts) break;
      const bool own = i >= parts_0;
      if (own) i -= parts_0;
      const Place& p = own ? at[1] : at[0];
      const bool copied = kBatch < 8 && p.of > 1;  // (at most 32 rows of all sequences are one row tile, without copies)
      const int in_cta = copied ? i & 3 : 0;
      if (copied) i >>= 2;
      const float4* o = p.whole_o;
      const float2* w = p.whole_ml;
      int stride = p.whole_rows;
      if (p.parts > 1) {  // the last part of its first CTA, the first part of the others
        const long long slot = i == 0 ? 2LL * p.first + 1 : 2LL * (p.first + i);
        o = a.part_o + slot * (kHD / 4) * kPfRows + p.at;
        w = a.part_ml + slot * kPfRows + p.at;
        stride = kPfRows;
      }
      o += in_cta * p.apart;
      w += in_cta * p.apart;
      ml[j] = *w;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = o[static_cast<long long>(warp * 4 + e) * stride];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (i0 + j * kSplit >= parts) break;
      const float mx = fmaxf(m, ml[j].x);
      const float f = m == -INFINITY ? 0.0f : exp2f_ftz((m - mx) * sc);
      const float k = ml[j].x == -INFINITY ? 0.0f : exp2f_ftz((ml[j].x - mx) * sc);
      m = mx;
      l = l * f + ml[j].y * k;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e].x = x[e].x * f + v[j][e].x * k;
        x[e].y = x[e].y * f + v[j][e].y * k;
        x[e].z = x[e].z * f + v[j][e].z * k;
        x[e].w = x[e].w * f + v[j][e].w * k;
      }
    }
  }
  if constexpr (kSplit > 1) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) {
      const float m1 = __shfl_xor_sync(0xffffffffu, m, o), l1 = __shfl_xor_sync(0xffffffffu, l, o);
      const float mx = fmaxf(m, m1);
      const float f = m == -INFINITY ? 0.0f : exp2f_ftz((m - mx) * sc);
      const float k = m1 == -INFINITY ? 0.0f : exp2f_ftz((m1 - mx) * sc);
      m = mx;
      l = l * f + l1 * k;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e].x = x[e].x * f + __shfl_xor_sync(0xffffffffu, x[e].x, o) * k;
        x[e].y = x[e].y * f + __shfl_xor_sync(0xffffffffu, x[e].y, o) * k;
        x[e].z = x[e].z * f + __shfl_xor_sync(0xffffffffu, x[e].z, o) * k;
        x[e].w = x[e].w * f + __shfl_xor_sync(0xffffffffu, x[e].w, o) * k;
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
  const int head = h * a.group + g;
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

template <int kHD, bool kDual, class Args>
static rf_status launch_attn(const Args& a, int ctas, cudaStream_t s) {
  static uint64_t done = 0;
  using Cfg = AttnCfg<kHD, kDual>;
  static_assert(Cfg::kSmem <= 227 * 1024, "shared memory beyond the 227 KB a CTA may hold");
  static_assert(sizeof(AttnExchange) <= Cfg::kTileBytes, "the exchange does not fit into a query tile");
  rf_status st = set_smem_attr(reinterpret_cast<const void*>(&k_attn<kHD, kDual, Args>), Cfg::kSmem, &done);
  if (st != RF_OK) return st;
  ProfScope prof(s, RF_STAGE_ATTENTION);
  // CTAs of unlike work are launched when the kernel before is done: those that come up as its CTAs leave take their
  // places in the order in which these finish, and the ones with the prefix's products then end up side by side (64
  // sequences over 16,384 shared rows: 72 us as dependents, 63 so).
  if (Args::kPrefix && kDual) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kAtThreads);
    cfg.dynamicSmemBytes = Cfg::kSmem;
    cfg.stream = s;
    return cuda_check(cudaLaunchKernelEx(&cfg, k_attn<kHD, kDual, Args>, a), "k_attn launch");
  }
  return cuda_check(launch_dependent(k_attn<kHD, kDual, Args>, dim3(static_cast<unsigned>(ctas)), dim3(kAtThreads), Cfg::kSmem, s, 1, a),
                    "k_attn launch");
}

}  // namespace rf

using namespace rf;

extern "C" size_t rf_attn_workspace_bytes(const rf_attn_desc* desc) {
  if (check_attn_desc(desc) != RF_OK) return 0;
  return attn_layout(desc, nullptr).bytes;
}

// Checks of the tensors, and the kernel's arguments from them (all but its workspace); `tiles`: row tiles
// of an item.
static rf_status attn_args(const rf_attn_desc* d, const rf_bf16* q, const rf_bf16* k_cache, const rf_bf16* v_cache,
                           const int32_t* lens, const rf_bf16* k_draft, const rf_bf16* v_draft, const uint64_t* tree_mask,
                           rf_bf16* out, float* lse, int32_t* dev_status, int tiles, AttnArgs* args) {
  if (!q || !k_cache || !v_cache || !lens || !k_draft || !v_draft || !out)
    return fail(RF_ERR_INVALID_ARG, "tensor pointers must be non-NULL");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_draft) || !aligned16(v_draft) ||
      !aligned16(out))
    return fail(RF_ERR_ALIGN, "row buffers must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(lens) & 3u) || (reinterpret_cast<uintptr_t>(tree_mask) & 7u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(RF_ERR_ALIGN, "arrays must be aligned to their elements");
  AttnArgs& a = *args;
  const uint64_t H = d->n_kv_heads, n = d->n_nodes, B = d->n_seqs;
  a.lens = lens;
  a.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  a.v_draft = reinterpret_cast<const __nv_bfloat16*>(v_draft);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.dev_status = dev_status;
  a.timeout_ns = wait_timeout_ns();
  a.out_row = d->out_row_stride;
  a.out_seq = d->out_seq_stride;
  a.draft_row = d->draft_row_stride;
  a.draft_seq = d->draft_seq_stride;
  a.n_seqs = static_cast<int>(B);
  a.heads = static_cast<int>(H);
  a.group = static_cast<int>(d->n_q_heads / d->n_kv_heads);
  a.npt = kAtTile / a.group;
  a.n = static_cast<int>(n);
  a.capacity = static_cast<int>(d->capacity);
  a.words = static_cast<int>(RF_TREE_WORDS(n));
  a.scale = static_cast<float>(d->scale);
  const int64_t per = static_cast<int64_t>(a.npt) * tiles;  // nodes of an item
  a.m_items = static_cast<int>((n + per - 1) / per);
  int64_t draft_sum = 0;
  for (int64_t mt = 0; mt < a.m_items; ++mt) {
    const int64_t seen = tree_mask != nullptr ? static_cast<int64_t>(n) : std::min<int64_t>(n, (mt + 1) * per);
    draft_sum += (seen + kAtTile - 1) / kAtTile;
  }
  if (draft_sum >= (int64_t(1) << 31)) return fail(RF_ERR_SHAPE, "n_nodes is too large");
  a.draft_sum = static_cast<int>(draft_sum);
  return RF_OK;
}

// The tensor maps.
static rf_status attn_maps(const rf_attn_desc* d, const rf_bf16* q, const rf_bf16* k_cache, const rf_bf16* v_cache,
                           const rf_bf16* k_draft, const rf_bf16* v_draft, int nodes, AttnArgs* args) {
  AttnArgs& a = *args;
  const uint64_t hd = d->head_dim, H = d->n_kv_heads, Hq = d->n_q_heads, n = d->n_nodes, B = d->n_seqs, cap = d->capacity;
  rf_status st;
  // a box of a row tile: every head of the group, `nodes` nodes
  if ((st = make_tmap_bf16_4d(&a.tm_q, q, {hd, Hq, n, B}, {hd, (uint64_t)d->q_row_stride, (uint64_t)d->q_seq_stride},
                              {64, (uint32_t)a.group, (uint32_t)nodes, 1})) != RF_OK)
    return st;
  const uint64_t cs[3] = {hd, (uint64_t)d->cache_row_stride, (uint64_t)d->cache_seq_stride};
  const uint64_t ds[3] = {hd, (uint64_t)d->draft_row_stride, (uint64_t)d->draft_seq_stride};
  const uint64_t cd[4] = {hd, H, cap, B}, dd[4] = {hd, H, n, B};
  const uint32_t box[4] = {64, 1, kAtTile, 1};
  if ((st = make_tmap_bf16_4d(&a.tm_k, k_cache, cd, cs, box)) != RF_OK) return st;
  if ((st = make_tmap_bf16_4d(&a.tm_v, v_cache, cd, cs, box)) != RF_OK) return st;
  if ((st = make_tmap_bf16_4d(&a.tm_kd, k_draft, dd, ds, box)) != RF_OK) return st;
  return make_tmap_bf16_4d(&a.tm_vd, v_draft, dd, ds, box);
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
  const AttnLayout lay = attn_layout(d, workspace);
  AttnArgs a{};
  if ((st = attn_args(d, q, k_cache, v_cache, lens, k_draft, v_draft, tree_mask, out, lse, dev_status, lay.tiles, &a)) != RF_OK)
    return st;
  if (workspace == nullptr || workspace_bytes < lay.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(RF_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", lay.bytes, workspace_bytes);
  int sms = 0;
  if ((st = current_device(&sms)) != RF_OK) return st;
  if ((st = attn_maps(d, q, k_cache, v_cache, k_draft, v_draft, a.npt, &a)) != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.part_o = lay.part_o;
  a.part_ml = lay.part_ml;
  a.plan = lay.plan;
  const uint64_t hd = d->head_dim, H = d->n_kv_heads, n = d->n_nodes, B = d->n_seqs, cap = d->capacity;
  // no more CTAs than weight, which is at least the tiles
  const int64_t most = static_cast<int64_t>(B * H) * (a.m_items * static_cast<int64_t>((cap + kAtTile - 1) / kAtTile + kAtItemCost) + a.draft_sum);
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
  c.group = a.group;
  c.npt = a.npt;
  c.tiles = lay.tiles;
  c.ctas = ctas;
  c.scale = a.scale;
  // rows of an item that exist, in a tile's numbering (the first tile's are followed by a gap)
  const int tile_rows = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(n) * a.group, a.npt * a.group));
  const int rows = lay.tiles == 2 ? 2 * kAtTile : tile_rows;
  const bool few = rows <= 32 && B * H * a.m_items * 8 <= ctas;
  const dim3 grid(static_cast<unsigned>(ctas - 1), static_cast<unsigned>((rows + (few ? 7 : 31)) / (few ? 8 : 32)));
  ProfScope prof(s, RF_STAGE_ATTN_COMBINE);
  void (*combine)(CombineArgs) = hd == 128 ? (few ? k_attn_combine<128, 8, 4> : k_attn_combine<128, 4, 1>)
                                           : (few ? k_attn_combine<64, 8, 4> : k_attn_combine<64, 4, 1>);
  return cuda_check(launch_dependent(combine, grid, dim3(static_cast<unsigned>(2 * hd)), 0, s, 1, c),
                    "k_attn_combine launch");
}

// ------------------------------------------------------------------- with a prefix
static rf_status check_prefix_desc(const rf_prefix_attn_desc* d) {
  if (d == nullptr) return fail(RF_ERR_INVALID_ARG, "desc is NULL");
  const rf_status st = check_attn_desc(&d->attn);
  if (st != RF_OK) return st;
  if (d->prefix_capacity <= 0) return fail(RF_ERR_INVALID_ARG, "need prefix_capacity > 0");
  if (d->prefix_capacity > (int64_t(1) << 30)) return fail(RF_ERR_SHAPE, "need prefix_capacity <= 2^30");
  if (d->attn.n_seqs * d->attn.n_nodes > (int64_t(1) << 28) / d->attn.n_q_heads)
    return fail(RF_ERR_SHAPE, "need n_seqs * n_nodes * n_q_heads <= 2^28");
  if (d->prefix_row_stride < d->attn.n_kv_heads * d->attn.head_dim || d->prefix_row_stride % 8)
    return fail(RF_ERR_ALIGN, "prefix_row_stride must be a multiple of 8, >= n_kv_heads*head_dim");
  if (d->prefix_row_stride >= (int64_t(1) << 39)) return fail(RF_ERR_SHAPE, "strides must be < 2^39");
  return RF_OK;
}

struct PrefixLayout {
  float4 *part_o, *whole_o;
  float2 *part_ml, *whole_ml;
  int2* item_ctas;
  int tiles, p_nodes, p_seqs, p_split, p_items, m_items, rows, p_rows, pairs, own_heads, copies;
  size_t bytes;
};

static PrefixLayout prefix_layout(const rf_attn_desc* d, void* ws) {
  PrefixLayout l;
  const int64_t group = d->n_q_heads / d->n_kv_heads, npt = kAtTile / group, n = d->n_nodes, B = d->n_seqs, H = d->n_kv_heads;
  l.tiles = B * n * group > kAtTile ? 2 : 1;
  l.p_nodes = static_cast<int>(std::min(n, npt));
  l.p_seqs = static_cast<int>(n <= npt ? std::min(npt / n, std::max<int64_t>(B, 1)) : 1);
  l.p_split = static_cast<int>(n <= npt ? 1 : (n + npt - 1) / npt);
  const int64_t p_tiles = n <= npt ? (B + l.p_seqs - 1) / l.p_seqs : B * l.p_split;
  l.p_items = static_cast<int>((p_tiles + l.tiles - 1) / l.tiles);
  l.m_items = static_cast<int>((n + npt * l.tiles - 1) / (npt * l.tiles));
  l.p_rows = static_cast<int>(l.tiles * group * l.p_nodes * l.p_seqs);
  l.pairs = l.tiles == 2 && n <= npt;
  l.own_heads = static_cast<int>(l.pairs ? (H + 1) / 2 : H);
  l.copies = l.pairs && n * group <= 32 ? 4 : 1;
  l.rows = static_cast<int>(l.pairs ? 2 * l.copies * n * group : n <= npt ? n * group : l.tiles * npt * group);
  const size_t cut = static_cast<size_t>(2 * kAtMaxCtas) * kPfRows;
  const size_t whole = static_cast<size_t>(H) * l.p_items * l.p_rows + static_cast<size_t>(B) * l.own_heads * l.m_items * l.rows;
  Carve c(ws);
  l.part_o = c.take<float4>(cut * d->head_dim / 4);
  l.part_ml = c.take<float2>(cut);
  l.whole_o = c.take<float4>(whole * d->head_dim / 4);
  l.whole_ml = c.take<float2>(whole);
  l.item_ctas = c.take<int2>(static_cast<size_t>(H) * l.p_items + static_cast<size_t>(B) * l.own_heads * l.m_items);
  l.bytes = c.bytes();
  return l;
}

extern "C" size_t rf_prefix_attn_workspace_bytes(const rf_prefix_attn_desc* desc) {
  if (check_prefix_desc(desc) != RF_OK) return 0;
  return prefix_layout(&desc->attn, nullptr).bytes;
}

extern "C" rf_status rf_prefix_attention(const rf_prefix_attn_desc* desc, const rf_bf16* q, const rf_bf16* k_prefix,
                                         const rf_bf16* v_prefix, const int32_t* prefix_len, const rf_bf16* k_cache,
                                         const rf_bf16* v_cache, const int32_t* lens, const rf_bf16* k_draft,
                                         const rf_bf16* v_draft, const uint64_t* tree_mask, rf_bf16* out, float* lse,
                                         int32_t* dev_status, void* workspace, size_t workspace_bytes, rf_stream_t stream) {
  clear_error();
  rf_status st = check_prefix_desc(desc);
  if (st != RF_OK) return st;
  const rf_attn_desc* d = &desc->attn;
  if (tree_mask != nullptr && d->n_nodes > RF_TREE_MAX_NODES)
    return fail(RF_ERR_SHAPE, "n_nodes must be <= %d with a mask", RF_TREE_MAX_NODES);
  if (d->n_seqs == 0) return RF_OK;
  const PrefixLayout lay = prefix_layout(d, workspace);
  PrefixArgs a{};
  if ((st = attn_args(d, q, k_cache, v_cache, lens, k_draft, v_draft, tree_mask, out, lse, dev_status, lay.tiles, &a)) != RF_OK)
    return st;
  if (!k_prefix || !v_prefix || !prefix_len) return fail(RF_ERR_INVALID_ARG, "tensor pointers must be non-NULL");
  if (!aligned16(k_prefix) || !aligned16(v_prefix)) return fail(RF_ERR_ALIGN, "row buffers must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(prefix_len) & 3u) return fail(RF_ERR_ALIGN, "arrays must be aligned to their elements");
  if (workspace == nullptr || workspace_bytes < lay.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(RF_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", lay.bytes, workspace_bytes);
  int sms = 0;
  if ((st = current_device(&sms)) != RF_OK) return st;
  if ((st = attn_maps(d, q, k_cache, v_cache, k_draft, v_draft, lay.p_nodes, &a)) != RF_OK) return st;
  const uint64_t hd = d->head_dim, H = d->n_kv_heads, Hq = d->n_q_heads, n = d->n_nodes, B = d->n_seqs;
  const uint64_t ps[3] = {hd, (uint64_t)desc->prefix_row_stride, (uint64_t)desc->prefix_row_stride};
  const uint64_t pd[4] = {hd, H, (uint64_t)desc->prefix_capacity, 1};
  const uint32_t box[4] = {64, 1, kAtTile, 1};
  if ((st = make_tmap_bf16_4d(&a.tm_qp, q, {hd, Hq, n, B}, {hd, (uint64_t)d->q_row_stride, (uint64_t)d->q_seq_stride},
                              {64, (uint32_t)a.group, (uint32_t)lay.p_nodes, (uint32_t)lay.p_seqs})) != RF_OK)
    return st;
  if ((st = make_tmap_bf16_4d(&a.tm_kp, k_prefix, pd, ps, box)) != RF_OK) return st;
  if ((st = make_tmap_bf16_4d(&a.tm_vp, v_prefix, pd, ps, box)) != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.part_o = lay.part_o;
  a.part_ml = lay.part_ml;
  a.whole_o = lay.whole_o;
  a.whole_ml = lay.whole_ml;
  a.item_ctas = lay.item_ctas;
  a.prefix_len = prefix_len;
  a.prefix_capacity = static_cast<int>(desc->prefix_capacity);
  a.p_nodes = lay.p_nodes;
  a.p_seqs = lay.p_seqs;
  a.p_split = lay.p_split;
  a.p_items = lay.p_items;
  // With two row tiles, in tenths of a microsecond: a prefix tile takes 1.7 (products) to 2.0 (beside CTAs that stream
  // caches), a tile of a pair, two of each head's, 1.8, an item's first and last steps some 6. Where there are no pairs a
  // tile is as long whoever's it is, and an item weighs four of them, as in rf_tree_attention.
  a.w_item = lay.pairs ? 60 : 68;
  a.w_prefix = lay.pairs ? 20 : 17;
  a.w_own = lay.pairs ? 18 : 17;
  a.in_step = static_cast<int>((32 << 20) / (static_cast<int64_t>(kAtTile) * 4 * hd * H));  // 32 MB of keys and values
  a.pairs = lay.pairs;
  a.own_heads = lay.own_heads;
  a.copies = lay.copies;
  a.rows = lay.rows;
  a.p_rows = lay.p_rows;
  const int ctas = std::min(sms, kAtMaxCtas);
  if (hd == 128) st = lay.tiles == 2 ? launch_attn<128, true>(a, ctas, s) : launch_attn<128, false>(a, ctas, s);
  else st = lay.tiles == 2 ? launch_attn<64, true>(a, ctas, s) : launch_attn<64, false>(a, ctas, s);
  if (st != RF_OK) return st;
  JoinArgs j{};
  j.part_o = lay.part_o;
  j.part_ml = lay.part_ml;
  j.whole_o = lay.whole_o;
  j.whole_ml = lay.whole_ml;
  j.item_ctas = lay.item_ctas;
  j.lens = lens;
  j.prefix_len = prefix_len;
  j.out = a.out;
  j.lse = lse;
  j.out_row = a.out_row;
  j.out_seq = a.out_seq;
  j.n_seqs = a.n_seqs;
  j.n = a.n;
  j.heads = a.heads;
  j.group = a.group;
  j.npt = a.npt;
  j.tiles = lay.tiles;
  j.m_items = a.m_items;
  j.p_nodes = lay.p_nodes;
  j.p_seqs = lay.p_seqs;
  j.p_split = lay.p_split;
  j.p_items = lay.p_items;
  j.copies = lay.copies;
  j.pairs = lay.pairs;
  j.own_heads = lay.own_heads;
  j.rows = lay.rows;
  j.p_rows = lay.p_rows;
  j.ctas = ctas;
  j.capacity = a.capacity;
  j.prefix_capacity = a.prefix_capacity;
  j.scale = a.scale;
  const int64_t rows = static_cast<int64_t>(B * n) * a.group;  // of a KV head
  const bool few = (rows + 31) / 32 * static_cast<int64_t>(H) < sms, fewest = rows <= 32;
  const int64_t blocks = (rows + (few ? 7 : 31)) / (few ? 8 : 32);
  // (n_seqs * n_nodes * n_q_heads <= 2^28: with more than 65,535 heads the blocks of one are 512 at most)
  const bool along_x = H > 65535;
  const dim3 grid = along_x ? dim3(static_cast<unsigned>(H), static_cast<unsigned>(blocks))
                            : dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(H));
  ProfScope prof(s, RF_STAGE_ATTN_COMBINE);
  void (*join)(JoinArgs) =
      along_x     ? (hd == 128 ? k_prefix_join<128, 4, 1, true> : k_prefix_join<64, 4, 1, true>)
      : hd == 128 ? (!few ? k_prefix_join<128, 4, 1> : fewest ? k_prefix_join<128, 8, 4> : k_prefix_join<128, 4, 4>)
                  : (!few ? k_prefix_join<64, 4, 1> : fewest ? k_prefix_join<64, 8, 4> : k_prefix_join<64, 4, 4>);
  return cuda_check(launch_dependent(join, grid, dim3(static_cast<unsigned>(2 * hd)), 0, s, 1, j), "k_prefix_join launch");
}
