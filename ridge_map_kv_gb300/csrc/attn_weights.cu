// Accumulated attention weights of cached rows (rf_attn_weights).
//
// score_out[t] = decay score_in[t] + sum over queries c that see t of
//                exp(scale q_c.k_t - lse_c).
// The statistics are known, so a key's sum needs no other key: each key tile is read
// once, and what is written is one number a key. The product is taken as S = K Qᵀ, keys
// along the TMEM lanes: a thread owns a key and sums over its columns, so there is no
// reduction across threads but that of two warps where they share a key's columns.
//
// Bound: the keys' bytes up to a few hundred queries (2 hd bytes a key against 2 R hd
// flops and R exponentials); beyond, the exponentials and the product. Measured (128 channels):
// 16 paths of up to 7 nodes, 32 heads on 8, over 913 to 16,384 rows: 62 us, 4.9 TB/s; the last 64
// of 32,768 rows, 20 heads on 2: 24 us, of which 8 are launch and queries (27.5 us with the
// queries gathered row by row); the exponentials of 672 columns a key fill most of the rest.
//
// The queries of a KV head (nodes of the path times query heads, R of them) stay in
// shared memory, up to 640 rows of 128 channels; the product takes them in steps of up
// to 256 columns, two of which are in TMEM at a time. More queries are taken in further
// launches. Units (128-key tiles) of all sequences and heads are cut into equal shares,
// one per CTA.
//
//   warps 0-3, 4-7   sums: a thread is a key. Where a tile takes one step, the two groups
//                    of warps take alternate tiles (a tile's work is a chain of waits and
//                    few instructions then, and two chains run side by side); else the
//                    first group takes a step's first half of the columns, the other the
//                    second, and the halves meet in shared memory
//   warp 8           TMA: key tiles, in 64-channel slabs
//   warp 9           MMA
//   warps 10-13      the queries of the next (sequence, head), into the other of two buffers
//                    (or, where two do not fit, once the one is free): all nodes of a sequence
//                    as one TMA box a slab, those of a path gathered row by row
#include <algorithm>
#include <cmath>

#include "rf_device.cuh"
#include "rf_host.h"

namespace rf {

constexpr int kWtTile = 128;
constexpr int kWtThreads = 448;
constexpr int kWtLoaders = 128;      // threads of warps 10-13
constexpr int kWtMaxSeqs = 1024;     // lengths and counts are kept in shared memory
constexpr int kWtStep = 256;         // columns of a step
constexpr int kWtMaxStages = 12;
constexpr int kWtSlab = kWtTile * 128;
constexpr int kWtQBytes = 640 * 128 * 2;  // the most that queries may take
constexpr int kWtNever = INT32_MIN;       // position of a column that counts for no key
constexpr float kWtLog2e = 1.4426950408889634f;

struct WeightArgs {
  CUtensorMap tm_k, tm_q;  // tm_q: boxes of j_max nodes, if box
  const __nv_bfloat16* q;
  const float* lse;
  const int32_t* path;
  const int32_t* n_path;
  const int32_t* lens;
  const float* score_in;  // nullptr: decay is 0
  float* score_out;
  int32_t* dev_status;
  uint64_t timeout_ns;
  long long q_row, q_seq;
  int n_seqs, heads, group, n, capacity;
  int j0, j_max;   // this launch takes path positions j0 .. j0 + j_max - 1
  bool box;        // queries come as boxes
  int rows_cap;    // query rows of one buffer (a multiple of 16)
  int bufs;        // query buffers: 2 where that leaves the ring its stages, else 1
  int stages;
  float scale, decay;
};

struct WeightShared {
  uint64_t full[kWtMaxStages], empty[kWtMaxStages];
  uint64_t q_full[2], q_empty[2], q_box[2], t_full[2], t_empty[2], half_full[4], mma_done;
  float half[4][kWtTile];  // the second warps' sums
  int b, h, t;             // first unit of the share
  long long units;
  uint32_t tmem;
  int abort;
};

// A CTA's share, unit by unit; a thread alone or (kWarp) a converged warp walks it.
template <bool kWarp>
struct WeightWalk {
  const int *len, *cnt;
  int b, h, t, tiles, queries;  // queries: path positions of the sequence
  long long left;
  template <class T>
  static __device__ __forceinline__ T same(T x) {
    if constexpr (kWarp) return uniform(x);
    else return x;
  }
  __device__ __forceinline__ void look() {
    tiles = same((len[b] + kWtTile - 1) / kWtTile);
    queries = same(cnt[b]);
  }
  __device__ __forceinline__ WeightWalk(const WeightShared* sh, const int* len_, const int* cnt_) : len(len_), cnt(cnt_) {
    b = same(sh->b);
    h = same(sh->h);
    t = same(sh->t);
    left = same(sh->units);
    tiles = queries = 0;
    if (left > 0) look();
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  // True when the next unit belongs to another sequence or head.
  __device__ __forceinline__ bool last_of_item() const { return t + 1 == tiles || left == 1; }
  __device__ __forceinline__ void next(const WeightArgs& a) {
    --left;
    if (++t < tiles || left <= 0) return;
    t = 0;
    if (++h == a.heads) {
      h = 0;
      do ++b;
      while (same(len[b]) <= 0);
      look();
    }
  }
  // Query rows of the item in this launch, and the columns and number of its steps.
  __device__ __forceinline__ int rows(const WeightArgs& a) const { return min(max(queries - a.j0, 0), a.j_max) * a.group; }
};
__device__ __forceinline__ int weight_steps(int rows) { return max(1, (rows + kWtStep - 1) / kWtStep); }
// Columns of a step: equal shares, multiples of 16.
__device__ __forceinline__ int weight_cols(int rows) {
  const int s = weight_steps(rows);
  return max(16, ((rows + s - 1) / s + 15) & ~15);
}

// Adds the weights 2^(s sc + nl) of N columns.
template <int N>
__device__ __forceinline__ void add_weights(const uint32_t (&r)[N], const float* nl, float sc, float2& s0, float2& s1) {
  const float2 sc2 = make_float2(sc, sc);
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(nl + i);
    const float2 x = fma_x2(make_float2(u2f(r[i]), u2f(r[i + 1])), sc2, make_float2(l.x, l.y));
    const float2 y = fma_x2(make_float2(u2f(r[i + 2]), u2f(r[i + 3])), sc2, make_float2(l.z, l.w));
    s0 = add_x2(s0, make_float2(exp2f_ftz(x.x), exp2f_ftz(x.y)));
    s1 = add_x2(s1, make_float2(exp2f_ftz(y.x), exp2f_ftz(y.y)));
  }
}

template <int kHD>
__global__ void __launch_bounds__(kWtThreads, 1) k_attn_weights(const __grid_constant__ WeightArgs a) {
  constexpr int kSlabs = kHD / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int q_slab = a.rows_cap * 128;  // a multiple of 1 KB: rows_cap is one of 16
  uint8_t* p = smem + a.bufs * kSlabs * q_slab + a.stages * kWtSlab;
  WeightShared* sh = reinterpret_cast<WeightShared*>(p);
  float* neg_lse = reinterpret_cast<float*>(p + ((sizeof(WeightShared) + 15) & ~size_t(15)));  // -lse log2 e, a column each
  int* position = reinterpret_cast<int*>(neg_lse + a.bufs * a.rows_cap);  // a column's path position, from j0
  int* len = position + a.bufs * a.rows_cap;
  int* cnt = len + a.n_seqs;
  const uint32_t s_q = smem_u32(smem), s_ring = s_q + a.bufs * kSlabs * q_slab;
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh->abort;
  const uint64_t timeout = a.timeout_ns;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->q_full[i], kWtLoaders);
      mbar_init(&sh->q_empty[i], 9);
      mbar_init(&sh->q_box[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->t_full[i], 1);
      mbar_init(&sh->t_empty[i], 8);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh->half_full[i], 4);
    mbar_init(&sh->mma_done, 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) tma_prefetch_desc(&a.tm_k);
  if (warp == 10 && lane == 0 && a.box) tma_prefetch_desc(&a.tm_q);
  if (warp == 9) {
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();
  // Lengths and counts, one warp a sequence: -1 for what may not be touched.
  for (int b = warp; b < a.n_seqs; b += kWtThreads / 32) {
    const int m = a.lens[b], c = a.n_path != nullptr ? a.n_path[b] : a.n;
    bool bad = m < 0 || m > a.capacity || c < 0 || c > a.n || c > m;
    if (!bad && a.path != nullptr)
      for (int j = lane; j < c; j += 32) {
        const int i = a.path[static_cast<long long>(b) * a.n + j];
        bad |= i < 0 || i >= a.n;
      }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (bad) record_status(a.dev_status, RF_ERR_INVALID_ARG);
      len[b] = bad || (a.j0 > 0 && c <= a.j0) ? -1 : m;
      cnt[b] = bad ? 0 : c;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {  // this CTA's share
    auto units_of = [&](int b) -> long long {
      return b < a.n_seqs ? static_cast<long long>(a.heads) * ((max(len[b], 0) + kWtTile - 1) / kWtTile) : 0;
    };
    long long total = 0;
    for (int b = lane; b < a.n_seqs; b += 32) total += units_of(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const long long shares = min(static_cast<long long>(gridDim.x), total);
    long long units = 0;
    int fb = 0, fh = 0, ft = 0;
    if (blockIdx.x < shares) {
      const long long first = share_start(total, static_cast<int>(blockIdx.x), static_cast<int>(shares));
      units = share_start(total, static_cast<int>(blockIdx.x) + 1, static_cast<int>(shares)) - first;
      long long base = 0;
      for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
        const long long own = units_of(b0 + lane);
        long long x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, first < base + x);
        if (hit) {
          const int at = __ffs(hit) - 1;
          fb = b0 + at;
          const long long r = first - base - __shfl_sync(0xffffffffu, x - own, at);
          const long long per_head = quick_div(__shfl_sync(0xffffffffu, own, at), a.heads);
          fh = static_cast<int>(quick_div(r, per_head));
          ft = static_cast<int>(r - fh * per_head);
          break;
        }
        base += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    if (lane == 0) {
      sh->b = fb;
      sh->h = fh;
      sh->t = ft;
      sh->units = units;
    }
  }
  __syncthreads();
  const uint32_t tmem = uniform(sh->tmem);

  if (warp == 8) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      for (WeightWalk<false> w(sh, len, cnt); w.more(); w.next(a)) {
#pragma unroll
        for (int c = 0; c < kSlabs; ++c) {
          if (!mbar_wait(&sh->empty[stage], phase ^ 1u, abort_flag, timeout)) goto load_done;
          mbar_arrive_expect_tx(&sh->full[stage], kWtSlab);
          tma_load_4d(s_ring + stage * kWtSlab, &a.tm_k, smem_u32(&sh->full[stage]), c * 64, w.h, w.t * kWtTile, w.b);
          ++issued;
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    load_done:
      int dummy = 0;
      for (long long i = (issued > a.stages ? issued - a.stages : 0); i < issued; ++i)
        mbar_wait(&sh->full[i % a.stages], static_cast<uint32_t>((i / a.stages) & 1), &dummy, timeout);
    }
  } else if (warp == 9) {
    const uint32_t issue = lane == 0;
    int stage = 0;
    uint32_t phase = 0, step = 0, item = 0;
    int qb = 0;         // query buffer of the item
    int steps = 0, cols = 0;
    uint32_t idesc = 0;
    bool fresh = true;  // the next unit starts an item
    auto wait = [&](uint64_t* bar, uint32_t par) {  // whole warp
      const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, timeout));
      if (ok) tc_fence_after();
      return ok;
    };
    for (WeightWalk<true> w(sh, len, cnt); w.more(); w.next(a)) {
      if (fresh) {
        qb = a.bufs == 2 ? item & 1u : 0;
        if (!wait(&sh->q_full[qb], (a.bufs == 2 ? item >> 1 : item) & 1u)) goto mma_done;
        ++item;
        steps = weight_steps(w.rows(a));
        cols = weight_cols(w.rows(a));
        idesc = make_idesc_bf16(kWtTile, cols, 0, 0);
      }
      int st[kSlabs];
#pragma unroll
      for (int c = 0; c < kSlabs; ++c) {
        st[c] = stage;
        if (!wait(&sh->full[stage], phase)) goto mma_done;
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      for (int i = 0; i < steps; ++i, ++step) {
        const uint32_t buf = step & 1u;
        if (!wait(&sh->t_empty[buf], ((step >> 1) & 1u) ^ 1u)) goto mma_done;
#pragma unroll
        for (int k = 0; k < kHD / 16; ++k)
          tc_mma_bf16_warp(tmem + buf * kWtStep, make_sdesc_sw128(s_ring + st[k / 4] * kWtSlab + (k % 4) * 32, 16, 1024),
                           make_sdesc_sw128(s_q + (qb * kSlabs + k / 4) * q_slab + i * cols * 128 + (k % 4) * 32, 16, 1024),
                           idesc, k > 0 ? 1u : 0u, issue);
        tc_commit_warp(&sh->t_full[buf], issue);
      }
#pragma unroll
      for (int c = 0; c < kSlabs; ++c) tc_commit_warp(&sh->empty[st[c]], issue);
      fresh = w.last_of_item();
      if (fresh) tc_commit_warp(&sh->q_empty[qb], issue);
    }
  mma_done:
    tc_commit_warp(&sh->mma_done, issue);
    if (lane == 0) {
      int dummy = 0;
      mbar_wait(&sh->mma_done, 0, &dummy, timeout);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // Warp w of the four takes rows 32 w .. 32 w + 31 of every 128. A lane looks up one row's
    // address; the copies of all rows are on their way before the statistics are looked at.
    const int w0 = (warp - 10) * 32;
    uint32_t item = 0;
    constexpr int kPieces = kHD / 8, kRowsAtOnce = 32 / kPieces, kGroups = kWtQBytes / (2 * kHD) / kWtLoaders + 1;
    for (WeightWalk<true> w(sh, len, cnt); w.more(); ++item) {
      const int qb = a.bufs == 2 ? item & 1u : 0;
      const uint32_t par = ((a.bufs == 2 ? item >> 1 : item) & 1u) ^ 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(&sh->q_empty[qb], par, abort_flag, timeout))) break;
      const int rows = w.rows(a), cols = weight_cols(rows) * weight_steps(rows);
      const uint32_t q0 = s_q + qb * kSlabs * q_slab;
      const int boxed = a.box ? a.j_max * a.group : 0;  // rows that a box brings
      if (a.box) {
        if (warp == 10 && lane == 0) {
          mbar_arrive_expect_tx(&sh->q_box[qb], kSlabs * boxed * 128);
#pragma unroll
          for (int c = 0; c < kSlabs; ++c) tma_load_4d(q0 + c * q_slab, &a.tm_q, smem_u32(&sh->q_box[qb]), c * 64, w.h * a.group, a.j0, w.b);
        }
        __syncwarp();
      }
      // Row of the lane in each group: its statistic, and its query's address (0: a row beyond the
      // queries, to be filled with zeros).
      float stat[kGroups];
      unsigned long long row_at[kGroups];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int r = w0 + g * kWtLoaders + lane;
        stat[g] = -INFINITY;
        row_at[g] = 0ull;
        if (r < rows) {
          const int j = a.j0 + r / a.group;
          const int node = a.path != nullptr ? a.path[static_cast<long long>(w.b) * a.n + j] : j;
          const long long head = static_cast<long long>(w.h) * a.group + r % a.group;
          stat[g] = a.lse[(static_cast<long long>(w.b) * a.n + node) * (static_cast<long long>(a.heads) * a.group) + head];
          row_at[g] = reinterpret_cast<unsigned long long>(a.q + w.b * a.q_seq + node * a.q_row + head * kHD);
        }
      }
      const int pc = lane % kPieces;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int r0 = w0 + g * kWtLoaders;
        if (r0 >= cols) break;
        if (r0 + kWtLoaders / 4 <= boxed) continue;
        unsigned long long from[kPieces];  // all shuffles before the first copy, which none would pass
#pragma unroll
        for (int i = 0; i < kPieces; ++i) from[i] = __shfl_sync(0xffffffffu, row_at[g], i * kRowsAtOnce + lane / kPieces);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int rr = r0 + i * kRowsAtOnce + lane / kPieces;
          const uint32_t dst = q0 + (pc / 8) * q_slab + rr * 128 + (((pc & 7) ^ (rr & 7)) << 4);
          if (rr >= boxed && rr < cols)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                         "l"((from[i] != 0ull ? from[i] : reinterpret_cast<unsigned long long>(a.q)) + pc * 16ull),
                         "r"(from[i] != 0ull ? 16 : 0)
                         : "memory");
        }
      }
      // A query that sees nothing (-inf) adds nothing: its row becomes 0, whatever its bits are,
      // and its column -inf.
      unsigned empty = 0;  // bit g: the lane's row of group g
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int r = w0 + g * kWtLoaders + lane;
        if (r < rows && stat[g] == -INFINITY) empty |= 1u << g;
        if (r < cols) {
          neg_lse[qb * a.rows_cap + r] = stat[g] == -INFINITY ? -INFINITY : -stat[g] * kWtLog2e;
          position[qb * a.rows_cap + r] = r < rows && stat[g] != -INFINITY ? r / a.group : kWtNever;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (a.box && !__all_sync(0xffffffffu, mbar_wait(&sh->q_box[qb], par ^ 1u, abort_flag, timeout))) {
        int dummy = 0;  // the box lands before the CTA may exit
        mbar_wait(&sh->q_box[qb], par ^ 1u, &dummy, timeout);
        break;
      }
      if (__any_sync(0xffffffffu, empty != 0u)) {  // the copies of a row are other lanes', complete after this
        __syncwarp();
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
          if ((empty >> g) & 1u) {
            const int r = w0 + g * kWtLoaders + lane;
            for (int pc = 0; pc < kPieces; ++pc)
              st_shared_v4(q0 + (pc / 8) * q_slab + r * 128 + ((pc & 7) << 4), 0, 0, 0, 0);
          }
      }
      fence_proxy_async_shared();
      mbar_arrive(&sh->q_full[qb]);
      // on to the next item
      while (!w.last_of_item()) w.next(a);
      w.next(a);
    }
  } else {
    const int part = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float sc = a.scale * kWtLog2e;
    uint32_t step = 0, halves = 0, item = 0;
    int qb = 0, rows = 0, steps = 0, cols = 0, c0 = 0, c1 = 0, m = 0, c = 0;
    const float* item_lse = neg_lse;
    bool fresh = true;
    // The scores so far come from memory a unit ahead.
    auto place = [&](const WeightWalk<true>& w) {
      return (static_cast<long long>(w.b) * a.heads + w.h) * a.capacity + w.t * kWtTile + row;
    };
    auto old_score = [&](const WeightWalk<true>& w) {
      return a.score_in != nullptr && w.more() && w.t * kWtTile + row < len[w.b] ? a.score_in[place(w)] : 0.0f;
    };
    WeightWalk<true> ahead(sh, len, cnt);
    float old_next = old_score(ahead);
    for (WeightWalk<true> w(sh, len, cnt); w.more(); w.next(a)) {
      const float old = old_next;
      ahead.next(a);
      old_next = old_score(ahead);
      if (fresh) {
        qb = a.bufs == 2 ? item & 1u : 0;
        const uint32_t par = (a.bufs == 2 ? item >> 1 : item) & 1u;
        if (!__all_sync(0xffffffffu, mbar_wait(&sh->q_full[qb], par, abort_flag, timeout))) goto sum_done;
        ++item;
        rows = w.rows(a);
        steps = weight_steps(rows);
        cols = weight_cols(rows);
        const int first = ((cols / 16 + 1) / 2) * 16;  // columns of the first warps
        c0 = steps == 1 || part == 0 ? 0 : first;
        c1 = steps == 1 || part == 1 ? cols : first;
        m = len[w.b];
        c = w.queries;
        item_lse = neg_lse + qb * a.rows_cap;
      }
      fresh = w.last_of_item();
      const bool mine = steps > 1 || (step & 1u) == static_cast<uint32_t>(part);
      const int key = w.t * kWtTile + row;
      float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
      if (mine) {
        // The first query sees rows up to m - c; the j-th up to m - c + j.
        const bool masked = rows == 0 || (w.t + 1) * kWtTile > m - c + a.j0 + 1;
        for (int i = 0; i < steps; ++i) {
          const uint32_t buf = (step + i) & 1u;
          if (!__all_sync(0xffffffffu, mbar_wait(&sh->t_full[buf], ((step + i) >> 1) & 1u, abort_flag, timeout)))
            goto sum_done;
          tc_fence_after();
          const uint32_t from = tmem + lanes + buf * kWtStep;
          const float* lse0 = item_lse + i * cols;
          bool by_column = masked;
          if (!masked) {
            const float2 b0 = s0, b1 = s1;
            int x = c0;
            for (; x + 32 <= c1; x += 32) {
              uint32_t r[32];
              tmem_ld32(from + x, r);
              tmem_wait_ld32(r);
              add_weights(r, lse0 + x, sc, s0, s1);
            }
            if (x < c1) {
              uint32_t r[16];
              tmem_ld16(from + x, r);
              tmem_wait_ld16(r);
              add_weights(r, lse0 + x, sc, s0, s1);
            }
            // A key with an infinity gives NaN in the columns of zeros (beyond the queries, or of one
            // that sees nothing), which do not count: its warp takes the step again without them.
            const float sum = (s0.x + s0.y) + (s1.x + s1.y);
            if (__any_sync(0xffffffffu, sum != sum)) {
              s0 = b0;
              s1 = b1;
              by_column = true;
            }
          }
          if (by_column) {
            for (int x = c0; x < c1; x += 16) {
              uint32_t r[16];
              tmem_ld16(from + x, r);
              tmem_wait_ld16(r);
              const int* pos = position + qb * a.rows_cap + i * cols + x;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float y = exp2f_ftz(fmaf(u2f(r[e]), sc, lse0[x + e]));
                s0.x += key - (m - c + a.j0) <= pos[e] ? y : 0.0f;
              }
            }
          }
          // Eight arrivals hand a step's columns back: one a warp, or two where four warps read it.
          tc_fence_before();
          __syncwarp();
          if (lane < (steps > 1 ? 1 : 2)) mbar_arrive(&sh->t_empty[buf]);
        }
      }
      step += steps;
      if (fresh && lane == 0) mbar_arrive(&sh->q_empty[qb]);  // neg_lse is read no more
      const float sum = (s0.x + s0.y) + (s1.x + s1.y);
      if (steps == 1) {
        if (mine && key < m) a.score_out[place(w)] = old * a.decay + sum;
      } else {
        // The two warps of a key meet. The second ones reach their fourth next meeting only after
        // the first ones have handed back a step of the second next, hence are done with slot and
        // barrier of this one.
        float* slot = sh->half[halves & 3u];
        if (part == 1) {
          slot[row] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->half_full[halves & 3u]);
        } else {
          if (!__all_sync(0xffffffffu, mbar_wait(&sh->half_full[halves & 3u], (halves >> 2) & 1u, abort_flag, timeout)))
            goto sum_done;
          if (key < m) a.score_out[place(w)] = old * a.decay + (sum + slot[row]);
        }
        ++halves;
      }
    }
  sum_done:;
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sh->abort) record_status(a.dev_status, RF_ERR_TIMEOUT);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int kHD>
static rf_status launch_weights(WeightArgs a, int ctas, size_t smem, cudaStream_t s) {
  static uint64_t done = 0;
  rf_status st = set_smem_attr(reinterpret_cast<const void*>(&k_attn_weights<kHD>), 227 * 1024, &done);
  if (st != RF_OK) return st;
  ProfScope prof(s, RF_STAGE_ATTN_WEIGHTS);
  return cuda_check(launch_dependent(k_attn_weights<kHD>, dim3(static_cast<unsigned>(ctas)), dim3(kWtThreads), smem, s, 1, a),
                    "k_attn_weights launch");
}

static rf_status check_weights(const rf_attn_desc* d) {
  rf_status st = check_attn_desc(d);
  if (st != RF_OK) return st;
  if (d->n_seqs > kWtMaxSeqs) return fail(RF_ERR_SHAPE, "n_seqs must be <= %d", kWtMaxSeqs);
  return RF_OK;
}

}  // namespace rf

using namespace rf;

extern "C" size_t rf_attn_weights_workspace_bytes(const rf_attn_desc* desc) {
  return check_weights(desc) == RF_OK ? 256 : 0;
}

extern "C" rf_status rf_attn_weights(const rf_attn_desc* d, const rf_bf16* q, const float* lse, const int32_t* path,
                                     const int32_t* n_path, const rf_bf16* k_cache, const int32_t* lens, double decay,
                                     const float* score_in, float* score_out, int32_t* dev_status, void* workspace,
                                     size_t workspace_bytes, rf_stream_t stream) {
  clear_error();
  rf_status st = check_weights(d);
  if (st != RF_OK) return st;
  if (!std::isfinite(decay)) return fail(RF_ERR_INVALID_ARG, "decay must be finite");
  if (d->n_seqs == 0) return RF_OK;
  if (!q || !lse || !k_cache || !lens || !score_out || (decay != 0.0 && !score_in) || (path == nullptr) != (n_path == nullptr))
    return fail(RF_ERR_INVALID_ARG, "tensor pointers must be non-NULL, path and n_path both or neither");
  if (!aligned16(q) || !aligned16(k_cache)) return fail(RF_ERR_ALIGN, "row buffers must be 16-byte aligned");
  const uintptr_t bits = reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(path) |
                         reinterpret_cast<uintptr_t>(n_path) | reinterpret_cast<uintptr_t>(lens) |
                         reinterpret_cast<uintptr_t>(score_in) | reinterpret_cast<uintptr_t>(score_out);
  if (bits & 3u) return fail(RF_ERR_ALIGN, "arrays must be 4-byte aligned");
  if (workspace == nullptr || workspace_bytes < 256 || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(RF_ERR_WORKSPACE, "workspace needs 256 bytes, 256-byte aligned (got %zu)", workspace_bytes);
  int sms = 0;
  if ((st = current_device(&sms)) != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint64_t hd = d->head_dim, H = d->n_kv_heads, B = d->n_seqs, cap = d->capacity;
  WeightArgs a{};
  if ((st = make_tmap_bf16_4d(&a.tm_k, k_cache, {hd, H, cap, B},
                              {hd, (uint64_t)d->cache_row_stride, (uint64_t)d->cache_seq_stride}, {64, 1, kWtTile, 1})) != RF_OK)
    return st;
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.lse = lse;
  a.path = path;
  a.n_path = n_path;
  a.lens = lens;
  a.dev_status = dev_status;
  a.timeout_ns = wait_timeout_ns();
  a.q_row = d->q_row_stride;
  a.q_seq = d->q_seq_stride;
  a.n_seqs = static_cast<int>(B);
  a.heads = static_cast<int>(H);
  a.group = static_cast<int>(d->n_q_heads / d->n_kv_heads);
  a.n = static_cast<int>(d->n_nodes);
  a.capacity = static_cast<int>(cap);
  a.scale = static_cast<float>(d->scale);
  // As many path positions a launch as their query rows fit in shared memory.
  const int64_t most = kWtQBytes / (2 * static_cast<int64_t>(hd));
  a.j_max = static_cast<int>(std::min<int64_t>(d->n_nodes, std::max<int64_t>(most / a.group, 1)));
  // A box holds up to 256 nodes (fewer query heads a KV head than three: gathered).
  a.box = path == nullptr && a.j_max <= 256;
  if (a.box && (st = make_tmap_bf16_4d(&a.tm_q, q, {hd, (uint64_t)d->n_q_heads, (uint64_t)d->n_nodes, B},
                                       {hd, (uint64_t)d->q_row_stride, (uint64_t)d->q_seq_stride},
                                       {64, (uint32_t)a.group, (uint32_t)a.j_max, 1})) != RF_OK)
    return st;
  // Steps round a launch's rows up by at most 16 columns each.
  const int rows = a.j_max * a.group;
  const int steps = std::max(1, (rows + kWtStep - 1) / kWtStep);
  a.rows_cap = std::max(16, (((rows + steps - 1) / steps + 15) & ~15)) * steps;
  // A second query buffer lets the next item's queries come in early, where the ring keeps at
  // least five slabs beside it (80 KB: more than the bytes in flight that hide memory's latency).
  // With one buffer the ring gets what is left: three slabs beside 640 query rows of 128 channels,
  // two with a thousand sequences as well.
  auto fixed = [&](int bufs) {
    return 1024 + static_cast<size_t>(bufs) * a.rows_cap * (hd * 2 + 8) + ((sizeof(WeightShared) + 15) & ~size_t(15)) +
           static_cast<size_t>(B) * 8;
  };
  constexpr size_t kMost = 227 * 1024;
  a.bufs = fixed(2) + 5 * kWtSlab <= kMost ? 2 : 1;
  a.stages = static_cast<int>(std::min<size_t>((kMost - fixed(a.bufs)) / kWtSlab, kWtMaxStages));
  const size_t smem = fixed(a.bufs) + static_cast<size_t>(a.stages) * kWtSlab;
  const int64_t units = static_cast<int64_t>(B * H) * static_cast<int64_t>((cap + kWtTile - 1) / kWtTile);
  const int ctas = static_cast<int>(std::min<int64_t>(units, sms));
  for (int64_t j0 = 0; j0 < d->n_nodes; j0 += a.j_max) {
    a.j0 = static_cast<int>(j0);
    a.decay = j0 == 0 ? static_cast<float>(decay) : 1.0f;
    a.score_in = j0 == 0 ? (decay != 0.0 ? score_in : nullptr) : score_out;
    a.score_out = score_out;
    st = hd == 128 ? launch_weights<128>(a, ctas, smem, s) : launch_weights<64>(a, ctas, smem, s);
    if (st != RF_OK) return st;
  }
  return RF_OK;
}
