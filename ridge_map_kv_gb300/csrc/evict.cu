// Eviction of cache rows by accumulated attention weight (rf_evict).
//
// Per layer, sequence and KV head ("unit") the min(len, keep) rows of the highest rank
// stay. Attention does not depend on the order of its rows, so nothing is compacted: the
// rows that stay beyond `keep` move into the holes below it, the fewest rows that can
// move. Sources lie beyond `keep` and destinations below, so the moves of a unit are
// independent of one another and run in any order, in place.
//
//   k_evict_select  one CTA a unit, a warp a contiguous run of rows and a lane one row of
//                   each 32. Rank keys stay in registers or shared memory (beyond 49,152
//                   rows they are formed anew from memory in every pass). The keep-th
//                   largest is searched by counting the keys that reach a candidate, two
//                   instructions a key and one barrier a step, bit by bit from the
//                   highest bit in which keys differ until just `keep` keys reach one, about
//                   20 steps for 4,000 different scores. (Interpolating on the counts took
//                   more steps, since rows that are sure to stay lie far off; histograms of
//                   8-bit digits take 3 passes, but their shared-memory atomics took 35 us
//                   for 16,384 rows.) Ranks among equals and the places of
//                   holes and movers come from ballots. It also writes the scores and
//                   positions of the rows that stay in place.
//   k_evict_move    the listed rows of K and V, their scores and positions. (No launch of its
//                   own where the capacity leaves a unit 128 moves at most.)
//
// Bound: reading scores and positions and writing the kept ones (16 bytes a row) and the
// moved rows' bytes twice; at a few rows a step, the latency of the selection. Measured (heads of
// 128 channels): half of 320 units at 4,103 rows with 4,096 to stay 9.8 us, of which the counting
// steps are most; 160 units of 16,384 rows with 4,096 to stay 122 us, of which the moves take 81
// (at the memory's rate) and the selection 42 (instructions, and a second wave of 8 CTAs).
#include <algorithm>

#include "rf_device.cuh"
#include "rf_host.h"

namespace rf {

constexpr int kMoveRows = 64;    // moves of one CTA of k_evict_move
constexpr int kOwnMoves = 128;   // at most: k_evict_select moves the rows itself

struct EvictArgs {
  const int32_t* lens;
  const int32_t* next_pos;
  const float* score_in;
  const int32_t* pos_in;
  float* score_out;
  int32_t* pos_out;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int32_t* moves;    // [units][2][max_moves]: destinations, sources
  int32_t* n_moves;  // [units]
  int32_t* new_lens;
  int32_t* dev_status;
  long long row_stride, seq_stride, layer_stride, max_moves;
  int n_seqs, heads, head_dim, capacity, keep, sink, recent;
  bool moves_too;  // k_evict_select also moves the rows and writes new_lens
};

// Order-preserving integer of a rank: larger scores give larger keys, -0 equals 0, NaN
// counts as -inf, rows that are sure to stay as +inf.
__device__ __forceinline__ unsigned rank_key(float score, bool sure) {
  float f = score != score ? -INFINITY : score;
  if (sure) f = INFINITY;
  const unsigned u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr size_t kSelKeyBytes = 192 * 1024;  // of shared memory for keys

template <int kThreads>
struct SelShared {
  int count[2][kThreads / 32];  // by the parity of the step
  int warp_a[kThreads / 32];
  int warp_b[kThreads / 32];
  int n_moves;
  int32_t moves[2][kOwnMoves];  // destinations and sources, where the CTA moves the rows itself
};

// Exclusive scan over the CTA's warps of one value per warp, in shared memory.
template <int kThreads>
__device__ __forceinline__ void scan_warps(int* v) {
  __syncthreads();
  if (threadIdx.x < 32) {
    const int own = threadIdx.x < kThreads / 32 ? v[threadIdx.x] : 0;
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (static_cast<int>(threadIdx.x) >= o) x += y;
    }
    if (threadIdx.x < kThreads / 32) v[threadIdx.x] = x - own;
  }
  __syncthreads();
}

__device__ __forceinline__ int32_t length_after(const EvictArgs& a, int len) {
  return len > a.keep && len <= a.capacity ? a.keep : len;
}

// m moves of a unit, by the whole CTA.
template <int kThreads>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int unit, const int32_t* dst, const int32_t* src, int m) {
  const int h = unit % a.heads, lb = unit / a.heads, b = lb % a.n_seqs, l = lb / a.n_seqs;
  const long long head = l * a.layer_stride + b * a.seq_stride + static_cast<long long>(h) * a.head_dim;
  const int pieces = a.head_dim / 8;
#pragma unroll 4
  for (int x = threadIdx.x; x < m * pieces; x += kThreads) {
    const int i = x / pieces, c = (x - i * pieces) * 8;
    const long long from = head + static_cast<long long>(src[i]) * a.row_stride + c;
    const long long to = head + static_cast<long long>(dst[i]) * a.row_stride + c;
    const uint4 k = *reinterpret_cast<const uint4*>(a.k + from), v = *reinterpret_cast<const uint4*>(a.v + from);
    *reinterpret_cast<uint4*>(a.k + to) = k;
    *reinterpret_cast<uint4*>(a.v + to) = v;
  }
  const long long base = static_cast<long long>(unit) * a.capacity;
  for (int i = threadIdx.x; i < m; i += kThreads) {
    a.score_out[base + dst[i]] = a.score_in[base + src[i]];
    a.pos_out[base + dst[i]] = a.pos_in[base + src[i]];
  }
}

// Rows are taken in groups of 32, one a lane: warp w owns the groups from w * per_warp on,
// kItems at a time (a "load" of groups). kKeys says where keys are between passes.
enum { kInRegisters, kInShared, kInMemory };  // (one load a warp), (formed once), (formed in every pass)
template <int kThreads, int kItems, int kKeys, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm) k_evict_select(const __grid_constant__ EvictArgs a) {
  static_assert(kItems <= 32, "a lane remembers one group's ballot");
  constexpr int kWarps = kThreads / 32;
  constexpr int kSelBatch = kItems < 8 ? kItems : 8;  // rows of a thread whose loads are in flight together
  __shared__ SelShared<kThreads> sh;
  pdl_wait();  // (no early release: waiting CTAs of the next kernel would take this one's places)
  const int unit = blockIdx.x;
  const int b = (unit / a.heads) % a.n_seqs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = a.lens[b];
  // rows from position `newest` on are sure to stay (saturated: positions are 32-bit)
  const int newest = static_cast<int>(max(static_cast<long long>(a.next_pos[b]) - a.recent, -2147483648ll));
  const long long base = static_cast<long long>(unit) * a.capacity;
  const float* score = a.score_in + base;
  const int32_t* pos = a.pos_in + base;
  if (a.moves_too && tid == 0 && unit % a.heads == 0 && unit / a.heads < a.n_seqs) a.new_lens[b] = length_after(a, len);
  if (len < 0 || len > a.capacity) {
    if (tid == 0) {
      a.n_moves[unit] = 0;
      record_status(a.dev_status, RF_ERR_INVALID_ARG);
    }
    return;
  }
  const int keep = a.keep;
  const bool copy = a.score_out != a.score_in || a.pos_out != a.pos_in;
  // Rows [t0, t0 + 32 n) of a warp, lane by lane: those in `mine` (bit i: row t0 + 32 i + lane)
  // are copied to the outputs, eight at a time.
  auto copy_rows = [&](int t0, unsigned mine) {
#pragma unroll
    for (int i0 = 0; i0 < kItems; i0 += kSelBatch) {
      if (__ballot_sync(0xffffffffu, (mine >> i0) & ((1u << kSelBatch) - 1u)) == 0) continue;
      float f[kSelBatch];
      int32_t q[kSelBatch];
#pragma unroll
      for (int i = 0; i < kSelBatch; ++i) {
        if ((mine >> (i0 + i)) & 1u) {
          f[i] = score[t0 + (i0 + i) * 32 + lane];
          q[i] = pos[t0 + (i0 + i) * 32 + lane];
        }
      }
#pragma unroll
      for (int i = 0; i < kSelBatch; ++i) {
        if ((mine >> (i0 + i)) & 1u) {
          a.score_out[base + t0 + (i0 + i) * 32 + lane] = f[i];
          a.pos_out[base + t0 + (i0 + i) * 32 + lane] = q[i];
        }
      }
    }
  };
  const int groups = (len + 31) / 32, per_warp = (groups + kWarps - 1) / kWarps;
  const int g0 = min(warp * per_warp, groups), g1 = min(g0 + per_warp, groups);  // this warp's groups
  if (len <= keep) {
    if (copy)
      for (int g = g0; g < g1; g += kItems) {
        unsigned mine = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i) mine |= g + i < g1 && (g + i) * 32 + lane < len ? 1u << i : 0u;
        copy_rows(g * 32, mine);
      }
    if (tid == 0) a.n_moves[unit] = 0;
    return;
  }
  // Keys of a load of groups from g on; 0, which is below every key, where there is no row.
  auto load_keys = [&](int g, unsigned (&k)[kItems]) {
#pragma unroll
    for (int i0 = 0; i0 < kItems; i0 += kSelBatch) {
      float f[kSelBatch];
      int32_t q[kSelBatch];
#pragma unroll
      for (int i = 0; i < kSelBatch; ++i) {
        const int t = min((g + i0 + i) * 32 + lane, len - 1);
        if (i0 + i < kItems) {
          f[i] = score[t];
          q[i] = pos[t];
        }
      }
#pragma unroll
      for (int i = 0; i < kSelBatch; ++i)
        if (i0 + i < kItems) {
          const int t = (g + i0 + i) * 32 + lane;
          k[i0 + i] = g + i0 + i < g1 && t < len ? rank_key(f[i], q[i] < a.sink || q[i] >= newest) : 0u;
        }
    }
  };
  unsigned keys[kItems];
  extern __shared__ unsigned shared_keys[];  // a warp touches its own groups' alone
  if constexpr (kKeys == kInRegisters) load_keys(g0, keys);
  if constexpr (kKeys == kInShared) {
    for (int g = g0; g < g1; g += kItems) {
      load_keys(g, keys);
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (g + i < g1) shared_keys[(g + i) * 32 + lane] = keys[i];
    }
  }
  // Calls f(first group, keys) for each of the warp's loads.
  auto each = [&](auto f) {
    if constexpr (kKeys == kInRegisters) {
      f(g0, keys);
    } else {
      for (int g = g0; g < g1; g += kItems) {
        if constexpr (kKeys == kInShared) {
#pragma unroll
          for (int i = 0; i < kItems; ++i) keys[i] = g + i < g1 ? shared_keys[(g + i) * 32 + lane] : 0u;
        } else {
          load_keys(g, keys);
        }
        f(g, keys);
      }
    }
  };
  // Sum over the CTA of a value per warp's lane 0 (`parity` alternates between calls).
  auto cta_sum = [&](int warp_value, int parity) {
    if (lane == 0) sh.count[parity][warp] = warp_value;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.count[parity][lane] : 0);
  };
  // The smallest and the largest key.
  unsigned lo = 0xffffffffu, hi = 0;
  each([&](int, const unsigned (&k)[kItems]) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      hi = max(hi, k[i]);
      lo = min(lo, k[i] != 0u ? k[i] : 0xffffffffu);
    }
  });
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lane == 0) {
    sh.warp_a[warp] = static_cast<int>(hi);
    sh.warp_b[warp] = static_cast<int>(lo);
  }
  __syncthreads();
  hi = __reduce_max_sync(0xffffffffu, lane < kWarps ? static_cast<unsigned>(sh.warp_a[lane]) : 0u);
  lo = __reduce_min_sync(0xffffffffu, lane < kWarps ? static_cast<unsigned>(sh.warp_b[lane]) : 0xffffffffu);
  const int top = hi == lo ? -1 : 31 - __clz(hi ^ lo);  // highest bit that differs
  // bar: the largest value with the bits found so far that at least `keep` keys reach;
  // reach: how many do. Without ties it is just `keep`.
  unsigned bar = top < 0 ? hi : top == 31 ? 0u : hi & (0xffffffffu << (top + 1));
  int reach = len, above = 0;  // above: keys known to be greater than any that share bar's bits
#pragma unroll 1
  for (int bit = top; bit >= 0 && reach != keep; --bit) {
    const unsigned c = bar | (1u << bit);
    int n = 0;
    each([&](int, const unsigned (&k)[kItems]) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) n += k[i] >= c;
    });
    n = cta_sum(__reduce_add_sync(0xffffffffu, n), bit & 1);
    if (n >= keep) {
      bar = c;
      reach = n;
    } else {
      above = n;
    }
  }
  const bool ties = reach != keep;  // then bar is a key, and some of those equal to it leave
  const int left = keep - above;    // how many of them stay
  __syncthreads();
  const unsigned below = (1u << lane) - 1u;
  int eq = 0;  // keys equal to bar in earlier groups
  if (ties) {
    int n = 0;
    each([&](int, const unsigned (&k)[kItems]) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) n += __popc(__ballot_sync(0xffffffffu, k[i] == bar));
    });
    if (lane == 0) sh.warp_a[warp] = n;
    scan_warps<kThreads>(sh.warp_a);
    eq = sh.warp_a[warp];
  }
  const int eq0 = eq;
  // The rows of a load that stay: bit i of the result for the lane's own rows, and lane i's
  // `group` for group i's 32 rows.
  auto who_stays = [&](const unsigned (&k)[kItems], unsigned& group) {
    unsigned own = 0;
    group = 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      bool stay = k[i] >= bar && k[i] != 0u;
      if (ties) {
        const unsigned m = __ballot_sync(0xffffffffu, k[i] == bar);
        if (k[i] == bar) stay = eq + __popc(m & below) < left;
        eq += __popc(m);
      }
      const unsigned m = __ballot_sync(0xffffffffu, stay);
      if (lane == i) group = m;
      own |= stay ? 1u << i : 0u;
    }
    return own;
  };
  // Of group g's rows that exist and lie below `keep` (lane's group: bit masks).
  auto rows_below = [&](int row0, int end) {  // bits of rows row0 .. row0 + 31 below `end`
    const int n = end - row0;
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  };
  int holes = 0, movers = 0;       // of the warp
  unsigned own_first = 0, m_first = 0;  // of its one load (kInRegisters)
  each([&](int g, const unsigned (&k)[kItems]) {
    unsigned m;
    own_first = who_stays(k, m);
    m_first = m;
    const int row0 = (g + lane) * 32;
    const unsigned low = lane < kItems && g + lane < g1 ? rows_below(row0, keep) : 0u;
    holes += __popc(~m & low & rows_below(row0, len));
    movers += lane < kItems ? __popc(m & ~rows_below(row0, keep)) : 0;
  });
  holes = __reduce_add_sync(0xffffffffu, holes);
  movers = __reduce_add_sync(0xffffffffu, movers);
  __syncthreads();
  if (lane == 0) {
    sh.warp_a[warp] = holes;
    sh.warp_b[warp] = movers;
  }
  scan_warps<kThreads>(sh.warp_a);
  scan_warps<kThreads>(sh.warp_b);
  int hole = sh.warp_a[warp], mover = sh.warp_b[warp];
  if (warp == kWarps - 1 && lane == 0) {
    a.n_moves[unit] = mover + movers;  // as many holes as movers
    sh.n_moves = mover + movers;
  }
  int32_t* dst = a.moves_too ? sh.moves[0] : a.moves + static_cast<long long>(unit) * 2 * a.max_moves;
  int32_t* src = a.moves_too ? sh.moves[1] : dst + a.max_moves;
  eq = eq0;
  each([&](int g, const unsigned (&k)[kItems]) {
    unsigned m = m_first;
    const unsigned own = kKeys == kInRegisters ? own_first : who_stays(k, m);
    const int row0 = (g + lane) * 32;
    const unsigned low = rows_below(row0, keep);
    const bool mine = lane < kItems && g + lane < g1;
    const unsigned mh = mine ? ~m & low & rows_below(row0, len) : 0u, mm = mine ? m & ~low : 0u;
    // where each group's holes and movers start in the lists
    int h = __popc(mh), v = __popc(mm);
    const int oh = h, ov = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, h, o), z = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) {
        h += y;
        v += z;
      }
    }
    const int h_all = __shfl_sync(0xffffffffu, h, 31), v_all = __shfl_sync(0xffffffffu, v, 31);
    h += hole - oh;
    v += mover - ov;
    for (unsigned todo = __ballot_sync(0xffffffffu, (mh | mm) != 0u); todo != 0u; todo &= todo - 1u) {
      const int i = __ffs(todo) - 1, t = (g + i) * 32 + lane;
      const unsigned gh = __shfl_sync(0xffffffffu, mh, i), gm = __shfl_sync(0xffffffffu, mm, i);
      const int bh = __shfl_sync(0xffffffffu, h, i), bm = __shfl_sync(0xffffffffu, v, i);
      if ((gh >> lane) & 1u) dst[bh + __popc(gh & below)] = t;
      if ((gm >> lane) & 1u) src[bm + __popc(gm & below)] = t;
    }
    hole += h_all;
    mover += v_all;
    if (copy) {
      unsigned in_place = own;  // the lane's rows that stay below `keep`
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if ((g + i) * 32 + lane >= keep) in_place &= ~(1u << i);
      copy_rows(g * 32, in_place);
    }
  });
  if (a.moves_too) {
    __syncthreads();
    move_rows<kThreads>(a, unit, dst, src, sh.n_moves);
  }
}

__global__ void __launch_bounds__(256) k_evict_move(const __grid_constant__ EvictArgs a) {
  pdl_wait();
  const int unit = blockIdx.y;
  const int n = a.n_moves[unit];
  const int i0 = blockIdx.x * kMoveRows;
  if (unit == 0 && i0 == 0) {  // new_lens may be lens, which k_evict_select has read
    for (int b = threadIdx.x; b < a.n_seqs; b += 256) a.new_lens[b] = length_after(a, a.lens[b]);
  }
  const int m = min(n - i0, kMoveRows);
  const int32_t* dst = a.moves + static_cast<long long>(unit) * 2 * a.max_moves + i0;
  if (m > 0) move_rows<256>(a, unit, dst, dst + a.max_moves, m);
}

// Whether no two rows of a cache, to all of which the calls write, lie on one another. As a rule
// layers, sequences and rows are nested, in any order: each stride spans all that lies inside it.
// Otherwise all differences of two places are looked at (up to 2^20 of them).
static bool rows_apart(const rf_cache_desc* d) {
  using Wide = __int128;
  struct Dim {
    int64_t n, stride;
  } dim[3] = {{d->capacity, d->row_stride}, {d->n_seqs, d->seq_stride}, {d->n_layers, d->layer_stride}};
  const Wide row = d->n_kv_heads * d->head_dim;
  std::sort(dim, dim + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  Wide span = row;
  bool nested = true;
  for (const Dim& x : dim) {
    if (x.n <= 1) continue;
    nested &= x.stride >= span;
    span += static_cast<Wide>(x.n - 1) * x.stride;
  }
  if (nested) return true;
  std::sort(dim, dim + 3, [](const Dim& x, const Dim& y) { return x.n > y.n; });
  for (const Dim& x : dim)
    if (x.n > 1 && x.stride < row) return false;
  if (dim[1].n * dim[2].n > (int64_t(1) << 20)) return false;
  const Wide most = dim[0].n - 1, step = dim[0].stride;
  for (int64_t i = 0; i < dim[1].n; ++i)
    for (int64_t j = i == 0 ? 1 : 1 - dim[2].n; j < dim[2].n; ++j) {
      const Wide x = static_cast<Wide>(i) * dim[1].stride + static_cast<Wide>(j) * dim[2].stride;
      for (int near = -1; near <= 1; ++near) {  // places of the first dimension around -x
        const Wide y = x + std::min(std::max(near - x / step, -most), most) * step;
        if (y < row && -y < row) return false;
      }
    }
  return true;
}

rf_status check_cache_desc(const rf_cache_desc* d) {
  if (d == nullptr) return fail(RF_ERR_INVALID_ARG, "desc is NULL");
  if (d->n_layers < 0 || d->n_seqs < 0 || d->n_kv_heads <= 0 || d->head_dim <= 0 || d->capacity <= 0)
    return fail(RF_ERR_INVALID_ARG, "need n_layers, n_seqs >= 0, n_kv_heads, head_dim, capacity > 0");
  if (d->head_dim % 8 != 0 || d->head_dim > 256) return fail(RF_ERR_SHAPE, "head_dim must be a multiple of 8, at most 256");
  if (d->capacity > (int64_t(1) << 24) || d->n_seqs > 65535 || d->n_layers > 65535 || d->n_kv_heads > 65535)
    return fail(RF_ERR_SHAPE, "need capacity <= 2^24, n_layers, n_seqs, n_kv_heads <= 65535");
  if (d->row_stride < d->n_kv_heads * d->head_dim || d->row_stride % 8 || d->seq_stride % 8 || d->layer_stride % 8 ||
      d->seq_stride < 0 || d->layer_stride < 0)
    return fail(RF_ERR_ALIGN, "cache strides must be multiples of 8, the row stride >= n_kv_heads*head_dim");
  if (!rows_apart(d)) return fail(RF_ERR_ALIGN, "rows, sequences and layers must not overlap");
  return RF_OK;
}

struct EvictLayout {
  int32_t* moves;
  int32_t* n_moves;
  int64_t max_moves;
  size_t bytes;
};

static EvictLayout evict_layout(const rf_cache_desc* d, int64_t keep, void* ws) {
  EvictLayout l;
  const int64_t units = d->n_layers * d->n_seqs * d->n_kv_heads;
  l.max_moves = std::max<int64_t>(std::min(keep, d->capacity - keep), 0);
  Carve c(ws);
  l.moves = c.take<int32_t>(static_cast<size_t>(units * 2 * l.max_moves));
  l.n_moves = c.take<int32_t>(static_cast<size_t>(units));
  l.bytes = std::max<size_t>(c.bytes(), 256);
  return l;
}

static rf_status check_evict(const rf_cache_desc* d, int64_t keep) {
  rf_status st = check_cache_desc(d);
  if (st != RF_OK) return st;
  if (keep < 1) return fail(RF_ERR_INVALID_ARG, "keep must be >= 1");
  const int64_t units = d->n_layers * d->n_seqs * d->n_kv_heads;
  if (units > 65535) return fail(RF_ERR_SHAPE, "n_layers * n_seqs * n_kv_heads must be <= 65535");
  return RF_OK;
}

}  // namespace rf

using namespace rf;

extern "C" size_t rf_evict_workspace_bytes(const rf_cache_desc* desc, int64_t keep) {
  if (check_evict(desc, keep) != RF_OK) return 0;
  return evict_layout(desc, keep, nullptr).bytes;
}

extern "C" rf_status rf_evict(const rf_cache_desc* d, int64_t keep, int64_t n_sink, int64_t n_recent,
                              const int32_t* lens, const int32_t* next_pos, rf_bf16* k_cache, rf_bf16* v_cache,
                              const float* score_in, const int32_t* pos_in, float* score_out, int32_t* pos_out,
                              int32_t* new_lens, int32_t* dev_status, void* workspace, size_t workspace_bytes,
                              rf_stream_t stream) {
  clear_error();
  rf_status st = check_evict(d, keep);
  if (st != RF_OK) return st;
  if (n_sink < 0 || n_recent < 0 || n_sink >= (int64_t(1) << 31) || n_recent >= (int64_t(1) << 31))
    return fail(RF_ERR_INVALID_ARG, "n_sink and n_recent must be in [0, 2^31)");
  if (d->n_layers == 0 || d->n_seqs == 0) return RF_OK;
  if (!lens || !next_pos || !k_cache || !v_cache || !score_in || !pos_in || !score_out || !pos_out || !new_lens)
    return fail(RF_ERR_INVALID_ARG, "tensor pointers must be non-NULL");
  if (!aligned16(k_cache) || !aligned16(v_cache)) return fail(RF_ERR_ALIGN, "caches must be 16-byte aligned");
  const uintptr_t bits = reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(next_pos) |
                         reinterpret_cast<uintptr_t>(score_in) | reinterpret_cast<uintptr_t>(pos_in) |
                         reinterpret_cast<uintptr_t>(score_out) | reinterpret_cast<uintptr_t>(pos_out) |
                         reinterpret_cast<uintptr_t>(new_lens);
  if (bits & 3u) return fail(RF_ERR_ALIGN, "arrays must be 4-byte aligned");
  if (new_lens != lens && overlap(new_lens, d->n_seqs, lens, d->n_seqs))
    return fail(RF_ERR_INVALID_ARG, "new_lens must be lens or lie apart from it");
  const EvictLayout lay = evict_layout(d, keep, workspace);
  if (workspace == nullptr || workspace_bytes < lay.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(RF_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", lay.bytes, workspace_bytes);
  int sms = 0;
  if ((st = current_device(&sms)) != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  EvictArgs a{};
  a.lens = lens;
  a.next_pos = next_pos;
  a.score_in = score_in;
  a.pos_in = pos_in;
  a.score_out = score_out;
  a.pos_out = pos_out;
  a.k = reinterpret_cast<__nv_bfloat16*>(k_cache);
  a.v = reinterpret_cast<__nv_bfloat16*>(v_cache);
  a.moves = lay.moves;
  a.n_moves = lay.n_moves;
  a.new_lens = new_lens;
  a.dev_status = dev_status;
  a.row_stride = d->row_stride;
  a.seq_stride = d->seq_stride;
  a.layer_stride = d->layer_stride;
  a.max_moves = lay.max_moves;
  a.n_seqs = static_cast<int>(d->n_seqs);
  a.heads = static_cast<int>(d->n_kv_heads);
  a.head_dim = static_cast<int>(d->head_dim);
  a.capacity = static_cast<int>(d->capacity);
  a.keep = static_cast<int>(std::min(keep, d->capacity));
  a.sink = static_cast<int>(n_sink);
  a.recent = static_cast<int>(n_recent);
  // One launch where few rows can move, so that a unit's CTA moves them by itself (half of 320
  // units over the 4,096 rows that stay, by 64 rows: 13.2 us, 15.0 in two launches; by 128: 14.7
  // and 15.7; 8 units over 2,000 rows by 64: 9.8 and 10.4; by 256: 12.3 and 11.0); not where
  // new_lens is written over lens or next_pos, which every CTA reads.
  const bool apart = !overlap(new_lens, d->n_seqs, lens, d->n_seqs) && !overlap(new_lens, d->n_seqs, next_pos, d->n_seqs);
  a.moves_too = apart && lay.max_moves <= kOwnMoves;
  const unsigned units = static_cast<unsigned>(d->n_layers * d->n_seqs * d->n_kv_heads);
  {
    ProfScope prof(s, RF_STAGE_EVICT_SELECT);
    // By the cache's capacity: every warp pays for a step's sums and barrier, so few warps with
    // many keys each, in registers while they fit (16,384 rows in 160 units: 47 us on 1,024
    // threads; with keys in shared memory 54 us on 512 threads and 59 us on 1,024). 17 keys a
    // thread, not 16, so that a cache of a power of two of rows fits with a sixteenth more for
    // the rows drafted since. Whole calls, 160 units down to 4,096 rows: 17,408 rows 124 us in
    // registers, 17,409 rows 173 us and 32,768 rows 197 us in shared memory, 49,152 rows 243 us
    // there, 49,153 rows 578 us with keys formed anew.
    cudaError_t e = cudaSuccess;
    const size_t key_bytes = (static_cast<size_t>(d->capacity) + 31) / 32 * 128;
    if (d->capacity <= 128 * 17) {
      e = launch_dependent(k_evict_select<128, 17, kInRegisters, 4>, dim3(units), dim3(128), 0, s, 1, a);
    } else if (d->capacity <= 256 * 17) {
      e = launch_dependent(k_evict_select<256, 17, kInRegisters, 3>, dim3(units), dim3(256), 0, s, 1, a);
    } else if (d->capacity <= 512 * 17) {
      e = launch_dependent(k_evict_select<512, 17, kInRegisters, 2>, dim3(units), dim3(512), 0, s, 1, a);
    } else if (d->capacity <= 1024 * 17) {
      e = launch_dependent(k_evict_select<1024, 17, kInRegisters, 1>, dim3(units), dim3(1024), 0, s, 1, a);
    } else if (key_bytes <= kSelKeyBytes) {
      static uint64_t done = 0;
      const void* fn = reinterpret_cast<const void*>(&k_evict_select<1024, 16, kInShared, 1>);
      if ((st = set_smem_attr(fn, kSelKeyBytes, &done)) != RF_OK) return st;
      e = launch_dependent(k_evict_select<1024, 16, kInShared, 1>, dim3(units), dim3(1024), key_bytes, s, 1, a);
    } else {
      e = launch_dependent(k_evict_select<1024, 16, kInMemory, 1>, dim3(units), dim3(1024), 0, s, 1, a);
    }
    if ((st = cuda_check(e, "k_evict_select launch")) != RF_OK) return st;
  }
  if (a.moves_too) return RF_OK;
  ProfScope prof(s, RF_STAGE_EVICT_MOVE);
  const unsigned chunks = static_cast<unsigned>(std::max<int64_t>((lay.max_moves + kMoveRows - 1) / kMoveRows, 1));
  return cuda_check(launch_dependent(k_evict_move, dim3(chunks, units), dim3(256), 0, s, 1, a), "k_evict_move launch");
}
