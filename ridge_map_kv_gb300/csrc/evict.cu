// Eviction of cache rows by accumulated attention weight (rf_evict).
//
// Per layer, sequence and KV head ("unit") the min(len, keep) rows of the highest rank
// stay. Attention does not depend on the order of its rows, so nothing is compacted: the
// rows that stay beyond `keep` move into the holes below it, the fewest rows that can
// move. Sources lie beyond `keep` and destinations below, so the moves of a unit are
// independent of one another and run in any order, in place.
//
//   k_evict_select  one CTA a unit, a warp a contiguous run of rows and a lane one row of
//                   each 32. Rank keys stay in registers (up to 32 a thread; beyond
//                   32,768 rows they are formed anew from memory in every pass). The
//                   keep-th largest comes from a radix selection of 11 + 11 + 10 bits;
//                   ranks among equals and the places of holes and movers come from
//                   ballots. It also writes the scores and positions of the rows that
//                   stay in place.
//   k_evict_move    the listed rows of K and V, their scores and positions.
//
// Bound: reading scores and positions and writing the kept ones (16 bytes a row) and the
// moved rows' bytes twice; at a few rows a step, the latency of the selection.
#include <algorithm>

#include "rf_device.cuh"
#include "rf_host.h"

namespace rf {

constexpr int kSelBins = 2048;
constexpr int kMoveRows = 64;                // moves of one CTA of k_evict_move

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
};

// Order-preserving integer of a rank: larger scores give larger keys, -0 equals 0, NaN
// counts as -inf, rows that are sure to stay as +inf.
__device__ __forceinline__ unsigned rank_key(float score, bool sure) {
  float f = score != score ? -INFINITY : score;
  if (sure) f = INFINITY;
  const unsigned u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int kThreads>
struct SelShared {
  int hist[kSelBins];
  int warp_a[kThreads / 32];
  int warp_b[kThreads / 32];
  unsigned prefix;
  int left;
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

// kItems keys a thread in registers, or 0: formed from memory in every pass.
template <int kThreads, int kItems>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) k_evict_select(const __grid_constant__ EvictArgs a) {
  constexpr int kWarps = kThreads / 32;
  __shared__ SelShared<kThreads> sh;
  pdl_launch_dependents();
  const int unit = blockIdx.x;
  const int b = (unit / a.heads) % a.n_seqs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = a.lens[b];
  const long long base = static_cast<long long>(unit) * a.capacity;
  const float* score = a.score_in + base;
  const int32_t* pos = a.pos_in + base;
  if (len < 0 || len > a.capacity) {
    if (tid == 0) {
      a.n_moves[unit] = 0;
      record_status(a.dev_status, RF_ERR_INVALID_ARG);
    }
    return;
  }
  const int keep = a.keep;
  if (len <= keep) {
#pragma unroll 4
    for (int t = tid; t < len; t += kThreads) {
      a.score_out[base + t] = score[t];
      a.pos_out[base + t] = pos[t];
    }
    if (tid == 0) a.n_moves[unit] = 0;
    return;
  }
  const long long newest = static_cast<long long>(a.next_pos[b]) - a.recent;
  // Warp w owns rows [r0, r1), lane i of it rows r0 + i, r0 + 32 + i, ...
  const int run = ((len + kWarps - 1) / kWarps + 31) & ~31;
  const int r0 = min(warp * run, len), r1 = min(r0 + run, len);
  auto key_of = [&](int t) {
    const int p = pos[t];
    return rank_key(score[t], p < a.sink || p >= newest);
  };
  unsigned keys[kItems > 0 ? kItems : 1];
  if constexpr (kItems > 0) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int t = r0 + i * 32 + lane;
      keys[i] = t < r1 ? key_of(t) : 0u;
    }
  }
  // Calls f(row, key, whether the row is one of the warp's) for all of a thread's rows, in
  // order; every lane of a warp makes the same calls.
  auto each = [&](auto f) {
    if constexpr (kItems > 0) {
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (r0 + i * 32 < r1) f(r0 + i * 32 + lane, keys[i], r0 + i * 32 + lane < r1);
    } else {
      for (int t = r0 + lane; t - lane < r1; t += 32) f(t, t < r1 ? key_of(t) : 0u, t < r1);
    }
  };
  // The keep-th largest key, digit by digit: among the keys that share the digits found
  // so far, the bin that holds the rank still wanted.
  unsigned prefix = 0, mask = 0;
  int left = keep;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const unsigned digit = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kSelBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    each([&](int, unsigned k, bool in) {
      if (in && (k & mask) == prefix) atomicAdd(&sh.hist[(k >> shift) & digit], 1);
    });
    __syncthreads();
    // Thread i holds kBins bins from the top down: an inclusive scan.
    constexpr int kBins = kSelBins / kThreads;
    int h[kBins], x = 0;
#pragma unroll
    for (int j = 0; j < kBins; ++j) {
      h[j] = sh.hist[kSelBins - 1 - (kBins * tid + j)];
      x += h[j];
    }
    const int own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh.warp_a[warp] = x;
    scan_warps<kThreads>(sh.warp_a);
    int before = sh.warp_a[warp] + x - own;             // keys in higher bins
    if (before < left && before + own >= left) {        // one thread
#pragma unroll
      for (int j = 0; j < kBins; ++j) {
        if (before < left && before + h[j] >= left) {
          sh.prefix = static_cast<unsigned>(kSelBins - 1 - (kBins * tid + j)) << shift;
          sh.left = left - before;
        }
        before += h[j];
      }
    }
    __syncthreads();
    prefix |= sh.prefix;
    mask |= digit << shift;
    left = sh.left;
  }
  const unsigned bar = prefix;  // rows above stay, and the first `left` of those equal to it
  const unsigned below = (1u << lane) - 1u;
  int n_eq = 0;
  each([&](int, unsigned k, bool in) { n_eq += __popc(__ballot_sync(0xffffffffu, in && k == bar)); });
  __syncthreads();
  if (lane == 0) sh.warp_a[warp] = n_eq;
  scan_warps<kThreads>(sh.warp_a);
  const int eq0 = sh.warp_a[warp];
  int eq = eq0;
  auto stays = [&](unsigned k, bool in) {  // warp-collective; eq: equal rows before these 32
    const bool same = in && k == bar;
    const unsigned m = __ballot_sync(0xffffffffu, same);
    const bool stay = in && (k > bar || (same && eq + __popc(m & below) < left));
    eq += __popc(m);
    return stay;
  };
  int holes = 0, movers = 0;
  each([&](int t, unsigned k, bool in) {
    const bool stay = stays(k, in);
    holes += __popc(__ballot_sync(0xffffffffu, in && t < keep && !stay));
    movers += __popc(__ballot_sync(0xffffffffu, t >= keep && stay));
  });
  __syncthreads();
  if (lane == 0) {
    sh.warp_a[warp] = holes;
    sh.warp_b[warp] = movers;
  }
  scan_warps<kThreads>(sh.warp_a);
  scan_warps<kThreads>(sh.warp_b);
  int hole = sh.warp_a[warp], mover = sh.warp_b[warp];
  int32_t* dst = a.moves + static_cast<long long>(unit) * 2 * a.max_moves;
  int32_t* src = dst + a.max_moves;
  const bool copy = a.score_out != a.score_in || a.pos_out != a.pos_in;
  eq = eq0;
  each([&](int t, unsigned k, bool in) {
    const bool stay = stays(k, in);
    const bool is_hole = in && t < keep && !stay, is_mover = t >= keep && stay;
    const unsigned mh = __ballot_sync(0xffffffffu, is_hole), mm = __ballot_sync(0xffffffffu, is_mover);
    if (is_hole) dst[hole + __popc(mh & below)] = t;
    if (is_mover) src[mover + __popc(mm & below)] = t;
    hole += __popc(mh);
    mover += __popc(mm);
    if (copy && stay && t < keep) {
      a.score_out[base + t] = score[t];
      a.pos_out[base + t] = pos[t];
    }
  });
  if (warp == kWarps - 1 && lane == 0) a.n_moves[unit] = mover;  // as many holes as movers
}

__global__ void __launch_bounds__(256) k_evict_move(const __grid_constant__ EvictArgs a) {
  pdl_wait();
  const int unit = blockIdx.y;
  const int n = a.n_moves[unit];
  const int i0 = blockIdx.x * kMoveRows;
  if (unit == 0 && i0 == 0) {  // new_lens may be lens, which k_evict_select has read
    for (int b = threadIdx.x; b < a.n_seqs; b += 256) {
      const int len = a.lens[b];
      a.new_lens[b] = len > a.keep && len <= a.capacity ? a.keep : len;
    }
  }
  const int m = min(n - i0, kMoveRows);
  if (m <= 0) return;
  const int h = unit % a.heads, lb = unit / a.heads, b = lb % a.n_seqs, l = lb / a.n_seqs;
  const int32_t* dst = a.moves + static_cast<long long>(unit) * 2 * a.max_moves + i0;
  const int32_t* src = dst + a.max_moves;
  const long long head = l * a.layer_stride + b * a.seq_stride + static_cast<long long>(h) * a.head_dim;
  const int pieces = a.head_dim / 8;
#pragma unroll 4
  for (int x = threadIdx.x; x < m * pieces; x += 256) {
    const int i = x / pieces, c = (x - i * pieces) * 8;
    const long long from = head + static_cast<long long>(src[i]) * a.row_stride + c;
    const long long to = head + static_cast<long long>(dst[i]) * a.row_stride + c;
    const uint4 k = *reinterpret_cast<const uint4*>(a.k + from), v = *reinterpret_cast<const uint4*>(a.v + from);
    *reinterpret_cast<uint4*>(a.k + to) = k;
    *reinterpret_cast<uint4*>(a.v + to) = v;
  }
  const long long base = static_cast<long long>(unit) * a.capacity;
  for (int i = threadIdx.x; i < m; i += 256) {
    a.score_out[base + dst[i]] = a.score_in[base + src[i]];
    a.pos_out[base + dst[i]] = a.pos_in[base + src[i]];
  }
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
  // rows of one cache must not lie on one another: the calls write to them
  const int64_t span = (d->capacity - 1) * d->row_stride + d->n_kv_heads * d->head_dim;
  if ((d->n_seqs > 1 && d->seq_stride < span && d->layer_stride < span) ||
      (d->n_seqs > 1 && d->seq_stride == 0) || (d->n_layers > 1 && d->layer_stride == 0))
    return fail(RF_ERR_ALIGN, "layers and sequences must not overlap");
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
  const unsigned units = static_cast<unsigned>(d->n_layers * d->n_seqs * d->n_kv_heads);
  {
    ProfScope prof(s, RF_STAGE_EVICT_SELECT);
    // Threads and keys a thread by the cache's capacity: small CTAs leave room for several on
    // an SM, and a CTA of 1,024 threads has 64 registers a thread for 32 keys.
    if (d->capacity <= 2048) k_evict_select<256, 8><<<units, 256, 0, s>>>(a);
    else if (d->capacity <= 8192) k_evict_select<512, 16><<<units, 512, 0, s>>>(a);
    else if (d->capacity <= 32768) k_evict_select<1024, 32><<<units, 1024, 0, s>>>(a);
    else k_evict_select<1024, 0><<<units, 1024, 0, s>>>(a);
  }
  if ((st = cuda_check(cudaGetLastError(), "k_evict_select launch")) != RF_OK) return st;
  ProfScope prof(s, RF_STAGE_EVICT_MOVE);
  const unsigned chunks = static_cast<unsigned>(std::max<int64_t>((lay.max_moves + kMoveRows - 1) / kMoveRows, 1));
  return cuda_check(launch_dependent(k_evict_move, dim3(chunks, units), dim3(256), 0, s, a), "k_evict_move launch");
}
