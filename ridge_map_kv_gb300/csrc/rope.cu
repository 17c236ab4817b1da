// Rotary positions in general form (rf_rope): both channel pairings, part of a head,
// frequencies stretched for long contexts, given positions, the transposed rotation,
// bf16 or fp32 rows.
//
// Pair i of a head at position p: (x1, x2) -> m (x1 c - x2 s, x2 c + x1 s), with c, s of
// the angle p f_i. Each row is read once and written once and a pair costs six
// operations, so memory is the bound at any row count that fills the GPU. Measured: 32,768
// rows of 48 bf16 heads 120 us (6.7 TB/s read and written, 0.99 of a plain copy), 8,191 rows of
// 40 fp32 heads 51 us (6.6 TB/s).
//
// A thread takes one or two 16-byte pieces of a head, at the same channels of `hpt` heads:
// in the half layout a piece of the first half and its partner of the second, in the
// interleaved one a piece of whole pairs. Its angles are formed once and serve all of its
// heads, four of which are loaded before any is stored. Neighbouring lanes take
// neighbouring pieces, so a warp's accesses are whole sectors. Where rot_dim or head_dim
// does not divide into such pieces a thread takes one pair at a time instead.
#include <algorithm>
#include <cmath>

#include "rf_device.cuh"
#include "rf_host.h"
#include "rope.cuh"

namespace rf {

struct RopeArgs {
  const void* in;
  void* out;
  const int32_t* positions;
  long long ld_in, ld_out, pos_offset;
  int n_rows, n_heads, head_dim, rot, hpt, items;  // items: chunks of a head
  float amp, sign;
};

// kWide: 16-byte pieces; else one pair (or two channels that do not turn) a thread.
template <class T, bool kWide, bool kHalf>
struct RopeShape {
  static constexpr int kVec = kWide ? 16 / static_cast<int>(sizeof(T)) : kHalf ? 1 : 2;  // channels of a piece
  static constexpr int kPieces = kHalf ? 2 : 1;
  static constexpr int kChannels = kVec * kPieces;                                       // of a thread and head
  static constexpr int kPairs = kChannels / 2;
};
constexpr int kRopeHeads = 4;  // heads whose loads are in flight together

template <class T, bool kWide, bool kHalf>
__global__ void __launch_bounds__(256) k_rope(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTable tab) {
  using S = RopeShape<T, kWide, kHalf>;
  pdl_launch_dependents();
  pdl_wait();
  const unsigned idx = blockIdx.x * 256u + threadIdx.x;
  if (idx >= static_cast<unsigned>(a.n_rows) * static_cast<unsigned>(a.items)) return;
  const int row = static_cast<int>(idx / static_cast<unsigned>(a.items));
  const int item = static_cast<int>(idx - static_cast<unsigned>(row) * static_cast<unsigned>(a.items));
  const int h0 = static_cast<int>(blockIdx.y) * a.hpt, h1 = min(h0 + a.hpt, a.n_heads);
  const int pair0 = item * S::kPairs;
  const bool turns = 2 * pair0 < a.rot;
  if (!turns && a.in == a.out) return;
  // First channels of the thread's pieces. Channels that do not turn follow one another.
  const int c1 = kHalf && turns ? pair0 : item * S::kChannels;
  const int c2 = kHalf && turns ? pair0 + (a.rot >> 1) : c1 + S::kVec;
  const T* in = static_cast<const T*>(a.in) + row * a.ld_in;
  T* out = static_cast<T*>(a.out) + row * a.ld_out;
  float c[S::kPairs], s[S::kPairs];
  if (turns) {
    const long long p = a.positions != nullptr ? static_cast<long long>(a.positions[row]) : row + a.pos_offset;
#pragma unroll
    for (int i = 0; i < S::kPairs; ++i) {
      turn_cs<T>(static_cast<unsigned long long>(p), tab.g[pair0 + i], c[i], s[i]);
      c[i] *= a.amp;
      s[i] *= a.amp * a.sign;
    }
  } else {
#pragma unroll
    for (int i = 0; i < S::kPairs; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
  }
  for (int h = h0; h < h1; h += kRopeHeads) {
    alignas(16) T u[kRopeHeads][S::kVec], w[kRopeHeads][S::kVec];
#pragma unroll
    for (int j = 0; j < kRopeHeads; ++j) {
      if (h + j >= h1) break;
      const int at = (h + j) * a.head_dim;
      load_vec(in + at + c1, u[j]);
      if constexpr (kHalf) load_vec(in + at + c2, w[j]);
    }
#pragma unroll
    for (int j = 0; j < kRopeHeads; ++j) {
      if (h + j >= h1) break;
      if (turns) {
#pragma unroll
        for (int i = 0; i < S::kPairs; ++i) {
          T& d1 = kHalf ? u[j][i] : u[j][(2 * i) % S::kVec];
          T& d2 = kHalf ? w[j][i] : u[j][(2 * i + 1) % S::kVec];
          const float x1 = to_f(d1), x2 = to_f(d2);
          from_f(d1, x1 * c[i] - x2 * s[i]);
          from_f(d2, x2 * c[i] + x1 * s[i]);
        }
      }
      const int at = (h + j) * a.head_dim;
      store_vec(out + at + c1, u[j]);
      if constexpr (kHalf) store_vec(out + at + c2, w[j]);
    }
  }
}

// The frequency table. theta^(-2i/r) is the product of two powers, one of i mod 8 and one
// of i - i mod 8: 8 + r/16 calls of pow instead of r/2, each factor within an ulp.
RopeTable rope_table(const rf_rope_desc* d) {
  RopeTable t{};
  const int r = static_cast<int>(d->rot_dim), n = r / 2;
  const double pi = 3.14159265358979323846;
  double theta = d->theta;
  if (d->scaling == RF_ROPE_SCALE_BASE) theta *= std::pow(d->factor, r / (r - 2.0));
  double lo[8], hi[kRopeMaxPairs / 8];
  for (int i = 0; i < std::min(n, 8); ++i) lo[i] = std::pow(theta, -2.0 * i / r);
  for (int i = 0; i < (n + 7) / 8; ++i) hi[i] = i == 0 ? 1.0 : std::pow(theta, -16.0 * i / r);
  double ramp_lo = 0.0, ramp_hi = 0.0;
  if (d->scaling == RF_ROPE_SCALE_RAMP) {
    auto at = [&](double turns) { return r * std::log(d->original_rows / (turns * 2.0 * pi)) / (2.0 * std::log(theta)); };
    ramp_lo = std::max(std::floor(at(d->high_turns)), 0.0);
    ramp_hi = std::min(std::ceil(at(d->low_turns)), r - 1.0);
  }
  auto clamp01 = [](double x) { return std::min(std::max(x, 0.0), 1.0); };
  for (int i = 0; i < n; ++i) {
    double f = lo[i & 7] * hi[i >> 3];
    switch (d->scaling) {
      case RF_ROPE_SCALE_LINEAR: f /= d->factor; break;
      case RF_ROPE_SCALE_WAVELENGTH: {
        const double w = clamp01((d->original_rows * f / (2.0 * pi) - d->low_turns) / (d->high_turns - d->low_turns));
        f *= w + (1.0 - w) / d->factor;
        break;
      }
      case RF_ROPE_SCALE_RAMP: {
        const double w = clamp01((i - ramp_lo) / std::max(ramp_hi - ramp_lo, 0.001));
        f *= (1.0 - w) + w / d->factor;
        break;
      }
      default: break;
    }
    // A frequency of a turn or more per position wraps like the angle itself.
    double turns = f / (2.0 * pi);
    turns -= std::floor(turns);
    t.g[i] = static_cast<unsigned long long>(std::ldexp(turns, 64));
  }
  return t;
}

rf_status check_rope(const rf_rope_desc* d) {
  if (d == nullptr) return fail(RF_ERR_INVALID_ARG, "desc is NULL");
  if (d->n_rows < 0 || d->n_heads <= 0 || d->head_dim <= 0 || d->rot_dim <= 0)
    return fail(RF_ERR_INVALID_ARG, "need n_rows >= 0, n_heads, head_dim, rot_dim > 0");
  if (!(d->theta > 0.0) || !std::isfinite(d->theta)) return fail(RF_ERR_INVALID_ARG, "theta must be > 0");
  if (!std::isfinite(d->amplitude)) return fail(RF_ERR_INVALID_ARG, "amplitude must be finite");
  if (d->layout != RF_ROPE_HALF && d->layout != RF_ROPE_INTERLEAVED) return fail(RF_ERR_INVALID_ARG, "unknown layout");
  if (d->dtype != RF_BF16 && d->dtype != RF_F32) return fail(RF_ERR_INVALID_ARG, "unknown dtype");
  if (d->scaling < RF_ROPE_SCALE_NONE || d->scaling > RF_ROPE_SCALE_RAMP)
    return fail(RF_ERR_INVALID_ARG, "unknown scaling");
  if (d->scaling != RF_ROPE_SCALE_NONE && (!(d->factor >= 1.0) || !std::isfinite(d->factor)))
    return fail(RF_ERR_INVALID_ARG, "factor must be >= 1");
  if (d->scaling == RF_ROPE_SCALE_WAVELENGTH || d->scaling == RF_ROPE_SCALE_RAMP) {
    if (!(d->original_rows > 0.0) || !(d->low_turns > 0.0) || !(d->high_turns > d->low_turns) ||
        !std::isfinite(d->original_rows) || !std::isfinite(d->high_turns))
      return fail(RF_ERR_INVALID_ARG, "need original_rows > 0 and 0 < low_turns < high_turns");
  }
  if (d->scaling == RF_ROPE_SCALE_RAMP && !(d->theta > 1.0)) return fail(RF_ERR_INVALID_ARG, "theta must be > 1");
  if (d->head_dim % 8 != 0 || d->head_dim > 256) return fail(RF_ERR_SHAPE, "head_dim must be a multiple of 8, at most 256");
  if (d->rot_dim % 2 != 0 || d->rot_dim > d->head_dim) return fail(RF_ERR_SHAPE, "rot_dim must be even, at most head_dim");
  if (d->scaling == RF_ROPE_SCALE_BASE && d->rot_dim <= 2) return fail(RF_ERR_SHAPE, "a stretched base needs rot_dim > 2");
  if (d->n_rows > (int64_t(1) << 24)) return fail(RF_ERR_SHAPE, "n_rows must be <= 2^24");
  if (d->n_heads > 65535) return fail(RF_ERR_SHAPE, "n_heads must be <= 65535");
  const int64_t w = d->n_heads * d->head_dim;
  if (d->ld_in < w || d->ld_out < w || d->ld_in % 8 != 0 || d->ld_out % 8 != 0)
    return fail(RF_ERR_ALIGN, "row strides must be >= n_heads*head_dim and multiples of 8");
  return RF_OK;
}

template <class T, bool kWide, bool kHalf>
static cudaError_t launch_rope(RopeArgs& a, const RopeTable& t, int sms, cudaStream_t s) {
  a.items = a.head_dim / RopeShape<T, kWide, kHalf>::kChannels;
  // Heads per thread: as many (multiples of the four that are loaded together) as still
  // leave two waves of threads; all of them one by one in the smallest calls.
  const long long threads1 = static_cast<long long>(a.n_rows) * a.items;
  a.hpt = 1;
  while (a.hpt < 16 && threads1 * a.n_heads / (2 * a.hpt) >= 4096LL * sms) a.hpt *= 2;
  const dim3 grid(static_cast<unsigned>((threads1 + 255) / 256), static_cast<unsigned>((a.n_heads + a.hpt - 1) / a.hpt));
  return launch_dependent(k_rope<T, kWide, kHalf>, grid, dim3(256), 0, s, 1, a, t);
}
template <class T>
static cudaError_t launch_rope(RopeArgs& a, const RopeTable& t, bool half, int sms, cudaStream_t s) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  const int unit = half ? 2 * kVec : kVec;  // channels of a thread and head
  const bool wide = a.rot % unit == 0 && a.head_dim % unit == 0;
  if (half) {
    if (wide) return launch_rope<T, true, true>(a, t, sms, s);
    return launch_rope<T, false, true>(a, t, sms, s);
  } else {
    if (wide) return launch_rope<T, true, false>(a, t, sms, s);
    return launch_rope<T, false, false>(a, t, sms, s);
  }
}

// Masks and positions of drafted trees, one CTA a sequence. A thread per node climbs its
// ancestors through the parents in shared memory; indices fall on the way up, so its
// mask words come out one after another, the highest first.
__global__ void __launch_bounds__(1024) k_tree_build(int n, int words, const int32_t* parents,
                                                     const int32_t* next_pos, unsigned long long* mask,
                                                     int32_t* positions, int32_t* dev_status) {
  __shared__ int up[RF_TREE_MAX_NODES];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x, i = threadIdx.x;
  bool bad = false;
  if (i < n) {
    const int p = parents[static_cast<long long>(b) * n + i];
    up[i] = p;
    bad = i == 0 ? p != -1 : (p < 0 || p >= i);
  }
  if (__syncthreads_or(bad)) {
    if (i == 0) record_status(dev_status, RF_ERR_INVALID_ARG);
    return;
  }
  if (i >= n) return;
  const long long node = static_cast<long long>(b) * n + i;
  int depth = -1, at = i;
  for (int w = words - 1; w >= 0; --w) {
    unsigned long long m = 0;
    while (at >= 0 && (at >> 6) == w) {
      m |= 1ull << (at & 63);
      at = up[at];
      ++depth;
    }
    if (mask != nullptr) mask[node * words + w] = m;
  }
  if (positions != nullptr) positions[node] = next_pos[b] + depth;
}

}  // namespace rf

using namespace rf;

extern "C" rf_status rf_rope(const rf_rope_desc* desc, const void* in, void* out, const int32_t* positions,
                             rf_stream_t stream) {
  clear_error();
  rf_status st = check_rope(desc);
  if (st != RF_OK) return st;
  if (desc->n_rows == 0) return RF_OK;
  if (!in || !out) return fail(RF_ERR_INVALID_ARG, "in and out must be non-NULL");
  if (!aligned16(in) || !aligned16(out)) return fail(RF_ERR_ALIGN, "in and out must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return fail(RF_ERR_ALIGN, "positions must be 4-byte aligned");
  if (in == out && desc->ld_in != desc->ld_out) return fail(RF_ERR_INVALID_ARG, "in place needs ld_out = ld_in");
  int sms = 0;
  if ((st = current_device(&sms)) != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RopeTable tab = rope_table(desc);
  RopeArgs a{};
  a.in = in;
  a.out = out;
  a.positions = positions;
  a.ld_in = desc->ld_in;
  a.ld_out = desc->ld_out;
  a.pos_offset = desc->pos_offset;
  a.n_rows = static_cast<int>(desc->n_rows);
  a.n_heads = static_cast<int>(desc->n_heads);
  a.head_dim = static_cast<int>(desc->head_dim);
  a.rot = static_cast<int>(desc->rot_dim);
  a.amp = desc->amplitude == 0.0 ? 1.0f : static_cast<float>(desc->amplitude);
  a.sign = desc->transpose ? -1.0f : 1.0f;
  const bool half = desc->layout == RF_ROPE_HALF;
  ProfScope prof(s, RF_STAGE_ROPE);
  return cuda_check(desc->dtype == RF_BF16 ? launch_rope<__nv_bfloat16>(a, tab, half, sms, s)
                                           : launch_rope<float>(a, tab, half, sms, s),
                    "k_rope launch");
}

extern "C" rf_status rf_tree_build(int64_t n_seqs, int64_t n_nodes, const int32_t* parents, const int32_t* next_pos,
                                   uint64_t* mask, int32_t* positions, int32_t* dev_status, rf_stream_t stream) {
  clear_error();
  if (n_seqs < 0 || n_nodes <= 0) return fail(RF_ERR_INVALID_ARG, "need n_seqs >= 0, n_nodes > 0");
  if (n_nodes > RF_TREE_MAX_NODES || n_seqs > (int64_t(1) << 24))
    return fail(RF_ERR_SHAPE, "n_nodes must be <= %d, n_seqs <= 2^24", RF_TREE_MAX_NODES);
  if (n_seqs == 0) return RF_OK;
  if (!parents || (positions && !next_pos)) return fail(RF_ERR_INVALID_ARG, "parents (and next_pos for positions) must be non-NULL");
  if ((reinterpret_cast<uintptr_t>(parents) & 3u) || (reinterpret_cast<uintptr_t>(next_pos) & 3u) ||
      (reinterpret_cast<uintptr_t>(mask) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return fail(RF_ERR_ALIGN, "arrays must be aligned to their elements");
  int sms = 0;
  rf_status st = current_device(&sms);
  if (st != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope prof(s, RF_STAGE_TREE_BUILD);
  return cuda_check(launch_dependent(k_tree_build, dim3(static_cast<unsigned>(n_seqs)),
                                     dim3(static_cast<unsigned>((n_nodes + 31) / 32 * 32)), 0, s, 1,
                                     static_cast<int>(n_nodes), static_cast<int>(RF_TREE_WORDS(n_nodes)), parents, next_pos,
                                     reinterpret_cast<unsigned long long*>(mask), positions, dev_status),
                    "k_tree_build launch");
}
