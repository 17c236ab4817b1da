// Norms of queries and keys, head by head, with the rotation in the same pass (rf_norm_rope),
// and their gradient (rf_norm_rope_backward).
//
// Forward, a head x of d channels: r = (mean(x^2) + eps)^-1/2, y = m R (g x r), with R the
// rotation of rf_rope. Backward, from dy: u = m R^T dy; dg = sum over rows and heads of u x r;
// w = g u; dx = r (w - x r^2 mean(w x)), since dr/dx = -r^3 x / d.
//
// Every row is read and written once, so memory is the bound. The lanes that share a head
// (a power of two up to 32, in one warp) hold two 16-byte pieces of it each: its sums are
// exchanged by shuffles and nothing is read twice. Channels' angles and gains are formed once
// for the heads of a row. A thread's pieces of its next heads are on their way to shared memory
// while it works on those that are there (asynchronous copies; each thread reads what it copied
// itself, so there is no barrier); with the pieces loaded to registers instead the forward pass
// took 151 us for 126 and the backward pass 69 for 60, as fewer bytes were in flight. Measured,
// of bf16 heads of 128: 32,768 rows of 48 in 124 us (6.5 TB/s), 0.96 of a plain copy's rate; the
// gradient of 8,191 rows of 40 in 54.5 us (4.6 TB/s; 60 before its products were packed in
// pairs), where neither memory (53% of its peak) nor issue slots (46%) are full: 16 warps an SM
// take one head after another through rotation, exchanges, root and stores; a step of 8 rows of
// 48 in 5 us, which is a launch. fp32: 8,191 rows of 40 in 57 us (5.9 TB/s), their gradient in 93
// (5.4 TB/s); rows of few heads are bound by their angles, which serve those only: 32,768 of 3 in 39.5 us
// (2.5 TB/s). Where half of the channels turn, a lane's pieces lie further apart: 32,768 rows of
// 48 bf16 heads in 153 us. Three forms say which pieces those are:
//   kPieces   halves turn against each other and divide into pieces: a piece of the first half
//             and its partner of the second, as in rf_rope
//   kPairs    neighbouring channels turn against each other: any two pieces
//   kShared   halves that do not divide into pieces: any two pieces, partners read from shared
//             memory (16-byte accesses of global memory even so). Of bf16 rows it holds an angle for
//             each channel, and 20 bytes of the forward pass and 112 of the backward pass do not find a
//             register
//
// The gains' gradients are sums over all rows: a thread keeps its channels' sums over its run of
// heads, a CTA joins its threads' and leaves a row of partial sums in the workspace, and
// k_gain_sum adds those in order. No atomics, so that the order, and the result, depends on the
// sizes alone.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "rf_device.cuh"
#include "rf_host.h"
#include "rope.cuh"

namespace rf {

constexpr int kNormThreads = 256;
constexpr int kNormMaxCtas = 1024;  // of the backward pass: bounds the workspace

enum NormForm { kPieces, kPairs, kShared };

struct NormArgs {
  const void* in;
  const void* q_gain;
  const void* k_gain;
  const void* dy;      // backward
  void* out;           // y, or dx
  float* part;         // backward: [ctas][head_dim] partial sums, NULL: not wanted
  const int32_t* positions;
  long long ld_in, ld_dy, ld_out, pos_offset;
  int n_rows, n_heads, n_q, head_dim, rot;
  int lanes;           // of a head, as a power of two
  int hpt;             // heads of a row that a thread takes
  int q_ctas;          // backward: CTAs of the query heads, the others take the key heads
  float amp, eps;
};

// A lane's place in a head.
template <class T, int kForm>
struct NormLane {
  static constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  static constexpr int kChannels = 2 * kVec;
  static constexpr int kAngles = kForm == kShared ? kChannels : kVec;
  using Raw = T[2][kVec];
  int start[2];  // first channels of its pieces
  bool ok[2];    // whether they exist
  bool turns;    // kPieces: its channels turn
  float c[kAngles], s[kAngles], g[kChannels];

  __device__ __forceinline__ void place(const NormArgs& a, int lane) {
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {  // (a group without a row turns zeros)
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
    if (kForm == kPieces) {
      turns = 2 * lane * kVec < a.rot;
      start[0] = turns ? lane * kVec : lane * kChannels;
      start[1] = turns ? start[0] + (a.rot >> 1) : start[0] + kVec;
      ok[0] = ok[1] = lane * kChannels < a.head_dim;
    } else {
      start[0] = lane * kVec;
      start[1] = (lane + a.lanes) * kVec;
      ok[0] = start[0] < a.head_dim;
      ok[1] = start[1] < a.head_dim;
    }
  }
  // Angles at position p; sign -1 for the transpose.
  __device__ __forceinline__ void angles(const NormArgs& a, const RopeTable& tab, long long p, float sign) {
    const unsigned long long q = static_cast<unsigned long long>(p);
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
      int pair;
      if (kForm == kPieces) {
        pair = turns && ok[0] ? start[0] + i : -1;
      } else if (kForm == kPairs) {
        const int ch = start[2 * i / kVec] + 2 * i % kVec;
        pair = ch < a.rot ? ch >> 1 : -1;
      } else {
        const int ch = start[i / kVec] + i % kVec;
        pair = ch < a.rot ? (2 * ch < a.rot ? ch : ch - (a.rot >> 1)) : -1;
      }
      if (pair >= 0) {
        turn_cs<T>(q, tab.g[pair], c[i], s[i]);
        c[i] *= a.amp;
        s[i] *= a.amp * sign;
        if (kForm == kShared && 2 * (start[i / kVec] + i % kVec) < a.rot) s[i] = -s[i];
      }
    }
  }
  __device__ __forceinline__ void gains(const void* gain) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      alignas(16) T v[kVec];
      const bool there = gain != nullptr && ok[p];
      if (there) load_vec(static_cast<const T*>(gain) + start[p], v);
#pragma unroll
      for (int i = 0; i < kVec; ++i) g[p * kVec + i] = there ? to_f(v[i]) : 1.0f;
    }
  }
  // Copies a head's pieces to `slot` (of this thread, its second piece kNormThreads places on), and reads them there.
  __device__ __forceinline__ void copy(uint32_t slot, const T* head) const {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      if (ok[p]) copy_async16(slot + p * kNormThreads * 16, head + start[p]);
  }
  __device__ __forceinline__ void take(uint32_t slot, Raw& v) const {
#pragma unroll
    for (int p = 0; p < 2; ++p) *reinterpret_cast<uint4*>(v[p]) = ld_shared_v4(slot + p * kNormThreads * 16);
  }
  // Zeros in the places of pieces that do not exist: nothing is copied there.
  __device__ __forceinline__ void clear(uint32_t slot) const {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      if (!ok[p]) st_shared_v4(slot + p * kNormThreads * 16, 0, 0, 0, 0);
  }
  __device__ __forceinline__ void widen(const T (&v)[2][kVec], float (&x)[kChannels]) const {
#pragma unroll
    for (int i = 0; i < kChannels; ++i) x[i] = to_f(v[i / kVec][i % kVec]);
  }
  __device__ __forceinline__ void store(T* head, const float (&x)[kChannels]) const {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      alignas(16) T v[kVec];
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<__nv_bfloat162*>(v + i) = __floats2bfloat162_rn(x[p * kVec + i], x[p * kVec + i + 1]);
        } else {
          v[i] = x[p * kVec + i];
          v[i + 1] = x[p * kVec + i + 1];
        }
      }
      if (ok[p]) store_vec(head + start[p], v);
    }
  }
  // Whether a gain is an infinity or NaN, or may become an infinity by an inverse root (2^63 at most).
  __device__ __forceinline__ bool odd_gains() const {
    float zero = 0.0f;
#pragma unroll
    for (int i = 0; i < kChannels; ++i) zero = fmaf(g[i] * 0x1p63f, 0.0f, zero);
    return zero != zero;
  }
  // Turns a head's channels; `sh`: the head's channels in shared memory (kShared; whole warp). Channels that do not turn
  // have an angle of 0; 0 times an infinity or NaN of one would be a NaN of another, so where there may be one they are left
  // alone (kOdd; done so always, heads of which a part turns took 2 to 6% longer).
  template <bool kOdd>
  __device__ __forceinline__ void turn(const NormArgs& a, float* sh, float (&x)[kChannels]) const {
    if (kForm == kPieces) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        if (kOdd && !turns) break;
        const float x1 = x[i], x2 = x[kVec + i];
        x[i] = x1 * c[i] - x2 * s[i];
        x[kVec + i] = x2 * c[i] + x1 * s[i];
      }
    } else if (kForm == kPairs) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        if (kOdd && start[2 * i / kVec] + 2 * i % kVec >= a.rot) continue;
        const float x1 = x[2 * i], x2 = x[2 * i + 1];
        x[2 * i] = x1 * c[i] - x2 * s[i];
        x[2 * i + 1] = x2 * c[i] + x1 * s[i];
      }
    } else {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kChannels; i += 4)
        if (ok[i / kVec])
          *reinterpret_cast<float4*>(sh + start[i / kVec] + i % kVec) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kChannels; ++i) {
        const int ch = start[i / kVec] + i % kVec;
        if (ok[i / kVec] && ch < a.rot) x[i] = x[i] * c[i] + sh[2 * ch < a.rot ? ch + (a.rot >> 1) : ch - (a.rot >> 1)] * s[i];
      }
    }
  }
};

// The same for a head in packed pairs of channels.
template <bool kOdd, class T, int kForm>
__device__ __forceinline__ void turn_x2(const NormArgs& a, const NormLane<T, kForm>& l, float* sh,
                                        float2 (&x)[NormLane<T, kForm>::kChannels / 2]) {
  constexpr int kHalf = NormLane<T, kForm>::kVec / 2;
  if constexpr (kForm == kPieces) {
    if (kOdd && !l.turns) return;
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      const float2 c = make_float2(l.c[2 * i], l.c[2 * i + 1]), s = make_float2(l.s[2 * i], l.s[2 * i + 1]);
      const float2 x1 = x[i], x2 = x[kHalf + i];
      x[i] = fma_x2(x1, c, mul_x2(x2, make_float2(-s.x, -s.y)));
      x[kHalf + i] = fma_x2(x2, c, mul_x2(x1, s));
    }
  } else {
    float y[4 * kHalf];
#pragma unroll
    for (int i = 0; i < 2 * kHalf; ++i) {
      y[2 * i] = x[i].x;
      y[2 * i + 1] = x[i].y;
    }
    l.template turn<kOdd>(a, sh, y);
#pragma unroll
    for (int i = 0; i < 2 * kHalf; ++i) x[i] = make_float2(y[2 * i], y[2 * i + 1]);
  }
}

// A thread's places for pieces in flight: `kHeads` heads (of one array) in each of kNormStages. Two stages carry both
// passes: three or four change their times by less than 3%, or cost a small call its ramp (22 and 25 us for 20).
constexpr int kNormStages = 2;
constexpr size_t norm_ring_bytes(int heads) {
  return static_cast<size_t>(kNormStages) * heads * 2 * kNormThreads * 16;
}
template <int kHeads>
__device__ __forceinline__ uint32_t norm_slot(uint32_t ring, int stage, int j) {
  return ring + static_cast<uint32_t>(((stage * kHeads + j) * 2 * kNormThreads + static_cast<int>(threadIdx.x)) * 16);
}

// Two neighbouring channels in fp32.
__device__ __forceinline__ float2 pair_of(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(v));
}
// Sums over the lanes of a head.
__device__ __forceinline__ void head_sums(float& x, float& y, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) {
    const float dx = __shfl_xor_sync(0xffffffffu, x, o), dy = __shfl_xor_sync(0xffffffffu, y, o);
    x += dx;
    y += dy;
  }
}
__device__ __forceinline__ float head_sum(float x, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// (v)^-1/2: the SFU's for bf16 rows, rounded operations for fp32 ones.
template <class T>
__device__ __forceinline__ float inverse_root(float v) {
  if constexpr (sizeof(T) == 2) return rsqrtf(v);
  else return __frcp_rn(__fsqrt_rn(v));
}

constexpr int kNormHeads = 4;  // heads that a thread takes together

// kPart: some channels do not turn (kPieces, kPairs).
template <class T, int kForm, bool kPart>
__global__ void __launch_bounds__(kNormThreads, 2) k_norm_rope(const __grid_constant__ NormArgs a,
                                                            const __grid_constant__ RopeTable tab) {
  using Lane = NormLane<T, kForm>;
  __shared__ __align__(16) float staged[kForm == kShared ? kNormThreads * Lane::kChannels : 4];
  pdl_launch_dependents();
  pdl_wait();
  const unsigned idx = blockIdx.x * static_cast<unsigned>(kNormThreads) + threadIdx.x;
  const int at = static_cast<int>(idx) & (a.lanes - 1);
  const int row_of = static_cast<int>(idx / static_cast<unsigned>(a.lanes));
  const bool live = row_of < a.n_rows;  // (the others keep their warp's exchanges whole)
  const int row = live ? row_of : a.n_rows - 1;
  float* sh = staged + (kForm == kShared ? (threadIdx.x - at) * Lane::kChannels : 0);
  Lane l;
  l.place(a, at);
  const T* in = static_cast<const T*>(a.in) + row * a.ld_in;
  T* out = static_cast<T*>(a.out) + row * a.ld_out;
  const int h0 = static_cast<int>(blockIdx.y) * a.hpt, h1 = min(h0 + a.hpt, a.n_heads);
  const float part = 1.0f / static_cast<float>(a.head_dim);
  extern __shared__ __align__(16) uint8_t norm_smem[];
  const uint32_t ring = smem_u32(norm_smem);
  // Up to kNormHeads heads that are all queries or all keys.
  auto batch_end = [&](int h) { return min(h + kNormHeads, h < a.n_q ? min(h1, a.n_q) : h1); };
  int ahead = h0, filled = 0;  // the next batch to be copied, and its stage
  auto copy_next = [&] {
    if (ahead < h1) {
      const int end = batch_end(ahead);
#pragma unroll
      for (int j = 0; j < kNormHeads; ++j)
        if (ahead + j < end) l.copy(norm_slot<kNormHeads>(ring, filled, j), in + (ahead + j) * a.head_dim);
      ahead = end;
    }
    copy_async_commit();
    filled = filled + 1 == kNormStages ? 0 : filled + 1;
  };
#pragma unroll
  for (int j = 0; j < kNormStages * kNormHeads; ++j) l.clear(norm_slot<kNormHeads>(ring, 0, j));
#pragma unroll
  for (int i = 0; i < kNormStages - 1; ++i) copy_next();
  l.angles(a, tab, a.positions != nullptr ? static_cast<long long>(a.positions[row]) : row + a.pos_offset, 1.0f);
  int stage = 0;
  bool odd = false;
  for (int h = h0; h < h1;) {
    const int end = batch_end(h);
    copy_next();
    if (h == h0 || h == a.n_q) l.gains(h < a.n_q ? a.q_gain : a.k_gain);
    copy_async_wait<kNormStages - 1>();
    alignas(16) typename Lane::Raw v[kNormHeads];
    float x[Lane::kChannels], r[kNormHeads];
#pragma unroll
    for (int j = 0; j < kNormHeads; ++j) {
      if (h + j >= end) break;
      l.take(norm_slot<kNormHeads>(ring, stage, j), v[j]);
      l.widen(v[j], x);
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < Lane::kChannels; ++i) ss += x[i] * x[i];
      r[j] = ss;
    }
#pragma unroll
    for (int j = 0; j < kNormHeads; ++j)
      if (h + j < end) r[j] = inverse_root<T>(head_sum(r[j], a.lanes) * part + a.eps);
    if (kPart && (h == h0 || h == a.n_q)) odd = l.odd_gains();
    auto finish = [&](auto with_odd) {
#pragma unroll
      for (int j = 0; j < kNormHeads; ++j) {
        if (h + j >= end) break;
        l.widen(v[j], x);
#pragma unroll
        for (int i = 0; i < Lane::kChannels; ++i) x[i] *= r[j] * l.g[i];
        l.template turn<with_odd.value>(a, sh, x);
        if (live) l.store(out + (h + j) * a.head_dim, x);
      }
    };
    if (kPart && odd) finish(std::true_type());
    else finish(std::false_type());
    h = end;
    stage = stage + 1 == kNormStages ? 0 : stage + 1;
  }
}

constexpr int kNormBackHeads = 2;

template <class T, int kForm, bool kPart>
__global__ void __launch_bounds__(kNormThreads, 2) k_norm_rope_backward(const __grid_constant__ NormArgs a,
                                                                        const __grid_constant__ RopeTable tab) {
  using Lane = NormLane<T, kForm>;
  constexpr int kC = Lane::kChannels;
  __shared__ __align__(16) float staged[kForm == kShared ? kNormThreads * kC : 8 * 256];
  pdl_launch_dependents();
  pdl_wait();
  const bool keys = static_cast<int>(blockIdx.x) >= a.q_ctas;
  const int cta = static_cast<int>(blockIdx.x) - (keys ? a.q_ctas : 0);
  const int ctas = keys ? static_cast<int>(gridDim.x) - a.q_ctas : a.q_ctas;
  const int first = keys ? a.n_q : 0, heads = keys ? a.n_heads - a.n_q : a.n_q;
  const int at = static_cast<int>(threadIdx.x) & (a.lanes - 1);
  const int group = static_cast<int>(threadIdx.x) / a.lanes, groups = kNormThreads / a.lanes;
  float* sh = staged + (kForm == kShared ? (threadIdx.x - at) * kC : 0);
  Lane l;
  l.place(a, at);
  l.gains(keys ? a.k_gain : a.q_gain);
  // The kind's heads, kNormBackHeads of a row together, in the order of the rows: each group takes an equal run of
  // them, so that it forms a row's angles once, and as many copies are in flight at the end of a run as before.
  const int batches = (heads + kNormBackHeads - 1) / kNormBackHeads;  // of a row
  const long long total = static_cast<long long>(a.n_rows) * batches, all_groups = static_cast<long long>(ctas) * groups;
  const long long me = static_cast<long long>(cta) * groups + group;
  const long long t0 = total * me / all_groups, t1 = total * (me + 1) / all_groups;
  const int turns = static_cast<int>((total + all_groups - 1) / all_groups);  // (every group of a warp makes as many)
  const float part = 1.0f / static_cast<float>(a.head_dim);
  float2 g[kC / 2], dg[kC / 2];
#pragma unroll
  for (int i = 0; i < kC / 2; ++i) {
    g[i] = make_float2(l.g[2 * i], l.g[2 * i + 1]);
    dg[i] = make_float2(0.0f, 0.0f);
  }
  extern __shared__ __align__(16) uint8_t norm_smem[];
  const uint32_t ring = smem_u32(norm_smem);
  struct Spot {  // a batch: its place in the run, its row and place in the row
    long long t;
    int row, batch;
  };
  auto advance = [&](Spot& p) {
    ++p.t;
    if (++p.batch == batches) {
      p.batch = 0;
      ++p.row;
    }
  };
  auto has = [&](const Spot& p, int j) { return p.t < t1 && p.batch * kNormBackHeads + j < heads; };
  Spot now{t0, static_cast<int>(t0 / batches), 0};
  now.batch = static_cast<int>(t0 - static_cast<long long>(now.row) * batches);
  Spot next = now;
  int filled = 0, stage = 0;
  auto copy_next = [&] {
#pragma unroll
    for (int j = 0; j < kNormBackHeads; ++j)
      if (has(next, j)) {
        const long long h = first + next.batch * kNormBackHeads + j;
        l.copy(norm_slot<2 * kNormBackHeads>(ring, filled, 2 * j), static_cast<const T*>(a.in) + next.row * a.ld_in + h * a.head_dim);
        l.copy(norm_slot<2 * kNormBackHeads>(ring, filled, 2 * j + 1), static_cast<const T*>(a.dy) + next.row * a.ld_dy + h * a.head_dim);
      }
    advance(next);
    copy_async_commit();
    filled = filled + 1 == kNormStages ? 0 : filled + 1;
  };
#pragma unroll
  for (int j = 0; j < kNormStages * 2 * kNormBackHeads; ++j) l.clear(norm_slot<2 * kNormBackHeads>(ring, 0, j));
#pragma unroll
  for (int i = 0; i < kNormStages - 1; ++i) copy_next();
  for (int i = 0; i < turns; ++i) {
    copy_next();
    if (now.t < t1 && (i == 0 || now.batch == 0))
      l.angles(a, tab, a.positions != nullptr ? static_cast<long long>(a.positions[now.row]) : now.row + a.pos_offset, -1.0f);
    __syncwarp();
    copy_async_wait<kNormStages - 1>();
#pragma unroll
    for (int j = 0; j < kNormBackHeads; ++j) {
      const bool there = has(now, j);
      alignas(16) typename Lane::Raw raw;
      float2 x[kC / 2], w[kC / 2];
      l.take(norm_slot<2 * kNormBackHeads>(ring, stage, 2 * j), raw);
#pragma unroll
      for (int i = 0; i < kC / 2; ++i) x[i] = pair_of(&raw[0][0] + 2 * i);
      l.take(norm_slot<2 * kNormBackHeads>(ring, stage, 2 * j + 1), raw);
#pragma unroll
      for (int i = 0; i < kC / 2; ++i) w[i] = pair_of(&raw[0][0] + 2 * i);
      if (!there) {  // (what lies there is of an earlier batch, or nothing)
#pragma unroll
        for (int i = 0; i < kC / 2; ++i) x[i] = w[i] = make_float2(0.0f, 0.0f);
      }
      turn_x2<false>(a, l, sh, w);
      float2 ss2 = make_float2(0.0f, 0.0f), dot2 = ss2;
#pragma unroll
      for (int i = 0; i < kC / 2; ++i) {
        ss2 = fma_x2(x[i], x[i], ss2);
        dot2 = fma_x2(mul_x2(w[i], g[i]), x[i], dot2);
      }
      float ss = ss2.x + ss2.y, dot = dot2.x + dot2.y;
      head_sums(ss, dot, a.lanes);
      if (kPart && !isfinite(dot)) {  // as with any infinity or NaN of w: the pieces are turned once more, each channel by itself
        l.take(norm_slot<2 * kNormBackHeads>(ring, stage, 2 * j + 1), raw);
#pragma unroll
        for (int i = 0; i < kC / 2; ++i) w[i] = there ? pair_of(&raw[0][0] + 2 * i) : make_float2(0.0f, 0.0f);
        turn_x2<true>(a, l, sh, w);
      }
      const float r = inverse_root<T>(ss * part + a.eps);
      const float b = dot * part * (r * r) * r;
      const float2 rr = make_float2(r, r), bb = make_float2(-b, -b);
      float y[kC];
#pragma unroll
      for (int i = 0; i < kC / 2; ++i) {
        const float2 u = mul_x2(w[i], rr);
        dg[i] = fma_x2(u, x[i], dg[i]);
        const float2 v = fma_x2(u, g[i], mul_x2(x[i], bb));
        y[2 * i] = v.x;
        y[2 * i + 1] = v.y;
      }
      if (there)
        l.store(static_cast<T*>(a.out) + now.row * a.ld_out +
                    static_cast<long long>(first + now.batch * kNormBackHeads + j) * a.head_dim, y);
    }
    advance(now);
    stage = stage + 1 == kNormStages ? 0 : stage + 1;
  }
  if (a.part == nullptr) return;
  // The CTA's sums: its groups' lanes by shuffles, then its warps through shared memory.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kC / 2; ++i)
    for (int o = a.lanes; o < 32; o <<= 1) {
      dg[i].x += __shfl_xor_sync(0xffffffffu, dg[i].x, o);
      dg[i].y += __shfl_xor_sync(0xffffffffu, dg[i].y, o);
    }
  __syncthreads();
  if (lane < a.lanes) {
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if (l.ok[i / Lane::kVec]) staged[warp * 256 + l.start[i / Lane::kVec] + i % Lane::kVec] = i & 1 ? dg[i / 2].y : dg[i / 2].x;
  }
  __syncthreads();
  for (int ch = threadIdx.x; ch < a.head_dim; ch += kNormThreads) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; ++w) sum += staged[w * 256 + ch];
    a.part[static_cast<long long>(blockIdx.x) * a.head_dim + ch] = sum;
  }
}

// d_gain[c] = the sum of the CTAs' rows. Block (x, y): channels 32 x .. 32 x + 31 of the query
// gain (y = 0) or the key gain; a warp takes every eighth row.
__global__ void __launch_bounds__(256) k_gain_sum(const float* part, int head_dim, int q_ctas, int ctas, float* dq, float* dk) {
  __shared__ float sums[8][32];
  pdl_wait();
  float* out = blockIdx.y == 0 ? dq : dk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.y == 0 ? 0 : q_ctas, c1 = blockIdx.y == 0 ? q_ctas : ctas;
  const int ch = blockIdx.x * 32 + lane;
  if (out == nullptr) return;
  float sum = 0.0f;
  if (ch < head_dim) {
#pragma unroll 8
    for (int c = c0 + warp; c < c1; c += 8) sum += part[static_cast<long long>(c) * head_dim + ch];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && ch < head_dim) {
#pragma unroll
    for (int w = 1; w < 8; ++w) sum += sums[w][lane];
    out[ch] = sum;
  }
}

static rf_status check_norm_rope(const rf_norm_rope_desc* d) {
  if (d == nullptr) return fail(RF_ERR_INVALID_ARG, "desc is NULL");
  const rf_status st = check_rope(&d->rope);
  if (st != RF_OK) return st;
  if (d->rope.transpose) return fail(RF_ERR_INVALID_ARG, "transpose must be 0 (the gradient has its own call)");
  if (d->n_q_heads < 0 || d->n_q_heads > d->rope.n_heads)
    return fail(RF_ERR_INVALID_ARG, "need 0 <= n_q_heads <= n_heads");
  const float eps = static_cast<float>(d->eps);
  if (!(eps >= 1.1754944e-38f) || !std::isfinite(eps)) return fail(RF_ERR_INVALID_ARG, "eps must be > 0 and normal in fp32");
  return RF_OK;
}

// Arguments that both passes share, and the lanes of a head.
static NormArgs norm_args(const rf_norm_rope_desc* d, NormForm* form) {
  const rf_rope_desc& r = d->rope;
  NormArgs a{};
  a.pos_offset = r.pos_offset;
  a.n_rows = static_cast<int>(r.n_rows);
  a.n_heads = static_cast<int>(r.n_heads);
  a.n_q = static_cast<int>(d->n_q_heads);
  a.head_dim = static_cast<int>(r.head_dim);
  a.rot = static_cast<int>(r.rot_dim);
  a.amp = r.amplitude == 0.0 ? 1.0f : static_cast<float>(r.amplitude);
  a.eps = static_cast<float>(d->eps);
  const int channels = r.dtype == RF_BF16 ? 16 : 8;  // of a lane
  *form = r.layout == RF_ROPE_INTERLEAVED ? kPairs
          : a.rot % channels == 0 && a.head_dim % channels == 0 ? kPieces
                                                                 : kShared;
  a.lanes = 1;
  while (a.lanes * channels < a.head_dim) a.lanes *= 2;
  return a;
}

template <class T, int kForm, bool kPart>
static rf_status launch_norm(NormArgs& a, const RopeTable& t, int sms, cudaStream_t s) {
  // Heads per thread: as many as still leave two waves of threads, so that a small call spreads
  // over the GPU and a large one forms its angles once for many heads.
  const long long threads1 = static_cast<long long>(a.n_rows) * a.lanes;
  a.hpt = 1;
  while (a.hpt < 16 && threads1 * a.n_heads / (2 * a.hpt) >= 4096LL * sms) a.hpt *= 2;
  const dim3 grid(static_cast<unsigned>((threads1 + kNormThreads - 1) / kNormThreads),
                  static_cast<unsigned>((a.n_heads + a.hpt - 1) / a.hpt));
  static uint64_t done = 0;
  const rf_status st = set_smem_attr(reinterpret_cast<const void*>(&k_norm_rope<T, kForm, kPart>), norm_ring_bytes(kNormHeads), &done);
  if (st != RF_OK) return st;
  return cuda_check(launch_dependent(k_norm_rope<T, kForm, kPart>, grid, dim3(kNormThreads), norm_ring_bytes(kNormHeads), s, 1, a, t),
                    "k_norm_rope launch");
}
template <class T>
static rf_status launch_norm(NormArgs& a, const RopeTable& t, NormForm form, int sms, cudaStream_t s) {
  const bool part = a.rot < a.head_dim;
  if (form == kPieces) return part ? launch_norm<T, kPieces, true>(a, t, sms, s) : launch_norm<T, kPieces, false>(a, t, sms, s);
  if (form == kPairs) return part ? launch_norm<T, kPairs, true>(a, t, sms, s) : launch_norm<T, kPairs, false>(a, t, sms, s);
  return launch_norm<T, kShared, false>(a, t, sms, s);
}

// CTAs of the backward pass: two an SM, no more than there are batches to share out among their groups, the query
// heads' and the key heads' in proportion.
static int norm_ctas(const NormArgs& a, int sms, int* q_ctas) {
  const int groups = kNormThreads / a.lanes;
  const long long most = std::min(2 * sms, kNormMaxCtas - 1);
  auto needed = [&](long long h) { return (a.n_rows * ((h + kNormBackHeads - 1) / kNormBackHeads) + groups - 1) / groups; };
  const int n_k = a.n_heads - a.n_q;
  const long long q = std::min<long long>(needed(a.n_q), std::max<long long>(a.n_q > 0, most * a.n_q / a.n_heads));
  const long long k = std::min<long long>(needed(n_k), std::max<long long>(n_k > 0, most - most * a.n_q / a.n_heads));
  *q_ctas = static_cast<int>(q);
  return static_cast<int>(q + k);
}

template <class T, int kForm, bool kPart>
static rf_status launch_norm_backward(const NormArgs& a, const RopeTable& t, int ctas, cudaStream_t s) {
  static uint64_t done = 0;
  constexpr size_t bytes = norm_ring_bytes(2 * kNormBackHeads);
  const rf_status st = set_smem_attr(reinterpret_cast<const void*>(&k_norm_rope_backward<T, kForm, kPart>), bytes, &done);
  if (st != RF_OK) return st;
  return cuda_check(launch_dependent(k_norm_rope_backward<T, kForm, kPart>, dim3(static_cast<unsigned>(ctas)), dim3(kNormThreads), bytes, s,
                                     1, a, t),
                    "k_norm_rope_backward launch");
}
template <class T>
static rf_status launch_norm_backward(const NormArgs& a, const RopeTable& t, NormForm form, int ctas, cudaStream_t s) {
  const bool part = a.rot < a.head_dim;
  if (form == kPieces)
    return part ? launch_norm_backward<T, kPieces, true>(a, t, ctas, s) : launch_norm_backward<T, kPieces, false>(a, t, ctas, s);
  if (form == kPairs)
    return part ? launch_norm_backward<T, kPairs, true>(a, t, ctas, s) : launch_norm_backward<T, kPairs, false>(a, t, ctas, s);
  return launch_norm_backward<T, kShared, false>(a, t, ctas, s);
}

}  // namespace rf

using namespace rf;

extern "C" rf_status rf_norm_rope(const rf_norm_rope_desc* d, const void* in, const void* q_gain, const void* k_gain,
                                  void* out, const int32_t* positions, rf_stream_t stream) {
  clear_error();
  rf_status st = check_norm_rope(d);
  if (st != RF_OK) return st;
  if (d->rope.n_rows == 0) return RF_OK;
  if (!in || !out) return fail(RF_ERR_INVALID_ARG, "in and out must be non-NULL");
  if (!aligned16(in) || !aligned16(out) || !aligned16(q_gain) || !aligned16(k_gain))
    return fail(RF_ERR_ALIGN, "rows and gains must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return fail(RF_ERR_ALIGN, "positions must be 4-byte aligned");
  if (in == out && d->rope.ld_in != d->rope.ld_out) return fail(RF_ERR_INVALID_ARG, "in place needs ld_out = ld_in");
  int sms = 0;
  if ((st = current_device(&sms)) != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RopeTable tab = rope_table(&d->rope);
  NormForm form;
  NormArgs a = norm_args(d, &form);
  a.in = in;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.out = out;
  a.positions = positions;
  a.ld_in = d->rope.ld_in;
  a.ld_out = d->rope.ld_out;
  ProfScope prof(s, RF_STAGE_NORM_ROPE);
  return d->rope.dtype == RF_BF16 ? launch_norm<__nv_bfloat16>(a, tab, form, sms, s) : launch_norm<float>(a, tab, form, sms, s);
}

extern "C" size_t rf_norm_rope_backward_workspace_bytes(const rf_norm_rope_desc* d) {
  if (check_norm_rope(d) != RF_OK) return 0;
  Carve c(nullptr);
  c.take<float>(static_cast<size_t>(kNormMaxCtas) * d->rope.head_dim);
  return c.bytes();
}

extern "C" rf_status rf_norm_rope_backward(const rf_norm_rope_desc* d, const void* in, const void* q_gain,
                                           const void* k_gain, const void* d_out, const int32_t* positions, void* d_in,
                                           float* d_q_gain, float* d_k_gain, void* workspace, size_t workspace_bytes,
                                           rf_stream_t stream) {
  clear_error();
  rf_status st = check_norm_rope(d);
  if (st != RF_OK) return st;
  const bool sums = d_q_gain != nullptr || d_k_gain != nullptr;
  if (d->rope.n_rows > 0 && (!in || !d_out || !d_in)) return fail(RF_ERR_INVALID_ARG, "in, d_out and d_in must be non-NULL");
  if (!aligned16(in) || !aligned16(d_out) || !aligned16(d_in) || !aligned16(q_gain) || !aligned16(k_gain))
    return fail(RF_ERR_ALIGN, "rows and gains must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(d_q_gain) | reinterpret_cast<uintptr_t>(d_k_gain)) & 3u)
    return fail(RF_ERR_ALIGN, "arrays must be aligned to their elements");
  if (d_in == d_out && d->rope.ld_in != d->rope.ld_out)
    return fail(RF_ERR_INVALID_ARG, "d_in over d_out needs ld_out = ld_in");
  const int64_t hd = d->rope.head_dim;
  if (overlap(d_q_gain, hd, d_k_gain, hd)) return fail(RF_ERR_INVALID_ARG, "the gains' gradients must lie apart");
  const size_t need = rf_norm_rope_backward_workspace_bytes(d);
  if (sums && (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
    return fail(RF_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", need, workspace_bytes);
  if (d->rope.n_rows == 0 && !sums) return RF_OK;
  int sms = 0;
  if ((st = current_device(&sms)) != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RopeTable tab = rope_table(&d->rope);
  NormForm form;
  NormArgs a = norm_args(d, &form);
  a.in = in;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.dy = d_out;
  a.out = d_in;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.positions = positions;
  a.ld_in = d->rope.ld_in;
  a.ld_dy = d->rope.ld_out;
  a.ld_out = d->rope.ld_in;
  const int ctas = norm_ctas(a, sms, &a.q_ctas);
  if (ctas > 0) {
    ProfScope prof(s, RF_STAGE_NORM_ROPE);
    st = d->rope.dtype == RF_BF16 ? launch_norm_backward<__nv_bfloat16>(a, tab, form, ctas, s)
                                  : launch_norm_backward<float>(a, tab, form, ctas, s);
    if (st != RF_OK) return st;
  }
  if (!sums) return RF_OK;
  ProfScope prof(s, RF_STAGE_NORM_ROPE);
  return cuda_check(launch_dependent(k_gain_sum, dim3(static_cast<unsigned>((hd + 31) / 32), 2), dim3(256), 0, s, 1,
                                     static_cast<const float*>(a.part), static_cast<int>(hd), a.q_ctas, ctas, d_q_gain,
                                     d_k_gain),
                    "k_gain_sum launch");
}
