// Sampling from logits by temperature, top-k, top-p and min-p, from given random numbers (rf_sample).
//
// In the order of falling logit, the lowest token first among equals, each filter keeps a first
// run of the tokens: the first k; of those the shortest run whose mass reaches p of theirs; of those
// the ones of at least min_p of the first one's weight. So what stays is a run too, and is given by its
// last token. Weights are w = 2^-t, t = (max - logit) log2(e) / T.
//
// Where the runs end is decided as in 64 bits. Logits are compared as they are. Masses are integers,
// so that sums do not depend on their order: t is a sum of two fp32 numbers, and 2^-t comes from a table
// of 64 powers and a polynomial, within about 2^-39 of the greatest weight (token_mass). In fp32 sums a
// flat row's nucleus would end a token early or late every few dozen rows.
//
// One cluster of up to eight CTAs a row, each with a share of the vocabulary, which it reads once for the
// maximum and then again, from L2:
//   few tokens (top-k of at most 128)   The threads of the cluster form 128 (or 64, ...) groups. The least
//             of the groups' maxima is a logit that at least so many tokens reach: what lies below it
//             cannot stay. The others, a few hundred, are listed and sorted; all filters and the draw then
//             take the list alone.
//   any other  A table of counts and masses by octaves of weight (each thread adds to 24 entries of its own
//             in shared memory: no atomics). A run's end lies in one octave; finer tables, of 2048 bins
//             over the octave's (logit, token) pairs, narrow it down to a few tokens, which are sorted. A
//             pass over all then adds up the weights and draws, another writes probabilities.
//
// Bound: the logits' bytes (and the probabilities'), beside some 40 operations a token where masses
// are formed.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "rf_device.cuh"
#include "rf_host.h"

namespace rf {
namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kSampleCtas = 8;        // CTAs of a cluster (the portable limit)
constexpr int kSampleShare = 2048;    // least tokens of a CTA
constexpr int kOctaves = 24;          // the last one holds every smaller weight as well
constexpr int kBins = 2048;
constexpr int kListed = 1024;         // tokens that are sorted at most
constexpr int kFewTokens = 128;       // top-k up to which tokens are listed at once: G groups leave about
                                      // G (ln G + 0.6) tokens, some 700 of 128
constexpr int kSampleMaxVocab = 1 << 20;
constexpr int kMassBits = 40;         // a weight of 1, within its octave
constexpr int kCommonBits = 43;       // a weight of 1, over all octaves: 2^20 of them are 2^63
static_assert(kSampleMaxVocab / kSampleThreads < (1 << (64 - kMassBits - 12)), "a thread's counts and masses share 64 bits");

struct PowerTable {
  unsigned long long t[65];  // 2^(40 - i/64)
};

struct SampleArgs {
  const void* logits;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* noise;
  float* probs;
  int32_t* token;
  float* logprob;
  int32_t* n_kept;
  int32_t* dev_status;
  long long ld_logits, ld_noise, ld_probs;
  int vocab;
};

// A token's place in the order: falling logit, then rising token. -0 and 0 are equal.
__device__ __forceinline__ unsigned rising_key(float x) {
  const unsigned b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(unsigned k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ unsigned long long place_of(float x, int i) {
  return (static_cast<unsigned long long>(~rising_key(x)) << 20) | static_cast<unsigned>(i);
}
__device__ __forceinline__ float place_value(unsigned long long p) { return key_value(~static_cast<unsigned>(p >> 20)); }
__device__ __forceinline__ int place_token(unsigned long long p) { return static_cast<int>(p & 0xfffffu); }

struct Scale {
  float m, c, c_lo;  // the row's maximum; log2(e) / T = c + c_lo
};

// t = (m - x) c as hi + lo, to about 2^-46 of itself.
__device__ __forceinline__ void distance(const Scale& s, float x, float& hi, float& lo) {
  const float d = s.m - x, b = d - s.m;
  const float e = (s.m - (d - b)) - (x + b);  // m - x = d + e
  hi = d * s.c;
  lo = fmaf(d, s.c, -hi);
  lo = fmaf(d, s.c_lo, lo);
  lo = fmaf(e, s.c, lo);
}
// 2^-t in fp32 (0 below 2^-126).
__device__ __forceinline__ float weight_of(const Scale& s, float x) {
  float hi, lo;
  distance(s, x, hi, lo);
  return hi < 150.0f ? exp2f_ftz(-hi) * fmaf(lo, -0.693147181f, 1.0f) : 0.0f;
}

// A token's octave and its mass there, 2^(40 + octave - t). With r = t - its whole part = k/64 + r',
// 2^-r = 2^(-k/64) (1 - q), q = z - z^2/2 + z^3/6 - z^4/24, z = r' ln 2 < 0.0055: the next term is
// 2^-44. z is kept as a sum of two numbers; the other terms are below 2^-16, their rounding below 2^-39.
__device__ __forceinline__ int token_mass(const Scale& s, float x, const unsigned long long* power, unsigned long long& mass) {
  float hi, lo;
  distance(s, x, hi, lo);
  if (!(hi < static_cast<float>(kOctaves + kMassBits))) {
    mass = 0;
    return kOctaves - 1;
  }
  const int n = static_cast<int>(hi);
  const float r = hi - static_cast<float>(n);
  constexpr float kRound = 12582912.0f;  // 1.5 2^23: adding it rounds to whole numbers
  const float y = fmaf(r, 64.0f, kRound);
  const int k = __float_as_int(y) - 0x4b400000;
  const float rest = fmaf(y - kRound, -0.015625f, r);
  const float a = rest + lo, b = lo - (a - rest);
  constexpr float kLn2 = 0.693147182f, kLn2Lo = -1.90465421e-9f;
  const float z = a * kLn2;
  float tail = fmaf(a, kLn2, -z);
  tail = fmaf(a, kLn2Lo, tail);
  tail = fmaf(b, kLn2, tail);
  tail = fmaf(-z * z, fmaf(-z, fmaf(-z, 0.0416666667f, 0.166666667f), 0.5f), tail);
  // q in units of 2^-38
  const float u = fmaf(z, 16777216.0f, kRound);
  const float left = fmaf(u - kRound, -5.9604644775390625e-8f, z) + tail;
  const int q = (__float_as_int(u) - 0x4b400000) * 16384 + (__float_as_int(fmaf(left, 274877906944.0f, kRound)) - 0x4b400000);
  const unsigned long long p = power[k];
  const long long cut = (static_cast<long long>(static_cast<int>((p + 512) >> 10)) * q) >> 28;
  const int octave = min(n, kOctaves - 1);
  mass = (p - static_cast<unsigned long long>(cut)) >> (n - octave);
  return octave;
}
// An octave's mass over all octaves, rounded down.
__device__ __forceinline__ unsigned long long common_mass(unsigned long long mass, int octave) {
  return (mass << (kCommonBits - kMassBits)) >> octave;
}

// f(first token, values) for the tokens v0 <= i < v1 of a row: 16 bytes at a time between the row's
// first and last 16-byte boundaries, one token at a time outside them. A thread's tokens rise.
template <class T, class F>
__device__ __forceinline__ void for_tokens(const T* row, int v0, int v1, F f) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T)), kBatch = 2;
  const int tid = threadIdx.x;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row + v0) & 15u) / sizeof(T));
  const int head = min(v1 - v0, (kVec - off) % kVec);
  auto one = [&](int i) {
    float x[1];
    if constexpr (sizeof(T) == 2) x[0] = __bfloat162float(row[i]);
    else x[0] = row[i];
    f(i, x);
  };
  if (tid < head) one(v0 + tid);
  const int first = v0 + head, pieces = (v1 - first) / kVec;
  for (int p0 = tid; p0 < pieces; p0 += kBatch * kSampleThreads) {
    uint4 raw[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (p0 + j * kSampleThreads < pieces) raw[j] = reinterpret_cast<const uint4*>(row + first)[p0 + j * kSampleThreads];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (p0 + j * kSampleThreads >= pieces) break;
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
      float x[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if constexpr (sizeof(T) == 2) x[e] = u2f(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        else x[e] = u2f(w[e]);
      }
      f(first + (p0 + j * kSampleThreads) * kVec, x);
    }
  }
  const int last = first + pieces * kVec + tid;
  if (last < v1) one(last);
}

struct SampleShared {
  unsigned long long power[65];
  unsigned long long warp_sum[kSampleWarps];
  unsigned warp_count[kSampleWarps];
  float warp_key[kSampleWarps];
  // from every CTA of the cluster, by the parity of the turn
  unsigned long long best[2][kSampleCtas];
  unsigned least[2][kSampleCtas];
  float sum[2][kSampleCtas];
  unsigned kept[2][kSampleCtas];
  unsigned listed[2][kSampleCtas];
  // counts and masses by octaves: every CTA's, then the row's
  unsigned octave_count[kSampleCtas][kOctaves];
  unsigned long long octave_mass[kSampleCtas][kOctaves];
  unsigned count[kOctaves];
  unsigned long long mass[kOctaves];
  // where a run ends
  unsigned long long found_place, found_mass;
  unsigned found_bin, found_count, found_in;
  int n_list;
  double min_away;  // T ln(min_p)
  float lowest;     // the least logit that min_p lets pass
};
// One area for what is not needed at the same time: the threads' octaves, or tables and lists.
struct SampleTables {
  unsigned long long mass[kBins];      // of this CTA
  unsigned count[kBins];
  unsigned long long all_mass[kBins];  // of the cluster
  unsigned all_count[kBins];
  unsigned long long own_place[kListed], own_mass[kListed];
  unsigned long long place[kListed], list_mass[kListed];
};
constexpr size_t kSampleArea = std::max(sizeof(SampleTables), sizeof(unsigned long long) * kOctaves * kSampleThreads);

// What all threads of a row's cluster know.
struct Row {
  int rank, ctas, v0, v1;
  Scale scale;
  bool top_inf;  // the maximum is +inf: those tokens share all weight, as if theirs were 0 and all others' -inf
  int turn;
};

// A logit as the filters see it: NaN as -inf.
__device__ __forceinline__ float seen(const Row& r, float x) {
  x = fmaxf(x, -INFINITY);
  return r.top_inf ? (x == INFINITY ? 0.0f : -INFINITY) : x;
}

__device__ __forceinline__ unsigned long long warp_max(unsigned long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// The sums of the pairs of the CTA's threads before this one (whole CTA).
__device__ __forceinline__ void before_sums(SampleShared& sh, unsigned& count, unsigned long long& mass) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned c = count;
  unsigned long long m = mass;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned c1 = __shfl_up_sync(0xffffffffu, c, o);
    const unsigned long long m1 = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) {
      c += c1;
      m += m1;
    }
  }
  __syncthreads();
  if (lane == 31) {
    sh.warp_count[warp] = c;
    sh.warp_sum[warp] = m;
  }
  __syncthreads();
  unsigned c0 = 0;
  unsigned long long m0 = 0;
  for (int w = 0; w < warp; ++w) {
    c0 += sh.warp_count[w];
    m0 += sh.warp_sum[w];
  }
  count = c0 + c - count;
  mass = m0 + m - mass;
}

// Sorts the list by place (whole CTA), padded to a power of two with places beyond all.
__device__ __forceinline__ void sort_list(SampleTables& t, int n) {
  int size = 2;
  while (size < n) size *= 2;
  for (int i = n + static_cast<int>(threadIdx.x); i < size; i += kSampleThreads) {
    t.place[i] = ~0ull;
    t.list_mass[i] = 0;
  }
  __syncthreads();
  for (int k = 2; k <= size; k *= 2) {
    for (int j = k / 2; j > 0; j /= 2) {
      for (int p = threadIdx.x; p < size / 2; p += kSampleThreads) {
        const int i = 2 * p - (p & (j - 1)), o = i + j;
        const unsigned long long a = t.place[i], b = t.place[o];
        if ((a > b) == ((i & k) == 0)) {
          t.place[i] = b;
          t.place[o] = a;
          const unsigned long long m = t.list_mass[i];
          t.list_mass[i] = t.list_mass[o];
          t.list_mass[o] = m;
        }
      }
      __syncthreads();
    }
  }
}

// Every CTA's listed tokens into the lists of all; false (for all of the cluster) where they are more
// than a list holds. sh.n_list tokens were counted by this CTA, of which own_place has the first ones.
__device__ __forceinline__ bool join_lists(cg::cluster_group& cl, SampleShared& sh, SampleTables& t, Row& r, int* n) {
  __syncthreads();
  const int own = sh.n_list;
  if (threadIdx.x < static_cast<unsigned>(r.ctas)) *cl.map_shared_rank(&sh.listed[r.turn & 1][r.rank], threadIdx.x) = own;
  cl.sync();
  int before = 0, all = 0;
  for (int c = 0; c < r.ctas; ++c) {
    const int x = static_cast<int>(sh.listed[r.turn & 1][c]);
    all += x;
    if (c < r.rank) before += x;
  }
  ++r.turn;
  *n = all;
  if (all > kListed) return false;
  for (int x = threadIdx.x; x < own * r.ctas; x += kSampleThreads) {
    const int c = x / own, i = x - c * own;
    *cl.map_shared_rank(&t.place[before + i], c) = t.own_place[i];
    *cl.map_shared_rank(&t.list_mass[before + i], c) = t.own_mass[i];
  }
  cl.sync();
  return true;
}

// Where a run ends: its last token's place, and the mass up to there, the token's own included.
struct End {
  unsigned long long place, mass;
};

// The end of the run of `target` tokens (kByMass false), or of the shortest run of mass `target`, from the
// octaves' table. Every CTA of the cluster comes to the same result.
template <bool kByMass, class T>
__device__ End find_end(cg::cluster_group& cl, SampleShared& sh, SampleTables& t, Row& r, const T* row, float temperature,
                        unsigned long long target) {
  int octave = 0;
  unsigned long long base = 0;  // mass before the octave
  for (; octave < kOctaves - 1; ++octave) {
    const unsigned long long step = kByMass ? common_mass(sh.mass[octave], octave) : sh.count[octave];
    if (target <= step) break;
    target -= step;
    base += common_mass(sh.mass[octave], octave);
  }
  unsigned in = sh.count[octave];
  if (kByMass) target = ((target << octave) + ((1ull << (kCommonBits - kMassBits)) - 1)) >> (kCommonBits - kMassBits);
  unsigned long long inside = 0;  // mass of the octave before the range below
  // The octave's places, a little wider than it is: what is not of the octave is left out by its octave.
  const float step = temperature * 0.693147181f;
  float high = r.scale.m - step * static_cast<float>(octave), low = r.scale.m - step * static_cast<float>(octave + 1);
  const float slack = 4e-6f * (fabsf(r.scale.m) + step * static_cast<float>(octave + 1));
  high = octave == 0 ? r.scale.m : fminf(high + slack, r.scale.m);
  low = octave == kOctaves - 1 ? -FLT_MAX : fmaxf(low - slack, -FLT_MAX);
  unsigned long long lo = place_of(high, 0), hi = place_of(low, kSampleMaxVocab - 1);
  auto place_in = [&](float x, int i, unsigned long long& p, unsigned long long& m) {
    if (!(x > -INFINITY)) return false;
    p = place_of(x, i);
    if (p < lo || p > hi) return false;
    return token_mass(r.scale, x, sh.power, m) == octave;
  };
  while (in > kListed) {
    const int width = 64 - __clzll(static_cast<long long>(hi - lo));
    const int shift = max(0, width - 11);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kSampleThreads) {
      t.mass[i] = 0;
      t.count[i] = 0;
    }
    __syncthreads();
    for_tokens(row, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e) {
        unsigned long long p, m;
        if (place_in(seen(r, x[e]), i + e, p, m)) {
          const int bin = static_cast<int>((p - lo) >> shift);
          atomicAdd(&t.count[bin], 1u);
          atomicAdd(&t.mass[bin], m);
        }
      }
    });
    __syncthreads();
    cl.sync();
    // the CTA's share of the bins, summed over the cluster and given to all
    const int per = kBins / r.ctas;
    for (int i = threadIdx.x; i < per; i += kSampleThreads) {
      const int bin = r.rank * per + i;
      unsigned c = 0;
      unsigned long long m = 0;
      for (int k = 0; k < r.ctas; ++k) {
        c += *cl.map_shared_rank(&t.count[bin], k);
        m += *cl.map_shared_rank(&t.mass[bin], k);
      }
      for (int k = 0; k < r.ctas; ++k) {
        *cl.map_shared_rank(&t.all_count[bin], k) = c;
        *cl.map_shared_rank(&t.all_mass[bin], k) = m;
      }
    }
    cl.sync();
    const int b0 = threadIdx.x * (kBins / kSampleThreads);
    unsigned c = 0;
    unsigned long long m = 0;
#pragma unroll
    for (int i = 0; i < kBins / kSampleThreads; ++i) {
      c += t.all_count[b0 + i];
      m += t.all_mass[b0 + i];
    }
    if (threadIdx.x == 0) {  // (logits that change under the kernel: all CTAs still agree)
      sh.found_bin = 0;
      sh.found_count = sh.found_in = 0;
      sh.found_mass = 0;
    }
    before_sums(sh, c, m);
#pragma unroll
    for (int i = 0; i < kBins / kSampleThreads; ++i) {
      const unsigned c1 = c + t.all_count[b0 + i];
      const unsigned long long m1 = m + t.all_mass[b0 + i];
      if (kByMass ? (m < target && target <= m1) : (c < target && target <= c1)) {
        sh.found_bin = b0 + i;
        sh.found_count = c;
        sh.found_mass = m;
        sh.found_in = c1 - c;
      }
      c = c1;
      m = m1;
    }
    __syncthreads();
    lo += static_cast<unsigned long long>(sh.found_bin) << shift;
    hi = min(hi, lo + ((1ull << shift) - 1));
    in = sh.found_in;
    inside += sh.found_mass;
    target -= kByMass ? sh.found_mass : sh.found_count;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  for_tokens(row, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
    for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e) {
      unsigned long long p, m;
      if (place_in(seen(r, x[e]), i + e, p, m)) {
        const int at = atomicAdd(&sh.n_list, 1);
        if (at < kListed) {
          t.own_place[at] = p;
          t.own_mass[at] = m;
        }
      }
    }
  });
  int n = 0;
  join_lists(cl, sh, t, r, &n);
  n = min(n, kListed);
  if (threadIdx.x == 0) {  // (as above)
    sh.found_place = hi;
    sh.found_mass = 0;
  }
  sort_list(t, n);
  const int i0 = threadIdx.x * 2;
  unsigned c = 0;
  unsigned long long m = 0;
  for (int i = i0; i < min(i0 + 2, n); ++i) m += t.list_mass[i];
  before_sums(sh, c, m);
  for (int i = i0; i < min(i0 + 2, n); ++i) {
    const unsigned long long m1 = m + t.list_mass[i];
    if (kByMass ? (m < target && target <= m1) : static_cast<unsigned long long>(i + 1) == target) {
      sh.found_place = t.place[i];
      sh.found_mass = m1;
    }
    m = m1;
  }
  __syncthreads();
  const End end{sh.found_place, base + common_mass(inside + sh.found_mass, octave)};
  __syncthreads();
  return end;
}

// The least mass that a run must reach: p of `all`, rounded up, at least 1.
__device__ __forceinline__ unsigned long long mass_target(float p, unsigned long long all) {
  const unsigned long long f = __float2ull_rz(p * 18446744073709551616.0f);  // p < 1
  return max(1ull, __umul64hi(f, all) + (f * all != 0));
}

template <class T>
__global__ void __launch_bounds__(kSampleThreads, 2) k_sample(const __grid_constant__ SampleArgs a,
                                                              const __grid_constant__ PowerTable powers) {
  extern __shared__ __align__(16) uint8_t area[];
  __shared__ SampleShared sh;
  SampleTables& t = *reinterpret_cast<SampleTables*>(area);
  cg::cluster_group cl = cg::this_cluster();
  Row r{};
  r.rank = static_cast<int>(cl.block_rank());
  r.ctas = static_cast<int>(cl.num_blocks());
  const long long row_of = blockIdx.x / static_cast<unsigned>(r.ctas);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = ((a.vocab + r.ctas - 1) / r.ctas + 7) & ~7;
  r.v0 = min(r.rank * share, a.vocab);
  r.v1 = min(r.v0 + share, a.vocab);
  pdl_launch_dependents();
  for (int i = tid; i < 65; i += kSampleThreads) sh.power[i] = powers.t[i];
  if (tid == 0) sh.n_list = 0;
  cl.barrier_arrive();  // (waited for below: every CTA of the cluster runs before another writes to it)
  pdl_wait();
  const T* row = static_cast<const T*>(a.logits) + row_of * a.ld_logits;
  float* probs = a.probs != nullptr ? a.probs + row_of * a.ld_probs : nullptr;
  const float temperature = a.temperature != nullptr ? a.temperature[row_of] : 1.0f;
  const int top_k = a.top_k != nullptr ? a.top_k[row_of] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[row_of] : 1.0f;
  const float min_p = a.min_p != nullptr ? a.min_p[row_of] : 0.0f;
  const bool good = (temperature == 0.0f || (temperature >= 0x1p-100f && temperature <= 0x1p100f)) && top_k >= 0 &&
                    top_p >= 0.0f && min_p >= 0.0f && min_p <= 1.0f;

  // The maximum and its lowest token; the threads' maxima.
  float top = -INFINITY;
  int top_i = 0;
  if (good)
    for_tokens(row, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e)
        if (x[e] > top) {
          top = x[e];
          top_i = i + e;
        }
    });
  if (min_p > 0.0f && tid == kSampleThreads - 1) sh.min_away = static_cast<double>(temperature) * log(static_cast<double>(min_p));
  const unsigned long long mine =
      top > -INFINITY ? (static_cast<unsigned long long>(rising_key(top)) << 32) | (0xffffffffu - static_cast<unsigned>(top_i)) : 0ull;
  unsigned long long best = warp_max(mine);
  // few tokens: groups of threads of this CTA, at least top_k of them in the cluster
  int groups = 0;
  unsigned least = 0xffffffffu;
  if (top_k > 0 && top_k <= kFewTokens) {
    groups = 1;
    while (groups * r.ctas < top_k) groups *= 2;
    const int size = kSampleThreads / groups;  // threads of a group, a power of two
    unsigned k = rising_key(top);
    for (int o = 1; o < min(size, 32); o <<= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
    if (size < 32) k = __reduce_min_sync(0xffffffffu, k);
    if (lane == 0) sh.warp_count[warp] = k;
  }
  if (lane == 0) sh.warp_sum[warp] = best;
  __syncthreads();
  if (warp == 0) {
    best = warp_max(lane < kSampleWarps ? sh.warp_sum[lane] : 0ull);
    if (groups > 0) {
      unsigned k = lane < kSampleWarps ? sh.warp_count[lane] : 0u;
      for (int o = 1; o < kSampleThreads / groups / 32; o <<= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
      least = __reduce_min_sync(0xffffffffu, lane < kSampleWarps ? k : 0xffffffffu);
    }
  }
  cl.barrier_wait();
  if (warp == 0 && lane < r.ctas) {
    *cl.map_shared_rank(&sh.best[0][r.rank], lane) = best;
    *cl.map_shared_rank(&sh.least[0][r.rank], lane) = least;
  }
  cl.sync();
  best = 0;
  for (int c = 0; c < r.ctas; ++c) {
    best = max(best, sh.best[0][c]);
    least = c == 0 ? sh.least[0][c] : min(least, sh.least[0][c]);
  }
  r.turn = 1;

  auto token_of = [](unsigned long long pair) { return static_cast<int>(0xffffffffu - static_cast<unsigned>(pair & 0xffffffffu)); };
  auto zero_probs = [&] {
    if (probs != nullptr)
      for (int i = r.v0 + tid; i < r.v1; i += kSampleThreads) probs[i] = 0.0f;
  };
  auto answer = [&](int token, float logprob, int kept) {
    if (a.token != nullptr) a.token[row_of] = token;
    if (a.logprob != nullptr) a.logprob[row_of] = logprob;
    if (a.n_kept != nullptr) a.n_kept[row_of] = kept;
  };
  if (best == 0) {  // nothing to choose from, or a setting out of range
    zero_probs();
    if (r.rank == 0 && tid == 0) {
      answer(-1, -INFINITY, 0);
      if (!good) record_status(a.dev_status, RF_ERR_INVALID_ARG);
    }
    return;
  }
  const int first = token_of(best);
  r.scale.m = key_value(static_cast<unsigned>(best >> 32));
  if (temperature == 0.0f) {
    zero_probs();
    __syncthreads();
    if (probs != nullptr && tid == 0 && first >= r.v0 && first < r.v1) probs[first] = 1.0f;
    if (r.rank == 0 && tid == 0) answer(first, 0.0f, 1);
    return;
  }
  r.top_inf = r.scale.m == INFINITY;
  if (r.top_inf) {
    r.scale.m = 0.0f;
    least = least == rising_key(INFINITY) ? rising_key(0.0f) : 0u;
  }
  {
    constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596303e-8f;
    r.scale.c = kLog2e / temperature;
    r.scale.c_lo = (fmaf(-r.scale.c, temperature, kLog2e) + kLog2eLo) / temperature;
  }
  if (tid == 0) {
    float f = -INFINITY;
    if (min_p > 0.0f) f = __double2float_ru(static_cast<double>(r.scale.m) + sh.min_away);
    sh.lowest = f;
  }
  __syncthreads();
  const float lowest = sh.lowest;

  const float* noise = a.noise != nullptr ? a.noise + row_of * a.ld_noise : nullptr;
  auto pair_of = [](float score, int i) {
    return (static_cast<unsigned long long>(__float_as_uint(score)) << 32) | (0xffffffffu - static_cast<unsigned>(i));
  };
  auto score_of = [&](float w, int i) { return w > 0.0f ? __fdiv_rn(w, noise[i]) : 0.0f; };
  auto logprob_of = [&](float x, float total) {
    float hi, lo;
    distance(r.scale, x, hi, lo);
    return -(hi + lo) * 0.693147181f - logf(total);
  };

  // Few tokens: list what reaches the least group's maximum.
  int n = 0;
  if (groups > 0 && least > rising_key(-INFINITY)) {
    for_tokens(row, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e) {
        const float y = seen(r, x[e]);
        if (rising_key(y) >= least) {
          const int at = atomicAdd(&sh.n_list, 1);
          if (at < kListed) {
            unsigned long long m;
            const int octave = token_mass(r.scale, y, sh.power, m);
            t.own_place[at] = place_of(y, i + e);
            t.own_mass[at] = common_mass(m, octave);
          }
        }
      }
    });
    if (join_lists(cl, sh, t, r, &n)) {
      sort_list(t, n);
      int kept = min(top_k, n);
      if (top_p < 1.0f) {
        const int i0 = tid * 2;
        unsigned c = 0;
        unsigned long long m = 0;
        for (int i = i0; i < min(i0 + 2, n); ++i) m += t.list_mass[i];
        before_sums(sh, c, m);
        unsigned long long x = m;
        for (int i = i0; i < min(i0 + 2, n); ++i) {
          x += t.list_mass[i];
          if (i == kept - 1) sh.found_mass = x;
        }
        __syncthreads();
        const unsigned long long target = mass_target(top_p, sh.found_mass);
        for (int i = i0; i < min(i0 + 2, n); ++i) {
          const unsigned long long m1 = m + t.list_mass[i];
          if (m < target && target <= m1) sh.found_count = i + 1;
          m = m1;
        }
        __syncthreads();
        kept = min(kept, static_cast<int>(sh.found_count));
      }
      // (at most top_k tokens, a quarter of the threads)
      kept = __syncthreads_count(tid < kept && place_value(t.place[tid]) >= lowest);
      float w = 0.0f, score = 0.0f;
      int i = 0;
      if (tid < kept) {
        i = place_token(t.place[tid]);
        w = weight_of(r.scale, place_value(t.place[tid]));
        if (a.token != nullptr && r.rank == 0) score = score_of(w, i);
      }
      float total = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      const unsigned long long pick = warp_max(tid < kept ? pair_of(score, i) : 0ull);
      if (lane == 0) {
        sh.warp_key[warp] = total;
        sh.warp_sum[warp] = pick;
      }
      zero_probs();
      __syncthreads();
      total = 0.0f;
      best = 0;
      for (int x = 0; x < kFewTokens / 32; ++x) {
        total += sh.warp_key[x];
        best = max(best, sh.warp_sum[x]);
      }
      if (probs != nullptr && tid < kept && i >= r.v0 && i < r.v1) probs[i] = w / total;
      // the token's own thread, or the first one's where none is drawn
      if (r.rank == 0 && tid < kept && i == (a.token != nullptr ? token_of(best) : place_token(t.place[0])))
        answer(i, logprob_of(place_value(t.place[tid]), total), kept);
      return;
    }
  }

  // Any number of tokens. The last one that stays, by logit and token:
  float last = -INFINITY;
  int last_i = -1;
  if ((top_k > 0 && top_k < a.vocab) || top_p < 1.0f) {
    unsigned long long* column = reinterpret_cast<unsigned long long*>(area) + tid;
    __syncthreads();
#pragma unroll
    for (int o = 0; o < kOctaves; ++o) column[o * kSampleThreads] = 0;
    for_tokens(row, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e) {
        const float y = seen(r, x[e]);
        if (y > -INFINITY) {
          unsigned long long m;
          const int o = token_mass(r.scale, y, sh.power, m);
          column[o * kSampleThreads] += m + (1ull << 52);
        }
      }
    });
    __syncthreads();
    for (int o = warp; o < kOctaves; o += kSampleWarps) {
      const unsigned long long* of = reinterpret_cast<const unsigned long long*>(area) + o * kSampleThreads + lane;
      unsigned c = 0;
      unsigned long long m = 0;
#pragma unroll
      for (int i = 0; i < kSampleThreads; i += 32) {
        c += static_cast<unsigned>(of[i] >> 52);
        m += of[i] & ((1ull << 52) - 1);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) {
        c += __shfl_xor_sync(0xffffffffu, c, s);
        m += __shfl_xor_sync(0xffffffffu, m, s);
      }
      if (lane < r.ctas) {
        *cl.map_shared_rank(&sh.octave_count[r.rank][o], lane) = c;
        *cl.map_shared_rank(&sh.octave_mass[r.rank][o], lane) = m;
      }
    }
    cl.sync();
    if (tid < kOctaves) {
      unsigned c = 0;
      unsigned long long m = 0;
      for (int k = 0; k < r.ctas; ++k) {
        c += sh.octave_count[k][tid];
        m += sh.octave_mass[k][tid];
      }
      sh.count[tid] = c;
      sh.mass[tid] = m;
    }
    __syncthreads();
    unsigned long long all = 0;
    unsigned valid = 0;
    for (int o = 0; o < kOctaves; ++o) {
      all += common_mass(sh.mass[o], o);
      valid += sh.count[o];
    }
    End end{~0ull, all};
    if (top_k > 0 && static_cast<unsigned>(top_k) < valid) end = find_end<false>(cl, sh, t, r, row, temperature, top_k);
    if (top_p < 1.0f) {
      const End by_mass = find_end<true>(cl, sh, t, r, row, temperature, mass_target(top_p, end.mass));
      end.place = min(end.place, by_mass.place);
    }
    if (end.place != ~0ull) {
      last = place_value(end.place);
      last_i = place_token(end.place);
    }
  }
  if (lowest > last) {
    last = lowest;
    last_i = kSampleMaxVocab;
  }
  auto stays = [&](float x, int i) { return x > last || (x == last && i <= last_i); };
  float total = 0.0f;
  unsigned kept = 0;
  best = 0;
  for_tokens(row, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
    for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e) {
      const float y = seen(r, x[e]);
      if (stays(y, i + e)) {
        const float w = weight_of(r.scale, y);
        total += w;
        ++kept;
        if (a.token != nullptr) best = max(best, pair_of(score_of(w, i + e), i + e));
      }
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  kept = __reduce_add_sync(0xffffffffu, kept);
  best = warp_max(best);
  __syncthreads();
  if (lane == 0) {
    sh.warp_key[warp] = total;
    sh.warp_count[warp] = kept;
    sh.warp_sum[warp] = best;
  }
  __syncthreads();
  if (warp == 0) {
    total = lane < kSampleWarps ? sh.warp_key[lane] : 0.0f;
    kept = lane < kSampleWarps ? sh.warp_count[lane] : 0u;
    best = warp_max(lane < kSampleWarps ? sh.warp_sum[lane] : 0ull);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    kept = __reduce_add_sync(0xffffffffu, kept);
    if (lane < r.ctas) {
      *cl.map_shared_rank(&sh.sum[r.turn & 1][r.rank], lane) = total;
      *cl.map_shared_rank(&sh.kept[r.turn & 1][r.rank], lane) = kept;
      *cl.map_shared_rank(&sh.best[r.turn & 1][r.rank], lane) = best;
    }
  }
  cl.sync();
  total = 0.0f;
  kept = 0;
  best = 0;
  for (int c = 0; c < r.ctas; ++c) {
    total += sh.sum[r.turn & 1][c];
    kept += sh.kept[r.turn & 1][c];
    best = max(best, sh.best[r.turn & 1][c]);
  }
  // The CTA that holds the token answers: its logit is read before probabilities are written over it.
  const int token = a.token != nullptr ? token_of(best) : first;
  if (tid == 0 && token >= r.v0 && token < r.v1) {
    float x;
    if constexpr (sizeof(T) == 2) x = __bfloat162float(row[token]);
    else x = row[token];
    answer(token, logprob_of(seen(r, x), total), static_cast<int>(kept));
  }
  if (probs == nullptr) return;
  __syncthreads();
  const float inverse = 1.0f / total;
  for_tokens(row, r.v0, r.v1, [&](int i, const auto& x) {
    constexpr int kN = static_cast<int>(sizeof(x) / sizeof(float));
    float p[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const float y = seen(r, x[e]);
      p[e] = stays(y, i + e) ? weight_of(r.scale, y) * inverse : 0.0f;
    }
    if (kN % 4 == 0 && (reinterpret_cast<uintptr_t>(probs + i) & 15u) == 0) {
#pragma unroll
      for (int e = 0; e + 3 < kN; e += 4) *reinterpret_cast<float4*>(probs + i + e) = make_float4(p[e], p[e + 1], p[e + 2], p[e + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e) probs[i + e] = p[e];
    }
  });
}

template <class T>
static rf_status launch_sample(const SampleArgs& a, int64_t rows, int sms, cudaStream_t s) {
  static uint64_t done = 0;
  rf_status st = set_smem_attr(reinterpret_cast<const void*>(&k_sample<T>), kSampleArea, &done);
  if (st != RF_OK) return st;
  PowerTable p;
  for (int i = 0; i <= 64; ++i) p.t[i] = static_cast<unsigned long long>(std::llrint(std::ldexp(std::exp2(-i / 64.0), kMassBits)));
  // a power of two of CTAs a row: as many as run at once, each with enough tokens for its threads
  unsigned ctas = 1;
  while (ctas < kSampleCtas && static_cast<int64_t>(ctas) * kSampleShare < a.vocab && rows * ctas * 2 <= 2 * sms) ctas *= 2;
  ProfScope prof(s, RF_STAGE_SAMPLE);
  return cuda_check(launch_dependent(k_sample<T>, dim3(static_cast<unsigned>(rows) * ctas), dim3(kSampleThreads), kSampleArea, s,
                                     ctas, a, p),
                    "k_sample launch");
}

}  // namespace rf

using namespace rf;

extern "C" rf_status rf_sample(const rf_sample_desc* d, const void* logits, const float* temperature, const int32_t* top_k,
                               const float* top_p, const float* min_p, const float* noise, float* probs, int32_t* token,
                               float* logprob, int32_t* n_kept, int32_t* dev_status, rf_stream_t stream) {
  clear_error();
  if (d == nullptr) return fail(RF_ERR_INVALID_ARG, "desc is NULL");
  if (d->n_rows < 0 || d->vocab <= 0) return fail(RF_ERR_INVALID_ARG, "need n_rows >= 0, vocab > 0");
  if (d->dtype != RF_BF16 && d->dtype != RF_F32) return fail(RF_ERR_INVALID_ARG, "unknown dtype");
  if (d->reserved != 0) return fail(RF_ERR_INVALID_ARG, "reserved must be 0");
  if (d->vocab > kSampleMaxVocab || d->n_rows > (int64_t(1) << 24))
    return fail(RF_ERR_SHAPE, "vocab must be <= 2^20, n_rows <= 2^24");
  if (d->ld_logits < d->vocab || (noise != nullptr && d->ld_noise < d->vocab) || (probs != nullptr && d->ld_probs < d->vocab))
    return fail(RF_ERR_ALIGN, "row strides must be >= vocab");
  if (d->n_rows == 0) return RF_OK;
  if (!logits || (!token && !probs)) return fail(RF_ERR_INVALID_ARG, "logits, and token or probs, must be non-NULL");
  if ((token != nullptr) != (noise != nullptr)) return fail(RF_ERR_INVALID_ARG, "token and noise belong together");
  if (logprob && !token) return fail(RF_ERR_INVALID_ARG, "logprob is the token's");
  const uintptr_t bits = reinterpret_cast<uintptr_t>(temperature) | reinterpret_cast<uintptr_t>(top_k) |
                         reinterpret_cast<uintptr_t>(top_p) | reinterpret_cast<uintptr_t>(min_p) |
                         reinterpret_cast<uintptr_t>(noise) | reinterpret_cast<uintptr_t>(probs) |
                         reinterpret_cast<uintptr_t>(token) | reinterpret_cast<uintptr_t>(logprob) |
                         reinterpret_cast<uintptr_t>(n_kept);
  const uintptr_t size = d->dtype == RF_BF16 ? 2 : 4;
  if ((bits & 3u) || (reinterpret_cast<uintptr_t>(logits) & (size - 1)))
    return fail(RF_ERR_ALIGN, "arrays must be aligned to their elements");
  if (d->ld_logits > (int64_t(1) << 36) || (noise && d->ld_noise > (int64_t(1) << 36)) || (probs && d->ld_probs > (int64_t(1) << 36)))
    return fail(RF_ERR_SHAPE, "row strides must be <= 2^36");
  const bool in_place = static_cast<const void*>(probs) == logits && d->dtype == RF_F32 && d->ld_probs == d->ld_logits;
  const int64_t span = (d->n_rows - 1) * d->ld_logits + d->vocab, wide = (d->n_rows - 1) * d->ld_probs + d->vocab;
  if (probs != nullptr && !in_place && overlap(static_cast<const char*>(logits), span * static_cast<int64_t>(size), probs, wide))
    return fail(RF_ERR_INVALID_ARG, "probs must be the logits (fp32, the same stride) or lie apart from them");
  int sms = 0;
  rf_status st = current_device(&sms);
  if (st != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  SampleArgs a{};
  a.logits = logits;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.noise = noise;
  a.probs = probs;
  a.token = token;
  a.logprob = logprob;
  a.n_kept = n_kept;
  a.dev_status = dev_status;
  a.ld_logits = d->ld_logits;
  a.ld_noise = d->ld_noise;
  a.ld_probs = d->ld_probs;
  a.vocab = static_cast<int>(d->vocab);
  return d->dtype == RF_BF16 ? launch_sample<__nv_bfloat16>(a, d->n_rows, sms, s) : launch_sample<float>(a, d->n_rows, sms, s);
}
