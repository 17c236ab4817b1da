// Sampling from logits by temperature, top-k, top-p and min-p, from given random numbers (rf_sample).
//
// In the order of falling logit, the lowest token first among equals, each filter keeps a first
// run of the tokens: the first k; of those the shortest run whose mass reaches p of theirs; of those
// the ones of at least min_p of the first one's weight. So what stays is a run too, and is given by its
// last token. Weights are w = 2^-t, t = (max - logit) log2(e) / T.
//
// Where the runs end is decided by integers of 64 bits. Logits are compared as they are. Masses are integers,
// so that sums do not depend on their order: t falls into one of 2,048 bins of 1/64 each; within a bin the
// weights differ by a factor 1 - q that a polynomial of the rest of t gives to 2^-29, with the rounding to whole
// numbers, so a bin needs the count of its tokens and the sum of their q, additions of integers to shared memory. The
// last bin's are off by 2^-53 of the greatest weight, and a bin's sum by 2^-42 of it. In fp32 sums a flat row's
// nucleus would end a token early or late every few dozen rows.
//
// One cluster of up to eight CTAs a row, each with a share of the vocabulary, which it reads once for the
// maximum and then again, from L2:
//   few tokens (top-k of at most 256)   The threads of the cluster form 2 k groups or more. What lies below the
//             k-th greatest of the groups' maxima, which k tokens reach, cannot stay. The others, some 1.4 k, are
//             listed and sorted; all filters and the draw then take the list alone. (The least maximum of k groups
//             leaves k (ln k + 0.6) tokens, and of 128 in one row of 20 more than a list holds.)
//   any other  The bins' table is built and summed over the cluster. A run's end lies in one bin, whose tokens
//             are listed and narrowed down to 32 by tables over their (logit, token) pairs (as they are before,
//             where a list does not hold them). A pass over all then adds up the weights that stay and draws,
//             another writes probabilities.
//
// Bound: the logits' bytes (and the probabilities') from memory are the floor. What takes the time of a row with a
// nucleus is some 80 instructions a token (bf16; a third of the issue slots) and the waits between its passes,
// each behind barriers of the cluster. Measured: one row of 32,000 in 9 to 11 us with a top-k of 1 to 256, 14 to 18
// without, of which some ten such barriers are most; 64 fp32 rows of 131,072 in 14 to 18 us with such a top-k, 64 bf16
// rows with nuclei in 43.8 us; 256 fp32 rows of 131,072 with every filter and their probabilities in 145 us
// (1.9 TB/s); 48 unfiltered rows of 100,003 with theirs in 32 us (1.8 TB/s).
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cstddef>
#include <cmath>

#include "rf_device.cuh"
#include "rf_host.h"

namespace rf {
namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kSampleCtas = 8;        // CTAs of a cluster (the portable limit)
constexpr int kSampleShare = 2048;    // least tokens of a CTA
constexpr int kSampleLong = 32768;    // tokens from which on a row has two CTAs at least
constexpr int kBins = 2048;           // of the table of masses: 64 an octave; the last one holds all smaller weights
constexpr int kListed = 1024;         // tokens that are listed at most
constexpr int kFewTokens = 256;       // top-k up to which tokens are listed at once
static_assert(2 * kFewTokens <= kSampleThreads && kSampleWarps * kSampleCtas <= 2 * kFewTokens, "groups of a cluster");
constexpr int kSampleMaxVocab = 1 << 20;
constexpr unsigned kSparse = 64;      // where more than one token in so many stays, the noise is read along with the
                                      // logits; below that only at the tokens that stay, each a wait of its own (64
                                      // bf16 rows of 131,072 with nuclei: 47.5 us that way for all, 43.8 with this
                                      // rule, the same with 32 for 64, 45.4 with 4)
constexpr int kMassBits = 29;         // a weight of 1, within its bin
constexpr int kCommonBits = 42;       // a weight of 1, over all bins
constexpr int kCountShift = 43;       // a bin's entry: its count above the sum of 2^22 + q 2^29, each below 2^23
static_assert(kSampleMaxVocab < 1 << (64 - kCountShift) && (static_cast<long long>(kSampleMaxVocab) << 23) <= 1ll << kCountShift,
              "all tokens may share a bin, whose count and sum share 64 bits");

struct PowerTable {
  unsigned long long t[64];  // 2^(63 - i/64)
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

// A token's place in the order: falling logit, then rising token. -0 and 0 are equal. A bf16 logit takes 16
// bits, so that tables over places tell its many equals apart by their tokens the sooner.
__device__ __forceinline__ unsigned rising_key(float x) {
  const unsigned b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(unsigned k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
template <bool kShort>
__device__ __forceinline__ unsigned long long place_of(float x, int i) {
  return (static_cast<unsigned long long>(~rising_key(x) >> (kShort ? 16 : 0)) << 20) | static_cast<unsigned>(i);
}
template <bool kShort>
__device__ __forceinline__ float place_value(unsigned long long p) {
  const unsigned k = static_cast<unsigned>(p >> 20);
  if (!kShort) return key_value(~k);
  return __uint_as_float((k & 0x8000u ? k : 0x7fffu ^ k) << 16);
}
__device__ __forceinline__ int place_token(unsigned long long p) { return static_cast<int>(p & 0xfffffu); }

struct Scale {
  float m, c, c_lo;  // the row's reference (see reference_of); log2(e) / T = c + c_lo
};

// What the weights of a bf16 row are relative to: the maximum, or 0 where that is next to it (all weights then change by
// less than 2^0.005, which cancels out).
__device__ __forceinline__ float reference_of(float top, float c) { return fabsf(top) * c < 0.005f ? 0.0f : top; }
// What the rounding of the difference d = m - x leaves of it. fp32: as for any two numbers, five operations. bf16 (kShort),
// two: d is exact unless one of the two is more than 2^15 times the other. If m is, m - d is exact and the rest is
// what it differs from x by; if x is, then m is 0 and d exact, or t beyond 160 and the weight 0 all the same.
template <bool kShort>
__device__ __forceinline__ float rounded_off(const Scale& s, float x, float d) {
  if (kShort) return (s.m - d) - x;
  const float b = d - s.m;
  return (s.m - (d - b)) - (x + b);
}
// t = (m - x) c as hi + lo, to about 2^-46 of itself.
template <bool kShort>
__device__ __forceinline__ void distance(const Scale& s, float x, float& hi, float& lo) {
  const float d = s.m - x;
  hi = d * s.c;
  lo = fmaf(d, s.c, -hi);
  lo = fmaf(d, s.c_lo, lo);
  lo = fmaf(rounded_off<kShort>(s, x, d), s.c, lo);
}
// The same of two bf16 tokens, in packed operations with the bits of the scalar ones. (256 rows of 131,072, unfiltered, with
// their probabilities: 96 us, 102 in scalar operations.)
__device__ __forceinline__ void distance_x2(const Scale& s, float2 x, float2& hi, float2& lo) {
  const float2 m = make_float2(s.m, s.m), c = make_float2(s.c, s.c), minus = make_float2(-1.0f, -1.0f);
  const float2 d = fma_x2(x, minus, m);
  hi = mul_x2(d, c);
  lo = fma_x2(d, c, make_float2(-hi.x, -hi.y));
  lo = fma_x2(d, make_float2(s.c_lo, s.c_lo), lo);
  lo = fma_x2(fma_x2(x, minus, fma_x2(d, minus, m)), c, lo);
}
// 2^-t in fp32 (0 below 2^-126).
__device__ __forceinline__ float weight_at(float hi, float lo) {
  return hi < 150.0f ? exp2f_ftz(-hi) * fmaf(lo, -0.693147181f, 1.0f) : 0.0f;
}
template <bool kShort>
__device__ __forceinline__ float weight_of(const Scale& s, float x) {
  float hi, lo;
  distance<kShort>(s, x, hi, lo);
  return weight_at(hi, lo);
}

constexpr float kRound = 12582912.0f;  // 1.5 2^23: adding it rounds to whole numbers
constexpr float kLastNear = kRound + static_cast<float>(kBins - 2);
// t in 64ths of an octave, as kRound + a whole number and the rest, within 0.54 (anything where t is beyond all bins).
template <bool kShort>
__device__ __forceinline__ void parts_of(const Scale& s, float x, float& whole, float& rest) {
  const float c = 64.0f * s.c, d = s.m - x;
  whole = fmaf(d, c, kRound);
  rest = fmaf(d, c, kRound - whole);
  rest = fmaf(d, 64.0f * s.c_lo, rest);
  rest = fmaf(rounded_off<kShort>(s, x, d), c, rest);
}
// The bin of t: the whole number nearest to 64 t, or the last.
__device__ __forceinline__ int near_bin(float whole) { return __float_as_int(whole) - 0x4b400000; }
// A bin's entry is its count above a sum (kCountShift). What a token adds to the sum: in the bins, 2^22 + 2^29 q with
// 2^-t = 2^(-bin/64) (1 - q), q = z - z^2/2 + z^3/6, z = ln 2 / 64 of the rest, within 0.0059 (the next term is 2^-34); in
// the last one 2^22 times the weight as a part of 2^(-2047/64): at most 1.006 2^22.
__device__ __forceinline__ unsigned bin_part(float rest) {
  constexpr float k1 = 5814539.98f, k2 = 31486.9687f, k3 = 113.672415f;
  return __float_as_uint(fmaf(fmaf(fmaf(rest, k3, -k2), rest, k1), rest, kRound)) - 0x4b000000u;
}
template <bool kShort>
__device__ __forceinline__ unsigned tail_part(const Scale& s, float x) {
  float hi, lo;
  distance<kShort>(s, x, hi, lo);
  return hi < 150.0f ? __float2uint_rn(exp2f_ftz(((kBins - 1) / 64.0f - hi) - lo) * 4194304.0f) : 0u;
}
struct Mass {
  int bin;
  unsigned part;
};
template <bool kShort>
__device__ __forceinline__ Mass mass_of(const Scale& s, float x) {
  float whole, rest;
  parts_of<kShort>(s, x, whole, rest);
  if (whole <= kLastNear) return {near_bin(whole), bin_part(rest)};
  return {kBins - 1, tail_part<kShort>(s, x)};
}
__device__ __forceinline__ unsigned long long entry_of(unsigned part) { return (1ull << kCountShift) + part; }
__device__ __forceinline__ unsigned entry_count(unsigned long long e) { return static_cast<unsigned>(e >> kCountShift); }
// An entry's mass, in units of 2^-29 of its bin's weight.
__device__ __forceinline__ unsigned long long entry_mass(unsigned long long e, int bin) {
  const unsigned long long sum = e & ((1ull << kCountShift) - 1);
  return bin < kBins - 1 ? (e >> kCountShift) * ((1ull << kMassBits) + (1ull << 22)) - sum : sum << (kMassBits - 22);
}
// That mass in units of 2^-42, rounded down: mass 2^13 2^(-bin/64). (mass < 2^50)
__device__ __forceinline__ unsigned long long common_mass(const unsigned long long* power, unsigned long long mass, int bin) {
  return __umul64hi(mass << (kCommonBits - kMassBits + 1), power[bin & 63]) >> (bin >> 6);
}

// A logit of a row whose maximum is +inf, as the filters see it.
__device__ __forceinline__ float infinite(float x) { return x == INFINITY ? 0.0f : -INFINITY; }

// f(first token, values, others) for the tokens v0 <= i < v1 of a row: 16 bytes at a time between the row's
// first and last 16-byte boundaries, one token at a time outside them; the next pieces are on their way while f
// works on the last ones, so that its code stands here twice and not once for each piece in flight (four pieces
// loaded at a time, and f unrolled for them, took 5% longer). A thread's tokens rise. `other`: a
// second row that is read along with the first (kOther). `top_inf` as in Row. NaN comes as it is: it fails every
// comparison.
template <bool kOther, class T, class F>
__device__ __forceinline__ void for_both(const T* row, const float* other, bool top_inf, int v0, int v1, F f) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T)), kBatch = kOther ? 1 : 2;
  const int tid = threadIdx.x;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row + v0) & 15u) / sizeof(T));
  const int head = min(v1 - v0, (kVec - off) % kVec);
  auto one = [&](int i) {
    float x[1], e[1] = {};
    if constexpr (sizeof(T) == 2) x[0] = __bfloat162float(row[i]);
    else x[0] = row[i];
    if constexpr (kOther) e[0] = other[i];
    if (top_inf) x[0] = infinite(x[0]);
    f(i, x, e);
  };
  if (tid < head) one(v0 + tid);
  const int first = v0 + head, pieces = (v1 - first) / kVec;
  const bool even = (reinterpret_cast<uintptr_t>(other + first) & 15u) == 0;
  uint4 raw[kBatch] = {}, next[kBatch] = {};
  alignas(16) float e[kBatch][kOther ? kVec : 1], after[kBatch][kOther ? kVec : 1];
  auto load = [&](int p0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int p = p0 + j * kSampleThreads;
      if (p >= pieces) break;
      next[j] = reinterpret_cast<const uint4*>(row + first)[p];
      if constexpr (kOther) {
        const float* o = other + first + p * kVec;
        if (even) {
#pragma unroll
          for (int k = 0; k < kVec; k += 4) *reinterpret_cast<float4*>(after[j] + k) = *reinterpret_cast<const float4*>(o + k);
        } else {
#pragma unroll
          for (int k = 0; k < kVec; ++k) after[j][k] = o[k];
        }
      }
    }
  };
  load(tid);
#pragma unroll 1
  for (int p0 = tid; p0 < pieces; p0 += kBatch * kSampleThreads) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      raw[j] = next[j];
#pragma unroll
      for (int k = 0; k < (kOther ? kVec : 1); ++k) e[j][k] = after[j][k];
    }
    load(p0 + kBatch * kSampleThreads);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (p0 + j * kSampleThreads >= pieces) break;
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
      float x[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        if constexpr (sizeof(T) == 2) x[k] = u2f(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
        else x[k] = u2f(w[k]);
      }
      if (top_inf) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) x[k] = infinite(x[k]);
      }
      f(first + (p0 + j * kSampleThreads) * kVec, x, e[j]);
    }
  }
  const int last = first + pieces * kVec + tid;
  if (last < v1) one(last);
}
template <class T, class F>
__device__ __forceinline__ void for_tokens(const T* row, bool top_inf, int v0, int v1, F f) {
  for_both<false>(row, nullptr, top_inf, v0, v1, [&](int i, const auto& x, const auto&) { f(i, x); });
}

struct SampleShared {
  unsigned long long power[64];
  unsigned long long warp_sum[kSampleWarps];
  unsigned warp_count[kSampleWarps];
  float warp_total[kSampleWarps];
  // from every CTA of the cluster, by the parity of the turn
  unsigned long long best[2][kSampleCtas];
  unsigned group[2 * kFewTokens];  // (or one a warp of the cluster, which are fewer)
  float sum[2][kSampleCtas];
  unsigned kept[2][kSampleCtas];
  unsigned listed[2][kSampleCtas];
  // where a run ends
  unsigned long long found_place, found_mass;
  unsigned found_bin, found_count, found_in;
  unsigned least;
  int n_list;
  double min_away;  // T ln(min_p)
  float lowest;     // the least logit that min_p lets pass
};
struct SampleTables {
  unsigned count[kBins], low[kBins], high[kBins];  // this CTA's counts and sums, by additions of 32 bits
  unsigned long long all[kBins];    // the cluster's, of the weights' bins
  unsigned long long finer[kBins];  // the cluster's, of finer tables
  unsigned long long own_place[kListed], place[kListed];
};

// What all threads of a row's cluster know.
struct Row {
  int rank, ctas, v0, v1;
  Scale scale;
  float top;     // the maximum
  bool top_inf;  // the maximum is +inf: those tokens share all weight, as if theirs were 0 and all others' -inf
  int turn;
};

__device__ __forceinline__ unsigned long long warp_max(unsigned long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// A key that at least k of the groups' maxima reach, about the greatest such (one warp): halving the range between the
// least and the greatest one until just k do, or 20 times.
__device__ __forceinline__ void least_of_groups(SampleShared& sh, int groups, int k) {
  constexpr int kEach = 2 * kFewTokens / 32;
  const int lane = threadIdx.x & 31;
  unsigned key[kEach], lo = 0xffffffffu, hi = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    key[i] = i * 32 + lane < groups ? sh.group[i * 32 + lane] : 0u;
    if (i * 32 + lane < groups) {
      lo = min(lo, key[i]);
      hi = max(hi, key[i]);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi) + 1;
  for (int turn = 0; turn < 20 && hi - lo > 1; ++turn) {
    const unsigned mid = lo + (hi - lo) / 2;
    int reach = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) reach += key[i] >= mid;
    reach = __reduce_add_sync(0xffffffffu, reach);
    if (reach >= k) lo = mid;
    else hi = mid;
    if (reach == k) break;
  }
  if (lane == 0) sh.least = lo;
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
#pragma unroll
  for (int w = 0; w < kSampleWarps - 1; ++w)
    if (w < warp) {
      c0 += sh.warp_count[w];
      m0 += sh.warp_sum[w];
    }
  count = c0 + c - count;
  mass = m0 + m - mass;
}

// Sorts the list by place (whole CTA), padded to a power of two with places beyond all: a bitonic network with
// an element a thread (two for the longest lists), which exchanges within warps by shuffles and between them
// through the two lists in turns, one barrier an exchange. (With all exchanges in shared memory 300 tokens took 6 us.)
__device__ __forceinline__ void sort_list(SampleTables& t, int n) {
  static_assert(kListed == 2 * kSampleThreads, "two elements a thread");
  const int tid = threadIdx.x;
  int size = 32;
  while (size < n) size *= 2;
  unsigned long long v[2] = {tid < n ? t.place[tid] : ~0ull, tid + kSampleThreads < n ? t.place[tid + kSampleThreads] : ~0ull};
  const bool two = size > kSampleThreads;
  unsigned long long* from = t.own_place;
  unsigned long long* other = t.place;
  auto keep = [](unsigned long long a, unsigned long long b, bool least) { return (a < b) == least ? a : b; };
  __syncthreads();
  for (int k = 2; k <= size; k *= 2) {
    for (int j = k / 2; j > 0; j /= 2) {
      const bool least = ((tid & j) == 0) == ((tid & k) == 0);
      if (j >= 32) {
        if (j == kSampleThreads) {
          const unsigned long long a = v[0], b = v[1];
          v[0] = min(a, b);
          v[1] = max(a, b);
          continue;
        }
        if (tid < size) from[tid] = v[0];
        if (two) from[tid + kSampleThreads] = v[1];
        __syncthreads();
        if (tid < size) v[0] = keep(v[0], from[tid ^ j], least);
        if (two) v[1] = keep(v[1], from[(tid ^ j) + kSampleThreads], ((tid & j) == 0) == (((tid + kSampleThreads) & k) == 0));
        unsigned long long* x = from;
        from = other;
        other = x;
      } else {
        v[0] = keep(v[0], __shfl_xor_sync(0xffffffffu, v[0], j), least);
        if (two) v[1] = keep(v[1], __shfl_xor_sync(0xffffffffu, v[1], j), ((tid & j) == 0) == (((tid + kSampleThreads) & k) == 0));
      }
    }
  }
  __syncthreads();
  if (tid < size) t.place[tid] = v[0];
  if (two) t.place[tid + kSampleThreads] = v[1];
  __syncthreads();
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
  }
  cl.sync();
  return true;
}

// Adds a token's part to a bin of this CTA's. (An addition of 64 bits to shared memory is a loop that tries until no
// other lane is in its way; a carry out of the sum's low word comes once in some 500 additions.)
__device__ __forceinline__ void add_to(SampleTables& t, int bin, unsigned count, unsigned part) {
  atomicAdd(&t.count[bin], count);
  if (atomicAdd(&t.low[bin], part) > ~part) atomicAdd(&t.high[bin], 1u);
}

__device__ __forceinline__ unsigned long long own_entry(const SampleTables& t, int bin) {
  return (static_cast<unsigned long long>(t.count[bin]) << kCountShift) + (static_cast<unsigned long long>(t.high[bin]) << 32) + t.low[bin];
}

// The CTAs' tables, summed over the cluster (a power of two of CTAs): each CTA sends the others their parts of its
// bins, sums the part that it gets and sends that to all. Stores to other CTAs' shared memory do not wait, as loads
// do. The parts arrive where the lists are otherwise: `again` if another CTA may still be reading one.
__device__ __forceinline__ void join_tables(cg::cluster_group& cl, SampleTables& t, unsigned long long* all, const Row& r, bool again) {
  static_assert(2 * kListed == kBins && offsetof(SampleTables, place) == offsetof(SampleTables, own_place) + kListed * 8,
                "the lists hold a table");
  __syncthreads();
  if (again) cl.sync();
  const int per = kBins / r.ctas;
#pragma unroll
  for (int i = 0; i < kBins / kSampleThreads; ++i) {
    const int bin = static_cast<int>(threadIdx.x) + i * kSampleThreads, to = bin / per;
    cl.map_shared_rank(t.own_place, to)[r.rank * per + bin - to * per] = own_entry(t, bin);
  }
  cl.sync();
  for (int i = threadIdx.x; i < per; i += kSampleThreads) {
    unsigned long long e = 0;
    for (int k = 0; k < r.ctas; ++k) e += t.own_place[k * per + i];
    for (int k = 0; k < r.ctas; ++k) cl.map_shared_rank(all, k)[r.rank * per + i] = e;
  }
  cl.sync();
}
__device__ __forceinline__ void clear_table(SampleTables& t) {
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kSampleThreads) t.count[i] = t.low[i] = t.high[i] = 0;
  __syncthreads();
}

// Where a run ends: its last token's place, the mass up to there, the token's own included, and the count of tokens
// up to the end of that token's bin.
struct End {
  unsigned long long place, mass;
  unsigned about;
};

constexpr int kEach = kBins / kSampleThreads;  // bins of a thread
// The mass of a table's bin: a bin of weights (weights_bin < 0) in common units, or one of a finer table over those of
// one bin in that bin's units.
__device__ __forceinline__ unsigned long long mass_in(const SampleShared& sh, unsigned long long e, int bin, int weights_bin) {
  return weights_bin < 0 ? common_mass(sh.power, entry_mass(e, bin), bin) : entry_mass(e, weights_bin);
}
// Counts and masses of the bins before this thread's (whole CTA).
__device__ __forceinline__ void before_bins(SampleShared& sh, const unsigned long long* table, int weights_bin, unsigned& count,
                                            unsigned long long& mass) {
  count = 0;
  mass = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int bin = threadIdx.x * kEach + i;
    count += entry_count(table[bin]);
    mass += mass_in(sh, table[bin], bin, weights_bin);
  }
  before_sums(sh, count, mass);
}

// The end of the run of `target` tokens (kByMass false), or of the shortest run of mass `target`, from the
// bins' table and what lies before each thread's part of it. Every CTA of the cluster comes to the same result.
template <bool kByMass, class T>
__device__ End find_end(cg::cluster_group& cl, SampleShared& sh, SampleTables& t, Row& r, const T* row, float temperature,
                        unsigned long long target, unsigned count, unsigned long long mass) {
  constexpr bool kShort = sizeof(T) == 2;
  // The bin of the run's end, from the counts and masses before each thread's bins.
  auto find_bin = [&](const unsigned long long* table, int weights_bin, unsigned long long mass_before, unsigned c, unsigned long long m) {
    __syncthreads();
    if (threadIdx.x == 0) {  // (logits that change under the kernel: all CTAs still agree)
      sh.found_bin = 0;
      sh.found_count = sh.found_in = 0;
      sh.found_mass = 0;
    }
    __syncthreads();
    // the mass before, as the target counts it
    auto common = [&](unsigned long long x) { return weights_bin < 0 ? x : common_mass(sh.power, mass_before + x, weights_bin); };
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = threadIdx.x * kEach + i;
      const unsigned c1 = c + entry_count(table[at]);
      const unsigned long long m1 = m + mass_in(sh, table[at], at, weights_bin);
      if (kByMass ? (common(m) < target && target <= common(m1)) : (c < target && target <= c1)) {
        sh.found_bin = at;
        sh.found_count = c;
        sh.found_mass = m;
        sh.found_in = c1 - c;
      }
      c = c1;
      m = m1;
    }
    __syncthreads();
  };
  find_bin(t.all, -1, 0, count, mass);
  const int bin = static_cast<int>(sh.found_bin);
  unsigned in = sh.found_in;
  const unsigned about = sh.found_count + in;
  const unsigned long long base = sh.found_mass;  // of the bins before, in common units
  target -= kByMass ? base : sh.found_count;      // from here on within the bin
  unsigned long long inside = 0;                  // mass of the bin before the range below
  // The bin's logits, a little wider than it is, so that most others fall out by a comparison.
  const float step = temperature * (0.693147181f / 64.0f), begin = static_cast<float>(bin) - 0.5f;
  const float slack = 4e-6f * (fabsf(r.scale.m) + step * static_cast<float>(bin + 1));
  const float high = fminf(r.scale.m - step * begin + slack, r.top);
  const float low = bin == kBins - 1 ? -FLT_MAX : fmaxf(r.scale.m - step * (static_cast<float>(bin) + 0.5f) - slack, -FLT_MAX);
  unsigned long long lo = place_of<kShort>(high, 0), hi = place_of<kShort>(low, kSampleMaxVocab - 1);
  auto place_in = [&](float x, int i, unsigned long long& p, unsigned& part) {
    if (!(x >= low && x <= high)) return false;
    const Mass m = mass_of<kShort>(r.scale, x);
    part = m.part;
    p = place_of<kShort>(x, i);
    return m.bin == bin && p >= lo && p <= hi;
  };
  while (in > kListed) {
    const int width = 64 - __clzll(static_cast<long long>(hi - lo));
    const int shift = max(0, width - 11);
    clear_table(t);
    for_tokens(row, r.top_inf, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e) {
        unsigned long long p;
        unsigned part;
        if (place_in(x[e], i + e, p, part)) add_to(t, static_cast<int>((p - lo) >> shift), 1, part);
      }
    });
    join_tables(cl, t, t.finer, r, true);
    before_bins(sh, t.finer, bin, count, mass);
    find_bin(t.finer, bin, inside, count, mass);
    lo += static_cast<unsigned long long>(sh.found_bin) << shift;
    hi = min(hi, lo + ((1ull << shift) - 1));
    in = sh.found_in;
    inside += sh.found_mass;
    if (!kByMass) target -= sh.found_count;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  for_tokens(row, r.top_inf, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
    for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e) {
      unsigned long long p;
      unsigned part;
      if (place_in(x[e], i + e, p, part)) {
        const int at = atomicAdd(&sh.n_list, 1);
        if (at < kListed) t.own_place[at] = p;
      }
    }
  });
  int n = 0;
  join_lists(cl, sh, t, r, &n);
  n = min(n, kListed);
  // Tables over the list's places narrow it down to a warp's tokens. (Sorting it took 8 us of 1,000 tokens, a table takes
  // 1.5. Places differ, so that the loop ends.)
  unsigned long long *list = t.place, *rest = t.own_place;
  while (n > 32 && lo < hi) {
    const int shift = max(0, 64 - __clzll(static_cast<long long>(hi - lo)) - 11);
    clear_table(t);
    for (int i = threadIdx.x; i < n; i += kSampleThreads) {
      if (list[i] < lo || list[i] > hi) continue;  // (logits that change under the kernel)
      add_to(t, static_cast<int>((list[i] - lo) >> shift), 1, mass_of<kShort>(r.scale, place_value<kShort>(list[i])).part);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) t.finer[threadIdx.x + i * kSampleThreads] = own_entry(t, threadIdx.x + i * kSampleThreads);
    if (threadIdx.x == 0) sh.n_list = 0;
    __syncthreads();
    before_bins(sh, t.finer, bin, count, mass);
    find_bin(t.finer, bin, inside, count, mass);
    lo += static_cast<unsigned long long>(sh.found_bin) << shift;
    hi = min(hi, lo + ((1ull << shift) - 1));
    inside += sh.found_mass;
    if (!kByMass) target -= sh.found_count;
    for (int i = threadIdx.x; i < n; i += kSampleThreads)
      if (list[i] >= lo && list[i] <= hi) rest[atomicAdd(&sh.n_list, 1)] = list[i];
    __syncthreads();
    n = sh.n_list;
    unsigned long long* x = list;
    list = rest;
    rest = x;
  }
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    n = min(n, 32);
    if (lane == 0) {  // (as above)
      sh.found_place = hi;
      sh.found_mass = 0;
    }
    __syncwarp();
    const unsigned long long place = lane < n ? list[lane] : ~0ull;
    const Mass mass_here = mass_of<kShort>(r.scale, place_value<kShort>(place));
    const unsigned long long own = lane < n ? entry_mass(entry_of(mass_here.part), bin) : 0ull;
    unsigned long long m = 0, rank = 0;
    for (int i = 0; i < n; ++i) {
      const unsigned long long other = __shfl_sync(0xffffffffu, place, i), its = __shfl_sync(0xffffffffu, own, i);
      if (other < place) {
        m += its;
        ++rank;
      }
    }
    if (lane < n && (kByMass ? (common_mass(sh.power, inside + m, bin) < target && target <= common_mass(sh.power, inside + m + own, bin))
                             : rank + 1 == target)) {
      sh.found_place = place;
      sh.found_mass = m + own;
    }
  }
  __syncthreads();
  const End end{sh.found_place, base + common_mass(sh.power, inside + sh.found_mass, bin), about};
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
  constexpr bool kShort = sizeof(T) == 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = ((a.vocab + r.ctas - 1) / r.ctas + 7) & ~7;
  r.v0 = min(r.rank * share, a.vocab);
  r.v1 = min(r.v0 + share, a.vocab);
  pdl_launch_dependents();
  if (tid < 64) sh.power[tid] = powers.t[tid];
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

  // The threads' maxima; at temperature 0, where nothing else is done, with their lowest tokens.
  float top = -INFINITY;
  int top_i = 0;
  if (temperature == 0.0f && good)
    for_tokens(row, false, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e)
        if (x[e] > top) {
          top = x[e];
          top_i = i + e;
        }
    });
  else if (good)
    for_tokens(row, false, r.v0, r.v1, [&](int, const auto& x) {
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e) top = fmaxf(top, x[e]);
    });
  if (min_p > 0.0f && tid == kSampleThreads - 1) sh.min_away = static_cast<double>(temperature) * log(static_cast<double>(min_p));
  const unsigned long long mine =
      top > -INFINITY ? (static_cast<unsigned long long>(rising_key(top)) << 32) | (0xffffffffu - static_cast<unsigned>(top_i)) : 0ull;
  unsigned long long best = warp_max(mine);
  // few tokens: groups of up to 32 threads of this CTA, at least twice top_k of them in the cluster
  int groups = 0;
  unsigned group_max = rising_key(top);
  if (top_k > 0 && top_k <= kFewTokens) {
    groups = kSampleWarps;
    while (groups * r.ctas < 2 * top_k) groups *= 2;
    for (int o = 1; o < kSampleThreads / groups; o <<= 1) group_max = max(group_max, __shfl_xor_sync(0xffffffffu, group_max, o));
  }
  if (lane == 0) sh.warp_sum[warp] = best;
  __syncthreads();
  cl.barrier_wait();
  if (groups > 0 && tid % (kSampleThreads / groups) == 0)
    for (int c = 0; c < r.ctas; ++c) cl.map_shared_rank(sh.group, c)[r.rank * groups + tid / (kSampleThreads / groups)] = group_max;
  if (warp == 0) {
    best = warp_max(lane < kSampleWarps ? sh.warp_sum[lane] : 0ull);
    if (lane < r.ctas) *cl.map_shared_rank(&sh.best[0][r.rank], lane) = best;
  }
  cl.sync();
  best = 0;
  for (int c = 0; c < r.ctas; ++c) best = max(best, sh.best[0][c]);
  if (groups > 0) {  // (whole cluster, each CTA the same)
    if (warp == 0) least_of_groups(sh, groups * r.ctas, top_k);
    __syncthreads();
  }
  r.turn = 1;

  auto token_of = [](unsigned long long pair) { return static_cast<int>(0xffffffffu - static_cast<unsigned>(pair & 0xffffffffu)); };
  auto zero_probs = [&] {
    if (probs == nullptr) return;
    const int head = min(r.v1 - r.v0, static_cast<int>(4 - ((reinterpret_cast<uintptr_t>(probs + r.v0) >> 2) & 3)) & 3);
    const int v = r.v0 + head, pieces = (r.v1 - v) / 4;
    if (tid < head) probs[r.v0 + tid] = 0.0f;
    for (int i = tid; i < pieces; i += kSampleThreads) reinterpret_cast<float4*>(probs + v)[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (v + pieces * 4 + tid < r.v1) probs[v + pieces * 4 + tid] = 0.0f;
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
  r.top = key_value(static_cast<unsigned>(best >> 32));
  if (temperature == 0.0f) {
    const int first = token_of(best);
    zero_probs();
    __syncthreads();
    if (probs != nullptr && tid == 0 && first >= r.v0 && first < r.v1) probs[first] = 1.0f;
    if (r.rank == 0 && tid == 0) answer(first, 0.0f, 1);
    return;
  }
  r.top_inf = r.top == INFINITY;
  if (r.top_inf) r.top = 0.0f;
  {
    constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596303e-8f;
    r.scale.c = kLog2e / temperature;
    r.scale.c_lo = (fmaf(-r.scale.c, temperature, kLog2e) + kLog2eLo) / temperature;
    r.scale.m = kShort ? reference_of(r.top, r.scale.c) : r.top;
  }
  if (tid == 0) {
    float f = -INFINITY;
    if (min_p > 0.0f) f = __double2float_ru(static_cast<double>(r.top) + sh.min_away);
    sh.lowest = f;
  }
  __syncthreads();
  const float lowest = sh.lowest;

  const float* noise = a.noise != nullptr ? a.noise + row_of * a.ld_noise : nullptr;
  auto pair_of = [](float score, int i) {
    return (static_cast<unsigned long long>(__float_as_uint(score)) << 32) | (0xffffffffu - static_cast<unsigned>(i));
  };
  auto score_of = [](float w, float e) { return w > 0.0f ? __fdividef(w, e) : 0.0f; };
  auto logprob_of = [&](float x, float total) {
    float hi, lo;
    distance<kShort>(r.scale, x, hi, lo);
    return -(hi + lo) * 0.693147181f - logf(total);
  };

  // No token that stays has a score: its noise is no number above 0.
  auto no_score = [&](int kept) {
    if (r.rank != 0 || tid != 0) return;
    answer(-1, -INFINITY, kept);
    record_status(a.dev_status, RF_ERR_INVALID_ARG);
  };

  // Few tokens: list what reaches the least of the top_k greatest group maxima.
  int n = 0;
  if (groups > 0 && !r.top_inf && sh.least > rising_key(-INFINITY)) {
    const float from = key_value(sh.least);
    for_tokens(row, r.top_inf, r.v0, r.v1, [&](int i, const auto& x) {
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e)
        if (x[e] >= from) {
          const int at = atomicAdd(&sh.n_list, 1);
          if (at < kListed) t.own_place[at] = place_of<kShort>(x[e], i + e);
        }
    });
    if (join_lists(cl, sh, t, r, &n)) {
      sort_list(t, n);
      int kept = min(top_k, n);
      if (top_p < 1.0f) {
        // (of the first top_k, up to half of the threads)
        unsigned c = 0;
        unsigned long long each = 0;
        if (tid < kept) {
          const Mass m = mass_of<kShort>(r.scale, place_value<kShort>(t.place[tid]));
          each = common_mass(sh.power, entry_mass(entry_of(m.part), m.bin), m.bin);
        }
        unsigned long long m = each;
        before_sums(sh, c, m);
        if (tid == kept - 1) sh.found_mass = m + each;
        __syncthreads();
        const unsigned long long target = mass_target(top_p, sh.found_mass);
        if (tid < kept && m < target && target <= m + each) sh.found_count = tid + 1;
        __syncthreads();
        kept = min(kept, static_cast<int>(sh.found_count));
      }
      kept = __syncthreads_count(tid < kept && place_value<kShort>(t.place[tid]) >= lowest);
      float w = 0.0f, score = 0.0f;
      int i = 0;
      if (tid < kept) {
        i = place_token(t.place[tid]);
        w = weight_of<kShort>(r.scale, place_value<kShort>(t.place[tid]));
        if (a.token != nullptr && r.rank == 0) score = score_of(w, noise[i]);
      }
      float total = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      const unsigned long long pick = warp_max(tid < kept && score >= 0.0f ? pair_of(score, i) : 0ull);
      if (lane == 0) {
        sh.warp_total[warp] = total;
        sh.warp_sum[warp] = pick;
      }
      zero_probs();
      __syncthreads();
      total = 0.0f;
      best = 0;
      for (int x = 0; x < kFewTokens / 32; ++x) {
        total += sh.warp_total[x];
        best = max(best, sh.warp_sum[x]);
      }
      if (probs != nullptr && tid < kept && i >= r.v0 && i < r.v1) probs[i] = w / total;
      // the token's own thread, or the first one's where none is drawn
      if (a.token != nullptr && best == 0) no_score(kept);
      else if (r.rank == 0 && tid < kept && i == (a.token != nullptr ? token_of(best) : place_token(t.place[0])))
        answer(i, logprob_of(place_value<kShort>(t.place[tid]), total), kept);
      return;
    }
  }

  // Any number of tokens. The last one that stays, by logit and token:
  float last = -INFINITY;
  int last_i = -1;
  unsigned about = static_cast<unsigned>(a.vocab);  // of them
  if ((top_k > 0 && top_k < a.vocab) || top_p < 1.0f) {
    clear_table(t);
    unsigned long long tail = 0;
    for_tokens(row, r.top_inf, r.v0, r.v1, [&](int, const auto& x) {
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(x) / sizeof(float)); ++e) {
        float whole, rest;
        parts_of<kShort>(r.scale, x[e], whole, rest);
        if (whole <= kLastNear) add_to(t, near_bin(whole), 1, bin_part(rest));
        else if (x[e] > -INFINITY) tail += (1ull << kCountShift) + tail_part<kShort>(r.scale, x[e]);  // (many share the last bin)
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tail += __shfl_xor_sync(0xffffffffu, tail, o);
    if (lane == 0 && tail != 0) {
      add_to(t, kBins - 1, entry_count(tail), static_cast<unsigned>(tail));
      atomicAdd(&t.high[kBins - 1], static_cast<unsigned>(tail >> 32) & ((1u << (kCountShift - 32)) - 1u));
    }
    join_tables(cl, t, t.all, r, false);
    unsigned before;
    unsigned long long mass_before;
    before_bins(sh, t.all, -1, before, mass_before);
    unsigned valid = 0;
    unsigned long long all = 0;
#pragma unroll
    for (int w = 0; w < kSampleWarps; ++w) {
      valid += sh.warp_count[w];
      all += sh.warp_sum[w];
    }
    End end{~0ull, all, valid};
    if (top_k > 0 && static_cast<unsigned>(top_k) < valid)
      end = find_end<false>(cl, sh, t, r, row, temperature, top_k, before, mass_before);
    if (top_p < 1.0f) {
      const End by_mass = find_end<true>(cl, sh, t, r, row, temperature, mass_target(top_p, end.mass), before, mass_before);
      end.place = min(end.place, by_mass.place);
      end.about = min(end.about, by_mass.about);
    }
    if (end.place != ~0ull) {
      last = place_value<kShort>(end.place);
      last_i = place_token(end.place);
      about = end.about;
    }
  }
  if (lowest > last) {
    last = lowest;
    last_i = kSampleMaxVocab;
    about = 0;  // (unknown)
  }
  auto stays = [&](float x, int i) { return x > last || (x == last && i <= last_i); };
  float total = 0.0f, leader = -1.0f;  // the greatest score and its token: the lowest, as a thread's tokens rise
  unsigned kept = 0;
  int lead_i = 0;
  auto count = [&](int i, float w, float e) {
    total += w;
    ++kept;
    const float score = score_of(w, e);
    if (score > leader) {
      leader = score;
      lead_i = i;
    }
  };
  auto count_in = [&](int i, const auto& x, const auto& e) {
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(x) / sizeof(float)); ++j)
      if (stays(x[j], i + j)) count(i + j, weight_of<kShort>(r.scale, x[j]), e[j]);
  };
  auto count_dense = [&](int i, const auto& x, const auto& e) {
    constexpr int kN = static_cast<int>(sizeof(x) / sizeof(float));
    if constexpr (kShort && kN > 1) {
#pragma unroll
      for (int j = 0; j < kN; j += 2) {
        float2 hi, lo;
        distance_x2(r.scale, make_float2(x[j], x[j + 1]), hi, lo);
        if (stays(x[j], i + j)) count(i + j, weight_at(hi.x, lo.x), e[j]);
        if (stays(x[j + 1], i + j + 1)) count(i + j + 1, weight_at(hi.y, lo.y), e[j + 1]);
      }
    } else {
      count_in(i, x, e);
    }
  };
  if (noise != nullptr && about > static_cast<unsigned>(a.vocab) / kSparse) {  // the noise comes along with the logits
    for_both<true>(row, noise, r.top_inf, r.v0, r.v1, count_dense);
  } else {
    for_tokens(row, r.top_inf, r.v0, r.v1, [&](int i, const auto& x) {
      constexpr int kN = static_cast<int>(sizeof(x) / sizeof(float));
      float e[kN], top = -INFINITY;
#pragma unroll
      for (int j = 0; j < kN; ++j) top = fmaxf(top, x[j]);
      if (!(top >= last)) return;
#pragma unroll
      for (int j = 0; j < kN; ++j) e[j] = noise != nullptr && stays(x[j], i + j) ? noise[i + j] : 1.0f;
      count_in(i, x, e);
    });
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  kept = __reduce_add_sync(0xffffffffu, kept);
  best = warp_max(leader >= 0.0f ? pair_of(leader, lead_i) : 0ull);
  __syncthreads();
  if (lane == 0) {
    sh.warp_total[warp] = total;
    sh.warp_count[warp] = kept;
    sh.warp_sum[warp] = best;
  }
  __syncthreads();
  if (warp == 0) {
    total = lane < kSampleWarps ? sh.warp_total[lane] : 0.0f;
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
  const int token = token_of(best);
  if (a.token != nullptr && best == 0) {
    no_score(static_cast<int>(kept));
  } else if (tid == 0 && (a.token != nullptr ? token >= r.v0 && token < r.v1 : r.rank == 0)) {
    float x = r.top;
    if (a.token != nullptr && !r.top_inf) {
      if constexpr (kShort) x = __bfloat162float(row[token]);
      else x = row[token];
    }
    answer(token, logprob_of(x, total), static_cast<int>(kept));
  }
  if (probs == nullptr) return;
  __syncthreads();
  const float inverse = 1.0f / total;
  for_tokens(row, r.top_inf, r.v0, r.v1, [&](int i, const auto& x) {
    constexpr int kN = static_cast<int>(sizeof(x) / sizeof(float));
    float p[kN];
    if constexpr (kShort && kN > 1) {
#pragma unroll
      for (int e = 0; e < kN; e += 2) {
        float2 hi, lo;
        distance_x2(r.scale, make_float2(x[e], x[e + 1]), hi, lo);
        p[e] = stays(x[e], i + e) ? weight_at(hi.x, lo.x) * inverse : 0.0f;
        p[e + 1] = stays(x[e + 1], i + e + 1) ? weight_at(hi.y, lo.y) * inverse : 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e) p[e] = stays(x[e], i + e) ? weight_of<kShort>(r.scale, x[e]) * inverse : 0.0f;
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
  rf_status st = set_smem_attr(reinterpret_cast<const void*>(&k_sample<T>), sizeof(SampleTables), &done);
  if (st != RF_OK) return st;
  PowerTable p;
  for (int i = 0; i < 64; ++i) p.t[i] = static_cast<unsigned long long>(std::ldexp(std::exp2(-i / 64.0), 63));
  // CTAs a row: a power of two, as many as run at once, each with enough tokens for its threads; long rows at least
  // two, so that rows that take longer than others are shared out and fewer are in L2 at a time (256 rows of
  // 131,072, half of them without a small top-k: 177 us with one, 145 with two, 149 with four, 190 with eight).
  unsigned ctas = a.vocab >= kSampleLong ? 2 : 1;
  while (ctas < kSampleCtas && static_cast<int64_t>(ctas) * kSampleShare < a.vocab && rows * ctas * 2 <= 2 * sms) ctas *= 2;
  ProfScope prof(s, RF_STAGE_SAMPLE);
  return cuda_check(launch_dependent(k_sample<T>, dim3(static_cast<unsigned>(rows) * ctas), dim3(kSampleThreads), sizeof(SampleTables), s,
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
  const auto span = [&](int64_t ld) { return (d->n_rows - 1) * ld + d->vocab; };
  if (probs != nullptr && !in_place &&
      overlap(static_cast<const char*>(logits), span(d->ld_logits) * static_cast<int64_t>(size), probs, span(d->ld_probs)))
    return fail(RF_ERR_INVALID_ARG, "probs must be the logits (fp32, the same stride) or lie apart from them");
  // A row's CTAs write probabilities while others still read noise. Rows of one stride may lie beside each other.
  if (probs != nullptr && noise != nullptr && overlap(noise, span(d->ld_noise), probs, span(d->ld_probs))) {
    const int64_t ld = d->ld_noise;
    const int64_t from = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(probs) - reinterpret_cast<uintptr_t>(noise)) / 4 % ld + ld) % ld;
    if (ld != d->ld_probs || from < d->vocab || ld - from < d->vocab)
      return fail(RF_ERR_INVALID_ARG, "probs must lie apart from the noise");
  }
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
