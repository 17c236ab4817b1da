// What the calls that turn rows by their positions share (rope.cu, norm_rope.cu): the frequency
// table, the angles and 16-byte accesses.
#pragma once
#include "rf_device.cuh"
#include "rf_host.h"

namespace rf {

constexpr int kRopeMaxPairs = 128;

// Fixed-point turns per position, as in RopeFreqs: g[i] = 2^64 f_i / 2 pi.
struct RopeTable {
  unsigned long long g[kRopeMaxPairs];
};

// The table of a description, and the checks of it (rope.cu).
RopeTable rope_table(const rf_rope_desc* d);
rf_status check_rope(const rf_rope_desc* d);

// cos and sin of the angle q g. bf16 rows: the SFU on the reduced angle (absolute error
// about 2^-21, a thirtieth of a bf16 rounding); fp32 rows: to the last bits of fp32,
// from the fraction of a turn itself, so that no rounding of pi enters.
template <class T>
__device__ __forceinline__ void turn_cs(unsigned long long q, unsigned long long g, float& c, float& s) {
  const int turns = static_cast<int>(static_cast<unsigned>((q * g) >> 32));
  if constexpr (sizeof(T) == 2) __sincosf(static_cast<float>(turns) * 1.4629180792671596e-9f, &s, &c);  // 2 pi / 2^32
  else sincospif(static_cast<float>(turns) * 4.6566128730773926e-10f, &s, &c);                         // 2 / 2^32
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

template <class T, int N>
__device__ __forceinline__ void load_vec(const T* p, T (&v)[N]) {
  if constexpr (N * sizeof(T) == 16) {
    *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i];
  }
}
template <class T, int N>
__device__ __forceinline__ void store_vec(T* p, const T (&v)[N]) {
  if constexpr (N * sizeof(T) == 16) {
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = v[i];
  }
}

}  // namespace rf
