// Verification of drafted tokens (rf_verify_draft) and the accepted rows' way into the
// cache (rf_commit_draft).
//
// The walk: from the root, children x of the current node are tried in index order. With
// k refusals so far the target's row p has become r_k, r_0 = p, Z_0 = 1,
//   r_{j+1} = max(r_j / Z_j - q, 0),  Z_{j+1} = sum r_{j+1}     (or, for children chosen
//   outright, r_{j+1} = r_j without its token),
// and x is accepted when u q(x) Z_k < r_k(x). A test needs r_k at one token only, which
// the chain above gives from p and q at that token, so the walk itself reads three
// numbers a node, fetched for every node at once beforehand. A whole row is read where a
// sum Z is needed (a refused child with a sibling behind it) and once at the end, for
// the lowest argmax of r / noise. What bounds a call is the latency of these steps: with the
// commit of 32 layers, a chain of 5 over 32,000 tokens takes 12 us, 16 trees of 64 nodes over
// 131,072 tokens 28 to 38 us, by the walks, for 29 MB that must be read.
//
// One cluster of CTAs a sequence: every thread follows the same walk through shared
// memory, each CTA sums or scans its share of the vocabulary and writes the result into the
// shared memory of all, and all join the shares in a fixed order. A thread keeps its tokens' r
// and q of the current node in registers (up to 16: 131,072 tokens in a cluster), so a refusal
// costs one quotient a token; larger vocabularies form r_k anew from p and q each time (such
// trees over 131,072 tokens 28 us, over 131,076 tokens 71 us, over 262,144 tokens 78 us).
#include <cooperative_groups.h>

#include <algorithm>

#include "rf_device.cuh"
#include "rf_host.h"

namespace rf {
namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 1024;
constexpr int kVerifyCtas = 8;      // CTAs of a cluster (the portable limit)
constexpr int kVerifyBatch = 8;     // values of each row that a thread has in flight (long rows)
constexpr int kVerifySlots = 16;    // tokens of a thread that stay in registers
constexpr int kVerifyShare = 2048;  // least tokens of a CTA

struct VerifyArgs {
  const float* target;
  const float* draft;
  const int32_t* tokens;
  const int32_t* parents;
  const float* u;
  const float* noise;
  int32_t* path;
  int32_t* n_path;
  int32_t* next_token;
  int32_t* dev_status;
  long long ld_target, ld_draft, ld_noise;
  int n, vocab;
};

// Tokens of a CTA: whole 16-byte groups.
__host__ __device__ inline int verify_share(int vocab, int ctas) { return ((vocab + ctas - 1) / ctas + 3) & ~3; }

// What one form has, so that the other cannot read it. With draft probabilities, for each refusal
// at the current node: 1 / Z_j and the least order (quotient_order) of what is divided by it quickly.
template <bool kDraft>
struct VerifyRefused {
  float inverse[RF_TREE_MAX_NODES];
  unsigned least[RF_TREE_MAX_NODES];
};
// Without: its node.
template <>
struct VerifyRefused<false> {
  int refused[RF_TREE_MAX_NODES];
};
template <bool kDraft>
struct VerifyShared : VerifyRefused<kDraft> {
  int up[RF_TREE_MAX_NODES];
  int token[RF_TREE_MAX_NODES];
  float u[RF_TREE_MAX_NODES];
  float p[RF_TREE_MAX_NODES];  // target probability of the node's token at its parent
  float q[RF_TREE_MAX_NODES];
  float z[RF_TREE_MAX_NODES];  // Z_j of the refusals at the current node
  int path[RF_TREE_MAX_NODES];
  float part_sum[2][kVerifyCtas];  // the CTAs' shares, by the parity of the turn
  unsigned long long part_best[2][kVerifyCtas];
  float warp_sum[kVerifyThreads / 32];
  unsigned long long warp_best[kVerifyThreads / 32];
};

// x / z, correctly rounded, for many x and one z: with y the correctly rounded 1/z, the
// remainder of x y corrects it (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990). For significands that was checked one by one: every
// divisor with all dividends whose quotient lies within 24 / 2z units of a rounding boundary,
// 535 million pairs. It takes 1/z, the quotient and the remainder to be normal numbers:
// divisors from 2^-100 to 2^16 and dividends from 2^-100 on (or 0; a divisor of 1 takes any).
// The others, of rows that are nearly empty or hold almost nothing, are divided.
__device__ __forceinline__ float quotient(float x, float z, float y) {
  const float q = __fmul_rn(x, y);
  return __fmaf_rn(__fmaf_rn(-q, z, x), y, q);
}
// The bits of x less 1, so that 0 is larger than any; and the least of them that quotient() takes
// for a divisor.
__device__ __forceinline__ unsigned quotient_order(float x) { return __float_as_uint(x) - 1u; }
__device__ __forceinline__ unsigned quotient_least(float z) {
  return z == 1.0f ? 0u : z >= 0x1p-100f && z <= 0x1p16f ? __float_as_uint(0x1p-100f) - 1u : 0xffffffffu;
}

// r_k(t) from p(t), q(t) and the refusals.
template <bool kDraft>
__device__ __forceinline__ float residual(const VerifyShared<kDraft>& sh, float p, float q, int t, int k) {
  float r = p;
  for (int j = 0; j < k; ++j) {
    if constexpr (kDraft) {
      const float x = quotient_order(r) >= sh.least[j] ? quotient(r, sh.z[j], sh.inverse[j]) : __fdiv_rn(r, sh.z[j]);
      r = fmaxf(__fsub_rn(x, q), 0.0f);
    } else r = sh.token[sh.refused[j]] == t ? 0.0f : r;
  }
  return r;
}

// f(t, p(t), q(t), e(t)) for the tokens v0 <= t < v1 of this thread; q and e may be NULL.
template <class F>
__device__ __forceinline__ void scan_row(int v0, int v1, const float* p, const float* q, const float* e, F f) {
  for (int t0 = v0 + static_cast<int>(threadIdx.x); t0 < v1; t0 += kVerifyThreads * kVerifyBatch) {
    float pv[kVerifyBatch], qv[kVerifyBatch], ev[kVerifyBatch];
#pragma unroll
    for (int i = 0; i < kVerifyBatch; ++i) {
      const int t = t0 + i * kVerifyThreads;
      pv[i] = t < v1 ? p[t] : 0.0f;
      qv[i] = q != nullptr && t < v1 ? q[t] : 0.0f;
      ev[i] = e != nullptr && t < v1 ? e[t] : 1.0f;
    }
#pragma unroll
    for (int i = 0; i < kVerifyBatch; ++i) {
      const int t = t0 + i * kVerifyThreads;
      if (t < v1) f(t, pv[i], qv[i], ev[i]);
    }
  }
}

// kFit: a CTA's share fits in its threads' registers.
template <bool kDraft, bool kFit>
__global__ void __launch_bounds__(kVerifyThreads, 1) k_verify(const __grid_constant__ VerifyArgs a) {
  __shared__ VerifyShared<kDraft> sh;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = static_cast<int>(cl.block_rank()), ctas = static_cast<int>(cl.num_blocks());
  const long long b = blockIdx.x / static_cast<unsigned>(ctas);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.n;
  const int share = verify_share(a.vocab, ctas);
  const int v0 = min(rank * share, a.vocab), v1 = min(v0 + share, a.vocab);
  pdl_launch_dependents();
  cl.barrier_arrive();  // (waited for below: every CTA of the cluster runs before another writes to it)
  pdl_wait();
  // The noise is read in any case; the root's rows more often than not.
  for (int t = v0 + tid * 32; t < v1; t += kVerifyThreads * 32) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.noise + b * a.ld_noise + t));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.target + b * n * a.ld_target + t));
    if (kDraft) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.draft + b * n * a.ld_draft + t));
  }
  bool bad = false;
  for (int i = tid; i < n; i += kVerifyThreads) {
    const int p = a.parents[b * n + i];
    const int t = i > 0 ? a.tokens[b * n + i] : 0;
    sh.up[i] = p;
    sh.token[i] = t;
    sh.u[i] = i > 0 ? a.u[b * n + i] : 0.0f;
    const bool wrong = i == 0 ? p != -1 : (p < 0 || p >= i || t < 0 || t >= a.vocab);
    bad |= wrong;
    if (i > 0 && !wrong) {
      const long long row = b * n + p;
      sh.p[i] = a.target[row * a.ld_target + t];
      sh.q[i] = kDraft ? a.draft[row * a.ld_draft + t] : 1.0f;
    }
  }
  bad = __syncthreads_or(bad);
  cl.barrier_wait();
  if (bad) {  // every CTA of the cluster sees the same
    if (rank == 0) {
      for (int i = tid; i < n; i += kVerifyThreads) a.path[b * n + i] = -1;
      if (tid == 0) {
        a.n_path[b] = 0;
        a.next_token[b] = -1;
        record_status(a.dev_status, RF_ERR_INVALID_ARG);
      }
    }
    return;
  }
  auto set_z = [&](int j, float z) {
    sh.z[j] = z;
    if constexpr (kDraft) {
      sh.inverse[j] = __frcp_rn(z);
      sh.least[j] = quotient_least(z);
    }
  };
  int cur = 0, k = 0, n_acc = 1, turn = 0;
  if (tid == 0) {
    sh.path[0] = 0;
    set_z(0, 1.0f);
  }
  __syncthreads();

  // The thread's tokens v0 + tid, v0 + tid + 1024, ...: r after `applied` refusals at `cur`
  // (-1: not read yet), and q.
  const int slots = (v1 - v0 + kVerifyThreads - 1) / kVerifyThreads;
  float r[kFit ? kVerifySlots : 1], q[kFit && kDraft ? kVerifySlots : 1];
  int applied = -1;
  auto bring = [&] {
    if constexpr (kFit) {
      if (applied < 0 || applied > k) {
        const float* p = a.target + (b * n + cur) * a.ld_target;
        const float* d = kDraft ? a.draft + (b * n + cur) * a.ld_draft : nullptr;
#pragma unroll
        for (int i = 0; i < kVerifySlots; ++i) {
          const int t = v0 + tid + i * kVerifyThreads;
          r[i] = t < v1 ? p[t] : 0.0f;
          if constexpr (kDraft) q[i] = t < v1 ? d[t] : 0.0f;
        }
        applied = 0;
      }
      for (; applied < k; ++applied) {
        if constexpr (kDraft) {
          const float z = sh.z[applied], y = sh.inverse[applied];
          unsigned order = 0xffffffffu;
#pragma unroll
          for (int i = 0; i < kVerifySlots; ++i) order = min(order, quotient_order(r[i]));
          if (order >= sh.least[applied]) {
#pragma unroll
            for (int i = 0; i < kVerifySlots; ++i)
              if (i < slots) r[i] = fmaxf(__fsub_rn(quotient(r[i], z, y), q[i]), 0.0f);
          } else {
#pragma unroll
            for (int i = 0; i < kVerifySlots; ++i)
              if (i < slots) r[i] = fmaxf(__fsub_rn(__fdiv_rn(r[i], z), q[i]), 0.0f);
          }
        } else {
          const int gone = sh.token[sh.refused[applied]] - v0 - tid;
#pragma unroll
          for (int i = 0; i < kVerifySlots; ++i)
            if (i < slots) r[i] = gone == i * kVerifyThreads ? 0.0f : r[i];
        }
      }
    }
  };
  // The next child of `cur` after node `c`, or n: 32 nodes at a time.
  auto next_child = [&](int c) {
    for (int c0 = c + 1; c0 < n; c0 += 32) {
      const unsigned hit = __ballot_sync(0xffffffffu, c0 + lane < n && sh.up[c0 + lane] == cur);
      if (hit) return c0 + __ffs(hit) - 1;
    }
    return n;
  };
  int c = next_child(0);
  while (c < n) {
    const float rx = residual(sh, sh.p[c], sh.q[c], sh.token[c], k);
    if (__fmul_rn(__fmul_rn(sh.u[c], sh.q[c]), sh.z[k]) < rx) {
      __syncthreads();  // the refusals of the node left behind are read no more
      if (tid == 0) {
        sh.path[n_acc] = c;
        set_z(0, 1.0f);
      }
      ++n_acc;
      cur = c;
      k = 0;
      applied = -1;
      c = next_child(c);
      __syncthreads();
      continue;
    }
    const int sibling = next_child(c);
    if constexpr (!kDraft) {
      if (tid == 0) sh.refused[k] = c;
      __syncthreads();
    }
    ++k;
    if (sibling < n) {
      // Z_k, this CTA's share, then the cluster's
      float sum = 0.0f;
      if constexpr (kFit) {
        bring();
#pragma unroll
        for (int i = 0; i < kVerifySlots; ++i)
          if (i < slots) sum += r[i];
      } else {
        scan_row(v0, v1, a.target + (b * n + cur) * a.ld_target, kDraft ? a.draft + (b * n + cur) * a.ld_draft : nullptr,
                 nullptr, [&](int t, float pt, float qt, float) { sum += residual(sh, pt, qt, t, k); });
      }
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) sh.warp_sum[warp] = sum;
      __syncthreads();
      if (warp == 0) {
        float s = lane < kVerifyThreads / 32 ? sh.warp_sum[lane] : 0.0f;
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane < ctas) *cl.map_shared_rank(&sh.part_sum[turn & 1][rank], lane) = s;
      }
      cl.sync();
      float z = lane < ctas ? sh.part_sum[turn & 1][lane] : 0.0f;
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      ++turn;
      if (z > 0.0f) {
        if (tid == 0) set_z(k, z);
      } else {
        --k;  // nothing would be left: the residual stays, and is read anew
        applied = -1;
      }
      __syncthreads();
    }
    c = sibling;
  }

  // The lowest argmax of r / noise: the score's bits (scores are >= 0) above the
  // complement of the token.
  const float* e = a.noise + b * a.ld_noise;
  int token = 0;
  while (true) {
    unsigned long long best = 0;
    auto look = [&](int t, float rt, float et) {
      const float score = rt > 0.0f ? __fdiv_rn(rt, et) : 0.0f;
      best = max(best, (static_cast<unsigned long long>(__float_as_uint(score)) << 32) |
                           (0xffffffffu - static_cast<unsigned>(t)));
    };
    if constexpr (kFit) {
      float ev[kVerifySlots];
#pragma unroll
      for (int i = 0; i < kVerifySlots; ++i) {
        const int t = v0 + tid + i * kVerifyThreads;
        ev[i] = t < v1 ? e[t] : 1.0f;
      }
      bring();
#pragma unroll
      for (int i = 0; i < kVerifySlots; ++i) {
        const int t = v0 + tid + i * kVerifyThreads;
        if (t < v1) look(t, r[i], ev[i]);
      }
    } else {
      scan_row(v0, v1, a.target + (b * n + cur) * a.ld_target, kDraft ? a.draft + (b * n + cur) * a.ld_draft : nullptr, e,
               [&](int t, float pt, float qt, float et) { look(t, residual(sh, pt, qt, t, k), et); });
    }
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) sh.warp_best[warp] = best;
    __syncthreads();
    if (warp == 0) {
      unsigned long long m = lane < kVerifyThreads / 32 ? sh.warp_best[lane] : 0ull;
      for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane < ctas) *cl.map_shared_rank(&sh.part_best[turn & 1][rank], lane) = m;
    }
    cl.sync();
    unsigned long long m = lane < ctas ? sh.part_best[turn & 1][lane] : 0ull;
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    ++turn;
    token = static_cast<int>(0xffffffffu - static_cast<unsigned>(m & 0xffffffffu));
    // All zero: the last refusal's residual is empty, so the one before it stands.
    if ((m >> 32) != 0 || k == 0) break;
    --k;
    __syncthreads();
  }
  if (rank == 0) {
    for (int i = tid; i < n; i += kVerifyThreads) a.path[b * n + i] = i < n_acc ? sh.path[i] : -1;
    if (tid == 0) {
      a.n_path[b] = n_acc;
      a.next_token[b] = token;
    }
  }
}

struct CommitArgs {
  const int32_t* path;
  const int32_t* n_path;
  const int32_t* lens;
  const int32_t* next_pos;
  const __nv_bfloat16* kd;
  const __nv_bfloat16* vd;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  float* score;
  int32_t* pos;
  int32_t* new_lens;
  int32_t* new_next_pos;
  int32_t* dev_status;
  long long row_stride, seq_stride, layer_stride, draft_row, draft_seq, draft_layer;
  int n_seqs, heads, width, capacity, n;  // width = heads * head_dim
  int lens_here;  // k_commit itself writes the lengths (new ones lie apart from its inputs)
};

// Whether sequence b's rows may be appended (whole CTA).
__device__ __forceinline__ bool commit_ok(const CommitArgs& a, int b, int cnt, int len) {
  bool bad = cnt < 0 || cnt > a.n || len < 0 || len > a.capacity - cnt;
  if (!bad)
    for (int j = threadIdx.x; j < cnt; j += blockDim.x) {
      const int i = a.path[static_cast<long long>(b) * a.n + j];
      bad |= i < 0 || i >= a.n;
    }
  return !__syncthreads_or(bad);
}

__device__ __forceinline__ void write_lens(const CommitArgs& a, int b, bool ok, int cnt, int len, int next) {
  if (!ok) record_status(a.dev_status, RF_ERR_INVALID_ARG);
  if (a.new_lens != nullptr) a.new_lens[b] = len + (ok ? cnt : 0);
  if (a.new_next_pos != nullptr) a.new_next_pos[b] = next + (ok ? cnt : 0);
}

// Layer blockIdx.x, sequence blockIdx.y.
__global__ void __launch_bounds__(256) k_commit(const __grid_constant__ CommitArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int l = blockIdx.x, b = blockIdx.y;
  const int cnt = a.n_path[b], len = a.lens[b];
  const bool ok = commit_ok(a, b, cnt, len);
  if (a.lens_here && l == 0 && threadIdx.x == 0) write_lens(a, b, ok, cnt, len, a.next_pos != nullptr ? a.next_pos[b] : 0);
  if (!ok) return;
  const int pieces = a.width / 8;
#pragma unroll 4
  for (int x = threadIdx.x; x < cnt * pieces; x += 256) {
    const int j = x / pieces, c = (x - j * pieces) * 8;
    const long long src = l * a.draft_layer + b * a.draft_seq +
                          static_cast<long long>(a.path[static_cast<long long>(b) * a.n + j]) * a.draft_row + c;
    const long long dst = l * a.layer_stride + b * a.seq_stride + static_cast<long long>(len + j) * a.row_stride + c;
    const uint4 k = *reinterpret_cast<const uint4*>(a.kd + src), v = *reinterpret_cast<const uint4*>(a.vd + src);
    *reinterpret_cast<uint4*>(a.k + dst) = k;
    *reinterpret_cast<uint4*>(a.v + dst) = v;
  }
  for (int x = threadIdx.x; x < cnt * a.heads; x += 256) {
    const int h = x / cnt, j = x - h * cnt;
    const long long at = ((static_cast<long long>(l) * a.n_seqs + b) * a.heads + h) * a.capacity + len + j;
    if (a.score != nullptr) a.score[at] = 0.0f;
    if (a.pos != nullptr) a.pos[at] = a.next_pos[b] + j;
  }
}

// Where new lengths or positions are written over lens, next_pos or n_path, they are written behind
// all of k_commit's reads: by a dependent launch, one CTA a sequence.
__global__ void __launch_bounds__(64) k_commit_lens(const __grid_constant__ CommitArgs a) {
  pdl_wait();
  const int b = blockIdx.x;
  const int cnt = a.n_path[b], len = a.lens[b];
  const int next = a.next_pos != nullptr ? a.next_pos[b] : 0;
  const bool ok = commit_ok(a, b, cnt, len);
  if (threadIdx.x == 0) write_lens(a, b, ok, cnt, len, next);
}

}  // namespace rf

using namespace rf;

extern "C" rf_status rf_verify_draft(const rf_verify_desc* d, const float* target, const float* draft,
                                     const int32_t* tokens, const int32_t* parents, const float* u, const float* noise,
                                     int32_t* path, int32_t* n_path, int32_t* next_token, int32_t* dev_status,
                                     rf_stream_t stream) {
  clear_error();
  if (d == nullptr) return fail(RF_ERR_INVALID_ARG, "desc is NULL");
  if (d->n_seqs < 0 || d->n_nodes <= 0 || d->vocab <= 0)
    return fail(RF_ERR_INVALID_ARG, "need n_seqs >= 0, n_nodes, vocab > 0");
  if (d->n_nodes > RF_TREE_MAX_NODES || d->vocab > (int64_t(1) << 31) - 65536 || d->n_seqs > (int64_t(1) << 24))
    return fail(RF_ERR_SHAPE, "n_nodes must be <= %d, vocab <= 2^31 - 65536, n_seqs <= 2^24", RF_TREE_MAX_NODES);
  if (d->ld_target < d->vocab || d->ld_noise < d->vocab || (draft != nullptr && d->ld_draft < d->vocab))
    return fail(RF_ERR_ALIGN, "row strides must be >= vocab");
  if (d->n_seqs == 0) return RF_OK;
  if (!target || !noise || !path || !n_path || !next_token || !parents || (d->n_nodes > 1 && (!tokens || !u)))
    return fail(RF_ERR_INVALID_ARG, "tensor pointers must be non-NULL");
  const uintptr_t bits = reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft) |
                         reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(parents) |
                         reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(noise) |
                         reinterpret_cast<uintptr_t>(path) | reinterpret_cast<uintptr_t>(n_path) |
                         reinterpret_cast<uintptr_t>(next_token);
  if (bits & 3u) return fail(RF_ERR_ALIGN, "arrays must be 4-byte aligned");
  int sms = 0;
  rf_status st = current_device(&sms);
  if (st != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  VerifyArgs a{};
  a.target = target;
  a.draft = draft;
  a.tokens = tokens;
  a.parents = parents;
  a.u = u;
  a.noise = noise;
  a.path = path;
  a.n_path = n_path;
  a.next_token = next_token;
  a.dev_status = dev_status;
  a.ld_target = d->ld_target;
  a.ld_draft = d->ld_draft;
  a.ld_noise = d->ld_noise;
  a.n = static_cast<int>(d->n_nodes);
  a.vocab = static_cast<int>(d->vocab);
  // a power of two of CTAs, so many that each has a few tokens a thread
  unsigned ctas = 1;
  while (ctas < kVerifyCtas && static_cast<int64_t>(ctas) * kVerifyShare < d->vocab) ctas *= 2;
  ProfScope prof(s, RF_STAGE_VERIFY);
  const bool fit = verify_share(a.vocab, static_cast<int>(ctas)) <= kVerifyThreads * kVerifySlots;
  void (*kernel)(VerifyArgs) = draft != nullptr ? (fit ? k_verify<true, true> : k_verify<true, false>)
                                                : (fit ? k_verify<false, true> : k_verify<false, false>);
  return cuda_check(launch_dependent(kernel, dim3(static_cast<unsigned>(d->n_seqs) * ctas), dim3(kVerifyThreads), 0, s, ctas, a),
                    "k_verify launch");
}

extern "C" rf_status rf_commit_draft(const rf_cache_desc* d, int64_t n_nodes, int64_t draft_row_stride,
                                     int64_t draft_seq_stride, int64_t draft_layer_stride, const int32_t* path,
                                     const int32_t* n_path, const int32_t* lens, const int32_t* next_pos,
                                     const rf_bf16* k_draft, const rf_bf16* v_draft, rf_bf16* k_cache, rf_bf16* v_cache,
                                     float* score, int32_t* pos, int32_t* new_lens, int32_t* new_next_pos,
                                     int32_t* dev_status, rf_stream_t stream) {
  clear_error();
  rf_status st = check_cache_desc(d);
  if (st != RF_OK) return st;
  if (n_nodes <= 0) return fail(RF_ERR_INVALID_ARG, "need n_nodes > 0");
  if (n_nodes > (int64_t(1) << 20)) return fail(RF_ERR_SHAPE, "n_nodes must be <= 2^20");
  const int64_t width = d->n_kv_heads * d->head_dim;
  if (draft_row_stride < width || draft_row_stride % 8 || draft_seq_stride % 8 || draft_layer_stride % 8 ||
      draft_seq_stride < 0 || draft_layer_stride < 0)
    return fail(RF_ERR_ALIGN, "draft strides must be multiples of 8, the row stride >= n_kv_heads*head_dim");
  if (n_nodes * (width / 8) >= (int64_t(1) << 31) || n_nodes * d->n_kv_heads >= (int64_t(1) << 31))
    return fail(RF_ERR_SHAPE, "n_nodes * n_kv_heads * head_dim is too large");
  if (d->n_seqs == 0) return RF_OK;
  if (!path || !n_path || !lens || (d->n_layers > 0 && (!k_draft || !v_draft || !k_cache || !v_cache)) ||
      (!next_pos && (pos || new_next_pos)))
    return fail(RF_ERR_INVALID_ARG, "tensor pointers must be non-NULL");
  if (!aligned16(k_draft) || !aligned16(v_draft) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(RF_ERR_ALIGN, "row buffers must be 16-byte aligned");
  const uintptr_t bits = reinterpret_cast<uintptr_t>(path) | reinterpret_cast<uintptr_t>(n_path) |
                         reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(next_pos) |
                         reinterpret_cast<uintptr_t>(score) | reinterpret_cast<uintptr_t>(pos) |
                         reinterpret_cast<uintptr_t>(new_lens) | reinterpret_cast<uintptr_t>(new_next_pos);
  if (bits & 3u) return fail(RF_ERR_ALIGN, "arrays must be 4-byte aligned");
  // Lengths written over an input, element by element, wait for all of k_commit's reads; no order
  // would be right where arrays overlap otherwise.
  bool over_inputs = false;
  for (const int32_t* w : {new_lens, new_next_pos}) {
    if (overlap(w, d->n_seqs, path, d->n_seqs * n_nodes))
      return fail(RF_ERR_INVALID_ARG, "new_lens and new_next_pos must lie apart from path");
    for (const int32_t* r : {lens, next_pos, n_path}) {
      if (!overlap(w, d->n_seqs, r, d->n_seqs)) continue;
      if (w != r) return fail(RF_ERR_INVALID_ARG, "new_lens and new_next_pos must not overlap an input in part");
      over_inputs = true;
    }
  }
  int sms = 0;
  if ((st = current_device(&sms)) != RF_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CommitArgs a{};
  a.path = path;
  a.n_path = n_path;
  a.lens = lens;
  a.next_pos = next_pos;
  a.kd = reinterpret_cast<const __nv_bfloat16*>(k_draft);
  a.vd = reinterpret_cast<const __nv_bfloat16*>(v_draft);
  a.k = reinterpret_cast<__nv_bfloat16*>(k_cache);
  a.v = reinterpret_cast<__nv_bfloat16*>(v_cache);
  a.score = score;
  a.pos = pos;
  a.new_lens = new_lens;
  a.new_next_pos = new_next_pos;
  a.dev_status = dev_status;
  a.row_stride = d->row_stride;
  a.seq_stride = d->seq_stride;
  a.layer_stride = d->layer_stride;
  a.draft_row = draft_row_stride;
  a.draft_seq = draft_seq_stride;
  a.draft_layer = draft_layer_stride;
  a.n_seqs = static_cast<int>(d->n_seqs);
  a.heads = static_cast<int>(d->n_kv_heads);
  a.width = static_cast<int>(width);
  a.capacity = static_cast<int>(d->capacity);
  a.n = static_cast<int>(n_nodes);
  a.lens_here = d->n_layers > 0 && !over_inputs;
  if (d->n_layers > 0) {
    ProfScope prof(s, RF_STAGE_COMMIT);
    st = cuda_check(launch_dependent(k_commit, dim3(static_cast<unsigned>(d->n_layers), static_cast<unsigned>(d->n_seqs)),
                                     dim3(256), 0, s, 1, a),
                    "k_commit launch");
    if (st != RF_OK) return st;
  }
  if (a.lens_here) return RF_OK;
  ProfScope prof(s, RF_STAGE_COMMIT);
  return cuda_check(launch_dependent(k_commit_lens, dim3(static_cast<unsigned>(d->n_seqs)), dim3(64), 0, s, 1, a),
                    "k_commit_lens launch");
}
