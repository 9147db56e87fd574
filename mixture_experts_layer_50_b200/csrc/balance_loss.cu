// The balance loss of a routed batch, its per-expert counts and its gradient.
//
// "Основы MoE", "Вспомогательный лосс Switch Transformer": with f_i the share of the top-k
// assignments that went to expert i and P_i its router probability averaged over the tokens,
//   L = alpha * E * sum_i f_i P_i.
// f is made of counts and has no gradient; with p_t the probabilities of token t (softmax, or
// sigmoid affinities normalised to sum 1), T tokens and g the gradient of L,
//   dL/dz_ti = g alpha E / T * p_ti u_ti (f_i - sum_j f_j p_tj),
//   u_ti = 1 (softmax), 1 - sigma(z_ti) (sigmoid).
// As sum_j p_tj = 1, any constant may be taken off f: the kernel uses f_i - 1/E, so that a
// nearly balanced batch loses no digits in the difference.
//
// Two launches.  Clusters of kCountCtas blocks, one for every kCountIds assignments, count them
// (integers; a cluster's counts meet over distributed shared memory and are written once) and
// clear the accumulators of the second launch, so nothing has to be zero before the call.  Then
// every token's row is read once: its probabilities give its gradient row, and add to P.  P is
// added up in 64-bit fixed point, which makes its value independent of the order of the atomic
// additions; the last block to finish turns the sums into P and the loss.  (Additions to shared
// memory bound the count: one cluster took 15 us for 16384 tokens of six experts.)
//
// Bound: one read of the logits and one write of the gradient; small batches by the two launches
// (64 tokens of 256 experts and 8191 of 8 take 7.3 us each in a captured graph).  For 16384 padded
// tokens of 384 experts the reads and writes are 7.8 us of 19.0: the count takes 5 us, its
// additions and its cluster's meeting; in the row pass a scheduler issues in 49 % of its slots with 38 %
// of an SM's threads (80 registers hold twelve experts a lane, the next token's logits and the
// sums of P), and warps wait for two or three reductions per token.  Reading a token ahead and 16
// bytes at a time took the whole from 37.6 to 21.5 us; starting the row pass beside the count, with
// its first logits on their way and all counts in flight at once, to 20.2 us; larger blocks, to 19.0.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kCountCtas = 8;
constexpr int kCountThreads = 1024;
constexpr int kCountUnroll = 4;
constexpr int kCountIds = 8192, kMaxCounts = 16;
constexpr float kFarSum = 5.9604645e-8f;  // 2^-24: a sum of sigmoids below it

// Scratch of one call (device): sums [E] u64, the clusters' counts [n][E] and tokens [n], and
// the ticket.
struct LossScratch {
  unsigned long long* sums;
  int32_t* counts;
  int32_t* tokens;
  unsigned* ticket;
  int n;  // clusters
};
LossScratch scratch_of(void* p, int E, int n) {
  LossScratch s;
  s.sums = static_cast<unsigned long long*>(p);
  s.counts = reinterpret_cast<int32_t*>(s.sums + E);
  s.tokens = s.counts + (size_t)kMaxCounts * E;
  s.ticket = reinterpret_cast<unsigned*>(s.tokens + kMaxCounts);
  s.n = n;
  return s;
}

__global__ void __cluster_dims__(kCountCtas, 1, 1) __launch_bounds__(kCountThreads)
    balance_count_kernel(const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
                         int64_t N, int E, int k, int32_t* __restrict__ counts, LossScratch out,
                         int* status) {
  pdl_wait();
  pdl_release();  // the row pass may load logits: what made them has ended
  extern __shared__ int32_t s_count[];  // [E], then the block's tokens
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  for (int i = threadIdx.x; i <= E; i += kCountThreads) s_count[i] = 0;
  __syncthreads();
  bool bad = false;
  // N * k is below 2^30 (checked on the host), so are all indices
  const uint32_t stride = gridDim.x * kCountThreads, nk = (uint32_t)(N * k);
  const uint32_t first = blockIdx.x * kCountThreads + threadIdx.x;
  for (uint32_t i = first; i < nk; i += kCountUnroll * stride) {
    // all loads of a turn are in flight before its first addition
    int e[kCountUnroll];
    bool on[kCountUnroll];
#pragma unroll
    for (int j = 0; j < kCountUnroll; ++j) {
      const uint32_t at = i + j * stride;
      on[j] = at < nk;
      e[j] = on[j] ? ids[at] : 0;
    }
    if (mask != nullptr) {
#pragma unroll
      for (int j = 0; j < kCountUnroll; ++j)
        if (on[j]) on[j] = mask[(i + j * stride) / (uint32_t)k] != 0;
    }
#pragma unroll
    for (int j = 0; j < kCountUnroll; ++j) {
      if (!on[j]) continue;
      if (e[j] >= 0 && e[j] < E)
        atomicAdd(&s_count[e[j]], 1);
      else
        bad = true;
    }
  }
  if (mask != nullptr) {
    int n = 0;
    for (uint32_t t = first; t < (uint32_t)N; t += stride)
      n += mask[t] != 0;
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if ((threadIdx.x & 31) == 0 && n != 0) atomicAdd(&s_count[E], n);
  }
  if (bad) report_status(status, kStatusInvalidInput);
  cluster.sync();
  const int c = (int)blockIdx.x / kCountCtas;
  for (int e = rank * kCountThreads + threadIdx.x; e <= E; e += kCountCtas * kCountThreads) {
    int n = 0;
    for (int b = 0; b < kCountCtas; ++b) n += cluster.map_shared_rank(s_count, b)[e];
    if (e == E) {
      out.tokens[c] = mask != nullptr ? n : c == 0 ? (int32_t)N : 0;
      continue;
    }
    out.counts[c * E + e] = n;
    if (counts != nullptr) counts[e] = n;  // (given where there is one cluster)
    if (c == 0) out.sums[e] = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *out.ticket = 0;
  cluster.sync();  // no block leaves while another reads its counts
}

struct LossArgs {
  const float* logits;
  const uint8_t* mask;
  int64_t N;
  int E;
  float alpha;
  const float* grad_loss;  // the gradient of the loss (device), or null: 1
  float* loss;
  int32_t* counts;  // where the count kernel has not written them
  float* P;
  float* dlogits;
  int accumulate;
  int want_sums;
  int k;
  float fixed_scale;  // power of two; N * fixed_scale < 2^62
  LossScratch s;
};

template <int kTeam>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
  for (int o = kTeam / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int kTeam>
__device__ __forceinline__ float team_max(float v) {
#pragma unroll
  for (int o = kTeam / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// kTeam lanes own a token.  Lane i of the team holds kEpl experts: i, i + kTeam, ..., or with
// kVec, in runs of four, 4 i ... 4 i + 3, 4 (i + kTeam) ....
template <int kTeam, bool kVec>
__device__ __forceinline__ int expert_of(int ti, int j) {
  return kVec ? 4 * (ti + j / 4 * kTeam) + j % 4 : ti + j * kTeam;
}

// (An expert a lane: six blocks on an SM need 40 registers, which the sigmoid form is told to keep
// to; with 48 16384 tokens of 32 experts take 14.5 us, with 40 12.1.)
template <int kTeam, int kEpl, bool kVec, bool kSigmoid, int kLossThreads>
__global__ void __launch_bounds__(kLossThreads, kSigmoid && kEpl == 1 ? 6 : 0)
    balance_loss_kernel(const LossArgs a) {
  constexpr int kTeams = kLossThreads / kTeam;
  extern __shared__ float s_f[];  // f [E]; then [kTeams][E] sums
  const int E = a.E;
  float* const s_p = s_f + E;
  const int ti = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
  // a token's logits, -infinity where there are none
  auto load = [&](int64_t t, float (&z)[kEpl]) {
    const bool live = t < a.N && (a.mask == nullptr || a.mask[t] != 0);
#pragma unroll
    for (int j = 0; j < kEpl; j += kVec ? 4 : 1) {
      const int e = expert_of<kTeam, kVec>(ti, j);
      const bool in = live && e < E;
      if constexpr (kVec) {
        const float4 v = in ? __ldg(reinterpret_cast<const float4*>(a.logits + t * E + e))
                            : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        z[j] = v.x;
        z[j + 1] = v.y;
        z[j + 2] = v.z;
        z[j + 3] = v.w;
      } else {
        z[j] = in ? __ldg(a.logits + t * E + e) : -INFINITY;
      }
    }
    return live;
  };
  // The first tokens' logits are on their way before the counts are there: the count kernel lets
  // this one start after all that came before itself has ended.
  float next[kEpl];
  bool next_live = load((int64_t)blockIdx.x * kTeams + team, next);
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int T = __reduce_add_sync(0xffffffffu, lane < a.s.n ? a.s.tokens[lane] : 0);
  const double per = 1.0 / ((double)(T > 0 ? T : 1) * a.k);
  for (int e = threadIdx.x; e < E; e += kLossThreads) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < kMaxCounts; ++c)
      if (c < a.s.n) n += a.s.counts[c * E + e];
    s_f[e] = (float)(n * per);
    s_p[e] = (float)(n * per - 1.0 / E);
    if (a.counts != nullptr && blockIdx.x == 0) a.counts[e] = n;
  }
  __syncthreads();
  const float g = (a.grad_loss != nullptr ? *a.grad_loss : 1.f) * a.alpha * (float)E /
                  (float)(T > 0 ? T : 1);
  float f0[kEpl], acc[kEpl];
#pragma unroll
  for (int j = 0; j < kEpl; ++j) {
    const int e = expert_of<kTeam, kVec>(ti, j);
    f0[j] = e < E ? s_p[e] : 0.f;
    acc[j] = 0.f;
  }
  // every team of the block takes the same number of steps: the shuffles need whole warps
  const int64_t step = (int64_t)gridDim.x * kTeams;
  for (int64_t t0 = (int64_t)blockIdx.x * kTeams; t0 < a.N; t0 += step) {
    const int64_t t = t0 + team;
    const bool live = next_live;
    float p[kEpl], u[kEpl];
#pragma unroll
    for (int j = 0; j < kEpl; ++j) p[j] = next[j];
    if (t0 + step < a.N) next_live = load(t + step, next);
    float sum = 0.f;
    if (kSigmoid) {
#pragma unroll
      for (int j = 0; j < kEpl; ++j) {
        // with q = exp(-|z|): sigma and 1 - sigma are 1 / (1 + q) and q / (1 + q), whichever way
        const float q = expf(-fabsf(p[j])), big = 1.f / (1.f + q), small = q * big;
        const bool neg = p[j] < 0.f;
        u[j] = neg ? big : small;
        p[j] = neg ? small : big;
        sum += p[j];
      }
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < kEpl; ++j) m = fmaxf(m, p[j]);
      m = team_max<kTeam>(m);
      // a row without any finite logit has no probabilities: all 0, and no gradient
      if (m == -INFINITY) m = 0.f;
#pragma unroll
      for (int j = 0; j < kEpl; ++j) {
        p[j] = expf(p[j] - m);
        sum += p[j];
      }
    }
    sum = team_sum<kTeam>(sum);
    if constexpr (kSigmoid) {
      // Sigmoids that are all below 2^-24 lose their digits further down and end as 0, while their
      // shares are as good as any; 1 + exp(z) is 1 there, and the shares are the softmax.  The
      // logits are read again, for which ordinary rows pay nothing; a masked token has none.
      const bool far = live && sum < kFarSum;
      if (__any_sync(0xffffffffu, far)) {
        float m = -INFINITY, far_sum = 0.f;
        if (far) {
          load(t, p);
#pragma unroll
          for (int j = 0; j < kEpl; ++j) m = fmaxf(m, p[j]);
        }
        m = team_max<kTeam>(m);
        if (m == -INFINITY) m = 0.f;
        if (far) {
#pragma unroll
          for (int j = 0; j < kEpl; ++j) {
            p[j] = expf(p[j] - m);
            far_sum += p[j];
          }
        }
        far_sum = team_sum<kTeam>(far_sum);
        if (far) sum = far_sum;
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
      p[j] *= inv;
      acc[j] += p[j];
      dot = fmaf(p[j], f0[j], dot);
    }
    if (a.dlogits == nullptr) continue;
    dot = team_sum<kTeam>(dot);
    if (t >= a.N) continue;
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
      p[j] = live ? g * (p[j] * (f0[j] - dot)) : 0.f;
      if (kSigmoid && live) p[j] *= u[j];
    }
    if (a.accumulate && !live) continue;
#pragma unroll
    for (int j = 0; j < kEpl; j += kVec ? 4 : 1) {
      const int e = expert_of<kTeam, kVec>(ti, j);
      if (e >= E) continue;
      float* dz = a.dlogits + t * E + e;
      if constexpr (kVec) {
        float4 v = make_float4(p[j], p[j + 1], p[j + 2], p[j + 3]);
        if (a.accumulate) {
          const float4 o = *reinterpret_cast<const float4*>(dz);
          v.x += o.x;
          v.y += o.y;
          v.z += o.z;
          v.w += o.w;
        }
        *reinterpret_cast<float4*>(dz) = v;
      } else {
        *dz = a.accumulate ? *dz + p[j] : p[j];
      }
    }
  }
  if (!a.want_sums) return;
  __syncthreads();  // f - 1/E has been read
#pragma unroll
  for (int j = 0; j < kEpl; ++j) {
    const int e = expert_of<kTeam, kVec>(ti, j);
    if (e < E) s_p[team * E + e] = acc[j];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kLossThreads) {
    float v = 0.f;
    for (int i = 0; i < kTeams; ++i) v += s_p[i * E + e];
    // sums stay below 2^62: the top bit is free to stand for a NaN (or an infinity, which has no
    // place in the sums either)
    if (!(v < INFINITY))
      atomicOr(&a.s.sums[e], 1ull << 63);
    else if (v != 0.f)
      atomicAdd(&a.s.sums[e], (unsigned long long)((double)v * (double)a.fixed_scale));
  }
  __shared__ bool s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();  // the block's additions come before its ticket
    s_last = atomicAdd(a.s.ticket, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  double part = 0.0;
  for (int e = threadIdx.x; e < E; e += kLossThreads) {
    const unsigned long long v = __ldcg(&a.s.sums[e]);
    const double Pe = (v >> 63) ? (double)NAN
                                : (double)v / ((double)a.fixed_scale * (T > 0 ? T : 1));
    if (a.P != nullptr) a.P[e] = (float)Pe;
    part += (double)s_f[e] * Pe;
  }
  __shared__ double s_sum[kLossThreads];
  s_sum[threadIdx.x] = part;
  for (int w = 512; w > 0; w >>= 1) {
    __syncthreads();
    if (threadIdx.x < w && threadIdx.x + w < kLossThreads) s_sum[threadIdx.x] += s_sum[threadIdx.x + w];
  }
  if (threadIdx.x == 0 && a.loss != nullptr)
    a.loss[0] = (float)((double)a.alpha * E * s_sum[0]);
}

template <int kTeam, int kEpl, bool kVec, bool kSigmoid, int kThreads>
cudaError_t launch_blocks(const LossArgs& a, int64_t blocks, cudaStream_t stream) {
  const size_t smem = sizeof(float) * a.E * (1 + (a.want_sums ? kThreads / kTeam : 1));
  return launch_pdl(balance_loss_kernel<kTeam, kEpl, kVec, kSigmoid, kThreads>, (unsigned)blocks,
                    kThreads, smem, stream, a);
}

template <int kTeam, int kEpl, bool kVec, bool kSigmoid>
cudaError_t launch_teams(const LossArgs& a, int sms, cudaStream_t stream) {
  // blocks of 256 threads that the registers let be on an SM at once
  constexpr int kPerSm = kEpl <= 2 ? 6 : kEpl == 4 ? 5 : kEpl == 8 ? (kSigmoid ? 3 : 4)
                       : kEpl == 12 ? (kSigmoid ? 2 : 3) : kEpl == 16 ? 2 : 1;
  const int64_t want = (a.N + 256 / kTeam - 1) / (256 / kTeam);
  const int64_t most = kPerSm * (int64_t)sms;
  // Many experts and tokens for all SMs: the same threads in one or two blocks on an SM, which read
  // the counts and add up their sums once (16384 tokens of 384 experts: 19.0 us, 20.2 us in blocks
  // of 256).
  if constexpr (kEpl >= 8 && kEpl <= 16)
    if (want > most) {
      constexpr int kBlocks = kPerSm == 4 ? 2 : 1;
      return launch_blocks<kTeam, kEpl, kVec, kSigmoid, 256 * kPerSm / kBlocks>(a, kBlocks * sms,
                                                                                stream);
    }
  return launch_blocks<kTeam, kEpl, kVec, kSigmoid, 256>(
      a, want < 1 ? 1 : want < most ? want : most, stream);
}

template <int kTeam, int kEpl, bool kVec>
cudaError_t launch_rows(const LossArgs& a, bool sigmoid, int sms, cudaStream_t stream) {
  return sigmoid ? launch_teams<kTeam, kEpl, kVec, true>(a, sms, stream)
                 : launch_teams<kTeam, kEpl, kVec, false>(a, sms, stream);
}

// More than 64 experts: 16 bytes at a time where rows start on 16 bytes.
template <int kEpl>
cudaError_t launch_wide(const LossArgs& a, bool sigmoid, int sms, cudaStream_t stream) {
  const auto off = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits);
  return a.E % 4 == 0 && off % 16 == 0 ? launch_rows<32, kEpl, true>(a, sigmoid, sms, stream)
                                       : launch_rows<32, kEpl, false>(a, sigmoid, sms, stream);
}

}  // namespace

size_t balance_loss_scratch_bytes(int E) {
  return (size_t)E * (8 + 4 * kMaxCounts) + 4 * kMaxCounts + 8;
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask,
                                int64_t N, int E, int k, int score_fn, float alpha,
                                const float* grad_loss, float* loss, int32_t* counts, float* P,
                                float* dlogits, int accumulate, void* scratch, int* status,
                                cudaStream_t stream, int* launches) {
  const bool rows = loss != nullptr || P != nullptr || dlogits != nullptr;
  int64_t n = rows ? (N * k + kCountIds - 1) / kCountIds : 1;
  n = n < 1 ? 1 : n < kMaxCounts ? n : kMaxCounts;
  const LossScratch s = scratch_of(scratch, E, (int)n);
  cudaError_t e = launch_pdl(balance_count_kernel, (unsigned)n * kCountCtas, kCountThreads,
                             sizeof(int32_t) * (E + 1), stream, ids, mask, N, E, k,
                             n == 1 ? counts : nullptr, s, status);
  ++*launches;
  if (e != cudaSuccess) return e;
  if (!rows) return cudaSuccess;
  LossArgs a{logits, mask, N, E, alpha, grad_loss, loss, n == 1 ? nullptr : counts, P, dlogits,
             accumulate, loss != nullptr || P != nullptr, k, 0.f, s};
  a.fixed_scale = 1.f;
  for (int64_t v = N; v < (int64_t)1 << 61; v = (v < 1 ? 1 : v) * 2) a.fixed_scale *= 2.f;
  ++*launches;
  const int sms = tc::num_sms();
  const bool sg = score_fn == 1;
  if (E <= 8) return launch_rows<8, 1, false>(a, sg, sms, stream);
  if (E <= 16) return launch_rows<16, 1, false>(a, sg, sms, stream);
  if (E <= 32) return launch_rows<32, 1, false>(a, sg, sms, stream);
  if (E <= 64) return launch_rows<32, 2, false>(a, sg, sms, stream);
  if (E <= 128) return launch_wide<4>(a, sg, sms, stream);
  if (E <= 256) return launch_wide<8>(a, sg, sms, stream);
  if (E <= 384) return launch_wide<12>(a, sg, sms, stream);
  if (E <= 512) return launch_wide<16>(a, sg, sms, stream);
  return launch_wide<32>(a, sg, sms, stream);
}

}  // namespace moe
