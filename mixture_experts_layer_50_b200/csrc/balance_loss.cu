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
// Two launches.  A cluster of kCountCtas blocks counts the assignments (integers; the blocks'
// counts meet over distributed shared memory) and clears the accumulators of the second launch,
// so nothing has to be zero before the call.  Then every token's row is read once: its
// probabilities give its gradient row, and add to P.  P is added up in 64-bit fixed point,
// which makes its value independent of the order of the atomic additions; the last block to
// finish turns the sums into P and the loss.
//
// Bound: one read of the logits and one write of the gradient.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kCountCtas = 8;
constexpr int kCountThreads = 512;
constexpr int kLossThreads = 256;

// Scratch of one call (device): sums [E] u64, f0 [E], f [E], then T and the ticket.
struct LossScratch {
  unsigned long long* sums;
  float* f0;
  float* f;
  int32_t* n_tokens;
  unsigned* ticket;
};
LossScratch scratch_of(void* p, int E) {
  LossScratch s;
  s.sums = static_cast<unsigned long long*>(p);
  s.f0 = reinterpret_cast<float*>(s.sums + E);
  s.f = s.f0 + E;
  s.n_tokens = reinterpret_cast<int32_t*>(s.f + E);
  s.ticket = reinterpret_cast<unsigned*>(s.n_tokens + 1);
  return s;
}

__global__ void __cluster_dims__(kCountCtas, 1, 1) __launch_bounds__(kCountThreads)
    balance_count_kernel(const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
                         int64_t N, int E, int k, int32_t* __restrict__ counts, LossScratch out,
                         int* status) {
  pdl_wait();
  extern __shared__ int32_t s_count[];  // [E], then the block's tokens
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  for (int i = threadIdx.x; i <= E; i += kCountThreads) s_count[i] = 0;
  __syncthreads();
  bool bad = false;
  // N * k is below 2^30 (checked on the host), so are all indices
  const uint32_t stride = kCountCtas * kCountThreads, nk = (uint32_t)(N * k);
  for (uint32_t i = rank * kCountThreads + threadIdx.x; i < nk; i += stride) {
    if (mask != nullptr && mask[i / (uint32_t)k] == 0) continue;
    const int e = ids[i];
    if (e >= 0 && e < E)
      atomicAdd(&s_count[e], 1);
    else
      bad = true;
  }
  if (mask != nullptr) {
    int n = 0;
    for (uint32_t t = rank * kCountThreads + threadIdx.x; t < (uint32_t)N; t += stride)
      n += mask[t] != 0;
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if ((threadIdx.x & 31) == 0 && n != 0) atomicAdd(&s_count[E], n);
  }
  if (bad) report_status(status, kStatusInvalidInput);
  cluster.sync();
  int64_t tokens = N;
  if (mask != nullptr) {
    tokens = 0;
    for (int b = 0; b < kCountCtas; ++b) tokens += cluster.map_shared_rank(s_count, b)[E];
  }
  const double per = 1.0 / ((double)(tokens > 0 ? tokens : 1) * k);
  for (int e = rank * kCountThreads + threadIdx.x; e < E; e += kCountCtas * kCountThreads) {
    int c = 0;
    for (int b = 0; b < kCountCtas; ++b) c += cluster.map_shared_rank(s_count, b)[e];
    if (counts != nullptr) counts[e] = c;
    out.f[e] = (float)(c * per);
    out.f0[e] = (float)(c * per - 1.0 / E);
    out.sums[e] = 0;
  }
  if (rank == 0 && threadIdx.x == 0) {
    *out.n_tokens = (int32_t)tokens;
    *out.ticket = 0;
  }
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
  float* P;
  float* dlogits;
  int accumulate;
  int want_sums;
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

// kTeam lanes own a token; lane i of the team holds experts i, i + kTeam, ...: kEpl of them.
template <int kTeam, int kEpl, bool kSigmoid>
__global__ void __launch_bounds__(kLossThreads) balance_loss_kernel(const LossArgs a) {
  constexpr int kTeams = kLossThreads / kTeam;
  pdl_wait();
  extern __shared__ float s_p[];  // [kTeams][E]
  const int E = a.E;
  const int ti = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
  const int T = *a.s.n_tokens;
  const float g = (a.grad_loss != nullptr ? *a.grad_loss : 1.f) * a.alpha * (float)E /
                  (float)(T > 0 ? T : 1);
  float f0[kEpl], acc[kEpl];
#pragma unroll
  for (int j = 0; j < kEpl; ++j) {
    const int e = ti + j * kTeam;
    f0[j] = e < E ? a.s.f0[e] : 0.f;
    acc[j] = 0.f;
  }
  // every team of the block takes the same number of steps: the shuffles need whole warps
  for (int64_t t0 = (int64_t)blockIdx.x * kTeams; t0 < a.N; t0 += (int64_t)gridDim.x * kTeams) {
    const int64_t t = t0 + team;
    const bool live = t < a.N && (a.mask == nullptr || a.mask[t] != 0);
    const float* z = a.logits + t * E;
    float p[kEpl], u[kEpl];
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
      const int e = ti + j * kTeam;
      p[j] = live && e < E ? z[e] : -INFINITY;
    }
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
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
      p[j] *= inv;
      acc[j] += p[j];
      dot = fmaf(p[j], f0[j], dot);
    }
    dot = team_sum<kTeam>(dot);
    if (a.dlogits != nullptr && t < a.N) {
      float* dz = a.dlogits + t * E;
#pragma unroll
      for (int j = 0; j < kEpl; ++j) {
        const int e = ti + j * kTeam;
        if (e >= E) continue;
        float v = live ? g * (p[j] * (f0[j] - dot)) : 0.f;
        if (kSigmoid && live) v *= u[j];
        if (!a.accumulate)
          dz[e] = v;
        else if (live)
          dz[e] += v;
      }
    }
  }
  if (!a.want_sums) return;
#pragma unroll
  for (int j = 0; j < kEpl; ++j) {
    const int e = ti + j * kTeam;
    if (e < E) s_p[team * E + e] = acc[j];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kLossThreads) {
    float v = 0.f;
    for (int i = 0; i < kTeams; ++i) v += s_p[i * E + e];
    // sums stay below 2^62: the top bit is free to stand for a NaN
    if (v != v)
      atomicOr(&a.s.sums[e], 1ull << 63);
    else if (v != 0.f)
      atomicAdd(&a.s.sums[e], (unsigned long long)((double)v * (double)a.fixed_scale));
  }
  __shared__ bool s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(a.s.ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double part = 0.0;
  for (int e = threadIdx.x; e < E; e += kLossThreads) {
    const unsigned long long v = __ldcg(&a.s.sums[e]);
    const double Pe = (v >> 63) ? (double)NAN
                                : (double)v / ((double)a.fixed_scale * (T > 0 ? T : 1));
    if (a.P != nullptr) a.P[e] = (float)Pe;
    part += (double)a.s.f[e] * Pe;
  }
  __shared__ double s_sum[kLossThreads];
  s_sum[threadIdx.x] = part;
  for (int w = kLossThreads / 2; w > 0; w >>= 1) {
    __syncthreads();
    if (threadIdx.x < w) s_sum[threadIdx.x] += s_sum[threadIdx.x + w];
  }
  if (threadIdx.x == 0 && a.loss != nullptr)
    a.loss[0] = (float)((double)a.alpha * E * s_sum[0]);
}

template <int kTeam, int kEpl>
cudaError_t launch_rows(const LossArgs& a, bool sigmoid, int sms, cudaStream_t stream) {
  constexpr int kTeams = kLossThreads / kTeam;
  const size_t smem = a.want_sums ? sizeof(float) * kTeams * a.E : 0;
  const int64_t want = (a.N + kTeams - 1) / kTeams;
  const int grid = (int)(want < 1 ? 1 : want < 4 * sms ? want : 4 * sms);
  return sigmoid ? launch_pdl(balance_loss_kernel<kTeam, kEpl, true>, grid, kLossThreads, smem,
                              stream, a)
                 : launch_pdl(balance_loss_kernel<kTeam, kEpl, false>, grid, kLossThreads, smem,
                              stream, a);
}

}  // namespace

size_t balance_loss_scratch_bytes(int E) { return (size_t)E * 16 + 8; }

cudaError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask,
                                int64_t N, int E, int k, int score_fn, float alpha,
                                const float* grad_loss, float* loss, int32_t* counts, float* P,
                                float* dlogits, int accumulate, void* scratch, int* status,
                                cudaStream_t stream, int* launches) {
  const LossScratch s = scratch_of(scratch, E);
  cudaError_t e = launch_pdl(balance_count_kernel, kCountCtas, kCountThreads,
                             sizeof(int32_t) * (E + 1), stream, ids, mask, N, E, k, counts, s,
                             status);
  ++*launches;
  if (e != cudaSuccess) return e;
  if (loss == nullptr && P == nullptr && dlogits == nullptr) return cudaSuccess;
  LossArgs a{logits, mask, N, E, alpha, grad_loss, loss, P, dlogits, accumulate,
             loss != nullptr || P != nullptr, 0.f, s};
  a.fixed_scale = 1.f;
  for (int64_t v = N; v < (int64_t)1 << 61; v = (v < 1 ? 1 : v) * 2) a.fixed_scale *= 2.f;
  ++*launches;
  const int sms = tc::num_sms();
  const bool sg = score_fn == 1;
  if (E <= 8) return launch_rows<8, 1>(a, sg, sms, stream);
  if (E <= 16) return launch_rows<16, 1>(a, sg, sms, stream);
  if (E <= 32) return launch_rows<32, 1>(a, sg, sms, stream);
  if (E <= 64) return launch_rows<32, 2>(a, sg, sms, stream);
  if (E <= 128) return launch_rows<32, 4>(a, sg, sms, stream);
  if (E <= 256) return launch_rows<32, 8>(a, sg, sms, stream);
  if (E <= 384) return launch_rows<32, 12>(a, sg, sms, stream);
  if (E <= 512) return launch_rows<32, 16>(a, sg, sms, stream);
  return launch_rows<32, 32>(a, sg, sms, stream);
}

}  // namespace moe
