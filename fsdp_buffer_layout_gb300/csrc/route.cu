// route.cu — the mixture-of-experts router: scores, top-k choice, gates,
// per-expert counts and the balance loss, and the gradient of its logits.
//
// With s the scores (softmax or sigmoid of the logits x), q = s / Z their
// share, C the chosen experts, D = sum_C s + 1e-20 and dg the gates' gradient:
//   gates:   d s_e  = route_scale (dg_e - sum_C dg s / D) / D   (e in C, renorm)
//                   = route_scale dg_e                          (e in C, else)
//   balance: d s_e += b_e                                        softmax (Z = 1)
//                  += (b_e - sum_j b_j q_j) / Z                  sigmoid
//            with b_e = loss_scale coef_s n_se, the counts taken as constants;
//   logits:  d x_e  = s_e (d s_e - sum_j s_j d s_j)              softmax
//                   = s_e (1 - s_e) d s_e                        sigmoid
//
// A warp takes a token; lane l holds experts l, l + 32, ... in registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "objective.cuh"

namespace vsf {
namespace {

using namespace obj;

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kMaxTopK = 32;
constexpr int64_t kMaxExperts = 512;
// Sums of shares are kept in fixed point, 2^-40 a unit: integer additions
// give the same sum in any order. A share is at most 1, so 2^23 tokens fit.
constexpr double kShareUnit = 1099511627776.0;

struct RouteIn {
  int64_t T_, ld, sequences;
  int32_t E, K, score, renorm;
  float scale, balance;
  const float* bias;
  const uint8_t* live;
  const int64_t* starts;  // NULL: one sequence of T_ tokens
};

// The sequence that holds token t, or -1: the last one that starts at or
// before t. Always below `sequences`, whatever the starts hold.
__device__ __forceinline__ int64_t sequence_of(const RouteIn& p, int64_t t) {
  if (p.starts == nullptr) return 0;
  int64_t lo = 0, hi = p.sequences;  // starts[lo] <= t < starts[hi], if any
  if (t < p.starts[0] || t >= p.starts[p.sequences]) return -1;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (p.starts[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Order-preserving 32-bit key of a float: larger is better, -0 equals +0,
// NaN comes after every number. 0 is below every key.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}

// Scores of a token's experts from its logits, in place; returns Z.
template <int N>
__device__ __forceinline__ float scores(float (&x)[N], int32_t E, int32_t score, int lane) {
  if (score == VSF_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, x[j]);
    m = warp_max(m);
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      x[j] = lane + 32 * j < E ? expf(x[j] - m) : 0.f;
      z += x[j];
    }
    z = warp_sum(z);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = x[j] / z;
    return 1.f;
  }
  float z = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    x[j] = lane + 32 * j < E ? 1.f / (1.f + expf(-x[j])) : 0.f;
    z += x[j];
  }
  return warp_sum(z) + 1e-20f;
}

template <typename T, int N>
__device__ __forceinline__ void load_token(float (&x)[N], const T* row, int32_t E, int lane) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = lane + 32 * j;
    x[j] = e < E ? to_f(row[e]) : -INFINITY;
  }
}

template <typename T, int N>
__global__ void __launch_bounds__(kRouteThreads)
    route_kernel(const T* logits, RouteIn p, int32_t* idx, float* gates, int32_t* seq_counts,
                 unsigned long long* seq_share, int32_t* seq_tokens, WsHead* head) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kRouteWarps;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5); t < p.T_; t += warps) {
    if (p.live != nullptr && p.live[t] == 0) {
      for (int k = lane; k < p.K; k += 32) {
        idx[t * p.K + k] = -1;
        gates[t * p.K + k] = 0.f;
      }
      continue;
    }
    float x[N];
    uint32_t key[N];
    load_token(x, logits + t * p.ld, p.E, lane);
    if (p.bias == nullptr) {
#pragma unroll
      for (int j = 0; j < N; ++j) key[j] = order_key(x[j]);
    }
    const float z = scores(x, p.E, p.score, lane);
    if (p.bias != nullptr) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (lane + 32 * j < p.E) key[j] = order_key(x[j] + p.bias[lane + 32 * j]);
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (lane + 32 * j >= p.E) key[j] = 0u;
    const int64_t seq = sequence_of(p, t);
    float mine = 0.f, sum = 0.f;  // lane k keeps choice k's score
    int chosen = -1;
    for (int k = 0; k < p.K; ++k) {
      uint32_t best = 0;
      int be = INT32_MAX;
      float bs = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (key[j] > best) {
          best = key[j];
          be = lane + 32 * j;
          bs = x[j];
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint32_t ok = __shfl_xor_sync(~0u, best, o);
        const int oe = __shfl_xor_sync(~0u, be, o);
        const float os = __shfl_xor_sync(~0u, bs, o);
        if (ok > best || (ok == best && oe < be)) {
          best = ok;
          be = oe;
          bs = os;
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (lane + 32 * j == be) key[j] = 0u;
      if (lane == k) {
        chosen = be;
        mine = bs;
      }
      sum += bs;
    }
    if (lane < p.K) {
      idx[t * p.K + lane] = chosen;
      gates[t * p.K + lane] = p.renorm ? p.scale * mine / (sum + 1e-20f) : p.scale * mine;
      if (seq >= 0) atomicAdd(&seq_counts[seq * p.E + chosen], 1);
    }
    if (seq >= 0) {
      bool bad = false;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = lane + 32 * j;
        if (e >= p.E) continue;
        const float q = x[j] / z;
        bad |= q != q;
        if (q > 0.f)
          atomicAdd(&seq_share[seq * p.E + e], (unsigned long long)((double)q * kShareUnit + 0.5));
      }
      if (bad) head->nan = 1u;
      if (lane == 0) atomicAdd(&seq_tokens[seq], 1);
    }
  }
}

// Counts over all sequences, the sequences' coefficients and the balance loss.
__global__ void __launch_bounds__(512)
    route_finish_kernel(RouteIn p, const int32_t* seq_counts, const unsigned long long* seq_share,
                        const int32_t* seq_tokens, int32_t* counts, float* seq_coef, float* loss,
                        WsHead* head) {
  __shared__ double part[16];
  __shared__ int full;  // sequences with a live token
  if (threadIdx.x == 0) full = 0;
  __syncthreads();
  int mine = 0;
  for (int64_t s = threadIdx.x; s < p.sequences; s += 512) mine += seq_tokens[s] > 0;
  if (mine) atomicAdd(&full, mine);
  __syncthreads();
  for (int64_t s = threadIdx.x; s < p.sequences; s += 512) {
    const double n = seq_tokens[s];
    seq_coef[s] = n > 0 ? (float)((double)p.balance * p.E / (p.K * n * n * full)) : 0.f;
  }
  double l = 0.0;
  for (int e = threadIdx.x; e < p.E; e += 512) {
    int c = 0;
    for (int64_t s = 0; s < p.sequences; ++s) {
      const int n_se = seq_counts[s * p.E + e];
      c += n_se;
      if (n_se) {
        const double n = seq_tokens[s];
        l += (double)p.balance * p.E / (p.K * n * n * full) * n_se *
             ((double)seq_share[s * p.E + e] / kShareUnit);
      }
    }
    counts[e] = c;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = l;
  __syncthreads();
  if (threadIdx.x == 0) {
    l = 0.0;
    for (int w = 0; w < 16; ++w) l += part[w];
    *loss = head->nan ? NAN : (float)l;
    head->nan = 0u;
  }
}

template <typename T, int N>
__global__ void __launch_bounds__(kRouteThreads)
    route_grad_kernel(const T* logits, RouteIn p, const int32_t* idx, const float* d_gates,
                      const int32_t* seq_counts, const float* seq_coef, float loss_scale, T* grad,
                      int64_t grad_ld) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kRouteWarps;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5); t < p.T_; t += warps) {
    T* g = grad + t * grad_ld;
    if (p.live != nullptr && p.live[t] == 0) {
      for (int e = lane; e < p.E; e += 32) g[e] = from_f<T>(0.f);
      continue;
    }
    float x[N], ds[N];
    load_token(x, logits + t * p.ld, p.E, lane);
    const float z = scores(x, p.E, p.score, lane);
#pragma unroll
    for (int j = 0; j < N; ++j) ds[j] = 0.f;
    if (d_gates != nullptr) {
      const int mine = lane < p.K ? idx[t * p.K + lane] : -1;
      const float dg = lane < p.K ? d_gates[t * p.K + lane] : 0.f;
      float picked = 0.f;  // lane k: the score of choice k
      for (int k = 0; k < p.K; ++k) {
        const int e = __shfl_sync(~0u, mine, k);
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (e >= 0 && (e >> 5) == j) v = x[j];
        v = __shfl_sync(~0u, v, e & 31);
        if (lane == k && e >= 0 && e < p.E) picked = v;
      }
      float pull = dg;
      if (p.renorm) {
        const float down = warp_sum(picked) + 1e-20f;
        const float dot = warp_sum(dg * picked) / down;
        pull = (dg - dot) / down;
      }
      pull *= p.scale;
      for (int k = 0; k < p.K; ++k) {
        const int e = __shfl_sync(~0u, mine, k);
        const float v = __shfl_sync(~0u, pull, k);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (lane + 32 * j == e) ds[j] = v;
      }
    }
    const int64_t seq = sequence_of(p, t);
    if (seq >= 0 && loss_scale != 0.f) {
      const float f = loss_scale * seq_coef[seq];
      float b[N], dot = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = lane + 32 * j;
        b[j] = e < p.E ? f * (float)seq_counts[seq * p.E + e] : 0.f;
        dot += b[j] * x[j];
      }
      if (p.score == VSF_SCORE_SIGMOID) dot = warp_sum(dot) / z;
      else dot = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) ds[j] += (b[j] - dot) / z;
    }
    float dot = 0.f;
    if (p.score == VSF_SCORE_SOFTMAX) {
#pragma unroll
      for (int j = 0; j < N; ++j) dot += x[j] * ds[j];
      dot = warp_sum(dot);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = lane + 32 * j;
      if (e < p.E)
        g[e] = from_f<T>(p.score == VSF_SCORE_SOFTMAX ? x[j] * (ds[j] - dot)
                                                      : x[j] * (1.f - x[j]) * ds[j]);
    }
  }
}

// ------------------------------------------------------------- host side
struct RouteWs {
  WsHead* head;
  int32_t* tokens;             // [sequences] live tokens
  unsigned long long* share;   // [sequences * E] sums of shares
  static size_t tokens_bytes(int64_t sequences) { return (size_t)((sequences * 4 + 15) / 16 * 16); }
  static size_t bytes(int64_t E, int64_t sequences) {
    return sizeof(WsHead) + tokens_bytes(sequences) + (size_t)(E * sequences) * 8;
  }
  RouteWs(void* ws, int64_t sequences) {
    unsigned char* b = static_cast<unsigned char*>(ws);
    head = reinterpret_cast<WsHead*>(b);
    tokens = reinterpret_cast<int32_t*>(b + sizeof(WsHead));
    share = reinterpret_cast<unsigned long long*>(b + sizeof(WsHead) + tokens_bytes(sequences));
  }
};

vsf_status check_route(const char* who, const void* logits, int32_t dtype, int64_t T_, int64_t E,
                       int64_t ld, const int64_t* starts, int64_t sequences,
                       const vsf_route_hparams* hp) {
  const std::string w(who);
  if (hp == nullptr || (T_ > 0 && logits == nullptr)) return fail(VSF_ERR_ARG, w + ": NULL pointer");
  if (dtype != VSF_BF16 && dtype != VSF_FP32) return fail(VSF_ERR_ARG, w + ": bad dtype");
  if (T_ < 0 || T_ > (1 << 23) || E < 1 || E > kMaxExperts || ld < E || ld > (int64_t(1) << 40) ||
      sequences < 1 || sequences > (1 << 20) || (starts == nullptr && sequences != 1))
    return fail(VSF_ERR_ARG, w + ": sizes out of range");
  if (hp->top_k < 1 || hp->top_k > std::min<int64_t>(E, kMaxTopK) ||
      (hp->score != VSF_SCORE_SOFTMAX && hp->score != VSF_SCORE_SIGMOID) ||
      !std::isfinite(hp->route_scale) || !std::isfinite(hp->balance))
    return fail(VSF_ERR_ARG, w + ": hyper-parameters out of range");
  if (!aligned(logits, dtype == VSF_BF16 ? 2 : 4) || !aligned(starts, 8))
    return fail(VSF_ERR_ALIGN, w + ": pointer alignment");
  return VSF_OK;
}

RouteIn route_in(int64_t T_, int64_t E, int64_t ld, const float* bias, const uint8_t* live,
                 const int64_t* starts, int64_t sequences, const vsf_route_hparams* hp) {
  return {T_, ld, sequences, (int32_t)E, hp->top_k, hp->score, hp->renorm != 0,
          hp->route_scale, hp->balance, bias, live, starts};
}

unsigned route_grid(int64_t T_) {
  return (unsigned)std::min<int64_t>((T_ + kRouteWarps - 1) / kRouteWarps, 152 * 8);
}

template <typename T, int N>
void route_launch(const void* logits, const RouteIn& p, int32_t* idx, float* gates,
                  int32_t* seq_counts, const RouteWs& w, cudaStream_t st) {
  route_kernel<T, N><<<route_grid(p.T_), kRouteThreads, 0, st>>>(
      static_cast<const T*>(logits), p, idx, gates, seq_counts, w.share, w.tokens, w.head);
}

template <typename T, int N>
void grad_launch(const void* logits, const RouteIn& p, const int32_t* idx, const float* d_gates,
                 const int32_t* seq_counts, const float* seq_coef, float loss_scale, void* grad,
                 int64_t grad_ld, cudaStream_t st) {
  route_grad_kernel<T, N><<<route_grid(p.T_), kRouteThreads, 0, st>>>(
      static_cast<const T*>(logits), p, idx, d_gates, seq_counts, seq_coef, loss_scale,
      static_cast<T*>(grad), grad_ld);
}

// Calls f<N> for the registers a lane needs to hold its share of E experts.
#define VSF_BY_EXPERTS(E, F, ...)                    \
  do {                                               \
    if ((E) <= 32) F<T, 1>(__VA_ARGS__);             \
    else if ((E) <= 64) F<T, 2>(__VA_ARGS__);        \
    else if ((E) <= 128) F<T, 4>(__VA_ARGS__);       \
    else if ((E) <= 256) F<T, 8>(__VA_ARGS__);       \
    else F<T, 16>(__VA_ARGS__);                      \
  } while (0)

template <typename T>
void route_by_experts(const void* logits, const RouteIn& p, int32_t* idx, float* gates,
                      int32_t* seq_counts, const RouteWs& w, cudaStream_t st) {
  VSF_BY_EXPERTS(p.E, route_launch, logits, p, idx, gates, seq_counts, w, st);
}

template <typename T>
void grad_by_experts(const void* logits, const RouteIn& p, const int32_t* idx,
                     const float* d_gates, const int32_t* seq_counts, const float* seq_coef,
                     float loss_scale, void* grad, int64_t grad_ld, cudaStream_t st) {
  VSF_BY_EXPERTS(p.E, grad_launch, logits, p, idx, d_gates, seq_counts, seq_coef, loss_scale,
                 grad, grad_ld, st);
}

}  // namespace
}  // namespace vsf

using namespace vsf;

extern "C" {

size_t vsf_route_workspace_bytes(int64_t experts, int64_t sequences) {
  if (experts < 1 || experts > kMaxExperts || sequences < 1 || sequences > (1 << 20)) return 0;
  return RouteWs::bytes(experts, sequences);
}

vsf_status vsf_route(const void* logits, int32_t dtype, int64_t T, int64_t E, int64_t ld,
                     const float* bias, const uint8_t* live, const int64_t* seq_starts,
                     int64_t sequences, const vsf_route_hparams* hp, int32_t* idx, float* gates,
                     int32_t* counts, float* loss, int32_t* seq_counts, float* seq_coef,
                     void* d_workspace, size_t ws_bytes, void* stream) {
  vsf::Range nvtx_range("vsf_route");
  const char* who = "vsf_route";
  vsf_status s = check_route(who, logits, dtype, T, E, ld, seq_starts, sequences, hp);
  if (s != VSF_OK) return s;
  if ((T > 0 && (idx == nullptr || gates == nullptr)) || counts == nullptr || loss == nullptr ||
      seq_counts == nullptr || seq_coef == nullptr || d_workspace == nullptr)
    return fail(VSF_ERR_ARG, "vsf_route: NULL pointer");
  if (ws_bytes < RouteWs::bytes(E, sequences))
    return fail(VSF_ERR_ARG, "vsf_route: workspace too small");
  if (!aligned(d_workspace, 16) || !aligned(bias, 4) || !aligned(idx, 4) || !aligned(gates, 4) ||
      !aligned(counts, 4) || !aligned(loss, 4) || !aligned(seq_counts, 4) || !aligned(seq_coef, 4))
    return fail(VSF_ERR_ALIGN, "vsf_route: pointer alignment");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const RouteWs w(d_workspace, sequences);
  const RouteIn p = route_in(T, E, ld, bias, live, seq_starts, sequences, hp);
  cudaError_t e = cudaMemsetAsync(w.tokens, 0, RouteWs::bytes(E, sequences) - sizeof(WsHead), st);
  if (e == cudaSuccess) e = cudaMemsetAsync(seq_counts, 0, (size_t)(sequences * E) * 4, st);
  if (e != cudaSuccess) return cuda_error(e, who);
  if (T > 0) {
    if (dtype == VSF_BF16) route_by_experts<uint16_t>(logits, p, idx, gates, seq_counts, w, st);
    else route_by_experts<float>(logits, p, idx, gates, seq_counts, w, st);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, who);
  }
  route_finish_kernel<<<1, 512, 0, st>>>(p, seq_counts, w.share, w.tokens, counts, seq_coef, loss,
                                         w.head);
  e = cudaGetLastError();
  return e == cudaSuccess ? VSF_OK : cuda_error(e, who);
}

vsf_status vsf_route_grad(const void* logits, int32_t dtype, int64_t T, int64_t E, int64_t ld,
                          const uint8_t* live, const int64_t* seq_starts, int64_t sequences,
                          const vsf_route_hparams* hp, const int32_t* idx, const float* d_gates,
                          const int32_t* seq_counts, const float* seq_coef, float loss_scale,
                          void* grad, int64_t grad_ld, void* stream) {
  vsf::Range nvtx_range("vsf_route_grad");
  const char* who = "vsf_route_grad";
  vsf_status s = check_route(who, logits, dtype, T, E, ld, seq_starts, sequences, hp);
  if (s != VSF_OK) return s;
  if (seq_counts == nullptr || seq_coef == nullptr || (T > 0 && (idx == nullptr || grad == nullptr)))
    return fail(VSF_ERR_ARG, "vsf_route_grad: NULL pointer");
  if (grad_ld < E || grad_ld > (int64_t(1) << 40) || !std::isfinite(loss_scale))
    return fail(VSF_ERR_ARG, "vsf_route_grad: grad_ld or loss_scale out of range");
  const int64_t size = dtype == VSF_BF16 ? 2 : 4;
  if (!aligned(idx, 4) || !aligned(d_gates, 4) || !aligned(seq_counts, 4) ||
      !aligned(seq_coef, 4) || !aligned(grad, size))
    return fail(VSF_ERR_ALIGN, "vsf_route_grad: pointer alignment");
  if (T == 0) return VSF_OK;
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(logits), g0 = reinterpret_cast<uintptr_t>(grad);
  if (x0 < g0 + ((T - 1) * grad_ld + E) * size && g0 < x0 + ((T - 1) * ld + E) * size &&
      !(x0 == g0 && ld == grad_ld))
    return fail(VSF_ERR_ARG, "vsf_route_grad: grad overlaps the logits in part");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const RouteIn p = route_in(T, E, ld, nullptr, live, seq_starts, sequences, hp);
  if (dtype == VSF_BF16)
    grad_by_experts<uint16_t>(logits, p, idx, d_gates, seq_counts, seq_coef, loss_scale, grad,
                              grad_ld, st);
  else
    grad_by_experts<float>(logits, p, idx, d_gates, seq_counts, seq_coef, loss_scale, grad,
                           grad_ld, st);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VSF_OK : cuda_error(e, who);
}

}  // extern "C"
