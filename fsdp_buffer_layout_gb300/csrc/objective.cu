// objective.cu — losses over a model's logits and their gradients: token log
// probabilities, the clipped policy loss with a KL term, and the preference
// loss of pairs.
//
// All three rest on one row operation. For a row x of logits with maximum m,
//   s = sum_v exp((x_v - m) / temperature),
//   ln p(y) = (x_y - m) / temperature - ln s,
//   d loss / d x_v = a (1[v = y] - exp((x_v - m) / temperature) / s),
// where a = d loss / d ln p(y) / temperature depends on the token alone
// (policy) or on its pair of sequences (preference).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "objective.cuh"

namespace vsf {
namespace {

using namespace obj;

constexpr int kTokenThreads = 512;

constexpr int kMaxPipeClusters = 1024;  // clusters whose sums the workspace holds

// Workspace: the head, the pipelined kernel's sums per cluster, then per token
// {m, s, x_y} and the gradient's coefficient, then per pair the loss and the margin.
struct ObjectiveWs {
  static constexpr size_t kFront = sizeof(WsHead) + (3 * (size_t)kMaxPipeClusters + 2) * 8;
  WsHead* head;
  double* partial;  // [3 * kMaxPipeClusters] sums of clusters or CTAs
  double* total;    // sum of the live weights, where a launch of its own adds it up
  float4* row;    // [tokens] maximum, sum and target's logit of a live row
  float* coef;    // [tokens] a of a token; 0: no gradient
  float2* pair;   // [pairs] loss and beta h
  static size_t bytes(int64_t tokens, int64_t pairs) {
    return kFront + (size_t)((tokens * 20 + 15) / 16 * 16) + (size_t)pairs * 8;
  }
  ObjectiveWs(void* ws, int64_t tokens) {
    unsigned char* p = static_cast<unsigned char*>(ws);
    head = reinterpret_cast<WsHead*>(p);
    partial = reinterpret_cast<double*>(p + sizeof(WsHead));
    total = partial + 3 * kMaxPipeClusters;
    row = reinterpret_cast<float4*>(p + kFront);
    coef = reinterpret_cast<float*>(row + tokens);
    pair = reinterpret_cast<float2*>(p + kFront + (tokens * 20 + 15) / 16 * 16);
  }
};

// Rows of logits and their targets.
template <typename T>
struct Rows {
  const T* x;
  int64_t ld;
  int64_t T_;
  int32_t V;
  const int64_t* target;
  const float* weight;  // NULL: 1
  Log2Scale c;
  float inv_tf;
  double inv_t;
};

struct Token {
  int64_t y;
  float w;
};
template <typename T>
__device__ __forceinline__ Token token_at(const Rows<T>& r, int64_t t) {
  if (t >= r.T_) return {-1, 0.f};
  return {r.target[t], r.weight != nullptr ? r.weight[t] : 1.f};
}

// The target of a live token, or -1.
template <typename T>
__device__ __forceinline__ int32_t live_target(const Rows<T>& r, Token k, uint32_t* err) {
  if (k.y < 0 || k.w == 0.f) return -1;
  if (k.y >= r.V) {
    if (err != nullptr) atomicOr(err, kErrTarget);
    return -1;
  }
  return (int32_t)k.y;
}
template <typename T>
__device__ __forceinline__ int32_t live_target(const Rows<T>& r, int64_t t, uint32_t* err) {
  return live_target(r, token_at(r, t), err);
}

// ln s = k ln 2 + f, with |f| at most 0.41, where logf's absolute error is
// below 3e-8 (logf(s) itself would round at 5e-7 for s in the thousands). The
// mean relative error of s itself, which would add up over a sequence, was
// measured at -0.4e-8 (32000 words) to -1.7e-8 (logits of five times the spread).
struct LogSum {
  float k, f;
};
__device__ __forceinline__ LogSum log_sum(float s) {
  float k = 0.f, f = s;
  if (s >= 1.1754944e-38f && s < INFINITY) {
    const uint32_t b = __float_as_uint(s);
    const uint32_t e = (b + 0x00400000u) >> 23;  // f in [0.75, 1.5)
    k = (float)((int)e - 127);
    f = __uint_as_float(b - ((e - 127u) << 23));
  }
  return {k, logf(f)};
}

// ln p(y) - ref in fp32, with d = x_y - m: the large parts cancel first. ln 2 =
// 355/512 - 2.12194440e-4 (the split of Cody and Waite): k times the first is
// exact.
__device__ __forceinline__ float log_ratio(float d, float inv_t, float ref, LogSum s) {
  const float a = __fmaf_rn(d, inv_t, -ref);
  return __fmaf_rn(-s.k, 0.693359375f, a) - __fmaf_rn(s.k, -2.12194440e-4f, s.f);
}
// The same to about fp32's last bit of the difference itself, for sums over a
// sequence: the rounding errors of the product and the two large differences
// are kept and added (Dekker's and Knuth's exact transformations).
__device__ __forceinline__ float exact_log_ratio(float d, float inv_t, float ref, LogSum s) {
  const float p = __fmul_rn(d, inv_t), ep = __fmaf_rn(d, inv_t, -p);
  auto minus = [](float a, float b, float& err) {  // a - b, and what rounding took off
    const float v = __fsub_rn(a, b), t = __fsub_rn(v, a);
    err = __fsub_rn(__fsub_rn(a, __fsub_rn(v, t)), __fadd_rn(b, t));
    return v;
  };
  float e1, e2;
  const float a = minus(p, ref, e1);
  const float c = minus(a, __fmul_rn(s.k, 0.693359375f), e2);
  const float low = __fadd_rn(__fadd_rn(ep, e1), e2);
  // an infinite or NaN difference has no error worth keeping
  return __fsub_rn(c, __fmaf_rn(s.k, -2.12194440e-4f, s.f)) + (low - low == 0.f ? low : 0.f);
}
// ln p(y) in fp64.
__device__ __forceinline__ double log_prob(float d, float s, double inv_t) {
  const LogSum l = log_sum(s);
  return (double)d * inv_t - ((double)l.k * 0.69314718055994530942 + (double)l.f);
}

struct MaxSum {
  float m, s;
};

// Joins by expf, whose mean error is a tenth of ex2's: a term passes several
// joins on its way to the row's sum.
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float inv_t) {
  const float m = fmaxf(a.m, b.m), z = finite_max(m);
  return {m, a.s * expf((a.m - z) * inv_t) + b.s * expf((b.m - z) * inv_t)};
}

struct PolicyIn {
  const float *old_logp, *ref_logp, *adv;
  float lo, hi, beta, scale;  // the ratio's clip bounds; loss factors
  int mean;
};

// One token's policy and KL terms and d(policy + beta kl)/d logp, from
// logp - old, u = ref - logp and its advantage.
struct PolicyTerm {
  float policy, kl, slope;
};

__device__ __forceinline__ PolicyTerm policy_term(const PolicyIn& p, float ahead, float u, float a) {
  PolicyTerm o;
  const float ratio = expf(ahead);
  // (past fp32 above 88: 0 times a ratio that is finite in truth is 0)
  const float freed = a == 0.f && ahead < INFINITY ? 0.f : ratio * a;
  const float held = fminf(fmaxf(ratio, p.lo), p.hi) * a;
  const bool clipped = freed > held;  // a NaN ratio is not clipped away
  o.policy = -(clipped ? held : freed);
  o.slope = clipped ? 0.f : -freed;
  o.kl = 0.f;
  if (p.beta != 0.f) {
    const float e = expm1f(u);
    // exp(u) - 1 - u; near 0 by its series, whose first terms do not cancel
    o.kl = fabsf(u) < 0.25f
               ? u * u * (0.5f + u * (1.f / 6 + u * (1.f / 24 + u * (1.f / 120 + u * (1.f / 720 + u * (1.f / 5040))))))
               : e - u;
    o.slope -= p.beta * e;
  }
  return o;
}

__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) v += part[w];
  return v;
}

// Policy loss of every token in one CTA, and the gradient's coefficients.
template <typename T>
__global__ void __launch_bounds__(kTokenThreads)
    policy_tokens_kernel(Rows<T> r, PolicyIn p, const float4* row, float* coef, float* stats,
                         WsHead* head) {
  __shared__ double part[kTokenThreads / 32];
  take_turn();
  double n = 0.0;
  for (int64_t t = threadIdx.x; t < r.T_; t += kTokenThreads)
    if (live_target(r, t, nullptr) >= 0) n += r.weight != nullptr ? (double)r.weight[t] : 1.0;
  n = block_sum(n, part);
  const double f = (double)p.scale / (p.mean && n != 0.0 ? n : 1.0);
  double pol = 0.0, kl = 0.0;
  for (int64_t t = threadIdx.x; t < r.T_; t += kTokenThreads) {
    if (live_target(r, t, nullptr) < 0) {
      coef[t] = 0.f;
      continue;
    }
    const double w = r.weight != nullptr ? (double)r.weight[t] : 1.0;
    const float4 ms = row[t];
    const double lp = log_prob(ms.z - ms.x, ms.y, r.inv_t);
    const PolicyTerm o =
        policy_term(p, (float)(lp - (double)p.old_logp[t]),
                    p.beta != 0.f ? (float)((double)p.ref_logp[t] - lp) : 0.f, p.adv[t]);
    pol += w * (double)o.policy;
    kl += w * (double)o.kl;
    coef[t] = (float)(f * w * r.inv_t * (double)o.slope);
  }
  pol = block_sum(pol, part) * f;
  kl = block_sum(kl, part) * f;
  if (threadIdx.x == 0) {
    stats[0] = (float)(pol + (p.beta != 0.f ? (double)p.beta * kl : 0.0));
    stats[1] = (float)pol;
    stats[2] = (float)kl;
    stats[3] = (float)n;
    head->rows = 1;
  }
}

struct PairIn {
  const float* ref_logp;
  const int64_t* starts;
  float* rewards;
  int64_t pairs;
  float beta, smoothing, margin, scale;
  int kind, average;
};

__device__ __forceinline__ int64_t clamp_start(int64_t v, int64_t T_) {
  return v < 0 ? 0 : v > T_ ? T_ : v;
}

// One pair a CTA: both log ratios, the loss, and its tokens' coefficients; the
// last CTA to finish adds up the pairs, in their order. Tokens in front of the
// first sequence and behind the last one get the coefficient 0. All in fp32 but
// the sum over pairs: fp64 runs at a 64th of the rate here, and a version in
// fp64 took 40 us for two pairs.
constexpr int kPairThreads = 512;  // half of them a sequence

template <typename T>
__global__ void __launch_bounds__(kPairThreads)
    pair_kernel(Rows<T> r, PairIn p, const float4* row, float* coef, float2* pair, float* stats,
                WsHead* head) {
  constexpr int kSide = kPairThreads / 2;
  __shared__ float2 part[kPairThreads / 32];
  __shared__ bool last;
  // (the gradient's CTAs set up while rows are still summed ended up unevenly
  // on the SMs: 291 us instead of 262 for 16 pairs of 384 x 32000)
  take_turn(false);
  const int64_t q = blockIdx.x;
  const int side = threadIdx.x / kSide, tid = threadIdx.x & (kSide - 1);
  const int64_t first = clamp_start(p.starts[side * p.pairs + q], r.T_);
  const int64_t end = clamp_start(p.starts[side * p.pairs + q + 1], r.T_);
  float d = 0.f, n = 0.f;
  for (int64_t t = first + tid; t < end; t += kSide) {
    const Token k = token_at(r, t);
    const float4 ms = row[t];
    const float ref = p.ref_logp != nullptr ? p.ref_logp[t] : 0.f;
    if (live_target(r, k, nullptr) < 0) continue;
    d += k.w * exact_log_ratio(ms.z - ms.x, r.inv_tf, ref, log_sum(ms.y));
    n += k.w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    d += __shfl_xor_sync(~0u, d, o);
    n += __shfl_xor_sync(~0u, n, o);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(d, n);
  __syncthreads();
  float ratio[2], length[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    d = n = 0.f;
#pragma unroll
    for (int w = 0; w < kSide / 32; ++w) {
      d += part[s * (kSide / 32) + w].x;
      n += part[s * (kSide / 32) + w].y;
    }
    length[s] = p.average && n != 0.f ? n : 1.f;
    ratio[s] = d / length[s];
  }
  if (tid == 0 && p.rewards != nullptr)
    p.rewards[side * p.pairs + q] = p.beta * (side ? ratio[1] : ratio[0]);
  const float h = ratio[0] - ratio[1];
  float loss, slope;
  if (p.kind == VSF_PREF_SIGMOID) {
    const float z = p.beta * h - p.margin;
    const float away = expf(-fabsf(z)), tail = log1pf(away);
    const float up = (z < 0.f ? away : 1.f) / (1.f + away);  // s(z)
    const float down = (z < 0.f ? 1.f : away) / (1.f + away);  // 1 - s(z)
    // without smoothing a rejected token of probability 0 costs nothing (z = inf)
    const float swapped = tail + (z < 0.f ? 0.f : z);
    loss = (1.f - p.smoothing) * (tail - (z > 0.f ? 0.f : z)) +
           (p.smoothing != 0.f ? p.smoothing * swapped : 0.f);
    slope = p.beta * (p.smoothing * up - (1.f - p.smoothing) * down);
  } else {
    const float gap = h - 0.5f / p.beta;
    loss = gap * gap;
    slope = 2.f * gap;
  }
  if (threadIdx.x == 0) {
    pair[q] = make_float2(loss, p.beta * h);
    __threadfence();
    last = atomicAdd(&head->ticket, 1u) + 1 == gridDim.x;
    __threadfence();
  }
  const float a = (side ? -1.f : 1.f) * p.scale / (float)p.pairs * slope /
                  (side ? length[1] : length[0]) * r.inv_tf;
  for (int64_t t = first + tid; t < end; t += kSide) {
    const Token k = token_at(r, t);
    coef[t] = live_target(r, k, nullptr) < 0 ? 0.f : a * k.w;
  }
  if (q == 0) {
    const int64_t b = clamp_start(p.starts[0], r.T_);
    for (int64_t t = threadIdx.x; t < b; t += kPairThreads) coef[t] = 0.f;
    for (int64_t t = clamp_start(p.starts[2 * p.pairs], r.T_) + threadIdx.x; t < r.T_;
         t += kPairThreads)
      coef[t] = 0.f;
  }
  __syncthreads();
  if (!last || threadIdx.x >= 32) return;
  double l = 0.0, m = 0.0;
  for (int64_t i = threadIdx.x; i < p.pairs; i += 32) {
    const float2 v = __ldcg(pair + i);
    l += (double)v.x;
    m += (double)v.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    l += __shfl_xor_sync(~0u, l, o);
    m += __shfl_xor_sync(~0u, m, o);
  }
  if (threadIdx.x == 0) {
    stats[0] = (float)((double)p.scale * l / (double)p.pairs);
    stats[1] = (float)(m / (double)p.pairs);
    head->ticket = 0;
    head->rows = 1;
  }
}

#include "mbarrier.cuh"
#include "row_pipe.cuh"
#include "row_regs.cuh"

// ------------------------------------------------------------- host side
struct RowsArg {
  const void* logits;
  int32_t dtype;
  int64_t T_, V, ld;
  const int64_t* target;
  const float* weight;
  float inv_t;
};

vsf_status check_rows(const char* who, const RowsArg& a, void* ws, size_t ws_bytes,
                      int64_t pairs) {
  const std::string w(who);
  if (a.dtype != VSF_BF16 && a.dtype != VSF_FP32) return fail(VSF_ERR_ARG, w + ": bad dtype");
  if (a.T_ < 0 || a.T_ > INT32_MAX || a.V < 1 || a.V > INT32_MAX || a.ld < a.V ||
      a.ld > (int64_t(1) << 40))
    return fail(VSF_ERR_ARG, w + ": sizes out of range");
  if (!(a.inv_t > 0.f && a.inv_t <= kMaxInvTemperature))
    return fail(VSF_ERR_ARG, w + ": inv_temperature must be positive and at most 2^127");
  if (ws == nullptr || (a.T_ > 0 && (a.logits == nullptr || a.target == nullptr)))
    return fail(VSF_ERR_ARG, w + ": NULL pointer");
  if (ws_bytes < ObjectiveWs::bytes(a.T_, pairs))
    return fail(VSF_ERR_ARG, w + ": workspace too small");
  if (!aligned(ws, 16) || !aligned(a.logits, a.dtype == VSF_BF16 ? 2 : 4) ||
      !aligned(a.target, 8) || !aligned(a.weight, 4))
    return fail(VSF_ERR_ALIGN, w + ": pointer alignment");
  return VSF_OK;
}

vsf_status check_grad(const char* who, const RowsArg& a, const void* grad, int64_t grad_ld) {
  if (grad == nullptr) return VSF_OK;
  const int64_t size = a.dtype == VSF_BF16 ? 2 : 4;
  if (grad_ld < a.V || grad_ld > (int64_t(1) << 40))
    return fail(VSF_ERR_ARG, std::string(who) + ": grad_ld out of range");
  if (!aligned(grad, size)) return fail(VSF_ERR_ALIGN, std::string(who) + ": pointer alignment");
  if (a.T_ == 0) return VSF_OK;
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(a.logits);
  const uintptr_t g0 = reinterpret_cast<uintptr_t>(grad);
  const uintptr_t x1 = x0 + ((a.T_ - 1) * a.ld + a.V) * size;
  const uintptr_t g1 = g0 + ((a.T_ - 1) * grad_ld + a.V) * size;
  if (x0 < g1 && g0 < x1 && !(x0 == g0 && a.ld == grad_ld))
    return fail(VSF_ERR_ARG, std::string(who) + ": grad overlaps the logits in part");
  return VSF_OK;
}

template <typename T>
Rows<T> rows_of(const RowsArg& a) {
  Rows<T> r;
  r.x = static_cast<const T*>(a.logits);
  r.ld = a.ld;
  r.T_ = a.T_;
  r.V = (int32_t)a.V;
  r.target = a.target;
  r.weight = a.weight;
  r.c = log2_scale(a.inv_t);
  r.inv_tf = a.inv_t;
  r.inv_t = (double)a.inv_t;
  return r;
}

constexpr int kPipeWarps = 16;

// Clusters of C CTAs of a kernel that fit on the current device at a time,
// looked up once per device and size; 0 with *e set where that fails.
template <typename T, bool POLICY>
int pipe_clusters(int C, cudaError_t* e) {
  using Shape = PipeShape<kPipeWarps>;
  static std::mutex mu;
  static int cached[64][5] = {};
  int dev = 0;
  if ((*e = cudaGetDevice(&dev)) != cudaSuccess) return 0;
  if (dev < 0 || dev >= 64) {
    *e = cudaErrorInvalidDevice;
    return 0;
  }
  int slot = 0;
  while ((1 << slot) < C) ++slot;
  std::lock_guard<std::mutex> lock(mu);
  int& n = cached[dev][slot];
  if (n == 0) {
    auto fn = row_pipe_kernel<T, kPipeWarps, POLICY>;
    constexpr uint32_t smem = pipe_smem<kPipeWarps>();
    *e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (*e != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C * 64);
    cfg.blockDim = dim3(Shape::threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int got = 0;
    *e = cudaOccupancyMaxActiveClusters(&got, fn, &cfg);
    if (*e != cudaSuccess) return 0;
    n = std::max(1, std::min(got, kMaxPipeClusters));
  }
  return n;
}

// CTAs that share a row (0: none that holds it), and whether two rows' shares
// fit the ring. `hold`: a share stays in the ring until its gradient is
// written. With few rows, more CTAs a row as long as their number fits the SMs
// (rows beyond the short ones give each of 8 at least 256 vectors). In us, policy
// loss with gradient and log probabilities, calls of a graph, with 1, 2, 4 and 8
// CTAs a row; * is taken:
//   8 x 32000 bf16     9.4, 9.1, 9.2, 9.2*     5.3, 5.3, 5.1, 5.2*
//   48 x 32000 bf16    9.5, 9.4*, 11.2, 13.6   5.3, 5.6*, 6.9, 8.6
//   100 x 32000 bf16   9.8*, 11.9, 13.5, 18.8  5.4*, 7.1, 8.4, 11.8
//   19 x 131072 bf16   10.1, 10.1, 10.2, 11.5* 8.6, 6.9, 6.0, 7.0*
//   19 x 50021 fp32    9.5, 9.6, 9.6, 11.3*    6.9, 6.1, 5.7, 6.8*
// More clusters than run at a time cost a second turn: 76 of 2, 36 of 4 and 15 of
// 8 CTAs were found to fit (a cluster keeps to one GPC), so for 16 to 19 rows and
// for 37 and 38 the rule takes one doubling too many, for about 1.5 us.
struct PipeSplit {
  int C;
  bool ahead;
};
template <typename T>
PipeSplit pipe_split(int64_t T_, int64_t V, bool hold) {
  using Shape = PipeShape<kPipeWarps>;
  const int64_t nvec = V / Vec<T>::n;
  auto chunks = [&](int C) { return (nvec / C + 1 + Shape::chunk_vecs - 1) / Shape::chunk_vecs; };
  PipeSplit s = {1, true};
  if (hold) {
    while (s.C <= 8 && 2 * chunks(s.C) > Shape::slots) s.C *= 2;
    if (s.C > 8) s = {chunks(8) <= Shape::slots ? 8 : 0, false};
    if (s.C == 0) return s;
  }
  while (s.C < 8 && T_ * s.C * 2 <= kSms * (16 / kPipeWarps)) s.C *= 2;
  return s;
}

template <typename T, bool POLICY>
cudaError_t launch_pipe(PipeArgs<T>& a, int C, cudaStream_t st) {
  using Shape = PipeShape<kPipeWarps>;
  cudaError_t e = cudaSuccess;
  const int most = pipe_clusters<T, POLICY>(C, &e);
  if (most == 0) return e;
  return launch_behind(row_pipe_kernel<T, kPipeWarps, POLICY>,
                       (unsigned)(C * std::max<int64_t>(1, std::min<int64_t>(most, a.r.T_))),
                       Shape::threads, pipe_smem<kPipeWarps>(), C, st, a);
}

// Rows short enough for the registers of 8 warps at 8 vectors a thread. Policy
// loss of 4096 rows, registers against pipeline: 1000 words 16 and 52 us, 8000
// words 48 and 64, 16000 words 66 and 73 (bf16); 16 vectors a thread would win 4
// percent at 20000 words and lose 11 at 32000.
template <typename T>
bool short_rows(int64_t V) {
  return V / Vec<T>::n <= 8 * kRegsThreads;
}

// Up to this many tokens every CTA adds up the weights for itself; beyond, a
// launch of its own does it once. In us, own sums against the launch, 1000 words:
// 1024 tokens 9.4 and 9.9, 2048 13.4 and 11.9, 4096 19.1 and 16.0, 8192 24.6 and
// 21.1; 16000 words: 1024 tokens 24.0 and 22.8, 4096 59.5 and 58.6.
constexpr int64_t kSumTokens = 2048;

template <typename T, bool POLICY, int G, int NV>
cudaError_t launch_regs_as(const PipeArgs<T>& a, const ObjectiveWs& w, cudaStream_t st) {
  const int64_t rows = 8 / G, most = kSms * regs_ctas(NV);
  const unsigned grid =
      (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, (a.r.T_ + rows - 1) / rows));
  static_assert(kSms * 4 <= kMaxPipeClusters, "the workspace holds a sum of every CTA");
  const double* total = nullptr;
  if (POLICY && a.p.mean && a.r.T_ > kSumTokens) {
    total = w.total;
    const unsigned n = (unsigned)std::min<int64_t>(64, (a.r.T_ + 8 * kSumThreads - 1) / (8 * kSumThreads));
    const cudaError_t e = launch_behind(weight_sum_kernel, n, kSumThreads, 0, 1, st, a.r.target, a.r.weight,
                                        a.r.T_, a.r.V, w.partial, w.total, w.head);
    if (e != cudaSuccess) return e;
  }
  return launch_behind(row_regs_kernel<T, G, NV, POLICY>, grid, kRegsThreads, 0, 1, st, a, total);
}

template <typename T, bool POLICY>
cudaError_t launch_regs(const PipeArgs<T>& a, const ObjectiveWs& w, cudaStream_t st) {
  const int64_t nvec = a.r.V / Vec<T>::n;
  if (nvec <= 4 * 32) return launch_regs_as<T, POLICY, 1, 4>(a, w, st);
  if (nvec <= 4 * 64) return launch_regs_as<T, POLICY, 2, 4>(a, w, st);
  if (nvec <= 4 * 128) return launch_regs_as<T, POLICY, 4, 4>(a, w, st);
  if (nvec <= 4 * 256) return launch_regs_as<T, POLICY, 8, 4>(a, w, st);
  return launch_regs_as<T, POLICY, 8, 8>(a, w, st);
}

template <typename T>
cudaError_t launch_stats(const Rows<T>& r, float4* row, float* logp, const ObjectiveWs& w,
                         cudaStream_t st) {
  if (r.T_ == 0) return cudaSuccess;
  PipeArgs<T> a = {};
  a.r = r;
  a.row = row;
  a.logp = logp;
  a.head = w.head;
  if (short_rows<T>(r.V)) return launch_regs<T, false>(a, w, st);
  return launch_pipe<T, false>(a, pipe_split<T>(r.T_, r.V, false).C, st);
}

template <typename T>
cudaError_t launch_grad(const Rows<T>& r, const ObjectiveWs& w, void* grad, int64_t grad_ld,
                        cudaStream_t st) {
  if (r.T_ == 0 || grad == nullptr) return cudaSuccess;
  const int32_t pieces =
      (int32_t)std::max<int64_t>(1, (r.V / Vec<T>::n + kGradPiece - 1) / kGradPiece);
  return launch_behind(row_grad_kernel<T>, (unsigned)std::min<int64_t>(r.T_ * pieces, kSms * kGradCtas),
                       kGradThreads, 0, 1, st, r, (const float4*)w.row, (const float*)w.coef,
                       static_cast<T*>(grad), grad_ld, pieces);
}

template <typename T>
cudaError_t policy(const RowsArg& a, const PolicyIn& p, float* stats, float* logp, void* grad,
                   int64_t grad_ld, const ObjectiveWs& w, cudaStream_t st) {
  const Rows<T> r = rows_of<T>(a);
  PipeArgs<T> k = {};
  k.r = r;
  k.p = p;
  k.grad = static_cast<T*>(grad);
  k.grad_ld = grad_ld;
  k.logp = logp;
  k.stats = stats;
  k.head = w.head;
  k.partial = w.partial;
  if (short_rows<T>(r.V)) return launch_regs<T, true>(k, w, st);
  const PipeSplit split = pipe_split<T>(r.T_, r.V, true);
  if (split.C > 0) {
    k.ahead = split.ahead;
    return launch_pipe<T, true>(k, split.C, st);
  }
  // a row too long for a cluster's shared memory: statistics, then gradient
  cudaError_t e = launch_stats(r, w.row, logp, w, st);
  if (e != cudaSuccess) return e;
  e = launch_behind(policy_tokens_kernel<T>, 1, kTokenThreads, 0, 1, st, r, p, (const float4*)w.row,
                    w.coef, stats, w.head);
  if (e != cudaSuccess) return e;
  return launch_grad(r, w, grad, grad_ld, st);
}

template <typename T>
cudaError_t preference(const RowsArg& a, const PairIn& p, float* stats, float* logp, void* grad,
                       int64_t grad_ld, const ObjectiveWs& w, cudaStream_t st) {
  const Rows<T> r = rows_of<T>(a);
  cudaError_t e = launch_stats(r, w.row, logp, w, st);
  if (e != cudaSuccess) return e;
  e = launch_behind(pair_kernel<T>, (unsigned)p.pairs, kPairThreads, 0, 1, st, r, p,
                    (const float4*)w.row, w.coef, w.pair, stats, w.head);
  if (e != cudaSuccess) return e;
  return launch_grad(r, w, grad, grad_ld, st);
}

}  // namespace
}  // namespace vsf

using namespace vsf;

extern "C" {

size_t vsf_objective_workspace_bytes(int64_t tokens, int64_t pairs) {
  if (tokens < 0 || tokens > INT32_MAX || pairs < 0 || pairs > INT32_MAX) return 0;
  return ObjectiveWs::bytes(tokens, pairs);
}

vsf_status vsf_objective_workspace_init(void* d_workspace, size_t bytes, void* stream) {
  vsf::Range nvtx_range("vsf_objective_workspace_init");
  if (d_workspace == nullptr || bytes < sizeof(WsHead))
    return fail(VSF_ERR_ARG, "vsf_objective_workspace_init: NULL or too small");
  if (!aligned(d_workspace, 16))
    return fail(VSF_ERR_ALIGN, "vsf_objective_workspace_init: workspace alignment");
  const cudaError_t e = cudaMemsetAsync(d_workspace, 0, bytes, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSF_OK : cuda_error(e, "vsf_objective_workspace_init");
}

vsf_status vsf_token_logprobs(const void* logits, int32_t dtype, int64_t T, int64_t V, int64_t ld,
                              const int64_t* targets, float inv_temperature, float* logp,
                              void* d_workspace, size_t ws_bytes, void* stream) {
  vsf::Range nvtx_range("vsf_token_logprobs");
  const RowsArg a = {logits, dtype, T, V, ld, targets, nullptr, inv_temperature};
  const vsf_status s = check_rows("vsf_token_logprobs", a, d_workspace, ws_bytes, 0);
  if (s != VSF_OK) return s;
  if (T > 0 && logp == nullptr) return fail(VSF_ERR_ARG, "vsf_token_logprobs: NULL pointer");
  if (!aligned(logp, 4)) return fail(VSF_ERR_ALIGN, "vsf_token_logprobs: pointer alignment");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const ObjectiveWs w(d_workspace, T);
  const cudaError_t e =
      dtype == VSF_BF16 ? launch_stats(rows_of<uint16_t>(a), nullptr, logp, w, st)
                        : launch_stats(rows_of<float>(a), nullptr, logp, w, st);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, "vsf_token_logprobs");
}

vsf_status vsf_policy_loss(const void* logits, int32_t dtype, int64_t T, int64_t V, int64_t ld,
                           const int64_t* targets, const float* old_logp, const float* ref_logp,
                           const float* advantages, const float* weights,
                           const vsf_policy_hparams* hp, float* stats, float* logp, void* grad,
                           int64_t grad_ld, void* d_workspace, size_t ws_bytes, void* stream) {
  vsf::Range nvtx_range("vsf_policy_loss");
  const char* who = "vsf_policy_loss";
  if (hp == nullptr || stats == nullptr) return fail(VSF_ERR_ARG, "vsf_policy_loss: NULL pointer");
  const RowsArg a = {logits, dtype, T, V, ld, targets, weights, hp->inv_temperature};
  vsf_status s = check_rows(who, a, d_workspace, ws_bytes, 0);
  if (s == VSF_OK) s = check_grad(who, a, grad, grad_ld);
  if (s != VSF_OK) return s;
  if (T > 0 && (old_logp == nullptr || advantages == nullptr ||
                (hp->kl_beta != 0.f && ref_logp == nullptr)))
    return fail(VSF_ERR_ARG, "vsf_policy_loss: NULL pointer");
  if (!(hp->clip_low >= 0.f && hp->clip_low <= 1.f && hp->clip_high >= 0.f) ||
      !std::isfinite(hp->kl_beta) || !std::isfinite(hp->scale))
    return fail(VSF_ERR_ARG, "vsf_policy_loss: hyper-parameters out of range");
  if (!aligned(old_logp, 4) || !aligned(ref_logp, 4) || !aligned(advantages, 4) ||
      !aligned(stats, 4) || !aligned(logp, 4))
    return fail(VSF_ERR_ALIGN, "vsf_policy_loss: pointer alignment");
  const PolicyIn p = {old_logp,
                      ref_logp,
                      advantages,
                      1.f - hp->clip_low,
                      1.f + hp->clip_high,
                      hp->kl_beta,
                      hp->scale,
                      hp->mean != 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const ObjectiveWs w(d_workspace, T);
  const cudaError_t e = dtype == VSF_BF16
                            ? policy<uint16_t>(a, p, stats, logp, grad, grad_ld, w, st)
                            : policy<float>(a, p, stats, logp, grad, grad_ld, w, st);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, who);
}

vsf_status vsf_preference_loss(const void* logits, int32_t dtype, int64_t T, int64_t V, int64_t ld,
                               const int64_t* targets, const float* ref_logp,
                               const float* weights, const int64_t* seq_starts, int64_t pairs,
                               const vsf_preference_hparams* hp, float* stats, float* rewards,
                               float* logp, void* grad, int64_t grad_ld, void* d_workspace,
                               size_t ws_bytes, void* stream) {
  vsf::Range nvtx_range("vsf_preference_loss");
  const char* who = "vsf_preference_loss";
  if (hp == nullptr || stats == nullptr || seq_starts == nullptr)
    return fail(VSF_ERR_ARG, "vsf_preference_loss: NULL pointer");
  if (pairs < 1 || pairs > (1 << 24))
    return fail(VSF_ERR_ARG, "vsf_preference_loss: pairs out of range");
  const RowsArg a = {logits, dtype, T, V, ld, targets, weights, hp->inv_temperature};
  vsf_status s = check_rows(who, a, d_workspace, ws_bytes, pairs);
  if (s == VSF_OK) s = check_grad(who, a, grad, grad_ld);
  if (s != VSF_OK) return s;
  if ((hp->kind != VSF_PREF_SIGMOID && hp->kind != VSF_PREF_SQUARED) || !(hp->beta > 0.f) ||
      !std::isfinite(hp->beta) || !(hp->smoothing >= 0.f && hp->smoothing <= 0.5f) ||
      !std::isfinite(hp->margin) || !std::isfinite(hp->scale))
    return fail(VSF_ERR_ARG, "vsf_preference_loss: hyper-parameters out of range");
  if (!aligned(ref_logp, 4) || !aligned(seq_starts, 8) || !aligned(stats, 4) ||
      !aligned(rewards, 4) || !aligned(logp, 4))
    return fail(VSF_ERR_ALIGN, "vsf_preference_loss: pointer alignment");
  const PairIn p = {ref_logp,   seq_starts,    rewards,   pairs,    hp->beta,
                    hp->smoothing, hp->margin, hp->scale, hp->kind, hp->average != 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const ObjectiveWs w(d_workspace, T);
  const cudaError_t e = dtype == VSF_BF16
                            ? preference<uint16_t>(a, p, stats, logp, grad, grad_ld, w, st)
                            : preference<float>(a, p, stats, logp, grad, grad_ld, w, st);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, who);
}

}  // extern "C"
