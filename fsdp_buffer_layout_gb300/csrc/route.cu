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
// A group of L lanes (8 or a warp) takes a token and holds its experts in
// registers, N a lane. A CTA takes a run of tokens, one sequence of it after the
// other, so that the sequence's sums stay in registers. Instructions bound the
// large sizes (256 experts: 1 KB of logits a token against some hundred
// instructions a warp), so the common form, 32 N experts in aligned rows, is
// compiled apart: no checks of the expert's number, the score's kind known,
// 16-byte loads and stores. 65536 tokens of 256 experts (fp32, sigmoid, bias, top
// 8) take 49 us forward and 27 us back, against 10 and 10 to 20 of HBM time; the
// issue slots are two thirds full, with some 600 and 350 instructions a token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>

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
constexpr float kShareUnit = 1099511627776.f;

struct RouteIn {
  int64_t T_, ld, sequences;
  int32_t E, K, score, renorm;
  float scale, balance;
  const float* bias;
  const uint8_t* live;
  const int64_t* starts;  // NULL: one sequence of T_ tokens
  float c;                // log2(e)
};

// The sequences of a run of tokens [pos, end), in turn. Tokens in front of the
// first start have sequence -1, those behind the last one `sequences`. Whatever
// the starts hold, every token comes once and the walk ends.
struct Walk {
  int64_t pos, end, seq, stop;  // tokens [pos, stop) belong to seq
  __device__ __forceinline__ void bound(const RouteIn& p) {
    const int64_t v = p.starts == nullptr || seq >= p.sequences ? end : p.starts[seq + 1];
    stop = v < pos ? pos : v > end ? end : v;
  }
  __device__ __forceinline__ void settle(const RouteIn& p) {  // on to one with tokens
    for (bound(p); stop == pos && pos < end; bound(p)) ++seq;
  }
  // All lanes of a warp together: a step of the search looks at 32 starts.
  __device__ __forceinline__ Walk(const RouteIn& p, int64_t first, int64_t last)
      : pos(first), end(last), seq(0) {
    if (p.starts != nullptr) {
      const int64_t n = p.sequences + 1;
      int64_t lo = -1, hi = n;  // starts[lo] <= pos < starts[hi]
      while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32;
        const int64_t at = lo + ((threadIdx.x & 31) + 1) * step;
        const bool in = at < hi && p.starts[at < n ? at : n - 1] <= pos;
        const int k = __ffs(~__ballot_sync(~0u, in)) - 1;  // steps taken; -1: all 32
        lo += (k < 0 ? 32 : k) * step;
        if (lo + step < hi) hi = lo + step;
      }
      seq = lo;
    }
    settle(p);
  }
  __device__ __forceinline__ bool done() const { return pos >= end; }
  __device__ __forceinline__ bool inside(const RouteIn& p) const {
    return seq >= 0 && seq < p.sequences;
  }
  __device__ __forceinline__ void next(const RouteIn& p) {
    pos = stop;
    ++seq;
    settle(p);
  }
};

// Order-preserving 32-bit key of a number: larger is better, -0 equals +0.
// Numbers lie above 1, the key of NaN; 0 is below every key. The caller tells
// whether a NaN may be there.
__device__ __forceinline__ uint32_t order_key(float v) {
  const int b = __float_as_int(v + 0.f);
  return (uint32_t)(b ^ (b >> 31 | (int)0x80000000));
}

// How a lane holds experts. Full: E = L N, each lane V adjacent experts at a
// time, which are one load; else expert `lane + L j` in register j.
template <typename T, int L, int N, bool FULL>
struct Hold {
  static constexpr int V = FULL ? (N * (int)sizeof(T) < 16 ? N : 16 / (int)sizeof(T)) : 1;
  static constexpr bool kWarp = L == 32;
  static constexpr int kLanes = L;
  static __device__ __forceinline__ int expert(int lane, int j) {
    return FULL ? j / V * (L * V) + lane * V + j % V : lane + L * j;
  }
  static __device__ __forceinline__ bool has(int lane, int j, int E) {
    return FULL || lane + L * j < E;
  }
};
template <int B>
struct Bytes;
template <>
struct Bytes<2> { using type = uint16_t; };
template <>
struct Bytes<4> { using type = uint32_t; };
template <>
struct Bytes<8> { using type = uint2; };
template <>
struct Bytes<16> { using type = uint4; };

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (L == 32) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
  }
}

// 1 / (1 + exp(-x)): ex2.approx and rcp.approx and the rounding of x log2(e).
__device__ __forceinline__ float rcp(float v) {  // 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float sigmoid(float x, float c) { return rcp(1.f + ex2(-x * c)); }

// A token's scores from its logits, in place: the largest logit and 1 / sum of
// the softmax (0 and 1 for sigmoids), with which score_of gives one logit's
// score again, and Z.
struct Norm {
  float m, inv, z;
};
template <typename H, int L, int N>
__device__ __forceinline__ Norm scores(float (&x)[N], bool softmax, int E, float c, int lane) {
  float sum = 0.f;
  if (softmax) {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) m = fmaxf(m, x[j]);
    m = group_max<L>(m);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      x[j] = H::has(lane, j, E) ? ex2((x[j] - m) * c) : 0.f;
      sum += x[j];
    }
    const float inv = rcp(group_sum<L>(sum));
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] *= inv;
    return {m, inv, 1.f};
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    x[j] = H::has(lane, j, E) ? sigmoid(x[j], c) : 0.f;
    sum += x[j];
  }
  return {0.f, 1.f, group_sum<L>(sum) + 1e-20f};
}
__device__ __forceinline__ float score_of(float x, Norm n, bool softmax, float c) {
  return softmax ? ex2((x - n.m) * c) * n.inv : sigmoid(x, c);
}

// A token's logits as they lie in memory, on their way while the token before
// it is worked on.
template <typename H, typename T, int N>
struct Raw {
  static constexpr int V = H::V;
  using Piece = typename Bytes<V * (int)sizeof(T)>::type;
  union {
    Piece p[N / V];
    T t[N];
  };
  bool on;
  __device__ __forceinline__ void fetch(const T* row, int E, int lane, bool live) {
    on = live;
#pragma unroll
    for (int j = 0; j < N; j += V)
      if (on && H::has(lane, j, E)) p[j / V] = *reinterpret_cast<const Piece*>(row + H::expert(lane, j));
  }
  // (of a whole warp's token: only where it is live)
  __device__ __forceinline__ void get(float (&x)[N], int E, int lane) const {
#pragma unroll
    for (int j = 0; j < N; ++j)
      x[j] = (H::kWarp || on) && H::has(lane, j, E) ? to_f(t[j]) : -INFINITY;
  }
};

// A lane's part in a token's choice: expert e takes place `rank` of the K, or
// none (rank >= K).
struct Choice {
  int e, rank;
};

// The K experts of largest key, ties to the lowest, the k-th in lane k of the
// group. Keys are lost. Round by round, the group's largest key is found and
// taken out.
template <typename H, int N>
__device__ __forceinline__ Choice choose_rounds(uint32_t (&key)[N], int K, int lane) {
  int mine = -1;
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
    int be = H::expert(lane, 0);
#pragma unroll
    for (int j = 1; j < N; ++j)
      if (key[j] > best) {
        best = key[j];
        be = H::expert(lane, j);
      }
    int e;
    if constexpr (H::kLanes == 32) {
      const uint32_t top = __reduce_max_sync(~0u, best);
      e = (int)__reduce_min_sync(~0u, best == top ? (uint32_t)be : 0xffffffffu);
    } else {
#pragma unroll
      for (int o = H::kLanes / 2; o > 0; o >>= 1) {
        const uint32_t key2 = __shfl_xor_sync(~0u, best, o);
        const int e2 = __shfl_xor_sync(~0u, be, o);
        if (key2 > best || (key2 == best && e2 < be)) {
          best = key2;
          be = e2;
        }
      }
      e = be;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (H::expert(lane, j) == e) key[j] = 0u;
    if (lane == k) mine = e;
  }
  return {mine, lane};
}

// The same with fewer and less dependent instructions where a lane holds several
// keys. A bound from below leaves few candidates, which go to a lane each; a
// candidate's rank is the number of better ones, counted in shared memory
// (rounds over the candidates took two dependent warp reductions a choice). Up
// to 8 choices, the smallest of the largest keys of 8 groups of 4 lanes bounds
// them (at least 8 keys reach it; 22 on average, as many as it takes to draw
// each of 8 kinds); with more choices, or more than 32 candidates, the K-th
// largest of the lanes' largest keys. Where that leaves more than 32 as well
// (equal keys), the rounds above.
struct __align__(16) Candidates {
  uint2 c[32];  // expert (inverted: the lower is the better), key
};
__device__ __forceinline__ uint64_t merit(uint2 c) { return (uint64_t)c.y << 32 | c.x; }
template <typename H, int N>
__device__ __forceinline__ int gather(const uint32_t (&key)[N], uint32_t bound, int lane,
                                      Candidates& c) {
  int n = 0;
  const uint32_t below = (1u << lane) - 1;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const bool in = key[j] >= bound;
    const uint32_t all = __ballot_sync(~0u, in);
    const int at = n + __popc(all & below);
    if (in && at < 32) c.c[at] = make_uint2(~(uint32_t)H::expert(lane, j), key[j]);
    n += __popc(all);
  }
  return n;
}
template <typename H, int N>
__device__ __forceinline__ Choice choose(uint32_t (&key)[N], int K, int lane, Candidates& cand) {
  if (N == 1) return choose_rounds<H, N>(key, K, lane);
  uint32_t lane_max = key[0];
#pragma unroll
  for (int j = 1; j < N; ++j) lane_max = max(lane_max, key[j]);
  uint32_t four = max(lane_max, __shfl_xor_sync(~0u, lane_max, 1));
  four = max(four, __shfl_xor_sync(~0u, four, 2));
  uint32_t bound = __reduce_min_sync(~0u, four);
  int n = 0;
#pragma unroll 1
  for (bool tight = K > 8;; tight = true) {
    if (tight)
      for (int k = 0; k < K;) {
        bound = __reduce_max_sync(~0u, lane_max);
        const bool hit = lane_max == bound;
        k += __popc(__ballot_sync(~0u, hit));
        if (hit) lane_max = 0u;
      }
    n = gather<H, N>(key, max(bound, 1u), lane, cand);
    if (n <= 32) break;
    if (tight) return choose_rounds<H, N>(key, K, lane);
    __syncwarp();
  }
  if (lane >= n) cand.c[lane] = make_uint2(0u, 0u);
  __syncwarp();
  const uint2 own = cand.c[lane];
  const uint64_t mine = merit(own);
  int rank = 0;
  const uint4* two = reinterpret_cast<const uint4*>(cand.c);
#pragma unroll 4
  for (int i = 0; 2 * i < n; ++i) {
    const uint4 v = two[i];
    rank += (int)(merit(make_uint2(v.x, v.y)) > mine) + (int)(merit(make_uint2(v.z, v.w)) > mine);
  }
  __syncwarp();
  return {(int)~own.x, lane < n ? rank : 32};
}

// Sums of the calls' workspace, zero between calls.
struct RouteSums {
  int32_t* tokens;            // [sequences] live tokens
  int32_t* count;             // [sequences * E] choices
  unsigned long long* share;  // [sequences * E] sums of shares
};

struct RouteOut {
  int32_t* idx;
  float* gates;
  int32_t* counts;
  float* loss;
  int32_t* seq_counts;
  float* seq_coef;
};

// Experts [e0, e0 + en) of all sequences: copies the counts out, adds up their
// totals, the balance loss and (first part) the sequences' coefficients, and
// zeroes the sums. A thread keeps to one expert and every G-th sequence. The
// loss of this part goes to thread 0.
__device__ float route_finish(const RouteIn& p, const RouteSums& w, const RouteOut& o, int e0,
                              int en, bool first) {
  __shared__ int total[kMaxExperts];
  __shared__ float part[kRouteWarps];
  const int tid = threadIdx.x;
  for (int e = tid; e < en; e += kRouteThreads) total[e] = 0;
  int mine = 0;
  for (int64_t s = tid; s < p.sequences; s += kRouteThreads) mine += __ldcg(w.tokens + s) > 0;
  // (sequences with a live token; also orders total[] before its use)
  int full = 0;
  {
    __shared__ int sum;
    if (tid == 0) sum = 0;
    __syncthreads();
    if (mine) atomicAdd(&sum, mine);
    __syncthreads();
    full = sum;
  }
  const float f = full > 0 ? p.balance * (float)p.E / ((float)p.K * (float)full) : 0.f;
  int width = 1;  // threads side by side on the experts
  while (width < en && width < kRouteThreads) width *= 2;
  const int G = kRouteThreads / width;
  float l = 0.f;
  for (int e = tid & (width - 1); e < en; e += width) {
    int c = 0;
#pragma unroll 4
    for (int64_t s = tid / width; s < p.sequences; s += G) {
      const int64_t at = s * p.E + e0 + e;
      const int n = __ldcg(w.count + at);
      const unsigned long long share = __ldcg(w.share + at);
      const float t = (float)__ldcg(w.tokens + s);
      o.seq_counts[at] = n;
      w.count[at] = 0;
      w.share[at] = 0ull;
      c += n;
      if (n) l += f / (t * t) * ((float)n * ((float)share / kShareUnit));
    }
    if (G == 1) total[e] = c;
    else if (c) atomicAdd(&total[e], c);
  }
  if (first)
    for (int64_t s = tid; s < p.sequences; s += kRouteThreads) {
      const float t = (float)__ldcg(w.tokens + s);
      o.seq_coef[s] = t > 0.f ? f / (t * t) : 0.f;
    }
  l = group_sum<32>(l);
  if ((tid & 31) == 0) part[tid >> 5] = l;
  __syncthreads();
  for (int e = tid; e < en; e += kRouteThreads) o.counts[e0 + e] = total[e];
  l = 0.f;
  for (int i = 0; i < kRouteWarps; ++i) l += part[i];
  return l;
}

// The call's end, by one thread: the loss, and the head as the next call wants
// it. Where a loss has used the workspace, its rows lay among the sums.
__device__ __forceinline__ void route_close(WsHead* head, float* loss, float l) {
  static_assert(offsetof(WsHead, nan) == 8 && offsetof(WsHead, rows) == 12, "nan, rows: one load");
  const uint2 seen = __ldcg(reinterpret_cast<const uint2*>(&head->nan));
  if (seen.y) atomicOr(&head->err, kErrShared);
  *loss = seen.x | seen.y ? NAN : l;
  head->nan = 0u;
  head->ticket = 0u;
}

// CTAs an SM: registers for the token ahead as well. At 256 experts 3 run in 76 us
// (65536 tokens, both ways) where 4, which spill, take 90 and 2 take 88; at 32
// experts (4 a lane) 4 run in 33 where 3 and 6 take 38; at 512 2 run in 179 where
// 3 take 325 and 1 takes 182 (rows not full).
constexpr int route_ctas(int n) { return n <= 4 ? 4 : n <= 8 ? 3 : 2; }

// SCORE: the score's kind, or -1 where it is known at run time only.
template <typename T, int L, int N, bool FULL, int SCORE>
__global__ void __launch_bounds__(kRouteThreads, route_ctas(N))
    route_kernel(const T* logits, const __grid_constant__ RouteIn p,
                 const __grid_constant__ RouteSums w, const __grid_constant__ RouteOut o,
                 WsHead* head, int32_t finish) {
  using H = Hold<T, L, N, FULL>;
  constexpr int kGroups = kRouteThreads / L;
  __shared__ float share[kGroups][N * L];  // sums of shares of each group
  __shared__ int32_t count[N * L];         // choices of the CTA
  __shared__ Candidates cand[kRouteWarps];
  __shared__ int tokens, last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & (L - 1), group = tid / L;
  for (int e = tid; e < N * L; e += kRouteThreads) count[e] = 0;
  if (tid == 0) tokens = 0;
  __syncthreads();
  take_turn();
  const bool softmax = SCORE < 0 ? p.score == VSF_SCORE_SOFTMAX : SCORE == VSF_SCORE_SOFTMAX;
  const float c = p.c;
  float bias[N];
  bool strange = false;  // a NaN in the bias
#pragma unroll
  for (int j = 0; j < N; ++j) {
    bias[j] = p.bias != nullptr && H::has(lane, j, p.E) ? p.bias[H::expert(lane, j)] : 0.f;
    strange |= bias[j] != bias[j];
  }
  strange = __any_sync(~0u, strange);
  const int64_t per = (p.T_ + gridDim.x - 1) / gridDim.x;
  const int64_t from = min((int64_t)blockIdx.x * per, p.T_);
  for (Walk run(p, from, min(from + per, p.T_)); !run.done(); run.next(p)) {
    const bool counted = run.inside(p);
    float acc[N];
    int seen = 0;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.f;
    // the groups of a warp go round together: shuffles span them
    Raw<H, T, N> next;
    auto fetch = [&](int64_t t) {
      const bool live = t < run.stop && (p.live == nullptr || p.live[t] != 0);
      next.fetch(logits + (live ? t : run.pos) * p.ld, p.E, lane, live);
    };
    int64_t t = run.pos + warp * (32 / L) + (tid & 31) / L;
    fetch(t);
    for (int64_t t0 = run.pos + warp * (32 / L); t0 < run.stop; t0 += kGroups, t += kGroups) {
      const bool in = t < run.stop, on = next.on;
      const T* row = logits + (on ? t : run.pos) * p.ld;
      if (L == 32 && !on) {
        if (lane < p.K) {
          o.idx[t * p.K + lane] = -1;
          o.gates[t * p.K + lane] = 0.f;
        }
        fetch(t + kGroups);
        continue;
      }
      float x[N];
      uint32_t key[N];
      next.get(x, p.E, lane);
      fetch(t + kGroups);
      if (p.bias == nullptr) {
#pragma unroll
        for (int j = 0; j < N; ++j) key[j] = order_key(x[j]);
      }
      const Norm norm = scores<H, L, N>(x, softmax, p.E, c, lane);
      if (p.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < N; ++j) key[j] = order_key(x[j] + bias[j]);
      }
      const bool odd = norm.z != norm.z || norm.inv != norm.inv;  // a NaN somewhere
      if (__any_sync(~0u, odd) || strange) {
        // NaN after every number: of a logit, or, with a bias, of a sum
        Raw<H, T, N> again;
        float y[N];
        again.fetch(row, p.E, lane, on);
        again.get(y, p.E, lane);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (p.bias != nullptr) y[j] = x[j] + bias[j];
          if (y[j] != y[j]) key[j] = 1u;
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (!H::has(lane, j, p.E)) key[j] = 0u;
      const Choice mine = L == 32 && N > 1 ? choose<H, N>(key, p.K, lane, cand[warp])
                                           : choose_rounds<H, N>(key, p.K, lane);
      float score = 0.f;
      if (on && mine.rank < p.K) score = score_of(to_f(row[mine.e]), norm, softmax, c);
      const float sum = group_sum<L>(score) + 1e-20f;
      if (in && mine.rank < p.K) {
        o.idx[t * p.K + mine.rank] = on ? mine.e : -1;
        o.gates[t * p.K + mine.rank] =
            on ? p.scale * (p.renorm ? __fdividef(score, sum) : score) : 0.f;
        if (on && counted) atomicAdd(&count[mine.e], 1);
      }
      if (on) {
        const float inv = softmax ? 1.f : rcp(norm.z);
        bad |= odd;
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = __fmaf_rn(x[j], inv, acc[j]);
        ++seen;
      }
    }
    if (!counted) continue;
#pragma unroll
    for (int j = 0; j < N; ++j) share[group][H::expert(lane, j)] = acc[j];
    if (lane == 0 && seen > 0) atomicAdd(&tokens, seen);
    if (bad) head->nan = 1u;
    __syncthreads();
    for (int e = tid; e < p.E; e += kRouteThreads) {
      float q = 0.f;
      for (int g = 0; g < kGroups; ++g) q += share[g][e];
      const int64_t at = run.seq * p.E + e;
      if (q > 0.f) atomicAdd(w.share + at, (unsigned long long)__float2ull_rn(q * kShareUnit));
      if (count[e] > 0) atomicAdd(w.count + at, count[e]);
      count[e] = 0;
    }
    if (tid == 0) {
      if (tokens > 0) atomicAdd(w.tokens + run.seq, tokens);
      tokens = 0;
    }
    __syncthreads();
  }
  if (!finish) return;
  if (gridDim.x > 1) {  // the last CTA finishes
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      last = atomicAdd(&head->ticket, 1u) + 1 == gridDim.x;
      __threadfence();
    }
    __syncthreads();
    if (!last) return;
  }
  const float l = route_finish(p, w, o, 0, p.E, true);
  for (int64_t s = tid; s < p.sequences; s += kRouteThreads) w.tokens[s] = 0;
  if (tid == 0) route_close(head, o.loss, l);
}

// The finish as a launch of its own, for many sequences: 32 experts a CTA.
constexpr int kFinishExperts = 32;
static_assert(kMaxExperts / kFinishExperts <= 16, "parts of the loss in the head");
__global__ void __launch_bounds__(kRouteThreads)
    route_finish_kernel(const __grid_constant__ RouteIn p, const __grid_constant__ RouteSums w,
                        const __grid_constant__ RouteOut o, WsHead* head) {
  __shared__ int last;
  const int e0 = blockIdx.x * kFinishExperts, tid = threadIdx.x;
  take_turn();
  const float l = route_finish(p, w, o, e0, min(kFinishExperts, p.E - e0), blockIdx.x == 0);
  if (tid == 0) {
    head->part[blockIdx.x] = l;
    __threadfence();
    last = atomicAdd(&head->ticket, 1u) + 1 == gridDim.x;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  for (int64_t s = tid; s < p.sequences; s += kRouteThreads) w.tokens[s] = 0;
  if (tid == 0) {
    float sum = 0.f;
    for (uint32_t i = 0; i < gridDim.x; ++i) sum += __ldcg(&head->part[i]);
    route_close(head, o.loss, sum);
  }
}

template <typename T, int L, int N, bool FULL, int SCORE>
__global__ void __launch_bounds__(kRouteThreads, route_ctas(N))
    route_grad_kernel(const T* logits, const __grid_constant__ RouteIn p, const int32_t* idx,
                      const float* d_gates, const int32_t* seq_counts, const float* seq_coef,
                      float loss_scale, T* grad, int64_t grad_ld) {
  using H = Hold<T, L, N, FULL>;
  constexpr int kGroups = kRouteThreads / L, V = H::V;
  __shared__ __align__(16) float pulled[kGroups][N * L];  // the gates' pull; zero between tokens
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & (L - 1);
  float* pull = pulled[tid / L];
#pragma unroll
  for (int j = 0; j < N; ++j) pull[lane + L * j] = 0.f;
  __syncwarp();
  take_turn();
  const bool softmax = SCORE < 0 ? p.score == VSF_SCORE_SOFTMAX : SCORE == VSF_SCORE_SOFTMAX;
  const float c = p.c;
  const int64_t per = (p.T_ + gridDim.x - 1) / gridDim.x;
  const int64_t from = min((int64_t)blockIdx.x * per, p.T_);
  for (Walk run(p, from, min(from + per, p.T_)); !run.done(); run.next(p)) {
    float b[N];  // the balance loss's pull on each share
    const bool balanced = run.inside(p) && loss_scale != 0.f;
    const float f = balanced ? loss_scale * seq_coef[run.seq] : 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j)
      b[j] = balanced && H::has(lane, j, p.E)
                 ? f * (float)seq_counts[run.seq * p.E + H::expert(lane, j)]
                 : 0.f;
    Raw<H, T, N> next;
    int next_e = -1;  // lane k: choice k and its gate's gradient
    float next_dg = 0.f;
    auto fetch = [&](int64_t t) {
      const bool live = t < run.stop && (p.live == nullptr || p.live[t] != 0);
      next.fetch(logits + (live ? t : run.pos) * p.ld, p.E, lane, live);
      next_e = -1;
      if (live && d_gates != nullptr && lane < p.K) {
        next_e = idx[t * p.K + lane];
        next_dg = d_gates[t * p.K + lane];
      }
    };
    int64_t t = run.pos + warp * (32 / L) + (tid & 31) / L;
    fetch(t);
    for (int64_t t0 = run.pos + warp * (32 / L); t0 < run.stop; t0 += kGroups, t += kGroups) {
      const bool in = t < run.stop, on = next.on;
      float x[N];
      if (L == 32 && !on) {
        fetch(t + kGroups);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (H::has(lane, j, p.E)) grad[t * grad_ld + H::expert(lane, j)] = from_f<T>(0.f);
        continue;
      }
      next.get(x, p.E, lane);
      int e = next_e;
      float dg = next_dg, xe = 0.f;
      if (e >= 0 && e < p.E) {
        xe = to_f(logits[t * p.ld + e]);
      } else {
        e = -1;
        dg = 0.f;
      }
      fetch(t + kGroups);
      const Norm norm = scores<H, L, N>(x, softmax, p.E, c, lane);
      float ds[N];
      if (d_gates != nullptr) {
        float v = dg;
        if (p.renorm) {
          const float s = e >= 0 ? score_of(xe, norm, softmax, c) : 0.f;
          const float inv = rcp(group_sum<L>(s) + 1e-20f);
          v = (dg - group_sum<L>(dg * s) * inv) * inv;
        }
        if (e >= 0) pull[e] = p.scale * v;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < N; ++j) ds[j] = pull[H::expert(lane, j)];
        __syncwarp();
        if (e >= 0) pull[e] = 0.f;
        __syncwarp();
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) ds[j] = 0.f;
      }
      float dot = 0.f;
      if (softmax) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          ds[j] += b[j];
          dot = __fmaf_rn(x[j], ds[j], dot);
        }
        dot = group_sum<L>(dot);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] *= ds[j] - dot;
      } else {
        const float inv = rcp(norm.z);
        if (balanced) {
#pragma unroll
          for (int j = 0; j < N; ++j) dot = __fmaf_rn(b[j], x[j], dot);
          dot = group_sum<L>(dot) * inv;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (balanced) ds[j] = __fmaf_rn(b[j] - dot, inv, ds[j]);
          x[j] = x[j] * (1.f - x[j]) * ds[j];
        }
      }
      if (in) {
        T* g = grad + t * grad_ld;
        using Piece = typename Bytes<V * (int)sizeof(T)>::type;
#pragma unroll
        for (int j = 0; j < N; j += V) {
          if (!H::has(lane, j, p.E)) continue;
          union {
            Piece p;
            T t[V];
          } u;
#pragma unroll
          for (int v = 0; v < V; ++v) u.t[v] = from_f<T>(on ? x[j + v] : 0.f);
          *reinterpret_cast<Piece*>(g + H::expert(lane, j)) = u.p;
        }
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------- host side
struct RouteWs {
  static size_t tokens_bytes(int64_t sequences) { return (size_t)((sequences * 4 + 15) / 16 * 16); }
  static size_t count_bytes(int64_t E, int64_t sequences) {
    return (size_t)((E * sequences * 4 + 15) / 16 * 16);
  }
  static size_t bytes(int64_t E, int64_t sequences) {
    return sizeof(WsHead) + tokens_bytes(sequences) + count_bytes(E, sequences) +
           (size_t)(E * sequences) * 8;
  }
  WsHead* head;
  RouteSums sums;
  RouteWs(void* ws, int64_t E, int64_t sequences) {
    unsigned char* b = static_cast<unsigned char*>(ws);
    head = reinterpret_cast<WsHead*>(b);
    b += sizeof(WsHead);
    sums.tokens = reinterpret_cast<int32_t*>(b);
    b += tokens_bytes(sequences);
    sums.count = reinterpret_cast<int32_t*>(b);
    b += count_bytes(E, sequences);
    sums.share = reinterpret_cast<unsigned long long*>(b);
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
          hp->route_scale, hp->balance, bias, live, starts, 1.44269504f};
}

// CTAs: 16 tokens and one a group at least, no more than run at a time.
template <int L, int N>
unsigned route_grid(int64_t T_) {
  const int64_t least = std::max(16, kRouteThreads / L);
  return (unsigned)std::max<int64_t>(
      1, std::min<int64_t>((T_ + least - 1) / least, kSms * route_ctas(N)));
}

// Up to here the last CTA of the router finishes; beyond, a launch of its own:
// for 33 sequences of 256 experts the last CTA alone took 12 us.
constexpr int64_t kFinishInside = 2048;

template <typename T, int L, int N, bool FULL, int SCORE>
cudaError_t route_launch(const void* logits, const RouteIn& p, const RouteOut& o, const RouteWs& w,
                         cudaStream_t st) {
  const bool inside = p.E * p.sequences <= kFinishInside;
  const cudaError_t e = launch_behind(route_kernel<T, L, N, FULL, SCORE>, route_grid<L, N>(p.T_),
                                      kRouteThreads, 0, 1, st, static_cast<const T*>(logits), p,
                                      w.sums, o, w.head, (int32_t)inside);
  if (e != cudaSuccess || inside) return e;
  return launch_behind(route_finish_kernel, (p.E + kFinishExperts - 1) / kFinishExperts,
                       kRouteThreads, 0, 1, st, p, w.sums, o, w.head);
}

template <typename T, int L, int N, bool FULL, int SCORE>
cudaError_t grad_launch(const void* logits, const RouteIn& p, const int32_t* idx,
                        const float* d_gates, const int32_t* seq_counts, const float* seq_coef,
                        float loss_scale, void* grad, int64_t grad_ld, cudaStream_t st) {
  return launch_behind(route_grad_kernel<T, L, N, FULL, SCORE>, route_grid<L, N>(p.T_),
                       kRouteThreads, 0, 1, st, static_cast<const T*>(logits), p, idx, d_gates,
                       seq_counts, seq_coef, loss_scale, static_cast<T*>(grad), grad_ld);
}

// F<T, lanes a token, experts a lane, full, score> for the experts of p; wide:
// every row of the arrays starts on a 16-byte boundary. Both ways, 65536 tokens,
// fp32, sigmoid, bias, top 8 (in brackets softmax, top 2), in us:
// - Up to 8 choices four tokens share a warp: a warp a token spends most of its
//   instructions on what does not depend on the number of experts. With 32
//   experts 35 (29) against 53 (46), with 64 50 (43) against 58 (55).
// - Full rows have code of their own: with 32 experts 32 (25) against 35 (29),
//   with 64 41 (30) against 50 (43), with 256 76 against 100, with 512 123
//   against 179.
// - With 128 full 8 lanes take 58 (40), a warp 60 (56), not full a warp 68; with
//   256 two tokens a warp take 103 against 76.
#define VSF_FULL(F, L, N, ...)                                                           \
  (p.score == VSF_SCORE_SOFTMAX ? F<T, L, N, true, VSF_SCORE_SOFTMAX>(__VA_ARGS__)       \
                                : F<T, L, N, true, VSF_SCORE_SIGMOID>(__VA_ARGS__))
#define VSF_BY_EXPERTS(F, wide, ...)                                  \
  do {                                                                \
    if (p.K <= 8) {                                                   \
      if ((wide) && p.E == 32) return VSF_FULL(F, 8, 4, __VA_ARGS__); \
      if ((wide) && p.E == 64) return VSF_FULL(F, 8, 8, __VA_ARGS__); \
      if ((wide) && p.E == 128) return VSF_FULL(F, 8, 16, __VA_ARGS__); \
      if (p.E <= 8) return F<T, 8, 1, false, -1>(__VA_ARGS__);        \
      if (p.E <= 16) return F<T, 8, 2, false, -1>(__VA_ARGS__);       \
      if (p.E <= 32) return F<T, 8, 4, false, -1>(__VA_ARGS__);       \
      if (p.E <= 64) return F<T, 8, 8, false, -1>(__VA_ARGS__);       \
    }                                                                 \
    if ((wide) && p.E == 128) return VSF_FULL(F, 32, 4, __VA_ARGS__); \
    if ((wide) && p.E == 256) return VSF_FULL(F, 32, 8, __VA_ARGS__); \
    if ((wide) && p.E == 512) return VSF_FULL(F, 32, 16, __VA_ARGS__); \
    if (p.E <= 32) return F<T, 32, 1, false, -1>(__VA_ARGS__);        \
    if (p.E <= 64) return F<T, 32, 2, false, -1>(__VA_ARGS__);        \
    if (p.E <= 128) return F<T, 32, 4, false, -1>(__VA_ARGS__);       \
    if (p.E <= 256) return F<T, 32, 8, false, -1>(__VA_ARGS__);       \
    return F<T, 32, 16, false, -1>(__VA_ARGS__);                      \
  } while (0)

// Whether rows of T at this stride start on 16-byte boundaries.
template <typename T>
bool wide_rows(const void* p, int64_t ld) {
  return aligned(p, 16) && ld * (int64_t)sizeof(T) % 16 == 0;
}

template <typename T>
cudaError_t route_by_experts(const void* logits, const RouteIn& p, const RouteOut& o,
                             const RouteWs& w, cudaStream_t st) {
  VSF_BY_EXPERTS(route_launch, wide_rows<T>(logits, p.ld), logits, p, o, w, st);
}

template <typename T>
cudaError_t grad_by_experts(const void* logits, const RouteIn& p, const int32_t* idx,
                            const float* d_gates, const int32_t* seq_counts,
                            const float* seq_coef, float loss_scale, void* grad, int64_t grad_ld,
                            cudaStream_t st) {
  VSF_BY_EXPERTS(grad_launch, wide_rows<T>(logits, p.ld) && wide_rows<T>(grad, grad_ld), logits, p,
                 idx, d_gates, seq_counts, seq_coef, loss_scale, grad, grad_ld, st);
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
  const RouteWs w(d_workspace, E, sequences);
  const RouteIn p = route_in(T, E, ld, bias, live, seq_starts, sequences, hp);
  const RouteOut o = {idx, gates, counts, loss, seq_counts, seq_coef};
  const cudaError_t e = dtype == VSF_BF16 ? route_by_experts<uint16_t>(logits, p, o, w, st)
                                          : route_by_experts<float>(logits, p, o, w, st);
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
  const cudaError_t e =
      dtype == VSF_BF16
          ? grad_by_experts<uint16_t>(logits, p, idx, d_gates, seq_counts, seq_coef, loss_scale,
                                      grad, grad_ld, st)
          : grad_by_experts<float>(logits, p, idx, d_gates, seq_counts, seq_coef, loss_scale, grad,
                                   grad_ld, st);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, who);
}

}  // extern "C"
