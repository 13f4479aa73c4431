// row_scores.cuh — a row's log probability, entropy and top alternatives, and the
// gradient of all three. Included by objective.cu after row_regs.cuh.
//
// With z_v = (x_v - m) / temperature, s = sum_v exp(z_v), u = sum_v z_v exp(z_v):
//   ln p_v = z_v - ln s,   entropy = ln s - u / s,
//   d ln p_w / d x_v   = (1[v = w] - p_v) / temperature,
//   d entropy / d x_v  = -p_v (z_v - u / s) / temperature.
// So the gradient of a ln p_y + h entropy + sum_j b_j ln p_(top_j) is
//   (a 1[v = y] + sum_j b_j 1[v = top_j] - p_v (a + sum_j b_j + h (z_v - u / s))) / temperature.
//
// A row is cut into pieces, a warp takes a piece: {m, s, u} of its elements, and
// each lane's largest element. What a lane has of a piece is a group: there are at
// most 1024 of them in most rows, and the k largest elements lie in those groups
// whose maxima are not below the k-th largest of all groups' maxima. A second launch,
// a warp a row, joins the pieces and ranks the elements of those groups (32 times 512
// bytes at most, unless maxima are equal); where equal ones are too many, it goes
// through the whole row.
//
// m is a reference for the exponents, not the maximum: the largest of a lane's first
// vectors, moved only where an element lies 16 units of ln 2 above it. A sum's terms
// then reach 2^23 at most, and no lane waits for another.

// Order of floats as whole numbers: -0 as 0; 0 is left for "no element".
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((int32_t)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((int32_t)k < 0 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(~0u, v); }

constexpr int kScoreThreads = 256;
constexpr int kScoreCtas = 4;        // an SM (gradient)
constexpr int kPartCtas = 3;         // an SM (sums)
constexpr int kScoreBatch = 4;       // vectors of a lane on their way at a time
constexpr int kMaxTop = 32;

// How rows are cut: `spans` of 32 vectors, pieces of 2^piece spans. The elements in
// front of a row's first 16-byte boundary belong to the first piece, those behind
// the last vector to the last.
struct ScoreCut {
  int32_t spans, piece, pieces;
};

template <typename T>
struct ScoreArgs {
  Rows<T> r;  // (a row is live where target >= 0)
  ScoreCut cut;
  int32_t K;
  float4* part;    // [T, pieces] m, s, u (in units of ln 2), -
  uint32_t* keys;  // [T, pieces, 32] of the lanes' maxima, written where K > 0
  float *logp, *entropy, *top_logp;
  float4* norm;    // [T] m, s, u / s, -
  int32_t* top_idx;
  WsHead* head;
};

// exp2 terms of a pair: z in units of ln 2, kept from -inf (whose term is 0, but
// whose product with it would be NaN); NaN goes through.
__device__ __forceinline__ void score_terms(F2 x, F2 nm, const PairScale& c, F2& z, F2& e) {
  const F2 d = f2_add(x, nm);
  float a, b;
  f2_get(f2_fma(d, c.hi, f2_mul(d, c.lo)), a, b);
  asm("max.NaN.f32 %0, %1, 0fC3480000;" : "=f"(a) : "f"(a));  // -200
  asm("max.NaN.f32 %0, %1, 0fC3480000;" : "=f"(b) : "f"(b));
  z = f2(a, b);
  e = f2(ex2(a), ex2(b));
}

// In the sums the same is reached by raising the logits themselves to a floor 200
// units of ln 2 below the maximum (or the next smaller logit, where they are that
// far apart), whose term is 0 as well: one instruction for two bf16 logits. Not
// where that floor is out of range (`far`: maxima next to the type's lowest value,
// inverse temperatures below 2^-110) or its z could be (above 64).
__device__ __forceinline__ bool far_temperature(float inv_t) { return inv_t < 7.7e-34f || inv_t > 64.f; }
__device__ __forceinline__ uint32_t score_floor(float m, float units, uint16_t) {
  const uint32_t f = __bfloat16_as_ushort(__float2bfloat16_rd(__fsub_rd(m, units)));
  return f | f << 16;
}
__device__ __forceinline__ uint32_t score_floor(float m, float units, float) {
  return __float_as_uint(__fsub_rd(m, units));
}
__device__ __forceinline__ uint32_t raised(uint32_t w, uint32_t floor, uint16_t) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(floor));
  return r;
}
__device__ __forceinline__ uint32_t raised(uint32_t w, uint32_t floor, float) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(w)), "f"(__uint_as_float(floor)));
  return __float_as_uint(r);
}

// What a lane has of a piece.
template <typename T>
struct ScoreSums {
  float m = -INFINITY, most = -INFINITY;  // the reference; where it is moved
  F2 nm = f2(0.f, 0.f);
  uint32_t floor;
  F2 sum0 = f2(0.f, 0.f), sum1 = f2(0.f, 0.f), zum0 = f2(0.f, 0.f), zum1 = f2(0.f, 0.f);
  __device__ __forceinline__ ScoreSums(float units) : floor(score_floor(0.f, units, T())) {}
  // bm: the largest of the elements to be added; units: 200 units of ln 2
  __device__ __forceinline__ void to(float bm, Log2Scale c, float units) {
    if (!(bm > most)) return;
    if (m != -INFINITY) {
      const float d = fmaxf(__fmaf_rn(m - bm, c.hi, (m - bm) * c.lo), -1e20f), f = ex2(d);
      const F2 dd = f2(d, d), ff = f2(f, f);
      zum0 = f2_mul(f2_fma(sum0, dd, zum0), ff);
      zum1 = f2_mul(f2_fma(sum1, dd, zum1), ff);
      sum0 = f2_mul(sum0, ff);
      sum1 = f2_mul(sum1, ff);
    }
    m = bm;
    most = __fmaf_rn(units, 0.08f, m);
    nm = f2(-m, -m);
    floor = score_floor(m, units, T());
  }
  __device__ __forceinline__ bool out_of_range() const { return floor == Vec<T>::lowest; }
  // c: this thread's factor, rounded down or up (Log2Scale)
  template <bool FAR>
  __device__ __forceinline__ void add(const uint4& v, F2 c) {
    Pairs<T> q;
    if (FAR)
      unpack(v, q);
    else
      unpack(make_uint4(raised(v.x, floor, T()), raised(v.y, floor, T()), raised(v.z, floor, T()),
                        raised(v.w, floor, T())), q);
#pragma unroll
    for (int i = 0; i < Vec<T>::n / 2; ++i) {
      const F2 t = f2_mul(f2_add(q.p[i], nm), c);
      float a, b;
      f2_get(t, a, b);
      if (FAR) {
        asm("max.NaN.f32 %0, %1, 0fC3480000;" : "=f"(a) : "f"(a));
        asm("max.NaN.f32 %0, %1, 0fC3480000;" : "=f"(b) : "f"(b));
      }
      const F2 z = f2(a, b), e = f2(ex2(a), ex2(b));
      if (i & 1) {
        sum1 = f2_add(sum1, e);
        zum1 = f2_fma(z, e, zum1);
      } else {
        sum0 = f2_add(sum0, e);
        zum0 = f2_fma(z, e, zum0);
      }
    }
  }
};

// {m, s, u} of a piece and its lanes' keys; a warp a piece. Two batches of loads
// are on their way at a time. (A ring of bulk copies for each warp, across pieces, took
// 14 instructions an element instead of 9 and 227 us instead of 188 for 4096 x 131072
// bf16, 3/4 live, with 20 alternatives.)
template <typename T>
__global__ void __launch_bounds__(kScoreThreads, kPartCtas)
    score_part_kernel(const __grid_constant__ ScoreArgs<T> a) {
  constexpr int VE = Vec<T>::n, B = kScoreBatch;
  const int lane = threadIdx.x & 31;
  const Rows<T>& r = a.r;
  const float c1 = (uint32_t)threadIdx.x * 2654435769u < r.c.ups ? r.c.up : r.c.hi;
  const F2 cc = f2(c1, c1);
  const bool far = far_temperature(r.inv_tf);
  const float units = 200.f / r.c.hi;
  take_turn();
  const int32_t pieces = a.cut.pieces;
  const int64_t step = (int64_t)gridDim.x * (kScoreThreads / 32);
  const int64_t step_t = step / pieces, first = (int64_t)blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
  const int32_t step_p = (int32_t)(step - step_t * pieces);
  int64_t t = first / pieces;
  int32_t p = (int32_t)(first - t * pieces);
  for (; t < r.T_; t += step_t, p += step_p) {
    if (p >= pieces) {
      p -= pieces;
      if (++t >= r.T_) break;
    }
    if (live_target(r, t, p == 0 ? &a.head->err : nullptr) < 0) continue;
    const T* x = r.x + t * r.ld;
    const Span s = span_of(x, r.V);
    const uint4* in = reinterpret_cast<const uint4*>(x + s.head) + lane;
    const int32_t v0 = (p << a.cut.piece) * 32, v1 = min(v0 + (32 << a.cut.piece), s.nvec);
    ScoreSums<T> sums(units);
    float top = -INFINITY;
    int32_t v = v0;
    if (!far && v + 32 * B <= v1) {
      // whole batches, by turns in two sets of registers
      uint4 q0[B], q1[B];
      auto load = [&](uint4 (&q)[B], int32_t at) {
#pragma unroll
        for (int j = 0; j < B; ++j) q[j] = __ldcs(in + at + 32 * j);
      };
      auto add = [&](const uint4 (&q)[B]) -> bool {
        const float bm = largest(q, T());
        top = fmaxf(top, bm);
        sums.to(bm, r.c, units);
        if (__any_sync(~0u, sums.out_of_range())) return false;
#pragma unroll
        for (int j = 0; j < B; ++j) sums.template add<false>(q[j], cc);
        v += 32 * B;
        return true;
      };
      load(q0, v);
      while (true) {
        const bool more1 = v + 64 * B <= v1;
        if (more1) load(q1, v + 32 * B);
        if (!add(q0) || !more1) break;
        const bool more0 = v + 64 * B <= v1;
        if (more0) load(q0, v + 32 * B);
        if (!add(q1) || !more0) break;
      }
    }
#pragma unroll 1
    for (; v < v1; v += 32) {  // less than a batch, or what is out of range
      uint4 q[1] = {make_uint4(Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest)};
      if (v + lane < v1) q[0] = __ldcs(in + v);
      const float bm = largest(q, T());
      top = fmaxf(top, bm);
      sums.to(bm, r.c, units);
      sums.template add<true>(q[0], cc);
    }
    if (a.K > 0) a.keys[(t * pieces + p) * 32 + lane] = v0 + lane < v1 ? order_key(top) : 0;
    if (p == 0 || p + 1 == pieces) {
      // the loose elements, in front of the vectors and behind them
      const int32_t tail = s.head + s.nvec * VE;
      int32_t loose = -1;
      if (p == 0 && lane < s.head) loose = lane;
      if (p + 1 == pieces && lane >= 16 && lane - 16 < r.V - tail) loose = tail + (lane - 16);
      if (loose >= 0) {
        const float xl = to_f(x[loose]);
        sums.to(xl, r.c, units);
        const PairScale c2 = {f2(r.c.hi, r.c.hi), f2(r.c.lo, r.c.lo)};
        const float z = -finite_max(sums.m);
        F2 zz, ee;
        score_terms(f2(xl, -INFINITY), f2(z, z), c2, zz, ee);
        sums.sum0 = f2_add(sums.sum0, ee);
        sums.zum0 = f2_fma(zz, ee, sums.zum0);
      }
    }
    // the lanes' join, by expf (see the join of the losses' sums)
    float s0, s1, s2, s3, u0, u1, u2, u3;
    f2_get(sums.sum0, s0, s1);
    f2_get(sums.sum1, s2, s3);
    f2_get(sums.zum0, u0, u1);
    f2_get(sums.zum1, u2, u3);
    const float m = warp_max(sums.m), d = sums.m - finite_max(m), f = expf(d * r.inv_tf);
    const float own = (s0 + s1) + (s2 + s3);
    const float shift = fmaxf(__fmaf_rn(d, r.c.hi, d * r.c.lo), -1e20f);
    const float sum = warp_sum(own == 0.f ? 0.f : f * own);
    const float zum = warp_sum(own == 0.f ? 0.f : f * __fmaf_rn(own, shift, (u0 + u1) + (u2 + u3)));
    if (lane == 0) a.part[t * pieces + p] = make_float4(m, sum, zum, 0.f);
  }
}

// The best of a warp's candidates: larger key first, then lower index. Lane i of
// the list holds the i-th best.
struct Best {
  uint32_t key;
  int32_t idx;
};
__device__ __forceinline__ bool in_front(uint32_t key, int32_t idx, const Best& b) {
  return key > b.key || (key == b.key && idx < b.idx);
}
__device__ __forceinline__ void insert(Best& list, uint32_t key, int32_t idx, int lane) {
  const int at = __popc(__ballot_sync(~0u, !in_front(key, idx, list)));
  const uint32_t k = __shfl_up_sync(~0u, list.key, 1);
  const int32_t i = __shfl_up_sync(~0u, list.idx, 1);
  if (lane == at) list = {key, idx};
  else if (lane > at) list = {k, i};
}

// The K best of n entries in shared memory, in any order, into lanes 0 .. K-1: each
// entry's place is the number of those in front of it. A lane without one gets {0, -1}.
__device__ __forceinline__ Best best_of(const Best* list, int n, int K, Best* out, int lane) {
  out[lane] = {0, -1};
  __syncwarp();
  for (int i0 = 0; i0 < n; i0 += 32) {
    const Best own = i0 + lane < n ? list[i0 + lane] : Best{0, INT32_MAX};
    int at = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const Best b = list[j];
      at += in_front(b.key, b.idx, own);
    }
    if (i0 + lane < n && at < K) out[at] = own;
  }
  __syncwarp();
  return out[lane];
}

// The K best of a whole row, in its order: where equal elements are too many to be
// gathered. Once the list has K elements, a later one belongs to it only if it is
// larger than the K-th, so most vectors cost their load and their maximum.
template <typename T>
__device__ __noinline__ Best best_of_row(const T* x, int32_t V, int K, int lane) {
  constexpr int VE = Vec<T>::n, B = 4;
  Best list = {0, INT32_MAX};
  // the elements k[] of the lanes, a lane's from index `base` on; 0: none
  auto take = [&](uint32_t (&k)[VE], int32_t base) {
    while (true) {
      uint32_t mine = 0;
      int32_t which = 0;
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (k[e] > mine) {
          mine = k[e];
          which = e;
        }
      const uint32_t last = __shfl_sync(~0u, list.key, K - 1);
      const uint32_t top = warp_max(mine > last ? mine : 0u);
      if (top == 0) break;
      const int from = __ffs(__ballot_sync(~0u, mine == top)) - 1;
      insert(list, top, __shfl_sync(~0u, base + which, from), lane);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (lane == from && e == which) k[e] = 0;
    }
  };
  const Span s = span_of(x, V);
  const int32_t tail = s.head + s.nvec * VE;
  uint32_t k[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) k[e] = 0;
  if (lane < s.head) k[0] = order_key(to_f(x[lane]));
  take(k, lane);
  const uint4* in = reinterpret_cast<const uint4*>(x + s.head);
  for (int32_t v = 0; v < s.nvec; v += 32 * B) {
    uint4 q[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      q[j] = make_uint4(Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest);
      if (v + 32 * j + lane < s.nvec) q[j] = in[v + 32 * j + lane];
    }
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int32_t at = v + 32 * j + lane;
      const uint4 one[1] = {q[j]};
      const uint32_t last = __shfl_sync(~0u, list.key, K - 1);
      if (!__any_sync(~0u, at < s.nvec && order_key(largest(one, T())) > last)) continue;
      Pairs<T> pr;
      unpack(q[j], pr);
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) {
        float f0, f1;
        f2_get(pr.p[e], f0, f1);
        k[2 * e] = at < s.nvec ? order_key(f0) : 0;
        k[2 * e + 1] = at < s.nvec ? order_key(f1) : 0;
      }
      take(k, s.head + at * VE);
    }
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) k[e] = 0;
  if (lane < V - tail) k[0] = order_key(to_f(x[tail + lane]));
  take(k, tail + lane);
  return list;
}

// Joins a row's pieces and picks its alternatives; a warp a row.
constexpr int kScoreCandidates = 128;
template <typename T>
__global__ void __launch_bounds__(kScoreThreads)
    score_row_kernel(const __grid_constant__ ScoreArgs<T> a) {
  constexpr int VE = Vec<T>::n, W = kScoreThreads / 32, C = kScoreCandidates;
  __shared__ Best groups[W][C];
  __shared__ Best elements[W][C];
  __shared__ Best sorted[W][32];
  __shared__ int32_t counts[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Rows<T>& r = a.r;
  take_turn();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.head->rows = 1;
  const int64_t t = (int64_t)blockIdx.x * W + warp;
  if (t >= r.T_) return;
  const int32_t y = live_target(r, t, nullptr);
  if (y < 0) {
    if (lane == 0) {
      a.logp[t] = 0.f;
      a.entropy[t] = 0.f;
      a.norm[t] = make_float4(0.f, 1.f, 0.f, 0.f);
    }
    if (lane < a.K) {
      a.top_idx[t * a.K + lane] = -1;
      a.top_logp[t * a.K + lane] = 0.f;
    }
    return;
  }
  const T* x = r.x + t * r.ld;
  const float xy = to_f(x[y]);
  // ---- each lane's largest key of the groups lane, lane + 32, ...
  const int32_t n_keys = a.cut.pieces * 32;
  const uint32_t* keys = a.keys + t * n_keys + lane;
  uint32_t best = 0;
  if (a.K > 0) {
#pragma unroll 8
    for (int32_t g = 0; g < n_keys; g += 32) best = max(best, keys[g]);
  }
  // ---- the pieces
  float m = -INFINITY, sum = 0.f, zum = 0.f;
  const float4* part = a.part + t * a.cut.pieces;
  for (int32_t p = lane; p < a.cut.pieces; p += 32) m = fmaxf(m, part[p].x);
  m = warp_max(m);
  for (int32_t p = lane; p < a.cut.pieces; p += 32) {
    const float4 q = part[p];
    if (q.y == 0.f) continue;  // (nothing but -inf; a NaN goes on)
    const float d0 = q.x - finite_max(m);
    const float d = fmaxf(__fmaf_rn(d0, r.c.hi, d0 * r.c.lo), -1e20f);
    const float f = expf(d0 * r.inv_tf);
    sum += f * q.y;
    zum += f * __fmaf_rn(q.y, d, q.z);
  }
  sum = warp_sum(sum);
  zum = warp_sum(zum);
  const LogSum ls = log_sum(sum);
  const float mean = zum / sum * 0.693147181f;  // of z, by p
  if (lane == 0) {
    a.logp[t] = log_ratio(xy - m, r.inv_tf, 0.f, ls);
    a.entropy[t] = __fmaf_rn(ls.k, 0.693359375f, __fmaf_rn(ls.k, -2.12194440e-4f, ls.f) - mean);
    a.norm[t] = make_float4(m, sum, mean, 0.f);
  }
  if (a.K == 0) return;
  if (!(sum > 0.f && sum < INFINITY)) {  // a NaN, a +inf or only -inf
    if (lane < a.K) {
      a.top_idx[t * a.K + lane] = -1;
      a.top_logp[t * a.K + lane] = NAN;
    }
    return;
  }
  // ---- the groups that count. The K-th largest of the lanes' largest keys is not
  // above the K-th largest key: groups below it are left out, the others ranked.
  int before = 0;
#pragma unroll
  for (int l = 0; l < 32; ++l) {
    const uint32_t k = __shfl_sync(~0u, best, l);
    before += k > best || (k == best && l < lane);
  }
  const uint32_t least =
      max(1u, __shfl_sync(~0u, best, __ffs(__ballot_sync(~0u, before == a.K - 1)) - 1));
  int n_groups = 0;
  for (int32_t g = 0; g < n_keys; g += 32) {
    const uint32_t k = keys[g];
    const uint32_t in = __ballot_sync(~0u, k >= least);
    const int to = n_groups + __popc(in & ((1u << lane) - 1));
    if (k >= least && to < C) groups[warp][to] = {k, g + lane};
    n_groups += __popc(in);
  }
  __syncwarp();
  Best list = {0, -1};
  bool whole = n_groups > C;
  if (!whole) {
    const uint32_t last = __shfl_sync(~0u, best_of(groups[warp], n_groups, a.K, sorted[warp], lane).key, a.K - 1);
    const float low = last == 0 ? -INFINITY : key_value(last);
    // ---- their elements that are not below the K-th group's maximum, and the loose ones
    const Span s = span_of(x, r.V);
    const int32_t tail = s.head + s.nvec * VE;
    if (lane == 0) counts[warp] = 0;
    __syncwarp();
    auto gather = [&](float v, int32_t idx) {
      if (v >= low) {
        const int to = atomicAdd(&counts[warp], 1);
        if (to < C) elements[warp][to] = {order_key(v), idx};
      }
    };
    if (lane < s.head) gather(to_f(x[lane]), lane);
    if (lane < r.V - tail) gather(to_f(x[tail + lane]), tail + lane);
    const uint4* in = reinterpret_cast<const uint4*>(x + s.head);
    const int log = a.cut.piece;  // a group has 2^log vectors
    const int64_t n_vecs = (int64_t)n_groups << log;
    constexpr int B = 4;
    for (int64_t i0 = lane; i0 < n_vecs; i0 += 32 * B) {
      uint4 q[B];
      int32_t at[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int64_t i = i0 + 32 * j;
        at[j] = -1;
        if (i >= n_vecs) continue;
        const Best g = groups[warp][i >> log];
        if (g.key < last) continue;
        const int32_t v = ((((g.idx >> 5) << log) + (int32_t)(i & ((1 << log) - 1))) << 5) + (g.idx & 31);
        if (v >= s.nvec) continue;
        at[j] = v;
        q[j] = in[v];
      }
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (at[j] < 0) continue;
        const uint4 one[1] = {q[j]};
        if (!(largest(one, T()) >= low)) continue;
        Pairs<T> pr;
        unpack(q[j], pr);
        const int32_t base = s.head + at[j] * VE;
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) {
          float f0, f1;
          f2_get(pr.p[e], f0, f1);
          gather(f0, base + 2 * e);
          gather(f1, base + 2 * e + 1);
        }
      }
    }
    __syncwarp();
    const int found = counts[warp];
    whole = found > C;
    if (!whole) list = best_of(elements[warp], found, a.K, sorted[warp], lane);
  }
  if (whole) list = best_of_row(x, r.V, a.K, lane);
  if (lane < a.K) {
    a.top_idx[t * a.K + lane] = list.idx;
    a.top_logp[t * a.K + lane] = log_ratio(key_value(list.key) - m, r.inv_tf, 0.f, ls);
  }
}

// ------------------------------------------------------------- the gradient
template <typename T>
struct ScoreGradArgs {
  Rows<T> r;
  ScoreCut cut;
  int32_t K;
  const float4* norm;
  const int32_t* top_idx;
  const float *d_logp, *d_entropy, *d_top;  // each may be NULL
  T* grad;
  int64_t grad_ld;
};

// A warp a piece of a row, as in the sums.
template <typename T>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtas)
    score_grad_kernel(const __grid_constant__ ScoreGradArgs<T> a) {
  constexpr int VE = Vec<T>::n, B = kScoreBatch;
  const int lane = threadIdx.x & 31;
  const Rows<T>& r = a.r;
  const PairScale c2 = {f2(r.c.hi, r.c.hi), f2(r.c.lo, r.c.lo)};
  take_turn();
  const int32_t pieces = a.cut.pieces;
  const int64_t step = (int64_t)gridDim.x * (kScoreThreads / 32);
  const int64_t step_t = step / pieces, first = (int64_t)blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
  const int32_t step_p = (int32_t)(step - step_t * pieces);
  int64_t t = first / pieces;
  int32_t p = (int32_t)(first - t * pieces);
  for (; t < r.T_; t += step_t, p += step_p) {
    if (p >= pieces) {
      p -= pieces;
      if (++t >= r.T_) break;
    }
    const int32_t y = live_target(r, t, nullptr);
    const T* x = r.x + t * r.ld;
    T* g = a.grad + t * a.grad_ld;
    // what a lane writes is counted from the gradient's 16-byte boundaries
    const Span s = span_of(g, r.V);
    const int32_t v0 = (p << a.cut.piece) * 32;
    const int32_t v1 = p + 1 == pieces ? s.nvec : min(v0 + (32 << a.cut.piece), s.nvec);
    const int32_t tail = s.head + s.nvec * VE;
    int32_t loose = -1;
    if (p == 0 && lane < s.head) loose = lane;
    if (p + 1 == pieces && lane >= 16 && lane - 16 < r.V - tail) loose = tail + (lane - 16);
    uint4* out = reinterpret_cast<uint4*>(g + s.head) + lane;
    if (y < 0) {
      for (int32_t v = v0; v + lane < v1; v += 32) __stcs(out + v, make_uint4(0, 0, 0, 0));
      if (loose >= 0) g[loose] = from_f<T>(0.f);
      continue;
    }
    const float4 nm4 = a.norm[t];
    const float da = a.d_logp != nullptr ? a.d_logp[t] : 0.f;
    const float dh = a.d_entropy != nullptr ? a.d_entropy[t] : 0.f;
    const float db = lane < a.K && a.d_top != nullptr ? a.d_top[t * a.K + lane] : 0.f;
    const int32_t ti = lane < a.K && a.d_top != nullptr ? a.top_idx[t * a.K + lane] : -1;
    const float pull = da + warp_sum(db);
    const float z0 = finite_max(nm4.x);
    const float scale = -r.inv_tf / nm4.y;
    const float h = scale * dh, c0 = scale * __fmaf_rn(-dh, nm4.z, pull), h2 = h * 0.693147181f;
    // e (c0 + h z): p_v times what pulls on all elements
    auto common = [&](float v) {
      F2 z, e;
      score_terms(f2(v, v), f2(-z0, -z0), c2, z, e);
      float za, zb, ea, eb;
      f2_get(z, za, zb);
      f2_get(e, ea, eb);
      return ea * __fmaf_rn(h2, za, c0);
    };
    // The elements with a pull of their own, read before anything is written (the
    // gradient may be written over the logits): the target, by lane 0 where no
    // alternative is it, and the alternatives, an index that comes twice by its
    // first lane.
    auto here = [&](int32_t v) {  // whether this piece writes element v
      const int32_t q = v - s.head;
      if (v < 0 || v >= r.V) return false;
      if (q < 0) return p == 0;
      if (q >= s.nvec * VE) return p + 1 == pieces;
      return q / VE >= v0 && q / VE < v1;
    };
    const bool my = here(ti);
    const uint32_t marked = __ballot_sync(~0u, my);
    float own = 0.f, xt = 0.f;
    bool first_of = my;
    if (marked != 0) {
      for (uint32_t left = marked; left != 0; left &= left - 1) {
        const int j = __ffs(left) - 1;
        const float bj = __shfl_sync(~0u, db, j);
        if (__shfl_sync(~0u, ti, j) == ti) {
          own += bj;
          if (j < lane) first_of = false;
        }
      }
      if (ti == y) own += da;
      if (my) xt = to_f(x[ti]);
    }
    const bool target = here(y) && __ballot_sync(~0u, my && ti == y) == 0;
    float xy = 0.f;
    if (target && lane == 0) xy = to_f(x[y]);
    float xl = 0.f;
    if (loose >= 0) xl = to_f(x[loose]);
    __syncwarp();
    const F2 nz = f2(-z0, -z0), c02 = f2(c0, c0), h22 = f2(h2, h2);
    if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0) {
      const uint4* in = reinterpret_cast<const uint4*>(x + s.head) + lane;
      for (int32_t v = v0; v < v1; v += 32 * B) {
        uint4 q[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (v + 32 * j + lane < v1) q[j] = __ldcs(in + v + 32 * j);
#pragma unroll
        for (int j = 0; j < B; ++j) {
          if (v + 32 * j + lane >= v1) break;
          Pairs<T> w;
          unpack(q[j], w);
          float o[VE];
#pragma unroll
          for (int i = 0; i < VE / 2; ++i) {
            F2 z, e;
            score_terms(w.p[i], nz, c2, z, e);
            f2_get(f2_mul(e, f2_fma(h22, z, c02)), o[2 * i], o[2 * i + 1]);
          }
          __stcs(out + v + 32 * j, pack_vec<T>(o));
        }
      }
    } else {
      const int32_t e1 = v1 * VE;
      for (int32_t e = v0 * VE + lane; e < e1; e += 32) g[s.head + e] = from_f<T>(common(to_f(x[s.head + e])));
    }
    if (loose >= 0) g[loose] = from_f<T>(common(xl));
    __syncwarp();
    if (first_of) g[ti] = from_f<T>(__fmaf_rn(r.inv_tf, own, common(xt)));
    if (target && lane == 0) g[y] = from_f<T>(__fmaf_rn(r.inv_tf, da, common(xy)));
  }
}
