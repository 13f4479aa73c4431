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
// the largest element of each of its groups of consecutive elements (a group is
// what one load instruction of the warp covers, 512 bytes, more only in rows that
// have over 1000 of them). A second launch, a warp a row, joins the pieces and
// picks the alternatives: the k largest elements (ties to the lowest index) lie in
// the k groups of largest maxima (ties to the lowest group). For were one of them
// in another group, each of those k groups would hold an element in front of it.
// So it reads 512 k bytes of the row again, whatever the logits are.

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
constexpr int kScoreCtas = 4;        // an SM
constexpr int kScoreBatch = 4;       // vectors of a lane on their way at a time
constexpr int kMaxGroupsRow = 1024;  // groups of a row, its loose elements among them
constexpr int kMaxTop = 32;

// How rows are cut: `spans` of 32 vectors, pieces of 2^piece spans, groups of
// 2^group. Group 0 are the elements in front of the first vector, the last one
// those behind the last vector.
struct ScoreCut {
  int32_t spans, piece, group;
  int32_t pieces, groups;
};

template <typename T>
struct ScoreArgs {
  Rows<T> r;  // (a row is live where target >= 0)
  ScoreCut cut;
  int32_t K;
  float4* part;    // [T, pieces] m, s, u (in units of ln 2), -
  uint32_t* keys;  // [T, groups], written where K > 0
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

// {m, s, u} of a piece and its groups' keys; a warp a piece.
template <typename T>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtas)
    score_part_kernel(const __grid_constant__ ScoreArgs<T> a) {
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
    if (live_target(r, t, p == 0 ? &a.head->err : nullptr) < 0) continue;
    const T* x = r.x + t * r.ld;
    const Span s = span_of(x, r.V);
    const uint4* in = reinterpret_cast<const uint4*>(x + s.head) + lane;
    uint32_t* keys = a.K > 0 ? a.keys + t * a.cut.groups : nullptr;
    const int32_t span0 = p << a.cut.piece, span1 = min(span0 + (1 << a.cut.piece), a.cut.spans);
    float m = -INFINITY;
    F2 sum0 = f2(0.f, 0.f), sum1 = sum0, zum0 = sum0, zum1 = sum0;
    auto raise = [&](float bm) {  // a new maximum, the same in all lanes
      if (!(bm > m)) return;
      if (m != -INFINITY) {
        const float d = fmaxf(__fmaf_rn(m - bm, r.c.hi, (m - bm) * r.c.lo), -1e20f), f = ex2(d);
        const F2 f2d = f2(d, d), ff = f2(f, f);
        zum0 = f2_mul(f2_fma(sum0, f2d, zum0), ff);
        zum1 = f2_mul(f2_fma(sum1, f2d, zum1), ff);
        sum0 = f2_mul(sum0, ff);
        sum1 = f2_mul(sum1, ff);
      }
      m = bm;
    };
    // the loose elements, in front of the vectors (first piece) and behind them (last)
    const int32_t tail = s.head + s.nvec * VE;
    int32_t loose = -1;
    if (p == 0 && lane < s.head) loose = lane;
    if (p + 1 == pieces && lane >= 16 && lane - 16 < r.V - tail) loose = tail + (lane - 16);
    if (p == 0 || p + 1 == pieces) {
      const float xl = loose >= 0 ? to_f(x[loose]) : -INFINITY;
      if (keys != nullptr) {
        const uint32_t k = loose >= 0 ? order_key(xl) : 0;
        const uint32_t front = warp_max(lane < 16 ? k : 0), back = warp_max(lane < 16 ? 0 : k);
        if (lane == 0 && p == 0) keys[0] = front;
        if (lane == 0 && p + 1 == pieces) keys[a.cut.groups - 1] = back;
      }
      raise(warp_max(xl));
      F2 z, e;
      const float nm = -finite_max(m);
      score_terms(f2(xl, xl), f2(nm, nm), c2, z, e);
      float z0, z1, e0, e1;
      f2_get(z, z0, z1);
      f2_get(e, e0, e1);
      if (loose >= 0) {
        sum0 = f2(e0, 0.f);
        zum0 = f2(z0 * e0, 0.f);
      }
    }
    uint32_t group_key = 0;
    for (int32_t b = span0; b < span1; b += B) {
      uint4 v[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        v[j] = make_uint4(Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest);
        const int32_t at = (b + j) * 32;
        if (b + j < span1 && at + lane < s.nvec) v[j] = __ldcs(in + at);
      }
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const uint4 one[1] = {v[j]};
        const float gm = warp_max(largest(one, T()));
        top = fmaxf(top, gm);
        if (keys != nullptr && b + j < span1) {
          group_key = max(group_key, (b + j) * 32 < s.nvec ? order_key(gm) : 0u);
          const int32_t next = b + j + 1;
          if ((next & ((1 << a.cut.group) - 1)) == 0 || next == a.cut.spans) {
            if (lane == 0) keys[1 + (b + j >> a.cut.group)] = group_key;
            group_key = 0;
          }
        }
      }
      raise(top);
      const float z = -finite_max(m);
      const F2 nm = f2(z, z);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        Pairs<T> q;
        unpack(v[j], q);
#pragma unroll
        for (int i = 0; i < VE / 2; i += 2) {
          F2 z0, e0, z1, e1;
          score_terms(q.p[i], nm, c2, z0, e0);
          score_terms(q.p[i + 1], nm, c2, z1, e1);
          sum0 = f2_add(sum0, e0);
          sum1 = f2_add(sum1, e1);
          zum0 = f2_fma(z0, e0, zum0);
          zum1 = f2_fma(z1, e1, zum1);
        }
      }
    }
    float s0, s1, s2, s3, u0, u1, u2, u3;
    f2_get(sum0, s0, s1);
    f2_get(sum1, s2, s3);
    f2_get(zum0, u0, u1);
    f2_get(zum1, u2, u3);
    const float sum = warp_sum((s0 + s1) + (s2 + s3)), zum = warp_sum((u0 + u1) + (u2 + u3));
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

// Joins a row's pieces and picks its alternatives; a warp a row.
template <typename T>
__global__ void __launch_bounds__(kScoreThreads)
    score_row_kernel(const __grid_constant__ ScoreArgs<T> a) {
  constexpr int VE = Vec<T>::n, NG = kMaxGroupsRow / 32;
  const int lane = threadIdx.x & 31;
  const Rows<T>& r = a.r;
  take_turn();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.head->rows = 1;
  const int64_t t = (int64_t)blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
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
  // ---- the K groups of largest maxima; lane i holds the i-th
  const uint32_t* keys = a.keys + t * a.cut.groups;
  uint32_t key[NG];
  uint32_t best = 0;
  int32_t at = 0;
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    key[j] = 0;
    if (j * 32 >= a.cut.groups) continue;
    if (j * 32 + lane < a.cut.groups) key[j] = keys[j * 32 + lane];
    if (key[j] > best) {
      best = key[j];
      at = j;
    }
  }
  Best group = {0, -1};
  for (int i = 0; i < a.K; ++i) {
    const uint32_t top = warp_max(best);
    if (top == 0) break;  // fewer groups than that
    const int32_t g = (int32_t)__reduce_min_sync(~0u, best == top ? (uint32_t)(at * 32 + lane) : ~0u);
    if (lane == i) group = {top, g};
    if (lane == (g & 31)) {
      best = 0;
      const int32_t out = at;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if (j * 32 >= a.cut.groups) continue;
        if (j == out) key[j] = 0;
        if (key[j] > best) {
          best = key[j];
          at = j;
        }
      }
    }
  }
  // ---- their elements. None below the last group's maximum is among the K.
  const Span s = span_of(x, r.V);
  const uint4* in = reinterpret_cast<const uint4*>(x + s.head) + lane;
  const int32_t tail = s.head + s.nvec * VE;
  Best list = {__shfl_sync(~0u, group.key, a.K - 1), INT32_MAX};
  for (int i = 0; i < a.K; ++i) {
    const uint32_t gk = __shfl_sync(~0u, group.key, i);
    const int32_t g = __shfl_sync(~0u, group.idx, i);
    // (lanes behind the list's K are never looked at)
    if (g < 0 || gk < __shfl_sync(~0u, list.key, a.K - 1)) break;
    const bool loose = g == 0 || g + 1 == a.cut.groups;
    const int32_t v0 = loose ? 0 : (g - 1 << a.cut.group) * 32;
    const int32_t v1 = loose ? 32 : min(v0 + (32 << a.cut.group), s.nvec);
    for (int32_t v = v0; v < v1; v += 32) {
      float f[VE];
      int32_t base;
      int n = VE;  // elements of this lane
      if (loose) {
        base = (g == 0 ? 0 : tail) + lane;
        n = lane < (g == 0 ? s.head : r.V - tail) ? 1 : 0;
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = 0.f;
        if (n) f[0] = to_f(x[base]);
      } else {
        base = s.head + (v + lane) * VE;
        n = v + lane < v1 ? VE : 0;
        uint4 q = make_uint4(0, 0, 0, 0);
        if (n) q = in[v];
        Pairs<T> pr;
        unpack(q, pr);
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) f2_get(pr.p[e], f[2 * e], f[2 * e + 1]);
      }
      uint32_t k[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) k[e] = e < n ? order_key(f[e]) : 0;
      while (true) {
        uint32_t mine = 0;
        int32_t which = 0;
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (k[e] > mine) {
            mine = k[e];
            which = e;
          }
        const Best last = {__shfl_sync(~0u, list.key, a.K - 1), __shfl_sync(~0u, list.idx, a.K - 1)};
        const bool good = mine != 0 && in_front(mine, base + which, last);
        const uint32_t top = warp_max(good ? mine : 0u);
        if (top == 0) break;
        const int from = __ffs(__ballot_sync(~0u, good && mine == top)) - 1;
        insert(list, top, __shfl_sync(~0u, base + which, from), lane);
        if (lane == from) {
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (e == which) k[e] = 0;
        }
      }
    }
  }
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
