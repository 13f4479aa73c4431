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
// whose maxima are not below the k-th largest of all groups' maxima. A second launch, a
// CTA a row, joins the pieces and ranks the elements of those groups (k times 512 bytes
// or little more, unless maxima are equal); where equal ones are too many, it goes
// through the whole row. Few rows take one launch for both, a CTA a row.
//
// m is a reference for the exponents, not the maximum: the largest of a lane's first
// vectors, moved only where an element lies more than 16 units of ln 2 above it (that
// border rounded down to a float). A sum's terms then reach 2^16 at most, and no lane
// waits for another.
//
// Measured (GB300): the sums of 4096 x 131072 bf16, 3/4 live, take 125 us, 95 percent
// of the copy rate, bound by HBM with 62 percent of the issue slots in use (7.5
// instructions an element); 5, 20 and 32 alternatives add 10, 26 and 40 us, bound by a
// row's chain of loads and ranks, some 3700 instructions. The gradient reads and writes
// 4096 x 32000 in 76 us, 89 percent of the copy rate. Measured and not kept: a row
// finished by the warp that is done last with it (a fence and a count a piece: 270 us
// without alternatives, 890 with 20); chunks of rows whose launches overlap (168 us in
// two, 188 in four, against 155); groups of 64 or 32 bytes side by side, read with
// 32-byte loads (sums 130 us instead of 125, all with 20 alternatives 148 or 151
// instead of 151).

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
constexpr int kPartCtas = 3;         // an SM
constexpr int kScoreBatch = 4;       // vectors of a lane on their way at a time
constexpr int kMaxTop = 32;

// How rows are cut: spans of 32 vectors, `pieces` of 2^piece spans. The elements in
// front of a row's first 16-byte boundary belong to the first piece, those behind
// the last vector to the last.
struct ScoreCut {
  int32_t piece, pieces;
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
  // bm: the largest of the elements to be added; units: ScoreLane's
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
    most = __fmaf_rd(units, 0.08f, m);
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

// What the sums of a launch's rows have in common.
struct ScoreLane {
  F2 cc;  // this thread's factor, rounded down or up (Log2Scale)
  // 200 units of ln 2; less where inverse temperatures are below 2^-120, so that a
  // twelfth of them above the lowest logit is in range
  float units;
  bool far;
  __device__ __forceinline__ ScoreLane(const Log2Scale& c, float inv_t)
      : units(fminf(200.f / c.hi, 2.1e38f)), far(far_temperature(inv_t)) {
    const float c1 = (uint32_t)threadIdx.x * 2654435769u < c.ups ? c.up : c.hi;
    cc = f2(c1, c1);
  }
};

// A piece of a row, and where its vectors lie.
template <typename T>
struct Piece {
  const uint4* in = nullptr;  // the row's first vector, and this lane's offset
  int64_t t = -1;
  int32_t p = 0, head = 0, v = 0, v1 = 0;
  __device__ __forceinline__ bool whole(bool far) const { return !far && v + 32 * kScoreBatch <= v1; }
  __device__ __forceinline__ void load(uint4 (&q)[kScoreBatch], int32_t at) const {
#pragma unroll
    for (int j = 0; j < kScoreBatch; ++j) q[j] = __ldcs(in + at + 32 * j);
  }
  // with its first vectors on their way
  __device__ __forceinline__ void open(const ScoreArgs<T>& a, bool far, uint4 (&q)[kScoreBatch]) {
    const T* x = a.r.x + t * a.r.ld;
    const Span s = span_of(x, a.r.V);
    in = reinterpret_cast<const uint4*>(x + s.head) + (threadIdx.x & 31);
    head = s.head;
    v = (p << a.cut.piece) * 32;
    v1 = min(v + (32 << a.cut.piece), s.nvec);
    if (whole(far)) load(q, v);
  }
};

// {m, s, u} of a piece whose first vectors q0 holds; one warp. Two batches of loads are
// on their way at a time; ahead(key), with this lane's key, is called when the last
// of them have been added, and may open the next piece in their place.
template <typename T, typename Ahead>
__device__ __forceinline__ float4 piece_sums(const ScoreArgs<T>& a, const ScoreLane& c, Piece<T>& piece,
                                             uint4 (&q0)[kScoreBatch], Ahead ahead) {
  constexpr int VE = Vec<T>::n, B = kScoreBatch;
  const Rows<T>& r = a.r;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = piece.t;
  const int32_t p0 = piece.p, v0 = piece.v;
  int32_t& v = piece.v;
  const int32_t& v1 = piece.v1;
  ScoreSums<T> sums(c.units);
  float top = -INFINITY;
  if (piece.whole(c.far)) {
    // whole batches, by turns in two sets of registers
    uint4 q1[B];
    auto add = [&](const uint4 (&q)[B]) -> bool {
      const float bm = largest(q, T());
      top = fmaxf(top, bm);
      sums.to(bm, r.c, c.units);
      if (__any_sync(~0u, sums.out_of_range())) return false;
#pragma unroll
      for (int j = 0; j < B; ++j) sums.template add<false>(q[j], c.cc);
      v += 32 * B;
      return true;
    };
    while (true) {
      const bool more1 = v + 64 * B <= v1;
      if (more1) piece.load(q1, v + 32 * B);
      if (!add(q0) || !more1) break;
      const bool more0 = v + 64 * B <= v1;
      if (more0) piece.load(q0, v + 32 * B);
      if (!add(q1) || !more0) break;
    }
  }
#pragma unroll 1
  for (; v < v1; v += 32) {  // less than a batch, or what is out of range
    uint4 q[1] = {make_uint4(Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest)};
    if (v + lane < v1) q[0] = __ldcs(piece.in + v);
    const float bm = largest(q, T());
    top = fmaxf(top, bm);
    sums.to(bm, r.c, c.units);
    sums.template add<true>(q[0], c.cc);
  }
  const int32_t head0 = piece.head;
  ahead(v0 + lane < v1 ? order_key(top) : 0u);
  if (p0 == 0 || p0 + 1 == a.cut.pieces) {
    // the loose elements, in front of the vectors and behind them
    const T* x = r.x + t0 * r.ld;
    const int32_t tail = head0 + (r.V - head0) / VE * VE;
    int32_t loose = -1;
    if (p0 == 0 && lane < head0) loose = lane;
    if (p0 + 1 == a.cut.pieces && lane >= 16 && lane - 16 < r.V - tail) loose = tail + (lane - 16);
    if (loose >= 0) {
      const float xl = to_f(x[loose]);
      sums.to(xl, r.c, c.units);
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
  return make_float4(m, sum, zum, 0.f);
}

// The pieces of many rows; a warp a piece, the first vectors of the next one on their
// way while one is finished. (A ring of bulk copies for each warp, across pieces, took
// 14 instructions an element instead of 9 and 227 us instead of 188 for 4096 x 131072
// bf16, 3/4 live, with 20 alternatives.)
template <typename T>
__global__ void __launch_bounds__(kScoreThreads, kPartCtas)
    score_part_kernel(const __grid_constant__ ScoreArgs<T> a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Rows<T>& r = a.r;
  const ScoreLane c(r.c, r.inv_tf);
  take_turn();
  const int32_t pieces = a.cut.pieces, step = (int32_t)gridDim.x * (kScoreThreads / 32);
  const int32_t step_t = step / pieces, step_p = step % pieces;
  // the piece ahead and its row's target
  const int32_t first = (int32_t)blockIdx.x * (kScoreThreads / 32) + warp;
  int64_t t_next = first / pieces;
  int32_t p_next = first % pieces;
  int64_t y_next = t_next < r.T_ ? r.target[t_next] : -1;
  Piece<T> piece;
  uint4 q0[kScoreBatch];
  // to the next piece of a live row; those of masked rows are left out
  auto find = [&]() {
    while (t_next < r.T_) {
      piece.t = t_next;
      piece.p = p_next;
      const int64_t y = y_next;
      t_next += step_t;
      p_next += step_p;
      if (p_next >= pieces) {
        p_next -= pieces;
        ++t_next;
      }
      y_next = t_next < r.T_ ? r.target[t_next] : -1;
      if (y >= 0 && y < r.V) return;
      if (y >= 0 && piece.p == 0 && lane == 0) atomicOr(&a.head->err, kErrTarget);
    }
    piece.t = -1;
  };
  find();
  if (piece.t >= 0) piece.open(a, c.far, q0);
  while (piece.t >= 0) {
    const int64_t t0 = piece.t;
    const int32_t p0 = piece.p;
    const float4 part = piece_sums(a, c, piece, q0, [&](uint32_t key) {
      if (a.K > 0) a.keys[(t0 * pieces + p0) * 32 + lane] = key;
      find();
      if (piece.t >= 0) piece.open(a, c.far, q0);
    });
    if (lane == 0) a.part[t0 * pieces + p0] = part;
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

// The K best of part `part` of `parts` of a whole row, in its order: where equal
// elements are too many to be gathered. Once the list has K elements, a later one
// belongs to it only if it is larger than the K-th, so most vectors cost their load
// and their maximum. One warp; lane i holds the i-th best.
template <typename T>
__device__ __noinline__ Best best_of_part(const T* x, int32_t V, int K, int part, int parts, int lane) {
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
  if (part == 0 && lane < s.head) k[0] = order_key(to_f(x[lane]));
  take(k, lane);
  const uint4* in = reinterpret_cast<const uint4*>(x + s.head);
  const int32_t end = (int32_t)((int64_t)s.nvec * (part + 1) / parts);
  for (int32_t v = (int32_t)((int64_t)s.nvec * part / parts); v < end; v += 32 * B) {
    uint4 q[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      q[j] = make_uint4(Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest);
      if (v + 32 * j + lane < end) q[j] = in[v + 32 * j + lane];
    }
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int32_t at = v + 32 * j + lane;
      const uint4 one[1] = {q[j]};
      const uint32_t last = __shfl_sync(~0u, list.key, K - 1);
      if (!__any_sync(~0u, at < end && order_key(largest(one, T())) > last)) continue;
      Pairs<T> pr;
      unpack(q[j], pr);
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) {
        float f0, f1;
        f2_get(pr.p[e], f0, f1);
        k[2 * e] = at < end ? order_key(f0) : 0;
        k[2 * e + 1] = at < end ? order_key(f1) : 0;
      }
      take(k, s.head + at * VE);
    }
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) k[e] = 0;
  if (part + 1 == parts && lane < V - tail) k[0] = order_key(to_f(x[tail + lane]));
  take(k, tail + lane);
  return list;
}

__device__ __forceinline__ uint64_t entry(uint32_t key, int32_t idx) {
  return (uint64_t)key << 32 | (uint32_t)~idx;
}

constexpr int kRowScoreThreads = 128;  // of the row's finish
constexpr int kScoreCandidates = 128;  // groups, and elements, that are ranked
struct RowShared {
  // key and, inverted, index: the larger number is in front
  uint64_t groups[kScoreCandidates], sorted[kScoreCandidates], elements[kScoreCandidates];
  uint32_t least_of[32], last_of;
  int32_t n_groups, n_elements;
  float m, sum;
};

template <typename T>
__device__ __forceinline__ void masked_row(const ScoreArgs<T>& a, int64_t t) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    a.logp[t] = 0.f;
    a.entropy[t] = 0.f;
    a.norm[t] = make_float4(0.f, 1.f, 0.f, 0.f);
  }
  if (tid < a.K) {
    a.top_idx[t * a.K + tid] = -1;
    a.top_logp[t * a.K + tid] = 0.f;
  }
}

// Joins the pieces of row t, whose target is y, and picks its alternatives; a CTA of
// kRowScoreThreads. key: N of the row's keys each, key j * kRowScoreThreads + tid of
// them; part: the first warp's first pieces; parts: all of them.
template <int N, typename T>
__device__ __forceinline__ void finish_row(const ScoreArgs<T>& a, int64_t t, int32_t y, const uint32_t (&key)[N],
                                           float4 part, const float4* parts, RowShared& sh) {
  constexpr int VE = Vec<T>::n, C = kScoreCandidates, NT = kRowScoreThreads, W = NT / 32;
  static_assert(C == NT, "a thread ranks an entry");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Rows<T>& r = a.r;
  uint32_t best = 0;
  const T* x = r.x + t * r.ld;
  if (tid == 0) sh.n_groups = sh.n_elements = 0;
  // ---- the pieces, by the first warp
  if (warp == 0) {
    const float xy = lane == 0 ? to_f(x[y]) : 0.f;
    constexpr int NP = N / 8;  // of a lane
    float4 q[NP];
    float m = -INFINITY, sum = 0.f, zum = 0.f;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      q[j] = j == 0 ? part : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      if (j > 0 && 32 * j + lane < a.cut.pieces) q[j] = parts[32 * j + lane];
      m = fmaxf(m, q[j].x);
    }
    m = warp_max(m);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      if (q[j].y == 0.f) continue;  // (nothing but -inf; a NaN goes on)
      const float d0 = q[j].x - finite_max(m);
      const float d = fmaxf(__fmaf_rn(d0, r.c.hi, d0 * r.c.lo), -1e20f);
      const float f = expf(d0 * r.inv_tf);
      sum += f * q[j].y;
      zum += f * __fmaf_rn(q[j].y, d, q[j].z);
    }
    sum = warp_sum(sum);
    zum = warp_sum(zum);
    if (lane == 0) {
      const LogSum ls = log_sum(sum);
      const float mean = zum / sum * 0.693147181f;  // of z, by p
      a.logp[t] = log_ratio(xy - m, r.inv_tf, 0.f, ls);
      a.entropy[t] = __fmaf_rn(ls.k, 0.693359375f, __fmaf_rn(ls.k, -2.12194440e-4f, ls.f) - mean);
      a.norm[t] = make_float4(m, sum, mean, 0.f);
      sh.m = m;
      sh.sum = sum;
    }
  }
  if (a.K == 0) return;
  // ---- the groups that count. Each warp's n-th largest of its threads' largest keys,
  // n = K / W rounded up: there are K keys not below the least of them.
#pragma unroll
  for (int j = 0; j < N; ++j) best = max(best, key[j]);
  uint32_t least = 0;
  for (int i = 0; i < (a.K + W - 1) / W; ++i) {
    least = warp_max(best);
    if (lane == __ffs(__ballot_sync(~0u, best == least)) - 1) best = 0;
  }
  if (lane == 0) sh.least_of[warp] = least;
  __syncthreads();
  const float m = sh.m, sum = sh.sum;
  if (!(sum > 0.f && sum < INFINITY)) {  // a NaN, a +inf or only -inf
    if (tid < a.K) {
      a.top_idx[t * a.K + tid] = -1;
      a.top_logp[t * a.K + tid] = NAN;
    }
    return;
  }
  for (int w = 0; w < W; ++w) least = min(least, sh.least_of[w]);
  least = max(least, 1u);
  int mine = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) mine += key[j] >= least;
  int to = mine;  // entries of the warp up to this lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, to, o);
    if (lane >= o) to += v;
  }
  int first = 0;
  if (lane == 31) first = atomicAdd(&sh.n_groups, to);
  to += __shfl_sync(~0u, first, 31) - mine;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (key[j] < least) continue;
    if (to < C) sh.groups[to] = entry(key[j], j * NT + tid);
    ++to;
  }
  __syncthreads();
  // An entry's place is the number of entries in front of it, whatever their order.
  auto place = [&](const uint64_t* list, int n, uint64_t own) {
    int at = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) at += list[j] > own;
    return at;
  };
  auto put = [&](int at, uint64_t own) {
    if (at >= a.K) return;
    a.top_idx[t * a.K + at] = (int32_t)~(uint32_t)own;
    a.top_logp[t * a.K + at] = log_ratio(key_value((uint32_t)(own >> 32)) - m, r.inv_tf, 0.f, log_sum(sum));
  };
  const int ng = sh.n_groups;
  if (ng <= C) {
    if (tid == 0 && ng < a.K) sh.last_of = 0;
    if (tid < ng) {
      const uint64_t own = sh.groups[tid];
      const int at = place(sh.groups, ng, own);
      sh.sorted[at] = own;
      if (at == a.K - 1) sh.last_of = (uint32_t)(own >> 32);
    }
    __syncthreads();
    // ---- their elements that are not below the K-th group's maximum, and the loose ones
    const uint32_t last = sh.last_of;
    const int kept = __syncthreads_count(tid < ng && (uint32_t)(sh.sorted[tid] >> 32) >= last);
    const float low = last == 0 ? -INFINITY : key_value(last);
    const Span s = span_of(x, r.V);
    const int32_t tail = s.head + s.nvec * VE;
    auto gather = [&](float v, int32_t idx) {
      const int to = atomicAdd(&sh.n_elements, 1);
      if (to < C) sh.elements[to] = entry(order_key(v), idx);
    };
    if (tid < s.head && to_f(x[tid]) >= low) gather(to_f(x[tid]), tid);
    if (tid < r.V - tail && to_f(x[tail + tid]) >= low) gather(to_f(x[tail + tid]), tail + tid);
    const uint4* in = reinterpret_cast<const uint4*>(x + s.head);
    const int log = a.cut.piece;  // a group has 2^log vectors
    const int64_t n_vecs = (int64_t)kept << log;
    constexpr int B = 4;
    for (int64_t i0 = tid; i0 < n_vecs; i0 += NT * B) {
      uint4 q[B];
      int32_t at[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int64_t i = i0 + NT * j;
        at[j] = -1;
        if (i >= n_vecs) continue;
        const int32_t g = (int32_t)~(uint32_t)sh.sorted[i >> log];
        const int32_t v = ((((g >> 5) << log) + (int32_t)(i & ((1 << log) - 1))) << 5) + (g & 31);
        if (v >= s.nvec) continue;
        at[j] = v;
        q[j] = in[v];
      }
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (at[j] < 0) continue;
        Pairs<T> pr;
        unpack(q[j], pr);
        uint32_t hits = 0;
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) {
          float f0, f1;
          f2_get(pr.p[e], f0, f1);
          if (f0 >= low) hits |= 1u << (2 * e);
          if (f1 >= low) hits |= 2u << (2 * e);
        }
        for (; hits != 0; hits &= hits - 1) {
          const int32_t idx = s.head + at[j] * VE + __ffs(hits) - 1;
          gather(to_f(x[idx]), idx);
        }
      }
    }
    __syncthreads();
    const int n = sh.n_elements;
    if (n <= C) {
      if (tid < n) put(place(sh.elements, n, sh.elements[tid]), sh.elements[tid]);
      return;
    }
    __syncthreads();  // (n_elements and the lists have been read)
  }
  // ---- too many equal ones: the whole row, a part a warp
  static_assert(W * kMaxTop <= C, "the warps' lists are ranked together");
  const Best own = best_of_part(x, r.V, a.K, warp, W, lane);
  if (lane < a.K) sh.elements[warp * a.K + lane] = entry(own.key, own.idx);
  __syncthreads();
  if (tid < W * a.K && sh.elements[tid] >> 32 != 0)
    put(place(sh.elements, W * a.K, sh.elements[tid]), sh.elements[tid]);
}

// Finishes the rows whose pieces score_part_kernel has left, a CTA a row: what a call of
// 64 rows of 131072 takes longer with 20 alternatives than without is 3.5 us, with a
// warp a row it was 18, a chain of some ten loads. N: keys of a thread, 8 for up to 32
// pieces.
template <typename T, int N>
__global__ void __launch_bounds__(kRowScoreThreads, N == 8 ? 12 : 4)
    score_row_kernel(const __grid_constant__ ScoreArgs<T> a) {
  __shared__ RowShared sh;
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  take_turn();
  if (t == 0 && tid == 0) a.head->rows = 1;
  // the groups' keys and the pieces are on their way before the row is known to be live
  const int32_t n_keys = a.K > 0 ? a.cut.pieces * 32 : 0;
  const uint32_t* keys = a.keys + t * n_keys;
  const float4* parts = a.part + t * a.cut.pieces;
  uint32_t key[N];
#pragma unroll
  for (int j = 0; j < N; ++j) key[j] = j * kRowScoreThreads + tid < n_keys ? keys[j * kRowScoreThreads + tid] : 0;
  float4 part = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  if (tid < 32 && tid < a.cut.pieces) part = parts[tid];
  const int32_t y = live_target(a.r, t, nullptr);
  if (y < 0)
    masked_row(a, t);
  else
    finish_row<N>(a, t, y, key, part, parts, sh);
}

// Few rows: a CTA does all of a row, its pieces' sums and keys in shared memory, in one
// launch instead of two: 5.5 us instead of 6.0 for 8 rows of 32000 bf16 with 5
// alternatives, 8.9 instead of 14.1 for 152 of 131072. CTAS of NT threads an SM, so that
// all rows are in work at a time.
template <typename T, int NT, int CTAS>
__global__ void __launch_bounds__(NT, CTAS) score_one_kernel(const __grid_constant__ ScoreArgs<T> a) {
  __shared__ RowShared sh;
  __shared__ float4 parts[32];  // (at most 32 pieces)
  __shared__ uint32_t keys[1024];
  constexpr int N = 1024 / kRowScoreThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t = blockIdx.x;
  const ScoreLane c(a.r.c, a.r.inv_tf);
  take_turn();
  if (t == 0 && tid == 0) a.head->rows = 1;
  const int32_t y = live_target(a.r, t, tid == 0 ? &a.head->err : nullptr);
  if (y < 0) {
    masked_row(a, t);
    return;
  }
  for (int32_t p = warp; p < a.cut.pieces; p += NT / 32) {
    Piece<T> piece;
    uint4 q0[kScoreBatch];
    piece.t = t;
    piece.p = p;
    piece.open(a, c.far, q0);
    const float4 part = piece_sums(a, c, piece, q0, [&](uint32_t key) { keys[p * 32 + lane] = key; });
    if (lane == 0) parts[p] = part;
  }
  __syncthreads();
  if (tid >= kRowScoreThreads) return;  // (a barrier waits for the threads that are left)
  uint32_t key[N];
#pragma unroll
  for (int j = 0; j < N; ++j)
    key[j] = j * kRowScoreThreads + tid < a.cut.pieces * 32 ? keys[j * kRowScoreThreads + tid] : 0;
  const float4 part = tid < 32 && tid < a.cut.pieces ? parts[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
  finish_row<N>(a, t, y, key, part, parts, sh);
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
__global__ void __launch_bounds__(kScoreThreads, kPartCtas)
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
    // (all of a row's scalars on their way at a time)
    const float4 nm4 = a.norm[t];
    const float da = a.d_logp != nullptr ? a.d_logp[t] : 0.f;
    const float dh = a.d_entropy != nullptr ? a.d_entropy[t] : 0.f;
    const float db = lane < a.K && a.d_top != nullptr ? a.d_top[t * a.K + lane] : 0.f;
    const int32_t ti = lane < a.K && a.d_top != nullptr ? a.top_idx[t * a.K + lane] : -1;
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
    // the first vectors
    const bool same = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
    const uint4* in = reinterpret_cast<const uint4*>(x + s.head) + lane;
    uint4 q0[B], q1[B];
    auto load = [&](uint4 (&q)[B], int32_t v) {
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (v + 32 * j + lane < v1) q[j] = __ldcs(in + v + 32 * j);
    };
    if (same) load(q0, v0);
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
    if (same) {
      // by turns in two sets of registers
      auto put = [&](const uint4 (&q)[B], int32_t v) {
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
      };
      for (int32_t v = v0; v < v1; v += 64 * B) {
        load(q1, v + 32 * B);
        put(q0, v);
        load(q0, v + 64 * B);
        put(q1, v + 32 * B);
      }
    } else {
      for (int64_t e = (int64_t)v0 * VE + lane; e < (int64_t)v1 * VE; e += 32)
        g[s.head + e] = from_f<T>(common(to_f(x[s.head + e])));
    }
    if (loose >= 0) g[loose] = from_f<T>(common(xl));
    __syncwarp();
    if (first_of) g[ti] = from_f<T>(__fmaf_rn(r.inv_tf, own, common(xt)));
    if (target && lane == 0) g[y] = from_f<T>(__fmaf_rn(r.inv_tf, da, common(xy)));
  }
}
