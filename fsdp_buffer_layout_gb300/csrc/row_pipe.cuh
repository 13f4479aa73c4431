// row_pipe.cuh — the pipelined kernel over rows of logits: each live row's
// maximum and sum (and with them its log probability), or, for the policy
// loss, the row's gradient in the same pass over device memory. Included by
// objective.cu.
//
// A cluster of C CTAs takes a row, each CTA an equal share of its 16-byte
// vectors. A CTA has three kinds of warps:
//   producer  finds the cluster's rows (live ones and masked ones are dealt
//             out apart, so that every cluster gets as many), puts each into a
//             queue, and streams its share into a ring of shared-memory chunks
//             with bulk copies;
//   consumers (W warps) add up the terms exp(x - m) of each chunk with a
//             running maximum a thread and leave the warp's join to
//   the joiner, which joins the warps and, with 16-byte asynchronous stores
//             into every CTA of the cluster, the row, and computes what hangs
//             on it: the log probability, the policy's terms, the gradient's
//             coefficient.
// For the gradient the consumers read a row's share once more from shared
// memory, where the chunks have stayed, so logits cross the memory bus once and
// gradients once. They do so after the NEXT row's sums (`ahead`), so that
// nobody waits for the joiner: the ring then holds two rows' shares. No barrier
// spans the consumers; they meet the other warps at mbarriers alone.
//
// Elements in front of a row's first 16-byte boundary and behind its last one
// are read by single threads. A gradient row whose address differs from the
// logits' modulo 16 bytes is written element by element.
//
// Bounds and measurements (GB300, a call among others). Sums alone read at the
// rate of a plain copy: 4096 x 131072 bf16, 3/4 live, 118 us = 6.8 TB/s. The
// policy loss is bound by HBM where a CTA's share is long (8192 x 131072 bf16:
// 694 us, 6.2 TB/s read and written; clusters of 4 leave 8 of the 152 SMs idle)
// and by a row's fixed cost, about 1.8 us of the consumers' time however short
// the row, where it is not (4096 x 32000 bf16, 3/4 live: 80 us, 5.7 TB/s).
// A call costs some 10 us from its first load to its last sum.
//
// Every wait is bounded (mbarrier.cuh). After a timeout all waits of the CTA
// return at once and its warps leave their loops; the cluster then meets at
// its end as always, and waits a moment for messages still on their way.

// 16 bytes of a row as floats in pairs.
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int n = 8;
  static constexpr uint32_t lowest = 0xff80ff80u;  // -inf, -inf
};
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static constexpr uint32_t lowest = 0xff800000u;
};

// Pairs of floats in the packed fp32 instructions of sm_100 and later: one
// issue slot for two elements.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_get(F2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v.v));
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// The pairs of one vector.
template <typename T>
struct Pairs {
  F2 p[Vec<T>::n / 2];
};
__device__ __forceinline__ void unpack(const uint4& v, Pairs<uint16_t>& o) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o.p[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const uint4& v, Pairs<float>& o) {
  o.p[0] = f2(__uint_as_float(v.x), __uint_as_float(v.y));
  o.p[1] = f2(__uint_as_float(v.z), __uint_as_float(v.w));
}

// Largest element of a thread's vectors; NaN is passed over.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int N>
__device__ __forceinline__ float largest(const uint4 (&v)[N], uint16_t) {
  uint32_t m = Vec<uint16_t>::lowest;
#pragma unroll
  for (int i = 0; i < N; ++i)
    m = max_bf16x2(m, max_bf16x2(max_bf16x2(v[i].x, v[i].y), max_bf16x2(v[i].z, v[i].w)));
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}
template <int N>
__device__ __forceinline__ float largest(const uint4 (&v)[N], float) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i)
    m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y)),
                       fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w))));
  return m;
}

__device__ __forceinline__ F2 exp2_pair(F2 t) {
  float a, b;
  f2_get(t, a, b);
  return f2(ex2(a), ex2(b));
}

// exp((x - m) / temperature) of a pair, with nm = (-m, -m).
struct PairScale {
  F2 hi, lo;
};
__device__ __forceinline__ F2 exp_pair(F2 x, F2 nm, const PairScale& c) {
  const F2 d = f2_add(x, nm);
  float a, b;
  f2_get(f2_fma(d, c.hi, f2_mul(d, c.lo)), a, b);
  return f2(ex2(a), ex2(b));
}

// Whether a row's gradient may take its terms as 2^(x c - m c), one fused product
// an element instead of a difference and two products. m c is rounded once, so
// the exponent is off by half a unit of |m c|'s last place, in every term the
// same way: 2^-14 below 2^11, less than a 40th of what bf16's rounding takes (2^-9 to
// 2^-8). Not for fp32, nor for rows farther from 0 or temperatures nearer to it.
// m: as subtracted (finite_max).
template <typename T>
__device__ __forceinline__ bool short_exponent(float m, Log2Scale c) {
  return sizeof(T) == 2 && fabsf(m * c.hi) < 2048.f;
}

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cta_count() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// 16 bytes into the shared memory of the cluster's CTA `rank`, completing
// transaction bytes on its barrier.
__device__ __forceinline__ void put_async(uint32_t slot, uint32_t bar, uint32_t rank, float a,
                                          float b, float c) {
  uint32_t rs, rb;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rs) : "r"(slot), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(bar), "r"(rank));
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
          rs),
      "f"(a), "f"(b), "f"(c), "f"(0.f), "r"(rb)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float (&o)[Vec<T>::n]);
template <>
__device__ __forceinline__ uint4 pack_vec<uint16_t>(const float (&o)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(o[2 * i + 1]), "f"(o[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack_vec<float>(const float (&o)[4]) {
  return make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                    __float_as_uint(o[3]));
}

constexpr int kMaxPipeCluster = 16;
constexpr uint32_t kQueue = 8;  // rows handed on and not yet added up
constexpr int kList = 2048;     // rows of a cluster that its list holds

// W consumer warps, each thread `per` vectors of a chunk; the rings of an SM's
// CTAs have 192 KB together, six chunks each. W = 16 (one CTA an SM) measured best: 8192 x 131072
// bf16, policy loss: 694 us, against 754 for W = 8 (two CTAs, each with half the
// ring, so rows in twice as many pieces); 4096 x 32000, 3/4 live: 81 against 85.
// Before rows were listed in advance 4 vectors took 888 us, 2 took 1014 (a
// chunk's fixed cost shows) and 6 took 1006 (too few chunks).
template <int W>
struct PipeShape {
  static constexpr int per = 4;  // (a short chunk's end is written out for it)
  static constexpr int consumers = W * 32;
  static constexpr int threads = consumers + 64;
  static constexpr int chunk_vecs = per * consumers;
  static constexpr uint32_t chunk_bytes = chunk_vecs * 16;
  static constexpr uint32_t slots = (W * 13u * 1024u) / chunk_bytes;
  // full and empty of each slot; full, empty and parts ready of each queue
  // place; result ready, two; messages, two
  static constexpr uint32_t barriers = 2 * slots + 3 * kQueue + 4;
};
// A place in the ring: slot and how often the ring has gone round, modulo 2.
template <uint32_t N>
struct Place {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// A row as the producer hands it on. Its x_y has been read by then, so the
// gradient may be written over the logits.
struct RowItem {
  int32_t t;  // -1: no more rows
  int32_t y;  // -1: masked
  float w, xy, old, ref, adv;
};
struct PipeTail {  // shared memory behind the ring and its barriers
  float4 message[2][kMaxPipeCluster];
  float4 result[2];  // m, b = -a / s, a, x_y
  RowItem item[kQueue];
  MaxSum part[kQueue][16];
  double sum[16];
  uint32_t count[2][16];  // live tokens of each warp's, masked ones << 16
  int32_t rows[kList];    // the cluster's live rows from the front, masked ones from the back
  int32_t n_live, n_dead;
  uint32_t stop;
};

template <int W>
constexpr uint32_t pipe_smem() {
  return PipeShape<W>::slots * PipeShape<W>::chunk_bytes + 8 * PipeShape<W>::barriers +
         (uint32_t)sizeof(PipeTail) + 128;
}

template <typename T>
struct PipeArgs {
  Rows<T> r;
  PolicyIn p;
  T* grad;
  int64_t grad_ld;
  float4* row;   // statistics: {m, s, x_y} of a live row, or NULL
  float* logp;
  float* stats;  // policy: fp32[4]
  WsHead* head;
  double* partial;  // policy: {policy, kl, weight} sums of each cluster
  int32_t ahead;    // the ring holds two rows' shares
};

// Where a row's vectors lie: `head` elements, then nvec vectors, then a tail.
// (V may be 2^31 - 1: what is added to the tail's start is compared first.)
struct Span {
  int32_t head, nvec;
};
template <typename T>
__device__ __forceinline__ Span span_of(const T* p, int32_t V) {
  const int32_t skew = (int32_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int32_t)sizeof(T);
  const int32_t head = min(skew, V);
  return {head, (V - head) / Vec<T>::n};
}
// First vector of a CTA's share, in a cluster of 2^log CTAs.
__device__ __forceinline__ int32_t share(int32_t nvec, uint32_t rank, uint32_t log) {
  return (int32_t)(((int64_t)nvec * rank) >> log);
}

// Largest of a warp's values; NaN is passed over.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// Sum over the first N lanes (a power of two), in each of them.
template <int N = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
// The join of the maxima and sums of a warp's first N lanes, in those lanes;
// the others hold {-inf, 0}.
template <int N = 32>
__device__ __forceinline__ MaxSum warp_join(MaxSum v, float inv_t) {
  const float m = warp_max(v.m);
  return {m, warp_sum<N>(v.s * expf((v.m - finite_max(m)) * inv_t))};
}

// Zeroes the gradient row's share of this CTA.
template <typename T>
__device__ __noinline__ void zero_share(T* g, int32_t V, uint32_t rank, uint32_t log, int tid,
                                           int threads) {
  const Span s = span_of(g, V);
  uint4* v = reinterpret_cast<uint4*>(g + s.head);
  const int32_t end = share(s.nvec, rank + 1, log);
  for (int32_t i = share(s.nvec, rank, log) + tid; i < end; i += threads)
    __stcs(v + i, make_uint4(0, 0, 0, 0));
  const int32_t tail = s.head + s.nvec * Vec<T>::n;
  if (rank == 0 && tid < s.head) g[tid] = from_f<T>(0.f);
  if (rank + 1 == 1u << log && tid < V - tail) g[tail + tid] = from_f<T>(0.f);
}

// Whether the phase of the given parity is over; does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The waits of a whole warp: all of its lanes go on, or none does.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned* err,
                                          volatile uint32_t* stop) {
  return __all_sync(~0u, mbar_wait(bar, parity, err, stop));
}
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, unsigned* err,
                                                  volatile uint32_t* stop) {
  return __all_sync(~0u, mbar_wait_cluster(bar, parity, err, stop));
}

// The loss from the sums of n clusters or CTAs, in their order; one warp.
template <typename T>
__device__ __forceinline__ void policy_stats(const PipeArgs<T>& a, int64_t n, int lane) {
  constexpr int kAhead = 4;
  double v[3] = {0.0, 0.0, 0.0};
  for (int64_t c = lane; c < n; c += 32 * kAhead) {
    double u[kAhead][3];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int j = 0; j < 3; ++j) u[k][j] = c + 32 * k < n ? __ldcg(a.partial + 3 * (c + 32 * k) + j) : 0.0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int j = 0; j < 3; ++j) v[j] += u[k][j];
  }
  for (int j = 0; j < 3; ++j) v[j] = warp_sum(v[j]);
  if (lane == 0) {
    const double f = (double)a.p.scale / (a.p.mean && v[2] != 0.0 ? v[2] : 1.0);
    a.stats[0] = (float)(f * (v[0] + (a.p.beta != 0.f ? (double)a.p.beta * v[1] : 0.0)));
    a.stats[1] = (float)(f * v[0]);
    a.stats[2] = (float)(f * v[1]);
    a.stats[3] = (float)v[2];
    a.head->ticket = 0;
    a.head->rows = 1;
  }
}

// A row whose gradient is still to be written.
template <uint32_t SLOTS>
struct Pending {
  int64_t t;
  int32_t y, loose;
  float xl;  // the loose element
  int32_t head, begin, end;  // the row's first vector; the share's vectors
  uint32_t skew;             // the logits' address modulo 16
  Place<SLOTS> first;
};

template <typename T, int W, bool POLICY>
__global__ void __launch_bounds__(PipeShape<W>::threads, 16 / W)
    row_pipe_kernel(const __grid_constant__ PipeArgs<T> a) {
  using Shape = PipeShape<W>;
  constexpr int VE = Vec<T>::n;
  constexpr uint32_t slots = Shape::slots;
  extern __shared__ unsigned char raw[];
  unsigned char* ring =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~(uintptr_t)127);
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + slots * Shape::chunk_bytes);
  PipeTail* sh = reinterpret_cast<PipeTail*>(bars + Shape::barriers);
  const uint32_t full = smem_u32(bars), empty = full + 8 * slots;
  const uint32_t qfull = empty + 8 * slots, qempty = qfull + 8 * kQueue;
  const uint32_t pbar = qempty + 8 * kQueue, rbar = pbar + 8 * kQueue, xbar = rbar + 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t C = cta_count(), rank = C > 1 ? cta_rank() : 0;
  const uint32_t logC = 31 - __clz(C);
  const int64_t cluster = blockIdx.x / C, clusters = gridDim.x / C;
  const Rows<T>& r = a.r;
  // whether live and masked rows are dealt out apart, by a list; with a row a
  // cluster at most, or more than it holds, clusters take rows as they come
  const bool listed = r.T_ > clusters && 2 * (r.T_ / clusters + 1) <= kList;
  unsigned* err = &a.head->err;
  volatile uint32_t* stop = &sh->stop;

  if (tid == 0) {
    for (uint32_t s = 0; s < slots; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, W);
    }
    for (uint32_t s = 0; s < kQueue; ++s) {
      mbar_init(qfull + 8 * s, 1);
      mbar_init(qempty + 8 * s, W + 1);
      mbar_init(pbar + 8 * s, W);
    }
    for (uint32_t s = 0; s < 2; ++s) {
      mbar_init(rbar + 8 * s, 1);
      mbar_init(xbar + 8 * s, 1);
    }
    sh->stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  if (C > 1) cluster_sync();
  take_turn();

  if (warp == W) {  // -------------------------------------------- producer
    Place<slots> at;
    Place<kQueue> q;
    uint32_t issued = 0, queued = 0;  // counted up to the ring's and the queue's length
    // Hands a row on, which lane `from` holds, and streams its share. As many
    // chunks as the ring has room for are asked for before the row's scalars
    // are waited for, the others after the row is in the queue (the consumers
    // make room only for a row they know).
    auto hand_on = [&](const RowItem& item, int from) -> bool {
      const int32_t t = __shfl_sync(~0u, item.t, from), y = __shfl_sync(~0u, item.y, from);
      bool ok = true;
      if (queued == kQueue) {
        if (lane == 0) ok = mbar_wait(qempty + 8 * q.slot, q.phase ^ 1, err, stop);
        if (!__shfl_sync(~0u, (int)ok, 0)) return false;
      } else {
        ++queued;
      }
      const bool reads = t >= 0 && y >= 0;
      const T* x = r.x + (reads ? t * r.ld : 0);
      const Span s = span_of(x, r.V);
      const char* base = reinterpret_cast<const char*>(x + s.head);
      int32_t v = share(s.nvec, rank, logC);
      const int32_t end = reads ? share(s.nvec, rank + 1, logC) : v;
      auto stream = [&](bool wait) -> bool {
        for (; v < end; v += Shape::chunk_vecs) {
          if (issued == slots) {
            const uint32_t bar = empty + 8 * at.slot;
            if (wait ? !mbar_wait(bar, at.phase ^ 1, err, stop) : !mbar_test(bar, at.phase ^ 1))
              return false;
          } else {
            ++issued;
          }
          const uint32_t bytes = (uint32_t)min(end - v, (int32_t)Shape::chunk_vecs) * 16;
          mbar_expect_tx(full + 8 * at.slot, bytes);
          bulk_load(smem_u32(ring + at.slot * Shape::chunk_bytes), base + (int64_t)v * 16, bytes,
                    full + 8 * at.slot);
          at.next();
        }
        return true;
      };
      if (lane == 0) stream(false);
      __syncwarp();
      if (lane == from) {
        sh->item[q.slot] = item;
        mbar_arrive(qfull + 8 * q.slot);
      }
      q.next();
      __syncwarp();
      if (lane == 0) ok = stream(true);
      return __shfl_sync(~0u, (int)ok, 0) != 0;
    };
    auto fetch = [&](int t) -> RowItem {
      RowItem it = {t, -1, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (t < 0) return it;
      const Token k = token_at(r, it.t);
      it.y = live_target(r, k, nullptr);
      it.w = k.w;
      if (it.y < 0) return it;
      it.xy = to_f(r.x[(int64_t)it.t * r.ld + it.y]);
      if (POLICY) {
        it.old = a.p.old_logp[it.t];
        it.adv = a.p.adv[it.t];
        if (a.p.beta != 0.f) it.ref = a.p.ref_logp[it.t];
      }
      return it;
    };
    bool ok = true;
    if (listed) {  // the first row at once; the others when the list is there
      const RowItem now = fetch(lane == 0 ? (int)cluster : -1);
      if (POLICY || __shfl_sync(~0u, now.y, 0) >= 0) ok = hand_on(now, 0);
      asm volatile("bar.sync 1, %0;" ::"r"(Shape::threads) : "memory");
    }
    // Rows in turn, masked ones spread among the live ones; a lane fetches what
    // the joiner needs of a row, 32 rows at a time and as many ahead.
    const int n_live = listed ? sh->n_live : 0, n_rows = listed ? n_live + sh->n_dead : 0;
    auto row_at = [&](int i) -> int {
      if (!listed) {
        const int64_t t = cluster + i * clusters;
        return t < r.T_ ? (int)t : -1;
      }
      if (i >= n_rows) return -1;
      // of the first i rows, i n_live / n_rows rounded up are live
      const int before = (i * n_live + n_rows - 1) / n_rows;
      const int after = ((i + 1) * n_live + n_rows - 1) / n_rows;
      return after > before ? sh->rows[before] : sh->rows[kList - 1 - (i - before)];
    };
    RowItem next = fetch(row_at(lane));
    for (int i0 = 32; ok; i0 += 32) {
      const RowItem now = next;
      const int n = __popc(__ballot_sync(~0u, now.t >= 0));
      if (n == 32) next = fetch(row_at(i0 + lane));
      for (int j = 0; j < n && ok; ++j)
        if (POLICY || __shfl_sync(~0u, now.y, j) >= 0) ok = hand_on(now, j);
      if (n < 32) break;
    }
    if (ok) hand_on({-1, -1, 0.f, 0.f, 0.f, 0.f, 0.f}, 0);
    if (lane == 0) {
      // every copy issued has to land before the CTA may end
      const uint64_t deadline = global_ns() + kWaitNs;
      if (issued < slots) at = Place<slots>();
      else at.phase ^= 1;  // the oldest of the last `slots` chunks
      for (; issued > 0; --issued, at.next())
        if (!mbar_drain(full + 8 * at.slot, at.phase, deadline, err)) break;
    }
  } else {
    if (warp < W) {
      // Once through the tokens, 8 times 32 a warp at a time: the sum of the
      // live weights, which scales every gradient (each CTA adds it up for
      // itself, in the same order), and the cluster's rows.
      constexpr int kBlocks = 8;
      const bool first = cluster == 0 && rank == 0;
      const int step = (int)clusters, own = (int)cluster;
      float w2[2] = {0.f, 0.f};
      int lives = 0, deads = 0, buf = 0;
      for (int64_t t0 = 0; t0 < r.T_; t0 += W * kBlocks * 32, buf ^= 1) {
        const int64_t tw = t0 + warp * kBlocks * 32;
        uint32_t lb = 0, db = 0;  // lane j: live and masked tokens of block j
        Token k[kBlocks];
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) k[j] = token_at(r, tw + 32 * j + lane);
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
          const int64_t t = tw + 32 * j + lane;
          const int32_t y = live_target(r, k[j], first ? err : nullptr);
          if (y >= 0) w2[j & 1] += k[j].w;
          else if (first && t < r.T_ && a.logp != nullptr) a.logp[t] = 0.f;
          // (the first row of each cluster is not on its list)
          const bool late = t >= clusters && t < r.T_;
          const uint32_t l = __ballot_sync(~0u, y >= 0 && late);
          const uint32_t d = __ballot_sync(~0u, y < 0 && late);
          if (lane == j) {
            lb = l;
            db = d;
          }
        }
        if (!listed) continue;
        // live and masked tokens (at most 256 a warp) up to each block's end
        const uint32_t mine = __popc(lb) | __popc(db) << 16;
        uint32_t sum = mine;
#pragma unroll
        for (int o = 1; o < kBlocks; o <<= 1) {
          const uint32_t u = __shfl_up_sync(~0u, sum, o);
          if (lane >= o) sum += u;
        }
        if (lane == kBlocks - 1) sh->count[buf][warp] = sum;
        asm volatile("bar.sync 2, %0;" ::"r"(Shape::consumers) : "memory");
        uint32_t before = 0, all = 0;  // of the warps before this one; of all
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const uint32_t c = sh->count[buf][w];
          all += c;
          if (w < warp) before += c;
        }
        before += sum - mine;
        // numbers own, own + step, ... of all live (masked) tokens
        auto list = [&](uint32_t bits, int start, bool front) {
          int i = start <= own ? 0 : (int)((uint32_t)(start - own + step - 1) / (uint32_t)step);
          for (int at = own + i * step - start; at < __popc(bits); at += step, ++i) {
            uint32_t rest = bits;
            for (int d = 0; d < at; ++d) rest &= rest - 1;
            sh->rows[front ? i : kList - 1 - i] = (int)tw + 32 * lane + __ffs(rest) - 1;
          }
        };
        if (lane < kBlocks) {
          list(lb, lives + (int)(before & 0xffffu), true);
          if (POLICY) list(db, deads + (int)(before >> 16), false);
        }
        lives += (int)(all & 0xffffu);
        deads += (int)(all >> 16);
      }
      const double n = warp_sum((double)w2[0] + (double)w2[1]);
      if (lane == 0) sh->sum[warp] = n;
      if (tid == 0) {
        sh->n_live = lives > own ? (lives - own + step - 1) / step : 0;
        sh->n_dead = POLICY && deads > own ? (deads - own + step - 1) / step : 0;
      }
      if (listed) asm volatile("bar.arrive 1, %0;" ::"r"(Shape::threads) : "memory");
      else asm volatile("bar.arrive 1, %0;" ::"r"(Shape::threads - 32) : "memory");
    } else {
      if (listed) asm volatile("bar.sync 1, %0;" ::"r"(Shape::threads) : "memory");
      else asm volatile("bar.sync 1, %0;" ::"r"(Shape::threads - 32) : "memory");
    }
    Place<kQueue> q;
    if (warp == W + 1) {  // ------------------------------------------ joiner
      double factor = 0.0;
      if (POLICY) {
        factor = (double)a.p.scale;
        if (a.p.mean) {
          double all = 0.0;
          for (int w = 0; w < W; ++w) all += sh->sum[w];
          if (all != 0.0) factor /= all;
        }
      }
      const float scale = (float)(factor * r.inv_t);
      double sum = 0.0;  // lane 0: policy, lane 1: KL, lane 2: weight
      for (uint32_t done = 0;; q.next()) {
        if (!warp_wait(qfull + 8 * q.slot, q.phase, err, stop)) break;
        const RowItem now = sh->item[q.slot];
        if (now.t < 0) break;
        if (now.y < 0) {
          if (!warp_wait(pbar + 8 * q.slot, q.phase, err, stop)) break;
          if (lane == 0) mbar_arrive(qempty + 8 * q.slot);
          continue;
        }
        const uint32_t par = done & 1, phase = (done >> 1) & 1;
        ++done;
        if (!warp_wait(pbar + 8 * q.slot, q.phase, err, stop)) break;
        MaxSum ms = lane < W ? sh->part[q.slot][lane] : MaxSum{-INFINITY, 0.f};
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty + 8 * q.slot);
        ms = warp_join<W>(ms, r.inv_tf);
        if (C > 1) {
          const uint32_t bar = xbar + 8 * par;
          if (lane == 0) mbar_expect_tx(bar, C * 16);
          __syncwarp();
          if (lane < C) put_async(smem_u32(&sh->message[par][rank]), bar, lane, ms.m, ms.s, now.xy);
          if (!warp_wait_cluster(bar, phase, err, stop)) break;
          const float4 got = sh->message[par][lane < C ? lane : 0];
          ms = warp_join<kMaxPipeCluster>(lane < C ? MaxSum{got.x, got.y} : MaxSum{-INFINITY, 0.f},
                                          r.inv_tf);
        }
        // lane 0 (of the cluster's first lanes) holds the row's maximum and sum
        const LogSum ls = log_sum(ms.s);
        const float d = now.xy - ms.m;
        if (POLICY) {
          const PolicyTerm o = policy_term(a.p, log_ratio(d, r.inv_tf, now.old, ls),
                                           -log_ratio(d, r.inv_tf, now.ref, ls), now.adv);
          const float coef = scale * now.w * o.slope;
          if (lane == 0) {
            sh->result[par] = make_float4(ms.m, -coef / ms.s, coef, now.xy);
            mbar_arrive(rbar + 8 * par);
          }
          sum += (double)(lane == 0 ? now.w * o.policy : lane == 1 ? now.w * o.kl : now.w);
        }
        if (lane == 0 && rank == 0) {
          if (a.row != nullptr) a.row[now.t] = make_float4(ms.m, ms.s, now.xy, 0.f);
          if (a.logp != nullptr) a.logp[now.t] = log_ratio(d, r.inv_tf, 0.f, ls);
        }
      }
      if (POLICY && rank == 0) {
        // the last cluster to finish adds up all of them in their order
        uint32_t last = 0;
        if (lane < 3) {
          a.partial[3 * cluster + lane] = sum;
          __threadfence();
        }
        __syncwarp();
        if (lane == 0) {
          last = atomicAdd(&a.head->ticket, 1u) + 1 == (uint32_t)clusters;
          __threadfence();
        }
        if (__shfl_sync(~0u, last, 0)) policy_stats(a, clusters, lane);
      }
    } else {  // ---------------------------------------------------- consumers
      const PairScale c2 = {f2(r.c.hi, r.c.hi), f2(r.c.lo, r.c.lo)};
      // this thread's factor: log2(e) / temperature rounded down or up
      const float c1 = (uint32_t)tid * 2654435769u < r.c.ups ? r.c.up : r.c.hi;
      const F2 cc = f2(c1, c1);
      Place<slots> at;
      uint32_t written = 0;  // live rows whose gradient has been written
      // The gradient of a row from the chunks still in shared memory.
      auto write_grad = [&](const Pending<slots>& p) -> bool {
        const uint32_t par = written & 1, phase = (written >> 1) & 1;
        ++written;
        if (!warp_wait(rbar + 8 * par, phase, err, stop)) return false;
        const float4 res = sh->result[par];
        const int32_t begin = p.begin, end = p.end;
        const float z = finite_max(res.x), b = res.y, coef = res.z;
        T* g = a.grad + p.t * a.grad_ld;
        const bool same = (reinterpret_cast<uintptr_t>(g) & 15) == p.skew;
        const bool near = short_exponent<T>(z, r.c);
        const F2 nm = f2(-z, -z), b2 = f2(b, b), c0 = f2(r.c.hi, r.c.hi);
        const F2 kk = f2(-z * r.c.hi, -z * r.c.hi);
        uint4* gv = reinterpret_cast<uint4*>(g + p.head);
        Place<slots> from = p.first;
        for (int32_t v = begin; v < end; v += Shape::chunk_vecs, from.next()) {
          const unsigned char* chunk = ring + from.slot * Shape::chunk_bytes;
          if (a.grad == nullptr || coef == 0.f) {
          } else if (same) {
            const uint4* c = reinterpret_cast<const uint4*>(chunk) + tid;
            uint4* out = gv + v + tid;
            const int32_t n = end - v - tid;
            if (near) {
#pragma unroll
              for (int j = 0; j < Shape::per; ++j) {
                if (j * Shape::consumers >= n) break;
                Pairs<T> e;
                unpack(c[j * Shape::consumers], e);
                float o[VE];
#pragma unroll
                for (int i = 0; i < VE / 2; ++i)
                  f2_get(f2_mul(exp2_pair(f2_fma(e.p[i], c0, kk)), b2), o[2 * i], o[2 * i + 1]);
                __stcs(out + j * Shape::consumers, pack_vec<T>(o));
              }
            } else {
#pragma unroll(sizeof(T) == 2 ? 1 : Shape::per)
              for (int j = 0; j < Shape::per; ++j) {
                if (j * Shape::consumers >= n) break;
                Pairs<T> e;
                unpack(c[j * Shape::consumers], e);
                float o[VE];
#pragma unroll
                for (int i = 0; i < VE / 2; ++i)
                  f2_get(f2_mul(exp_pair(e.p[i], nm, c2), b2), o[2 * i], o[2 * i + 1]);
                __stcs(out + j * Shape::consumers, pack_vec<T>(o));
              }
            }
          } else {
            const T* c = reinterpret_cast<const T*>(chunk);
            const int32_t n = min(end - v, (int32_t)Shape::chunk_vecs) * VE;
            T* out = g + p.head + (int64_t)v * VE;
#pragma unroll 1
            for (int32_t i = tid; i < n; i += Shape::consumers)
              out[i] = from_f<T>(b * exp_scaled(to_f(c[i]) - z, r.c));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty + 8 * from.slot);
        }
        if (a.grad == nullptr) return true;
        if (coef == 0.f) {
          zero_share(g, r.V, rank, logC, tid, Shape::consumers);
          return true;
        }
        if (p.loose >= 0) {
          const float e = b * exp_scaled(p.xl - z, r.c);
          g[p.loose] = from_f<T>(p.loose == p.y ? e + coef : e);
        }
        // the target's element again, by the thread that wrote it
        const int32_t ye = p.y - p.head, yv = ye / VE;
        if (ye >= 0 && yv >= begin && yv < end &&
            tid == ((same ? yv - begin : ye - begin * VE) & (Shape::consumers - 1)))
          g[p.y] = from_f<T>(b * exp_scaled(res.w - z, r.c) + coef);
        return true;
      };
      Pending<slots> prev = {};
      prev.t = -1;
      bool ok = true;
      for (; ok; q.next()) {
        if (!warp_wait(qfull + 8 * q.slot, q.phase, err, stop)) {
          ok = false;
          break;
        }
        const RowItem it = sh->item[q.slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty + 8 * q.slot);
        if (it.t < 0) break;
        if (it.y < 0) {
          if (lane == 0) mbar_arrive(pbar + 8 * q.slot);
          if (a.grad != nullptr)
            zero_share(a.grad + (int64_t)it.t * a.grad_ld, r.V, rank, logC, tid, Shape::consumers);
          continue;
        }
        Pending<slots> row;
        row.t = it.t;
        row.y = it.y;
        row.first = at;
        const T* x = r.x + (int64_t)it.t * r.ld;
        const Span s = span_of(x, r.V);
        const int32_t begin = share(s.nvec, rank, logC), end = share(s.nvec, rank + 1, logC);
        row.head = s.head;
        row.begin = begin;
        row.end = end;
        row.skew = (uint32_t)(reinterpret_cast<uintptr_t>(x) & 15);
        row.loose = -1;
        if (rank == 0 && tid < s.head) row.loose = tid;
        const int32_t tail = s.head + s.nvec * VE;
        if (rank + 1 == C && tid >= 16 && tid - 16 < r.V - tail) row.loose = tail + (tid - 16);
        row.xl = -INFINITY;
        if (row.loose >= 0) row.xl = to_f(x[row.loose]);

        // ---- maximum and sum
        float m = -INFINITY;
        F2 sum0 = f2(0.f, 0.f), sum1 = sum0;
        auto add_up = [&](const auto& x4) {
          constexpr int n = sizeof(x4) / sizeof(uint4);
          const float bm = largest(x4, T());
          if (bm > m) {
            const float f = expf((m - bm) * r.inv_tf);
            sum0 = f2_mul(sum0, f2(f, f));
            sum1 = f2_mul(sum1, f2(f, f));
            m = bm;
          }
          const float z = -finite_max(m);
          const F2 nm = f2(z, z);
#pragma unroll
          for (int j = 0; j < n; ++j) {
            Pairs<T> p;
            unpack(x4[j], p);
#pragma unroll
            for (int i = 0; i < VE / 2; i += 2) {
              sum0 = f2_add(sum0, exp2_pair(f2_mul(f2_add(p.p[i], nm), cc)));
              sum1 = f2_add(sum1, exp2_pair(f2_mul(f2_add(p.p[i + 1], nm), cc)));
            }
          }
        };
        for (int32_t v = begin; v < end; v += Shape::chunk_vecs, at.next()) {
          if (!warp_wait(full + 8 * at.slot, at.phase, err, stop)) {
            ok = false;
            break;
          }
          const uint4* c = reinterpret_cast<const uint4*>(ring + at.slot * Shape::chunk_bytes) + tid;
          const int32_t n = end - v - tid;
          if (n > (Shape::per - 1) * Shape::consumers) {
            uint4 x4[Shape::per];
#pragma unroll
            for (int j = 0; j < Shape::per; ++j) x4[j] = c[j * Shape::consumers];
            add_up(x4);
          } else if (n > 2 * Shape::consumers) {
            const uint4 x3[3] = {c[0], c[Shape::consumers], c[2 * Shape::consumers]};
            add_up(x3);
          } else if (n > Shape::consumers) {
            const uint4 x2[2] = {c[0], c[Shape::consumers]};
            add_up(x2);
          } else if (n > 0) {
            const uint4 x1[1] = {c[0]};
            add_up(x1);
          }
          if (!POLICY) {
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * at.slot);
          }
        }
        if (!ok) break;
        float s0, s1, s2, s3;
        f2_get(sum0, s0, s1);
        f2_get(sum1, s2, s3);
        MaxSum ms = {m, (s0 + s1) + (s2 + s3)};
        if (row.loose >= 0) ms = join(ms, {row.xl, row.xl == -INFINITY ? 0.f : 1.f}, r.inv_tf);
        ms = warp_join(ms, r.inv_tf);
        if (lane == 0) {
          sh->part[q.slot][warp] = ms;
          mbar_arrive(pbar + 8 * q.slot);
        }
        if (POLICY) {
          if (!a.ahead) {
            ok = write_grad(row);
          } else {
            if (prev.t >= 0) ok = write_grad(prev);
            prev = row;
          }
        }
      }
      if (POLICY && a.ahead && ok && prev.t >= 0) write_grad(prev);
    }
  }
  __syncwarp();
  // no CTA leaves while another of its cluster may still write to it
  if (C > 1) {
    cluster_sync();
    if (*stop != 0u) {
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < 100000ull) {
      }
    }
  }
}

// ------------------------------------------------------------ gradient alone
// The gradient's rows where a row's coefficient is known only after the sums of
// all rows (preference loss), or its share of a cluster's shared memory is too
// long. A thread takes six vectors of a row at a time (four and eight are within
// 2 percent of it). Rows are taken last first: the pass before read them first
// to last, so that the end of the logits is still in L2 (75 of 221 MB measured).
// HBM bounds it: for 16 pairs of 384 x 32000 bf16, 3/4 live, the three kernels of
// the loss take 255 us, of which 175 here (443 MB read, 591 MB written).
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 6;
constexpr int kGradCtas = 4;  // an SM
constexpr int kGradPiece = kGradThreads * kGradVecs;  // vectors of a row at a time

// One piece of a gradient row: y < 0 or a = 0: zeros.
template <typename T>
__device__ __forceinline__ void grad_piece(const Rows<T>& r, int64_t t, int32_t piece,
                                           int32_t pieces, int32_t y, float a, const float4& st,
                                           T* grad, int64_t grad_ld) {
  constexpr int VE = Vec<T>::n;
  const int tid = threadIdx.x;
  const PairScale c2 = {f2(r.c.hi, r.c.hi), f2(r.c.lo, r.c.lo)};
  T* g = grad + t * grad_ld;
  const T* x = r.x + t * r.ld;
  const Span s = span_of(g, r.V);
  const int32_t begin = piece * kGradPiece;
  const int32_t end = piece + 1 == pieces ? s.nvec : min(s.nvec, begin + kGradPiece);
  const int32_t tail = s.head + s.nvec * VE;
  // the loose element of this thread, if any
  int32_t loose = -1;
  if (piece == 0 && tid < s.head) loose = tid;
  if (piece + 1 == pieces && tid >= 16 && tid - 16 < r.V - tail) loose = tail + (tid - 16);
  uint4* out = reinterpret_cast<uint4*>(g + s.head) + tid;
  if (y < 0 || a == 0.f) {
    for (int32_t v = begin; v + tid < end; v += kGradThreads)
      __stcs(out + v, make_uint4(0, 0, 0, 0));
    if (loose >= 0) g[loose] = from_f<T>(0.f);
    return;
  }
  const float z = finite_max(st.x), b = -a / st.y;
  if (loose >= 0) {
    const float e = b * exp_scaled(to_f(x[loose]) - z, r.c);
    g[loose] = from_f<T>(loose == y ? e + a : e);
  }
  const int32_t ye = y - s.head, yv = ye / VE;
  const bool mine = ye >= 0 && yv >= begin && yv < end;  // the target is in this piece
  if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0) {
    const bool near = short_exponent<T>(z, r.c);
    const F2 nm = f2(-z, -z), b2 = f2(b, b), c0 = f2(r.c.hi, r.c.hi);
    const F2 kk = f2(-z * r.c.hi, -z * r.c.hi);
    const uint4* in = reinterpret_cast<const uint4*>(x + s.head) + tid;
    for (int32_t v = begin; v < end; v += kGradPiece) {
      uint4 q[kGradVecs];
#pragma unroll
      for (int j = 0; j < kGradVecs; ++j)
        if (v + j * kGradThreads + tid < end) q[j] = __ldcs(in + v + j * kGradThreads);
#pragma unroll
      for (int j = 0; j < kGradVecs; ++j) {
        if (v + j * kGradThreads + tid >= end) break;
        Pairs<T> e;
        unpack(q[j], e);
        float o[VE];
#pragma unroll
        for (int k = 0; k < VE / 2; ++k)
          f2_get(f2_mul(near ? exp2_pair(f2_fma(e.p[k], c0, kk)) : exp_pair(e.p[k], nm, c2), b2),
                 o[2 * k], o[2 * k + 1]);
        __stcs(out + v + j * kGradThreads, pack_vec<T>(o));
      }
    }
    if (mine && tid == ((yv - begin) & (kGradThreads - 1)))
      g[y] = from_f<T>(b * exp_scaled(st.z - z, r.c) + a);
  } else {
    const int32_t first = s.head + begin * VE, n = (end - begin) * VE;
    for (int32_t k = tid; k < n; k += kGradThreads) {
      const float e = b * exp_scaled(to_f(x[first + k]) - z, r.c);
      g[first + k] = from_f<T>(first + k == y ? e + a : e);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kGradThreads, kGradCtas)
    row_grad_kernel(const __grid_constant__ Rows<T> r, const float4* row, const float* coef,
                    T* grad, int64_t grad_ld, int32_t pieces) {
  take_turn();
  const int64_t items = r.T_ * pieces;
  // what a piece needs of its row, on its way while the piece before is written
  int64_t t = 0;
  int32_t piece = 0;
  Token k = {-1, 0.f};
  float a = 0.f;
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fetch = [&](int64_t i) {
    if (i >= items) return;
    t = r.T_ - 1 - i / pieces;
    piece = (int32_t)(i % pieces);
    k = token_at(r, t);
    a = coef[t];
    st = row[t];
  };
  fetch(blockIdx.x);
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int64_t t0 = t;
    const int32_t piece0 = piece;
    const int32_t y = live_target(r, k, nullptr);
    const float a0 = a;
    const float4 st0 = st;
    fetch(i + gridDim.x);
    grad_piece(r, t0, piece0, pieces, y, a0, st0, grad, grad_ld);
  }
}
