// row_regs.cuh — the row operation for short rows (up to 32 KB), whose vectors
// fit the registers of G warps: one read, one write, no ring. The pipelined
// kernel hands rows from warp to warp, which takes about 1.8 us a row however
// short it is; here 3 to 32 rows are in flight on an SM instead. What bounds it
// is the chain from a row's loads over its sum and its scalars to its stores
// (policy loss, bf16: 4096 x 16000 66 us, 59 percent of the copy rate; 4096 x
// 1000 16 us); sums alone reach 5.4 us for 4096 x 1000. Included by objective.cu
// after row_pipe.cuh.
//
// Each group of G warps takes every n-th row. Its threads hold up to NV vectors
// each. The warps' joins meet in shared memory (G > 1) behind a barrier of the
// group, and every warp works out the row's scalars for itself.
constexpr int kRegsThreads = 256;
constexpr int regs_ctas(int nv) { return nv <= 4 ? 4 : 3; }  // an SM

// Sum of the live weights, for many tokens: up to 64 CTAs, the last of which adds
// up their sums in their order. The kernel behind it is set up and fetches its
// first tokens meanwhile (it is let go only after the kernels before this one
// have ended) and waits for the sum before its first row.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads)
    weight_sum_kernel(const int64_t* target, const float* weight, int64_t T_, int32_t V,
                      double* partial, double* total, WsHead* head) {
  __shared__ float part[32];
  const int tid = threadIdx.x;
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  float w = 0.f;
  const int64_t step = (int64_t)gridDim.x * kSumThreads;
#pragma unroll 4
  for (int64_t t = (int64_t)blockIdx.x * kSumThreads + tid; t < T_; t += step)
    if (target[t] >= 0 && target[t] < V) w += weight != nullptr ? weight[t] : 1.f;
  w = warp_sum(w);
  if ((tid & 31) == 0) part[tid >> 5] = w;
  __syncthreads();
  if (tid >= 32) return;
  const double s = warp_sum((double)part[tid]);
  if (gridDim.x == 1) {
    if (tid == 0) *total = s;
    return;
  }
  uint32_t last = 0;
  if (tid == 0) {
    partial[blockIdx.x] = s;
    __threadfence();
    last = atomicAdd(&head->ticket, 1u) + 1 == gridDim.x;
    __threadfence();
  }
  if (!__shfl_sync(~0u, last, 0)) return;
  double all = tid < gridDim.x ? __ldcg(partial + tid) : 0.0;
  if (tid + 32 < gridDim.x) all += __ldcg(partial + tid + 32);
  all = warp_sum(all);
  if (tid == 0) {
    *total = all;
    head->ticket = 0;
  }
}

template <typename T, int G, int NV, bool POLICY>
__global__ void __launch_bounds__(kRegsThreads, regs_ctas(NV))
    row_regs_kernel(const __grid_constant__ PipeArgs<T> a, const double* total) {
  constexpr int VE = Vec<T>::n, kGroups = 8 / G, kThreads = 32 * G;
  __shared__ float4 part[2][8];  // of each warp: m, s, x_y
  __shared__ double sums[8][3];
  __shared__ float weights[8];
  const Rows<T>& r = a.r;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = warp / G, gtid = tid & (kThreads - 1);
  const int64_t groups = (int64_t)gridDim.x * kGroups;
  const int64_t first = (int64_t)blockIdx.x * kGroups + group;
  const PairScale c2 = {f2(r.c.hi, r.c.hi), f2(r.c.lo, r.c.lo)};
  const float c1 = (uint32_t)gtid * 2654435769u < r.c.ups ? r.c.up : r.c.hi;
  const F2 cc = f2(c1, c1);
  // (behind weight_sum_kernel, inputs may be read before its end)
  if (total == nullptr) cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  Token next = token_at(r, first);
  float scale = 0.f;
  if (POLICY) {
    double n = 0.0;
    if (a.p.mean && total == nullptr) {  // few tokens: each CTA adds them up
      float w = 0.f;
      for (int64_t t = tid; t < r.T_; t += kRegsThreads) {
        const Token k = token_at(r, t);
        if (k.y >= 0 && k.y < r.V) w += k.w;
      }
      w = warp_sum(w);
      if (lane == 0) weights[warp] = w;
      __syncthreads();
      for (int i = 0; i < 8; ++i) n += (double)weights[i];
    } else if (a.p.mean) {
      cudaGridDependencySynchronize();
      n = __ldcg(total);
    }
    scale = (float)((double)a.p.scale / (a.p.mean && n != 0.0 ? n : 1.0) * r.inv_t);
  }
  double sum = 0.0;  // lane 0: policy, lane 1: KL, lane 2: weight
  int par = 0;
  for (int64_t t = first; t < r.T_; t += groups) {
    const int32_t y = live_target(r, next, gtid == 0 ? &a.head->err : nullptr);
    const float w = next.w;
    next = token_at(r, t + groups);
    if (y < 0) {
      if (POLICY && a.grad != nullptr) zero_share(a.grad + t * a.grad_ld, r.V, 0, 0, gtid, kThreads);
      if (gtid == 0 && a.logp != nullptr) a.logp[t] = 0.f;
      continue;
    }
    const T* x = r.x + t * r.ld;
    const Span s = span_of(x, r.V);
    const uint4* in = reinterpret_cast<const uint4*>(x + s.head) + gtid;
    uint4 q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      q[j] = make_uint4(Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest, Vec<T>::lowest);
      if (j * kThreads + gtid < s.nvec) q[j] = __ldcs(in + j * kThreads);
    }
    const int32_t tail = s.head + s.nvec * VE;
    int32_t loose = -1;
    if (gtid < s.head) loose = gtid;
    if (gtid >= 16 && gtid - 16 < r.V - tail) loose = tail + (gtid - 16);
    float xl = -INFINITY;
    if (loose >= 0) xl = to_f(x[loose]);
    float xy = 0.f, old = 0.f, ref = 0.f, adv = 0.f;
    if (G == 1 || warp % G == 0) xy = to_f(x[y]);
    if (POLICY) {
      old = a.p.old_logp[t];
      adv = a.p.adv[t];
      if (a.p.beta != 0.f) ref = a.p.ref_logp[t];
    }
    // ---- maximum and sum
    const float m = fmaxf(largest(q, T()), xl);
    const float z = -finite_max(m);
    const F2 nm = f2(z, z);
    F2 sum0 = f2(0.f, 0.f), sum1 = sum0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (j > 0 && j * kThreads >= s.nvec) break;
      Pairs<T> p;
      unpack(q[j], p);
#pragma unroll
      for (int i = 0; i < VE / 2; i += 2) {
        sum0 = f2_add(sum0, exp2_pair(f2_mul(f2_add(p.p[i], nm), cc)));
        sum1 = f2_add(sum1, exp2_pair(f2_mul(f2_add(p.p[i + 1], nm), cc)));
      }
    }
    float s0, s1, s2, s3;
    f2_get(sum0, s0, s1);
    f2_get(sum1, s2, s3);
    MaxSum ms = {m, (s0 + s1) + (s2 + s3)};
    if (loose >= 0) ms.s += exp_scaled(xl + z, r.c);
    ms = warp_join(ms, r.inv_tf);
    if (G > 1) {
      // x_y goes with the sums: it has been read before any warp of the group
      // may write the gradient over the logits
      if (lane == 0) part[par][warp] = make_float4(ms.m, ms.s, xy, 0.f);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(kThreads) : "memory");
      const float4 got = part[par][group * G + (lane < G ? lane : 0)];
      xy = __shfl_sync(~0u, got.z, 0);
      ms = warp_join<G>(lane < G ? MaxSum{got.x, got.y} : MaxSum{-INFINITY, 0.f}, r.inv_tf);
      ms.s = __shfl_sync(~0u, ms.s, 0);
      par ^= 1;
    }
    // ---- the row's scalars
    const LogSum ls = log_sum(ms.s);
    const float d = xy - ms.m;
    if (gtid == 0) {
      if (a.row != nullptr) a.row[t] = make_float4(ms.m, ms.s, xy, 0.f);
      if (a.logp != nullptr) a.logp[t] = log_ratio(d, r.inv_tf, 0.f, ls);
    }
    if (!POLICY) continue;
    const PolicyTerm o = policy_term(a.p, log_ratio(d, r.inv_tf, old, ls),
                                     -log_ratio(d, r.inv_tf, ref, ls), adv);
    const float coef = scale * w * o.slope;
    sum += (double)(lane == 0 ? w * o.policy : lane == 1 ? w * o.kl : w);
    // ---- the gradient
    if (a.grad == nullptr) continue;
    T* g = a.grad + t * a.grad_ld;
    if (coef == 0.f) {
      zero_share(g, r.V, 0, 0, gtid, kThreads);
      continue;
    }
    const float zm = finite_max(ms.m), b = -coef / ms.s;
    const bool near = short_exponent<T>(zm, r.c);
    const bool same = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
    const F2 nz = f2(-zm, -zm), b2 = f2(b, b), c0 = f2(r.c.hi, r.c.hi);
    const F2 kk = f2(-zm * r.c.hi, -zm * r.c.hi);
    uint4* out = reinterpret_cast<uint4*>(g + s.head) + gtid;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (j * kThreads + gtid >= s.nvec) break;
      Pairs<T> e;
      unpack(q[j], e);
      float v[VE];
#pragma unroll
      for (int i = 0; i < VE / 2; ++i)
        f2_get(f2_mul(near ? exp2_pair(f2_fma(e.p[i], c0, kk)) : exp_pair(e.p[i], nz, c2), b2),
               v[2 * i], v[2 * i + 1]);
      if (same) {
        __stcs(out + j * kThreads, pack_vec<T>(v));
      } else {
        T* at = g + s.head + (j * kThreads + gtid) * VE;
#pragma unroll
        for (int i = 0; i < VE; ++i) at[i] = from_f<T>(v[i]);
      }
    }
    if (loose >= 0) {
      const float e = b * exp_scaled(xl - zm, r.c);
      g[loose] = from_f<T>(loose == y ? e + coef : e);
    }
    // the target's element again, by the thread that wrote it
    const int32_t ye = y - s.head;
    if (ye >= 0 && ye / VE < s.nvec && gtid == (ye / VE & (kThreads - 1)))
      g[y] = from_f<T>(b * exp_scaled(xy - zm, r.c) + coef);
  }
  if (!POLICY) return;
  // the CTA's sums, then, by the last CTA to finish, all of them in their order
  if (lane < 3) sums[warp][lane] = warp % G == 0 ? sum : 0.0;
  __syncthreads();
  if (warp > 0) return;
  uint32_t last = 0;
  if (lane < 3) {
    double v = 0.0;
    for (int i = 0; i < 8; ++i) v += sums[i][lane];
    a.partial[3 * blockIdx.x + lane] = v;
    __threadfence();
  }
  __syncwarp();
  if (lane == 0) {
    last = atomicAdd(&a.head->ticket, 1u) + 1 == gridDim.x;
    __threadfence();
  }
  if (!__shfl_sync(~0u, last, 0)) return;
  policy_stats(a, gridDim.x, lane);
}
