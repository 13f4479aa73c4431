// dispatch.cu — tokens by expert: the router's choices sorted by expert, rows
// copied into that order, the experts' outputs combined with their gates, and
// the gradients of both.
//
// Choice c = t top_k + j of token t is the j-th expert it takes. The sort is a
// stable counting sort: place[c], the row of choice c, counts the choices of
// lower experts and the earlier ones of its own. With it
//   gather            rows[place[t, j]] = x[t]
//   its gradient      dx[t] = sum_j d_rows[place[t, j]]           (combine, gates 1)
//   combine           out[t] = sum_j g[t, j] y[place[t, j]]
//   its gradient      dy[place[t, j]] = g[t, j] d_out[t]
//                     dg[t, j] = sum_h d_out[t, h] y[place[t, j], h]
// All four go by token, so a token's row is read (or written) once, and sums
// over j keep their order: equal inputs give equal bits, without a floating atomic.
// HBM bounds all four: 32768 tokens of 2048 bf16, 8 of 256 experts each, 195 to 200,
// 177, 360 and 175 us (copy, combine, its gradient, the copy's), 6.1 to 6.9 TB/s read
// and written; the sort of their 262144 choices 18 us. A call on a few tokens takes 4 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <string>
#include <utility>

#include "objective.cuh"

namespace vsf {
namespace {

using namespace obj;

constexpr int64_t kMaxTokens = int64_t(1) << 23;
constexpr int kMaxChoices = 32;   // of a token
constexpr int kMaxSorted = 512;   // experts
constexpr int64_t kMaxWidth = int64_t(1) << 24;

// ------------------------------------------------------------------ the sort
// Each CTA takes a run of consecutive choices, each of its warps a part of the
// run. The first launch counts the runs' choices by expert, the second adds up
// the counts of the runs before its own (every CTA for itself: at most 64 runs
// of 512 counts, from L2) and places its run's choices in their order. Up to
// kSortOne choices one CTA does both in one launch. In us: 8192 choices of 32 experts
// by one CTA 10.1, by runs of 1024 6.7; 32768 of 32 by runs of 4096 8.9, of 1024 7.2;
// 262144 of 256 by runs of 4096 17.6, of 1024 18.5 (a CTA's share of the counts).
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxRuns = 64;
constexpr int64_t kSortRun = 1024;  // choices a CTA takes at least
constexpr int64_t kSortOne = 2048;

struct SortIn {
  const int32_t* idx;
  int32_t *starts, *source, *place;  // source: may be NULL
  int32_t* counts;                   // [runs, E]
  int64_t n, run;                    // choices; of a run
  int32_t E, runs;
};

// Choices of this warp: [begin, end) of its CTA's run.
__device__ __forceinline__ void warp_part(const SortIn& s, int64_t& begin, int64_t& end) {
  const int64_t first = blockIdx.x * s.run, last = min(s.n, first + s.run);
  const int64_t per = ((s.run + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  begin = min(last, first + (threadIdx.x >> 5) * per);
  end = min(last, begin + per);
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortIn s) {
  extern __shared__ int32_t hist[];  // [E]
  take_turn();
  for (int e = threadIdx.x; e < s.E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * s.run, last = min(s.n, first + s.run);
  for (int64_t c = first + threadIdx.x; c < last; c += kSortThreads) {
    const int32_t e = s.idx[c];
    if (e >= 0 && e < s.E) atomicAdd(hist + e, 1);  // (whole numbers: any order)
  }
  __syncthreads();
  for (int e = threadIdx.x; e < s.E; e += kSortThreads) s.counts[(int64_t)blockIdx.x * s.E + e] = hist[e];
}

template <bool ONE>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortIn s) {
  // a warp's counts, then the next row of its choices, by expert; behind them
  // the rows that lower experts and earlier runs take
  extern __shared__ int32_t next[];  // [kSortWarps, E], [E], [E]
  __shared__ int32_t sums[kSortWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = s.E;
  int32_t* before = next + kSortWarps * E;
  int32_t* all = before + E;
  take_turn();
  for (int i = tid; i < (kSortWarps + 2) * E; i += kSortThreads) next[i] = 0;
  __syncthreads();
  int64_t begin, end;
  warp_part(s, begin, end);
  int32_t* mine = next + warp * E;
  for (int64_t c = begin + lane; c < end; c += 32) {
    const int32_t e = s.idx[c];
    if (e >= 0 && e < E) atomicAdd(mine + e, 1);
  }
  if (!ONE) {
    // threads side by side on the experts, slices of the runs
    const int width = E <= 32 ? 32 : E <= 64 ? 64 : E <= 128 ? 128 : E <= 256 ? 256 : 512;
    const int slices = kSortThreads / width, slice = tid / width, e = tid & (width - 1);
    if (e < E) {
      int32_t pre = 0, sum = 0;
#pragma unroll 4
      for (int r = slice; r < s.runs; r += slices) {
        const int32_t v = __ldcg(s.counts + (int64_t)r * E + e);
        sum += v;
        if (r < (int)blockIdx.x) pre += v;
      }
      atomicAdd(before + e, pre);
      atomicAdd(all + e, sum);
    }
  }
  __syncthreads();
  // the warps' first rows within the run; the run's counts
  int32_t total = 0;
  if (tid < E) {
    int32_t at = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t v = next[w * E + tid];
      next[w * E + tid] = at;
      at += v;
    }
    total = ONE ? at : all[tid];
  }
  // the experts' first rows: a scan over at most 512 of them
  int32_t scan = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t v = __shfl_up_sync(~0u, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) sums[warp] = scan;
  __syncthreads();
  int32_t base = 0;
  for (int w = 0; w < kMaxSorted / 32; ++w)
    if (w < warp) base += sums[w];
  const int32_t first = base + scan - total;
  if (tid < E) {
    before[tid] += first;
    if (blockIdx.x == 0) {
      s.starts[tid] = first;
      if (tid == E - 1) s.starts[E] = first + total;
    }
  }
  if (tid == E - 1) sums[kSortWarps - 1] = first + total;  // (past the experts' warps, or read)
  __syncthreads();
  const int32_t routed = sums[kSortWarps - 1];
  for (int64_t c0 = begin; c0 < end; c0 += 32) {
    const int64_t c = c0 + lane;
    const int32_t e = c < end ? s.idx[c] : -1;
    const bool ok = e >= 0 && e < E;
    const uint32_t same = __match_any_sync(~0u, ok ? e : -1);
    const int rank = __popc(same & ((1u << lane) - 1));
    int32_t row = -1;
    if (ok) row = before[e] + mine[e] + rank;
    __syncwarp();
    if (ok && rank == 0) mine[e] += __popc(same);
    __syncwarp();
    if (c < end) {
      s.place[c] = row;
      if (s.source != nullptr && ok) s.source[row] = (int32_t)c;
    }
  }
  if (s.source != nullptr)
    for (int64_t r = (int64_t)routed + (int64_t)blockIdx.x * kSortThreads + tid; r < s.n;
         r += (int64_t)gridDim.x * kSortThreads)
      s.source[r] = -1;
}

// ------------------------------------------------------------- rows of tokens
// A row in units: 16 bytes where every row of a call starts on a 16-byte
// boundary (the elements behind the last whole unit one by one), else elements.
template <typename T, bool WIDE>
struct Unit;
template <typename T>
struct Unit<T, false> {
  using raw = T;
  static constexpr int n = 1;
  __device__ static __forceinline__ void get(const raw& r, float (&v)[1]) { v[0] = to_f(r); }
  __device__ static __forceinline__ raw put(const float (&v)[1]) { return from_f<T>(v[0]); }
};
template <>
struct Unit<float, true> {
  using raw = uint4;
  static constexpr int n = 4;
  __device__ static __forceinline__ void get(const raw& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  }
  __device__ static __forceinline__ raw put(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};
template <>
struct Unit<uint16_t, true> {
  using raw = uint4;
  static constexpr int n = 8;
  __device__ static __forceinline__ void get(const raw& r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static __forceinline__ raw put(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// L lanes take an item: a piece of a token's row, or a choice. A warp (L = 32), or, where
// a row is no longer than what 8 lanes hold and a token has no more than 8 choices, 8
// of them: 65536 tokens of 64 bf16, 8 choices each, took 23, 51 and 178 us (gather,
// combine, gradient) with a warp an item.
constexpr int kRowThreads = 256;
constexpr int kRowCtas = 8;  // an SM, at most
// Units of a lane in a piece, single elements and wide ones; more of the former pay for
// the copy and the sum (16384 tokens of 4097 bf16, 2 choices: sum 132 us with 4, 94 with
// 16), not for the gradient (159 us with 8, 182 with 16).
constexpr int kGatherUnits[2] = {16, 4}, kCombineUnits[2] = {16, 2}, kGradUnits[2] = {8, 4};

struct RowIn {
  int64_t T_, rows, ld, row_ld;  // tokens, rows; strides of the tokens' and of the rows' arrays
  int32_t K, H;
  const int32_t* place;
};

// The items of a group of lanes: (t, piece), every step-th. All groups of a warp go
// through as many; `on` is false where there is none.
template <int L>
struct Items {
  int64_t t, step_t;
  int32_t piece, step_p, pieces, left;
  __device__ __forceinline__ Items(int64_t T_, int32_t pieces_) : pieces(pieces_) {
    constexpr int G = 32 / L;
    const int64_t groups = (int64_t)gridDim.x * (kRowThreads / L), n = T_ * pieces;
    const int64_t warp0 = ((int64_t)blockIdx.x * kRowThreads + (threadIdx.x & ~31)) / L;
    const int64_t first = warp0 + (threadIdx.x & 31) / L;
    left = (int32_t)((n - warp0 + groups - 1) / groups);  // (of the warp's first group)
    if (warp0 >= n) left = 0;
    step_t = groups / pieces;
    step_p = (int32_t)(groups - step_t * pieces);
    t = first / pieces;
    piece = (int32_t)(first - t * pieces);
    static_assert(G >= 1, "");
  }
  __device__ __forceinline__ void next() {
    --left;
    t += step_t;
    piece += step_p;
    if (piece >= pieces) {
      piece -= pieces;
      ++t;
    }
  }
};

// rows[place[t, j]] = x[t]: a piece of a token's row, read once and written to the
// token's rows.
template <typename T, bool WIDE, int L>
__global__ void __launch_bounds__(kRowThreads)
    gather_kernel(const RowIn p, const T* __restrict__ x, T* __restrict__ rows, int32_t pieces) {
  using U = Unit<T, WIDE>;
  using raw = typename U::raw;
  constexpr int NU = kGatherUnits[WIDE];
  const int lane = threadIdx.x & (L - 1);
  const int32_t units = p.H / U::n, tail = units * U::n;
  take_turn();
  for (Items<L> it(p.T_, pieces); it.left > 0; it.next()) {
    const bool on = it.t < p.T_;
    int32_t row = on && lane < p.K ? p.place[it.t * p.K + lane] : -1;
    if (row >= p.rows) row = -1;
    const T* in = x + (on ? it.t : 0) * p.ld;
    const int32_t u0 = it.piece * (L * NU) + lane;
    const bool any = __any_sync(~0u, row >= 0);
    raw v[NU];
#pragma unroll
    for (int k = 0; k < NU; ++k)
      if (any && on && u0 + L * k < units) v[k] = reinterpret_cast<const raw*>(in)[u0 + L * k];
    const bool last = on && it.piece + 1 == pieces && tail + lane < p.H;
    T loose = T();
    if (last) loose = in[tail + lane];
    for (int j = 0; any && j < p.K; ++j) {
      const int32_t r = __shfl_sync(~0u, row, j, L);
      if (r < 0) continue;
      T* out = rows + (int64_t)r * p.row_ld;
#pragma unroll
      for (int k = 0; k < NU; ++k)
        if (u0 + L * k < units) reinterpret_cast<raw*>(out)[u0 + L * k] = v[k];
      if (last) out[tail + lane] = loose;
    }
  }
}

// out[t] = sum_j g[t, j] y[place[t, j]] (GATES), or the plain sum; in fp32, one
// choice after the other, rounded once. Four choices' loads are on their way at a time.
template <typename T, bool WIDE, bool GATES, int L>
__global__ void __launch_bounds__(kRowThreads)
    combine_kernel(const RowIn p, const T* __restrict__ y, const float* __restrict__ gates,
                   T* __restrict__ out, int32_t pieces) {
  using U = Unit<T, WIDE>;
  using raw = typename U::raw;
  constexpr int NU = kCombineUnits[WIDE], JB = 4;
  const int lane = threadIdx.x & (L - 1);
  const int32_t units = p.H / U::n, tail = units * U::n;
  take_turn();
  for (Items<L> it(p.T_, pieces); it.left > 0; it.next()) {
    const bool on = it.t < p.T_;
    int32_t row = on && lane < p.K ? p.place[it.t * p.K + lane] : -1;
    if (row >= p.rows) row = -1;
    const float gate = GATES && row >= 0 ? gates[it.t * p.K + lane] : 1.f;
    const int32_t u0 = it.piece * (L * NU) + lane;
    const bool last = on && it.piece + 1 == pieces && tail + lane < p.H;
    float acc[NU][U::n], loose = 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int q = 0; q < U::n; ++q) acc[k][q] = 0.f;
    for (int j0 = 0; j0 < p.K; j0 += JB) {
      raw v[JB][NU];
      int32_t r[JB];
      T lv[JB];
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        r[j] = __shfl_sync(~0u, row, (j0 + j) & (L - 1), L);
        if (j0 + j >= p.K) r[j] = -1;
        if (r[j] < 0) continue;
        const T* in = y + (int64_t)r[j] * p.row_ld;
#pragma unroll
        for (int k = 0; k < NU; ++k)
          if (u0 + L * k < units) v[j][k] = reinterpret_cast<const raw*>(in)[u0 + L * k];
        if (last) lv[j] = in[tail + lane];
      }
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        const float g = __shfl_sync(~0u, gate, (j0 + j) & (L - 1), L);
        if (r[j] < 0) continue;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
          float f[U::n];
          U::get(v[j][k], f);
#pragma unroll
          for (int q = 0; q < U::n; ++q) acc[k][q] = GATES ? __fmaf_rn(g, f[q], acc[k][q]) : acc[k][q] + f[q];
        }
        if (last) loose = GATES ? __fmaf_rn(g, to_f(lv[j]), loose) : loose + to_f(lv[j]);
      }
    }
    if (!on) continue;
    T* to = out + it.t * p.ld;
#pragma unroll
    for (int k = 0; k < NU; ++k)
      if (u0 + L * k < units) reinterpret_cast<raw*>(to)[u0 + L * k] = U::put(acc[k]);
    if (last) to[tail + lane] = from_f<T>(loose);
  }
}

// dy[place[t, j]] = g[t, j] d_out[t] and dg[t, j] = <d_out[t], y[place[t, j]]>, a choice
// at a time; the lanes of a token's choices read its row at about the same time, all
// but the first from L1 or L2. y and d_y may be the same rows.
template <typename T, bool WIDE, int L>
__global__ void __launch_bounds__(kRowThreads)
    combine_grad_kernel(const RowIn p, const T* __restrict__ d_out, const T* y, int64_t y_ld,
                        const float* __restrict__ gates, T* d_y, float* __restrict__ d_gates) {
  using U = Unit<T, WIDE>;
  using raw = typename U::raw;
  constexpr int NU = kGradUnits[WIDE];
  const int lane = threadIdx.x & (L - 1);
  const int32_t units = p.H / U::n, tail = units * U::n;
  take_turn();
  for (Items<L> it(p.T_, p.K); it.left > 0; it.next()) {
    const bool on = it.t < p.T_;
    const int64_t c = it.t * p.K + it.piece;
    const int32_t row = on ? p.place[c] : -1;
    const bool used = row >= 0 && row < p.rows;
    float dot[NU];
#pragma unroll
    for (int k = 0; k < NU; ++k) dot[k] = 0.f;
    if (used) {
      const float g = gates[c];
      const T* d = d_out + it.t * p.ld;
      const T* in = y + (int64_t)row * y_ld;
      T* to = d_y + (int64_t)row * p.row_ld;
      for (int32_t u0 = lane; u0 < units; u0 += L * NU) {
        raw a[NU], b[NU];
#pragma unroll
        for (int k = 0; k < NU; ++k)
          if (u0 + L * k < units) {
            a[k] = reinterpret_cast<const raw*>(d)[u0 + L * k];
            b[k] = reinterpret_cast<const raw*>(in)[u0 + L * k];
          }
#pragma unroll
        for (int k = 0; k < NU; ++k)
          if (u0 + L * k < units) {
            float fa[U::n], fb[U::n];
            U::get(a[k], fa);
            U::get(b[k], fb);
#pragma unroll
            for (int q = 0; q < U::n; ++q) {
              dot[k] = __fmaf_rn(fa[q], fb[q], dot[k]);
              fa[q] *= g;
            }
            reinterpret_cast<raw*>(to)[u0 + L * k] = U::put(fa);
          }
      }
      if (tail + lane < p.H) {
        const float a = to_f(d[tail + lane]);
        dot[0] = __fmaf_rn(a, to_f(in[tail + lane]), dot[0]);
        to[tail + lane] = from_f<T>(g * a);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k) sum += dot[k];
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (on && lane == 0) d_gates[c] = sum;
  }
}

// ------------------------------------------------------------- host side
int64_t run_of(int64_t n) {
  const int64_t run = std::max(kSortRun, (n + kMaxRuns - 1) / kMaxRuns);
  return (run + kSortWarps * 32 - 1) / (kSortWarps * 32) * (kSortWarps * 32);
}

// Counts of as many runs as any call of up to n choices takes. Their number falls
// where a run grows: 65536 choices are 64 runs, 65537 are 33.
size_t sort_bytes(int64_t n, int64_t E) {
  const int64_t runs = std::min<int64_t>(kMaxRuns, (n + kSortRun - 1) / kSortRun);
  return n <= kSortOne ? 16 : (size_t)((runs * E * 4 + 15) / 16 * 16);
}

bool sizes_ok(int64_t T_, int64_t K) {
  return T_ >= 0 && T_ <= kMaxTokens && K >= 1 && K <= kMaxChoices;
}

struct RowsArg {
  const char* who;
  int32_t dtype;
  int64_t T_, K, H;
  const int32_t* place;
};
// An array of n rows at stride ld.
struct Strided {
  const void* p;
  int64_t n, ld;
};

vsf_status check_rows(const RowsArg& a, std::initializer_list<Strided> in) {
  const std::string w(a.who);
  if (a.dtype != VSF_BF16 && a.dtype != VSF_FP32) return fail(VSF_ERR_ARG, w + ": bad dtype");
  if (!sizes_ok(a.T_, a.K) || a.H < 1 || a.H > kMaxWidth)
    return fail(VSF_ERR_ARG, w + ": sizes out of range");
  for (const Strided& s : in) {
    if (s.ld < a.H || !offsets_ok(s.n, s.ld)) return fail(VSF_ERR_ARG, w + ": stride out of range");
    if (a.T_ > 0 && s.p == nullptr) return fail(VSF_ERR_ARG, w + ": NULL pointer");
    if (!aligned(s.p, a.dtype == VSF_BF16 ? 2 : 4)) return fail(VSF_ERR_ALIGN, w + ": pointer alignment");
  }
  if (a.T_ > 0 && a.place == nullptr) return fail(VSF_ERR_ARG, w + ": NULL pointer");
  if (!aligned(a.place, 4)) return fail(VSF_ERR_ALIGN, w + ": pointer alignment");
  return VSF_OK;
}

Area area(const RowsArg& a, const Strided& s) {
  const int64_t size = a.dtype == VSF_BF16 ? 2 : 4;
  return {s.p, s.n, s.ld * size, a.H * size};
}
// A value a choice.
Area per_choice(const RowsArg& a, const void* p) {
  const int64_t bytes = a.T_ * a.K * 4;
  return {p, p != nullptr, bytes, bytes};
}
bool meets_any(const Area& out, std::initializer_list<Area> in) {
  return std::any_of(in.begin(), in.end(), [&](const Area& x) { return meet(out, x); });
}

bool all_wide(const RowsArg& a, std::initializer_list<Strided> in) {
  const int64_t size = a.dtype == VSF_BF16 ? 2 : 4;
  for (const Strided& s : in)
    if (!aligned(s.p, 16) || s.ld * size % 16 != 0) return false;
  return true;
}

// How a call's rows are taken: whether in wide units, by how many lanes, in how many
// pieces of `units` a lane; and its CTAs.
struct RowSplit {
  bool wide;
  int lanes;
  int32_t pieces;
  RowSplit(const RowsArg& a, std::initializer_list<Strided> in, const int (&units)[2]) : wide(all_wide(a, in)) {
    const int64_t n = wide ? a.H / (a.dtype == VSF_BF16 ? 8 : 4) : a.H;
    lanes = a.K <= 8 && n <= 8 * units[wide] ? 8 : 32;
    pieces = (int32_t)std::max<int64_t>(1, (n + lanes * units[wide] - 1) / (lanes * units[wide]));
  }
  unsigned grid(int64_t items) const {
    const int64_t of = kRowThreads / lanes;
    return (unsigned)std::min<int64_t>((items + of - 1) / of, kSms * kRowCtas);
  }
};
#define VSF_BY_SPLIT(F, T, s, ...)                                             \
  ((s).wide ? (s).lanes == 8 ? F<T, true, ##__VA_ARGS__, 8> : F<T, true, ##__VA_ARGS__, 32> \
            : (s).lanes == 8 ? F<T, false, ##__VA_ARGS__, 8> : F<T, false, ##__VA_ARGS__, 32>)

template <typename T>
cudaError_t launch_gather(const RowIn& p, const void* x, void* rows, const RowSplit& s, cudaStream_t st) {
  return launch_behind(VSF_BY_SPLIT(gather_kernel, T, s), s.grid(p.T_ * s.pieces), kRowThreads, 0, 1, st, p,
                       static_cast<const T*>(x), static_cast<T*>(rows), s.pieces);
}

template <typename T>
cudaError_t launch_combine(const RowIn& p, const void* y, const float* gates, void* out, const RowSplit& s,
                           cudaStream_t st) {
  auto fn = gates != nullptr ? VSF_BY_SPLIT(combine_kernel, T, s, true) : VSF_BY_SPLIT(combine_kernel, T, s, false);
  return launch_behind(fn, s.grid(p.T_ * s.pieces), kRowThreads, 0, 1, st, p, static_cast<const T*>(y), gates,
                       static_cast<T*>(out), s.pieces);
}

template <typename T>
cudaError_t launch_combine_grad(const RowIn& p, const void* d_out, const void* y, int64_t y_ld,
                                const float* gates, void* d_y, float* d_gates, const RowSplit& s,
                                cudaStream_t st) {
  return launch_behind(VSF_BY_SPLIT(combine_grad_kernel, T, s), s.grid(p.T_ * p.K), kRowThreads, 0, 1, st, p,
                       static_cast<const T*>(d_out), static_cast<const T*>(y), y_ld, gates,
                       static_cast<T*>(d_y), d_gates);
}

}  // namespace
}  // namespace vsf

using namespace vsf;

extern "C" {

size_t vsf_expert_sort_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts) {
  if (!sizes_ok(tokens, top_k) || experts < 1 || experts > kMaxSorted) return 0;
  return sort_bytes(tokens * top_k, experts);
}

vsf_status vsf_expert_sort(const int32_t* idx, int64_t T, int64_t top_k, int64_t E, int32_t* starts,
                           int32_t* source, int32_t* place, void* d_workspace, size_t ws_bytes,
                           void* stream) {
  vsf::Range nvtx_range("vsf_expert_sort");
  const char* who = "vsf_expert_sort";
  if (!sizes_ok(T, top_k) || E < 1 || E > kMaxSorted)
    return fail(VSF_ERR_ARG, "vsf_expert_sort: sizes out of range");
  if (starts == nullptr || d_workspace == nullptr || (T > 0 && (idx == nullptr || place == nullptr)))
    return fail(VSF_ERR_ARG, "vsf_expert_sort: NULL pointer");
  const int64_t n = T * top_k;
  if (ws_bytes < sort_bytes(n, E)) return fail(VSF_ERR_ARG, "vsf_expert_sort: workspace too small");
  if (!aligned(idx, 4) || !aligned(starts, 4) || !aligned(source, 4) || !aligned(place, 4) ||
      !aligned(d_workspace, 16))
    return fail(VSF_ERR_ALIGN, "vsf_expert_sort: pointer alignment");
  // what is written overlaps neither what is read nor each other
  const std::pair<const void*, int64_t> used[] = {
      {idx, n * 4}, {starts, (E + 1) * 4}, {source, source != nullptr ? n * 4 : 0}, {place, n * 4},
      {d_workspace, (int64_t)sort_bytes(n, E)}};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(used[i].first), b = reinterpret_cast<uintptr_t>(used[j].first);
      if (a < b + used[j].second && b < a + used[i].second)
        return fail(VSF_ERR_ARG, "vsf_expert_sort: arrays overlap");
    }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool one = n <= kSortOne;
  const int64_t run = one ? std::max<int64_t>(n, 1) : run_of(n);
  const int32_t runs = one ? 1 : (int32_t)((n + run - 1) / run);
  const SortIn s = {idx, starts, source, place, static_cast<int32_t*>(d_workspace),
                    n,   run,    (int32_t)E, runs};
  const unsigned smem = (unsigned)((kSortWarps + 2) * E * 4);
  auto fn = one ? sort_place_kernel<true> : sort_place_kernel<false>;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && !one)
    e = launch_behind(sort_count_kernel, runs, kSortThreads, (unsigned)(E * 4), 1, st, s);
  if (e == cudaSuccess) e = launch_behind(fn, runs, kSortThreads, smem, 1, st, s);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, who);
}

vsf_status vsf_expert_gather(const void* x, int32_t dtype, int64_t T, int64_t H, int64_t ld,
                             const int32_t* place, int64_t top_k, void* rows, int64_t rows_ld,
                             void* stream) {
  vsf::Range nvtx_range("vsf_expert_gather");
  const RowsArg a = {"vsf_expert_gather", dtype, T, top_k, H, place};
  const Strided in = {x, T, ld}, out = {rows, T * top_k, rows_ld};
  const vsf_status s = check_rows(a, {in, out});
  if (s != VSF_OK) return s;
  if (meets_any(area(a, out), {area(a, in), per_choice(a, place)}))
    return fail(VSF_ERR_ARG, "vsf_expert_gather: the output overlaps an input");
  if (T == 0) return VSF_OK;
  const RowIn p = {T, T * top_k, ld, rows_ld, (int32_t)top_k, (int32_t)H, place};
  const RowSplit w(a, {in, out}, kGatherUnits);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == VSF_BF16 ? launch_gather<uint16_t>(p, x, rows, w, st)
                                          : launch_gather<float>(p, x, rows, w, st);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, a.who);
}

vsf_status vsf_expert_combine(const void* y, int32_t dtype, int64_t T, int64_t H, int64_t y_ld,
                              const int32_t* place, const float* gates, int64_t top_k, void* out,
                              int64_t out_ld, void* stream) {
  vsf::Range nvtx_range("vsf_expert_combine");
  const RowsArg a = {"vsf_expert_combine", dtype, T, top_k, H, place};
  const Strided in = {y, T * top_k, y_ld}, to = {out, T, out_ld};
  const vsf_status s = check_rows(a, {in, to});
  if (s != VSF_OK) return s;
  if (!aligned(gates, 4)) return fail(VSF_ERR_ALIGN, "vsf_expert_combine: pointer alignment");
  if (meets_any(area(a, to), {area(a, in), per_choice(a, place), per_choice(a, gates)}))
    return fail(VSF_ERR_ARG, "vsf_expert_combine: the output overlaps an input");
  if (T == 0) return VSF_OK;
  const RowIn p = {T, T * top_k, out_ld, y_ld, (int32_t)top_k, (int32_t)H, place};
  const RowSplit w(a, {in, to}, kCombineUnits);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == VSF_BF16 ? launch_combine<uint16_t>(p, y, gates, out, w, st)
                                          : launch_combine<float>(p, y, gates, out, w, st);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, a.who);
}

vsf_status vsf_expert_combine_grad(const void* d_out, int32_t dtype, int64_t T, int64_t H,
                                   int64_t d_out_ld, const void* y, int64_t y_ld,
                                   const int32_t* place, const float* gates, int64_t top_k,
                                   void* d_y, int64_t d_y_ld, float* d_gates, void* stream) {
  vsf::Range nvtx_range("vsf_expert_combine_grad");
  const RowsArg a = {"vsf_expert_combine_grad", dtype, T, top_k, H, place};
  const Strided d = {d_out, T, d_out_ld}, in = {y, T * top_k, y_ld}, to = {d_y, T * top_k, d_y_ld};
  const vsf_status s = check_rows(a, {d, in, to});
  if (s != VSF_OK) return s;
  if (T > 0 && (gates == nullptr || d_gates == nullptr))
    return fail(VSF_ERR_ARG, "vsf_expert_combine_grad: NULL pointer");
  if (!aligned(gates, 4) || !aligned(d_gates, 4))
    return fail(VSF_ERR_ALIGN, "vsf_expert_combine_grad: pointer alignment");
  const Area from = per_choice(a, place), by = per_choice(a, gates), dg = per_choice(a, d_gates);
  if (meets_any(area(a, to), {area(a, d), from, by, dg}) ||
      (meet(area(a, to), area(a, in)) && !(y == d_y && y_ld == d_y_ld)))
    return fail(VSF_ERR_ARG, "vsf_expert_combine_grad: d_y overlaps another array (y in part)");
  if (meets_any(dg, {area(a, d), area(a, in), from, by}))
    return fail(VSF_ERR_ARG, "vsf_expert_combine_grad: d_gates overlaps an input");
  if (T == 0) return VSF_OK;
  const RowIn p = {T, T * top_k, d_out_ld, d_y_ld, (int32_t)top_k, (int32_t)H, place};
  const RowSplit w(a, {d, in, to}, kGradUnits);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == VSF_BF16
          ? launch_combine_grad<uint16_t>(p, d_out, y, y_ld, gates, d_y, d_gates, w, st)
          : launch_combine_grad<float>(p, d_out, y, y_ld, gates, d_y, d_gates, w, st);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, a.who);
}

}  // extern "C"
