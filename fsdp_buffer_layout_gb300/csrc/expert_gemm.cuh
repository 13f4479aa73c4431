// expert_gemm.cuh — the products of rows sorted by expert with their experts'
// weights, on the fifth-generation tensor cores (tcgen05, sm_103a). Included by
// experts.cu after tcgen05.cuh.
//
// Expert e owns rows [starts[e], starts[e + 1]) of x [R, K] and y [R, N] and the
// weights W[e] [N, K]. bf16 operands and outputs, fp32 accumulation in tensor
// memory, one rounding. The three products, as D[i][j] = sum_r A[i][r] B[j][r]:
//   kForward    y  = x W^T     i: N (A = W, K-major)    j: rows (x, K-major)   r: K
//   kInput      dx = dy W      i: K (A = W, MN-major)   j: rows (dy, K-major)  r: N
//   kWeight     dW = dy^T x    i: N (A = dy, MN-major)  j: K (x, MN-major)     r: rows
// The weights' side is the 256 lanes of a tile, the rows are its columns: a
// tensor-core product has 128 or 256 lanes but any multiple of 32 columns, and
// experts have any number of rows. So an expert with few rows costs a narrow tile,
// and one that streams its weights costs little more than their bytes. Columns
// behind an expert's last row are computed from what lies there (the next
// expert's rows, or zeros behind the last row of all) and not stored: columns do
// not mix. Where rows are what is summed over (kWeight) they would: there the rows
// of the last stage that are not the expert's, up to the next 16, are zeroed in
// shared memory before the products read them.
//
// Pairs of CTAs compute tiles of 256 lanes with cta_group::2, each CTA half of the
// lanes, as ns_gemm.cuh does: a ring of six stages of 64 of r, two accumulators.
//   warp 0      producer: this CTA's halves of both operands' stages;
//   warp 1      TMEM; one lane of the leader's issues the products;
//   warps 2..5  epilogue, in both CTAs;
//   warp 6      (kWeight) zeroes, in its CTA, the rows that are not the expert's.
// Persistent: one pair of CTAs for two SMs, tiles dealt out in turn. The tiles
// depend on starts, which is device memory: every CTA works out the experts'
// tiles for itself before it begins. Every wait is bounded (mbarrier.cuh), and a
// broken pipeline ends as in ns_gemm.cuh.
//
// Measured (GB300): 8 experts of 4096 rows, 4096 x 4096: 560 to 580 us forward, 1890
// to 1970 TFLOP/s (torch's one product of as many FLOPs 1870 to 1940 in the same
// runs); 32 of 1024 rows, 5632 x 2816: 550 to 575 us forward, 600 to 620 input
// gradient, 620 to 655 weight gradient; the tensor pipe is busy in 91 percent of the
// cycles, and calls in a row for longer than some 0.1 s are slower by the card's
// power limit (32 of 1024 rows, 5760 x 2880, for 2 s: 1603, 1538 and 1520 TFLOP/s, torch's
// batched products 1618, 1487 and 1423, its one product of 8192^3 1693). 32 experts of 16 rows, 5760 x 2880: 163 us, 6.6 TB/s of weights; their
// weight gradient 255 us, 4.2 TB/s written (torch's fill of as much: 4.0). Bound by a
// call's fixed 5 us, a tile's first loads and its epilogue (2 us) where there are few
// tiles of little depth.
// A tile sums its whole depth on one pair of SMs, 0.2 to 0.3 us for 64 of r, whatever
// number of pairs is idle, and has 256 lanes, however few the weights' side has. So few
// tiles of a long depth take several times their bytes' time: the weight gradients of 4
// experts of 8192 rows, 256 x 256, 41 us (5 us of bytes), of 2 of 65536 rows, 64 x 64, 179
// (5); forward of 4 of 64 rows, 8192 deep to 256 lanes, 28 (3). And a narrow side pays for
// 256 lanes: 8 experts of 4096 rows, forward 64 deep to 4096 lanes 103 us, its input
// gradient with 64 lanes and 4096 deep 56 (41 us of bytes each).
// Measured and not kept: eight epilogue warps (2700 rows of 13 experts, 1001 x 523, 10.1
// us instead of 10.8, but 626 instead of 614 for 32768 rows, 5760 x 2880); the
// accumulator's next columns read while the ones before are stored, which needs the
// weight gradient's copies to be 32 columns wide (305 us instead of 262 for the small
// one above); waiting threads that spin instead of sleep (554 us instead of 501).

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
// What is left of a wait whose first try failed, out of line: a call of a few tiles waits
// for its code as well (13 experts of some 200 rows, 1001 x 523, the three products: 41.4
// us, with a copy at each wait 42.1).
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, unsigned* err, volatile uint32_t* stop,
                                     uint64_t limit_ns) {
  return mbar_wait_rest(bar, parity, err, stop, limit_ns);
}
__device__ __noinline__ bool wait_on_cluster(uint32_t bar, uint32_t parity, unsigned* err,
                                             volatile uint32_t* stop, uint64_t limit_ns) {
  return mbar_wait_rest_cluster(bar, parity, err, stop, limit_ns);
}
__device__ __noinline__ bool wait_on_moving(uint32_t bar, uint32_t parity, unsigned* err,
                                            volatile uint32_t* stop, uint64_t limit_ns,
                                            const volatile uint32_t* moved) {
  return mbar_wait_rest_moving(bar, parity, err, stop, limit_ns, moved);
}
// The waits of a whole warp: all of its lanes go on, or none does.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned* err, volatile uint32_t* stop,
                                          uint64_t limit_ns) {
  return __all_sync(~0u, mbar_try(bar, parity) || wait_on(bar, parity, err, stop, limit_ns));
}
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, unsigned* err,
                                                  volatile uint32_t* stop, uint64_t limit_ns) {
  return __all_sync(~0u, mbar_try_cluster(bar, parity) || wait_on_cluster(bar, parity, err, stop, limit_ns));
}
// For a tile's end or the next mended stage: as long as the producer's stages go by.
__device__ __forceinline__ bool warp_wait_moving(uint32_t bar, uint32_t parity, unsigned* err,
                                                 volatile uint32_t* stop, uint64_t limit_ns,
                                                 const volatile uint32_t* moved) {
  return __all_sync(~0u, mbar_try(bar, parity) || wait_on_moving(bar, parity, err, stop, limit_ns, moved));
}

enum { kForward = 0, kInput = 1, kWeight = 2 };

constexpr int kXStages = 6;
constexpr int kXDepth = 64;                            // of r a stage
constexpr int kXLanes = 256;                           // of a tile
constexpr int kXCols = 256;                            // of a tile, at most
constexpr int kMaxGroups = 512;                        // experts
constexpr int kXBlock = 8;                             // pieces of rows side by side
constexpr int32_t kXBeat = 256 * kXDepth;              // of r, after which a producer says that it moves on
constexpr uint32_t kXHalf = 128 * kXDepth * 2;         // one operand's half of a stage: 16 KB
constexpr uint32_t kXStage = 2 * kXHalf;
constexpr uint32_t kXBars = 3 * kXStages + 5;
struct XTable {
  int32_t first[kMaxGroups + 1];  // tiles in front of each expert's
  int32_t start[kMaxGroups + 1];  // its first row
  uint32_t tmem, stop, moved;     // (moved: this CTA's producer, stages)
  int32_t most;                   // rows of a tile at most, 2^most (kForward, kInput)
  PairEnd end;
};
constexpr uint32_t kXOut = 4096;  // of each epilogue warp: 32 lanes x 64 columns, or two of 32 x 32
constexpr uint32_t kXSmem =
    kXStages * kXStage + 4 * kXOut + 8 * kXBars + (uint32_t)sizeof(XTable) + 1024;
static_assert(kXSmem <= 227 * 1024, "fits in shared memory");

struct ExpertArgs {
  const int32_t* starts;
  int32_t E, rows;    // experts; rows of the arrays
  int32_t lanes;      // extent of i
  int32_t cols;       // kWeight: extent of j
  int32_t depth;      // kForward, kInput: extent of r
  int32_t lane_tiles, col_tiles;
  uint16_t* out;
  int64_t ld, stride; // of out's rows; kWeight: of its experts
  PairLimits limits;
};

struct XTile {
  int32_t e, lane0;   // expert, first lane (of the pair)
  int32_t col0;       // first row (kWeight: first column)
  int32_t width;      // columns computed: a multiple of 32 (kWeight: 128 or 256)
  int32_t cols;       // columns stored
  int32_t row0, depth;  // what is summed over
};

// Of one CTA's copies into a stage; whether the stage of r from k0 on is mended (below).
__device__ __forceinline__ uint32_t stage_bytes(const XTile& q) {
  return kXHalf + (uint32_t)(q.width / 2) * (kXDepth * 2);
}
template <int KIND>
__device__ __forceinline__ bool mended_stage(const XTile& q, int32_t k0) {
  return KIND == kWeight && k0 + kXDepth > q.depth && (q.depth & 15) != 0;
}

// An expert's rows in tiles of at most `most`, as even as can be in units of 32: one of
// 256 and a narrow one would cost more than half a tile for the narrow one, and as many
// of one width compute up to an eighth too many. `most` is 256, or 128 where the tiles
// of that are no more than the pairs of CTAs: 4 experts of 256 rows, 1024 x 4096, 19.8 us
// instead of 25.3, 4 of 1190 rows, 64 x 4352, 21.7 instead of 26.3. (With 64 as well 19.7
// and 20.5, but 8 of 128 rows, 1024 x 4096, 20.5 instead of 20.0, weights read more often.)
constexpr int kXMost = 8, kXLeast = 7;  // 2^8, 2^7
__device__ __forceinline__ int32_t token_tiles(int32_t rows, int32_t most) { return (rows + (1 << most) - 1) >> most; }

// Tile t of the launch, for a converged warp; `e` moves on from tile to tile.
template <int KIND>
__device__ __forceinline__ XTile tile_at(const ExpertArgs& a, const XTable& x, int32_t t, int32_t& e) {
  XTile q;
  if (KIND == kWeight) {
    const int32_t per = a.lane_tiles * a.col_tiles;
    q.e = t / per;
    const int32_t k = t - q.e * per, col = k / a.lane_tiles;
    q.lane0 = (k - col * a.lane_tiles) * kXLanes;
    q.col0 = col * kXCols;
    q.cols = min(kXCols, a.cols - q.col0);
    q.width = q.cols > 128 ? 256 : 128;
    q.row0 = x.start[q.e];
    q.depth = x.start[q.e + 1] - q.row0;
  } else {
    // 32 experts at a time (one after the other the walk bound a launch of many small
    // experts: 512 of 4 rows, 256 x 64, 29 us instead of 16)
    for (int32_t n = 32; n == 32;) {
      const int32_t k = e + 1 + (int32_t)(threadIdx.x & 31);
      n = __popc(__ballot_sync(~0u, k <= a.E && t >= x.first[k]));
      e += n;
    }
    q.e = e;
    // eight pieces of rows at a time take a lane tile one after the other: its
    // weights come from memory once, and are asked for by fewer pairs at a time (2 to 4
    // percent for 32 experts of 1024 rows, against all lane tiles of a piece in turn)
    const int32_t begin = x.start[e], rows = x.start[e + 1] - begin, pieces = token_tiles(rows, x.most);
    int32_t k = t - x.first[e];
    const int32_t block = k / (kXBlock * a.lane_tiles) * kXBlock, n = min(kXBlock, pieces - block);
    k -= block * a.lane_tiles;
    const int32_t lane_tile = k / n, piece = block + k - lane_tile * n;
    q.lane0 = lane_tile * kXLanes;
    const int32_t unit = (rows + 31) / 32, unit0 = (int32_t)((int64_t)unit * piece / pieces);
    q.width = 32 * ((int32_t)((int64_t)unit * (piece + 1) / pieces) - unit0);
    q.col0 = begin + 32 * unit0;
    q.cols = min(q.width, begin + rows - q.col0);
    q.row0 = 0;
    q.depth = a.depth;
  }
  return q;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int KIND>
constexpr int kXThreads = KIND == kWeight ? 224 : 192;

// Tensor maps: the lanes' operand; the columns' operand, in boxes of 16, 32, 64 and
// 128 rows (kWeight: of 64 x 64, the first alone); the output, in boxes of 32 rows of
// 32 elements (kWeight: of 64).
// A copy to memory leaves out what lies behind a map's width in whole pieces of 16 bytes
// only: of the last piece it writes all. So the output's map ends at its last whole
// piece, whole_pieces(width), and the up to seven elements behind it are stored by the
// lanes, a row each (13 experts of some 200 rows, 1001 x 523, the three products: 42.4 us;
// by two lanes of 16 rows, or an element at a time, 47.0).
__host__ __device__ constexpr int32_t whole_pieces(int32_t width) { return width & ~7; }
// n elements, 1 to 7, of a piece in shared memory.
__device__ __forceinline__ void store_rest(uint16_t* to, uint32_t from, int32_t n) {
  uint32_t a, b, c, d;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(from));
  if (n & 4) {
    *reinterpret_cast<uint2*>(to) = make_uint2(a, b);
    to += 4;
    a = c;
    b = d;
  }
  if (n & 2) {
    *reinterpret_cast<uint32_t*>(to) = a;
    to += 2;
    a = b;
  }
  if (n & 1) *to = (uint16_t)a;
}
struct XMaps {
  CUtensorMap lanes, cols[4], out;
};

template <int KIND>
__global__ void __launch_bounds__(kXThreads<KIND>, 1)
    expert_gemm_kernel(const __grid_constant__ XMaps maps, const ExpertArgs g, unsigned* err) {
  constexpr bool AMN = KIND != kForward, BMN = KIND == kWeight;
  extern __shared__ __align__(1024) unsigned char raw[];
  unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t s0 = smem_u32(sm), out0 = s0 + kXStages * kXStage, bar0 = out0 + 4 * kXOut;
  XTable& table = *reinterpret_cast<XTable*>(sm + kXStages * kXStage + 4 * kXOut + 8 * kXBars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kXStages + s); };
  auto tfull_bar = [&](int i) { return bar0 + 8u * (2 * kXStages + i); };
  auto tempty_bar = [&](int i) { return bar0 + 8u * (2 * kXStages + 2 + i); };
  const uint32_t done_bar = bar0 + 8u * (2 * kXStages + 4);
  auto own_bar = [&](int s) { return done_bar + 8u + 8u * s; };
  volatile uint32_t* stop = &table.stop;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const bool leader = rank == 0;
  const int cid = blockIdx.x / 2, ncid = gridDim.x / 2;
  constexpr uint16_t kBoth = 3;

  if (threadIdx.x == 0) {
    table.stop = table.moved = table.end.loaded = table.end.early = 0u;
    for (int s = 0; s < kXStages; ++s) {
      // kWeight: both CTAs' warps 6 arrive for a mended stage, the leader's producer twice
      // for others (by one of its warps 6 after the other: a row more or less an expert
      // made 32 of 1024 rows, 5760 x 2880, 755 us instead of 730)
      mbar_init(full_bar(s), KIND == kWeight ? 2 : 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(own_bar(s), 1);  // kWeight: this CTA's copies of a stage to be mended
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull_bar(i), 1);
      mbar_init(tempty_bar(i), 8);  // every epilogue warp of both CTAs
    }
    mbar_init(done_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&table.tmem), 2 * kXCols);
    tmem_relinquish_pair();
  }
  take_turn();
  // the experts' rows, in order and inside the arrays whatever starts holds
  for (int e = threadIdx.x; e <= g.E; e += kXThreads<KIND>)
    table.start[e] = min(max(g.starts[e], 0), g.rows);
  __syncthreads();
  if (warp == 2) {
    // each lane takes a run of experts: their running maximum, their tiles
    const int per = (g.E + 32) / 32, begin = min(lane * per, g.E + 1), end = min(begin + per, g.E + 1);
    int32_t top = 0;
    for (int e = begin; e < end; ++e) table.start[e] = top = max(top, table.start[e]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(~0u, top, o);
      if (lane >= o) top = max(top, v);
    }
    int32_t low = __shfl_up_sync(~0u, top, 1);
    if (lane == 0) low = 0;
    for (int e = begin; e < end; ++e) table.start[e] = max(low, table.start[e]);
    __syncwarp();
    int32_t tiles = 0, narrow = 0;
    for (int e = begin; e < min(end, g.E); ++e) {
      const int32_t rows = table.start[e + 1] - table.start[e];
      tiles += token_tiles(rows, kXMost) * g.lane_tiles;
      narrow += token_tiles(rows, kXLeast) * g.lane_tiles;
    }
    int32_t most = kXMost;
    if (KIND != kWeight && __reduce_add_sync(~0u, narrow) <= ncid) {
      most = kXLeast;
      tiles = narrow;
    }
    if (lane == 0) table.most = most;
    int32_t at = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(~0u, at, o);
      if (lane >= o) at += v;
    }
    at -= tiles;
    for (int e = begin; e < end; ++e) {
      table.first[e] = at;
      if (e < g.E) at += token_tiles(table.start[e + 1] - table.start[e], most) * g.lane_tiles;
    }
  }
  tc_fence_before();
  cluster_barrier();
  tc_fence_after();
  const uint32_t tmem = table.tmem;
  // the leader's products write both CTAs' accumulators at the leader's address
  if (threadIdx.x == 0 && ld_peer_u32(peer_addr(smem_u32(&table.tmem), (uint32_t)(rank ^ 1))) != tmem) {
    atomicOr(err, 8u);
    table.stop = 1u;
    remote_stop(stop, (uint32_t)(rank ^ 1));
  }
  cluster_barrier();
  const int32_t ntiles =
      KIND == kWeight ? g.E * g.lane_tiles * g.col_tiles : table.first[g.E];
  const uint32_t leader_full0 = peer_addr(full_bar(0), 0);
  const uint32_t leader_tempty0 = peer_addr(tempty_bar(0), 0);
  auto halt_cluster = [&]() { remote_stop(stop, (uint32_t)(rank ^ 1)); };

  if (warp == 0) {
    if (__all_sync(~0u, *stop == 0u)) {
      // ---------------- producer (both CTAs), one lane of a whole warp as for the products
      const bool one = elect_one();
      const uint32_t own0 = peer_addr(own_bar(0), (uint32_t)rank);
      uint32_t it = 0, mended = 0, phases = 0;  // stages mended so far; how often, modulo 2
      const int32_t end = last_tile(g.limits, leader, ntiles, cid, ncid);
      int s = 0;
      uint32_t phase = 1;
      int32_t e = 0;
      bool halted = false;
      for (int32_t t = cid; t < end && !halted; t += ncid) {
        const XTile q = tile_at<KIND>(g, table, t, e);
        const int32_t half = q.width / 2;
        const int32_t lane0 = q.lane0 + rank * 128, col0 = q.col0 + rank * half;
        const int largest = 27 - __clz(half);  // box of 16 << largest rows
        const int32_t box = 16 << largest;
        const CUtensorMap* cols = &maps.cols[KIND == kWeight ? 0 : largest];
        const uint32_t bytes = stage_bytes(q);
        // (with a store and a comparison for each stage the weight gradient of 2 experts of
        // 16384 rows, 64 x 64, took 61.7 us instead of 55.4)
        for (int32_t k0 = 0, beat = 0; beat < q.depth && !halted;) {
          if (one) table.moved = it;
          beat = q.depth - beat > kXBeat ? beat + kXBeat : q.depth;
          for (; k0 < beat; k0 += kXDepth) {
            if (!warp_wait(empty_bar(s), phase, err, stop, g.limits.wait_ns)) {
              halted = true;
              if (one) halt_cluster();
              break;
            }
            ++it;
            uint32_t fb = leader_full0 + 8u * s;
            if (mended_stage<KIND>(q, k0)) {
              fb = own0 + 8u * s;  // warp 6 mends the stage and then arrives
              if (one) mbar_expect_tx(own_bar(s), bytes);
              mended |= 1u << s;
              phases ^= 1u << s;
            } else if (leader && one) {
              mbar_expect_tx(full_bar(s), 2 * bytes);
              if (KIND == kWeight) mbar_arrive(full_bar(s));
            }
            const uint32_t a = s0 + s * kXStage, b = a + kXHalf;
            if (!one) {
            } else if (KIND == kWeight) {
              const int32_t r = q.row0 + k0;
              tma3_g2s_pair(a, &maps.lanes, lane0, r, 0, fb);
              tma3_g2s_pair(a + 8192u, &maps.lanes, lane0 + 64, r, 0, fb);
              tma3_g2s_pair(b, &maps.cols[0], col0, r, 0, fb);
              if (half > 64) tma3_g2s_pair(b + 8192u, &maps.cols[0], col0 + 64, r, 0, fb);
            } else {
              if (AMN) {
                tma3_g2s_pair(a, &maps.lanes, lane0, k0, q.e, fb);
                tma3_g2s_pair(a + 8192u, &maps.lanes, lane0 + 64, k0, q.e, fb);
              } else {
                tma3_g2s_pair(a, &maps.lanes, k0, lane0, q.e, fb);
              }
              // the columns' half in boxes of 128, 64, 32 and 16 rows, each once at most
              // (seven of 16 for 112 rows ran at 970 TFLOP/s instead of 1470)
              tma3_g2s_pair(b, cols, k0, col0, 0, fb);
              for (int32_t rest = half - box, c = box; rest != 0;) {
                const int i = 27 - __clz(rest);
                tma3_g2s_pair(b + (uint32_t)c * 128u, &maps.cols[i], k0, col0 + c, 0, fb);
                c += 16 << i;
                rest -= 16 << i;
              }
            }
            __syncwarp();
            if (++s == kXStages) {
              s = 0;
              phase ^= 1u;
            }
          }
        }
      }
      // every copy lands before the CTA ends: the leader sees both CTAs' (the
      // follower's are covered by its wait and pair_end)
      if (one) {
        pair_loaded(table.end, it, leader && (halted || end < ntiles));
        const uint64_t deadline = global_ns() + kWaitNs;
        for (int s = 0; KIND == kWeight && s < kXStages; ++s)
          if (mended >> s & 1u) mbar_drain(own_bar(s), (phases >> s & 1u) ^ 1u, deadline, err);
        if (leader) {
          for (int s = 0; s < kXStages; ++s) {
            if (it > (uint32_t)s) {
              const uint32_t last = (it - 1 - s) / kXStages * kXStages + s;
              mbar_drain(full_bar(s), (last / kXStages) & 1u, deadline, err);
            }
          }
        }
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    if (leader && __all_sync(~0u, *stop == 0u)) {
      // ---------------- products (leader only). What is done for a stage has to fit the
      // tensor cores' time for it, 512 cycles of 256 columns. So the descriptors' low
      // words are counted on (their high words do not change), and the whole warp goes
      // through the loop, whose values are then the warp's and not a lane's; one lane
      // issues. (Of 44 stages a tile took, in us, of 32, 128 and 256 columns: one lane
      // and descriptors made anew 14.4, 14.6, 15.8; one lane 11.2, 11.4, 14.0; so 7.8,
      // 9.0, 13.9 = 2010 TFLOP/s.)
      const bool one = elect_one();
      constexpr uint64_t kDescA = operand_desc<AMN>(0u, 0), kDescB = operand_desc<BMN>(0u, 0);
      constexpr uint32_t kStepA = AMN ? 2048u >> 4 : 32u >> 4, kStepB = BMN ? 2048u >> 4 : 32u >> 4;
      const uint32_t a0 = (uint32_t)kDescA + (s0 >> 4), b0 = (uint32_t)kDescB + ((s0 + kXHalf) >> 4);
      int s = 0;
      uint32_t phase = 0;
      int32_t e = 0;
      int lt = 0;
      bool halted = false;
      for (int32_t t = cid; t < ntiles && !halted; t += ncid, ++lt) {
        const XTile q = tile_at<KIND>(g, table, t, e);
        const uint32_t idesc = umma_idesc_bf16(AMN, BMN, kXLanes, q.width);
        const int buf = lt & 1;
        if (!warp_wait_cluster(tempty_bar(buf), ((uint32_t)(lt >> 1) & 1u) ^ 1u, err, stop, g.limits.wait_ns)) {
          if (one) halt_cluster();
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * kXCols);
        uint32_t more = 0;
        for (int32_t left = q.depth; left > 0; left -= kXDepth) {
          if (!warp_wait_cluster(full_bar(s), phase, err, stop, g.limits.wait_ns)) {
            halted = true;
            if (one) halt_cluster();
            break;
          }
          tc_fence_after();
          const uint32_t a = a0 + (uint32_t)s * (kXStage >> 4), b = b0 + (uint32_t)s * (kXStage >> 4);
          auto step = [&](int kk, uint32_t accumulate) {
            umma_pair_words(d, a + kk * kStepA, (uint32_t)(kDescA >> 32), b + kk * kStepB,
                            (uint32_t)(kDescB >> 32), idesc, accumulate);
          };
          // (what a stage holds past the depth is zeros, or mended to the next 16)
          if (one) {
            step(0, more);
            if (left > 48) {
              step(1, 1);
              step(2, 1);
              step(3, 1);
            } else {
              if (left > 16) step(1, 1);
              if (left > 32) step(2, 1);
            }
            umma_pair_commit(empty_bar(s), kBoth);
          }
          __syncwarp();
          more = 1;
          if (++s == kXStages) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (!halted && one) umma_pair_commit(tfull_bar(buf), kBoth);
        __syncwarp();
      }
      if (one) {
        umma_pair_commit(done_bar, 1);  // this CTA only
        mbar_drain(done_bar, 0u, global_ns() + kWaitNs, err);
      }
      __syncwarp();
    }
  } else if (warp < 6) {
    // ---------------- epilogue (both CTAs): this CTA's 128 lanes
    const int quarter = warp & 3;
    int32_t e = 0;
    int lt = 0;
    uint32_t turn = 0;
    for (int32_t t = cid; t < ntiles; t += ncid, ++lt) {
      const int buf = lt & 1;
      if (!warp_wait_moving(tfull_bar(buf), (uint32_t)(lt >> 1) & 1u, err, stop, g.limits.wait_ns, &table.moved)) {
        if (lane == 0) halt_cluster();
        break;
      }
      tc_fence_after();
      // The accumulator is free once its last columns are in registers: said before
      // they are stored, as the arrival (a release) waits for the warp's stores.
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(leader_tempty0 + 8u * buf);
      };
      const XTile q = tile_at<KIND>(g, table, t, e);
      const int32_t i = q.lane0 + rank * 128 + 32 * quarter + lane;
      const uint32_t from = tmem + (uint32_t)(buf * kXCols) + ((uint32_t)(32 * quarter) << 16);
      if (KIND == kWeight) {
        // A lane holds 64 columns of its row at a time. Through shared memory, in
        // the swizzle of the tensor copies (16-byte piece p of row l at p ^ (l & 7)),
        // and out as one copy of 32 rows: 32 lanes' stores to 32 rows took 1640 us
        // for 32 experts of 1024 rows, 5760 x 2880.
        const uint32_t to = out0 + (uint32_t)quarter * kXOut;
        const uint32_t mine = to + (uint32_t)lane * 128u;
#pragma unroll 1
        for (int32_t c = 0; c < q.cols; c += 64) {
          uint32_t p[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            __syncwarp();
            tmem_ld32(from + c + 32 * h, r);
            if (h == 1 && c + 64 >= q.cols) release();
#pragma unroll
            for (int x = 0; x < 16; ++x)
              p[16 * h + x] = q.depth == 0 ? 0u : pack_bf16(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1]));
          }
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int w = 0; w < 8; ++w)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + (uint32_t)((w ^ (lane & 7)) * 16)),
                         "r"(p[4 * w]), "r"(p[4 * w + 1]), "r"(p[4 * w + 2]), "r"(p[4 * w + 3])
                         : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          const int32_t whole = whole_pieces(g.cols), at = whole - (q.col0 + c);  // (see whole_pieces)
          if (lane == 0 && at > 0 && q.lane0 + rank * 128 + 32 * quarter < g.lanes) {
            asm volatile(
                "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                    reinterpret_cast<uint64_t>(&maps.out)),
                "r"(q.col0 + c), "r"(q.lane0 + rank * 128 + 32 * quarter), "r"(q.e), "r"(to)
                : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
          if (whole != g.cols && at < 64 && i < g.lanes)
            store_rest(g.out + q.e * g.stride + i * g.ld + whole,
                       mine + (uint32_t)((at / 8 ^ (lane & 7)) * 16), g.cols - whole);
        }
      }
#pragma unroll 1
      for (int32_t c = 0; KIND != kWeight && c < q.cols; c += 32) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld32(from + c, r);
        if (c + 32 >= q.cols) release();
        {
          // Lane pairs trade columns: an even lane keeps column x and gets its
          // neighbour's, an odd one column x + 1, so that each has two adjacent
          // elements of a row. 32 whole rows go out through shared memory as one
          // copy, the last rows of an expert by the lanes themselves.
          const bool odd = lane & 1;
          const int32_t n = q.cols - c, i2 = i & ~1, whole = whole_pieces(g.lanes);  // (see whole_pieces)
          uint32_t p[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const uint32_t give = odd ? r[x] : r[x + 1];
            const uint32_t got = __shfl_xor_sync(~0u, give, 1);
            p[x / 2] = odd ? pack_bf16(__uint_as_float(got), __uint_as_float(r[x + 1]))
                           : pack_bf16(__uint_as_float(r[x]), __uint_as_float(got));
          }
          if (n >= 32) {
            const uint32_t to = out0 + (uint32_t)quarter * kXOut + (turn++ & 1u) * (kXOut / 2);
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            __syncwarp();
            const uint32_t mine = to + (odd ? 64u : 0u) + (uint32_t)(lane >> 1) * 4u;
#pragma unroll
            for (int x = 0; x < 16; ++x)
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(mine + (uint32_t)x * 128u), "r"(p[x]) : "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            const int32_t at = whole - (i - lane);
            if (whole != g.lanes && at >= 0 && at < 32)  // a lane a row
              store_rest(g.out + (int64_t)(q.col0 + c + lane) * g.ld + whole,
                         to + (uint32_t)(lane * 64 + at * 2), g.lanes - whole);
            if (lane == 0) {
              if (i < whole)
                asm volatile(
                    "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                        reinterpret_cast<uint64_t>(&maps.out)),
                    "r"(i), "r"(q.col0 + c), "r"(0), "r"(to)
                    : "memory");
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          } else {
            uint16_t* to = g.out + (int64_t)(q.col0 + c + (odd ? 1 : 0)) * g.ld + i2;
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              if (x + (odd ? 1 : 0) < n) {
                if (i2 + 1 < g.lanes)
                  *reinterpret_cast<uint32_t*>(to + (int64_t)x * g.ld) = p[x / 2];
                else if (i2 < g.lanes)
                  to[(int64_t)x * g.ld] = (uint16_t)p[x / 2];
              }
            }
          }
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else {
    // ---------------- mending (both CTAs): rows that are not the expert's
    uint32_t it = 0, phases = 0;
    int32_t e = 0;
    for (int32_t t = cid; t < ntiles; t += ncid) {
      const XTile q = tile_at<KIND>(g, table, t, e);
      it += (uint32_t)((q.depth + kXDepth - 1) / kXDepth);
      if ((q.depth & 15) == 0) continue;
      const int s = (it - 1) % kXStages;
      if (!warp_wait_moving(own_bar(s), phases >> s & 1u, err, stop, g.limits.wait_ns, &table.moved)) {
        if (lane == 0) halt_cluster();
        break;
      }
      const int32_t from = q.depth & (kXDepth - 1), rows = 16 - (q.depth & 15);
      const int boxes = 2 + q.width / 128;  // of 64 x 64: two of A, one or two of B
      // eight lanes a box, a row at a time
      unsigned char* a = sm + s * kXStage + (lane >> 3) * 8192 + from * 128 + (lane & 7) * 16;
      for (int i = 0; i < rows && (lane >> 3) < boxes; ++i)
        *reinterpret_cast<uint4*>(a + i * 128) = make_uint4(0, 0, 0, 0);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_full0 + 8u * s);
      phases ^= 1u << s;
    }
  }
  tc_fence_before();
  // no CTA frees TMEM or leaves while the pair's products or copies may touch it
  pair_end(table.end, leader, [&](uint32_t lead, uint32_t other) {
    uint32_t k = 0;  // stage
    int32_t e = 0;
    for (int32_t t = cid; t < ntiles && k < other; t += ncid) {
      const XTile q = tile_at<KIND>(g, table, t, e);
      for (int32_t k0 = 0; k0 < q.depth && k < other; k0 += kXDepth, ++k) {
        // (a mended stage's copies come to the other CTA's own barrier)
        if (k < lead || mended_stage<KIND>(q, k0) || lane != 0) continue;
        const uint32_t s = k % kXStages;
        mbar_expect_tx(full_bar(s), stage_bytes(q));
        if (KIND == kWeight) mbar_arrive(full_bar(s));
        mbar_drain(full_bar(s), (k / kXStages) & 1u, global_ns() + kWaitNs, err);
      }
      __syncwarp();
    }
  });
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * kXCols);
  }
}
