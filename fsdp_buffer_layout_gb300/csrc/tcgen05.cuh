// tcgen05.cuh — what the kernels on the fifth-generation tensor cores share
// (ns_gemm.cuh: Newton-Schulz products; expert_gemm.cuh: the experts'
// products): TMEM, pair MMAs, tensor copies and cluster barriers as inline PTX
// for sm_103a, how a pair ends that was stopped, the operands' descriptors, and the
// tensor maps' encoder. Included inside a namespace by each translation unit that uses
// it, after mbarrier.cuh.
#pragma once

// ---------------------------------------------------------------- PTX wrappers

// TMEM allocation of the CTA pair: one warp of each CTA executes it, and the
// pair gets `ncols` columns at the same address in both CTAs' TMEM.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D (both CTAs' TMEM) (+)= A (both CTAs' shared memory) * B^T, kind::f16
// (bf16 here), issued by one thread of the leader CTA.
__device__ __forceinline__ void umma_pair_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with the descriptors' two words.
__device__ __forceinline__ void umma_pair_words(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                                uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n"
      " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The mbarrier at `bar` in every CTA of cta_mask receives one arrival once
// every pair MMA this thread issued before has completed.
__device__ __forceinline__ void umma_pair_commit(uint32_t bar, uint16_t cta_mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"(cta_mask)
      : "memory");
}

// 32 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 3-D tensor copy (global -> this CTA's shared memory) of one box at
// (x, y, z), completing on an mbarrier of either CTA of the pair (bar: a
// shared::cluster address).
__device__ __forceinline__ void tma3_g2s_pair(uint32_t dst, const CUtensorMap* map, int x, int y,
                                              int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// The shared::cluster address of the same offset in cluster rank `rank`.
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t ld_peer_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_peer_u32(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
// Sets the stop flag at the same shared-memory offset in cluster rank `rank`.
__device__ __forceinline__ void remote_stop(volatile uint32_t* stop, uint32_t rank) {
  st_peer_u32(peer_addr(smem_u32(const_cast<uint32_t*>(stop)), rank), 1u);
}
// Arrival on an mbarrier of the cluster (release at cluster scope).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// How a pair ends whose waits have run out. Both CTAs' copies of a stage come to the
// leader's barrier, and the leader waits for the stages that it has asked for. The other
// CTA may have loaded up to a ring of stages more by the time it sees the stop flag: it
// must not leave while those are in flight. So a leader whose producer ends early says so
// to both CTAs, and behind the cluster barrier that follows it asks for what the other
// one has loaded more and waits for it (bounded), before either leaves.
struct PairEnd {
  uint32_t loaded;  // stages that this CTA's producer has loaded
  uint32_t early;   // the leader's has not loaded all of its tiles
};
__device__ __forceinline__ void pair_loaded(PairEnd& end, uint32_t stages, bool early) {
  end.loaded = stages;
  if (early) {
    end.early = 1u;
    st_peer_u32(peer_addr(smem_u32(&end.early), 1u), 1u);
  }
}
// The end of the tiles that a CTA's producer loads: all, but for a self-test.
__device__ __forceinline__ int32_t last_tile(const PairLimits& l, bool leader, int32_t tiles, int32_t first,
                                             int32_t step) {
  const int32_t n = leader ? l.tiles[0] : l.tiles[1];
  return n >= (tiles - first) / step + 1 ? tiles : first + n * step;
}
// Called by all threads of both CTAs; ask(lead, other), by the leader's first warp: for
// the stages from `lead` on.
template <typename Ask>
__device__ __forceinline__ void pair_end(const PairEnd& end, bool leader, Ask ask) {
  __syncthreads();
  cluster_barrier();
  if (*const_cast<const volatile uint32_t*>(&end.early) == 0u) return;
  if (leader && threadIdx.x < 32) ask(end.loaded, ld_peer_u32(peer_addr(smem_u32(&end.loaded), 1u)));
  __syncwarp();
  cluster_barrier();
}

// Shared-memory matrix descriptor of tcgen05 (128-byte swizzle): start
// address, leading- and stride-dimension byte offsets (all >> 4), the fixed
// version bits 46-48 = 0b001, swizzle mode 2 (128B) in bits 61-63.
__host__ __device__ constexpr uint64_t umma_smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor of kind::f16: fp32 accumulator (bits 4-5 = 1), bf16
// A and B (bits 7-9, 10-12 = 1), A / B MN-major flags (bits 15, 16), N >> 3
// (bits 17-22), M >> 4 (bits 24-28).
__host__ __device__ constexpr uint32_t umma_idesc_bf16(bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Operand layouts in a stage (both from 128-byte-swizzled tensor copies of
// this CTA's 128 rows):
//   K-major, 128 rows x 64 K: row r at r * 128 bytes; 8-row groups 1024 bytes
//     apart (stride offset); one MMA's 16 K elements are 32 bytes of each
//     row, so K step kk starts kk * 32 bytes in.
//   MN-major, 64 K rows x 128: two boxes of 64 MN elements x 64 K rows, 8 KB
//     each, side by side (leading offset 8192 between 64-element MN groups);
//     K row k at k * 128 bytes in its box, 8-row groups 1024 bytes apart; K
//     step kk starts kk * 16 rows = kk * 2048 bytes in.
template <bool kMN>
__host__ __device__ __forceinline__ constexpr uint64_t operand_desc(uint32_t base, int kk) {
  return kMN ? umma_smem_desc(base + kk * 2048u, 8192u, 1024u)
             : umma_smem_desc(base + kk * 32u, 16u, 1024u);
}

__device__ __forceinline__ uint16_t bf16_rn(float x) {
  const __nv_bfloat16 h = __float2bfloat16_rn(x);
  return *reinterpret_cast<const uint16_t*>(&h);
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against libcuda).
inline PFN_cuTensorMapEncodeTiled_v12000 gemm_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}
