// experts.cu — the products of rows sorted by expert with their experts' weights
// and both gradients: arguments, tensor maps and launches of expert_gemm.cuh.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <string>

#include "objective.cuh"

namespace vsf {
namespace {

using namespace obj;

#include "mbarrier.cuh"
#include "tcgen05.cuh"
#include "expert_gemm.cuh"

constexpr int64_t kMaxRows = int64_t(1) << 28;
constexpr int64_t kMaxSide = int64_t(1) << 24;

// An expert launch's arguments as the caller gives them: lhs are the rows' array
// (kWeight: d_y), rhs the weights (kWeight: x).
struct Product {
  const char* who;
  const int32_t* starts;
  int64_t rows, E, N, K;
  const uint16_t *rows_in, *other;
  int64_t rows_ld, other_ld, other_stride;  // other_stride: of weights
  uint16_t* out;
  int64_t out_ld, out_stride;
  unsigned* err;
};

bool tma_rows(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

vsf_status check(int kind, const Product& a) {
  const std::string w(a.who);
  if (a.rows < 0 || a.rows > kMaxRows || a.E < 1 || a.E > kMaxGroups || a.N < 1 || a.N > kMaxSide ||
      a.K < 1 || a.K > kMaxSide)
    return fail(VSF_ERR_ARG, w + ": sizes out of range");
  const int64_t in = kind == kForward ? a.K : a.N, to = kind == kForward ? a.N : a.K;
  auto stride_ok = [](int64_t n, int64_t ld, int64_t width) { return ld >= width && offsets_ok(n, ld); };
  const bool grad = kind == kWeight;
  if (!stride_ok(a.rows, a.rows_ld, in) || !stride_ok(grad ? a.rows : a.N, a.other_ld, a.K) ||
      !stride_ok(grad ? a.N : a.rows, a.out_ld, to))
    return fail(VSF_ERR_ARG, w + ": stride out of range");
  if (a.starts == nullptr || a.err == nullptr ||
      (a.rows > 0 && (a.rows_in == nullptr || a.other == nullptr || a.out == nullptr)) ||
      (kind == kWeight && a.out == nullptr))
    return fail(VSF_ERR_ARG, w + ": NULL pointer");
  // the experts' matrices
  const int64_t stride = a.E == 1 ? 0 : grad ? a.out_stride : a.other_stride;
  const int64_t whole = (a.N - 1) * (grad ? a.out_ld : a.other_ld) + a.K;
  if (a.E > 1 && !stride_ok(a.E, stride, whole))
    return fail(VSF_ERR_ARG, w + ": experts' stride out of range");
  if (!aligned(a.starts, 4) || !aligned(a.err, 4) || !tma_rows(a.rows_in, a.rows_ld) ||
      !tma_rows(a.other, a.other_ld) || !tma_rows(a.out, a.out_ld) ||
      stride % 8 != 0)
    return fail(VSF_ERR_ALIGN, w + ": rows have to start on 16-byte boundaries (strides of whole 8 elements)");
  // what is written overlaps nothing that is read
  auto rows_of = [](const uint16_t* p, int64_t n, int64_t ld, int64_t width) -> Area {
    return {p, n, 2 * ld, 2 * width};
  };
  auto matrices = [&](const uint16_t* p) -> Area {
    const int64_t bytes = 2 * ((a.E - 1) * stride + whole);
    return {p, 1, bytes, bytes};
  };
  const Area out = grad ? matrices(a.out) : rows_of(a.out, a.rows, a.out_ld, to);
  const int64_t starts_bytes = (a.E + 1) * 4;
  for (const Area& read : {rows_of(a.rows_in, a.rows, a.rows_ld, in),
                           grad ? rows_of(a.other, a.rows, a.other_ld, a.K) : matrices(a.other),
                           Area{a.starts, 1, starts_bytes, starts_bytes}})
    if (meet(out, read)) return fail(VSF_ERR_ARG, w + ": the output overlaps an input");
  return VSF_OK;
}

// Tensor map over [batch, rows, width] (row stride ld, batch stride bs, in
// elements), boxes of 64 elements x box_rows rows, 128-byte swizzle (or of 32
// elements, not swizzled); copies outside read zeros and write nothing, but for what is
// left of the 16 bytes that hold a row's last element.
vsf_status operand_map(CUtensorMap* map, const char* who, const uint16_t* p, int64_t width, int64_t rows,
                       int64_t batch, int64_t ld, int64_t bs, int box_rows, int box_width = 64) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = gemm_map_encoder();
  if (encode == nullptr) return fail(VSF_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(batch > 1 ? bs : ld) * 2};
  const cuuint32_t box[3] = {(cuuint32_t)box_width, (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p), dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            box_width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(VSF_ERR_CUDA, std::string(who) + ": cuTensorMapEncodeTiled failed (" +
                                  std::to_string((int)r) + ")");
  return VSF_OK;
}

// Pairs of CTAs that run at a time, looked up once a device and kind; 0 with *e
// set where that fails.
template <int KIND>
int expert_pairs(cudaError_t* e) {
  static std::mutex mu;
  static int cached[64] = {};
  int dev = 0;
  if ((*e = cudaGetDevice(&dev)) != cudaSuccess) return 0;
  if (dev < 0 || dev >= 64) {
    *e = cudaErrorInvalidDevice;
    return 0;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (cached[dev] == 0) {
    auto fn = expert_gemm_kernel<KIND>;
    *e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kXSmem);
    if (*e != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 64);
    cfg.blockDim = dim3(kXThreads<KIND>);
    cfg.dynamicSmemBytes = kXSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int got = 0;
    *e = cudaOccupancyMaxActiveClusters(&got, fn, &cfg);
    if (*e != cudaSuccess) return 0;
    cached[dev] = std::max(1, got);
  }
  return cached[dev];
}

template <int KIND>
vsf_status product(const Product& a, cudaStream_t st) {
  const int64_t lanes = KIND == kInput ? a.K : a.N;
  ExpertArgs g = {};
  g.starts = a.starts;
  g.E = (int32_t)a.E;
  g.rows = (int32_t)a.rows;
  g.lanes = (int32_t)lanes;
  g.cols = (int32_t)a.K;
  g.depth = (int32_t)(KIND == kForward ? a.K : a.N);
  g.lane_tiles = (int32_t)((lanes + kXLanes - 1) / kXLanes);
  g.col_tiles = (int32_t)((a.K + kXCols - 1) / kXCols);
  g.out = a.out;
  g.ld = a.out_ld;
  g.stride = a.out_stride;
  g.limits = pair_limits();
  // (an upper bound: the rows' share among the experts is device memory)
  const int64_t tiles = KIND == kWeight ? a.E * g.lane_tiles * g.col_tiles
                                        : (a.rows / kXCols + std::min(a.E, a.rows)) * g.lane_tiles;
  const int64_t narrow = KIND == kWeight ? tiles : ((a.rows >> kXLeast) + std::min(a.E, a.rows)) * g.lane_tiles;
  if (tiles > INT32_MAX / 4) return fail(VSF_ERR_ARG, std::string(a.who) + ": too many tiles");
  XMaps m;
  vsf_status s;
  // (a map has to have a width; where the output has no whole piece none is copied)
  const int64_t out_width = std::max<int64_t>(8, whole_pieces((int32_t)(KIND == kWeight ? a.K : lanes)));
  if (KIND == kWeight) {
    s = operand_map(&m.lanes, a.who, a.rows_in, a.N, a.rows, 1, a.rows_ld, 0, 64);
    if (s == VSF_OK) s = operand_map(&m.cols[0], a.who, a.other, a.K, a.rows, 1, a.other_ld, 0, 64);
    if (s == VSF_OK) s = operand_map(&m.out, a.who, a.out, out_width, a.N, a.E, a.out_ld, a.out_stride, 32);
    m.cols[1] = m.cols[2] = m.cols[3] = m.cols[0];
  } else {
    s = operand_map(&m.lanes, a.who, a.other, a.K, a.N, a.E, a.other_ld, a.other_stride,
                    KIND == kForward ? 128 : 64);
    for (int i = 0; i < 4 && s == VSF_OK; ++i)
      s = operand_map(&m.cols[i], a.who, a.rows_in, g.depth, a.rows, 1, a.rows_ld, 0, 16 << i);
    if (s == VSF_OK) s = operand_map(&m.out, a.who, a.out, out_width, a.rows, 1, a.out_ld, 0, 32, 32);
  }
  if (s != VSF_OK) return s;
  cudaError_t e = cudaSuccess;
  const int pairs = expert_pairs<KIND>(&e);
  if (pairs > 0)
    e = launch_behind(expert_gemm_kernel<KIND>, (unsigned)(2 * std::min<int64_t>(pairs, narrow)),
                      kXThreads<KIND>, kXSmem, 2, st, m, g, a.err);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, a.who);
}

// The weights' gradient where no expert has a row.
__global__ void __launch_bounds__(256)
    zero_weights_kernel(uint16_t* out, int64_t rows, int32_t N, int32_t K, int64_t ld, int64_t stride) {
  take_turn();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    uint16_t* to = out + r / N * stride + r % N * ld;
    for (int32_t k = threadIdx.x; k < K; k += 256) to[k] = 0;
  }
}

}  // namespace
}  // namespace vsf

using namespace vsf;

namespace {
std::mutex pair_limits_mu;
PairLimits pair_limits_now = {kWaitNs, {INT32_MAX, INT32_MAX}};
}  // namespace

PairLimits vsf::pair_limits() {
  std::lock_guard<std::mutex> lock(pair_limits_mu);
  return pair_limits_now;
}

extern "C" {

vsf_status vsf_selftest_pair_waits(uint64_t limit_ns, int32_t lead_tiles, int32_t other_tiles) {
  if (limit_ns > 1000000000ull) return fail(VSF_ERR_ARG, "vsf_selftest_pair_waits: limit above 1 s");
  std::lock_guard<std::mutex> lock(pair_limits_mu);
  pair_limits_now = {limit_ns > 0 ? limit_ns : kWaitNs,
                     {lead_tiles < 0 ? INT32_MAX : lead_tiles, other_tiles < 0 ? INT32_MAX : other_tiles}};
  return VSF_OK;
}

vsf_status vsf_expert_product(const uint16_t* x, int64_t rows, int64_t K, int64_t x_ld, const uint16_t* w,
                              int64_t E, int64_t N, int64_t w_ld, int64_t w_stride, const int32_t* starts,
                              uint16_t* y, int64_t y_ld, unsigned* d_err, void* stream) {
  vsf::Range nvtx_range("vsf_expert_product");
  const Product a = {"vsf_expert_product", starts, rows, E, N, K, x, w, x_ld, w_ld, w_stride, y, y_ld, 0, d_err};
  const vsf_status s = check(kForward, a);
  if (s != VSF_OK || rows == 0) return s;
  return product<kForward>(a, static_cast<cudaStream_t>(stream));
}

vsf_status vsf_expert_product_input_grad(const uint16_t* d_y, int64_t rows, int64_t N, int64_t d_y_ld,
                                         const uint16_t* w, int64_t E, int64_t K, int64_t w_ld,
                                         int64_t w_stride, const int32_t* starts, uint16_t* d_x,
                                         int64_t d_x_ld, unsigned* d_err, void* stream) {
  vsf::Range nvtx_range("vsf_expert_product_input_grad");
  const Product a = {"vsf_expert_product_input_grad", starts, rows, E, N, K, d_y, w, d_y_ld, w_ld, w_stride,
                     d_x, d_x_ld, 0, d_err};
  const vsf_status s = check(kInput, a);
  if (s != VSF_OK || rows == 0) return s;
  return product<kInput>(a, static_cast<cudaStream_t>(stream));
}

vsf_status vsf_expert_product_weight_grad(const uint16_t* d_y, int64_t rows, int64_t N, int64_t d_y_ld,
                                          const uint16_t* x, int64_t K, int64_t x_ld, int64_t E,
                                          const int32_t* starts, uint16_t* d_w, int64_t d_w_ld,
                                          int64_t d_w_stride, unsigned* d_err, void* stream) {
  vsf::Range nvtx_range("vsf_expert_product_weight_grad");
  const Product a = {"vsf_expert_product_weight_grad", starts, rows, E, N, K, d_y, x, d_y_ld, x_ld, 0, d_w,
                     d_w_ld, d_w_stride, d_err};
  const vsf_status s = check(kWeight, a);
  if (s != VSF_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows > 0) return product<kWeight>(a, st);
  const int64_t n = E * N;
  const cudaError_t e = launch_behind(zero_weights_kernel, (unsigned)std::min<int64_t>(n, kSms * 8), 256, 0, 1,
                                      st, d_w, n, (int32_t)N, (int32_t)K, d_w_ld, d_w_stride);
  return e == cudaSuccess ? VSF_OK : cuda_error(e, a.who);
}

}  // extern "C"
