// objective.cuh — what the training objectives' kernels share (objective.cu:
// the losses over logits; route.cu: the router): element access, the
// exponential, argument checks, and the head of their workspaces.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>
#include <string>
#include <utility>

#include "vsf_internal.h"

namespace vsf {

// First words of every objective workspace, zeroed by
// vsf_objective_workspace_init and left zero by each call (but for the error
// word, which the caller reads, and `rows`).
struct WsHead {
  uint32_t err;     // device error word: see vsf.h
  uint32_t ticket;  // CTAs of the running launch that have finished
  uint32_t nan;     // a NaN score was seen (router)
  uint32_t rows;    // a loss has left its rows' sums behind the head: not for a router
  float part[16];   // parts of a loss (router)
};
static_assert(sizeof(WsHead) % 16 == 0, "what follows the head is 16-byte aligned");

constexpr uint32_t kErrTarget = 16u;  // error-word bit: a target >= V
constexpr uint32_t kErrShared = 32u;  // error-word bit: a router on a loss's workspace

namespace obj {

constexpr int kSms = 152;  // of a GB300: no grid here has more CTAs than run at a time

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f<uint16_t>(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// 2^t by the special-function unit (ex2.approx: 2 ulp; 2^-inf = 0).
__device__ __forceinline__ float ex2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

// The factor c = log2(e) / temperature. One float's rounding error would act
// like a slightly different temperature, the same way for every token, and add
// up over a sequence's log ratios. So either as a sum of two floats, hi + lo
// (both positive, however small c is: -inf times either is -inf), or, where one
// product an element has to do, rounded down (hi) in some threads and up in the
// others, in such a share (ups / 2^32) that the mean is c. c has to fit fp32: 0
// times an infinite factor would be NaN.
struct Log2Scale {
  float hi, lo, up;
  uint32_t ups;
};
constexpr float kMaxInvTemperature = 1.7014118e38f;  // 2^127
inline Log2Scale log2_scale(float inv_t) {
  const double c = (double)inv_t * 1.4426950408889634074;
  float hi = (float)c;
  if ((double)hi >= c) hi = std::nextafter(hi, 0.f);
  const float up = std::nextafter(hi, INFINITY);
  const double part = (c - (double)hi) / ((double)up - (double)hi);
  const float lo = std::max((float)(c - (double)hi), std::numeric_limits<float>::denorm_min());
  return {hi, lo, up, (uint32_t)std::min(part * 4294967296.0, 4294967295.0)};
}

// exp(d / temperature) for d = x - max <= 0.
__device__ __forceinline__ float exp_scaled(float d, Log2Scale c) {
  return ex2(__fmaf_rn(d, c.hi, __fmul_rn(d, c.lo)));
}

// What a maximum is subtracted as: -inf - (-inf) would be NaN where a run of
// -inf logits comes first.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

// At the start of each kernel, before it touches global memory: the kernel
// behind it on the stream may be set up on the SMs already (early; where it was
// launched by launch_behind; it waits here in its turn), then wait for the end
// of the kernels before it.
__device__ __forceinline__ void take_turn(bool early = true) {
  if (early) cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
}

// A launch that may be set up while the kernel before it on the stream runs
// out, in clusters of C CTAs (C > 1). It pays for calls of a few microseconds:
// set-up, first loads of parameters and barriers come off each.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*fn)(P...), unsigned grid, unsigned threads, unsigned smem, int C,
                          cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, std::forward<A>(args)...);
}

inline vsf_status cuda_error(cudaError_t e, const char* who) {
  return fail(VSF_ERR_CUDA, std::string(who) + ": " + cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

}  // namespace obj
}  // namespace vsf
