// Internal declarations of the dense operators: products with one packed
// matrix (linear.cu) and the 16-bit gated feed-forward block (ffn.cu).
#pragma once

#include "moe_internal.cuh"

namespace moe {

// Columns a packed product takes at most: one token's activations (2 bytes a
// column), the blocks' initial sums (1 byte a column) and the weight ring
// share one SM's shared memory.
constexpr int kLinearMaxCols = 32768;

// Sizes of the 16-bit block: tile counts and coordinates fit 32 bits.
constexpr int kFfnMaxSize = 65536;
constexpr int kFfnMaxTokens = 1 << 22;

struct LinearCall {
  const uint8_t* codes;
  const void* scales;
  const float* row_scales;
  const float* bias;
  const void* x;
  void* y;
  int rows, cols, T;      // rows of the packed matrix (2I when gated)
  int block, half_levels, scale_fmt;
  int x_type, y_type, gated;
};

cudaError_t launch_linear(const LinearCall& c, int num_sms, cudaStream_t s);

struct FfnCall {
  int H, I, T, type;
  const void* w_gate_up;      // [2I][H]
  const void* w_down;         // [H][I]
  const void* x;              // [T][H]
  const void* dy;             // [T][H]
  void* y;                    // forward: [T][H]
  void* dx;                   // [T][H], or null
  void* dw_gate_up;           // [2I][H], or null
  void* dw_down;              // [H][I], or null
  void* ws;
};

size_t ffn_workspace_bytes(int H, int I, int T, bool backward);
cudaError_t launch_ffn_forward(const FfnCall& c, int num_sms, cudaStream_t s);
cudaError_t launch_ffn_backward(const FfnCall& c, int num_sms, cudaStream_t s);

// moe_capi.cu
int num_sms_of_current_device();
int status_of_cuda(cudaError_t e);

// launch_pdl with clusters of cg CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int cg, int grid, int threads, size_t smem, cudaStream_t s,
                           const Args&... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cg);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cg > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// One value rounded to a moe_type and stored at index `at`.
__device__ __forceinline__ void store_as(void* p, int type, size_t at, float v) {
  if (type == MOE_FP32) static_cast<float*>(p)[at] = v;
  else if (type == MOE_BF16) static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[at] = __float2half_rn(v);
}

}  // namespace moe
