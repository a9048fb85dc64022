// Launchers of the operators that close a training step (host side): the router's losses, the
// gradient norm, the AdamW step.  As in launch.h, the arguments are already validated by abi.cu and
// each launcher only enqueues kernels on `s`.
#pragma once

#include "launch.h"

namespace lrmoe {

// launch_pdl with clusters of `cluster` blocks (1: none).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                      cudaStream_t s, int cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

size_t balance_workspace(int T, int E, int B);
cudaError_t launch_balance(const void* logits, int T, int E, lrmoe_dtype dt, const int32_t* idx,
                           int k, lrmoe_score_fn fn, const int32_t* off, int B, float coef,
                           float z_coef, int32_t* counts, int32_t* stats, float* mean, float* loss,
                           void* ws, uint32_t* status, cudaStream_t s);
cudaError_t launch_balance_grad(const void* logits, int T, int E, lrmoe_dtype dt,
                                const int32_t* idx, int k, lrmoe_score_fn fn, const int32_t* off,
                                int B, float coef, float z_coef, const int32_t* counts,
                                const int32_t* stats, const float* dloss, const void* add,
                                void* dlogits, uint32_t* status, cudaStream_t s);

size_t grad_norm_workspace(int count);
cudaError_t launch_grad_norm(const lrmoe_tensor* t, int count, lrmoe_dtype dt, float max_norm,
                             float* out, void* ws, uint32_t* status, cudaStream_t s);

struct AdamwArgs {
  double lr, beta1, beta2;
  float eps;
  int step;
  const float* lr_dev;
  const int32_t* step_dev;
  const float* grad_scale;
  uint32_t seed;
  uint32_t* status;
};
cudaError_t launch_adamw(const lrmoe_tensor* t, int count, lrmoe_dtype pdt, lrmoe_dtype gdt,
                         int bits, const AdamwArgs& a, cudaStream_t s);

}  // namespace lrmoe
