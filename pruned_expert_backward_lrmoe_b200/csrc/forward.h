// Launchers of the layer's forward operators (host side); as in launch.h, the arguments are
// already validated by abi.cu and each launcher only enqueues kernels on `s`.
#pragma once

#include "launch.h"

namespace lrmoe {

cudaError_t launch_route(const void* logits, int T, int E, lrmoe_dtype dt, const float* bias, int k,
                         lrmoe_score_fn fn, int n_group, int topk_group, int renorm, float scale,
                         int32_t* idx, float* w, uint32_t* status, cudaStream_t s);
cudaError_t launch_route_grad(const void* logits, int T, int E, lrmoe_dtype dt, const int32_t* idx,
                              int k, lrmoe_score_fn fn, int renorm, float scale, const float* dw,
                              void* dlogits, uint32_t* status, cudaStream_t s);
cudaError_t launch_combine(const void* y, const int32_t* idx, const float* w, int T, int k, int E,
                           int H, lrmoe_dtype dt, const void* residual, void* Y, uint32_t* status,
                           cudaStream_t s);
cudaError_t launch_bias_grad(const void* rows, int rows_cap, const int32_t* offsets, int E, int N,
                             lrmoe_dtype dt, float* db, int accumulate, uint32_t* status,
                             cudaStream_t s, const char** why, uint64_t stall_ns = 0);
cudaError_t launch_swiglu_simt(const void* x, int n_src, int src_div, const int32_t* perm,
                               const int32_t* offsets, int rows_cap, const void* W,
                               const void* bias, int E, int H, int I, void* Ap, void* g, void* u,
                               void* a, uint32_t* status, cudaStream_t s);
cudaError_t launch_linear_simt(const void* rows, int rows_cap, const void* W, const void* bias,
                               const int32_t* offsets, int E, int K, int N, const void* residual,
                               const int32_t* perm, int n_out, void* out, uint32_t* status,
                               cudaStream_t s);
cudaError_t launch_swiglu_tc(const void* x, int n_src, int src_div, const int32_t* perm,
                             const int32_t* offsets, int rows_cap, const void* W, const void* bias,
                             int E, int H, int I, void* Ap, void* g, void* u, void* a,
                             uint32_t* status, cudaStream_t s, const char** why);
cudaError_t launch_linear_tc(const void* rows, int rows_cap, const void* W, const void* bias,
                             const int32_t* offsets, int E, int K, int N, const void* residual,
                             const int32_t* perm, int n_out, void* out, uint32_t* status,
                             cudaStream_t s, const char** why);

}  // namespace lrmoe
