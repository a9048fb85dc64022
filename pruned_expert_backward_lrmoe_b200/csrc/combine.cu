// The experts' outputs back in the token layout:
//
//   Y_t = RNE( residual_t + sum_{j ascending, slot j taken} w_tj y_tj )   in fp32
//
// The layer output sum_j w_tj y_tj is what the pruned backward of "LRMoE урезает обратный
// проход MoE ..." (section "Что делает LRMoE") differentiates.  HBM-bound: every row is read
// once, in 16-byte vectors, eight of a token's rows in flight together per lane.  T = 16384, top-8,
// H = 4096, residual: 222 us, 5.9 TB/s.
#include "common.cuh"
#include "forward.h"
#include "launch.h"

namespace lrmoe {
namespace {

template <lrmoe_dtype DT>
constexpr int per_vec() {
  return DT == LRMOE_BF16 ? 8 : 4;
}

// acc += w * v, element by element
template <lrmoe_dtype DT>
__device__ __forceinline__ void fma_vec(float (&acc)[per_vec<DT>()], float w, const uint4& v) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == LRMOE_BF16) {
      acc[2 * i] = fmaf(w, bf16_bits_to_f32(u[i] & 0xffffu), acc[2 * i]);
      acc[2 * i + 1] = fmaf(w, bf16_bits_to_f32(u[i] >> 16), acc[2 * i + 1]);
    } else {
      acc[i] = fmaf(w, __uint_as_float(u[i]), acc[i]);
    }
  }
}

template <lrmoe_dtype DT>
__device__ __forceinline__ uint4 round_vec(const float (&acc)[per_vec<DT>()]) {
  if constexpr (DT == LRMOE_BF16)
    return make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                      pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
  else
    return make_uint4(__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                      __float_as_uint(acc[3]));
}

constexpr int kCombineLoads = 8;  // rows of a token in flight per lane

// One warp per (token, 32-vector column chunk).  The residual may be the output itself: a
// lane reads its vector before it writes it.
template <lrmoe_dtype DT>
__global__ void __launch_bounds__(256) combine_kernel(const uint4* __restrict__ y,
                                                      const int32_t* __restrict__ idx,
                                                      const float* __restrict__ w, int T, int k,
                                                      int E, int V, const uint4* residual, uint4* Y,
                                                      uint32_t* __restrict__ status) {
  const int lane = threadIdx.x & 31;
  const int chunks = (V + 31) >> 5;
  const long long units = (long long)T * chunks;
  pdl_wait();
  pdl_trigger();
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < units;
       i += (long long)gridDim.x * 8) {
    const int t = (int)(i / chunks), c = ((int)(i % chunks) << 5) + lane;
    int e = lane < k ? __ldg(idx + (size_t)t * k + lane) : -1;
    if (e >= E) {
      raise_status(status, LRMOE_ST_BAD_EXPERT);
      e = -1;
    }
    const float wj = e >= 0 ? __ldg(w + (size_t)t * k + lane) : 0.0f;
    const unsigned taken = __ballot_sync(kFull, e >= 0);
    const uint4* rows = y + (size_t)t * k * V;
    float acc[per_vec<DT>()];
#pragma unroll
    for (int n = 0; n < per_vec<DT>(); ++n) acc[n] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += kCombineLoads) {
      uint4 v[kCombineLoads];
#pragma unroll
      for (int j = 0; j < kCombineLoads; ++j)
        v[j] = (j0 + j < k && ((taken >> (j0 + j)) & 1u) && c < V)
                   ? __ldg(rows + (size_t)(j0 + j) * V + c)
                   : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kCombineLoads; ++j) {
        if (j0 + j >= k) break;
        const float f = __shfl_sync(kFull, wj, j0 + j);
        if ((taken >> (j0 + j)) & 1u) fma_vec<DT>(acc, f, v[j]);
      }
    }
    if (c < V) {
      if (residual) fma_vec<DT>(acc, 1.0f, residual[(size_t)t * V + c]);
      Y[(size_t)t * V + c] = round_vec<DT>(acc);
    }
  }
}

}  // namespace

cudaError_t launch_combine(const void* y, const int32_t* idx, const float* w, int T, int k, int E,
                           int H, lrmoe_dtype dt, const void* residual, void* Y, uint32_t* status,
                           cudaStream_t s) {
  const int V = H / (dt == LRMOE_BF16 ? 8 : 4);
  const long long units = (long long)T * ((V + 31) / 32);
  long long blocks = (units + 7) / 8;
  const long long cap = (long long)num_sms() * 32;
  if (blocks > cap) blocks = cap;
  auto kern = dt == LRMOE_BF16 ? combine_kernel<LRMOE_BF16> : combine_kernel<LRMOE_F32>;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const uint4*>(y),
                    idx, w, T, k, E, V, static_cast<const uint4*>(residual), static_cast<uint4*>(Y),
                    status);
}

}  // namespace lrmoe
