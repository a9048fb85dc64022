// The experts' outputs back in the token layout, and the bias gradient of the experts' products.
//
//   combine:    Y_t = RNE( residual_t + sum_{j ascending, slot j taken} w_tj y_tj )   in fp32
//   bias grad:  db[e][n] = sum_{r in R_e} rows[r][n]                                   in fp32
//
// The layer output sum_j w_tj y_tj is what the pruned backward of "LRMoE урезает обратный
// проход MoE ..." (section "Что делает LRMoE") differentiates; the pages name no biases.
// Both are HBM-bound: every row is read once, in 16-byte vectors, with fixed sum orders (no
// atomics).
#include "common.cuh"
#include "grouped.cuh"
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

// A cluster of CTAs per (expert, chunk of kBiasVecs 16-byte vectors of columns).  The cluster's
// CTAs take neighbouring runs of the expert's rows (an expert with many rows would otherwise be
// one CTA's long tail, a single expert only a few CTAs); a thread sums every 16th row of its run
// in its vector's columns.  The 16 partial sums of a column are added in order, then the CTAs'
// sums in rank order by the first CTA, through distributed shared memory: no atomics, no
// workspace.
constexpr int kBiasVecs = 16;                   // 256-byte column chunks
constexpr int kBiasRows = 256 / kBiasVecs;      // rows in a pass of the block
constexpr int kBiasUnroll = 8;                  // rows in flight per thread

template <lrmoe_dtype DT>
__global__ void __launch_bounds__(256) bias_grad_kernel(const uint4* __restrict__ rows,
                                                        const int32_t* __restrict__ offsets, int E,
                                                        int V, float* __restrict__ db,
                                                        int accumulate, int rows_cap, int splits,
                                                        uint32_t* __restrict__ status) {
  constexpr int PER = per_vec<DT>();
  constexpr int COLS = kBiasVecs * PER;
  __shared__ float part[kBiasRows][COLS + 4];
  __shared__ float total[COLS];
  pdl_wait();
  pdl_trigger();
  const int vec = threadIdx.x % kBiasVecs, lane_row = threadIdx.x / kBiasVecs;
  const int chunks = (V + kBiasVecs - 1) / kBiasVecs;
  const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
  const long long b = blockIdx.x / splits;  // (expert, chunk)
  const int e = (int)(b / chunks), c = (int)(b % chunks) * kBiasVecs + vec;
  int r0 = offsets[e], r1 = offsets[e + 1];
  if (!idx_ok(r0, (long long)rows_cap + 1, status) || !idx_ok(r1, (long long)rows_cap + 1, status))
    r0 = r1 = 0;
  const int run = (r1 - r0 + splits - 1) / splits;  // >= 0 rows of each CTA
  const int lo = r0 + min(run * rank, r1 - r0), hi = min(lo + run, r1);
  float acc[PER];
#pragma unroll
  for (int n = 0; n < PER; ++n) acc[n] = 0.0f;
  if (c < V) {
    const uint4* at = rows + c;
    int r = lo + lane_row;
    for (; hi - r > (kBiasUnroll - 1) * kBiasRows; r += kBiasUnroll * kBiasRows) {
      uint4 v[kBiasUnroll];
#pragma unroll
      for (int i = 0; i < kBiasUnroll; ++i) v[i] = __ldg(at + (size_t)(r + i * kBiasRows) * V);
#pragma unroll
      for (int i = 0; i < kBiasUnroll; ++i) fma_vec<DT>(acc, 1.0f, v[i]);
    }
    for (; r < hi; r += kBiasRows) fma_vec<DT>(acc, 1.0f, __ldg(at + (size_t)r * V));
  }
#pragma unroll
  for (int n = 0; n < PER; ++n) part[lane_row][vec * PER + n] = acc[n];
  __syncthreads();
  const int col = threadIdx.x;
  float sum = 0.0f;
  if (col < COLS) {
    for (int i = 0; i < kBiasRows; ++i) sum += part[i][col];
    total[col] = sum;
  }
  if (splits > 1) {
    cluster_sync_all();  // every CTA's total is written
    if (rank == 0 && col < COLS) {
      for (int s = 1; s < splits; ++s) {
        float v;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(&total[col], s)));
        sum += v;
      }
    }
    cluster_sync_all();  // and read, before its CTA may leave
  }
  const int n = (int)(b % chunks) * COLS + col;
  if (rank == 0 && col < COLS && n < V * PER) {
    float* out = db + (size_t)e * V * PER + n;
    *out = accumulate ? *out + sum : sum;
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

cudaError_t launch_bias_grad(const void* rows, int rows_cap, const int32_t* offsets, int E, int N,
                             lrmoe_dtype dt, float* db, int accumulate, uint32_t* status,
                             cudaStream_t s) {
  const int V = N / (dt == LRMOE_BF16 ? 8 : 4);
  const long long units = (long long)E * ((V + kBiasVecs - 1) / kBiasVecs);
  // Split an expert's rows over a cluster (up to 8 CTAs, the portable size) while there are fewer
  // than eight CTAs per SM and a CTA would still have a few passes of rows on average.
  int splits = 1;
  while (splits < 8 && units * splits < 8ll * num_sms() &&
         (long long)rows_cap / ((long long)E * splits) >= 4 * kBiasRows)
    splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * splits));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  auto kern = dt == LRMOE_BF16 ? bias_grad_kernel<LRMOE_BF16> : bias_grad_kernel<LRMOE_F32>;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const uint4*>(rows), offsets, E, V, db,
                            accumulate, rows_cap, splits, status);
}

}  // namespace lrmoe
