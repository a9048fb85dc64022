// a4 for fp32 storage: variable-size grouped GEMMs in fp32 FFMA.
//
// "LRMoE урезает обратный проход MoE ...", section "Что делает LRMoE", bullet 5:
// grouped GEMMs of variable size over the compacted per-expert blocks, with
// no zero padding.  The tensor cores have no fp32 x fp32 kind that meets a
// 1e-5 relative error, so fp32 layers use this CUDA-core path (64x64 tiles,
// 16-deep K slices, 4x4 outputs per thread, persistent grid over a tile table
// built on the device from `offsets`).
#include "common.cuh"
#include "forward.h"
#include "grouped.cuh"
#include "launch.h"

namespace lrmoe {
namespace {

constexpr int BM = 64, BN = 64, BK = 16, NT = 256;

__device__ __forceinline__ float sigmoidf_(float x) { return 1.0f / (1.0f + expf(-x)); }

// D[r][n] = sum_k rows[r][k] W[e][k][n] for r in R_e; epilogue STORE or SWIGLU_BWD.
__global__ void __launch_bounds__(NT) dgrad_simt_kernel(
    const float* __restrict__ rows, const float* __restrict__ W,
    const int32_t* __restrict__ offsets, int E, int K, int N, int epi,
    const float* __restrict__ Gp, const float* __restrict__ Up, float* __restrict__ out,
    int rows_cap, uint32_t* __restrict__ status) {
  __shared__ int tstart[kMaxExperts + 1];
  __shared__ int scratch[33];
  __shared__ float As[BK][BM + 4];
  __shared__ float Bs[BK][BN];
  pdl_wait();
  pdl_trigger();
  const int n_tiles = (N + BN - 1) / BN;
  const int total = offsets_invalid(offsets, E, rows_cap, status)
                        ? 0 : build_dgrad_tiles(offsets, E, BM, n_tiles, tstart, scratch);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int e = find_group(tstart, E, t);
    const int local = t - tstart[e];
    const int mt = local / n_tiles, nt = local % n_tiles;
    const int row_beg = offsets[e] + mt * BM;
    const int row_end = offsets[e + 1];
    const int n0 = nt * BN;
    const float* We = W + (size_t)e * K * N;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += BK) {
      // A: 64 rows x 16 k, thread loads 4 (kk fastest)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int idx = tid + i * NT;
        const int r = idx >> 4, kk = idx & 15;
        const int gr = row_beg + r, gk = k0 + kk;
        As[kk][r] = (gr < row_end && gk < K) ? rows[(size_t)gr * K + gk] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int idx = tid + i * NT;
        const int kk = idx >> 6, n = idx & 63;
        const int gk = k0 + kk, gn = n0 + n;
        Bs[kk][n] = (gk < K && gn < N) ? We[(size_t)gk * N + gn] : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < BK; ++kk) {
        float av[4], bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = As[kk][ty * 4 + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) bv[j] = Bs[kk][tx * 4 + j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int gr = row_beg + ty * 4 + i;
      if (gr >= row_end) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int gn = n0 + tx * 4 + j;
        if (gn >= N) continue;
        const float d = acc[i][j];
        if (epi == LRMOE_EPI_SWIGLU_BWD) {
          const float g = Gp[(size_t)gr * N + gn];
          const float u = Up[(size_t)gr * N + gn];
          const float s = sigmoidf_(g);
          out[(size_t)gr * 2 * N + gn] = d * u * s * (1.0f + g * (1.0f - s));
          out[(size_t)gr * 2 * N + N + gn] = d * g * s;
        } else {
          out[(size_t)gr * N + gn] = d;
        }
      }
    }
  }
}

// dW[e][m][n] = sum_{r in R_e} grad[r][m] in[r][n]
__global__ void __launch_bounds__(NT) wgrad_simt_kernel(
    const float* __restrict__ grad, const float* __restrict__ in,
    const int32_t* __restrict__ offsets, int E, int N1, int N2, float* __restrict__ dW,
    int accumulate, int rows_cap, uint32_t* __restrict__ status) {
  __shared__ float As[BK][BM];
  __shared__ float Bs[BK][BN];
  pdl_wait();
  pdl_trigger();
  const int m_tiles = (N1 + BM - 1) / BM, n_tiles = (N2 + BN - 1) / BN;
  const int per_e = m_tiles * n_tiles;
  const int total = offsets_invalid(offsets, E, rows_cap, status) ? 0 : per_e * E;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int e = t / per_e;
    const int local = t % per_e;
    const int m0 = (local / n_tiles) * BM, n0 = (local % n_tiles) * BN;
    const int r_beg = offsets[e], r_end = offsets[e + 1];
    float acc[4][4] = {};
    for (int r0 = r_beg; r0 < r_end; r0 += BK) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int idx = tid + i * NT;
        const int kk = idx >> 6, c = idx & 63;
        const int r = r0 + kk;
        As[kk][c] = (r < r_end && m0 + c < N1) ? grad[(size_t)r * N1 + m0 + c] : 0.0f;
        Bs[kk][c] = (r < r_end && n0 + c < N2) ? in[(size_t)r * N2 + n0 + c] : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < BK; ++kk) {
        float av[4], bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = As[kk][ty * 4 + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) bv[j] = Bs[kk][tx * 4 + j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
      __syncthreads();
    }
    float* dWe = dW + (size_t)e * N1 * N2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + ty * 4 + i;
      if (m >= N1) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (n >= N2) continue;
        float* dst = dWe + (size_t)m * N2 + n;
        *dst = accumulate ? *dst + acc[i][j] : acc[i][j];
      }
    }
  }
}

// This thread's copies since the last commit become a group; wait until at most N groups are
// still in flight.
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Forward products against K-major weights: D[r][n] = sum_k A[r][k] W[e][n][k] for r in R_e.
//   SwiGLU (swiglu != 0): half of a tile's columns are gate rows, half the up rows of the same
//     features, and a thread holds both of a feature.  A row r = x[perm[r] / src_div].
//   linear: out[perm[r]] = D + bias + residual[perm[r]].
struct FpropF32 {
  const float* rows;
  const float* W;
  const int32_t* offsets;
  int E, K, N, swiglu;
  const int32_t* perm;
  int gather, src_div, n_out;
  const float* bias;
  const float* residual;
  float* out;
  float* g;
  float* u;
  float* a;
  int rows_cap;
  uint32_t* status;
};

// 128 CUDA-core multiply-adds a cycle and SM are the limit for large layers; the layers that fp32
// is for are small, and there the latency of a tile is: T = 1021, K = 256, N = 512, one expert,
// residual: 14.6 us; SwiGLU of 2042 pairs over 8 experts, H = 256, I = 384: 39.6 us, 20 TFLOP/s.
//
// Two fp32 multiply-adds in one instruction, each rounded as fmaf.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

// A thread makes RI rows x TN / 16 columns of the 64 x TN tile: the more, the fewer reads of
// shared memory per product, which is what bounds the slices (4 x 4 per thread: 143 us where
// 8 x 4 takes 125).
constexpr int RI = 8;
constexpr int TY = BM / RI;   // thread rows
constexpr int FT = 16 * TY;   // threads of a K group
constexpr int LR = FT / 4;    // tile rows that the threads load in a pass

// silu(g) * u = g / (1 + h^2) * u for g >= 0 and (g h / (1 + h^2)) u h for g < 0, h = exp(-|g| / 2): exp(-g)
// overflows from g = -88.7 on, where the product with a large u is still a normal number.  |g| h stays
// below 3/4, so no factor overflows before the result does.
__device__ __forceinline__ float silu_times(float g, float u) {
  const float h = expf(-0.5f * fabsf(g));
  const float f = g >= 0.0f ? 1.0f : h;
  return g * f / fmaf(h, h, 1.0f) * u * f;
}

// Ring of FS slices of K, copied asynchronously as they lie in memory; rows padded by four
// floats keep the 16-byte reads of neighbouring columns in different banks.  KS groups of FT threads
// take 16 of a slice's k each and add up at the end.
template <int TN, int KS>
struct FpropRing {
  static constexpr int D = BK * KS, P = D + 4, FS = 4;
  float A[FS][BM][P];
  float B[FS][TN][P];
};

template <int TN, int KS>
__global__ void __launch_bounds__(KS * FT) fprop_simt_kernel(const FpropF32 p) {
  constexpr int CJ = TN / 16;  // columns of a thread
  constexpr int AL = BM / LR, BL = TN > LR ? TN / LR : 1;
  using Ring = FpropRing<TN, KS>;
  constexpr int D = Ring::D, FS = Ring::FS;
  extern __shared__ __align__(16) uint8_t dynamic[];
  auto& As = reinterpret_cast<Ring*>(dynamic)->A;
  auto& Bs = reinterpret_cast<Ring*>(dynamic)->B;
  __shared__ int tstart[kMaxExperts + 1];
  __shared__ int scratch[33];
  __shared__ int src[BM];   // source row of each tile row (-1: none)
  __shared__ int dest[BM];  // output row of each tile row (-1: none)
  pdl_wait();
  const int E = p.E, K = p.K, N = p.N;
  const int feat = p.swiglu ? TN / 2 : TN;
  const int n_tiles = (N + feat - 1) / feat;
  const int total = offsets_invalid(p.offsets, E, p.rows_cap, p.status)
                        ? 0 : build_dgrad_tiles(p.offsets, E, BM, n_tiles, tstart, scratch);
  const int tid = threadIdx.x, group = tid / FT, part = tid % FT, tx = part & 15, ty = part >> 4;
  const int lr = tid / (D / 4), lk = tid % (D / 4) * 4;  // tile row and first k of its loads
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int e = find_group(tstart, E, t);
    const int local = t - tstart[e];
    const int row_beg = p.offsets[e] + (local / n_tiles) * BM;
    const int row_end = p.offsets[e + 1];
    const int n0 = (local % n_tiles) * feat;
    __syncthreads();  // the last tile's slices and dest have been read
    if (tid < BM) {
      const int r = row_beg + tid;
      int s = -1, d = -1;
      if (r < row_end) {
        s = d = r;
        if (p.perm) {
          d = p.perm[r];
          if (d < 0 || d >= p.n_out) {
            raise_status(p.status, LRMOE_ST_BAD_INDEX);
            s = d = -1;
          } else if (p.gather) {
            s = d / p.src_div;
          }
        }
      }
      src[tid] = s;
      dest[tid] = d;
    }
    __syncthreads();
    const float* ap[AL];  // this thread's rows of A and of W (nullptr: zeros)
    const float* wp[BL];
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int s = src[lr + i * LR];
      ap[i] = s < 0 ? nullptr : p.rows + (size_t)s * K;
    }
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int c = lr + i * LR;  // column of the tile
      int w = p.swiglu ? n0 + c % (TN / 2) : n0 + c;
      const bool ok = c < TN && w < N;
      if (p.swiglu && c >= TN / 2) w += N;
      wp[i] = ok ? p.W + ((size_t)e * (p.swiglu ? 2 * N : N) + w) * K : nullptr;
    }
    uint64_t acc2[RI][CJ] = {};  // sums over even k (low word) and odd k (high word)
    const int steps = (K + D - 1) / D;
    int in = 0, f = 0;  // slices of the ring to fill and to read
    auto fetch = [&](int step) {  // this thread's 16-byte pieces of a slice (K % 4 == 0)
      const int k = step * D + lk, f = in;
      in = in + 1 == FS ? 0 : in + 1;
      if (step < steps) {
#pragma unroll
        for (int i = 0; i < AL; ++i) {
          const bool ok = ap[i] && k < K;
          cp_async_16(&As[f][lr + i * LR][lk], ok ? ap[i] + k : p.rows, ok ? 16 : 0);
        }
#pragma unroll
        for (int i = 0; i < BL; ++i) {
          const bool ok = wp[i] && k < K;
          if (lr + i * LR < TN)
            cp_async_16(&Bs[f][lr + i * LR][lk], ok ? wp[i] + k : p.W, ok ? 16 : 0);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < FS - 1; ++i) fetch(i);
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      cp_async_wait_group<FS - 2>();
      __syncthreads();  // slice `step` is there for every thread, slice step - 1 is read
      fetch(step + FS - 1);
#pragma unroll
      for (int kk0 = 0; kk0 < BK; kk0 += 4) {
        const int kk = group * BK + kk0;
        ulonglong2 av[RI], bv[CJ];  // (k, k + 1), (k + 2, k + 3)
#pragma unroll
        for (int i = 0; i < RI; ++i)
          av[i] = *reinterpret_cast<const ulonglong2*>(&As[f][ty + TY * i][kk]);
#pragma unroll
        for (int j = 0; j < CJ; ++j)
          bv[j] = *reinterpret_cast<const ulonglong2*>(&Bs[f][tx + 16 * j][kk]);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
          for (int j = 0; j < CJ; ++j) fma2(acc2[i][j], av[i].x, bv[j].x);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
          for (int j = 0; j < CJ; ++j) fma2(acc2[i][j], av[i].y, bv[j].y);
      }
      f = f + 1 == FS ? 0 : f + 1;
    }
    float acc[RI][CJ];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < CJ; ++j)
        acc[i][j] = __uint_as_float((uint32_t)acc2[i][j]) + __uint_as_float((uint32_t)(acc2[i][j] >> 32));
    if constexpr (KS == 2) {  // each group finishes half of the thread's rows
      __syncthreads();        // the ring has been read
      float* swap = &As[0][0][0];
      static_assert(RI / 2 * CJ * 2 * FT <= FS * BM * Ring::P, "the sums fit into the ring");
#pragma unroll
      for (int i = 0; i < RI / 2; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j)
          swap[((group * RI / 2 + i) * CJ + j) * FT + part] = group ? acc[i][j] : acc[i + RI / 2][j];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < RI / 2; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j)
          acc[i][j] = (group ? acc[i + RI / 2][j] : acc[i][j]) +
                      swap[(((group ^ 1) * RI / 2 + i) * CJ + j) * FT + part];
    }
    // Not earlier: blocks of the next launch that move in during a launch of fewer tiles than SMs hold
    // crowd some SMs (128 tiles, back to back: 12.7 us with a trigger at the start, 11.1 here).
    if (t + (long long)gridDim.x >= total) pdl_trigger();
    // columns tx + 16 j of the tile: SwiGLU holds gate features tx (and tx + 16) and their ups
#pragma unroll
    for (int i = 0; i < RI / KS; ++i) {
      const int m = ty + TY * (i + group * RI / 2);
      const int d = dest[m];
      if (d < 0) continue;
      const size_t at = (size_t)d * N;
      if (p.swiglu) {
#pragma unroll
        for (int j = 0; j < CJ / 2; ++j) {
          const int n = n0 + tx + 16 * j;
          if (n >= N) continue;
          float g = acc[i][j], u = acc[i][CJ / 2 + j];
          if (p.bias) {
            g += p.bias[(size_t)e * 2 * N + n];
            u += p.bias[(size_t)e * 2 * N + N + n];
          }
          const float a = silu_times(g, u);
          if (p.g) p.g[at + n] = g;
          if (p.u) p.u[at + n] = u;
          if (p.a) p.a[at + n] = a;
          p.out[(size_t)(row_beg + m) * N + n] = a;
        }
      } else {
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
          const int n = n0 + tx + 16 * j;
          if (n >= N) continue;
          float v = acc[i][j];
          if (p.bias) v += p.bias[(size_t)e * N + n];
          if (p.residual) v += p.residual[at + n];
          p.out[at + n] = v;
        }
      }
    }
  }
}

cudaError_t fprop_simt(const FpropF32& p, cudaStream_t s) {
  auto tiles = [&](int tn) {  // an upper bound
    const int feat = p.swiglu ? tn / 2 : tn;
    return ((long long)p.rows_cap / BM + p.E) * ((p.N + feat - 1) / feat);
  };
  // 64-column tiles do more products per read of shared memory; 32-column ones with two K groups
  // spread a small product over more SMs and warps: 8192 x 512 x 512 125 and 134 us, 2048 x 256 x 256 over
  // four experts 19.4 and 14.5 (16.3 with one K group).
  const bool narrow = tiles(64) < 4ll * num_sms();
  const long long n = tiles(narrow ? 32 : 64), cap = 8ll * num_sms();
  auto launch = [&](auto kern, size_t ring, int threads) {
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring);
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, dim3((unsigned)(n < cap ? n : cap)), dim3(threads), ring, s, p);
  };
  return narrow ? launch(fprop_simt_kernel<32, 2>, sizeof(FpropRing<32, 2>), 2 * FT)
                : launch(fprop_simt_kernel<64, 1>, sizeof(FpropRing<64, 1>), FT);
}

}  // namespace

cudaError_t launch_swiglu_simt(const void* x, int n_src, int src_div, const int32_t* perm,
                               const int32_t* offsets, int rows_cap, const void* W,
                               const void* bias, int E, int H, int I, void* Ap, void* g, void* u,
                               void* a, uint32_t* status, cudaStream_t s) {
  const FpropF32 p{static_cast<const float*>(x), static_cast<const float*>(W), offsets, E, H, I, 1,
                   perm, perm != nullptr, src_div, perm ? n_src * src_div : rows_cap,
                   static_cast<const float*>(bias), nullptr, static_cast<float*>(Ap),
                   static_cast<float*>(g), static_cast<float*>(u), static_cast<float*>(a), rows_cap,
                   status};
  return fprop_simt(p, s);
}

cudaError_t launch_linear_simt(const void* rows, int rows_cap, const void* W, const void* bias,
                               const int32_t* offsets, int E, int K, int N, const void* residual,
                               const int32_t* perm, int n_out, void* out, uint32_t* status,
                               cudaStream_t s) {
  const FpropF32 p{static_cast<const float*>(rows), static_cast<const float*>(W), offsets, E, K, N,
                   0, perm, 0, 1, n_out, static_cast<const float*>(bias),
                   static_cast<const float*>(residual), static_cast<float*>(out), nullptr, nullptr,
                   nullptr, rows_cap, status};
  return fprop_simt(p, s);
}

cudaError_t launch_dgrad_simt(const void* rows, int rows_cap, const void* W,
                              const int32_t* offsets, int E, int K, int N, lrmoe_dtype dt,
                              lrmoe_epilogue epi, const void* Gp, const void* Up, void* out,
                              uint32_t* status, cudaStream_t s) {
  (void)dt;
  return launch_pdl(dgrad_simt_kernel, dim3(num_sms() * 4), dim3(NT), 0, s,
                    static_cast<const float*>(rows), static_cast<const float*>(W), offsets, E, K,
                    N, (int)epi, static_cast<const float*>(Gp), static_cast<const float*>(Up),
                    static_cast<float*>(out), rows_cap, status);
}

cudaError_t launch_wgrad_simt(const void* grad_rows, const void* in_rows, int rows_cap,
                              const int32_t* offsets, int E, int N1, int N2, lrmoe_dtype dt,
                              float* dW, int accumulate, uint32_t* status, cudaStream_t s) {
  (void)dt;
  return launch_pdl(wgrad_simt_kernel, dim3(num_sms() * 4), dim3(NT), 0, s,
                    static_cast<const float*>(grad_rows), static_cast<const float*>(in_rows),
                    offsets, E, N1, N2, dW, accumulate, rows_cap, status);
}

}  // namespace lrmoe
