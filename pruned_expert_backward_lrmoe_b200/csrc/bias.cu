// Bias gradient of the experts' products: db[e][n] = sum_{r in R_e} rows[r][n], in fp32.
//
// (The pages on LRMoE name no biases; the products' other gradients are the grouped dgrad and
// wgrad of the pruned backward.)
//
// HBM-bound: every row is read once.  A cluster of CTAs owns an (expert, 128-byte chunk of
// columns); its CTAs take neighbouring runs of the expert's rows.  Their number comes from the host,
// which knows only the mean length of an expert: clusters serve few experts and columns, so that a
// single expert is not a few CTAs' work.  With many of both there is one CTA to an (expert, chunk)
// however long the expert is, and a long one is their tail.  A CTA's rows come
// in through a ring of 6 TMA boxes of 64 rows x 128 bytes (48 KB on the way, four CTAs per SM):
// most of a typical expert's run is requested at once, which plain loads into registers could not
// hold.  Each of 256 threads adds two 16-byte vectors per box; a column's sums meet in the warp
// (shuffles), then over the eight warps, then over the cluster's CTAs through distributed shared
// memory, each in a fixed order: a sum of m rows in one CTA is m / 32 additions deep and 18 more.  No
// atomics, no workspace.  65536 rows of 1536 over 128 experts: 38 us, 5.3 TB/s (plain 16-byte loads,
// eight in flight: 59 us), half of them in one expert: 126 us; 16381 rows of 4096 of one expert: 27 us,
// 4.9 TB/s.
#include "forward.h"
#include "gemm_common.cuh"

namespace lrmoe {
namespace {

constexpr int kBoxRows = 64;
constexpr int kBoxBytes = kBoxRows * 128;
constexpr int kSlots = 6;
constexpr int kBiasThreads = 256 + 32;  // 8 adding warps, one copying warp
constexpr int kMaxSplits = 8;           // the portable cluster size

// STALL: the diagnostic, in which every CTA withholds its first box and waits give up after stall_ns.
template <lrmoe_dtype DT, bool STALL>
__global__ void __launch_bounds__(kBiasThreads) bias_grad_kernel(
    const __grid_constant__ CUtensorMap tm /* rows as 16-bit columns, 64 x 64 boxes */,
    const int32_t* __restrict__ offsets, int N, float* __restrict__ db, int accumulate, int rows_cap,
    int splits, uint64_t stall_ns, uint32_t* __restrict__ status) {
  constexpr int PER = DT == LRMOE_BF16 ? 8 : 4;  // values per 16-byte vector
  constexpr int COLS = 8 * PER;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t full[kSlots], empty[kSlots];
  __shared__ float total[COLS];
  __shared__ int abort_word, stopped;  // stopped: boxes issued, if not all
  volatile int* abort_flag = &abort_word;
  const uint64_t limit_ns = STALL ? stall_ns : kWaitLimitNs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 8);
    }
    *abort_flag = 0;
    stopped = 0x7fffffff;
    fence_barrier_init();
    tma_prefetch_desc(&tm);
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int chunks = (N + COLS - 1) / COLS;
  const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
  const int unit = blockIdx.x / splits;
  const int e = unit / chunks, chunk = unit - e * chunks;
  int r0 = offsets[e], r1 = offsets[e + 1];
  if (!idx_ok(r0, (long long)rows_cap + 1, status) ||
      !idx_ok((long long)r1 - r0, (long long)rows_cap - r0 + 1, status))
    r0 = r1 = 0;  // checked build: offsets out of range, or falling, are an empty expert
  const int rows = r1 > r0 ? r1 - r0 : 0;
  const int run = (rows + splits - 1) / splits;
  const int lo = min(run * rank, rows), mine = min(run, rows - lo);  // this CTA's rows
  const int boxes = (mine + kBoxRows - 1) / kBoxRows;
  float acc[PER];
#pragma unroll
  for (int n = 0; n < PER; ++n) acc[n] = 0.0f;
  if (warp == 8) {
    if (lane == 0) {
      for (int b = 0; b < boxes; ++b) {
        const int slot = b % kSlots;
        if (b >= kSlots &&
            !mbar_wait_bounded(&empty[slot], ((b / kSlots) & 1) ^ 1, abort_flag, status, limit_ns)) {
          stopped = b;
          break;
        }
        if (STALL && b == 0) continue;
        mbar_arrive_expect_tx(&full[slot], kBoxBytes);
        tma_load_2d(ring + slot * kBoxBytes, &tm, &full[slot], chunk * 64, r0 + lo + b * kBoxRows);
      }
    }
  } else {
    const int row = threadIdx.x >> 3, vec = threadIdx.x & 7;  // rows row, row + 32 of a box
    // the box's rows lie under the 128-byte swizzle (rows 32 apart alike)
    const uint8_t* at = ring + row * 128 + ((vec ^ (row & 7)) << 4);
    auto add = [&](const uint4& v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == LRMOE_BF16) {
          acc[2 * i] += bf16_bits_to_f32(w[i] & 0xffffu);
          acc[2 * i + 1] += bf16_bits_to_f32(w[i] >> 16);
        } else {
          acc[i] += __uint_as_float(w[i]);
        }
      }
    };
    int slot = 0;
    uint32_t phase = 0;
    for (int b = 0; b < boxes; ++b) {
      if (!__all_sync(kFull, mbar_wait_bounded(&full[slot], phase, abort_flag, status, limit_ns))) break;
      const uint4 v0 = *reinterpret_cast<const uint4*>(at + slot * kBoxBytes);
      const uint4 v1 = *reinterpret_cast<const uint4*>(at + slot * kBoxBytes + 32 * 128);
      __syncwarp();
      if (lane == 0 && b + kSlots < boxes) mbar_arrive(&empty[slot]);
      // rows past the run belong to others
      if (b * kBoxRows + row < mine) add(v0);
      if (b * kBoxRows + row + 32 < mine) add(v1);
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  __syncthreads();
  // a CTA whose wait ran out lets its copies land before it leaves its shared memory
  if (*abort_flag) {
    if (threadIdx.x == 0) {  // of each slot the last box that was started
      const int issued = min(boxes, stopped);
      for (int b = max(issued - kSlots, STALL ? 1 : 0); b < issued; ++b)
        mbar_wait_drain(&full[b % kSlots], (b / kSlots) & 1);
    }
    __syncthreads();
  }
  __shared__ float part[8][COLS];
  if (warp < 8) {
#pragma unroll
    for (int n = 0; n < PER; ++n) {  // the warp's four rows of each vector
      acc[n] += __shfl_xor_sync(kFull, acc[n], 8);
      acc[n] += __shfl_xor_sync(kFull, acc[n], 16);
      if (lane < 8) part[warp][lane * PER + n] = acc[n];
    }
  }
  __syncthreads();
  const int col = threadIdx.x;
  float sum = 0.0f;
  if (col < COLS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += part[i][col];
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
  const int n = chunk * COLS + col;
  if (rank == 0 && col < COLS && n < N) {
    float* out = db + (size_t)e * N + n;
    *out = accumulate ? *out + sum : sum;
  }
}

}  // namespace

cudaError_t launch_bias_grad(const void* rows, int rows_cap, const int32_t* offsets, int E, int N,
                             lrmoe_dtype dt, float* db, int accumulate, uint32_t* status,
                             cudaStream_t s, const char** why, uint64_t stall_ns) {
  // the copies see 16-bit columns whatever the type
  const uint64_t cols = (uint64_t)N * (dt == LRMOE_BF16 ? 1 : 2);
  CUtensorMap tm;
  if (!make_map_2d(&tm, rows, (uint64_t)rows_cap, cols, 64, kBoxRows)) {
    *why = "cuTensorMapEncodeTiled failed for the gradient rows";
    return cudaErrorInvalidValue;
  }
  const long long units = (long long)E * (long long)((cols + 63) / 64);
  // Split the experts' rows over clusters while there are fewer than eight CTAs per SM and a CTA
  // would still have a few boxes of rows on average (the lengths themselves stay on the device).
  int splits = 1;
  while (splits < kMaxSplits && units * splits < 8ll * num_sms() &&
         (long long)rows_cap / ((long long)E * splits) >= 4 * kBoxRows)
    splits *= 2;
  auto kern = dt == LRMOE_BF16 ? bias_grad_kernel<LRMOE_BF16, false> : bias_grad_kernel<LRMOE_F32, false>;
  if (stall_ns) kern = bias_grad_kernel<LRMOE_BF16, true>;
  const int smem = kSlots * kBoxBytes + 1024;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * splits));
  cfg.blockDim = dim3(kBiasThreads);
  cfg.dynamicSmemBytes = smem;
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
  return cudaLaunchKernelEx(&cfg, kern, tm, offsets, N, db, accumulate, rows_cap, splits, stall_ns,
                            status);
}

}  // namespace lrmoe
