// The experts' forward products for bf16 storage: variable-size grouped GEMMs against
// K-major weights, with the bias, the SwiGLU activation, the residual and the scatter to
// pair order in the epilogue.
//
//   SwiGLU: [g | u] = x_r . W_gu[e]^T + b[e],  a = silu(g) * u      (x_r gathered by perm)
//   linear: out     = rows_r . W[e]^T + b[e] + residual
//
// The expert feed-forward g = x W_gate^T, u = x W_up^T, a = silu(g) * u, y = a W_down^T is
// what the pruned backward of "LRMoE урезает обратный проход MoE ..." (section "Что делает
// LRMoE", bullet 1: the forward computes every pair) takes its saved tensors from.
//
// Mathematics: D = A . B^T with A = the expert's rows [m][K] and B = the expert's weights
// [N][K], both K-major, so A and B are staged alike: 64-deep K blocks as 128-byte rows under
// the 128-byte swizzle.  The accumulators stay in fp32 in tensor memory; bias, activation and
// residual are applied to the fp32 values and each output is rounded once, to bf16 (the stored
// g and u are rounded copies: a is formed from the unrounded ones).
//
// Tiles.  PAIR: a cluster of two CTAs shares one tcgen05.mma.cta_group::2 of 256 rows x 256
// columns; each CTA stages its 128 rows of A and 128 of the 256 rows of B.  One SM: 128 rows x
// 256 columns.  For SwiGLU the 256 columns are 128 gate rows and the 128 up rows of the same
// features, so that a thread finds g and u of a feature in its own tensor-memory lane and the
// activation needs no exchange.  An expert's rows go to PAIR tiles, a last tile of at most 128
// rows to a one-SM tile in a second launch that overlaps the first one's drain.
//
// Gathered rows come in by four-row TMA gathers, which the copy engine takes about 19 ns each
// (32 a K block and CTA: more than the block's products take).  So their PAIR tile is DOUBLE: 256
// rows x 512 columns, both accumulators at once, half the gathers per product.  For packed rows
// (and on one SM) the two accumulators alternate and a tile's epilogue runs under the next
// tile's products.  Single against DOUBLE, E = 128, top-8, under load: I = 768, T = 8192, gathered:
// H = 256 150 and 143 us, 1024 344 and 308, 2048 609 and 525; T = 16384, H = 4096, I = 1408 3.76 and
// 3.23 ms (3.14 and 2.70 in the first passes, before the power cap settles); packed 3.10 and 3.17 ms.
//
// Every tile has the same K depth, so tiles are dealt out in turn; there is no device-side
// scheduling state that two launches or two captured graphs could share.
//
// Roles: producer warps (one for packed rows; to gather, four share the four-row gathers: with
// one warp the T = 16384 layer below took 6.8 ms), one warp for tensor memory and MMA issue, eight
// epilogue warps.  Every wait is bounded (LRMOE_ST_TIMEOUT, then a clean exit).  No TMA multicast.
//
// What bounds it, and what it measured (B200, under load until the power cap settles):
//   SwiGLU, T = 16384, E = 128, top-8, H = 4096, I = 1408, gathered rows: 3.2-3.4 ms (900-950
//     TFLOP/s at 1.4 GHz, 1000 W: power); packed rows 3.1 ms; the same flops as one dense product
//     2.34 ms, cuBLAS 2.29.
//   linear, T = 8111, E = 128, top-8, K = 768, N = 2048: 0.26 ms, of which 45 us are the one-SM
//     launch reading half of the weights again; without any epilogue 0.23.  One dense 16384 x 1408 x
//     4096 product: 161 us, cuBLAS 151, without epilogue 143.
//   SwiGLU, T = 16 (a few rows per expert), H = 2048, I = 768: 80-86 us, linear, K = 768, N = 2048: 40 us;
//     the weights of the experts taken at 6.1-6.6 TB/s (HBM).
//   One expert that every token takes, T = 4096: SwiGLU, H = 2048, I = 1408 67 us (705 TFLOP/s), linear,
//     K = 1408, N = 2048, residual 32 us (731): two turns of tiles, the second one partly empty.
#include "forward.h"
#include "gemm_common.cuh"

namespace lrmoe {
namespace {

struct FpropParams {
  const int32_t* offsets;
  int E, K, N;              // N: output features (SwiGLU: I)
  const int32_t* perm;      // packed row -> pair (nullptr: identity)
  int src_div;              // GATHER: packed row r reads source row perm[r] / src_div
  int n_out;                // rows of the pair-order outputs
  const uint16_t* bias;     // [E][N] (SwiGLU: [E][2N]) or nullptr
  const uint16_t* residual; // linear: [n_out][N] or nullptr
  uint16_t* out;            // linear: [n_out][N]; SwiGLU: packed a [rows_cap][N]
  uint16_t* g;              // SwiGLU, each optional: pair-order [n_out][N]
  uint16_t* u;
  uint16_t* a;
  uint32_t* status;
  int part;                 // RowPart
  int late_wait;
  int rows_cap;
  int wide;                 // outputs' rows start on 32 bytes and N % 16 == 0
};

// 3D bf16 map over [E][N][K] (K-major weights of the forward products), box = 64 (K) x 128 (N)
// x 1, 128-B swizzle.
bool make_map_kmajor(CUtensorMap* m, const void* base, uint64_t E, uint64_t N, uint64_t K) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {K, N, E};
  cuuint64_t strides[2] = {K * 2, N * K * 2};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// DOUBLE: a PAIR tile of 256 rows x 512 columns (both accumulators at once, see fprop_kernel).
template <bool PAIR, bool DOUBLE>
struct FwdLayout {
  static constexpr int kStages = PAIR && !DOUBLE ? 6 : 4;
  static constexpr int kABytes = BM * BK * 2;                       // 16 KB
  static constexpr int kBBytes = (PAIR ? kBNT / 2 : kBNT) * BK * 2; // 16 KB / 32 KB
  static constexpr int kStageBytes = kABytes + (DOUBLE ? 2 : 1) * kBBytes;
  static constexpr int kBarOff = kStages * kStageBytes;
  static constexpr int kNumBars = 2 * kStages + 5;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kTableOff = kMiscOff + 16;
  __host__ __device__ static constexpr int table_ints(int E) { return 2 * (E + 1) + 33; }
  __host__ __device__ static constexpr int alloc(int E) {
    return kTableOff + table_ints(E) * 4 + 1024;
  }
};

struct FwdTile {
  int e, row0, row_end, n0;
};

// Output columns of an accumulator: SwiGLU features, each with its gate and up.
template <bool SWIGLU>
constexpr int kFeat = SWIGLU ? kBNT / 2 : kBNT;

template <bool SWIGLU, bool PAIR, bool DOUBLE>
__device__ __forceinline__ FwdTile decode_fwd(int t, const FpropParams& p, const int* offs,
                                              const int* tab, int nt) {
  FwdTile ti;
  ti.e = find_group(tab, p.E, t);
  const int local = t - tab[ti.e];
  ti.n0 = (local % nt) * kFeat<SWIGLU> * (DOUBLE ? 2 : 1);
  ti.row0 = dgrad_tile_row0(offs[ti.e], offs[ti.e + 1] - offs[ti.e], PAIR ? 2 * BM : BM, p.part,
                            local / nt);
  ti.row_end = offs[ti.e + 1];
  return ti;
}

// Four gathered rows (64 bf16 columns from c0) of a row-major matrix, box of one row.
__device__ __forceinline__ void tma_gather4(void* dst, const void* tmap, uint64_t* bar, int c0,
                                            const int (&r)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(r[0]), "r"(r[1]),
      "r"(r[2]), "r"(r[3])
      : "memory");
}

// The same with completion counted on a barrier of either CTA of the pair (cluster address).
__device__ __forceinline__ void tma_gather4_pair(void* dst, const void* tmap, uint32_t bar_cl,
                                                 int c0, const int (&r)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cl), "r"(c0), "r"(r[0]), "r"(r[1]),
      "r"(r[2]), "r"(r[3])
      : "memory");
}

// bf16 row segment [nb, nb + 32) of `orow`, columns >= N skipped.  wide: rows and columns lie on
// 32 bytes, so a thread writes whole sectors (linear, T = 8111, K = 768, N = 2048: 263 us against
// 293 with 16-byte stores; 217 and 247 in the first passes, before the power cap settles).
__device__ __forceinline__ void store_row32(const uint32_t (&r)[32], uint16_t* orow, int nb, int N,
                                            bool wide) {
  if (!wide) {
    epi_store_bf16(r, orow, nb, N);
    return;
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    if (nb + v * 16 < N) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = pack_bf16x2(__uint_as_float(r[16 * v + 2 * i]), __uint_as_float(r[16 * v + 2 * i + 1]));
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                       reinterpret_cast<uint64_t>(orow + nb + v * 16)),
                   "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                   "r"(w[7])
                   : "memory");
    }
  }
}

// silu(g) * u = g r u for g >= 0 and (g h r) u h for g < 0, h = exp(-|g| / 2), r = 1 / (1 + h^2) in
// [1/2, 1]: exp(-g) itself would overflow, and its reciprocal flush, from g = -87 on, where the product
// with a large u is still a normal number.  |g| h stays below 3/4, so no factor overflows before the
// result does.  h is the square of 2^(-|g| log2(e) / 4), which flushes only past |g| = 349 (the power of
// -|g| / 2 itself would need its range extended there, three more instructions).  2^x and 1/x are good to 2
// and 1 ulp of fp32 (2^-23) and x is off by 2^-23: 14 + |g| ulp in all, 1.1e-5 at |g| = 80; the result
// is rounded to bf16.
__device__ __forceinline__ float silu_times(float g, float u) {
  float q, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(fabsf(g) * -0.36067376f));
  const float h = q * q;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(h, h, 1.0f)));
  const float f = g >= 0.0f ? 1.0f : h;
  return g * f * r * u * f;
}

// 32 values of columns [nb, nb + 32) added to r (columns >= N skipped; N % 8 == 0).  Plain
// loads: the residual may be the output itself.
__device__ __forceinline__ void add_row32(uint32_t (&r)[32], const uint16_t* v, int nb, int N) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (nb + c * 8 < N) {
      const uint4 w = *reinterpret_cast<const uint4*>(v + nb + c * 8);
      const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[8 * c + 2 * i] = __float_as_uint(__uint_as_float(r[8 * c + 2 * i]) +
                                           bf16_bits_to_f32(h[i] & 0xffffu));
        r[8 * c + 2 * i + 1] = __float_as_uint(__uint_as_float(r[8 * c + 2 * i + 1]) +
                                               bf16_bits_to_f32(h[i] >> 16));
      }
    }
  }
}

// Producer warps.  Packed rows need one; gathered rows come in through four, since a warp's
// four-row loads issue one after another (about 40 ns each; eight warps cost the epilogue its
// registers: H = 2048, I = 768, T = 8192 549 us against 531).
template <bool GATHER>
constexpr int kProducers = GATHER ? 4 : 1;
template <bool GATHER>
constexpr int kFwdThreads = 32 * (kProducers<GATHER> + 1 + kEpiWarps);

template <bool SWIGLU, bool PAIR, bool GATHER, bool DOUBLE>
__global__ void __launch_bounds__(kFwdThreads<GATHER>, 1) fprop_kernel(
    const __grid_constant__ CUtensorMap tmA /* rows: 32-row boxes, or one-row boxes to gather */,
    const __grid_constant__ CUtensorMap tmB /* W [E][rows][K], 128-row boxes */,
    const FpropParams p) {
  using L = FwdLayout<PAIR, DOUBLE>;
  constexpr int FEAT = kFeat<SWIGLU>;
  constexpr int STAGES = L::kStages;
  constexpr int BN = kBNT;
  constexpr int kTileM = PAIR ? 2 * BM : BM;
  constexpr int NP = kProducers<GATHER>;
  const int E = p.E;
  uint32_t* status = p.status;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* full = bars;
  uint64_t* empty = bars + STAGES;
  uint64_t* tfull = bars + 2 * STAGES;       // [2]
  uint64_t* tempty = bars + 2 * STAGES + 2;  // [2]
  uint64_t* mma_done = bars + 2 * STAGES + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  int* tab = reinterpret_cast<int*>(smem + L::kTableOff);
  int* offs_s = tab + (E + 1);
  int* scratch = offs_s + (E + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const int first = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x;
  const int step = PAIR ? (int)gridDim.x >> 1 : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], (PAIR ? 2 : 1) * NP);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], (PAIR ? 2 : 1) * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == NP) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, 2 * BN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 2 * BN);
      tmem_relinquish();
    }
  }
  if constexpr (PAIR) cluster_sync_all();  // both CTAs' barriers exist before any remote arrival
  // A late-wait launch (the last tiles of the experts, behind the PAIR launch of the same
  // product) reads only what was complete when that launch started.
  if (!p.late_wait) {
    pdl_wait();
    pdl_trigger();
  }
  constexpr int kTileN = FEAT * (DOUBLE ? 2 : 1);
  const int nt = (p.N + kTileN - 1) / kTileN;
  int total = build_dgrad_tiles(p.offsets, E, kTileM, nt, tab, scratch, p.part);
  for (int i = threadIdx.x; i <= E; i += blockDim.x) offs_s[i] = p.offsets[i];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (offsets_invalid(offs_s, E, p.rows_cap, status)) total = 0;
  const uint32_t tmem_base = *tmem_slot;
  const int nk = (p.K + BK - 1) / BK;

  if (warp < NP) {
    // ---------------- producers ----------------
    // Every producer warp of both CTAs arrives on a block's barrier, also one without a group of
    // rows to load: no block completes without it, so none can fall a ring turn behind.
    int stage = 0;
    uint32_t phase = 0;
    uint32_t armed = 0, armed_par = 0;
    const uint32_t lead_full = PAIR ? cluster_addr(full, 0) : 0u;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const FwdTile ti = decode_fwd<SWIGLU, PAIR, DOUBLE>(t, p, offs_s, tab, nt);
      const int base = ti.row0 + rank * BM;  // this CTA's first row
      const uint32_t halves = DOUBLE && ti.n0 + FEAT < p.N ? 2 : 1;
      // Row groups of A with at least one of the expert's rows are loaded; what shared memory
      // holds in the others only reaches accumulator rows that are never stored.
      constexpr int unit = GATHER ? 4 : 32;
      auto groups = [&](int b) {
        int n = ti.row_end - b;
        n = n < 0 ? 0 : (n > BM ? BM : n);
        return (n + unit - 1) / unit;
      };
      const int mine = groups(base);
      constexpr uint32_t a_unit = (uint32_t)unit * BK * 2;
      // this lane's group: a producer warp has eight of the 32 four-row groups
      const int grp = GATHER ? warp * (32 / NP) + lane : lane;
      const bool load_a = grp < mine && (!GATHER || lane < 32 / NP);
      const uint32_t bytes =
          (uint32_t)mine * a_unit + halves * L::kBBytes +
          (PAIR ? (uint32_t)groups(ti.row0 + BM) * a_unit + halves * L::kBBytes : 0u);
      int src[4] = {0, 0, 0, 0};
      if (GATHER && load_a) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = base + grp * 4 + i;
          const int pr = r < ti.row_end ? __ldg(p.perm + r) : 0;
          // an entry out of range reads row 0; the epilogue flags it and stores nothing
          src[i] = pr >= 0 && pr < p.n_out ? pr / p.src_div : 0;
        }
      }
      const int brow = SWIGLU ? (rank ? p.N + ti.n0 : ti.n0) : ti.n0 + rank * (BN / 2);
      for (int kb = 0; kb < nk; ++kb) {
        if (!__all_sync(kFull, mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, status))) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + stage * L::kStageBytes;
        uint8_t* sb = sa + L::kABytes;
        if (leader) {
          if (lane == 0) {
            if (warp == 0)
              mbar_arrive_expect_tx(&full[stage], bytes);
            else
              mbar_arrive(&full[stage]);
          }
          armed |= 1u << stage;
          armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          __syncwarp();
          if (load_a) {
            if constexpr (GATHER)
              tma_gather4(sa + grp * a_unit, &tmA, &full[stage], kb * BK, src);
            else
              tma_load_2d(sa + grp * a_unit, &tmA, &full[stage], kb * BK, base + grp * 32);
          }
          if (warp == 0 && lane == 0) {
            tma_load_3d(sb, &tmB, &full[stage], kb * BK, brow, ti.e);
            if (DOUBLE && halves == 2)
              tma_load_3d(sb + L::kBBytes, &tmB, &full[stage], kb * BK, brow + FEAT, ti.e);
            if constexpr (!PAIR)
              tma_load_3d(sb + L::kBBytes / 2, &tmB, &full[stage], kb * BK,
                          SWIGLU ? p.N + ti.n0 : ti.n0 + BN / 2, ti.e);
          }
        } else {
          const uint32_t fb = lead_full + 8u * stage;
          if (load_a) {
            if constexpr (GATHER)
              tma_gather4_pair(sa + grp * a_unit, &tmA, fb, kb * BK, src);
            else
              tma_load_2d_pair(sa + grp * a_unit, &tmA, fb, kb * BK, base + grp * 32);
          }
          __syncwarp();
          if (lane == 0) {
            if (warp == 0) {
              tma_load_3d_pair(sb, &tmB, fb, kb * BK, brow, ti.e);
              if (DOUBLE && halves == 2)
                tma_load_3d_pair(sb + L::kBBytes, &tmB, fb, kb * BK, brow + FEAT, ti.e);
            }
            mbar_arrive_cluster_relaxed(fb);  // the bytes are counted by the barrier itself
          }
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // every load that was started lands before shared memory is released (the leader's
    // barriers count the peer's bytes too)
    if (leader && warp == 0 && lane == 0)
      for (int i = 0; i < STAGES; ++i)
        if ((armed >> i) & 1u) mbar_wait_drain<PAIR>(&full[i], (armed_par >> i) & 1u);
    __syncwarp();
  } else if (warp == NP) {
    if (leader) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc = idesc_bf16_f32(kTileM, BN, false, false);
      const uint32_t peer_empty = PAIR ? cluster_addr(empty, 1) : 0u;
      const uint32_t peer_tfull = PAIR ? cluster_addr(tfull, 1) : 0u;
      int stage = 0;
      uint32_t phase = 0, acc_par = 0;  // bit a: parity of accumulator a's uses so far
      bool ok = true;
      // the MMAs of one K block (lane 0): A times half h of B into accumulator acc
      auto multiply = [&](int st, int h, uint32_t acc, bool first_block) {
        const uint32_t a_addr = smem_u32(smem + st * L::kStageBytes);
        const uint32_t b_addr = a_addr + L::kABytes + h * L::kBBytes;
#pragma unroll
        for (int kk = 0; kk < BK / UK; ++kk) {
          const uint64_t adesc = smem_desc_sw128(a_addr + kk * 32, 16, 1024);
          const uint64_t bdesc = smem_desc_sw128(b_addr + kk * 32, 16, 1024);
          const uint32_t more = first_block && kk == 0 ? 0u : 1u;
          if constexpr (PAIR)
            tc_mma_f16_pair(tmem_base + acc * BN, adesc, bdesc, idesc, more);
          else
            tc_mma_f16(tmem_base + acc * BN, adesc, bdesc, idesc, more);
        }
      };
      auto commit = [&](uint64_t* bar, uint32_t peer_bar) {  // (lane 0) in both CTAs
        if constexpr (PAIR) {
          tc_commit_pair(smem_u32(bar));
          tc_commit_pair(peer_bar);
        } else {
          tc_commit(bar);
        }
      };
      auto wait_acc = [&](uint32_t acc) {  // drained by the epilogue
        const bool free_ = __all_sync(kFull, mbar_wait_bounded(&tempty[acc],
                                                               ((acc_par >> acc) & 1u) ^ 1u,
                                                               abort_flag, status));
        acc_par ^= 1u << acc;
        tc_fence_after();
        return free_;
      };
      auto wait_block = [&](int st, uint32_t ph) {
        const bool there =
            __all_sync(kFull, mbar_wait_bounded(&full[st], ph, abort_flag, status));
        tc_fence_after();
        return there;
      };
      uint32_t turn = 0;  // !DOUBLE: the tiles alternate between the accumulators
      for (int t = first; t < total && ok; t += step) {
        const FwdTile ti = decode_fwd<SWIGLU, PAIR, DOUBLE>(t, p, offs_s, tab, nt);
        const bool two = DOUBLE && ti.n0 + FEAT < p.N;
        const uint32_t acc = DOUBLE ? 0u : turn;
        turn ^= 1u;
        if (!(ok = wait_acc(acc))) break;
        int kb = 0;
        if (two) {
          // The second accumulator is drained after the first: meanwhile multiply the first
          // blocks into the first one, then catch up.
          const int head = min(STAGES - 1, nk);
          int st = stage;
          uint32_t ph = phase;
          for (int i = 0; i < head && ok; ++i) {
            if (!(ok = wait_block(st, ph))) break;
            if (lane == 0) multiply(st, 0, 0, i == 0);
            __syncwarp();
            if (++st == STAGES) {
              st = 0;
              ph ^= 1u;
            }
          }
          if (!ok || !(ok = wait_acc(1))) break;
          for (; kb < head; ++kb) {
            if (lane == 0) {
              multiply(stage, 1, 1, kb == 0);
              commit(&empty[stage], peer_empty + 8u * stage);
            }
            __syncwarp();
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        for (; kb < nk; ++kb) {
          if (!(ok = wait_block(stage, phase))) break;
          if (lane == 0) {
            multiply(stage, 0, acc, kb == 0);
            if (two) {
              if (kb + 1 == nk) commit(&tfull[0], peer_tfull);
              multiply(stage, 1, 1, false);
            }
            commit(&empty[stage], peer_empty + 8u * stage);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (lane == 0) {
          if (!two || nk < STAGES) commit(&tfull[acc], peer_tfull + 8u * acc);
          if (two) commit(&tfull[1], peer_tfull + 8u);
        }
        __syncwarp();
      }
      // every issued MMA has finished before tensor memory is released
      if (lane == 0) {
        if constexpr (PAIR)
          tc_commit_pair(smem_u32(mma_done));
        else
          tc_commit(mma_done);
      }
      __syncwarp();
      mbar_wait_drain(mma_done, 0);
    }
  } else {
    // ---------------- epilogue ----------------
    const int ew = warp - NP - 1;
    const int q = warp & 3, half = ew >> 2;
    const int row_in_tile = rank * BM + q * 32 + lane;
    const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16);
    const uint32_t lead_tempty = PAIR ? cluster_addr(tempty, 0) : 0u;
    const bool wide = p.wide != 0;
    uint32_t acc_par = 0, turn = 0;  // acc_par: bit a is the parity of accumulator a's uses
    auto release_acc = [&](uint32_t b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_remote(lead_tempty + 8u * b);
        else
          mbar_arrive(&tempty[b]);
      }
    };
    for (int t = first; t < total; t += step) {
      const FwdTile ti = decode_fwd<SWIGLU, PAIR, DOUBLE>(t, p, offs_s, tab, nt);
      const int row = ti.row0 + row_in_tile;
      bool row_ok = row < ti.row_end;
      int orow = row;
      if (row_ok && p.perm != nullptr) {
        orow = __ldg(p.perm + row);
        if (orow < 0 || orow >= p.n_out) {
          raise_status(status, LRMOE_ST_BAD_INDEX);
          row_ok = false;
        }
      }
      const int halves = DOUBLE && ti.n0 + FEAT < p.N ? 2 : 1;
      bool ok = true;
      for (int h = 0; h < halves; ++h) {
        const uint32_t b = DOUBLE ? (uint32_t)h : turn;
        ok = __all_sync(kFull, mbar_wait_bounded(&tfull[b], (acc_par >> b) & 1u, abort_flag, status));
        acc_par ^= 1u << b;
        if (!ok) break;
        tc_fence_after();
        const int c0 = ti.n0 + h * FEAT;  // first column of this accumulator
        if constexpr (SWIGLU) {
          const uint16_t* bias = p.bias ? p.bias + (size_t)ti.e * 2 * p.N : nullptr;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int f = half * 64 + c * 32;  // feature inside the accumulator
            const int nb = c0 + f;
            uint32_t rg[32], ru[32];
            tmem_ld_32x32b_x32(lane_base + b * BN + f, rg);
            tmem_ld_32x32b_x32(lane_base + b * BN + BN / 2 + f, ru);
            tmem_wait_ld();
            reg_fence(rg);
            reg_fence(ru);
            if (c == 1) release_acc(b);
            if (row_ok && nb < p.N) {
              if (bias) {
                add_row32(rg, bias, nb, p.N);
                add_row32(ru, bias + p.N, nb, p.N);
              }
              const size_t at = (size_t)orow * p.N;
              if (p.g) store_row32(rg, p.g + at, nb, p.N, wide);
              if (p.u) store_row32(ru, p.u + at, nb, p.N, wide);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                rg[i] = __float_as_uint(silu_times(__uint_as_float(rg[i]), __uint_as_float(ru[i])));
              if (p.a) store_row32(rg, p.a + at, nb, p.N, wide);
              store_row32(rg, p.out + (size_t)row * p.N, nb, p.N, wide);
            }
          }
        } else {
          const uint16_t* bias = p.bias ? p.bias + (size_t)ti.e * p.N : nullptr;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int col = half * 128 + c * 32;
            const int nb = c0 + col;
            uint32_t r[32];
            tmem_ld_32x32b_x32(lane_base + b * BN + col, r);
            tmem_wait_ld();
            reg_fence(r);
            if (c == 3) release_acc(b);
            if (row_ok && nb < p.N) {
              const size_t at = (size_t)orow * p.N;
              if (bias) add_row32(r, bias, nb, p.N);
              if (p.residual) add_row32(r, p.residual + at, nb, p.N);
              store_row32(r, p.out + at, nb, p.N, wide);
            }
          }
        }
      }
      if (!ok) break;
      turn ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after();
  if (warp == NP) {
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, 2 * BN);
    else
      tmem_dealloc(tmem_base, 2 * BN);
  }
  if (p.late_wait) {
    // this grid completes only after the kernel before it, so the next kernel in the
    // stream sees both launches' rows
    pdl_wait();
    pdl_trigger();
  }
}

template <bool SWIGLU, bool PAIR, bool GATHER, bool DOUBLE>
cudaError_t launch_fprop(const CUtensorMap& a, const CUtensorMap& b, FpropParams prm,
                         cudaStream_t s) {
  using L = FwdLayout<PAIR, DOUBLE>;
  const int smem = L::alloc(prm.E);
  if (smem > kSmemLimit) return cudaErrorInvalidConfiguration;
  auto kern = fprop_kernel<SWIGLU, PAIR, GATHER, DOUBLE>;
  // set on every launch (host-side only): a cached flag would go stale when the device's
  // context is reset
  cudaError_t err =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (err != cudaSuccess) return err;
  constexpr int feat = kFeat<SWIGLU> * (DOUBLE ? 2 : 1);
  constexpr int tile_m = PAIR ? 2 * BM : BM;
  const int nt = (prm.N + feat - 1) / feat;
  long long tiles = ((long long)prm.rows_cap / tile_m + prm.E) * nt;  // an upper bound
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kFwdThreads<GATHER>);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  const int units = PAIR ? num_sms() / 2 : num_sms();
  const int n = tiles < units ? (int)tiles : units;
  cfg.gridDim = dim3((PAIR ? 2 : 1) * n);
  return cudaLaunchKernelEx(&cfg, kern, a, b, prm);
}

template <bool SWIGLU, bool GATHER>
cudaError_t fprop(const void* rows, int n_rows, const void* W, int w_rows, FpropParams prm,
                  cudaStream_t s, const char** why) {
  CUtensorMap a, b;
  if (!make_map_2d(&a, rows, (uint64_t)n_rows, (uint64_t)prm.K, 64, GATHER ? 1 : 32) ||
      !make_map_kmajor(&b, W, (uint64_t)prm.E, (uint64_t)w_rows, (uint64_t)prm.K)) {
    *why = "cuTensorMapEncodeTiled failed for a forward operand";
    return cudaErrorInvalidValue;
  }
  auto on32 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 31u) == 0; };
  prm.wide = prm.N % 16 == 0 && on32(prm.out) && on32(prm.g) && on32(prm.u) && on32(prm.a);
  // At most 128 rows in all: no expert can fill more than a one-SM tile.  (Otherwise one-SM tiles
  // for the last rows and PAIR tiles for the rest: PAIR tiles for all rows measured the same at
  // T = 16384 and 257 us against 192 at T = 1024, H = 2048, I = 768.)
  const bool pairs = prm.rows_cap > BM;
  if (pairs) {
    prm.part = kRowsPairs;
    const cudaError_t e = launch_fprop<SWIGLU, true, GATHER, GATHER>(a, b, prm, s);
    if (e != cudaSuccess) return e;
  }
  prm.part = pairs ? kRowsTails : kRowsAll;
  prm.late_wait = pairs ? 1 : 0;
  return launch_fprop<SWIGLU, false, GATHER, false>(a, b, prm, s);
}

}  // namespace

cudaError_t launch_swiglu_tc(const void* x, int n_src, int src_div, const int32_t* perm,
                             const int32_t* offsets, int rows_cap, const void* W, const void* bias,
                             int E, int H, int I, void* Ap, void* g, void* u, void* a,
                             uint32_t* status, cudaStream_t s, const char** why) {
  FpropParams prm{};
  prm.offsets = offsets;
  prm.E = E;
  prm.K = H;
  prm.N = I;
  prm.perm = perm;
  prm.src_div = src_div;
  prm.n_out = perm ? n_src * src_div : rows_cap;
  prm.bias = static_cast<const uint16_t*>(bias);
  prm.out = static_cast<uint16_t*>(Ap);
  prm.g = static_cast<uint16_t*>(g);
  prm.u = static_cast<uint16_t*>(u);
  prm.a = static_cast<uint16_t*>(a);
  prm.status = status;
  prm.rows_cap = rows_cap;
  return perm ? fprop<true, true>(x, n_src, W, 2 * I, prm, s, why)
              : fprop<true, false>(x, n_src, W, 2 * I, prm, s, why);
}

cudaError_t launch_linear_tc(const void* rows, int rows_cap, const void* W, const void* bias,
                             const int32_t* offsets, int E, int K, int N, const void* residual,
                             const int32_t* perm, int n_out, void* out, uint32_t* status,
                             cudaStream_t s, const char** why) {
  FpropParams prm{};
  prm.offsets = offsets;
  prm.E = E;
  prm.K = K;
  prm.N = N;
  prm.perm = perm;
  prm.src_div = 1;
  prm.n_out = n_out;
  prm.bias = static_cast<const uint16_t*>(bias);
  prm.residual = static_cast<const uint16_t*>(residual);
  prm.out = static_cast<uint16_t*>(out);
  prm.status = status;
  prm.rows_cap = rows_cap;
  return fprop<false, false>(rows, rows_cap, W, N, prm, s, why);
}

}  // namespace lrmoe
