// The router's auxiliary losses and their gradient.
//
// With p_t the token's shares of the score (softmax, or sigmoids over their sum), c_be the pairs of
// expert e in sequence b, m_b their sum, n_b the sequence's tokens and B' the sequences that have any:
//   loss[0] = coef / B' sum_b (E / (m_b n_b)) sum_e c_be S_be,  S_be = sum_t p_te
//   loss[1] = z_coef / N sum_t lse_t^2
//   softmax dz = p (D - <D, p>),  sigmoid that times 1 - s,  D_e = dloss coef E c_be / (m_b n_b B')
//   dz += 2 dloss z_coef lse / N softmax(z)
//
// The batch is cut into runs of tokens, one block each; a run is cut again where a sequence ends.
// The piece of run c in sequence b writes its sums over tokens to row c + b of the workspace: along
// the batch each piece raises c or b or both, so that no two pieces share a row and a sequence's rows
// lie side by side.  A second kernel adds each sequence's rows in order (no atomics on floats: the
// same inputs give the same bits) and its last block adds the losses up.
//
// A group of SUB lanes takes a token, VPL values to a lane; groups of a warp take neighbouring tokens.
#include <math.h>

#include "common.cuh"
#include "step.h"

namespace lrmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRuns = 592;  // runs of tokens: four blocks to an SM

struct RowSums {  // of one piece of a run
  int tokens, pairs;
  float z;
  int unused;
};

struct BalanceParams {
  const void* logits;
  const int32_t* idx;
  const int32_t* off;  // nullptr: one sequence of all tokens
  int T, E, k, B, run, runs, col_blocks;
  float coef, z_coef;
  float* sums;    // [runs + B][E]
  int32_t* hist;  // [runs + B][E]
  RowSums* rows;  // [runs + B]
  float* part;    // [B][col_blocks], then [B] sums of lse^2
  unsigned* ticket;
  int32_t *counts, *stats;
  float *mean, *loss;
  uint32_t* status;
};

struct BalanceGradParams {
  const void* logits;
  const int32_t* idx;
  const int32_t* off;
  int T, E, k, B;
  float coef, z_coef;
  const int32_t *counts, *stats;
  const float* dloss;
  const void* add;
  void* dlogits;
  uint32_t* status;
};

// Values that a lane holds of a row: in vectors of 16 bytes, neighbouring lanes side by side, where rows
// are whole vectors (the tensor starts on 16 bytes), else one by one.
template <lrmoe_dtype DT, int VPL, int SUB, bool VEC>
struct Row {
  static constexpr int G = DT == LRMOE_BF16 ? 8 : 4;  // values of a vector
  static __device__ __forceinline__ int at(int i, int j) {
    return VEC ? ((i / G) * SUB + j) * G + i % G : i * SUB + j;
  }
  // Values past the row's end, and all of them without `live`, are `none`.
  static __device__ __forceinline__ void load(const void* z, size_t row, int E, int j, bool live,
                                              float none, float (&v)[VPL]) {
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < VPL / G; ++q) {
        const int e = (q * SUB + j) * G;
        const bool ok = live && e < E;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (ok)
          w = *reinterpret_cast<const uint4*>(static_cast<const char*>(z) + (row + e) * (16 / G));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < G; ++i) {
          float f;
          if constexpr (DT == LRMOE_BF16)
            f = (i & 1) ? __uint_as_float(u[i / 2] & 0xffff0000u) : bf16_bits_to_f32(u[i / 2] & 0xffffu);
          else
            f = __uint_as_float(u[i]);
          v[q * G + i] = ok ? f : none;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = at(i, j);
        float f = none;
        if (live && e < E) {
          if constexpr (DT == LRMOE_BF16)
            f = bf16_bits_to_f32(static_cast<const unsigned short*>(z)[row + e]);
          else
            f = static_cast<const float*>(z)[row + e];
        }
        v[i] = f;
      }
    }
  }
  static __device__ __forceinline__ void store(void* z, size_t row, int E, int j, const float (&v)[VPL]) {
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < VPL / G; ++q) {
        const int e = (q * SUB + j) * G;
        if (e >= E) continue;
        uint4 w;
        if constexpr (DT == LRMOE_BF16) {
          const float* f = v + q * G;
          w = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                         pack_bf16x2(f[6], f[7]));
        } else {
          const float* f = v + q * G;
          w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                         __float_as_uint(f[3]));
        }
        *reinterpret_cast<uint4*>(static_cast<char*>(z) + (row + e) * (16 / G)) = w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = at(i, j);
        if (e >= E) continue;
        if constexpr (DT == LRMOE_BF16)
          static_cast<unsigned short*>(z)[row + e] = (unsigned short)f32_to_bf16_bits_rne(v[i]);
        else
          static_cast<float*>(z)[row + e] = v[i];
      }
    }
  }
};

template <int SUB>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = SUB / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

template <int SUB>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = SUB / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

constexpr float kLog2e = 1.44269504088896341f;

// exp(x) for x <= 0 to 2^-21 or so of itself: x is a difference, so that its product's rounding is
// small beside it
__device__ __forceinline__ float exp_neg(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * kLog2e));
  return r;
}

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// exp(z - zmax) of the group's row into u; its sum and zmax come back (0 and 0 for a row without a
// finite logit).  NaN and +inf are found by their sum, which is then no number: such rows, and those
// without a finite logit, are done again with -inf in their place.
template <int VPL, int SUB>
__device__ __forceinline__ void softmax_terms(float (&v)[VPL], float (&u)[VPL], float& sum, float& zmax,
                                              uint32_t* status) {
  auto pass = [&]() {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, v[i]);
    zmax = group_max<SUB>(m);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      u[i] = exp_neg(v[i] - zmax);
      sum += u[i];
    }
    sum = group_sum<SUB>(sum);
  };
  pass();
  if (__any_sync(kFull, !(sum > 0.0f && sum < INFINITY))) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!(v[i] < INFINITY)) {
        raise_status(status, LRMOE_ST_NONFINITE);
        v[i] = -INFINITY;
      }
    pass();
    if (!(zmax > -INFINITY)) {
      sum = zmax = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) u[i] = 0.0f;
    }
  }
}

// sigmoid(z) of the group's row into u, all times one factor where their sum would be next to nothing;
// their sum comes back (0 for a row without a finite logit).
template <int VPL, int SUB>
__device__ __forceinline__ void sigmoid_terms(float (&v)[VPL], float (&u)[VPL], float& sum,
                                              uint32_t* status) {
  bool bad = false;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    bad |= !(v[i] < INFINITY);
    const float t = exp_neg(-fabsf(v[i]));
    const float r = rcp(1.0f + t);
    u[i] = v[i] >= 0.0f ? r : t * r;
    s += u[i];
  }
  sum = group_sum<SUB>(s);
  if (__any_sync(kFull, bad || !(sum > 1e-30f))) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (!(v[i] < INFINITY)) {
        raise_status(status, LRMOE_ST_NONFINITE);
        v[i] = -INFINITY;
      }
      m = fmaxf(m, v[i]);
    }
    const float base = fminf(group_max<SUB>(m), 0.0f);  // the factor is exp(-base)
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float t = exp_neg(-fabsf(v[i]));
      u[i] = v[i] > -INFINITY ? exp_neg(fminf(v[i], 0.0f) - base) * rcp(1.0f + t) : 0.0f;
      s += u[i];
    }
    sum = group_sum<SUB>(s);
  }
}

// Sequence of token t among those that are not empty: the last b with off[b] <= t.
__device__ __forceinline__ int find_sequence(const int32_t* off, int B, int t) {
  int lo = 0, hi = B;  // off[lo] <= t < off[hi], as far as the offsets rise
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(off + mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The slots of a group's token: how many name an expert.  They are counted in `hist` if there is one.
template <int SUB>
__device__ __forceinline__ int routed_slots(const int32_t* idx, int t, int k, int E, int j, bool live,
                                            int* hist, uint32_t* status) {
  int n = 0;
  for (int q = 0; q < k; q += SUB) {
    int e = -1;
    if (live && q + j < k) e = __ldg(idx + (size_t)t * k + q + j);
    if (e >= E) {
      raise_status(status, LRMOE_ST_BAD_EXPERT);
      e = -1;
    }
    if (hist != nullptr && e >= 0) atomicAdd(hist + e, 1);
    const unsigned set = __ballot_sync(kFull, e >= 0);
    if constexpr (SUB == 32)
      n += __popc(set);
    else
      n += __popc((set >> (threadIdx.x & 31 & ~(SUB - 1))) & ((1u << SUB) - 1u));
  }
  return n;
}

template <lrmoe_dtype DT, bool SIGMOID, int VPL, int SUB, bool VEC>
__global__ void __launch_bounds__(kThreads) balance_kernel(const BalanceParams p) {
  constexpr int TPW = 32 / SUB;  // tokens of a warp at a time
  using R = Row<DT, VPL, SUB, VEC>;
  extern __shared__ float smem[];  // [kWarps][E] sums, [E] counts
  const int E = p.E;
  int* hist = reinterpret_cast<int*>(smem + (size_t)kWarps * E);
  __shared__ RowSums warp_sums[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / SUB, j = lane % SUB;
  for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0u;
  const int t0 = blockIdx.x * p.run, t1 = min(p.T, t0 + p.run);
  int b = p.off ? find_sequence(p.off, p.B, t0) : 0;
  for (; b < p.B; ++b) {
    int lo = 0, hi = p.T;
    if (p.off) {
      lo = __ldg(p.off + b);
      if (lo >= t1) break;
      hi = __ldg(p.off + b + 1);
    }
    lo = max(lo, t0);
    hi = min(hi, t1);
    if (lo >= hi) continue;
    float col[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) col[i] = 0.0f;
    int tokens = 0, pairs = 0;
    float zz = 0.0f;
    __syncthreads();  // the counts are 0
    for (int first = lo + warp * TPW; first < hi; first += kWarps * TPW) {
      const int t = first + sub;
      const bool live = t < hi;
      float v[VPL], u[VPL], sum, zmax;
      R::load(p.logits, (size_t)t * E, E, j, live, live ? -INFINITY : 0.0f, v);
      const int n = routed_slots<SUB>(p.idx, t, p.k, E, j, live, hist, p.status);
      if constexpr (SIGMOID) {
        sigmoid_terms<VPL, SUB>(v, u, sum, p.status);
      } else {
        softmax_terms<VPL, SUB>(v, u, sum, zmax, p.status);
      }
      const float inv = n > 0 && sum > 0.0f ? rcp(sum) : 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) col[i] = fmaf(u[i], inv, col[i]);
      if (p.z_coef != 0.0f) {
        if constexpr (SIGMOID) softmax_terms<VPL, SUB>(v, u, sum, zmax, p.status);
        const float lse = sum > 0.0f ? zmax + logf(sum) : 0.0f;
        if (n > 0) zz = fmaf(lse, lse, zz);
      }
      tokens += n > 0;
      pairs += n;
    }
#pragma unroll
    for (int o = SUB; o < 32; o <<= 1) {  // the warp's groups
#pragma unroll
      for (int i = 0; i < VPL; ++i) col[i] += __shfl_xor_sync(kFull, col[i], o);
      tokens += __shfl_xor_sync(kFull, tokens, o);
      pairs += __shfl_xor_sync(kFull, pairs, o);
      zz += __shfl_xor_sync(kFull, zz, o);
    }
    if (sub == 0) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (R::at(i, j) < E) smem[(size_t)warp * E + R::at(i, j)] = col[i];
    }
    if (lane == 0) warp_sums[warp] = RowSums{tokens, pairs, zz, 0};
    __syncthreads();
    const size_t row = (size_t)blockIdx.x + b;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += smem[(size_t)w * E + e];
      p.sums[row * E + e] = s;
      p.hist[row * E + e] = hist[e];
      hist[e] = 0;
    }
    if (threadIdx.x == 0) {
      RowSums r{0, 0, 0.0f, 0};
      for (int w = 0; w < kWarps; ++w) {
        r.tokens += warp_sums[w].tokens;
        r.pairs += warp_sums[w].pairs;
        r.z += warp_sums[w].z;
      }
      p.rows[row] = r;
    }
  }
}

template <typename V>
__device__ __forceinline__ V block_sum(V v, V* scratch /* [kWarps + 1] */) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  V s = scratch[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s += scratch[w];
  return s;
}

// One block to COLS experts of a sequence: its pieces' rows are added in order.
template <int COLS>
__global__ void __launch_bounds__(kThreads) balance_sum_kernel(const BalanceParams p) {
  constexpr int ROWS = kThreads / COLS;  // rows at a time
  const int E = p.E;
  const int b = blockIdx.x / p.col_blocks, cb = blockIdx.x - b * p.col_blocks;
  const int c = threadIdx.x % COLS, r = threadIdx.x / COLS, e = cb * COLS + c;
  __shared__ float fsum[ROWS][COLS];
  __shared__ int isum[ROWS][COLS];
  __shared__ float fs[kWarps + 1];
  __shared__ int is[kWarps + 1];
  __shared__ bool last;
  pdl_wait();
  pdl_trigger();
  int lo = 0, hi = p.T;
  if (p.off) {
    lo = __ldg(p.off + b);
    hi = __ldg(p.off + b + 1);
    if (lo < 0 || hi > p.T || lo > hi) {
      if (cb == 0 && threadIdx.x == 0) raise_status(p.status, LRMOE_ST_BAD_INDEX);
      lo = min(max(lo, 0), p.T);
      hi = min(max(hi, lo), p.T);
    }
  }
  const int first = lo / p.run + b, rows = hi > lo ? (hi - 1) / p.run - lo / p.run + 1 : 0;
  float s = 0.0f;
  int n = 0;
  if (e < E) {
#pragma unroll 4
    for (int i = r; i < rows; i += ROWS) {
      s += p.sums[(size_t)(first + i) * E + e];
      n += p.hist[(size_t)(first + i) * E + e];
    }
  }
  fsum[r][c] = s;
  isum[r][c] = n;
  int tokens = 0, pairs = 0;
  float z = 0.0f;
  for (int i = threadIdx.x; i < rows; i += kThreads) {
    const RowSums q = p.rows[first + i];
    tokens += q.tokens;
    pairs += q.pairs;
    z += q.z;
  }
  tokens = block_sum(tokens, is);
  pairs = block_sum(pairs, is);
  z = block_sum(z, fs);
  float dot = 0.0f;
  if (r == 0 && e < E) {
    for (int i = 1; i < ROWS; ++i) {
      s += fsum[i][c];
      n += isum[i][c];
    }
    p.counts[(size_t)b * E + e] = n;
    p.mean[(size_t)b * E + e] = tokens > 0 ? s / (float)tokens : 0.0f;
    dot = (float)n * s;
  }
  dot = block_sum(dot, fs);
  if (threadIdx.x == 0) {
    p.part[blockIdx.x] = pairs > 0 ? dot * ((float)E / ((float)pairs * (float)tokens)) : 0.0f;
    if (cb == 0) {
      p.stats[2 * b] = tokens;
      p.stats[2 * b + 1] = pairs;
      p.part[(size_t)p.B * p.col_blocks + b] = z;
    }
    __threadfence();
    last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  // the last block: every other's part is written
  const volatile float* part = p.part;
  const volatile int32_t* stats = p.stats;
  float l = 0.0f;
  z = 0.0f;
  int all = 0, live = 0;
  for (long long i = threadIdx.x; i < (long long)p.B * p.col_blocks; i += kThreads) l += part[i];
  for (int i = threadIdx.x; i < p.B; i += kThreads) {
    z += part[(size_t)p.B * p.col_blocks + i];
    all += stats[2 * i];
    live += stats[2 * i] > 0;
  }
  l = block_sum(l, fs);
  z = block_sum(z, fs);
  all = block_sum(all, is);
  live = block_sum(live, is);
  if (threadIdx.x == 0) {
    p.stats[2 * p.B] = all;
    p.stats[2 * p.B + 1] = live;
    p.loss[0] = live > 0 ? p.coef * (l / (float)live) : 0.0f;
    p.loss[1] = all > 0 ? p.z_coef * (z / (float)all) : 0.0f;
  }
}

template <lrmoe_dtype DT, bool SIGMOID, int VPL, int SUB, bool VEC>
__global__ void __launch_bounds__(kThreads) balance_grad_kernel(const BalanceGradParams p) {
  constexpr int TPW = 32 / SUB;
  using R = Row<DT, VPL, SUB, VEC>;
  const int lane = threadIdx.x & 31, sub = lane / SUB, j = lane % SUB;
  const int E = p.E;
  pdl_wait();
  pdl_trigger();
  const int all = __ldg(p.stats + 2 * p.B), live_seqs = __ldg(p.stats + 2 * p.B + 1);
  const float d0 = p.dloss ? __ldg(p.dloss) : 1.0f, d1 = p.dloss ? __ldg(p.dloss + 1) : 1.0f;
  const float c0 = live_seqs > 0 ? p.coef * d0 * (float)E / (float)live_seqs : 0.0f;
  const float cz = all > 0 ? 2.0f * p.z_coef * d1 / (float)all : 0.0f;
  // a warp's tokens lie side by side, so that its sequence seldom changes
  const long long warps = (long long)gridDim.x * kWarps;
  const long long each = ((p.T + warps - 1) / warps + TPW - 1) / TPW * TPW;
  const long long w0 = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * each;
  const int end = (int)min((long long)p.T, w0 + each);
  int seq = -1, seq_lo = 0, seq_hi = 0;  // the sequence whose factors are in D
  float D[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) D[i] = 0.0f;
  for (long long first = w0; first < end; first += TPW) {
    const int t = (int)first + sub;
    const bool live = t < end;
    const size_t row = (size_t)t * E;
    if (live && (seq < 0 || t < seq_lo || t >= seq_hi)) {
      seq = p.off ? find_sequence(p.off, p.B, t) : 0;
      seq_lo = p.off ? __ldg(p.off + seq) : 0;
      seq_hi = p.off ? __ldg(p.off + seq + 1) : p.T;
      const float nm = (float)__ldg(p.stats + 2 * seq) * (float)__ldg(p.stats + 2 * seq + 1);
      const float f = nm > 0.0f ? c0 / nm : 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        D[i] = R::at(i, j) < E ? f * (float)__ldg(p.counts + (size_t)seq * E + R::at(i, j)) : 0.0f;
    }
    // rows behind the last sequence are not read
    const bool inside = live && t >= seq_lo && t < seq_hi;
    float v[VPL], u[VPL], sum, zmax;
    R::load(p.logits, row, E, j, inside, inside ? -INFINITY : 0.0f, v);
    const bool counts = routed_slots<SUB>(p.idx, t, p.k, E, j, inside, nullptr, p.status) > 0;
    float dz[VPL];
    if constexpr (SIGMOID) {
      sigmoid_terms<VPL, SUB>(v, u, sum, p.status);
      const float inv = counts && sum > 0.0f ? rcp(sum) : 0.0f;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) dot = fmaf(D[i], u[i], dot);
      dot = group_sum<SUB>(dot) * inv;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float t1 = exp_neg(-fabsf(v[i]));
        const float r = rcp(1.0f + t1);
        dz[i] = u[i] * inv * (D[i] - dot) * (v[i] >= 0.0f ? t1 * r : r);
      }
      if (p.z_coef != 0.0f) {
        softmax_terms<VPL, SUB>(v, u, sum, zmax, p.status);
        const float w = counts && sum > 0.0f ? cz * (zmax + logf(sum)) * rcp(sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) dz[i] = fmaf(w, u[i], dz[i]);
      }
    } else {
      softmax_terms<VPL, SUB>(v, u, sum, zmax, p.status);
      const float inv = counts && sum > 0.0f ? rcp(sum) : 0.0f;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) dot = fmaf(D[i], u[i], dot);
      dot = group_sum<SUB>(dot) * inv;
      if (p.z_coef != 0.0f && inv > 0.0f) dot -= cz * (zmax + logf(sum));
#pragma unroll
      for (int i = 0; i < VPL; ++i) dz[i] = u[i] * inv * (D[i] - dot);
    }
    if (p.add) {
      R::load(p.add, row, E, j, live, 0.0f, v);
#pragma unroll
      for (int i = 0; i < VPL; ++i) dz[i] += v[i];
    }
    if (live) R::store(p.dlogits, row, E, j, dz);
  }
}

// Lanes and values of a token by the number of experts; rows of whole 16-byte vectors or not.
template <template <lrmoe_dtype, bool, int, int, bool> class F, lrmoe_dtype DT, bool SIGMOID, bool VEC,
          typename P>
cudaError_t by_width(const P& p, cudaStream_t s) {
  if (p.E <= 32) return F<DT, SIGMOID, 8, 4, VEC>::run(p, s);
  if (p.E <= 64) return F<DT, SIGMOID, 8, 8, VEC>::run(p, s);
  if (p.E <= 128) return F<DT, SIGMOID, 8, 16, VEC>::run(p, s);
  if (p.E <= 256) return F<DT, SIGMOID, 8, 32, VEC>::run(p, s);
  if (p.E <= 512) return F<DT, SIGMOID, 16, 32, VEC>::run(p, s);
  return F<DT, SIGMOID, 32, 32, VEC>::run(p, s);
}

template <template <lrmoe_dtype, bool, int, int, bool> class F, typename P>
cudaError_t by_type(const P& p, lrmoe_dtype dt, bool sigmoid, cudaStream_t s) {
  if (dt == LRMOE_BF16) {
    if (p.E % 8 == 0)
      return sigmoid ? by_width<F, LRMOE_BF16, true, true>(p, s) : by_width<F, LRMOE_BF16, false, true>(p, s);
    return sigmoid ? by_width<F, LRMOE_BF16, true, false>(p, s) : by_width<F, LRMOE_BF16, false, false>(p, s);
  }
  if (p.E % 4 == 0)
    return sigmoid ? by_width<F, LRMOE_F32, true, true>(p, s) : by_width<F, LRMOE_F32, false, true>(p, s);
  return sigmoid ? by_width<F, LRMOE_F32, true, false>(p, s) : by_width<F, LRMOE_F32, false, false>(p, s);
}

template <lrmoe_dtype DT, bool SIGMOID, int VPL, int SUB, bool VEC>
struct Forward {
  static cudaError_t run(const BalanceParams& p, cudaStream_t s) {
    return launch_pdl(balance_kernel<DT, SIGMOID, VPL, SUB, VEC>, dim3(p.runs), dim3(kThreads),
                      sizeof(float) * (kWarps + 1) * (size_t)p.E, s, p);
  }
};

template <lrmoe_dtype DT, bool SIGMOID, int VPL, int SUB, bool VEC>
struct Backward {
  static cudaError_t run(const BalanceGradParams& p, cudaStream_t s) {
    const long long per = kWarps * (32 / SUB);
    long long blocks = (p.T + per - 1) / per;
    const long long cap = (long long)num_sms() * 8;
    if (blocks > cap) blocks = cap;
    return launch_pdl(balance_grad_kernel<DT, SIGMOID, VPL, SUB, VEC>, dim3((unsigned)blocks),
                      dim3(kThreads), 0, s, p);
  }
};

struct Plan {  // what the sizes alone fix
  int run, runs, cols, col_blocks;
  size_t hist, rows, part, ticket, total;  // offsets in the workspace (the sums come first)
};

Plan plan_of(int T, int E, int B) {
  Plan q;
  // runs of at least a block's tokens at a time
  const int sub = E <= 32 ? 4 : E <= 64 ? 8 : E <= 128 ? 16 : 32;
  const int at_a_time = kWarps * (32 / sub);
  q.run = (T + kMaxRuns - 1) / kMaxRuns;
  if (q.run < at_a_time) q.run = at_a_time;
  q.runs = (int)(((long long)T + q.run - 1) / q.run);
  q.cols = B >= 64 ? 64 : 8;
  q.col_blocks = (E + q.cols - 1) / q.cols;
  auto up = [](size_t n) { return (n + 15) & ~size_t(15); };
  const size_t pieces = (size_t)q.runs + B;
  q.hist = up(pieces * E * 4);
  q.rows = q.hist + up(pieces * E * 4);
  q.part = q.rows + up(pieces * sizeof(RowSums));
  q.ticket = q.part + up(((size_t)B * q.col_blocks + B) * 4);
  q.total = q.ticket + 16;
  return q;
}

}  // namespace

size_t balance_workspace(int T, int E, int B) { return plan_of(T, E, B).total; }

cudaError_t launch_balance(const void* logits, int T, int E, lrmoe_dtype dt, const int32_t* idx,
                           int k, lrmoe_score_fn fn, const int32_t* off, int B, float coef,
                           float z_coef, int32_t* counts, int32_t* stats, float* mean, float* loss,
                           void* ws, uint32_t* status, cudaStream_t s) {
  const Plan q = plan_of(T, E, B);
  char* w = static_cast<char*>(ws);
  BalanceParams p{};
  p.logits = logits;
  p.idx = idx;
  p.off = off;
  p.T = T;
  p.E = E;
  p.k = k;
  p.B = B;
  p.run = q.run;
  p.runs = q.runs;
  p.col_blocks = q.col_blocks;
  p.coef = coef;
  p.z_coef = z_coef;
  p.sums = reinterpret_cast<float*>(w);
  p.hist = reinterpret_cast<int32_t*>(w + q.hist);
  p.rows = reinterpret_cast<RowSums*>(w + q.rows);
  p.part = reinterpret_cast<float*>(w + q.part);
  p.ticket = reinterpret_cast<unsigned*>(w + q.ticket);
  p.counts = counts;
  p.stats = stats;
  p.mean = mean;
  p.loss = loss;
  p.status = status;
  cudaError_t e = by_type<Forward>(p, dt, fn == LRMOE_SCORE_SIGMOID, s);
  if (e != cudaSuccess) return e;
  const unsigned blocks = (unsigned)((long long)B * q.col_blocks);
  auto kern = q.cols == 64 ? balance_sum_kernel<64> : balance_sum_kernel<8>;
  return launch_pdl(kern, dim3(blocks), dim3(kThreads), 0, s, p);
}

cudaError_t launch_balance_grad(const void* logits, int T, int E, lrmoe_dtype dt,
                                const int32_t* idx, int k, lrmoe_score_fn fn, const int32_t* off,
                                int B, float coef, float z_coef, const int32_t* counts,
                                const int32_t* stats, const float* dloss, const void* add,
                                void* dlogits, uint32_t* status, cudaStream_t s) {
  const BalanceGradParams p{logits, idx,   off,   T,     E,   k,       B,
                            coef,   z_coef, counts, stats, dloss, add, dlogits, status};
  return by_type<Backward>(p, dt, fn == LRMOE_SCORE_SIGMOID, s);
}

}  // namespace lrmoe
