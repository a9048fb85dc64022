// Routing to experts and its gradient.
//
// The layer output sum_j w_tj y_tj takes its experts and weights from here (the pages on LRMoE
// start from routed pairs and say nothing of the router).  With s = softmax(z) or sigmoid(z):
//   order key   c_e = s_e + b_e (b steers the selection only, for balance)
//   groups      a group counts the sum of its two largest keys; the best topk_group groups stay
//   weights     w_j = scale * s_ej, or scale * s_ej / sum_i s_ei
// Ties go to the lower group and the lower expert.
//
// The order is that of keys computed in fp64, not of one fp32 rounding of them.  Without bias
// the score rises with the logit, so the logits themselves are compared.  Keys with a bias and
// group values are computed in fp32 with a bound on their error; where two neighbours in the order are nearer than
// that bound (about one token in a thousand) and are not the same logit and bias, the warp
// computes the keys of that token again in fp64 and selects by those.
//
// One warp per token.  Expert e = lane * VPL + i lives in register i of a lane, so the lowest
// lane that holds a maximum holds the lowest expert.
#include <math.h>

#include "common.cuh"
#include "launch.h"

namespace lrmoe {
namespace {

constexpr int kRouteWarps = 4;  // warps (tokens) per block

struct RouteParams {
  const void* logits;
  const float* bias;
  int T, E, k, groups, keep_groups, renorm;
  float scale;
  int32_t* idx;
  float* w;
  uint32_t* status;
};

template <lrmoe_dtype DT>
__device__ __forceinline__ float load_logit(const void* z, size_t i) {
  if constexpr (DT == LRMOE_BF16)
    return bf16_bits_to_f32(__ldg(static_cast<const unsigned short*>(z) + i));
  else
    return __ldg(static_cast<const float*>(z) + i);
}

// Logits e0 .. e0 + VPL of a row (-inf past its end).  With E a multiple of VPL every row starts
// on a multiple of the vector (the tensor starts on 16 bytes): 16-byte loads.
template <lrmoe_dtype DT, int VPL>
__device__ __forceinline__ void load_row(const void* z, size_t row, int e0, int E, float (&v)[VPL]) {
  constexpr int kBytes = VPL * (DT == LRMOE_BF16 ? 2 : 4);
  if constexpr (kBytes >= 8) {
    if (E % VPL == 0) {
      constexpr int kWords = kBytes / 4;
      uint32_t w[kWords];
      const char* at = static_cast<const char*>(z) + (row + e0) * (DT == LRMOE_BF16 ? 2 : 4);
      const bool ok = e0 < E;
#pragma unroll
      for (int i = 0; i < kWords; i += (kBytes >= 16 ? 4 : 2)) {
        if constexpr (kBytes >= 16) {
          const uint4 q = ok ? __ldg(reinterpret_cast<const uint4*>(at) + i / 4) : make_uint4(0, 0, 0, 0);
          w[i] = q.x;
          w[i + 1] = q.y;
          w[i + 2] = q.z;
          w[i + 3] = q.w;
        } else {
          const uint2 q = ok ? __ldg(reinterpret_cast<const uint2*>(at)) : make_uint2(0, 0);
          w[i] = q.x;
          w[i + 1] = q.y;
        }
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float f;
        if constexpr (DT == LRMOE_BF16)
          f = bf16_bits_to_f32((i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
        else
          f = __uint_as_float(w[i]);
        v[i] = ok ? f : -INFINITY;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    v[i] = e0 + i < E ? load_logit<DT>(z, row + e0 + i) : -INFINITY;
}

// Order-preserving bits of a float that is not NaN; every such value maps above 0, which marks
// an expert that cannot be chosen.
__device__ __forceinline__ uint32_t order_bits(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 orders as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// sigmoid without overflow on either side: exp(min(z, 0) - m) / (1 + exp(-|z|)) is
// exp(-m) * sigmoid(z).
__device__ __forceinline__ float sigmoid_scaled(float z, float m) {
  return expf(fminf(z, 0.0f) - m) / (1.0f + expf(-fabsf(z)));
}

// The two largest of (a1 >= a2) and (b1 >= b2), into a.
template <typename F>
__device__ __forceinline__ void merge_top2(F& a1, F& a2, F b1, F b2) {
  if (b1 > a1) {
    a2 = a1 > b2 ? a1 : b2;
    a1 = b1;
  } else {
    a2 = a2 > b1 ? a2 : b1;
  }
}

// fp64 selection over the keys key[0..E) of one token (shared memory, -inf: not to be chosen);
// one warp.  keep_groups_fp64 closes the experts of the groups that do not stay;
// topk_fp64 returns the expert of slot `lane` (-1: none left).
__device__ __noinline__ void keep_groups_fp64(double* key, int E, int G, int keep, int lane) {
  const double kNone = -INFINITY;
  const int n = E / G;
  double value = kNone;  // of group `lane`
  for (int g = 0; g < G; ++g) {
    double a1 = kNone, a2 = kNone;
    for (int i = lane; i < n; i += 32) merge_top2(a1, a2, key[g * n + i], kNone);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const double b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
      merge_top2(a1, a2, b1, b2);
    }
    if (lane == g && a1 > kNone) value = a2 > kNone ? a1 + a2 : a1;
  }
  int rank = 0;
  for (int g = 0; g < G; ++g) {
    const double v = __shfl_sync(kFull, value, g);
    rank += (v > value || (v == value && g < lane)) ? 1 : 0;
  }
  const unsigned kept = __ballot_sync(kFull, lane < G && rank < keep && value > kNone);
  __syncwarp();
  for (int e = lane; e < E; e += 32)
    if (!((kept >> (e / n)) & 1u)) key[e] = kNone;
  __syncwarp();
}

__device__ __noinline__ int topk_fp64(double* key, int E, int k, int lane) {
  const double kNone = -INFINITY;
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    double best = kNone;
    int at = E;
    for (int e = lane; e < E; e += 32)
      if (key[e] > best) {
        best = key[e];
        at = e;
      }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const double ob = __shfl_xor_sync(kFull, best, o);
      const int oa = __shfl_xor_sync(kFull, at, o);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (!(best > kNone)) break;  // uniform: nothing left
    if (lane == j) mine = at;
    if (lane == 0) key[at] = kNone;
    __syncwarp();
  }
  return mine;
}

template <lrmoe_dtype DT, bool SIGMOID, int VPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteParams p) {
  extern __shared__ double keys64[];  // [kRouteWarps][E], when a bias or groups are given
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = p.E, k = p.k, G = p.groups;
  const bool plain = p.bias == nullptr && G == 1;  // the order is that of the logits
  const int e0 = lane * VPL;
  const int n = E / G;
  // groups of whole lanes: a lane's experts belong to one group, a group to lpg neighbouring lanes
  const bool whole = n % VPL == 0;
  const int lpg = whole ? n / VPL : 1, my_group = lane / lpg;
  pdl_wait();
  pdl_trigger();
  for (int t = blockIdx.x * kRouteWarps + warp; t < p.T; t += gridDim.x * kRouteWarps) {
    const size_t row = (size_t)t * E;
    float z[VPL];
    load_row<DT, VPL>(p.logits, row, e0, E, z);
    bool bad = false;
    float zmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (isnan(z[i]) || z[i] == INFINITY) {
        bad = true;
        z[i] = -INFINITY;
      }
      zmax = fmaxf(zmax, z[i]);
    }
    float den = 1.0f;  // softmax denominator
    if (!SIGMOID && !(plain && p.renorm)) {
      zmax = warp_max(zmax);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (z[i] > -INFINITY) sum += expf(z[i] - zmax);
      den = warp_sum(sum);
    }
    // Order keys; 0 = cannot be chosen.  The scores in them are only good to the bound that the
    // checks below allow for (fast exponential and division: 2 + 1.2 |x| ulp, under 2e-5 relative
    // where a score is above 1e-35); the weights are computed again from the logits.
    uint32_t key[VPL];
    float smax = 0.0f;  // largest score of this lane
    const float rden = 1.0f / den;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      bool open = z[i] > -INFINITY;
      float c = z[i];
      if (!plain) {
        const float s = SIGMOID ? __fdividef(1.0f, 1.0f + __expf(fminf(-z[i], 87.0f)))
                                : __expf(z[i] - zmax) * rden;
        c = s;
        if (open) smax = fmaxf(smax, s);
        if (p.bias) {
          const float b = e0 + i < E ? __ldg(p.bias + e0 + i) : 0.0f;
          if (isnan(b) || b == INFINITY) bad = true;
          if (!(fabsf(b) < INFINITY)) open = false;
          c = s + b;
        }
      }
      key[i] = open ? order_bits(c) : 0u;
    }
    if (__any_sync(kFull, bad) && lane == 0) raise_status(p.status, LRMOE_ST_NONFINITE);
    bool sure = true;
    if (G > 1) {
      // value of each group: the sum of its two largest keys (0 bits: none)
      float value = -INFINITY;  // of group `lane`
      if (whole) {
        const int pos = lane - my_group * lpg;
        uint32_t a1 = 0u, a2 = 0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          a2 = max(a2, min(a1, key[i]));
          a1 = max(a1, key[i]);
        }
        for (int o = 1; o < lpg; o <<= 1) {  // lane pos 0 ends with the whole group
          const uint32_t b1 = __shfl_down_sync(kFull, a1, o), b2 = __shfl_down_sync(kFull, a2, o);
          if (pos + o < lpg) {
            a2 = max(max(a2, b2), min(a1, b1));
            a1 = max(a1, b1);
          }
        }
        float v = -INFINITY;
        if (a1 != 0u) v = a2 != 0u ? order_value(a1) + order_value(a2) : order_value(a1);
        v = __shfl_sync(kFull, v, lane < G ? lane * lpg : 0);
        if (lane < G) value = v;
      } else {
        for (int g = 0; g < G; ++g) {
          uint32_t a1 = 0u, a2 = 0u;
#pragma unroll
          for (int i = 0; i < VPL; ++i) {
            const int e = e0 + i;
            const uint32_t kv = e >= g * n && e < (g + 1) * n ? key[i] : 0u;
            a2 = max(a2, min(a1, kv));
            a1 = max(a1, kv);
          }
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) {
            const uint32_t b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
            a2 = max(max(a2, b2), min(a1, b1));
            a1 = max(a1, b1);
          }
          if (lane == g && a1 != 0u)
            value = a2 != 0u ? order_value(a1) + order_value(a2) : order_value(a1);
        }
      }
      int rank = 0;
      for (int g = 0; g < G; ++g) {
        const float v = __shfl_sync(kFull, value, g);
        rank += (v > value || (v == value && g < lane)) ? 1 : 0;
      }
      const bool open = lane < G && value > -INFINITY;
      const unsigned kept = __ballot_sync(kFull, open && rank < p.keep_groups);
      // the last kept value against the first that is not kept
      const float in = -warp_max((kept >> lane) & 1u ? -value : -INFINITY);
      const float out = warp_max(open && !((kept >> lane) & 1u) ? value : -INFINITY);
      if (out > -INFINITY && kept) {
        const float tol = 1e-4f * warp_max(smax) + 5e-7f * fmaxf(fabsf(in), fabsf(out)) + 1e-36f;
        sure = in - out > tol;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (e0 + i < E && !((kept >> (whole ? my_group : (e0 + i) / n)) & 1u)) key[i] = 0u;
        // inside the kept groups, without bias, the score rises with the logit
        if (p.bias == nullptr && key[i] != 0u) key[i] = order_bits(z[i]);
      }
    }
    // k rounds: the warp's largest key, its lowest holder, gone for the next round
    int mine = -1;           // expert of slot `lane`
    uint32_t mine_key = 0u;  // key of slot `lane` (lane k: the best one left)
    const int rounds = p.bias ? k + 1 : k;
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
    for (int j = 0; j < rounds; ++j) {
      const uint32_t top = __reduce_max_sync(kFull, best);
      if (top == 0u) break;
      const int owner = __ffs(__ballot_sync(kFull, best == top)) - 1;
      int at = 0;
      if (lane == owner) {
        // the lowest register that holds it (scanned from the highest), then the lane's next best
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
          if (key[i] == top) at = i;
        best = 0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          if (i == at) key[i] = 0u;
          best = max(best, key[i]);
        }
      }
      at = __shfl_sync(kFull, at, owner) + owner * VPL;
      if (lane == j) {
        mine = at;
        mine_key = top;
      }
    }
    float zj = mine >= 0 ? load_logit<DT>(p.logits, row + mine) : -INFINITY;
    if (p.bias) {
      // neighbours of the order that fp32 cannot tell apart
      const float c = mine >= 0 ? order_value(mine_key) : 0.0f;
      const float b = mine >= 0 ? __ldg(p.bias + mine) : 0.0f;
      const float s = fabsf(c - b) + 1.2e-7f * fabsf(c);  // the score, up to rounding
      const float c2 = __shfl_down_sync(kFull, c, 1), b2 = __shfl_down_sync(kFull, b, 1);
      const float s2 = __shfl_down_sync(kFull, s, 1), z2 = __shfl_down_sync(kFull, zj, 1);
      const int m2 = __shfl_down_sync(kFull, mine, 1);
      if (lane < k && mine >= 0 && lane < 31 && m2 >= 0) {
        const float tol = 5e-5f * fmaxf(s, s2) + 2.5e-7f * fmaxf(fabsf(c), fabsf(c2)) + 1e-36f;
        if (c - c2 <= tol && !(zj == z2 && b == b2)) sure = false;
      }
      if (lane == 31 && k == 32) sure = false;  // its neighbour has no lane: decide in fp64
      sure = __all_sync(kFull, sure);
    }
    if (!sure) {  // uniform across the warp
      double* kd = keys64 + (size_t)warp * E;
      double den64 = 1.0;
      if constexpr (!SIGMOID) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (z[i] > -INFINITY) sum += exp((double)z[i] - (double)zmax);
        den64 = warp_sum(sum);
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (e0 + i >= E) continue;
        double c = -INFINITY;
        const float b = p.bias ? __ldg(p.bias + e0 + i) : 0.0f;
        if (z[i] > -INFINITY && fabsf(b) < INFINITY) {
          c = SIGMOID ? 1.0 / (1.0 + exp(-(double)z[i]))
                      : exp((double)z[i] - (double)zmax) / den64;
          c += (double)b;
        }
        kd[e0 + i] = c;
      }
      __syncwarp();
      if (G > 1) keep_groups_fp64(kd, E, G, p.keep_groups, lane);
      if (p.bias == nullptr) {  // the score rises with the logit
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (e0 + i < E && kd[e0 + i] > -INFINITY) kd[e0 + i] = (double)z[i];
        __syncwarp();
      }
      mine = topk_fp64(kd, E, k, lane);
      __syncwarp();
      zj = mine >= 0 ? load_logit<DT>(p.logits, row + mine) : -INFINITY;
    }
    // weights of the slots
    const bool slot = lane < k;
    if (!slot) {
      mine = -1;
      zj = -INFINITY;
    }
    float s = 0.0f;
    if (p.renorm) {
      // relative to the largest chosen score: no underflow of all of them
      const float zc = warp_max(zj);
      if (mine >= 0) s = SIGMOID ? sigmoid_scaled(zj, fminf(zc, 0.0f)) : expf(zj - zc);
      const float sum = warp_sum(s);
      if (mine >= 0) s = s / sum;
    } else if (mine >= 0) {
      s = SIGMOID ? sigmoid_scaled(zj, 0.0f) : expf(zj - zmax) / den;
    }
    if (slot) {
      p.idx[(size_t)t * k + lane] = mine;
      p.w[(size_t)t * k + lane] = mine >= 0 ? s * p.scale : 0.0f;
    }
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
struct RouteGradParams {
  const void* logits;
  const int32_t* idx;
  const float* dw;
  int T, E, k;
  float scale;
  void* dlogits;
  uint32_t* status;
};

template <lrmoe_dtype DT, int VPL>
__device__ __forceinline__ void store_row(void* z, size_t row, int e0, int E, const float (&v)[VPL]) {
  constexpr int kBytes = VPL * (DT == LRMOE_BF16 ? 2 : 4);
  if constexpr (kBytes >= 8) {
    if (E % VPL == 0) {  // see load_row
      if (e0 >= E) return;
      char* at = static_cast<char*>(z) + (row + e0) * (DT == LRMOE_BF16 ? 2 : 4);
      uint32_t w[kBytes / 4];
#pragma unroll
      for (int i = 0; i < kBytes / 4; ++i) {
        if constexpr (DT == LRMOE_BF16)
          w[i] = f32_to_bf16_bits_rne(v[2 * i]) | (f32_to_bf16_bits_rne(v[2 * i + 1]) << 16);
        else
          w[i] = __float_as_uint(v[i]);
      }
#pragma unroll
      for (int i = 0; i < kBytes / 4; i += (kBytes >= 16 ? 4 : 2)) {
        if constexpr (kBytes >= 16)
          reinterpret_cast<uint4*>(at)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        else
          *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (e0 + i >= E) continue;
    if constexpr (DT == LRMOE_BF16)
      static_cast<unsigned short*>(z)[row + e0 + i] = (unsigned short)f32_to_bf16_bits_rne(v[i]);
    else
      static_cast<float*>(z)[row + e0 + i] = v[i];
  }
}

// Slots of one token: lane j < k holds expert, logit and d L / d (s_j or log s_j).
//   renormalised: p_j = s_j / S,  d_j = scale p_j (dw_j - sum_i p_i dw_i)       (= s_j dL/ds_j)
//   softmax:  dz_e = sum of d over the slots of e                        (renormalised)
//             dz_e = s_e (scale sum of dw over the slots of e - scale sum_i dw_i s_i)
//   sigmoid:  dz_e = (1 - s_e) sum over the slots of e of d_j, d_j = scale s_j dw_j if not renormalised
// Only the third form (softmax, not renormalised) reads the whole row; the others read the
// slots' logits and write zeros elsewhere.
template <lrmoe_dtype DT, bool SIGMOID, bool RENORM, int VPL>
__global__ void __launch_bounds__(256) route_grad_kernel(const RouteGradParams p) {
  constexpr bool DENSE = !SIGMOID && !RENORM;
  const int lane = threadIdx.x & 31;
  const int E = p.E, k = p.k;
  const int e0 = lane * VPL;
  pdl_wait();
  pdl_trigger();
  for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < p.T; t += gridDim.x * 8) {
    const size_t row = (size_t)t * E;
    int e = lane < k ? __ldg(p.idx + (size_t)t * k + lane) : -1;
    if (e >= E) {
      raise_status(p.status, LRMOE_ST_BAD_EXPERT);
      e = -1;
    }
    float z = e >= 0 ? load_logit<DT>(p.logits, row + e) : -INFINITY;
    if (e >= 0 && !(fabsf(z) < INFINITY)) {
      if (z != -INFINITY) raise_status(p.status, LRMOE_ST_NONFINITE);
      e = -1;
      z = -INFINITY;
    }
    const float dw = e >= 0 ? __ldg(p.dw + (size_t)t * k + lane) : 0.0f;
    float d = 0.0f;       // this slot's share of dz[e]
    float inv = 0.0f, dot = 0.0f;
    float v[DENSE ? VPL : 1];  // exp(z - zmax) of the lane's experts (0: not finite)
    if constexpr (RENORM) {
      const float zc = warp_max(z);
      float s = 0.0f;
      if (e >= 0) s = SIGMOID ? sigmoid_scaled(z, fminf(zc, 0.0f)) : expf(z - zc);
      const float sum = warp_sum(s);
      const float pj = e >= 0 ? s / sum : 0.0f;
      const float mean = warp_sum(pj * dw);
      d = p.scale * pj * (dw - mean);
      if (SIGMOID && e >= 0) d *= sigmoid_scaled(-z, 0.0f);
    } else if constexpr (SIGMOID) {
      if (e >= 0) d = p.scale * dw * sigmoid_scaled(z, 0.0f) * sigmoid_scaled(-z, 0.0f);
    } else {
      load_row<DT, VPL>(p.logits, row, e0, E, v);
      float m = -INFINITY;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (isnan(v[i]) || v[i] == INFINITY) {
          bad = true;
          v[i] = -INFINITY;
        }
        m = fmaxf(m, v[i]);
      }
      if (__any_sync(kFull, bad) && lane == 0) raise_status(p.status, LRMOE_ST_NONFINITE);
      const float zmax = warp_max(m);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        v[i] = v[i] > -INFINITY ? expf(v[i] - zmax) : 0.0f;
        sum += v[i];
      }
      sum = warp_sum(sum);
      inv = sum > 0.0f ? 1.0f / sum : 0.0f;
      dot = warp_sum(e >= 0 ? dw * (expf(z - zmax) * inv) : 0.0f);
      d = p.scale * dw;
    }
    // the row: every expert's value from the slots that name it, in slot order
    float acc[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int at = __shfl_sync(kFull, e, j) - e0;
      const float dj = __shfl_sync(kFull, d, j);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (at == i) acc[i] += dj;
    }
    if constexpr (DENSE) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = v[i] * inv * (acc[i] - p.scale * dot);
    }
    store_row<DT, VPL>(p.dlogits, row, e0, E, acc);
  }
}

template <lrmoe_dtype DT, bool SIGMOID>
cudaError_t route_by_width(const RouteParams& p, cudaStream_t s) {
  auto kern = route_kernel<DT, SIGMOID, 32>;
  if (p.E <= 32)
    kern = route_kernel<DT, SIGMOID, 1>;
  else if (p.E <= 64)
    kern = route_kernel<DT, SIGMOID, 2>;
  else if (p.E <= 128)
    kern = route_kernel<DT, SIGMOID, 4>;
  else if (p.E <= 256)
    kern = route_kernel<DT, SIGMOID, 8>;
  else if (p.E <= 512)
    kern = route_kernel<DT, SIGMOID, 16>;
  const bool plain = p.bias == nullptr && p.groups == 1;
  const size_t smem = plain ? 0 : sizeof(double) * (size_t)kRouteWarps * p.E;  // <= 32 KB
  long long blocks = ((long long)p.T + kRouteWarps - 1) / kRouteWarps;
  const long long cap = (long long)num_sms() * 32;
  if (blocks > cap) blocks = cap;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(32 * kRouteWarps), smem, s, p);
}

template <lrmoe_dtype DT, bool SIGMOID, bool RENORM>
cudaError_t route_grad_by_width(const RouteGradParams& p, cudaStream_t s) {
  auto kern = route_grad_kernel<DT, SIGMOID, RENORM, 32>;
  if (p.E <= 32)
    kern = route_grad_kernel<DT, SIGMOID, RENORM, 1>;
  else if (p.E <= 64)
    kern = route_grad_kernel<DT, SIGMOID, RENORM, 2>;
  else if (p.E <= 128)
    kern = route_grad_kernel<DT, SIGMOID, RENORM, 4>;
  else if (p.E <= 256)
    kern = route_grad_kernel<DT, SIGMOID, RENORM, 8>;
  else if (p.E <= 512)
    kern = route_grad_kernel<DT, SIGMOID, RENORM, 16>;
  long long blocks = ((long long)p.T + 7) / 8;
  const long long cap = (long long)num_sms() * 16;
  if (blocks > cap) blocks = cap;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, s, p);
}

template <lrmoe_dtype DT>
cudaError_t route_grad_by_fn(const RouteGradParams& p, bool sigmoid, bool renorm, cudaStream_t s) {
  if (sigmoid)
    return renorm ? route_grad_by_width<DT, true, true>(p, s) : route_grad_by_width<DT, true, false>(p, s);
  return renorm ? route_grad_by_width<DT, false, true>(p, s) : route_grad_by_width<DT, false, false>(p, s);
}

}  // namespace

cudaError_t launch_route(const void* logits, int T, int E, lrmoe_dtype dt, const float* bias, int k,
                         lrmoe_score_fn fn, int n_group, int topk_group, int renorm, float scale,
                         int32_t* idx, float* w, uint32_t* status, cudaStream_t s) {
  const RouteParams p{logits, bias, T, E, k, n_group, topk_group, renorm, scale, idx, w, status};
  const bool sg = fn == LRMOE_SCORE_SIGMOID;
  if (dt == LRMOE_BF16)
    return sg ? route_by_width<LRMOE_BF16, true>(p, s) : route_by_width<LRMOE_BF16, false>(p, s);
  return sg ? route_by_width<LRMOE_F32, true>(p, s) : route_by_width<LRMOE_F32, false>(p, s);
}

cudaError_t launch_route_grad(const void* logits, int T, int E, lrmoe_dtype dt, const int32_t* idx,
                              int k, lrmoe_score_fn fn, int renorm, float scale, const float* dw,
                              void* dlogits, uint32_t* status, cudaStream_t s) {
  const RouteGradParams p{logits, idx, dw, T, E, k, scale, dlogits, status};
  const bool sg = fn == LRMOE_SCORE_SIGMOID, rn = renorm != 0;
  return dt == LRMOE_BF16 ? route_grad_by_fn<LRMOE_BF16>(p, sg, rn, s)
                          : route_grad_by_fn<LRMOE_F32>(p, sg, rn, s);
}

}  // namespace lrmoe
