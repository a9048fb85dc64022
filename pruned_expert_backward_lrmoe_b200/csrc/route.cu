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
// group values are computed in fp32 with a bound on their error; where that leaves the order open
// (about one token in a thousand), the warp computes the keys of that token again in fp64 and
// selects by those.  With a bias and k = 32 the lanes hold 32 experts and none is left for the best one
// behind them, so the order is never known to be sure and every token of 32 or more open experts takes
// that way.
//
// One warp per token.  Expert e = lane * VPL + i lives in register i of a lane, so the lowest
// lane that holds a maximum holds the lowest expert.
//
// Bound by the latency and the number of a token's dependent steps (67-70% of the issue slots; the
// bytes would take 1-2 us).  Passes over several sets of inputs, T = 16384, bf16: E = 128, top-8: 9 us (440
// instructions a token), with a bias, sigmoid: 14.5 us (670); E = 256 in 8 groups, bias, sigmoid: 23 us
// (1040), softmax 27.6 (its kernels of up to 256 experts spill 52-92 bytes, the sigmoid ones do not).  A token
// that goes to fp64 takes 0.6 us more for the order of its slots, 3 us for its groups, 6 for all keys:
// E = 128 with a bias, sigmoid, k = 31: 54 us, k = 32: 111.  Where more than 32 keys pass the threshold
// (topk_by_threshold): E = 130, k = 16: 41 us, E = 300: 65.  One token: a launch.
// Gradient, device time: T = 16384, E = 128, top-8, renormalised: 5.3 us; softmax, not renormalised, the same 10.1,
// T = 8191, E = 160, bf16, top-6 5.9 us; latency and the bytes of the result.  A call takes 7.5 us.
#include <math.h>

#include "common.cuh"
#include "forward.h"
#include "launch.h"

namespace lrmoe {
namespace {

constexpr int kRouteWarps = 4;  // warps (tokens) per block

struct RouteParams {
  const void* logits;
  const float* bias;
  int T, E, k, groups, keep_groups, renorm;
  int n;    // experts of a group
  int lpg;  // lanes of a group, if a group is whole lanes of the kernel's width, else 0
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

// Order-preserving bits of a float that is not NaN (-0 orders as +0).  -inf marks an expert that
// cannot be chosen; its bits lie below those of every other value.
__device__ __forceinline__ uint32_t order_bits(float f) {
  const int b = __float_as_int(f + 0.0f);
  return (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}
constexpr uint32_t kShut = 0x007fffffu;  // order_bits(-inf)

__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

__device__ __forceinline__ float warp_max(float v) {
  return order_value(__reduce_max_sync(kFull, order_bits(v)));
}

// 1/x to one ulp, for keys that are checked against an error bound (see route_kernel)
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// Order-preserving bits of a double that is not NaN, and those of -inf (see order_bits).
__device__ __forceinline__ uint64_t order_bits64(double d) {
  const long long b = __double_as_longlong(d + 0.0);
  return (uint64_t)b ^ ((uint64_t)(b >> 63) | 0x8000000000000000ull);
}
constexpr uint64_t kShut64 = 0x000fffffffffffffull;

// fp64 selection over the keys key[0..E) of one token (shared memory, -inf: not to be chosen);
// one warp.  order_fp64 orders the experts of lanes 0 .. n - 1 and returns that of this lane's place.
// keys_fp64 computes all keys; kept_groups_fp64 returns the groups that stay, `sub`
// neighbouring lanes to a group; topk_fp64 returns the expert of slot `lane` (-1:
// none left).  Few tokens come here, so what counts is how long one takes, from cold instructions
// on, since the end of the launch waits for it: short loops.
template <lrmoe_dtype DT>
__device__ __noinline__ double sum_fp64(const void* logits, int E, size_t row, float zmax, int lane) {
  double sum = 0.0;  // the softmax's denominator
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const float z = load_logit<DT>(logits, row + e);
    if (z > -INFINITY && z < INFINITY) sum += exp((double)z - (double)zmax);
  }
  return warp_sum(sum);
}

template <lrmoe_dtype DT, bool SIGMOID>
__device__ __noinline__ void keys_fp64(const void* logits, const float* bias, int E, size_t row,
                                       float zmax, double* key, int lane) {
  const double inv = SIGMOID ? 1.0 : 1.0 / sum_fp64<DT>(logits, E, row, zmax, lane);
  __syncwarp();
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const float z = load_logit<DT>(logits, row + e), b = bias != nullptr ? __ldg(bias + e) : 0.0f;
    double s = exp(SIGMOID ? -(double)z : (double)z - (double)zmax);
    s = SIGMOID ? 1.0 / (1.0 + s) : s * inv;
    const bool open = z > -INFINITY && z < INFINITY && b > -INFINITY && b < INFINITY;
    key[e] = open ? s + (double)b : -INFINITY;
  }
  __syncwarp();
}

template <lrmoe_dtype DT, bool SIGMOID>
__device__ __noinline__ int order_fp64(const void* logits, int E, size_t row, float zmax, int mine,
                                       float z, float b, int n, uint64_t* box, int lane) {
  const double inv = SIGMOID ? 1.0 : 1.0 / sum_fp64<DT>(logits, E, row, zmax, lane);
  double v = exp(SIGMOID ? -(double)z : (double)z - (double)zmax);
  v = (SIGMOID ? 1.0 / (1.0 + v) : v * inv) + (double)b;
  int rank = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const double ov = __shfl_sync(kFull, v, i);
    const int om = __shfl_sync(kFull, mine, i);
    rank += ov > v || (ov == v && om < mine) ? 1 : 0;
  }
  if (lane < n) box[rank] = (uint64_t)mine;
  __syncwarp();
  if (lane < n) mine = (int)box[lane];
  __syncwarp();
  return mine;
}

__device__ __noinline__ unsigned kept_groups_fp64(const double* key, int E, int G, int keep, int lane) {
  const double kNone = -INFINITY;
  const int n = E / G, sub = 1 << (31 - __clz(32 / G)), mine = lane / sub;
  double a1 = kNone, a2 = kNone;
  if (mine < G) {
#pragma unroll 4
    for (int i = lane % sub; i < n; i += sub) merge_top2(a1, a2, key[mine * n + i], kNone);
  }
  for (int o = 1; o < sub; o <<= 1) {
    const double b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
    merge_top2(a1, a2, b1, b2);
  }
  double value = a2 > kNone ? a1 + a2 : a1;  // of group `lane`
  value = __shfl_sync(kFull, value, (lane * sub) & 31);
  if (lane >= G) value = kNone;
  int rank = 0;
#pragma unroll 4
  for (int g = 0; g < G; ++g) {
    const double v = __shfl_sync(kFull, value, g);
    rank += (v > value || (v == value && g < lane)) ? 1 : 0;
  }
  return __ballot_sync(kFull, rank < keep && value > kNone);
}

__device__ __noinline__ int topk_fp64(double* key, int E, int k, int lane) {
  uint64_t best;  // of this lane's experts: lane, lane + 32, ...
  int at;
  auto scan = [&] {
    best = kShut64;
    at = E;
    for (int e = lane; e < E; e += 32) {
      const uint64_t v = order_bits64(key[e]);
      if (v > best) {
        best = v;
        at = e;
      }
    }
  };
  scan();
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    const uint32_t high = __reduce_max_sync(kFull, (uint32_t)(best >> 32));
    bool top = (uint32_t)(best >> 32) == high;
    const uint32_t low = __reduce_max_sync(kFull, top ? (uint32_t)best : 0u);
    if ((((uint64_t)high << 32) | low) <= kShut64) break;  // uniform: nothing left
    top = top && (uint32_t)best == low;
    const int first = (int)__reduce_min_sync(kFull, top ? (unsigned)at : (unsigned)E);
    if (lane == j) mine = first;
    if (top && at == first) {
      key[at] = -INFINITY;
      scan();
    }
    __syncwarp();
  }
  return mine;
}

// The k experts of the largest keys in slot order, by threshold: at least k + 1 of the warp's keys
// reach the (k + 1)-th largest of the 32 lane maxima, and few more do while k is well below the number
// of lanes that hold experts (random logits, in the mean: 10 of 128 for k = 8, 22 for k = 16).  Lanes hold a
// power of two of experts, so E = 130 and 300 leave 17 and 19 lanes: for k = 16 more than 32 keys pass
// for 94% and 66% of the tokens (E = 72: 50%, 160: 39%, 384: 13%, 128 and 256: 0.2%; k <= 10: none).  Those that
// do are brought to one per lane and ranked by counting (key, lower
// expert first).  Lane j gets the j-th largest (mine, mine_key), for all that reach the threshold;
// whole: no expert is left behind them.
// False (nothing set) where more than 32 do.
template <int VPL>
__device__ __forceinline__ bool topk_by_threshold(const uint32_t (&key)[VPL], int k, int lane,
                                                  uint64_t* box, int& mine, uint32_t& mine_key,
                                                  bool& whole) {
  uint32_t best = key[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
  uint32_t bar = 0u;
  if (VPL > 1) {  // the largest maxima one after another, equal ones together
    uint32_t left = best;
    for (int seen = 0; seen <= k;) {
      bar = __reduce_max_sync(kFull, left);
      if (bar <= kShut) break;
      const bool top = left == bar;
      seen += __popc(__ballot_sync(kFull, top));
      if (top) left = 0u;
    }
  }
  whole = bar <= kShut;  // fewer lanes than that hold a key: take all keys
  if (whole) bar = kShut + 1u;
  int count = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool in = key[i] >= bar;
    const unsigned who = __ballot_sync(kFull, in);
    const int at = count + __popc(who & ((1u << lane) - 1u));
    if (in && at < 32) box[at] = ((uint64_t)key[i] << 32) | (uint32_t)~(lane * VPL + i);
    count += __popc(who);
  }
  __syncwarp();  // box is written, also for order_fp64 after a selection by rounds
  if (count > 32) return false;
  const uint64_t own = lane < count ? box[lane] : 0ull;
  if (lane >= count) box[lane] = 0ull;
  __syncwarp();
  int rank = 0;
  for (int c = 0; c < count; c += 4) {  // all lanes read one address: a broadcast
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(box + c);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(box + c + 2);
    rank += (a.x > own ? 1 : 0) + (a.y > own ? 1 : 0) + (b.x > own ? 1 : 0) + (b.y > own ? 1 : 0);
  }
  __syncwarp();
  if (lane < count) box[rank] = own;
  __syncwarp();
  if (lane < count) {
    const uint64_t got = box[lane];
    mine = (int)~(uint32_t)got;
    mine_key = (uint32_t)(got >> 32);
  }
  __syncwarp();  // before the next token's keys
  return true;
}

// The same in k + 1 rounds: the warp's largest key, its lowest holder, gone for the next round.
template <int VPL>
__device__ __noinline__ void topk_by_rounds(uint32_t (&key)[VPL], int k, int lane, int& mine,
                                            uint32_t& mine_key, bool& whole) {
  whole = false;
  for (int j = 0; j < (k < 31 ? k + 1 : 32); ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(kFull, best);
    whole = top <= kShut;
    if (whole) break;
    const int owner = __ffs(__ballot_sync(kFull, best == top)) - 1;
    int at = 0;
    if (lane == owner) {
      // the lowest register that holds it (scanned from the highest)
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        if (key[i] == top) at = i;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == at) key[i] = kShut;
    }
    at = __shfl_sync(kFull, at, owner) + owner * VPL;
    if (lane == j) {
      mine = at;
      mine_key = top;
    }
  }
}

// PLAIN: no bias and no groups, so that the order is that of the logits.
template <lrmoe_dtype DT, bool SIGMOID, bool PLAIN, int VPL>
__global__ void __launch_bounds__(32 * kRouteWarps, VPL <= 4 ? 8 : VPL == 8 ? 6 : VPL == 16 ? 4 : 2) route_kernel(const RouteParams p) {
  extern __shared__ double keys64[];  // [kRouteWarps][E], when a bias or groups are given
  __shared__ __align__(16) uint64_t boxes[kRouteWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = p.E, k = p.k, G = PLAIN ? 1 : p.groups;
  const float* biases = PLAIN ? nullptr : p.bias;
  const int e0 = lane * VPL;
  const int n = p.n;
  // groups of whole lanes: a lane's experts belong to one group, a group to lpg neighbouring lanes
  const bool whole = p.lpg > 0;
  const int lpg = p.lpg, my_group = G > 1 && whole ? lane / lpg : 0;
  pdl_wait();
  pdl_trigger();
  // this lane's biases; one that is not finite shuts its expert
  float bias[VPL];
  bool bad_bias = false;
  float low_bias = INFINITY;  // the lowest finite one
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    bias[i] = biases != nullptr && e0 + i < E ? __ldg(biases + e0 + i) : 0.0f;
    if (!(bias[i] < INFINITY)) {
      bad_bias = true;
      bias[i] = -INFINITY;
    }
    if (e0 + i < E && bias[i] > -INFINITY) low_bias = fminf(low_bias, bias[i]);
  }
  if (biases != nullptr) low_bias = -warp_max(-low_bias);
  // 64-bit: T may be near 2^31
  for (long long t = (long long)blockIdx.x * kRouteWarps + warp; t < p.T;
       t += (long long)gridDim.x * kRouteWarps) {
    const size_t row = (size_t)t * E;
    float z[VPL];
    load_row<DT, VPL>(p.logits, row, e0, E, z);
    bool bad = bad_bias;
    float zmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (!(z[i] < INFINITY)) {  // NaN or +inf
        bad = true;
        z[i] = -INFINITY;
      }
      if (!SIGMOID) zmax = fmaxf(zmax, z[i]);
    }
    if (__any_sync(kFull, bad) && lane == 0) raise_status(p.status, LRMOE_ST_NONFINITE);
    if (!SIGMOID && !(PLAIN && p.renorm)) zmax = warp_max(zmax);
    // Order keys, with a bound on the error of their scores (u = 2^-24).  The fast exponential of x
    // is off by 2 + 1.173 |x| ulp, (4 + 2.35 |x|) u relative; the reciprocal by 2 u.  sigmoid: with the
    // addition (7 + 2.35 (1 - s) |z|) u s.  softmax: z - zmax rounds by |z - zmax| u; the sum of the
    // exponentials has 36 additions and their mean error, |z - zmax| being ln E in the mean at most:
    // (73 + 3.35 |z - zmax|) u s.  With R the largest score there may be (1, or the softmax of
    // zmax), no score of at most S has an error of more than
    //   (A + 3.35 max(1, ln(R / S))) u S,  A = 7 or 73:
    // s |z - zmax| = s ln(R / s), and s |z| <= s ln(1 / s) for z < 0, rise with s up to R / e and stay
    // below 0.37 R; s (1 - s) z is below 0.23 for z > 0.
    // Scores under 2e-38 count as that or 0.
    constexpr float kErr = SIGMOID ? 7.0f : 73.0f;
    constexpr float kU = 6.0e-8f;  // a little above u
    uint32_t key[VPL];
    float rden = 1.0f;  // softmax: the largest score
    if constexpr (PLAIN) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = order_bits(z[i]);
    } else {
      float sc[VPL];
      if constexpr (SIGMOID) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) sc[i] = fast_rcp(1.0f + __expf(fminf(-z[i], 87.0f)));
      } else {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          sc[i] = z[i] > -INFINITY ? __expf(z[i] - zmax) : 0.0f;
          sum += sc[i];
        }
        rden = fast_rcp(warp_sum(sum));
#pragma unroll
        for (int i = 0; i < VPL; ++i) sc[i] *= rden;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        key[i] = order_bits(z[i] > -INFINITY ? sc[i] + bias[i] : -INFINITY);
    }
    double* kd = keys64 + (size_t)warp * E;
    unsigned kept = 0u;  // groups
    if (G > 1) {
      // lane g: the two largest keys of group g
      uint32_t top1 = kShut, top2 = kShut;
      if (whole) {
        const int pos = lane - my_group * lpg;
        uint32_t a1 = kShut, a2 = kShut;
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
        const int from = lane < G ? lane * lpg : 0;
        a1 = __shfl_sync(kFull, a1, from);
        a2 = __shfl_sync(kFull, a2, from);
        if (lane < G) top1 = a1, top2 = a2;
      } else {
        for (int g = 0; g < G; ++g) {
          uint32_t a1 = kShut, a2 = kShut;
#pragma unroll
          for (int i = 0; i < VPL; ++i) {
            const int e = e0 + i;
            const uint32_t kv = e >= g * n && e < (g + 1) * n ? key[i] : kShut;
            a2 = max(a2, min(a1, kv));
            a1 = max(a1, kv);
          }
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) {
            const uint32_t b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
            a2 = max(max(a2, b2), min(a1, b1));
            a1 = max(a1, b1);
          }
          if (lane == g) top1 = a1, top2 = a2;
        }
      }
      // the group's value is their sum (-inf: no expert left in it)
      const float c1 = order_value(top1), c2 = top2 > kShut ? order_value(top2) : 0.0f;
      const float value = c1 + c2;
      // the best ones, the lower of equal ones first
      uint32_t left = order_bits(value);
      for (int j = 0; j < p.keep_groups; ++j) {
        const uint32_t top = __reduce_max_sync(kFull, left);
        if (top <= kShut) break;
        const int g = __ffs(__ballot_sync(kFull, left == top)) - 1;
        kept |= 1u << g;
        if (lane == g) left = kShut;
      }
      // Sure if the kept values, less their errors, are above the others and theirs: two scores, the
      // rounding of their keys and that of the sum.
      const float R = SIGMOID ? 1.0f : rden;
      // (A NaN of a sum that overflows counts as not sure.)
      const float err = 2.0f * (kErr + 3.5f) * kU * R + 4.0f * kU * (fabsf(c1) + fabsf(c2)) + 1e-36f;
      const bool in = (kept >> lane) & 1u, out = !in && top1 > kShut;
      const float least = in ? fmaxf(value - err, -INFINITY) : INFINITY;
      const float most = out ? fminf(value + err, INFINITY) : -INFINITY;
      const uint32_t low = __reduce_min_sync(kFull, order_bits(least));
      const uint32_t high = __reduce_max_sync(kFull, order_bits(most));
      if (low <= high) {
        keys_fp64<DT, SIGMOID>(p.logits, biases, E, row, zmax, kd, lane);
        kept = kept_groups_fp64(kd, E, G, p.keep_groups, lane);
      }
      if (whole) {
        if (!((kept >> my_group) & 1u)) {
#pragma unroll
          for (int i = 0; i < VPL; ++i) key[i] = kShut;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (e0 + i < E && !((kept >> ((e0 + i) / n)) & 1u)) key[i] = kShut;
      }
      if (biases == nullptr) {  // inside the kept groups the score rises with the logit
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (key[i] != kShut) key[i] = order_bits(z[i]);
      }
    }
    int mine = -1;             // expert of slot `lane`
    uint32_t mine_key = kShut; // its key (lane k: the best one left)
    bool whole_order;  // no expert behind those of the lanes
    if (k == 32 || !topk_by_threshold<VPL>(key, k, lane, boxes[warp], mine, mine_key, whole_order))
      topk_by_rounds<VPL>(key, k, lane, mine, mine_key, whole_order);
    float zj = mine >= 0 ? load_logit<DT>(p.logits, row + mine) : -INFINITY;
    if (biases != nullptr) {
      // Is the order of the slots, and of the best expert left, sure?  Lane i compares expert i of
      // the order with all behind it.  Their keys are at most c2, that of i + 1, so none of their
      // scores is above S.  (Rounding the sums s + b keeps their order: only the rounding of c
      // and c2 counts.)
      const float c = mine >= 0 ? order_value(mine_key) : 0.0f;
      const float b = mine >= 0 ? __ldg(biases + mine) : 0.0f;
      const float R = SIGMOID ? 1.0f : rden;
      auto above = [&](float c2) {
        const float S = fmaxf(1e-36f, fminf(R, fmaxf(c - b, c2 - low_bias) +
                                                   2.0f * kU * (fabsf(c) + fabsf(c2) + fabsf(low_bias))));
        return c - c2 > 2.0f * kU * S * (kErr + 3.5f * fmaxf(1.0f, __logf(R / S))) +
                            2.0f * kU * (fabsf(c) + fabsf(c2)) + 1e-36f;
      };
      const float c2 = __shfl_down_sync(kFull, c, 1), b2 = __shfl_down_sync(kFull, b, 1);
      const float z2 = __shfl_down_sync(kFull, zj, 1);
      const unsigned have = __ballot_sync(kFull, mine >= 0);
      const bool pair = (have >> 1 >> lane) & 1u;  // lanes 0 .. n - 1 have an expert
      const bool same = pair && zj == z2 && b == b2;
      const unsigned close = __ballot_sync(kFull, pair && !same && !above(c2));
      // Equal experts are in their order already, and what is behind the second is behind the
      // first: the last comparison that counts is the first of unequal ones from slot k - 1 on.
      const unsigned equal = __ballot_sync(kFull, same) >> (k - 1);
      const int last = k - 1 + __ffs(~equal) - 1;
      const bool compared = (have >> 1 >> last) & 1u;
      bool sure = !(close & (0xffffffffu >> (31 - last))) && (compared || whole_order);
      if (!sure) {
        // If the slots' experts are above all that have no lane, the fp64 keys of the lanes decide.
        const int found = __popc(have);
        const float lowest = __shfl_sync(kFull, c, found - 1);
        if (whole_order || __all_sync(kFull, lane >= k || above(lowest))) {
          mine = order_fp64<DT, SIGMOID>(p.logits, E, row, zmax, mine, zj, b, found, boxes[warp], lane);
          zj = mine >= 0 ? load_logit<DT>(p.logits, row + mine) : -INFINITY;
          sure = true;
        }
      }
      if (!sure) {  // uniform across the warp
        keys_fp64<DT, SIGMOID>(p.logits, biases, E, row, zmax, kd, lane);
        if (G > 1) {
          for (int e = lane; e < E; e += 32)
            if (!((kept >> (e / n)) & 1u)) kd[e] = -INFINITY;
          __syncwarp();
        }
        mine = topk_fp64(kd, E, k, lane);
        zj = mine >= 0 ? load_logit<DT>(p.logits, row + mine) : -INFINITY;
      }
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
      const float sum = warp_sum(s);  // between 1/2 and 32
      s = mine >= 0 ? __fdividef(s, sum) : 0.0f;
    } else if constexpr (SIGMOID) {
      if (mine >= 0) s = sigmoid_scaled(zj, 0.0f);
    } else {
      float den = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) den += z[i] > -INFINITY ? expf(z[i] - zmax) : 0.0f;
      den = warp_sum(den);
      if (mine >= 0) s = expf(zj - zmax) / den;
    }
    if (slot) {
      p.idx[t * k + lane] = mine;
      p.w[t * k + lane] = mine >= 0 ? s * p.scale : 0.0f;
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
          w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
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

// An expert named by several slots: the first of them gets the sum over all, in slot order.  `tag`
// tells the experts of the warp's tokens apart; lanes without a slot have e < 0.  True for the
// lanes that write their expert's value.
__device__ __forceinline__ bool first_of_slots(int e, float& d, int tag, int lane) {
  const unsigned same = __match_any_sync(kFull, e >= 0 ? tag : ~lane);
  if (!__any_sync(kFull, (same & (same - 1u)) != 0u)) return e >= 0;
  const float own = d;
  d = 0.0f;
  for (int i = 0; i < 32; ++i) {
    const float di = __shfl_sync(kFull, own, i);
    if ((same >> i) & 1u) d += di;
  }
  return e >= 0 && lane == __ffs(same) - 1;
}

template <lrmoe_dtype DT>
__device__ __forceinline__ void store_logit(void* z, size_t i, float v) {
  if constexpr (DT == LRMOE_BF16)
    static_cast<unsigned short*>(z)[i] = (unsigned short)f32_to_bf16_bits_rne(v);
  else
    static_cast<float*>(z)[i] = v;
}

// One token's slots, slot j in lane j of the token's SUB lanes:
//   renormalised: p_j = s_j / S, d_j = scale p_j (dw_j - sum_i p_i dw_i), for sigmoid times (1 - s_j)
//   sigmoid:      d_j = scale dw_j s_j (1 - s_j)
// and dz_e = sum of d over the slots of e: the row is zeros but for the slots' experts, so only
// their logits are read.  SUB lanes take a token (k <= SUB), a warp 32 / SUB neighbouring tokens.
// A single renormalised slot (p = 1) gets exactly 0.
template <lrmoe_dtype DT, bool SIGMOID, bool RENORM, int SUB>
__global__ void __launch_bounds__(256) route_grad_sparse_kernel(const RouteGradParams p) {
  constexpr int kTokens = 32 / SUB;
  constexpr int kSize = DT == LRMOE_BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31, sub = lane / SUB, j = lane % SUB;
  const int E = p.E, k = p.k;
  auto sum = [](float v) {
#pragma unroll
    for (int o = SUB / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
  };
  const long long step = (long long)gridDim.x * 8 * kTokens;
  pdl_wait();
  pdl_trigger();
  for (long long t0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kTokens; t0 < p.T; t0 += step) {
    const long long t = t0 + sub;
    const bool live = t < p.T;
    const size_t row = (size_t)t * E;
    int e = live && j < k ? __ldg(p.idx + t * k + j) : -1;
    if (live) {  // zeros first; the slots' values follow
      char* at = static_cast<char*>(p.dlogits) + row * kSize;
      const int bytes = E * kSize;
      if (bytes % 16 == 0) {
        for (int i = j * 16; i < bytes; i += SUB * 16)
          *reinterpret_cast<uint4*>(at + i) = make_uint4(0, 0, 0, 0);
      } else if (bytes % 4 == 0) {
        for (int i = j * 4; i < bytes; i += SUB * 4) *reinterpret_cast<uint32_t*>(at + i) = 0u;
      } else {
        for (int i = j * 2; i < bytes; i += SUB * 2) *reinterpret_cast<unsigned short*>(at + i) = 0;
      }
    }
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
    const float dw = e >= 0 ? __ldg(p.dw + t * k + j) : 0.0f;
    float d = 0.0f;
    if constexpr (RENORM) {
      float zc = z;
#pragma unroll
      for (int o = SUB / 2; o >= 1; o >>= 1) zc = fmaxf(zc, __shfl_xor_sync(kFull, zc, o));
      float s = 0.0f;
      if (e >= 0) s = SIGMOID ? sigmoid_scaled(z, fminf(zc, 0.0f)) : expf(z - zc);
      const float total = sum(s);
      const float pj = e >= 0 ? s / total : 0.0f;
      const float mean = sum(pj * dw);
      d = p.scale * pj * (dw - mean);
      if (SIGMOID && e >= 0) d *= sigmoid_scaled(-z, 0.0f);
    } else {
      if (e >= 0) d = p.scale * dw * sigmoid_scaled(z, 0.0f) * sigmoid_scaled(-z, 0.0f);
    }
    const bool write = first_of_slots(e, d, (sub << 16) | e, lane);
    __syncwarp();  // the zeros are written before the values
    if (write) store_logit<DT>(p.dlogits, row + e, d);
  }
}

// Softmax, not renormalised: every logit gets a gradient,
//   dz_e = s_e (scale sum of dw over the slots of e - scale sum_i dw_i s_i):
// the row as if no slot named an expert, then the slots' experts again.
template <lrmoe_dtype DT, int VPL>
__global__ void __launch_bounds__(256) route_grad_dense_kernel(const RouteGradParams p) {
  const int lane = threadIdx.x & 31;
  const int E = p.E, k = p.k;
  const int e0 = lane * VPL;
  pdl_wait();
  pdl_trigger();
  for (long long t = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); t < p.T;
       t += (long long)gridDim.x * 8) {
    const size_t row = (size_t)t * E;
    float v[VPL];  // then exp(z - zmax) of the lane's experts (0: not finite)
    load_row<DT, VPL>(p.logits, row, e0, E, v);
    int e = lane < k ? __ldg(p.idx + t * k + lane) : -1;
    if (e >= E) {
      raise_status(p.status, LRMOE_ST_BAD_EXPERT);
      e = -1;
    }
    const float z = e >= 0 ? load_logit<DT>(p.logits, row + e) : -INFINITY;
    if (!(fabsf(z) < INFINITY)) e = -1;  // NaN and +inf are flagged with the row
    const float dw = e >= 0 ? __ldg(p.dw + t * k + lane) : 0.0f;
    float m = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (!(v[i] < INFINITY)) {
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
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const float sj = e >= 0 ? expf(z - zmax) * inv : 0.0f;
    const float dot = warp_sum(dw * sj);
    const float rest = -p.scale * dot * inv;
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] *= rest;
    store_row<DT, VPL>(p.dlogits, row, e0, E, v);
    float d = dw;
    const bool write = first_of_slots(e, d, e, lane);
    __syncwarp();  // the row is written before the slots' values
    if (write) store_logit<DT>(p.dlogits, row + e, sj * (p.scale * (d - dot)));
  }
}

template <lrmoe_dtype DT, bool SIGMOID, bool PLAIN>
cudaError_t route_by_width(RouteParams p, cudaStream_t s) {
  auto kern = route_kernel<DT, SIGMOID, PLAIN, 32>;
  int vpl = 32;  // experts of a lane
  if (p.E <= 32) {
    kern = route_kernel<DT, SIGMOID, PLAIN, 1>;
    vpl = 1;
  } else if (p.E <= 64) {
    kern = route_kernel<DT, SIGMOID, PLAIN, 2>;
    vpl = 2;
  } else if (p.E <= 128) {
    kern = route_kernel<DT, SIGMOID, PLAIN, 4>;
    vpl = 4;
  } else if (p.E <= 256) {
    kern = route_kernel<DT, SIGMOID, PLAIN, 8>;
    vpl = 8;
  } else if (p.E <= 512) {
    kern = route_kernel<DT, SIGMOID, PLAIN, 16>;
    vpl = 16;
  }
  p.n = p.E / p.groups;
  p.lpg = p.n % vpl == 0 ? p.n / vpl : 0;
  const size_t smem = PLAIN ? 0 : sizeof(double) * (size_t)kRouteWarps * p.E;  // <= 32 KB
  long long blocks = ((long long)p.T + kRouteWarps - 1) / kRouteWarps;
  // A warp keeps its biases over several tokens.  Tokens take unequal times (those that go to
  // fp64 and back 1.5 times as long and more), so more blocks than are resident at once: E = 256 in
  // groups, T = 16383, 16 to an SM 22.8 us, 8 to an SM 26; with wider rows the biases count for more.
  const long long cap = (long long)num_sms() * (p.E <= 256 ? 16 : 4);
  if (blocks > cap) blocks = cap;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(32 * kRouteWarps), smem, s, p);
}

template <lrmoe_dtype DT, bool SIGMOID>
cudaError_t route_by_order(const RouteParams& p, cudaStream_t s) {
  return p.bias == nullptr && p.groups == 1 ? route_by_width<DT, SIGMOID, true>(p, s)
                                            : route_by_width<DT, SIGMOID, false>(p, s);
}

template <lrmoe_dtype DT, bool SIGMOID, bool RENORM>
cudaError_t route_grad_sparse(const RouteGradParams& p, cudaStream_t s) {
  auto kern = route_grad_sparse_kernel<DT, SIGMOID, RENORM, 32>;
  int sub = 32;
  if (p.k <= 8) {
    kern = route_grad_sparse_kernel<DT, SIGMOID, RENORM, 8>;
    sub = 8;
  } else if (p.k <= 16) {
    kern = route_grad_sparse_kernel<DT, SIGMOID, RENORM, 16>;
    sub = 16;
  }
  const long long tokens = 8 * (32 / sub);  // of a block
  long long blocks = (p.T + tokens - 1) / tokens;
  const long long cap = (long long)num_sms() * 32;
  if (blocks > cap) blocks = cap;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, s, p);
}

template <lrmoe_dtype DT>
cudaError_t route_grad_dense(const RouteGradParams& p, cudaStream_t s) {
  auto kern = route_grad_dense_kernel<DT, 32>;
  if (p.E <= 32)
    kern = route_grad_dense_kernel<DT, 1>;
  else if (p.E <= 64)
    kern = route_grad_dense_kernel<DT, 2>;
  else if (p.E <= 128)
    kern = route_grad_dense_kernel<DT, 4>;
  else if (p.E <= 256)
    kern = route_grad_dense_kernel<DT, 8>;
  else if (p.E <= 512)
    kern = route_grad_dense_kernel<DT, 16>;
  long long blocks = ((long long)p.T + 7) / 8;
  const long long cap = (long long)num_sms() * 16;
  if (blocks > cap) blocks = cap;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, s, p);
}

template <lrmoe_dtype DT>
cudaError_t route_grad_by_fn(const RouteGradParams& p, bool sigmoid, bool renorm, cudaStream_t s) {
  if (!renorm) return sigmoid ? route_grad_sparse<DT, true, false>(p, s) : route_grad_dense<DT>(p, s);
  return sigmoid ? route_grad_sparse<DT, true, true>(p, s) : route_grad_sparse<DT, false, true>(p, s);
}

}  // namespace

cudaError_t launch_route(const void* logits, int T, int E, lrmoe_dtype dt, const float* bias, int k,
                         lrmoe_score_fn fn, int n_group, int topk_group, int renorm, float scale,
                         int32_t* idx, float* w, uint32_t* status, cudaStream_t s) {
  const RouteParams p{logits, bias, T, E, k, n_group, topk_group, renorm, 0, 0, scale, idx, w, status};
  const bool sg = fn == LRMOE_SCORE_SIGMOID;
  if (dt == LRMOE_BF16)
    return sg ? route_by_order<LRMOE_BF16, true>(p, s) : route_by_order<LRMOE_BF16, false>(p, s);
  return sg ? route_by_order<LRMOE_F32, true>(p, s) : route_by_order<LRMOE_F32, false>(p, s);
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
