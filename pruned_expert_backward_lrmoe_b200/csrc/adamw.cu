// The step that the layer's weight gradients are for: the norm over many gradient tensors and one
// AdamW step over many tensors at once.
//
//   norm = sqrt(sum g^2), factor = min(1, max_norm / norm)
//   g <- s g,  m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2
//   p <- p - lr wd p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// The list of tensors travels in the launch's parameters, so that a call needs no device memory for it
// and a captured call keeps its own.  Tiles of 2048 values are dealt to the blocks in turn; a warp takes
// 256 neighbouring values of a tile, lane l the values 4 l .. 4 l + 3 of each half.  That is the block of
// the 8-bit states, whose largest magnitudes are then one reduction over the warp.
//
// HBM-bound: every value is read and written once.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "step.h"

namespace lrmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 256;          // values of a warp, and to a scale
constexpr int kTile = 8 * kBlock;    // values of a block's turn
constexpr int kNormBlocks = 148 * 8; // at most, of a launch

constexpr int kFew = 24, kMany = 448;  // tensors of a launch: 1.8 KB or 32 KB of parameters

struct Item {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  long long n;
  float decay;   // lr-free weight decay
  unsigned end;  // tiles up to this tensor's last
};

template <int CAP>
struct Items {
  Item t[CAP];
};

// The tensor of `tile`, at or behind `at`.
template <int CAP>
__device__ __forceinline__ int find_item(const Items<CAP>& list, int count, int at, unsigned tile) {
  if (tile < list.t[at].end) return at;
  int lo = at + 1, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (tile < list.t[mid].end)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Four values from an address of a whole vector; past `left` they are 0 and not read.
template <lrmoe_dtype DT>
__device__ __forceinline__ void load4(const void* at, long long i, int left, float (&v)[4]) {
  if constexpr (DT == LRMOE_F32) {
    const float* a = static_cast<const float*>(at) + i;
    if (left >= 4) {
      const float4 q = *reinterpret_cast<const float4*>(a);
      v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = j < left ? a[j] : 0.0f;
    }
  } else {
    const unsigned short* a = static_cast<const unsigned short*>(at) + i;
    if (left >= 4) {
      const uint2 q = *reinterpret_cast<const uint2*>(a);
      v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
      v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = j < left ? bf16_bits_to_f32(a[j]) : 0.0f;
    }
  }
}

template <lrmoe_dtype DT>
__device__ __forceinline__ void store4(void* at, long long i, int left, const float (&v)[4]) {
  if constexpr (DT == LRMOE_F32) {
    float* a = static_cast<float*>(at) + i;
    if (left >= 4) {
      *reinterpret_cast<float4*>(a) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) a[j] = v[j];
    }
  } else {
    unsigned short* a = static_cast<unsigned short*>(at) + i;
    if (left >= 4) {
      *reinterpret_cast<uint2*>(a) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) a[j] = (unsigned short)f32_to_bf16_bits_rne(v[j]);
    }
  }
}

// e4m3 codes
__device__ __forceinline__ void load4_codes(const void* at, long long i, int left, float (&v)[4]) {
  const uint8_t* a = static_cast<const uint8_t*>(at) + i;
  uint32_t q = 0;
  if (left >= 4) {
    q = *reinterpret_cast<const uint32_t*>(a);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) q |= (uint32_t)a[j] << (8 * j);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)(q >> (16 * j))));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    v[2 * j] = lo;
    v[2 * j + 1] = hi;
  }
}

__device__ __forceinline__ void store4_codes(void* at, long long i, int left, const float (&v)[4]) {
  uint8_t* a = static_cast<uint8_t*>(at) + i;
  unsigned short lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
  const uint32_t q = lo | ((uint32_t)hi << 16);
  if (left >= 4) {
    *reinterpret_cast<uint32_t*>(a) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) a[j] = (uint8_t)(q >> (8 * j));
  }
}

// ---------------------------------------------------------------------------
// norm
// ---------------------------------------------------------------------------
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[32];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += part[w];
  return s;  // of thread 0
}

template <lrmoe_dtype DT, int CAP>
__global__ void __launch_bounds__(kThreads)
    norm_kernel(const __grid_constant__ Items<CAP> list, int count, double* __restrict__ partial) {
  const unsigned tiles = list.t[count - 1].end;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  double total = 0.0;
  int at = 0;
  for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    at = find_item(list, count, at, tile);
    const Item& it = list.t[at];
    const long long base = (long long)(tile - (at ? list.t[at - 1].end : 0u)) * kTile + warp * kBlock + lane * 4;
    float g[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long left = it.n - base - 128 * h;
      load4<DT>(it.g, base + 128 * h, (int)min(max(left, 0ll), 4ll), g[h]);
    }
    float s = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) s = fmaf(g[h][j], g[h][j], s);
    double d = s;
    if (!(s < 1e37f) || s < 1e-25f) {  // squares out of fp32's range, or all 0
      d = 0.0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) d = fma((double)g[h][j], (double)g[h][j], d);
    }
    total += d;
  }
  total = block_sum(total);
  if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

__global__ void __launch_bounds__(1024) norm_finish_kernel(const double* __restrict__ partial, int n,
                                                           float max_norm, float* __restrict__ out,
                                                           uint32_t* __restrict__ status) {
  pdl_wait();
  pdl_trigger();
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) s += partial[i];
  s = block_sum(s);
  if (threadIdx.x == 0) {
    const double norm = sqrt(s);
    const bool fine = norm - norm == 0.0;
    if (!fine) raise_status(status, LRMOE_ST_NONFINITE);
    out[0] = (float)norm;
    out[1] = !fine ? 0.0f : norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.0f;
  }
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
struct Hyper {
  float b1, a1, b2, a2;  // b and 1 - b
  float eps;
  float lr, rate, root;  // lr, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  double log_b1, log_b2;
  const float* lr_dev;
  const int32_t* step_dev;
  const float* grad_scale;
  uint32_t seed;
  int step, first;  // `first`: number of the launch's first tensor
  uint32_t* status;
};

__host__ __device__ __forceinline__ uint32_t mix(uint32_t h) {
  h ^= h >> 16;
  h *= 0x9E3779B1u;
  h ^= h >> 15;
  h *= 0x6A09E667u;
  return h ^ (h >> 16);
}

// x in [0, 448] to one of its two e4m3 neighbours: 16 random bits are added to the 20 that are
// dropped.  Below 2^-6 the values are 2^-9 apart, as they are from 2^-6 to 2^-5, where x is moved.
__device__ __forceinline__ float round_code(float x, uint32_t bits16) {
  const float low = x < 0.015625f ? 0.015625f : 0.0f;
  const uint32_t b = __float_as_uint(x + low) + (bits16 << 4);
  return __uint_as_float(b & 0xfff00000u) - low;
}

__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float warp_max_abs(float v) {  // v >= 0
  return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(v)));
}

// A block's scale and its inverse.
__device__ __forceinline__ void scale_of(float top, float& scale, float& inv) {
  scale = top > 0.0f ? fmaxf(top * (1.0f / 448.0f), 1.17549435e-38f) : 0.0f;
  inv = top > 0.0f ? 1.0f / scale : 0.0f;
}

template <lrmoe_dtype PDT, bool MASTER, lrmoe_dtype GDT, int BITS, int CAP>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ Items<CAP> list, int count, const __grid_constant__ Hyper hy) {
  constexpr bool kRandomParam = PDT == LRMOE_BF16 && !MASTER;
  constexpr lrmoe_dtype KDT = MASTER ? LRMOE_F32 : PDT;  // of the kept weights
  const unsigned tiles = list.t[count - 1].end;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float shared_hyper[3];
  pdl_wait();
  pdl_trigger();
  const float gs = hy.grad_scale ? __ldg(hy.grad_scale) : 1.0f;
  if (gs == 0.0f) return;
  float lr = hy.lr, rate = hy.rate, root = hy.root;
  int step = hy.step;
  if (hy.lr_dev || hy.step_dev) {
    if (hy.step_dev) step = max(__ldg(hy.step_dev), 1);
    if (threadIdx.x == 0) {
      const double l = hy.lr_dev ? (double)__ldg(hy.lr_dev) : (double)hy.lr;
      shared_hyper[0] = (float)l;
      shared_hyper[1] = (float)(l / -expm1(step * hy.log_b1));
      shared_hyper[2] = (float)(1.0 / sqrt(-expm1(step * hy.log_b2)));
    }
    __syncthreads();
    lr = shared_hyper[0];
    rate = shared_hyper[1];
    root = shared_hyper[2];
  }
  const uint32_t step_key = mix(mix(hy.seed) + (uint32_t)step);
  bool bad = false;
  int at = 0;
  for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    at = find_item(list, count, at, tile);
    const Item& it = list.t[at];
    const long long first = (long long)(tile - (at ? list.t[at - 1].end : 0u)) * kTile + warp * kBlock;
    if (first >= it.n) continue;
    const long long base = first + lane * 4;
    const float decay = lr * it.decay;
    void* kept = MASTER ? static_cast<void*>(it.master) : it.p;
    int left[2];
    float g[2][4], p[2][4], m[2][4], v[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      left[h] = (int)min(max(it.n - base - 128 * h, 0ll), 4ll);
      const long long i = base + 128 * h;
      load4<GDT>(it.g, i, left[h], g[h]);
      load4<KDT>(kept, i, left[h], p[h]);
      if constexpr (BITS == 32) {
        load4<LRMOE_F32>(it.m, i, left[h], m[h]);
        load4<LRMOE_F32>(it.v, i, left[h], v[h]);
      } else {
        load4_codes(it.m, i, left[h], m[h]);
        load4_codes(it.v, i, left[h], v[h]);
      }
    }
    float ms = 1.0f, vs = 1.0f;
    if constexpr (BITS == 8) {
      ms = it.m_scale[first / kBlock];
      vs = it.v_scale[first / kBlock];
    }
    uint32_t key = 0;
    if constexpr (BITS == 8 || kRandomParam) {
      key = mix(step_key + (uint32_t)(hy.first + at));
      key += (uint32_t)base + (uint32_t)(base >> 32) * 0x632BE5ABu;
    }
    float top_m = 0.0f, top_v = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float gg = g[h][j] * gs;
        const float m0 = BITS == 8 ? __fmul_rn(m[h][j], ms) : m[h][j];
        const float r0 = BITS == 8 ? v[h][j] * vs : 0.0f;
        const float v0 = BITS == 8 ? __fmul_rn(r0, r0) : v[h][j];
        // each product and sum rounded by itself, and an exact root: the codes depend on their last bits
        const float m1 = __fadd_rn(__fmul_rn(hy.b1, m0), __fmul_rn(hy.a1, gg));
        const float v1 = __fadd_rn(__fmul_rn(hy.b2, v0), __fmul_rn(__fmul_rn(hy.a2, gg), gg));
        const bool ok = v1 < INFINITY;
        bad |= !ok;
        const float r1 = __fsqrt_rn(v1);
        const float p0 = p[h][j];
        const float p1 = fmaf(-rate * m1, rcp_fast(fmaf(r1, root, hy.eps)), fmaf(-decay, p0, p0));
        m[h][j] = ok ? m1 : m0;
        v[h][j] = BITS == 8 ? (ok ? r1 : r0) : (ok ? v1 : v0);
        p[h][j] = ok ? p1 : p0;
        if constexpr (BITS == 8) {
          top_m = fmaxf(top_m, fabsf(m[h][j]));
          top_v = fmaxf(top_v, fabsf(v[h][j]));
        }
      }
    }
    float im = 0.0f, iv = 0.0f;
    if constexpr (BITS == 8) {
      scale_of(warp_max_abs(top_m), ms, im);
      scale_of(warp_max_abs(top_v), vs, iv);
      if (lane == 0) {
        it.m_scale[first / kBlock] = ms;
        it.v_scale[first / kBlock] = vs;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long i = base + 128 * h;
      if constexpr (BITS == 8 || kRandomParam) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = mix(key + 128 * h + j);
          if constexpr (BITS == 8) {
            m[h][j] = copysignf(round_code(fabsf(m[h][j]) * im, w & 0xffffu), m[h][j]);
            const float x = v[h][j] * iv;
            const float y = round_code(x, w >> 16);
            v[h][j] = x > 0.0f ? fmaxf(y, 0.001953125f) : y;
          }
          if constexpr (kRandomParam)
            p[h][j] = __uint_as_float((__float_as_uint(p[h][j]) + ((w * 0x9E3779B1u) >> 16)) & 0xffff0000u);
        }
      }
      if constexpr (MASTER) store4<LRMOE_F32>(it.master, i, left[h], p[h]);
      store4<PDT>(it.p, i, left[h], p[h]);
      if constexpr (BITS == 32) {
        store4<LRMOE_F32>(it.m, i, left[h], m[h]);
        store4<LRMOE_F32>(it.v, i, left[h], v[h]);
      } else {
        store4_codes(it.m, i, left[h], m[h]);
        store4_codes(it.v, i, left[h], v[h]);
      }
    }
  }
  if (bad) raise_status(hy.status, LRMOE_ST_NONFINITE);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// The next launch's tensors from `next` on (empty ones left out); their number.
template <int CAP>
int fill(Items<CAP>& list, const lrmoe_tensor* t, int count, int& next, int& first) {
  int n = 0;
  unsigned long long tiles = 0;
  first = next;
  for (; next < count && n < CAP; ++next) {
    const lrmoe_tensor& s = t[next];
    const unsigned long long more = ((unsigned long long)s.n + kTile - 1) / kTile;
    if (n > 0 && tiles + more > 0x7fffffffull) break;
    tiles += more;
    list.t[n++] = Item{s.param, s.master, s.grad, s.m, s.v, s.m_scale, s.v_scale, (long long)s.n,
                       s.weight_decay, (unsigned)tiles};
  }
  return n;
}

template <typename F>
cudaError_t over_launches(const lrmoe_tensor* t, int count, F&& f) {
  int next = 0, first = 0;
  while (next < count) {
    cudaError_t e;
    if (count - next <= kFew) {
      Items<kFew> list;
      const int n = fill(list, t, count, next, first);
      e = list.t[n - 1].end ? f(list, n, first) : cudaSuccess;
    } else {
      Items<kMany> list;
      const int n = fill(list, t, count, next, first);
      e = list.t[n - 1].end ? f(list, n, first) : cudaSuccess;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int CAP>
unsigned grid_of(const Items<CAP>& list, int n, int per_sm) {
  const unsigned tiles = list.t[n - 1].end, most = (unsigned)(num_sms() * per_sm);
  return tiles < most ? tiles : most;
}

}  // namespace

size_t grad_norm_workspace(int count) {
  return sizeof(double) * kNormBlocks * (size_t)((count + kMany - 1) / kMany + 1);
}

cudaError_t launch_grad_norm(const lrmoe_tensor* t, int count, lrmoe_dtype dt, float max_norm,
                             float* out, void* ws, uint32_t* status, cudaStream_t s) {
  double* partial = static_cast<double*>(ws);
  int n = 0;
  cudaError_t e = over_launches(t, count, [&](auto& list, int items, int) {
    constexpr int CAP = sizeof(list.t) / sizeof(Item);
    unsigned grid = grid_of(list, items, 8);
    if (grid > (unsigned)kNormBlocks) grid = kNormBlocks;
    auto kern = dt == LRMOE_BF16 ? norm_kernel<LRMOE_BF16, CAP> : norm_kernel<LRMOE_F32, CAP>;
    cudaError_t r = launch_pdl(kern, dim3(grid), dim3(kThreads), 0, s, list, items, partial + n);
    n += (int)grid;
    return r;
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_finish_kernel, dim3(1), dim3(1024), 0, s, partial, n, max_norm, out, status);
}

namespace {

template <lrmoe_dtype PDT, bool MASTER, int CAP>
auto pick(lrmoe_dtype gdt, int bits) {
  if (gdt == LRMOE_BF16)
    return bits == 8 ? adamw_kernel<PDT, MASTER, LRMOE_BF16, 8, CAP> : adamw_kernel<PDT, MASTER, LRMOE_BF16, 32, CAP>;
  return bits == 8 ? adamw_kernel<PDT, MASTER, LRMOE_F32, 8, CAP> : adamw_kernel<PDT, MASTER, LRMOE_F32, 32, CAP>;
}

}  // namespace

cudaError_t launch_adamw(const lrmoe_tensor* t, int count, lrmoe_dtype pdt, lrmoe_dtype gdt,
                         int bits, const AdamwArgs& a, cudaStream_t s) {
  Hyper h{};
  h.b1 = (float)a.beta1;
  h.a1 = (float)(1.0 - a.beta1);
  h.b2 = (float)a.beta2;
  h.a2 = (float)(1.0 - a.beta2);
  h.eps = a.eps;
  h.log_b1 = log(a.beta1);
  h.log_b2 = log(a.beta2);
  h.step = a.step < 1 ? 1 : a.step;
  h.lr = (float)a.lr;
  h.rate = (float)(a.lr / -expm1(h.step * h.log_b1));
  h.root = (float)(1.0 / sqrt(-expm1(h.step * h.log_b2)));
  h.lr_dev = a.lr_dev;
  h.step_dev = a.step_dev;
  h.grad_scale = a.grad_scale;
  h.seed = a.seed;
  h.status = a.status;
  bool master = false;
  for (int i = 0; i < count; ++i) master |= t[i].n > 0 && t[i].master != nullptr;
  return over_launches(t, count, [&](auto& list, int items, int first) {
    constexpr int CAP = sizeof(list.t) / sizeof(Item);
    h.first = first;
    auto kern = pdt == LRMOE_F32 ? pick<LRMOE_F32, false, CAP>(gdt, bits)
                : master         ? pick<LRMOE_BF16, true, CAP>(gdt, bits)
                                 : pick<LRMOE_BF16, false, CAP>(gdt, bits);
    return launch_pdl(kern, dim3(grid_of(list, items, 8)), dim3(kThreads), 0, s, list, items, h);
  });
}

}  // namespace lrmoe
