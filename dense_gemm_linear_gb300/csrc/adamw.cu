// AdamW over many tensors (dgl_adamw), with states in 32 bits or in 8.
//
//   g = s grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// One launch takes hundreds of tensors: their addresses travel in the kernel's
// parameters, so a call uploads nothing and a captured one stays valid.  The
// tensors are cut into chunks of 2048 elements that a persistent grid walks in
// order, 8 neighbouring elements a thread.  Every element is read and written
// once: the kernel is bound by HBM (28 bytes an element with fp32 weights,
// gradients and states, 14 with 8-bit states and bf16 gradients), and with 8-bit states nearly as
// much by its arithmetic.
//
// 8-bit states.  A block of 128 elements of a tensor has a power of two as its
// scale, so that scaling is exact; m is stored in E4M3 and v in E5M2 (its square
// root, which the update divides by, has then E4M3's relative step, and the
// 31 binades of v reach 15 of the root).  A step changes v by a thousandth
// where neighbouring codes are an eighth to a quarter apart: rounded to nearest, v would
// stay where its first few steps left it while 1 - b2^t grows, and updates
// would become many times too large.  Values are therefore rounded up or down
// at random, in proportion, which keeps the averages' expectations.  The random bits are
// SplitMix64's (Steele, Lea and Flood 2014) of seed, step and element.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dgl.h"
#include "elem.cuh"
#include "host.h"
#include "launch.h"
#include "ptx.cuh"

namespace dgl {

namespace {

using bf16 = __nv_bfloat16;

constexpr int kBlock = DGL_ADAMW_BLOCK;  // elements of an 8-bit state that share a scale
constexpr int kEach = 8;                 // elements a thread takes of a chunk
constexpr int kThreads = 256;
constexpr int kChunk = kEach * kThreads;
constexpr int kBlocksPerSm = 4;

enum : uint32_t {
  PARAM_F32 = 1,
  GRAD_F32 = 2,
  UNITS_32 = 4,  // every address allows units of 8 elements: 32 bytes of fp32, 16 of bf16, 8 of 8-bit states
  UNITS_16 = 8,  // units of at most 16 bytes
};

struct AdamTensor {
  void* p;
  const void* g;
  float* master;  // null: the parameter is its own
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  int64_t first_block;   // blocks of 128 in the call's tensors before this one
  uint32_t first_chunk;  // chunks in the launch's tensors before this one
  uint32_t kind;
  float decay;
};

struct AdamScalars {
  int64_t* steps;
  uint32_t* ticket;  // null: a further launch follows, which counts the step
  const float* grad_scale;
  const float* lr_at;
  double log_beta1, log_beta2;
  float lr, beta1, rest1, beta2, rest2, eps;  // rest: 1 - beta
  uint64_t seed;
  uint32_t chunks;
  int count;
};

// Room in a launch's parameters (at most 32764 bytes); few tensors take the
// small table, whose parameters are quicker to hand over.
constexpr int kFewTensors = 40, kManyTensors = 336;

template <int CAP>
struct AdamTable {
  AdamScalars s;
  AdamTensor t[CAP];
};
static_assert(sizeof(AdamTable<kManyTensors>) <= 32764, "kernel parameters");

// SplitMix64's increment and output function.
constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;
__device__ __forceinline__ uint64_t split_mix(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Products in pairs, and their sum one by one: fused into one rounding, as packed
// additions were, they would not give the bits that an 8-bit state depends on.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add_apart(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// Eight elements from p on, as far as they exist; 0 past them.  (Elements are in
// pairs, for the packed fp32 instructions.)
__device__ __forceinline__ void load8(const float* p, int have, uint32_t kind, float2 (&pairs)[kEach / 2]) {
  float(&f)[kEach] = reinterpret_cast<float(&)[kEach]>(pairs);
  if (have == kEach && (kind & UNITS_32)) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "l"(p));
  } else if (have == kEach && (kind & UNITS_16)) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) f[i] = i < have ? p[i] : 0.0f;
  }
}
__device__ __forceinline__ void load8(const bf16* p, int have, uint32_t kind, float2 (&pairs)[kEach / 2]) {
  float(&f)[kEach] = reinterpret_cast<float(&)[kEach]>(pairs);
  if (have == kEach && (kind & (UNITS_32 | UNITS_16))) {
    unpack<bf16, kEach>(load_unit<bf16, kEach>(p), f);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) f[i] = i < have ? __bfloat162float(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ uint2 load8(const uint8_t* p, int have, uint32_t kind) {
  if (have == kEach && (kind & (UNITS_32 | UNITS_16))) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (i < have) w[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store8(float* p, int have, uint32_t kind, const float2 (&pairs)[kEach / 2]) {
  const float(&f)[kEach] = reinterpret_cast<const float(&)[kEach]>(pairs);
  if (have == kEach && (kind & UNITS_32)) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                 "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
  } else if (have == kEach && (kind & UNITS_16)) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < have) p[i] = f[i];
  }
}
__device__ __forceinline__ void store8(bf16* p, int have, uint32_t kind, const float2 (&pairs)[kEach / 2]) {
  const float(&f)[kEach] = reinterpret_cast<const float(&)[kEach]>(pairs);
  if (have == kEach && (kind & (UNITS_32 | UNITS_16))) {
    store_unit<bf16, kEach>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < have) p[i] = __float2bfloat16_rn(f[i]);
  }
}
__device__ __forceinline__ void store8(uint8_t* p, int have, uint32_t kind, uint2 c) {
  if (have == kEach && (kind & (UNITS_32 | UNITS_16))) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < have) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i % 4)));
  }
}

// The values of eight E4M3 or E5M2 codes (E5M2 is the upper half of an fp16).
template <bool E4M3>
__device__ __forceinline__ void decode8(uint2 c, float scale, float2 (&f)[kEach / 2]) {
#pragma unroll
  for (int i = 0; i < kEach / 2; ++i) {
    const uint32_t word = i < 2 ? c.x : c.y;
    float2 v;
    if constexpr (E4M3) {
      const uint32_t two = i % 2 ? word >> 16 : word & 0xffffu;
      v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3)));
    } else {
      const uint32_t two = __byte_perm(word, 0, i % 2 ? 0x3424 : 0x1404);
      v = __half22float2(*reinterpret_cast<const __half2*>(&two));
    }
    f[i] = mul2(v, both(scale));
  }
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The upper bytes of four words.
__device__ __forceinline__ uint32_t upper_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Codes of eight values and their block's scale.  The block's largest finite
// magnitude (16 neighbouring threads) lands in [2^TOP, 2^(TOP + 1)).  Taken
// down by the difference of the formats' exponent biases, an fp32's exponent
// and leading fraction bits are the code, subnormal ones too (fp32's
// subnormals begin where the format's do): a random number below the
// last of them carries into the code as often as the rest of the fraction asks.
// A v above zero never becomes zero, which the update divides by; what is not
// finite becomes NaN, in a pass of its own that blocks without such a value
// need not pay for.
template <bool E4M3>
__device__ __forceinline__ uint2 encode8(const float2 (&f)[kEach / 2], const uint32_t (&random)[kEach], float& scale) {
  constexpr int kTop = E4M3 ? 7 : 14, kShift = E4M3 ? 20 : 21;
  float x[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) x[i] = i % 2 ? f[i / 2].y : f[i / 2].x;
  float top = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < kEach; ++i) top = max_or_nan(top, fabsf(x[i]));
#pragma unroll
  for (int o = 1; o < kBlock / kEach; o *= 2) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool finite = top < INFINITY;  // the same in all threads of the block
  if (__any_sync(0xffffffffu, !finite)) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) most = fmaxf(most, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.0f);
#pragma unroll
    for (int o = 1; o < kBlock / kEach; o *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    top = most;
  }
  // the scale and its reciprocal are normal numbers
  const uint32_t exponent = max(__float_as_uint(top) >> 23, 16u);
  scale = __uint_as_float((exponent - kTop) << 23);
  // 2^TOP over the largest's power of two, times 2^-120 or 2^-112: one factor
  // where that is a normal number, else two
  constexpr uint32_t kDown = E4M3 ? 120 : 112;
  const bool one = exponent + kDown < 254 + kTop;
  const float up = __uint_as_float((254 + kTop - exponent - (one ? kDown : 0)) << 23);
  const float down = one ? 1.0f : __uint_as_float((127 - kDown) << 23);
  uint32_t code[kEach];  // in the upper byte
  auto round = [&](int i, float scaled) {
    const uint32_t r = E4M3 ? (random[i] << 4 & 0xffff0u) | 8u : (random[i] >> 11 & 0x1fffe0u) | 16u;
    code[i] = __float_as_uint(scaled) + r;
    if constexpr (!E4M3) code[i] = max(code[i], x[i] > 0.0f ? 1u << kShift : 0u);
    code[i] <<= 24 - kShift;
  };
  if (__all_sync(0xffffffffu, one)) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) round(i, __fmul_rn(fabsf(x[i]), up));
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) round(i, __fmul_rn(__fmul_rn(fabsf(x[i]), up), down));
  }
  if (!finite) {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (!(fabsf(x[i]) < INFINITY)) code[i] = 0x7f000000u;
  }
  uint2 c = make_uint2(upper_bytes(code[0], code[1], code[2], code[3]), upper_bytes(code[4], code[5], code[6], code[7]));
  if constexpr (E4M3) {
    c.x |= 0x80808080u & upper_bytes(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    c.y |= 0x80808080u & upper_bytes(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
  }
  return c;
}

// m / (sqrt(v) root + eps) by the hardware's approximations, off by a few units
// in the last place.  They take subnormal numbers for zero: a v below 2^-126
// is nothing beside an eps past 1e-18; without one its root is taken in full.
__device__ __forceinline__ float quotient(float m, float v, float root, float eps) {
  float r, q;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(fmaf(r, root, eps)));
  return m * q;
}

template <bool EIGHT, int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) adamw_kernel(const __grid_constant__ AdamTable<CAP> a) {
  griddep_wait();
  griddep_launch_dependents();
  const AdamScalars& s = a.s;
  const int64_t steps = *s.steps + 1;
  const float grad_scale = s.grad_scale ? *s.grad_scale : 1.0f;
  const float lr = s.lr_at ? *s.lr_at : s.lr;
  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  const float size = lr / -expm1f(static_cast<float>(static_cast<double>(steps) * s.log_beta1));
  const float root = 1.0f / sqrtf(-expm1f(static_cast<float>(static_cast<double>(steps) * s.log_beta2)));
  const uint64_t key = EIGHT ? split_mix(s.seed + static_cast<uint64_t>(steps) * kGolden) : 0;

  // a range of chunks, and the tensor that its first lies in
  const uint32_t begin = static_cast<uint32_t>(static_cast<uint64_t>(s.chunks) * blockIdx.x / gridDim.x);
  const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(s.chunks) * (blockIdx.x + 1) / gridDim.x);
  int at = 0;
  for (int step = CAP; step > 0; step /= 2)
    while (at + step < s.count && a.t[at + step].first_chunk <= begin) at += step;
  for (uint32_t chunk = begin; chunk < end; ++chunk) {
    while (at + 1 < s.count && a.t[at + 1].first_chunk <= chunk) ++at;
    const AdamTensor& t = a.t[at];
    const uint32_t kind = t.kind;
    const int64_t e = static_cast<int64_t>(chunk - t.first_chunk) * kChunk + threadIdx.x * kEach;
    const int have = static_cast<int>(min(max(t.n - e, int64_t(0)), int64_t(kEach)));
    float2 p[kEach / 2], g[kEach / 2], m[kEach / 2], v[kEach / 2];
    if (kind & GRAD_F32) load8(static_cast<const float*>(t.g) + e, have, kind, g);
    else load8(static_cast<const bf16*>(t.g) + e, have, kind, g);
    if (t.master) load8(t.master + e, have, kind, p);
    else if (kind & PARAM_F32) load8(static_cast<const float*>(t.p) + e, have, kind, p);
    else load8(static_cast<const bf16*>(t.p) + e, have, kind, p);
    if constexpr (EIGHT) {
      const uint2 cm = load8(static_cast<const uint8_t*>(t.m) + e, have, kind);
      const uint2 cv = load8(static_cast<const uint8_t*>(t.v) + e, have, kind);
      const float ms = have > 0 ? t.m_scale[e / kBlock] : 0.0f, vs = have > 0 ? t.v_scale[e / kBlock] : 0.0f;
      decode8<true>(cm, ms, m);
      decode8<false>(cv, vs, v);
    } else {
      load8(static_cast<const float*>(t.m) + e, have, kind, m);
      load8(static_cast<const float*>(t.v) + e, have, kind, v);
    }
    const float fade = -lr * t.decay;
#pragma unroll
    for (int i = 0; i < kEach / 2; ++i) {
      g[i] = mul2(g[i], both(grad_scale));
      m[i] = add_apart(mul2(both(s.beta1), m[i]), mul2(both(s.rest1), g[i]));
      v[i] = add_apart(mul2(both(s.beta2), v[i]), mul2(both(s.rest2), mul2(g[i], g[i])));
    }
    if (s.eps > 1e-18f) {
#pragma unroll
      for (int i = 0; i < kEach / 2; ++i) {
        const float2 u = make_float2(quotient(m[i].x, v[i].x, root, s.eps), quotient(m[i].y, v[i].y, root, s.eps));
        p[i] = __ffma2_rn(both(-size), u, __ffma2_rn(both(fade), p[i], p[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEach / 2; ++i) {
        const float2 u = make_float2(m[i].x / fmaf(sqrtf(v[i].x), root, s.eps), m[i].y / fmaf(sqrtf(v[i].y), root, s.eps));
        p[i] = __ffma2_rn(both(-size), u, __ffma2_rn(both(fade), p[i], p[i]));
      }
    }
    if (t.master) store8(t.master + e, have, kind, p);
    if (kind & PARAM_F32) store8(static_cast<float*>(t.p) + e, have, kind, p);
    else store8(static_cast<bf16*>(t.p) + e, have, kind, p);
    if constexpr (EIGHT) {
      uint32_t random[kEach];
      uint64_t x = key + static_cast<uint64_t>((t.first_block * kBlock + e) / 2) * kGolden;
#pragma unroll
      for (int i = 0; i < kEach; i += 2) {
        x += kGolden;
        const uint64_t z = split_mix(x);
        random[i] = static_cast<uint32_t>(z);
        random[i + 1] = static_cast<uint32_t>(z >> 32);
      }
      float scale;
      const uint2 cm = encode8<true>(m, random, scale);
      const bool leads = threadIdx.x % (kBlock / kEach) == 0 && have > 0;
      if (leads) t.m_scale[e / kBlock] = scale;
      store8(static_cast<uint8_t*>(t.m) + e, have, kind, cm);
      const uint2 cv = encode8<false>(v, random, scale);
      if (leads) t.v_scale[e / kBlock] = scale;
      store8(static_cast<uint8_t*>(t.v) + e, have, kind, cv);
    } else {
      store8(static_cast<float*>(t.m) + e, have, kind, m);
      store8(static_cast<float*>(t.v) + e, have, kind, v);
    }
  }
  // the last block counts the step: every block has read it by then.  The
  // ticket wraps to zero by itself
  if (!s.ticket) return;
  __syncthreads();
  if (threadIdx.x == 0 && atomicInc(s.ticket, gridDim.x - 1) == gridDim.x - 1) *s.steps = steps;
}

dgl_status check_tensor(const dgl_adamw_tensor& t, int bits) {
  if (t.n < 0 || (t.param_dtype != DGL_OUT_BF16 && t.param_dtype != DGL_OUT_F32) ||
      (t.grad_dtype != DGL_OUT_BF16 && t.grad_dtype != DGL_OUT_F32))
    return DGL_ERR_ARG;
  if (t.n > (int64_t(1) << 40)) return DGL_ERR_SHAPE;
  if (!std::isfinite(t.weight_decay) || t.weight_decay < 0.0f) return DGL_ERR_ARG;
  if (t.n == 0) return DGL_OK;
  if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return DGL_ERR_ARG;
  if (t.master && t.param_dtype != DGL_OUT_BF16) return DGL_ERR_ARG;
  if (bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) return DGL_ERR_ARG;
  const uintptr_t state = bits == 8 ? 1 : 4;
  if (!aligned(t.param, t.param_dtype == DGL_OUT_F32 ? 4 : 2) || !aligned(t.grad, t.grad_dtype == DGL_OUT_F32 ? 4 : 2) ||
      !aligned(t.master, 4) || !aligned(t.exp_avg, state) || !aligned(t.exp_avg_sq, state))
    return DGL_ERR_ALIGN;
  if (bits == 8 && (!aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4))) return DGL_ERR_ALIGN;
  return DGL_OK;
}

// Whether every address of a tensor allows units of eight elements, of up to `most` bytes.
bool takes_units(const dgl_adamw_tensor& t, int bits, uintptr_t most) {
  const uintptr_t f32 = most, state = bits == 8 ? 8 : f32;
  return aligned(t.param, t.param_dtype == DGL_OUT_F32 ? f32 : 16) && aligned(t.grad, t.grad_dtype == DGL_OUT_F32 ? f32 : 16) &&
         aligned(t.master, f32) && aligned(t.exp_avg, state) && aligned(t.exp_avg_sq, state);
}

template <int CAP>
dgl_status launch(const AdamScalars& s, const AdamTensor* t, int bits, int num_sms, cudaStream_t stream) {
  AdamTable<CAP> a;
  a.s = s;
  std::copy(t, t + s.count, a.t);
  const unsigned grid =
      std::max(1u, std::min(s.chunks, static_cast<uint32_t>(num_sms) * static_cast<uint32_t>(kBlocksPerSm)));
  const cudaError_t e = bits == 8 ? launch_dependent(adamw_kernel<true, CAP>, grid, kThreads, stream, a)
                                  : launch_dependent(adamw_kernel<false, CAP>, grid, kThreads, stream, a);
  return e == cudaSuccess ? DGL_OK : DGL_ERR_CUDA;
}

dgl_status run_adamw(const dgl_adamw_desc& d, const dgl_adamw_tensor* tensors, int count, cudaStream_t stream) {
  if (count < 0 || (count > 0 && !tensors) || !d.steps || !d.ticket) return DGL_ERR_ARG;
  if (d.state_bits != 8 && d.state_bits != 32) return DGL_ERR_ARG;
  for (double beta : {d.beta1, d.beta2})
    if (!(beta >= 0.0 && beta < 1.0)) return DGL_ERR_ARG;
  if (!std::isfinite(d.lr) || !(d.eps >= 0.0) || !std::isfinite(d.eps)) return DGL_ERR_ARG;
  if (!aligned(d.steps, 8) || !aligned(d.ticket, 4) || !aligned(d.grad_scale, 4) || !aligned(d.lr_at, 4))
    return DGL_ERR_ALIGN;
  for (int i = 0; i < count; ++i) {
    const dgl_status st = check_tensor(tensors[i], d.state_bits);
    if (st != DGL_OK) return st;
  }
  int dev = 0;
  DeviceState* ds = nullptr;
  dgl_status st = get_device(&dev, &ds);
  if (st != DGL_OK) return st;

  AdamScalars s = {};
  s.steps = d.steps;
  s.grad_scale = d.grad_scale;
  s.lr_at = d.lr_at;
  s.log_beta1 = std::log(d.beta1);
  s.log_beta2 = std::log(d.beta2);
  s.lr = static_cast<float>(d.lr);
  s.beta1 = static_cast<float>(d.beta1);
  s.rest1 = static_cast<float>(1.0 - d.beta1);
  s.beta2 = static_cast<float>(d.beta2);
  s.rest2 = static_cast<float>(1.0 - d.beta2);
  s.eps = static_cast<float>(d.eps);
  s.seed = d.seed;
  AdamTensor table[kManyTensors];
  int64_t block = 0;
  int i = 0;
  do {
    int64_t chunk = 0;
    s.count = 0;
    for (; i < count && s.count < kManyTensors; ++i) {
      const dgl_adamw_tensor& t = tensors[i];
      const int64_t chunks = (t.n + kChunk - 1) / kChunk;
      if (chunk + chunks > UINT32_MAX / 2) break;  // (2^40 elements are 2^29 chunks: the first always fits)
      if (t.n > 0)
        table[s.count++] = AdamTensor{t.param,
                                      t.grad,
                                      t.master,
                                      t.exp_avg,
                                      t.exp_avg_sq,
                                      t.exp_avg_scale,
                                      t.exp_avg_sq_scale,
                                      t.n,
                                      block,
                                      static_cast<uint32_t>(chunk),
                                      (t.param_dtype == DGL_OUT_F32 ? PARAM_F32 : 0u) |
                                          (t.grad_dtype == DGL_OUT_F32 ? GRAD_F32 : 0u) |
                                          (takes_units(t, d.state_bits, 32)   ? UNITS_32
                                           : takes_units(t, d.state_bits, 16) ? UNITS_16
                                                                              : 0u),
                                      t.weight_decay};
      chunk += chunks;
      block += (t.n + kBlock - 1) / kBlock;
    }
    s.chunks = static_cast<uint32_t>(chunk);
    s.ticket = i == count ? d.ticket : nullptr;
    st = s.count <= kFewTensors ? launch<kFewTensors>(s, table, d.state_bits, ds->num_sms, stream)
                                : launch<kManyTensors>(s, table, d.state_bits, ds->num_sms, stream);
  } while (st == DGL_OK && i < count);
  return st;
}

}  // namespace
}  // namespace dgl

using namespace dgl;

extern "C" dgl_status dgl_adamw(const dgl_adamw_desc* desc, const dgl_adamw_tensor* tensors, int32_t count,
                                void* stream) {
  if (!desc) return DGL_ERR_ARG;
  return run_adamw(*desc, tensors, count, static_cast<cudaStream_t>(stream));
}
