// AdamW over many tensors (dgl_adamw), with states in 32 bits or in 8.
//
//   g = s grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// One launch takes hundreds of tensors: their addresses travel in the kernel's
// parameters, so a call uploads nothing and a captured one stays valid.  The
// tensors are cut into chunks of 2048 elements, of which a block takes a few, 8
// neighbouring elements a thread.  Every element is read and written once: the
// kernel is bound by HBM (28 bytes an element with fp32 weights, gradients and
// states, 14 with 8-bit states and bf16 gradients), and with 8-bit states nearly as
// much by its arithmetic.
//
// 8-bit states.  A block of 128 elements of a tensor has a power of two as its
// scale, so that scaling is exact; m is stored in E4M3 and v in E5M2 (its square
// root, which the update divides by, has then E4M3's relative step, and the 31
// binades of v reach 15 of the root).  A step changes v by a thousandth where
// neighbouring codes are an eighth to a quarter apart: rounded to nearest, v would
// stay where its first few steps left it while 1 - b2^t grows, and updates would
// become many times too large.  Values are therefore rounded up or down at random,
// in proportion, which keeps the averages' expectations.  The random bits are
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
constexpr int kEach = 8;  // neighbouring elements that a thread takes
constexpr int kThreads = 256;
constexpr int kChunk = kEach * kThreads;
// With 8-bit states the arithmetic bounds the kernel and its latency asks for
// warps: five blocks an SM, at 48 registers (304 M elements: 793 us; four blocks
// 821, three with the loads of two chunks under way 809).
template <bool EIGHT>
constexpr int kBlocksPerSm = EIGHT ? 5 : 4;
// Chunks that a block takes, where there are enough for many blocks: blocks that
// end and make room spread the work better over SMs of unequal speed than ones that
// stay (304 M elements, 32 bits: 1418 us with a resident grid, 1318 so), but each
// begins with what its elements share.
template <bool EIGHT>
constexpr uint32_t kBlockChunks = EIGHT ? 32 : 8;

enum : int {
  PARAM_F32 = 1,
  GRAD_F32 = 2,
  MASTER = 4,
  ANY_TYPES = 8,
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
  int types;
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
// small table, whose parameters are quicker to hand over (a step of 49 tensors from
// Python 10.4 us with the large one, 9.1 so; of 6 5.7 either with 40 places or 120).
constexpr int kFewTensors = 120, kManyTensors = 336;

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
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 add_apart(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// Eight elements on their way: fp32 in eight words, bf16 in four.
struct Eight {
  uint32_t w[kEach];
};

// Eight elements from element e of p on: as units, or one by one as far as they
// exist (0 past them).
__device__ __forceinline__ void load8(const void* p, int64_t e, bool f32, Eight& x) {
  if (f32) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]), "=r"(x.w[6]),
                   "=r"(x.w[7])
                 : "l"(static_cast<const float*>(p) + e));
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e);
    x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
  }
}
__device__ __forceinline__ void load8_guarded(const void* p, int64_t e, bool f32, int have, Eight& x) {
#pragma unroll
  for (int i = 0; i < kEach; ++i) x.w[i] = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (i >= have) continue;
    if (f32) x.w[i] = static_cast<const uint32_t*>(p)[e + i];
    else x.w[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[e + i]) << (16 * (i % 2));
  }
}
__device__ __forceinline__ uint2 load8_guarded(const uint8_t* p, int have) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (i < have) w[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
  return make_uint2(w[0], w[1]);
}
// (elements are in pairs, for the packed fp32 instructions)
__device__ __forceinline__ void values(const Eight& x, bool f32, float2 (&f)[kEach / 2]) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < kEach / 2; ++i) f[i] = make_float2(__uint_as_float(x.w[2 * i]), __uint_as_float(x.w[2 * i + 1]));
  } else {
#pragma unroll
    for (int i = 0; i < kEach / 2; ++i)
      f[i] = make_float2(__uint_as_float(x.w[i] << 16), __uint_as_float(x.w[i] & 0xffff0000u));
  }
}
__device__ __forceinline__ void store8(void* p, int64_t e, bool f32, const float2 (&f)[kEach / 2]) {
  if (f32) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(static_cast<float*>(p) + e), "f"(f[0].x),
                 "f"(f[0].y), "f"(f[1].x), "f"(f[1].y), "f"(f[2].x), "f"(f[2].y), "f"(f[3].x), "f"(f[3].y)
                 : "memory");
  } else {
    __nv_bfloat162 two[kEach / 2];
#pragma unroll
    for (int i = 0; i < kEach / 2; ++i) two[i] = __floats2bfloat162_rn(f[i].x, f[i].y);
    *reinterpret_cast<uint4*>(static_cast<bf16*>(p) + e) = *reinterpret_cast<uint4*>(two);
  }
}
__device__ __forceinline__ void store8_guarded(void* p, int64_t e, bool f32, int have, const float2 (&f)[kEach / 2]) {
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const float v = i % 2 ? f[i / 2].y : f[i / 2].x;
    if (i >= have) continue;
    if (f32) static_cast<float*>(p)[e + i] = v;
    else static_cast<bf16*>(p)[e + i] = __float2bfloat16_rn(v);
  }
}
__device__ __forceinline__ void store8_guarded(uint8_t* p, int have, uint2 c) {
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (i < have) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i % 4)));
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
// in the last place.  They take subnormal numbers for zero: a v below 2^-126,
// which adds less than 2^-63 root, is nothing beside an eps past 2^-39 root (1.8e-12
// for a root of 1, 5.8e-11 on the first step where beta2 is 0.999); with a smaller
// one the root and the quotient are taken in full.
__device__ __forceinline__ float quotient(float m, float v, float root, float eps) {
  float r, q;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(fmaf(r, root, eps)));
  return m * q;
}

// TYPES: the tensors' PARAM_F32, GRAD_F32 and MASTER, which are the same for all of
// a launch and whose addresses all allow units of 8 elements; or ANY_TYPES: each
// its own.
template <bool EIGHT, int TYPES, int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<EIGHT>) adamw_kernel(const __grid_constant__ AdamTable<CAP> a) {
  griddep_wait();
  griddep_launch_dependents();
  const AdamScalars& s = a.s;
  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t) (By each thread: by one for its block the
  // others waited longer than this takes, 816 -> 934 us.)
  const int64_t steps = *s.steps + 1;
  const float grad_scale = s.grad_scale ? *s.grad_scale : 1.0f;
  const float lr = s.lr_at ? *s.lr_at : s.lr;
  const float size = lr / -expm1f(static_cast<float>(static_cast<double>(steps) * s.log_beta1));
  const float root = rsqrtf(-expm1f(static_cast<float>(static_cast<double>(steps) * s.log_beta2)));
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
    constexpr bool kAny = TYPES == ANY_TYPES;
    const int types = kAny ? t.types : TYPES;
    const int64_t e = static_cast<int64_t>(chunk - t.first_chunk) * kChunk + threadIdx.x * kEach;
    void* const param = t.p;
    float* const master = t.master;
    const bool param_f32 = types & PARAM_F32, grad_f32 = types & GRAD_F32, mastered = types & MASTER;
    const int have = static_cast<int>(min(max(t.n - e, int64_t(0)), int64_t(kEach)));
    const bool whole = !kAny && have == kEach;
    Eight in_p, in_g, in_m, in_v;  // (of 8-bit states the first two words)
    if (whole) {
      load8(t.g, e, grad_f32, in_g);
      load8(mastered ? master : param, e, mastered || param_f32, in_p);
      if constexpr (EIGHT) {
        const uint2 cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + e);
        const uint2 cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + e);
        in_m.w[0] = cm.x, in_m.w[1] = cm.y, in_v.w[0] = cv.x, in_v.w[1] = cv.y;
      } else {
        load8(t.m, e, true, in_m);
        load8(t.v, e, true, in_v);
      }
    } else {
      load8_guarded(t.g, e, grad_f32, have, in_g);
      load8_guarded(mastered ? master : param, e, mastered || param_f32, have, in_p);
      if constexpr (EIGHT) {
        const uint2 cm = load8_guarded(static_cast<const uint8_t*>(t.m) + e, have);
        const uint2 cv = load8_guarded(static_cast<const uint8_t*>(t.v) + e, have);
        in_m.w[0] = cm.x, in_m.w[1] = cm.y, in_v.w[0] = cv.x, in_v.w[1] = cv.y;
      } else {
        load8_guarded(t.m, e, true, have, in_m);
        load8_guarded(t.v, e, true, have, in_v);
      }
    }
    float2 p[kEach / 2], g[kEach / 2], m[kEach / 2], v[kEach / 2];
    if constexpr (EIGHT) {
      const float m_scale = have > 0 ? t.m_scale[e / kBlock] : 0.0f, v_scale = have > 0 ? t.v_scale[e / kBlock] : 0.0f;
      decode8<true>(make_uint2(in_m.w[0], in_m.w[1]), m_scale, m);
      decode8<false>(make_uint2(in_v.w[0], in_v.w[1]), v_scale, v);
    } else {
      values(in_m, true, m);
      values(in_v, true, v);
    }
    values(in_g, grad_f32, g);
    values(in_p, mastered || param_f32, p);
    const float fade = -lr * t.decay;
#pragma unroll
    for (int i = 0; i < kEach / 2; ++i) {
      g[i] = mul2(g[i], both(grad_scale));
      m[i] = add_apart(mul2(both(s.beta1), m[i]), mul2(both(s.rest1), g[i]));
      v[i] = add_apart(mul2(both(s.beta2), v[i]), mul2(both(s.rest2), mul2(g[i], g[i])));
    }
    if (s.eps > 0x1p-39f * root) {
#pragma unroll
      for (int i = 0; i < kEach / 2; ++i) {
        const float2 u = make_float2(quotient(m[i].x, v[i].x, root, s.eps), quotient(m[i].y, v[i].y, root, s.eps));
        p[i] = fma2(both(-size), u, fma2(both(fade), p[i], p[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEach / 2; ++i) {
        const float2 u = make_float2(m[i].x / fmaf(sqrtf(v[i].x), root, s.eps), m[i].y / fmaf(sqrtf(v[i].y), root, s.eps));
        p[i] = fma2(both(-size), u, fma2(both(fade), p[i], p[i]));
      }
    }
    if (whole) {
      if (mastered) store8(master, e, true, p);
      store8(param, e, param_f32, p);
    } else {
      if (mastered) store8_guarded(master, e, true, have, p);
      store8_guarded(param, e, param_f32, have, p);
    }
    if constexpr (EIGHT) {
      uint32_t random[kEach];
      uint64_t x = key + static_cast<uint64_t>(t.first_block * kBlock + e) / 2 * kGolden;
#pragma unroll
      for (int i = 0; i < kEach; i += 2) {
        x += kGolden;
        const uint64_t z = split_mix(x);
        random[i] = static_cast<uint32_t>(z);
        random[i + 1] = static_cast<uint32_t>(z >> 32);
      }
      float m_scale, v_scale;
      const uint2 cm = encode8<true>(m, random, m_scale);
      const uint2 cv = encode8<false>(v, random, v_scale);
      if (threadIdx.x % (kBlock / kEach) == 0 && have > 0) {
        t.m_scale[e / kBlock] = m_scale;
        t.v_scale[e / kBlock] = v_scale;
      }
      if (whole) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + e) = cm;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + e) = cv;
      } else {
        store8_guarded(static_cast<uint8_t*>(t.m) + e, have, cm);
        store8_guarded(static_cast<uint8_t*>(t.v) + e, have, cv);
      }
    } else if (whole) {
      store8(t.m, e, true, m);
      store8(t.v, e, true, v);
    } else {
      store8_guarded(t.m, e, true, have, m);
      store8_guarded(t.v, e, true, have, v);
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

// A tensor's types, if every address allows units of eight elements: 32 bytes of
// fp32, 16 of bf16, 8 of 8-bit states.
int types_of(const dgl_adamw_tensor& t) {
  return (t.param_dtype == DGL_OUT_F32 ? PARAM_F32 : 0) | (t.grad_dtype == DGL_OUT_F32 ? GRAD_F32 : 0) |
         (t.master ? MASTER : 0);
}
bool takes_units(const dgl_adamw_tensor& t, int bits) {
  const uintptr_t state = bits == 8 ? 8 : 32;
  return aligned(t.param, t.param_dtype == DGL_OUT_F32 ? 32 : 16) && aligned(t.grad, t.grad_dtype == DGL_OUT_F32 ? 32 : 16) &&
         aligned(t.master, 32) && aligned(t.exp_avg, state) && aligned(t.exp_avg_sq, state);
}

template <bool EIGHT, int TYPES, int CAP>
dgl_status launch(const AdamScalars& s, const AdamTensor* t, int num_sms, cudaStream_t stream) {
  AdamTable<CAP> a;
  a.s = s;
  std::copy(t, t + s.count, a.t);
  const uint32_t resident = static_cast<uint32_t>(num_sms * kBlocksPerSm<EIGHT>);
  const unsigned grid = std::max(1u, std::min(s.chunks, std::max(resident, s.chunks / kBlockChunks<EIGHT>)));
  const cudaError_t e = launch_dependent(adamw_kernel<EIGHT, TYPES, CAP>, grid, kThreads, stream, a);
  return e == cudaSuccess ? DGL_OK : DGL_ERR_CUDA;
}

template <bool EIGHT, int TYPES>
dgl_status launch(const AdamScalars& s, const AdamTensor* t, int num_sms, cudaStream_t stream) {
  return s.count <= kFewTensors ? launch<EIGHT, TYPES, kFewTensors>(s, t, num_sms, stream)
                                : launch<EIGHT, TYPES, kManyTensors>(s, t, num_sms, stream);
}

template <bool EIGHT>
dgl_status launch(int types, const AdamScalars& s, const AdamTensor* t, int num_sms, cudaStream_t stream) {
  switch (types) {
    case 0: return launch<EIGHT, 0>(s, t, num_sms, stream);
    case PARAM_F32: return launch<EIGHT, PARAM_F32>(s, t, num_sms, stream);
    case GRAD_F32: return launch<EIGHT, GRAD_F32>(s, t, num_sms, stream);
    case PARAM_F32 | GRAD_F32: return launch<EIGHT, PARAM_F32 | GRAD_F32>(s, t, num_sms, stream);
    case MASTER: return launch<EIGHT, MASTER>(s, t, num_sms, stream);
    case MASTER | GRAD_F32: return launch<EIGHT, MASTER | GRAD_F32>(s, t, num_sms, stream);
    default: return launch<EIGHT, ANY_TYPES>(s, t, num_sms, stream);
  }
}

dgl_status run_adamw(const dgl_adamw_desc& d, const dgl_adamw_tensor* tensors, int count, cudaStream_t stream) {
  if (count < 0 || (count > 0 && !tensors) || !d.steps || !d.ticket) return DGL_ERR_ARG;
  if (d.state_bits != 8 && d.state_bits != 32) return DGL_ERR_ARG;
  for (double beta : {d.beta1, d.beta2})
    if (!(beta >= 0.0 && beta < 1.0)) return DGL_ERR_ARG;
  if (!std::isfinite(d.lr) || !(d.eps >= 0.0) || !std::isfinite(d.eps)) return DGL_ERR_ARG;
  if (!aligned(d.steps, 8) || !aligned(d.ticket, 4) || !aligned(d.grad_scale, 4) || !aligned(d.lr_at, 4))
    return DGL_ERR_ALIGN;
  uint32_t kinds = 0;  // of tensors that there are: bit `types`, or ANY_TYPES where units do not fit
  for (int i = 0; i < count; ++i) {
    const dgl_status st = check_tensor(tensors[i], d.state_bits);
    if (st != DGL_OK) return st;
    if (tensors[i].n > 0) kinds |= 1u << (takes_units(tensors[i], d.state_bits) ? types_of(tensors[i]) : ANY_TYPES);
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
  const bool eight = d.state_bits == 8;
  AdamTensor table[kManyTensors];
  if (kinds == 0) kinds = 1u << ANY_TYPES;  // nothing but a step to count
  // a launch for each kind, and for each table full; the last counts the step
  for (int types = 0; kinds != 0 && st == DGL_OK; ++types) {
    if (!(kinds >> types & 1)) continue;
    kinds &= ~(1u << types);
    int64_t block = 0, chunk = 0;
    s.count = 0;
    auto flush = [&](bool last) {
      s.chunks = static_cast<uint32_t>(chunk);
      s.ticket = last ? d.ticket : nullptr;
      st = eight ? launch<true>(types, s, table, ds->num_sms, stream) : launch<false>(types, s, table, ds->num_sms, stream);
      s.count = 0;
      chunk = 0;
    };
    for (int i = 0; i < count && st == DGL_OK; ++i) {
      const dgl_adamw_tensor& t = tensors[i];
      const int64_t first = block, chunks = (t.n + kChunk - 1) / kChunk;
      block += (t.n + kBlock - 1) / kBlock;
      if (t.n == 0 || (takes_units(t, d.state_bits) ? types_of(t) : ANY_TYPES) != types) continue;
      // (a tensor's 2^40 elements are 2^29 chunks)
      if (s.count == kManyTensors || chunk + chunks > UINT32_MAX / 2) flush(false);
      table[s.count++] =
          AdamTensor{t.param,          t.grad, t.master, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale, t.n,
                     first, static_cast<uint32_t>(chunk), types_of(t), t.weight_decay};
      chunk += chunks;
    }
    if (st == DGL_OK) flush(kinds == 0);
  }
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
