// Layer norm, forward and backward (dgl_layer_norm, dgl_layer_norm_grad).
//
// With h = (x - mean) rstd over the d elements of a row and u = dy w:
//   y  = h w + b
//   dx = rstd (u - mean_j u - h mean_j (u h))
//   dw = sum_rows dy h,  db = sum_rows dy
// Rows of up to 16384 elements are read once and held in registers, kElems
// elements a thread: the threads of a row (its lanes) are part of a warp, a warp,
// or a block of up to 1024.  A lane keeps the same columns from row to row, so the
// weight stays in its registers and the sums of dw and db are its own.  All sums
// and statistics are fp32; the variance is the sum of squares around the
// mean, never a difference of two large sums.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
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

constexpr int kElems = 16;                  // elements a thread holds of a row
constexpr int kWide = 1024 * kElems;        // the widest row that a block holds
constexpr int kMid = 512 * kElems;          // and with 128 registers a thread
constexpr int kSlowThreads = 512;           // a block of the kernels for wider rows
constexpr int kFewThreads = 128;            // a block whose rows take a warp or less

struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* w;
  const void* b;
  int w_f32;    // type of w and b
  int w_fits;   // they can be read in the row's units
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  const void* dy;
  int64_t lddy;
  void* dx;
  int64_t lddx;
  float* part;  // [blocks][2][d] sums of dw and db (null: not wanted)
  int64_t rows;
  int d;
  int lanes;    // lanes of a row: 1 to 32 (a power of two), or whole warps, then the block
  float eps;
};

__device__ __forceinline__ float element(const void* v, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(v)[i] : to_float(static_cast<const bf16*>(v)[i]);
}

// Sums over the lanes of a row: a power of two below 32, or a warp.
template <bool WARPS>
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (WARPS || o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over a row's warps, in every lane: lane k holds warp k's value (zero where
// there is none), and lanes 8 apart the same where there are at most eight.
constexpr int kFewWarps = 8;
__device__ __forceinline__ float warps_sum(float v, bool few) {
  if (!few) {
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
  }
#pragma unroll
  for (int o = kFewWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Two sums over a whole warp in six shuffles' steps instead of ten: the halves of
// the warp exchange what each does not go on with.  Lanes 0 to 15 return the
// first, 16 to 31 the second.
__device__ __forceinline__ float warp_sums(float a, float b) {
  const bool low = (threadIdx.x & 16) == 0;
  float v = low ? a : b;
  v += __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(v): the hardware's, off by two units in the last place, and a step of
// Newton's method.  (0 gives infinity, infinity 0.)
__device__ __forceinline__ float reciprocal_root(float v) {
  const float r = rsqrtf(v);
  const float better = fmaf(r * fmaf(-v * r, r, 1.0f), 0.5f, r);
  return r > 0.0f && r < INFINITY ? better : r;
}

// A lane's elements are in pairs, for the packed fp32 instructions.
__device__ __forceinline__ void put(float2 (&f)[kElems / 2], int i, float v) {
  if (i % 2) f[i / 2].y = v;
  else f[i / 2].x = v;
}
__device__ __forceinline__ float get(const float2 (&f)[kElems / 2], int i) { return i % 2 ? f[i / 2].y : f[i / 2].x; }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// Two fp32 operations in one instruction (a sixth fewer instructions in all).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// (x - mean) rstd, in two steps, of which the first is nearly exact.  (As x rstd -
// mean rstd, one instruction, a rounding of mean rstd remains where the row is equal
// elements or nearly so: 0.4 of 30000 with an eps of 1e-5.)
__device__ __forceinline__ float2 scaled(float2 x, float mean, float rstd) {
  return mul2(add2(x, both(-mean)), both(rstd));
}

// A lane's units of a row, on their way from memory.  Units of 4 bytes or more pass
// through shared memory: a lane copies its own units of DEPTH - 1 rows ahead
// (cp.async) and reads them back itself, so nothing synchronises, no register waits
// and far more is in flight than registers would hold.  bf16 rows off 4 bytes are
// held in registers, one row ahead.  Forward, 10240 x 2048 bf16: 23.4 us with one
// row ahead in registers, 16.4 so (17.0 with what has been added since), 18.7 with
// one bulk copy a row, whose arrival and release cost more instructions than the
// copies of 16 bytes.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void store_shared_zero(uint32_t to) {
  if constexpr (BYTES == 16)
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
  else
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(0) : "memory");
}
template <class U>
__device__ __forceinline__ U load_shared(uint32_t from) {
  U u;
  if constexpr (sizeof(U) == 16)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "r"(from)
                 : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(from) : "memory");
  return u;
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

template <class T, int VEC, bool RING>
struct RowUnits {
  static constexpr int U = kElems / VEC, kBytes = VEC * static_cast<int>(sizeof(T));
  static constexpr bool kRing = RING && kBytes >= 4;
  Unit<T, VEC> held[kRing ? 1 : U];
  const T* next;   // the lane's first unit of the row to be loaded
  int64_t step;    // elements from one of the group's rows to its next
  int apart;       // elements between the lane's units
  int count;       // units that the lane has
  uint32_t pitch;  // of a slot's units in shared memory
  uint32_t first, in, out, end;  // of the lane's slots: the first, the one to fill, the one to read, the last's end

  // ring: [depth][U][threads] units.  Units past a row's end are zeros, which no load writes.
  __device__ __forceinline__ void begin(const T* x, int64_t ld, int64_t row, int64_t stride, int lane, int lanes,
                                        int units, uint8_t* ring, int depth) {
    next = x + row * ld + lane * VEC;
    step = stride * ld;
    apart = lanes * VEC;
    count = lane < units ? (units - lane + lanes - 1) / lanes : 0;
    pitch = blockDim.x * kBytes;
    first = in = out = smem_u32(ring) + threadIdx.x * kBytes;
    end = first + depth * U * pitch;
    if constexpr (kRing) {
      if (count < U)
        for (int k = 0; k < depth; ++k) zero(first + k * U * pitch, count);
    }
  }
  __device__ __forceinline__ void zero(uint32_t slot, int from) {
    for (int i = from; i < U; ++i) store_shared_zero<kBytes>(slot + i * pitch);
  }
  // The next row; zeros where it does not exist.
  __device__ __forceinline__ void load(bool exists) {
    if constexpr (kRing) {
      if (exists) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (i < count) copy_async<kBytes>(in + i * pitch, next + i * apart);
      } else {
        zero(in, 0);
      }
      in += U * pitch;
      if (in == end) in = first;
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i)
        held[i] = exists && i < count ? load_unit_once<T, VEC>(next + i * apart) : Unit<T, VEC>{};
    }
    next += step;
  }
  __device__ __forceinline__ void get(float2 (&f)[kElems / 2]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float e[VEC];
      if constexpr (kRing) unpack<T, VEC>(load_shared<Unit<T, VEC>>(out + i * pitch), e);
      else unpack<T, VEC>(held[i], e);
#pragma unroll
      for (int j = 0; j < VEC; ++j) put(f, i * VEC + j, e[j]);
    }
    if constexpr (kRing) {
      out += U * pitch;
      if (out == end) out = first;
    }
  }
};

// Rows that a lane has under way and at hand: 160 KB of an SM's shared memory
// at the residencies below.
template <class T, int VEC>
constexpr int kDepth = VEC * sizeof(T) < 4 ? 2 : sizeof(T) == 2 ? 4 : 3;
template <class T, int VEC>
constexpr int kRingBytes = VEC * sizeof(T) < 4 ? 0 : kDepth<T, VEC> * kElems * static_cast<int>(sizeof(T));  // a thread

// The lanes of a group that is whole warps; `groups` in the block.
__device__ __forceinline__ void group_sync(int group, int lanes, int groups) {
  if (groups == 1) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
}

// The same columns of a vector (the weight or the bias); `fill` where there are
// none.  In units where its address allows: read element by element, a warp's 32
// lanes touch 32 sectors for each of 32 loads, and a grid's blocks spent half their
// time on that.
template <int VEC>
__device__ __forceinline__ void unit_columns(const void* v, int f32, int units_fit, float fill, int at,
                                             float (&e)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) e[j] = fill;
  if (!v) return;
  if (units_fit) {
    if (f32) unpack<float, VEC>(load_unit<float, VEC>(static_cast<const float*>(v) + at), e);
    else unpack<bf16, VEC>(load_unit<bf16, VEC>(static_cast<const bf16*>(v) + at), e);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) e[j] = element(v, f32, at + j);
  }
}
template <int VEC>
__device__ __forceinline__ void lane_columns(const void* v, int f32, int units_fit, float fill, int lane, int lanes,
                                             int units, float2 (&f)[kElems / 2]) {
#pragma unroll
  for (int i = 0; i < kElems / VEC; ++i) {
    const int at = lane + i * lanes;
    float e[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) e[j] = fill;
    if (at < units) unit_columns<VEC>(v, f32, units_fit, fill, at * VEC, e);
#pragma unroll
    for (int j = 0; j < VEC; ++j) put(f, i * VEC + j, e[j]);
  }
}

// Gives the elements past the lane's `count` units a value.
template <int VEC>
__device__ __forceinline__ void fill_row(float2 (&f)[kElems / 2], int count, float v) {
#pragma unroll
  for (int i = 0; i < kElems; ++i)
    if (i / VEC >= count) put(f, i, v);
}

// row: the lane's first unit.
template <class T, int VEC>
__device__ __forceinline__ void store_row(T* row, int apart, int count, const float2 (&f)[kElems / 2]) {
#pragma unroll
  for (int i = 0; i < kElems / VEC; ++i) {
    if (i >= count) continue;
    float e[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) e[j] = get(f, i * VEC + j);
    store_unit<T, VEC>(row + i * apart, e);
  }
}

// What elements are taken from before they are summed: anything that neither
// overflows nor is lost beside them.
__device__ __forceinline__ float within(float v) { return fabsf(v) < 0x1p100f ? v : 0.0f; }
__device__ __forceinline__ float finite(float v) { return fabsf(v) < INFINITY ? v : 0.0f; }

// sum / n: the quotient that is nearest, but for ties.
__device__ __forceinline__ float over(float sum, float n, float inv_n) {
  const float v = sum * inv_n;
  return fmaf(fmaf(-v, n, sum), inv_n, v);
}

// (to a few units in the last place; of a subnormal number 0)
__device__ __forceinline__ float root(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Where `far`, a row of fp32 elements by a group of lanes (WARPS: the block) from
// memory, in the steps of norm_forward_wide_kernel; the lanes of a warp enter together.
template <bool WARPS>
__device__ __noinline__ void far_row(const NormArgs& a, int64_t row, int lane, int lanes, bool far, float2* red) {
  const int in_warp = threadIdx.x & 31, end = far ? a.d : 0;
  const float d = static_cast<float>(a.d);
  const auto row_sums = [&](float u, float v) {
    if constexpr (!WARPS) return make_float2(lanes_sum<false>(u, lanes), lanes_sum<false>(v, lanes));
    const float sum = warp_sums(u, v);
    __syncthreads();
    if (in_warp == 0) red[threadIdx.x / 32].x = sum;
    if (in_warp == 16) red[threadIdx.x / 32].y = sum;
    __syncthreads();
    const float2 o = in_warp < lanes / 32 ? red[in_warp] : both(0.0f);
    return make_float2(warps_sum(o.x, false), warps_sum(o.y, false));
  };
  const float* x = static_cast<const float*>(a.x) + row * a.ldx;
  float* y = static_cast<float*>(a.y) + row * a.ldy;
  const float first = far ? within(x[0]) : 0.0f, own = lane < end ? within(x[lane]) : 0.0f;
  const float n = lane < end ? static_cast<float>((end - lane + lanes - 1) / lanes) : 0.0f;
  float t = 0.0f, s = 0.0f, q = 0.0f;
  for (int i = lane; i < end; i += lanes) t += x[i] - own;
  const float near = first + row_sums(fmaf(n, own - first, t), 0.0f).x / d;
  for (int i = lane; i < end; i += lanes) {
    const float c = x[i] - near;
    s += c;
    q = fmaf(c, c, q);
  }
  const float2 sums = row_sums(s, q);
  s = finite(sums.x);
  const float shift = s / d, rstd = reciprocal_root(fmaf(-shift, s, sums.y) / d + a.eps);
  for (int i = lane; i < end; i += lanes)
    y[i] = fmaf(((x[i] - near) - shift) * rstd, a.w ? element(a.w, a.w_f32, i) : 1.0f,
                a.b ? element(a.b, a.w_f32, i) : 0.0f);
  if (lane == 0 && far) {
    if (a.mean) a.mean[row] = near + shift;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// Forward.  A persistent grid; each group of lanes takes rows a grid's groups
// apart. THREADS: the most in a block.  1024, of rows past 8192: the weight does
// not fit beside a row in 64 registers and is read again for each row, from L1,
// which it has to itself: the next row waits in registers and not in shared memory.
// WARPS: a row has several warps, which are the block.
//
// Equal elements are their mean, and h is 0, whatever their size and rstd; elements
// far from zero beside their spread keep what they differ by.  A warp's sum of such bf16
// elements is exact or nearly so, and over() takes back what a product with 1 / n
// is rounded by.  A row of fp32 elements whose mean is past kFar times their
// standard deviation is gone over again, by what its elements are away from a lane's
// first: below, fp32's roundings of the sums move h by a few times kFar 2^-24.  (Done
// so for every row it took 13% longer where rows are off their units; 8192 x 4096 take
// 43 us, 264 where every row is far.)
constexpr float kFar = 64.0f;
template <class XT, int VEC, int THREADS, bool WARPS>
__global__ void __launch_bounds__(THREADS) norm_forward_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr bool kKeep = THREADS <= 512;
  constexpr int DEPTH = kKeep ? kDepth<XT, VEC> : 2;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2][32], red_far[sizeof(XT) == 4 ? 32 : 1];
  __shared__ uint32_t block_pending;
  const int lanes = a.lanes, lane = threadIdx.x % lanes, units = a.d / VEC;
  // (rows fit 31 bits)
  const int in_block = blockDim.x / lanes, groups = gridDim.x * in_block, nrows = static_cast<int>(a.rows);
  int row = blockIdx.x * in_block + threadIdx.x / lanes;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, in_warp = threadIdx.x & 31;
  const float d = static_cast<float>(a.d), inv_d = 1.0f / d;

  const int count = lane < units ? (units - lane + lanes - 1) / lanes : 0, apart = lanes * VEC;
  RowUnits<XT, VEC, kKeep> rows;
  rows.begin(static_cast<const XT*>(a.x), a.ldx, row, groups, lane, lanes, units, ring, DEPTH);
  int ahead = nrows - row;  // rows from the next to be loaded on, over all groups
#pragma unroll
  for (int k = 0; k < DEPTH - 1; ++k, ahead -= groups) {
    rows.load(ahead > 0);
    copy_async_commit();
  }

  // elements that the lane's warp (or smaller group) holds, and each warp of its block
  const bool full = units == lanes * (kElems / VEC);
  const float held = lanes_sum<WARPS>(static_cast<float>(count * VEC), lanes);
  const float inv_held = held > 0.0f ? 1.0f / held : 0.0f;
  const bool few = warps <= kFewWarps;
  const int other = few ? in_warp % kFewWarps : in_warp;  // the warp whose sums this lane takes up
  float2 counted = both(0.0f);  // of that warp: elements, and one over that
  if constexpr (WARPS) {
    if (in_warp == 0) red[0][warp] = make_float2(held, inv_held);
    __syncthreads();
    if (other < warps) counted = red[0][other];
    __syncthreads();
  }

  float2 w[kKeep ? kElems / 2 : 1], b[kKeep ? kElems / 2 : 1];
  if constexpr (kKeep) {
    lane_columns<VEC>(a.w, a.w_f32, a.w_fits, 1.0f, lane, lanes, units, w);
    lane_columns<VEC>(a.b, a.w_f32, a.w_fits, 0.0f, lane, lanes, units, b);
  }
  XT* y = static_cast<XT*>(a.y) + row * a.ldy + lane * VEC;
  const int64_t y_step = groups * a.ldy;
  // all lanes of a warp go round together: the rows of its groups may end apart
  const int turns = (nrows + groups - 1) / groups;
  // Rows of fp32 elements that are far wait until 32 have been looked at: with their
  // path inside the loop over rows, rows past 8192 took half as long again.
  constexpr bool kWait = sizeof(XT) == 4;
  for (int turn = 0; turn < turns;) {
    uint32_t pending = 0;  // (WARPS: the block's, in shared memory)
    if (kWait && WARPS && threadIdx.x == 0) block_pending = 0;
    const int end = kWait ? min(turns, turn + 32) : turns;
    for (; turn < end; ++turn, row += groups, y += y_step) {
      bool far = false;
      float2 f[kElems / 2];
      copy_async_wait<DEPTH - 2>();
      rows.get(f);
      rows.load(ahead > 0);
      ahead -= groups;
      copy_async_commit();
      // the warp's (or group's) mean and squares around it, then the block's
      float2 t = f[0], squares = both(0.0f);
#pragma unroll
      for (int i = 1; i < kElems / 2; ++i) t = add2(t, f[i]);
      float sum = lanes_sum<WARPS>(t.x + t.y, lanes), q, mean, centre;  // centre: what is still to be taken from f
      if constexpr (sizeof(XT) == 2) {
        const float m = over(sum, held, inv_held);
#pragma unroll
        for (int i = 0; i < kElems / 2; ++i) f[i] = add2(f[i], both(-m));
        if (!full) fill_row<VEC>(f, count, 0.0f);
#pragma unroll
        for (int i = 0; i < kElems / 2; ++i) squares = fma2(f[i], f[i], squares);
        q = lanes_sum<WARPS>(squares.x + squares.y, lanes);
        mean = m;
        if constexpr (WARPS) {
          float2* r = red[turn & 1];  // two in turn: one barrier a row
          if (in_warp == 0) r[warp] = make_float2(sum, q);
          __syncthreads();
          const float2 o = other < warps ? r[other] : both(0.0f);
          sum = warps_sum(o.x, few);
          mean = over(sum, d, inv_d);
          const float c = fmaf(-mean, counted.x, o.x);
          q = warps_sum(fmaf(c * counted.y, c, o.y), few);
        }
        centre = (mean - m) + fmaf(-mean, d, sum) * inv_d;
        if (!(fabsf(mean) < INFINITY)) mean = sum * inv_d;  // (an infinite sum's is infinite)
      } else {
        mean = sum * inv_held;
        if (full) {
#pragma unroll
          for (int i = 0; i < kElems / 2; ++i) {
            const float2 c = add2(f[i], both(-mean));
            squares = fma2(c, c, squares);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kElems / 2; ++i) {
            float2 c = add2(f[i], both(-mean));
            if (2 * i / VEC >= count) c.x = 0.0f;
            if ((2 * i + 1) / VEC >= count) c.y = 0.0f;
            squares = fma2(c, c, squares);
          }
        }
        q = lanes_sum<WARPS>(squares.x + squares.y, lanes);
        if constexpr (WARPS) {
          float2* r = red[turn & 1];
          if (in_warp == 0) r[warp] = make_float2(sum, q);
          __syncthreads();
          const float2 o = other < warps ? r[other] : both(0.0f);
          mean = warps_sum(o.x, few) * inv_d;
          const float c = fmaf(o.x, counted.y, -mean);
          q = warps_sum(fmaf(counted.x * c, c, o.y), few);
        }
        centre = mean;
        far = fabsf(mean) < INFINITY && !(fabsf(mean) <= kFar * root(q * inv_d) && q < INFINITY);
        if constexpr (!WARPS) pending |= far ? 1u << (turn & 31) : 0;
        else if (far && threadIdx.x == 0) block_pending |= 1u << (turn & 31);
      }
      const float rstd = reciprocal_root(fmaf(q, inv_d, a.eps));
      if (row >= nrows || far) continue;
      if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < kElems / 2; ++i) {
          // (what is left of bf16 elements is small: one instruction)
          const float2 h = sizeof(XT) == 2 ? fma2(f[i], both(rstd), both(-centre * rstd)) : scaled(f[i], centre, rstd);
          f[i] = fma2(h, w[i], b[i]);
        }
        store_row<XT, VEC>(y, apart, count, f);
      } else {
#pragma unroll
        for (int i = 0; i < kElems / VEC; ++i) {
          if (i >= count) continue;
          const int at = (lane + i * lanes) * VEC;
          float e[VEC], w_unit[VEC], b_unit[VEC];
          unit_columns<VEC>(a.w, a.w_f32, a.w_fits, 1.0f, at, w_unit);
          unit_columns<VEC>(a.b, a.w_f32, a.w_fits, 0.0f, at, b_unit);
#pragma unroll
          for (int j = 0; j < VEC; ++j) e[j] = fmaf((get(f, i * VEC + j) - centre) * rstd, w_unit[j], b_unit[j]);
          store_unit<XT, VEC>(y + i * apart, e);
        }
      }
      if (lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
    }
    if constexpr (kWait) {
      // (WARPS: all threads of a row have the same sums)
      if constexpr (WARPS) __syncthreads();
      const uint32_t all = WARPS ? block_pending : __reduce_or_sync(0xffffffffu, pending);
      if constexpr (WARPS) pending = all;
      for (uint32_t any = all; any != 0; any &= any - 1) {
        const int k = __ffs(any) - 1, back = ((turn - 1) & 31) + 1 - k;
        far_row<WARPS>(a, row - static_cast<int64_t>(back) * groups, lane, lanes, pending >> k & 1, red_far);
      }
      if constexpr (WARPS) __syncthreads();
    }
  }
}

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = lanes_sum<true>(v, 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) t += red[i];
  return t;
}

__device__ __forceinline__ float2 block_sums(float a, float b, float2* red) {
  const float v = warp_sums(a, b);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32].x = v;
  if ((threadIdx.x & 31) == 16) red[threadIdx.x / 32].y = v;
  __syncthreads();
  float2 t = both(0.0f);
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) t = add2(t, red[i]);
  return t;
}

// Forward of rows wider than a block holds, and of those past 8192 off their units: a
// block a row, three passes over it (the second and third from L2).
template <class XT>
__global__ void __launch_bounds__(kSlowThreads) norm_forward_wide_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float red[kSlowThreads / 32];
  __shared__ float2 reds[kSlowThreads / 32];
  const float d = static_cast<float>(a.d);
  const float n = static_cast<float>((a.d - static_cast<int>(threadIdx.x) + kSlowThreads - 1) / kSlowThreads);
  const XT* ahead = static_cast<const XT*>(a.x) + blockIdx.x * a.ldx;
  float x_first = to_float(ahead[0]), x_own = to_float(ahead[threadIdx.x]);  // the next row's first, the thread's first
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
    XT* y = static_cast<XT*>(a.y) + row * a.ldy;
    // `near`, the mean but for roundings, by what the elements are away from the
    // thread's first and that from the row's; then sums of what they are away from it
    const float first = within(x_first), own = within(x_own);
    float t = 0.0f;
    float2 sums = both(0.0f);  // of distances, of squares
#pragma unroll 4
    for (int i = threadIdx.x; i < a.d; i += kSlowThreads) t += to_float(x[i]) - own;
    if (row + gridDim.x < a.rows) {
      ahead = x + gridDim.x * a.ldx;
      x_first = to_float(ahead[0]);
      x_own = to_float(ahead[threadIdx.x]);
    }
    const float near = first + block_sum(fmaf(n, own - first, t), red) / d;
#pragma unroll 4
    for (int i = threadIdx.x; i < a.d; i += kSlowThreads) {
      const float c = to_float(x[i]) - near;
      sums.x += c;
      sums.y = fmaf(c, c, sums.y);
    }
    sums = block_sums(sums.x, sums.y, reds);
    const float s = finite(sums.x), shift = s / d, mean = near + shift;  // (an infinite mean stays one)
    const float rstd = reciprocal_root(fmaf(-shift, s, sums.y) / d + a.eps);
    for (int i = threadIdx.x; i < a.d; i += kSlowThreads)
      y[i] = from_float<XT>(fmaf(((to_float(x[i]) - near) - shift) * rstd, a.w ? element(a.w, a.w_f32, i) : 1.0f,
                                 a.b ? element(a.b, a.w_f32, i) : 0.0f));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// Backward.  As forward, with x and dy of a row; mean_j u and mean_j (u h) take one
// barrier a row.  The lanes' sums of dw and db leave as a row of `part` for each
// block. THREADS 512: a block of several groups fills an SM by itself, so that
// `part` has as many rows as there are SMs; the sums are in registers and the
// block's groups join theirs in shared memory.  THREADS 1024 (rows past 8192, one
// group): the sums are in shared memory, which only the lane itself reads and
// writes, and nothing is loaded ahead.
template <class XT, int VEC, int THREADS, bool WARPS>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr bool kKeep = THREADS <= 512;
  constexpr int DEPTH = kDepth<XT, VEC>;
  extern __shared__ __align__(16) uint8_t ring[];
  float* sums = reinterpret_cast<float*>(ring);  // [2 kElems][threads]
  __shared__ float2 red[2][32];
  const int lanes = a.lanes, lane = threadIdx.x % lanes, units = a.d / VEC;
  const int in_block = blockDim.x / lanes, group = threadIdx.x / lanes;
  const int groups = gridDim.x * in_block, nrows = static_cast<int>(a.rows);  // (rows fit 31 bits)
  int row = blockIdx.x * in_block + group;
  const int warp = threadIdx.x / 32, in_warp = threadIdx.x & 31;
  const int group_warps = lanes / 32;
  const bool few = group_warps <= kFewWarps;
  const int other = few ? in_warp % kFewWarps : in_warp;  // the group's warp whose sums this lane takes up
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const bool want_w = a.part != nullptr;

  const int count = lane < units ? (units - lane + lanes - 1) / lanes : 0, apart = lanes * VEC;
  RowUnits<XT, VEC, true> rows_x, rows_g;
  rows_x.begin(static_cast<const XT*>(a.x), a.ldx, row, groups, lane, lanes, units, ring, kKeep ? DEPTH : 0);
  rows_g.begin(static_cast<const XT*>(a.dy), a.lddy, row, groups, lane, lanes, units,
               ring + kRingBytes<XT, VEC> * blockDim.x, kKeep ? DEPTH : 0);
  int ahead = nrows - row;  // rows from the next to be loaded on, over all groups
  float next_mean = 0.0f, next_rstd = 0.0f;  // of the next row
  if (row < nrows) next_mean = a.mean[row], next_rstd = a.rstd[row];
  if constexpr (kKeep) {
#pragma unroll
    for (int k = 0; k < DEPTH - 1; ++k, ahead -= groups) {
      rows_x.load(ahead > 0);
      rows_g.load(ahead > 0);
      copy_async_commit();
    }
  }

  float2 dw[kKeep ? kElems / 2 : 1], db[kKeep ? kElems / 2 : 1];
  float2 wv[kElems / 2];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kElems / 2; ++i) dw[i] = db[i] = both(0.0f);
    lane_columns<VEC>(a.w, a.w_f32, a.w_fits, 1.0f, lane, lanes, units, wv);
  } else {
#pragma unroll
    for (int i = 0; i < 2 * kElems; ++i) sums[i * THREADS + threadIdx.x] = 0.0f;
  }
  XT* dx = static_cast<XT*>(a.dx) + row * a.lddx + lane * VEC;
  const int64_t dx_step = groups * a.lddx;
  const int turns = (nrows + groups - 1) / groups;
  for (int turn = 0; turn < turns; ++turn, row += groups, dx += dx_step) {
    // (a row that does not exist, and columns past the row's, are zeros of dy and add nothing)
    float2 h[kElems / 2], g[kElems / 2];
    const float mean = next_mean, rstd = next_rstd;
    next_mean = next_rstd = 0.0f;
    if (row < nrows - groups) next_mean = a.mean[row + groups], next_rstd = a.rstd[row + groups];
    if constexpr (kKeep) {
      copy_async_wait<DEPTH - 2>();
      rows_x.get(h);
      rows_g.get(g);
      rows_x.load(ahead > 0);
      rows_g.load(ahead > 0);
      ahead -= groups;
      copy_async_commit();
    } else {
      const int have = row < nrows ? count : 0;
#pragma unroll
      for (int i = 0; i < kElems / VEC; ++i) {
        float e[2][VEC] = {};
        if (i < have) {
          unpack<XT, VEC>(load_unit_once<XT, VEC>(rows_x.next + i * apart), e[0]);
          unpack<XT, VEC>(load_unit_once<XT, VEC>(rows_g.next + i * apart), e[1]);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          put(h, i * VEC + j, e[0][j]);
          put(g, i * VEC + j, e[1][j]);
        }
      }
      rows_x.next += rows_x.step;
      rows_g.next += rows_g.step;
      lane_columns<VEC>(a.w, a.w_f32, a.w_fits, 1.0f, lane, lanes, units, wv);
    }
#pragma unroll
    for (int i = 0; i < kElems / 2; ++i) h[i] = scaled(h[i], mean, rstd);
    if (want_w) {
      if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < kElems / 2; ++i) {
          dw[i] = fma2(g[i], h[i], dw[i]);
          db[i] = add2(db[i], g[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
          float* m = sums + i * THREADS + threadIdx.x;
          *m = fmaf(get(g, i), get(h, i), *m);
          m[kElems * THREADS] += get(g, i);
        }
      }
    }
    if (!a.dx) continue;
    float2 sum = both(0.0f), dot = both(0.0f);
#pragma unroll
    for (int i = 0; i < kElems / 2; ++i) {
      g[i] = mul2(g[i], wv[i]);  // u
      sum = add2(sum, g[i]);
      dot = fma2(g[i], h[i], dot);
    }
    float s, q;
    if constexpr (WARPS) {
      float2* r = red[turn & 1];
      const float v = warp_sums(sum.x + sum.y, dot.x + dot.y);
      if (in_warp == 0) r[warp].x = v;
      if (in_warp == 16) r[warp].y = v;
      group_sync(group, lanes, in_block);
      const float2 o = other < group_warps ? r[group * group_warps + other] : both(0.0f);
      s = warps_sum(o.x, few);
      q = warps_sum(o.y, few);
    } else {
      s = lanes_sum<false>(sum.x + sum.y, lanes);
      q = lanes_sum<false>(dot.x + dot.y, lanes);
    }
    if (row >= nrows) continue;
    s *= -inv_d * rstd;
    q *= -inv_d * rstd;
#pragma unroll
    for (int i = 0; i < kElems / 2; ++i) g[i] = fma2(g[i], both(rstd), fma2(h[i], both(q), both(s)));
    store_row<XT, VEC>(dx, apart, count, g);
  }
  if (!want_w) return;
  float* part = a.part + blockIdx.x * 2 * static_cast<int64_t>(a.d);
  if constexpr (kKeep) {
    const int stride = WARPS ? lanes : 32;  // the block's groups, or warps of smaller ones
    if (static_cast<int>(blockDim.x) > stride || lanes < 32) {
      // the groups of a warp, then of the block, in a fixed order
      for (int o = lanes; o < 32; o *= 2) {
#pragma unroll
        for (int i = 0; i < kElems / 2; ++i) {
          dw[i].x += __shfl_xor_sync(0xffffffffu, dw[i].x, o);
          dw[i].y += __shfl_xor_sync(0xffffffffu, dw[i].y, o);
          db[i].x += __shfl_xor_sync(0xffffffffu, db[i].x, o);
          db[i].y += __shfl_xor_sync(0xffffffffu, db[i].y, o);
        }
      }
      __syncthreads();  // (copies have all been waited for by their own threads)
#pragma unroll
      for (int i = 0; i < kElems; ++i) {
        sums[i * blockDim.x + threadIdx.x] = get(dw, i);
        sums[(kElems + i) * blockDim.x + threadIdx.x] = get(db, i);
      }
      __syncthreads();
      if (threadIdx.x >= lanes) return;
#pragma unroll
      for (int i = 0; i < kElems; ++i) {
        float sw = 0.0f, sb = 0.0f;
        for (int k = threadIdx.x; k < static_cast<int>(blockDim.x); k += stride) {
          sw += sums[i * blockDim.x + k];
          sb += sums[(kElems + i) * blockDim.x + k];
        }
        put(dw, i, sw);
        put(db, i, sb);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kElems / VEC; ++i) {
    const int at = lane + i * lanes;
    if (at >= units) continue;
    float e[2][VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if constexpr (kKeep) {
        e[0][j] = get(dw, i * VEC + j);
        e[1][j] = get(db, i * VEC + j);
      } else {
        e[0][j] = sums[(i * VEC + j) * THREADS + threadIdx.x];
        e[1][j] = sums[(kElems + i * VEC + j) * THREADS + threadIdx.x];
      }
    }
    store_unit<float, VEC>(part + at * VEC, e[0]);
    store_unit<float, VEC>(part + a.d + at * VEC, e[1]);
  }
}

// Backward of wider rows: the row's two sums, then dx; x and dy are read twice.
template <class XT>
__global__ void __launch_bounds__(kSlowThreads) norm_backward_wide_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float red[kSlowThreads / 32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
    const XT* dy = static_cast<const XT*>(a.dy) + row * a.lddy;
    XT* dx = static_cast<XT*>(a.dx) + row * a.lddx;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s = 0.0f, q = 0.0f;
    for (int i = threadIdx.x; i < a.d; i += kSlowThreads) {
      const float u = to_float(dy[i]) * (a.w ? element(a.w, a.w_f32, i) : 1.0f);
      s += u;
      q = fmaf(u, (to_float(x[i]) - mean) * rstd, q);
    }
    s = block_sum(s, red) / static_cast<float>(a.d);
    q = block_sum(q, red) / static_cast<float>(a.d);
    for (int i = threadIdx.x; i < a.d; i += kSlowThreads) {
      const float u = to_float(dy[i]) * (a.w ? element(a.w, a.w_f32, i) : 1.0f);
      dx[i] = from_float<XT>(rstd * (u - s - (to_float(x[i]) - mean) * rstd * q));
    }
  }
}

// And their dw and db: a thread a column, gridDim.y ranges of rows.
template <class XT>
__global__ void __launch_bounds__(256) norm_columns_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (col >= a.d) return;
  const int64_t share = (a.rows + gridDim.y - 1) / gridDim.y;
  const int64_t r0 = share * blockIdx.y, r1 = min(a.rows, r0 + share);
  const XT* x = static_cast<const XT*>(a.x);
  const XT* dy = static_cast<const XT*>(a.dy);
  float dw = 0.0f, db = 0.0f;
#pragma unroll 4
  for (int64_t r = r0; r < r1; ++r) {
    const float g = to_float(dy[r * a.lddy + col]);
    dw = fmaf(g, (to_float(x[r * a.ldx + col]) - a.mean[r]) * a.rstd[r], dw);
    db += g;
  }
  a.part[blockIdx.y * 2 * static_cast<int64_t>(a.d) + col] = dw;
  a.part[(blockIdx.y * 2 + 1) * static_cast<int64_t>(a.d) + col] = db;
}

// Sums of the rows of `part`, in a fixed order: 32 threads a column, each a range
// of rows, then the ranges in order.  Latency bounds it: with 8 threads a column,
// and so 19 rows a range instead of 5, it took 2 us longer.
constexpr int kReduceSlices = 32;
template <class DT>
__global__ void __launch_bounds__(32 * kReduceSlices)
    norm_reduce_kernel(const float* __restrict__ part, int64_t groups, int d, DT* __restrict__ dw, DT* __restrict__ db,
                       int add) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float red[kReduceSlices][32];
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;  // of 2 d
  const int slice = threadIdx.x / 32;
  const int64_t share = (groups + kReduceSlices - 1) / kReduceSlices, g1 = min(groups, share * (slice + 1));
  float s = 0.0f;
  if (col < 2 * static_cast<int64_t>(d)) {
#pragma unroll 8
    for (int64_t g = share * slice; g < g1; ++g) s += part[g * 2 * d + col];
  }
  red[slice][threadIdx.x % 32] = s;
  __syncthreads();
  if (slice != 0 || col >= 2 * static_cast<int64_t>(d)) return;
#pragma unroll
  for (int i = 1; i < kReduceSlices; ++i) s += red[i][threadIdx.x];
  DT* out = col < d ? (dw ? dw + col : nullptr) : (db ? db + (col - d) : nullptr);
  if (out) *out = from_float<DT>(add ? to_float(*out) + s : s);
}

// ---- host

int lanes_for(int64_t d) {
  const int64_t need = (d + kElems - 1) / kElems;
  if (need > 32) return static_cast<int>((need + 31) / 32 * 32);
  int lanes = 1;
  while (lanes < need) lanes *= 2;
  return lanes;
}

int threads_for(int lanes) { return lanes > 32 ? lanes : kFewThreads; }

struct BackwardPlan {
  int lanes, threads;
  int64_t grid, groups;  // blocks, rows of `part`
};

BackwardPlan backward_plan(int64_t rows, int64_t d, int num_sms) {
  BackwardPlan p;
  if (d > kWide) {
    p.lanes = p.threads = kSlowThreads;
    p.grid = std::min<int64_t>(rows, int64_t(4) * num_sms);
    p.groups = std::min<int64_t>(rows, 32);
    return p;
  }
  p.lanes = lanes_for(d);
  // one block an SM: its registers, at 512 threads, and its shared memory are full
  const int64_t in_block = std::max<int64_t>(1, d > kMid ? 1 : std::min<int64_t>(512 / p.lanes, rows));
  p.threads = static_cast<int>((in_block * p.lanes + 31) / 32 * 32);
  p.grid = std::min<int64_t>((rows * p.lanes + p.threads - 1) / p.threads, num_sms);
  p.groups = p.grid;
  return p;
}

constexpr int kMostSms = 160;  // workspaces are sized for this many

int64_t part_bytes(int64_t rows, int64_t d) {
  return std::max<int64_t>(backward_plan(rows, d, kMostSms).groups, 1) * 2 * d * static_cast<int64_t>(sizeof(float));
}

dgl_status check_extents(const dgl_norm_desc* n) {
  if (!n) return DGL_ERR_ARG;
  if (n->rows < 0 || n->d <= 0) return DGL_ERR_ARG;
  // (row numbers go past the last row by less than a grid's groups)
  if (n->rows > INT32_MAX - (1 << 20) || n->d > INT32_MAX / 8) return DGL_ERR_SHAPE;
  for (int32_t t : {n->x_dtype, n->w_dtype, n->dw_dtype})
    if (t != DGL_OUT_BF16 && t != DGL_OUT_F32) return DGL_ERR_ARG;
  return DGL_OK;
}

size_t size_of(int32_t dtype) { return dtype == DGL_OUT_F32 ? 4 : 2; }

// A matrix of the rows: its pitch, and by how many elements it can be accessed.
dgl_status check_matrix(const void* p, int64_t& ld, int64_t rows, int64_t d, size_t size, int64_t& vec) {
  if (!p) return DGL_ERR_ARG;
  if (ld == 0) ld = d;
  if (ld < d) return DGL_ERR_ARG;
  if (ld > INT32_MAX) return DGL_ERR_SHAPE;
  if (!aligned(p, size)) return DGL_ERR_ALIGN;
  while (vec > 1 && (!aligned(p, vec * size) || (rows > 1 && ld % vec != 0) || d % vec != 0)) vec /= 2;
  return DGL_OK;
}

// The units that there are kernels for: 16 bytes, of bf16 also 4, and single elements.
template <class XT, class F>
cudaError_t with_vec(int64_t vec, F f) {
  constexpr int kMost = 16 / static_cast<int>(sizeof(XT));
  if (vec == kMost) return f(XT{}, std::integral_constant<int, kMost>{});
  if constexpr (sizeof(XT) == 2)
    if (vec >= 2) return f(XT{}, std::integral_constant<int, 2>{});
  return f(XT{}, std::integral_constant<int, 1>{});
}

// Calls f with the element type and the access width as template arguments.
template <class F>
cudaError_t with_types(int32_t x_dtype, int64_t vec, F f) {
  return x_dtype == DGL_OUT_F32 ? with_vec<float>(vec, f) : with_vec<bf16>(vec, f);
}

// What the two calls check alike; fills a.
dgl_status prepare(dgl_norm_desc& n, bool backward, NormArgs& a, int64_t& vec) {
  const size_t xs = size_of(n.x_dtype), ws = size_of(n.w_dtype);
  vec = 16 / static_cast<int64_t>(xs);
  if (!aligned(n.weight, ws) || !aligned(n.bias, ws) || !aligned(n.mean, 4) || !aligned(n.rstd, 4))
    return DGL_ERR_ALIGN;
  dgl_status st;
  if (n.rows > 0) {
    if ((st = check_matrix(n.x, n.ldx, n.rows, n.d, xs, vec)) != DGL_OK) return st;
    if (!backward && (st = check_matrix(n.y, n.ldy, n.rows, n.d, xs, vec)) != DGL_OK) return st;
    if (backward) {
      if ((st = check_matrix(n.dy, n.lddy, n.rows, n.d, xs, vec)) != DGL_OK) return st;
      if (n.dx && (st = check_matrix(n.dx, n.lddx, n.rows, n.d, xs, vec)) != DGL_OK) return st;
      if (!n.mean || !n.rstd) return DGL_ERR_ARG;
    }
  }
  a = NormArgs{n.x,    n.ldx, n.weight, n.bias, n.w_dtype == DGL_OUT_F32,
               aligned(n.weight, 16) && aligned(n.bias, 16), n.y, n.ldy,  n.mean, n.rstd, n.dy, n.lddy, n.dx,
               n.lddx, nullptr, n.rows, static_cast<int>(n.d), 0, n.eps};
  return DGL_OK;
}

// A persistent grid of as many blocks as are resident together (one more an SM
// would run alone afterwards and double the time).
template <class X, int VEC, int THREADS, bool WARPS>
cudaError_t launch_forward(const NormArgs& a, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  static std::atomic<int> resident[33] = {};  // blocks of so many warps on an SM
  const auto kernel = norm_forward_kernel<X, VEC, THREADS, WARPS>;
  constexpr int kRing = THREADS <= 512 ? kRingBytes<X, VEC> : 0;
  const int threads = threads_for(a.lanes), smem = kRing * threads;
  cudaError_t e = cudaSuccess;
  if (kRing > 0 && (e = set_smem_attr_once(kernel, kRing * THREADS, done)) != cudaSuccess) return e;
  int fit = resident[threads / 32].load(std::memory_order_relaxed);
  if (fit == 0) {
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, threads, smem)) != cudaSuccess) return e;
    resident[threads / 32].store(fit = std::max(fit, 1), std::memory_order_relaxed);
  }
  const int64_t in_block = threads / a.lanes;
  const int64_t grid = std::min<int64_t>((a.rows + in_block - 1) / in_block, static_cast<int64_t>(fit) * num_sms);
  return launch_dependent_smem(kernel, static_cast<unsigned>(grid), threads, smem, stream, a);
}

template <class X, int VEC, int THREADS, bool WARPS>
cudaError_t launch_backward(const NormArgs& a, const BackwardPlan& plan, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int kSums = 2 * kElems * static_cast<int>(sizeof(float));  // a thread
  constexpr int kEach = THREADS <= 512 ? std::max(2 * kRingBytes<X, VEC>, kSums) : kSums;
  const auto kernel = norm_backward_kernel<X, VEC, THREADS, WARPS>;
  const cudaError_t e = set_smem_attr_once(kernel, kEach * THREADS, done);
  if (e != cudaSuccess) return e;
  // (the 1024-thread kernel's sums have a pitch of 1024)
  const int smem = kEach * (THREADS <= 512 ? plan.threads : THREADS);
  return launch_dependent_smem(kernel, static_cast<unsigned>(plan.grid), plan.threads, smem, stream, a);
}

dgl_status run_forward(dgl_norm_desc n, cudaStream_t stream) {
  NormArgs a;
  int64_t vec;
  dgl_status st = prepare(n, false, a, vec);
  if (st != DGL_OK) return st;
  if (!(n.eps >= 0.0f) || !std::isfinite(n.eps)) return DGL_ERR_ARG;
  int dev = 0;
  DeviceState* ds = nullptr;
  if ((st = get_device(&dev, &ds)) != DGL_OK) return st;
  if (n.rows == 0) return DGL_OK;
  // (past 8192 single elements spill where a block holds the row: 4000 x 12287 290 us in fp32, 110 so)
  if (n.d > kWide || (n.d > kMid && vec < (n.x_dtype == DGL_OUT_F32 ? 4 : 2))) {
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(n.rows, int64_t(4) * ds->num_sms));
    a.lanes = kSlowThreads;
    const cudaError_t e = with_types(n.x_dtype, 1, [&](auto x, auto) {
      return launch_dependent(norm_forward_wide_kernel<decltype(x)>, grid, kSlowThreads, stream, a);
    });
    return e == cudaSuccess ? DGL_OK : DGL_ERR_CUDA;
  }
  a.lanes = lanes_for(n.d);
  const cudaError_t e = with_types(n.x_dtype, vec, [&](auto x, auto v) {
    using X = decltype(x);
    constexpr int kVec = decltype(v)::value;
    if constexpr (kVec > 1)
      if (n.d > kMid) return launch_forward<X, kVec, 1024, true>(a, ds->num_sms, stream);
    return a.lanes > 32 ? launch_forward<X, kVec, 512, true>(a, ds->num_sms, stream)
                        : launch_forward<X, kVec, 512, false>(a, ds->num_sms, stream);
  });
  return e == cudaSuccess ? DGL_OK : DGL_ERR_CUDA;
}

template <class DT>
cudaError_t launch_reduce(const dgl_norm_desc& n, const float* part, int64_t groups, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((2 * n.d + 31) / 32);
  return launch_dependent(norm_reduce_kernel<DT>, grid, 32 * kReduceSlices, stream, part, groups, static_cast<int>(n.d),
                          static_cast<DT*>(n.dweight), static_cast<DT*>(n.dbias), n.accumulate);
}

dgl_status run_backward(dgl_norm_desc n, cudaStream_t stream) {
  const bool want_w = n.dweight || n.dbias;
  if (n.rows > 0 && !n.dx && !want_w) return DGL_ERR_ARG;
  if (n.accumulate != 0 && (n.accumulate != 1 || !want_w || n.dw_dtype != DGL_OUT_F32)) return DGL_ERR_ARG;
  NormArgs a;
  int64_t vec;
  dgl_status st = prepare(n, true, a, vec);
  if (st != DGL_OK) return st;
  const size_t dws = size_of(n.dw_dtype);
  if (!aligned(n.dweight, dws) || !aligned(n.dbias, dws)) return DGL_ERR_ALIGN;
  if (want_w && n.rows > 0) {
    if (!n.ws || n.ws_bytes < part_bytes(n.rows, n.d)) return DGL_ERR_ARG;
    if (!aligned(n.ws, 256)) return DGL_ERR_ALIGN;
  }
  int dev = 0;
  DeviceState* ds = nullptr;
  if ((st = get_device(&dev, &ds)) != DGL_OK) return st;
  if (ds->num_sms > kMostSms) return DGL_ERR_UNSUPPORTED;
  float* part = want_w && n.rows > 0 ? static_cast<float*>(n.ws) : nullptr;
  int64_t groups = 0;
  if (n.rows > 0) {
    const BackwardPlan plan = backward_plan(n.rows, n.d, ds->num_sms);
    const unsigned grid = static_cast<unsigned>(plan.grid);
    groups = plan.groups;
    a.lanes = plan.lanes;
    a.part = part;
    cudaError_t e = cudaSuccess;
    if (n.d > kWide) {
      if (n.dx)
        e = with_types(n.x_dtype, 1, [&](auto x, auto) {
          return launch_dependent(norm_backward_wide_kernel<decltype(x)>, grid, kSlowThreads, stream, a);
        });
      if (e == cudaSuccess && part) {
        const dim3 blocks(static_cast<unsigned>((n.d + 255) / 256), static_cast<unsigned>(groups));
        e = n.x_dtype == DGL_OUT_F32 ? launch_dependent(norm_columns_kernel<float>, blocks, 256, stream, a)
                                     : launch_dependent(norm_columns_kernel<bf16>, blocks, 256, stream, a);
      }
    } else {
      e = with_types(n.x_dtype, vec, [&](auto x, auto v) {
        using X = decltype(x);
        constexpr int kVec = decltype(v)::value;
        return n.d > kMid     ? launch_backward<X, kVec, 1024, true>(a, plan, stream)
               : a.lanes > 32 ? launch_backward<X, kVec, 512, true>(a, plan, stream)
                              : launch_backward<X, kVec, 512, false>(a, plan, stream);
      });
    }
    if (e != cudaSuccess) return DGL_ERR_CUDA;
  }
  if (!want_w || (n.rows == 0 && n.accumulate)) return DGL_OK;
  const cudaError_t e = n.dw_dtype == DGL_OUT_F32 ? launch_reduce<float>(n, part, groups, stream)
                                                  : launch_reduce<bf16>(n, part, groups, stream);
  return e == cudaSuccess ? DGL_OK : DGL_ERR_CUDA;
}

}  // namespace
}  // namespace dgl

using namespace dgl;

extern "C" {

dgl_status dgl_layer_norm_workspace(const dgl_norm_desc* norm, int64_t* bytes) {
  const dgl_status st = check_extents(norm);
  if (st != DGL_OK) return st;
  if (!bytes) return DGL_ERR_ARG;
  *bytes = norm->rows > 0 ? part_bytes(norm->rows, norm->d) : 0;
  return DGL_OK;
}

dgl_status dgl_layer_norm(const dgl_norm_desc* norm, void* stream) {
  const dgl_status st = check_extents(norm);
  return st != DGL_OK ? st : run_forward(*norm, static_cast<cudaStream_t>(stream));
}

dgl_status dgl_layer_norm_grad(const dgl_norm_desc* norm, void* stream) {
  const dgl_status st = check_extents(norm);
  return st != DGL_OK ? st : run_backward(*norm, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
