// Layer norm, forward and backward (dgl_layer_norm, dgl_layer_norm_grad).
//
// With h = (x - mean) rstd over the d elements of a row and u = dy w:
//   y  = h w + b
//   dx = rstd (u - mean_j u - h mean_j (u h))
//   dw = sum_rows dy h,  db = sum_rows dy
// Every kernel reads its matrices once and holds a row in registers, kElems
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

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's units of a row.
template <class T, int VEC>
struct RowUnits {
  static constexpr int U = kElems / VEC;
  Unit<T, VEC> u[U];

  __device__ __forceinline__ void load(const T* row, int lane, int lanes, int units) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int at = lane + i * lanes;
      if (at < units) u[i] = load_unit_once<T, VEC>(row + static_cast<int64_t>(at) * VEC);
      else u[i] = Unit<T, VEC>{};
    }
  }
  __device__ __forceinline__ void get(float (&f)[kElems]) const {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float e[VEC];
      unpack<T, VEC>(u[i], e);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[i * VEC + j] = e[j];
    }
  }
};

// The same columns of a vector (the weight or the bias); `fill` where there are none.
template <int VEC>
__device__ __forceinline__ void lane_columns(const void* v, int f32, float fill, int lane, int lanes, int units,
                                             float (&f)[kElems]) {
#pragma unroll
  for (int i = 0; i < kElems; ++i) {
    const int at = lane + i / VEC * lanes;
    f[i] = v && at < units ? element(v, f32, at * VEC + i % VEC) : fill;
  }
}

template <class T, int VEC>
__device__ __forceinline__ void store_row(T* row, int lane, int lanes, int units, const float (&f)[kElems]) {
#pragma unroll
  for (int i = 0; i < kElems / VEC; ++i) {
    const int at = lane + i * lanes;
    if (at >= units) continue;
    float e[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) e[j] = f[i * VEC + j];
    store_unit<T, VEC>(row + static_cast<int64_t>(at) * VEC, e);
  }
}

// Forward.  A persistent grid; each group of lanes takes rows a grid's groups
// apart and loads the next row while it works on this one.
// THREADS: the most in a block (1024: neither the weight nor the next row fit
// beside a row in 64 registers; the weight is read again for each row, from L1).
template <class XT, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_forward_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr bool kKeep = THREADS <= 512;
  __shared__ float2 red[2][32];
  const int lanes = a.lanes, lane = threadIdx.x % lanes, units = a.d / VEC;
  const bool whole = lanes > 32;  // the block is one group
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (blockDim.x / lanes);
  int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, in_warp = threadIdx.x & 31;
  const float inv_d = 1.0f / static_cast<float>(a.d);

  // elements that this lane holds, and its warp or group
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kElems / VEC; ++i) mine += lane + i * lanes < units ? VEC : 0;
  const float held = lanes_sum(static_cast<float>(mine), lanes < 32 ? lanes : 32);
  const float inv_held = held > 0.0f ? 1.0f / held : 0.0f;
  float other_held = 0.0f;  // of warp `in_warp`
  if (whole) {
    if (in_warp == 0) red[0][warp].x = held;
    __syncthreads();
    if (in_warp < warps) other_held = red[0][in_warp].x;
    __syncthreads();
  }

  float w[kElems], b[kElems];
  if constexpr (kKeep) {
    lane_columns<VEC>(a.w, a.w_f32, 1.0f, lane, lanes, units, w);
    lane_columns<VEC>(a.b, a.w_f32, 0.0f, lane, lanes, units, b);
  }
  const XT* x = static_cast<const XT*>(a.x);
  RowUnits<XT, VEC> next;
  // all lanes of a warp go round together: the rows of its groups may end apart
  const int64_t turns = (a.rows + groups - 1) / groups;
  if (kKeep && row < a.rows) next.load(x + row * a.ldx, lane, lanes, units);
  for (int64_t turn = 0; turn < turns; ++turn, row += groups) {
    const bool live = row < a.rows;
    float f[kElems];
    if constexpr (!kKeep) {
      if (live) next.load(x + row * a.ldx, lane, lanes, units);
    }
    next.get(f);
    if (kKeep && row + groups < a.rows) next.load(x + (row + groups) * a.ldx, lane, lanes, units);
    // the warp's (or group's) mean and squares around it, then the block's
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kElems; ++i) s += f[i];
    s = lanes_sum(s, lanes < 32 ? lanes : 32);
    float mean = s * inv_held, q = 0.0f;
#pragma unroll
    for (int i = 0; i < kElems; ++i) {
      const float c = lane + i / VEC * lanes < units ? f[i] - mean : 0.0f;
      q = fmaf(c, c, q);
    }
    q = lanes_sum(q, lanes < 32 ? lanes : 32);
    if (whole) {
      float2* r = red[turn & 1];  // two in turn: one barrier a row
      if (in_warp == 0) r[warp] = make_float2(s, q);
      __syncthreads();
      const float2 o = in_warp < warps ? r[in_warp] : make_float2(0.0f, 0.0f);
      const float warp_mean = other_held > 0.0f ? o.x / other_held : 0.0f;
      mean = lanes_sum(o.x, 32) * inv_d;
      const float c = warp_mean - mean;
      q = lanes_sum(fmaf(other_held * c, c, o.y), 32);
    }
    const float rstd = 1.0f / sqrtf(fmaf(q, inv_d, a.eps));
    if (!live) continue;
    if constexpr (!kKeep) {
      lane_columns<VEC>(a.w, a.w_f32, 1.0f, lane, lanes, units, w);
      lane_columns<VEC>(a.b, a.w_f32, 0.0f, lane, lanes, units, b);
    }
#pragma unroll
    for (int i = 0; i < kElems; ++i) f[i] = fmaf((f[i] - mean) * rstd, w[i], b[i]);
    store_row<XT, VEC>(static_cast<XT*>(a.y) + row * a.ldy, lane, lanes, units, f);
    if (lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = lanes_sum(v, 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) t += red[i];
  return t;
}

// Forward of rows wider than a block holds: a block a row, three passes over it
// (the second and third from L2).
template <class XT>
__global__ void __launch_bounds__(kSlowThreads) norm_forward_wide_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float red[kSlowThreads / 32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
    XT* y = static_cast<XT*>(a.y) + row * a.ldy;
    float s = 0.0f, q = 0.0f;
    for (int i = threadIdx.x; i < a.d; i += kSlowThreads) s += to_float(x[i]);
    const float mean = block_sum(s, red) / static_cast<float>(a.d);
    for (int i = threadIdx.x; i < a.d; i += kSlowThreads) {
      const float c = to_float(x[i]) - mean;
      q = fmaf(c, c, q);
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, red) / static_cast<float>(a.d) + a.eps);
    for (int i = threadIdx.x; i < a.d; i += kSlowThreads)
      y[i] = from_float<XT>(fmaf((to_float(x[i]) - mean) * rstd, a.w ? element(a.w, a.w_f32, i) : 1.0f, a.b ? element(a.b, a.w_f32, i) : 0.0f));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// Backward.  As forward, with x and dy of a row in registers; mean_j u and
// mean_j (u h) take one barrier a row.  The lane's sums of dw and db are in
// registers (THREADS 512) or, for rows past 8192, in shared memory, which only
// the lane itself reads and writes, and leave as a row of `part`.
template <class XT, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr bool kKeep = THREADS <= 512;
  extern __shared__ float sums[];  // !kKeep: [2][kElems][THREADS]
  __shared__ float2 red[2][32];
  const int lanes = a.lanes, lane = threadIdx.x % lanes, units = a.d / VEC;
  const bool whole = lanes > 32;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (blockDim.x / lanes);
  int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, in_warp = threadIdx.x & 31;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const bool want_w = a.part != nullptr;

  float dw[kKeep ? kElems : 1], db[kKeep ? kElems : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kElems; ++i) dw[i] = db[i] = 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < 2 * kElems; ++i) sums[i * THREADS + threadIdx.x] = 0.0f;
  }
  float wv[kElems];
  if constexpr (kKeep) lane_columns<VEC>(a.w, a.w_f32, 1.0f, lane, lanes, units, wv);
  RowUnits<XT, VEC> next_x, next_g;
  const int64_t turns = (a.rows + groups - 1) / groups;
  const XT* x = static_cast<const XT*>(a.x);
  const XT* dy = static_cast<const XT*>(a.dy);
  if (kKeep && row < a.rows) {
    next_x.load(x + row * a.ldx, lane, lanes, units);
    next_g.load(dy + row * a.lddy, lane, lanes, units);
  }
  for (int64_t turn = 0; turn < turns; ++turn, row += groups) {
    const bool live = row < a.rows;
    float h[kElems], g[kElems];
    if constexpr (!kKeep) {
      if (live) {
        next_x.load(x + row * a.ldx, lane, lanes, units);
        next_g.load(dy + row * a.lddy, lane, lanes, units);
      }
    }
    next_x.get(h);
    next_g.get(g);
    const float mean = live ? a.mean[row] : 0.0f, rstd = live ? a.rstd[row] : 0.0f;
    if (kKeep && row + groups < a.rows) {
      next_x.load(x + (row + groups) * a.ldx, lane, lanes, units);
      next_g.load(dy + (row + groups) * a.lddy, lane, lanes, units);
    }
    if constexpr (!kKeep) lane_columns<VEC>(a.w, a.w_f32, 1.0f, lane, lanes, units, wv);
    float s = 0.0f, q = 0.0f;
#pragma unroll
    for (int i = 0; i < kElems; ++i) {
      h[i] = (h[i] - mean) * rstd;
      // (a row that has ended, and columns past the row's, add nothing: g is zero there or unused)
      if (live && lane + i / VEC * lanes < units) {
        const float u = g[i] * wv[i];
        s += u;
        q = fmaf(u, h[i], q);
        if (want_w) {
          if constexpr (kKeep) {
            dw[i] = fmaf(g[i], h[i], dw[i]);
            db[i] += g[i];
          } else {
            float* m = sums + i * THREADS + threadIdx.x;
            *m = fmaf(g[i], h[i], *m);
            m[kElems * THREADS] += g[i];
          }
        }
      }
    }
    if (!a.dx) continue;
    s = lanes_sum(s, lanes < 32 ? lanes : 32);
    q = lanes_sum(q, lanes < 32 ? lanes : 32);
    if (whole) {
      float2* r = red[turn & 1];
      if (in_warp == 0) r[warp] = make_float2(s, q);
      __syncthreads();
      const float2 o = in_warp < warps ? r[in_warp] : make_float2(0.0f, 0.0f);
      s = lanes_sum(o.x, 32);
      q = lanes_sum(o.y, 32);
    }
    if (!live) continue;
    s *= inv_d;
    q *= inv_d;
#pragma unroll
    for (int i = 0; i < kElems; ++i) g[i] = rstd * (fmaf(g[i], wv[i], -s) - h[i] * q);
    store_row<XT, VEC>(static_cast<XT*>(a.dx) + row * a.lddx, lane, lanes, units, g);
  }
  if (!want_w) return;
  float* part = a.part + blockIdx.x * 2 * static_cast<int64_t>(a.d);
  if constexpr (kKeep) {
    if (!whole) {
      // the groups of the warp, then of the block's warps, in a fixed order
      __shared__ float across[kFewThreads / 32][2 * kElems][32];
#pragma unroll
      for (int i = 0; i < kElems; ++i) {
        for (int o = lanes; o < 32; o *= 2) {
          dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
          db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
        }
        across[warp][i][in_warp] = dw[i];
        across[warp][kElems + i][in_warp] = db[i];
      }
      __syncthreads();
      if (threadIdx.x >= lanes) return;
#pragma unroll
      for (int i = 0; i < kElems; ++i) {
        for (int k = 1; k < warps; ++k) {
          dw[i] += across[k][i][in_warp];
          db[i] += across[k][kElems + i][in_warp];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kElems; ++i) {
    const int at = lane + i / VEC * lanes;
    if (at >= units) continue;
    float* to = part + at * VEC + i % VEC;
    if constexpr (kKeep) {
      to[0] = dw[i];
      to[a.d] = db[i];
    } else {
      to[0] = sums[i * THREADS + threadIdx.x];
      to[a.d] = sums[(kElems + i) * THREADS + threadIdx.x];
    }
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

// Sums of the rows of `part`, in a fixed order: 8 threads a column, each
// a range of groups, then the eight in order.
template <class DT>
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* __restrict__ part, int64_t groups, int d,
                                                          DT* __restrict__ dw, DT* __restrict__ db, int add) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float red[8][32];
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;  // of 2 d
  const int slice = threadIdx.x / 32;
  const int64_t share = (groups + 7) / 8, g1 = min(groups, share * (slice + 1));
  float s = 0.0f;
  if (col < 2 * static_cast<int64_t>(d)) {
#pragma unroll 8
    for (int64_t g = share * slice; g < g1; ++g) s += part[g * 2 * d + col];
  }
  red[slice][threadIdx.x % 32] = s;
  __syncthreads();
  if (slice != 0 || col >= 2 * static_cast<int64_t>(d)) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x];
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

// Blocks of a persistent grid: `threads` a block, about `per_sm` threads on an SM.
int64_t grid_for(int64_t rows, int lanes, int threads, int per_sm, int num_sms) {
  const int64_t in_block = threads / lanes;
  const int64_t most = static_cast<int64_t>(num_sms) * std::max(1, per_sm / threads);
  return std::min((rows + in_block - 1) / in_block, most);
}

constexpr int kForwardThreads = 768, kBackwardThreads = 512;

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
  p.threads = threads_for(p.lanes);
  p.grid = grid_for(rows, p.lanes, p.threads, kBackwardThreads, num_sms);
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
  if (n->rows > INT32_MAX || n->d > INT32_MAX / 8) return DGL_ERR_SHAPE;
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

template <class XT, class F>
cudaError_t with_vec(int64_t vec, F f) {
  constexpr int kMost = 16 / static_cast<int>(sizeof(XT));
  if (vec >= kMost) return f(XT{}, std::integral_constant<int, kMost>{});
  if (vec >= 2 && sizeof(XT) == 2) return f(XT{}, std::integral_constant<int, 2>{});
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
  if (!aligned(n.weight, ws) || !aligned(n.bias, ws) || !aligned(n.mean, 4) || !aligned(n.rstd, 4)) return DGL_ERR_ALIGN;
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
  a = NormArgs{n.x,    n.ldx, n.weight, n.bias, n.w_dtype == DGL_OUT_F32, n.y, n.ldy,  n.mean, n.rstd, n.dy, n.lddy, n.dx,
               n.lddx, nullptr, n.rows, static_cast<int>(n.d), 0, n.eps};
  return DGL_OK;
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
  if (n.d > kWide) {
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(n.rows, int64_t(4) * ds->num_sms));
    a.lanes = kSlowThreads;
    const cudaError_t e = with_types(n.x_dtype, 1, [&](auto x, auto) {
      return launch_dependent(norm_forward_wide_kernel<decltype(x)>, grid, kSlowThreads, stream, a);
    });
    return e == cudaSuccess ? DGL_OK : DGL_ERR_CUDA;
  }
  a.lanes = lanes_for(n.d);
  const int threads = threads_for(a.lanes);
  const unsigned grid =
      static_cast<unsigned>(grid_for(n.rows, a.lanes, threads, n.d > kMid ? 1024 : kForwardThreads, ds->num_sms));
  const cudaError_t e = with_types(n.x_dtype, vec, [&](auto x, auto v) {
    using X = decltype(x);
    return n.d > kMid
               ? launch_dependent(norm_forward_kernel<X, decltype(v)::value, 1024>, grid, threads, stream, a)
               : launch_dependent(norm_forward_kernel<X, decltype(v)::value, 512>, grid, threads, stream, a);
  });
  return e == cudaSuccess ? DGL_OK : DGL_ERR_CUDA;
}

template <class DT>
cudaError_t launch_reduce(const dgl_norm_desc& n, const float* part, int64_t groups, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((2 * n.d + 31) / 32);
  return launch_dependent(norm_reduce_kernel<DT>, grid, 256, stream, part, groups, static_cast<int>(n.d),
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
        if (n.d <= kMid)
          return launch_dependent(norm_backward_kernel<X, kVec, 512>, grid, plan.threads, stream, a);
        static std::atomic<uint64_t> done{0};
        constexpr int kBytes = 2 * kElems * 1024 * static_cast<int>(sizeof(float));
        const cudaError_t err = set_smem_attr_once(norm_backward_kernel<X, kVec, 1024>, kBytes, done);
        if (err != cudaSuccess) return err;
        return launch_dependent_smem(norm_backward_kernel<X, kVec, 1024>, grid, plan.threads, kBytes, stream, a);
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
