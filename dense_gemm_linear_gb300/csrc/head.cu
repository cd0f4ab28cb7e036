// Losses of a linear head (dgl_linear_xent, dgl_linear_distill): validation,
// workspace, the per-row kernels and the calls into the tile kernel.
//
// Tokens are taken in chunks.  In units of log 2, with y = s log2(e) x . w:
//   prepare  (distill; one warp per row) the teacher's weights q, sorted by column
//   logits   (tile kernel, HEAD) y in fp32, never stored: per row and group of
//            columns a base B near its largest y and the sum of 2^(y - B), the
//            targets' accumulators, and for a gradient e = 2^(y - B) in fp16
//   finish   (one block per row) S = sum e, lse, loss, and for the gradient
//            dz = (grad s / m) (Q e / S - q) in bf16 in the place of e
//   dX = m dz W, dW = m dz^T x  (tile kernel)
// m, between 1 and 2, is the significand of one row's |grad s|: where all rows
// have the same grad (a mean) or none, grad s / m is a power of two, and the targets'
// entries, near -grad s in every row that does not predict them, do not all
// carry the rounding of that one number into dX and dW.
// T x V values take 2 bytes of workspace for the chunk's tokens, are written
// twice and read three times; the three products are 6 T V d operations.
// e needs the 11 bits of fp16 because it is rounded again, as dz, once S is
// known (in bf16 its rounding would add to dz's); a group's own maximum keeps
// it in fp16's range whatever the logits are.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "dgl.h"
#include "host.h"
#include "launch.h"
#include "plan.h"
#include "ptx.cuh"

namespace dgl {

namespace {

constexpr int kMaxK = DGL_DISTILL_MAX_K;
constexpr int kAbsent = INT_MAX - 1;  // the column of an absent entry; one more does not overflow
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kUnshift = 1.0f / 32768.0f;  // 2^-kHeadShift

// What a row asks of the softmax: xent (k == 0) one target, distill k entries.
struct HeadTargets {
  const int64_t* index;      // [T] targets or [T][k] entries
  int64_t ignore_index;      // xent
  const float* logits;       // distill: [T][k]
  const float* teacher_lse;  // distill: [T] or null
  float inv_temp;            // distill
  int k;                     // 0: xent
};

// A chunk's rows: what `prepare` (distill only) and the logits' epilogue leave.
struct HeadRows {
  int* column;       // [rows][k] kept entries sorted by column, then kAbsent
  float* q;          // [rows][k] their weights
  float4* sums;      // [rows] Q, sum q log q, state (1: has a loss, 0: none, -1: index out of range), 0
  uint8_t* start;    // [rows][start_ld] entries before each tile of columns
  int start_ld;
  int group_shift;   // a group is 2^group_shift columns, half a tile
  float* pick;       // [rows][max(k, 1)] accumulators of the entries
  float2* part;      // [rows][groups] (base B, sum of the exponentials relative to it)
  int groups;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kPrepareWarps = 4;

// Distill, one warp per row: the teacher's distribution over the row's entries
// in fp32, the entries sorted by column (an entry's place is the number of
// entries before it, k^2 comparisons by 32 lanes), and the number of them before
// each tile of columns.  Bound by latency: 4.7 us at k = 1, 7.6 us at
// k = 64 (1024 rows, V = 50257).
// PER: entries a lane holds (k at most 32 PER).
template <int PER>
__global__ void __launch_bounds__(32 * kPrepareWarps)
    head_prepare_kernel(HeadTargets tg, HeadRows rows, int n, int V) {
  // everything before is done once the logits' kernel may start: it loads its
  // operands beside this one and waits for it in its epilogue (PDL_BATCH_NEXT)
  griddep_wait();
  griddep_launch_dependents();
  __shared__ __align__(16) int s_col[kPrepareWarps][32 * PER];
  __shared__ int s_sorted[kPrepareWarps][32 * PER];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kPrepareWarps + warp;
  if (row >= n) return;
  const int k = tg.k;
  int col[PER];
  float l[PER];
  float high = -INFINITY;
  bool bad = false, some = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + 32 * i;
    col[i] = kAbsent;
    l[i] = -INFINITY;
    if (j < k) {
      const int64_t c64 = tg.index[static_cast<int64_t>(row) * k + j];
      bad |= c64 >= V;
      if (c64 >= 0 && c64 < V) {
        const float v = tg.logits[static_cast<int64_t>(row) * k + j];
        if (!(v == -INFINITY)) {  // minus infinity: no probability; NaN stays, and reaches the loss
          col[i] = static_cast<int>(c64);
          l[i] = v;
          high = fmaxf(high, v);
          some = true;
        }
      }
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  some = __any_sync(0xffffffffu, some);
  high = warp_max(high);
  // log q and q.  Without teacher_lse log q is (l - high) / temperature - log
  // sum: the difference to the row's largest logit is taken first, in which what
  // the logits have in common goes before anything is rounded, and nothing of
  // their size is added again (log sum is at most log k).
  const bool share = tg.teacher_lse != nullptr;
  const float whole = share ? tg.teacher_lse[row] : 0.0f;
  float lq[PER], q[PER];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    lq[i] = share ? fmaf(l[i], tg.inv_temp, -whole) : (l[i] - high) * tg.inv_temp;
    q[i] = col[i] != kAbsent ? expf(lq[i]) : 0.0f;
    sum += q[i];
  }
  float Q = sum = warp_sum(sum);
  if (!share && some) {
    const float log_sum = logf(sum);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      lq[i] -= log_sum;
      q[i] = __fdiv_rn(q[i], sum);
      total += q[i];
    }
    Q = warp_sum(total);
  }
  float qlogq = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) qlogq += q[i] != 0.0f ? q[i] * lq[i] : 0.0f;
  qlogq = warp_sum(qlogq);
  const int state = bad ? -1 : some ? 1 : 0;
  if (lane == 0) rows.sums[row] = make_float4(Q, qlogq, static_cast<float>(state), 0.0f);
  // sort by (column, position): an entry's place is the number before it
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (state != 1) col[i] = kAbsent;
    s_col[warp][lane + 32 * i] = col[i];
  }
  __syncwarp();
  // (entries past k are kAbsent, and come after every entry before k)
  int place[PER] = {};
#pragma unroll 2
  for (int o = 0; o < k; o += 4) {
    const int4 four = *reinterpret_cast<const int4*>(&s_col[warp][o]);
    const int other[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int i = 0; i < PER; ++i) place[i] += other[v] < col[i] + (o + v < lane + 32 * i);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (lane + 32 * i < k) {
      s_sorted[warp][place[i]] = col[i];
      rows.column[static_cast<int64_t>(row) * k + place[i]] = col[i];
      rows.q[static_cast<int64_t>(row) * k + place[i]] = q[i];
    }
  }
  __syncwarp();
  int kept = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) kept += col[i] != kAbsent;
  kept = __reduce_add_sync(0xffffffffu, kept);
#pragma unroll 4
  for (int g = lane; g < rows.start_ld; g += 32) {
    // entries with a column below the tile's first one (the last tile ends past V)
    const int64_t below = static_cast<int64_t>(g) << (rows.group_shift + 1);
    int lo = 0;
#pragma unroll
    for (int step = 32 * PER; step > 0; step >>= 1)
      if (lo + step <= kept && s_sorted[warp][lo + step - 1] < below) lo += step;
    rows.start[static_cast<int64_t>(row) * rows.start_ld + g] = static_cast<uint8_t>(lo);
  }
}

// m of a chunk: the significand of |grad s| of its first row whose grad s is a
// normal number (1 where none is).
__device__ __forceinline__ bool is_normal(float g) { return fabsf(g) >= 1.17549435e-38f && fabsf(g) < INFINITY; }
__device__ __forceinline__ float significand(float g) {
  return __uint_as_float((__float_as_uint(g) & 0x007FFFFFu) | 0x3F800000u);
}
// By a warp: m where one of the first 32 rows decides it (lane i holds row i's
// grad s, 0 past the last), else 0.
__device__ __forceinline__ float common_significand(float g) {
  const uint32_t normal = __ballot_sync(0xffffffffu, is_normal(g));
  const float first = __shfl_sync(0xffffffffu, g, normal ? __ffs(normal) - 1 : 0);
  return normal ? significand(first) : 0.0f;
}
// By a block, for a chunk that starts with 32 rows or more without a grad (a
// prompt that is masked by its weights): rows 32 .. n - 1, 4 THREADS at a time.
template <int THREADS>
__device__ float search_significand(const float* __restrict__ grad, float scale, int n, int* found) {
  for (int i0 = 32; i0 < n; i0 += 4 * THREADS) {
    int mine = INT_MAX;
#pragma unroll
    for (int u = 3; u >= 0; --u) {
      const int i = i0 + u * THREADS + threadIdx.x;
      if (i < n && is_normal(grad[i] * scale)) mine = i;
    }
    mine = __reduce_min_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0) found[threadIdx.x >> 5] = mine;
    __syncthreads();
    for (int w = 0; w < THREADS / 32; ++w) mine = min(mine, found[w]);
    if (mine != INT_MAX) return significand(grad[mine] * scale);
    __syncthreads();  // read by all before it is written again
  }
  return 1.0f;
}

// A gradient's blocks of short rows (or slices) are of 128 threads, so that all
// that an SM has room for hide each other's first and last steps, long rows'
// of 256 (128 / 256 threads, us in all: 1000 x 4095 x 512 38 / 43, 6000 x 11007 x
// 256 179 / 200, 4000 x 20000 x 256 224 / 228, 2000 x 32000 x 256 168.9 / 169.4,
// 1024 x 50257 x 512 180 / 177, 1500 x 50257 x 256 210 / 201).
constexpr int64_t kFinishShort = 32768;  // columns

// One block per row, and with few rows several, each for a slice of the
// vocabulary (gridDim.y; all of them reduce the row's statistics): statistics
// of the row's column groups -> loss and lse; with e (gradient), e -> dz in
// place (zero up to a multiple of 8 columns), and, when dW is asked for, x for
// dW = dz^T x, zero where the row has no gradient (0 x NaN would reach dW).  A
// gradient is bound by reading e and writing dz: 10240 x 50257 in 305 to 328 us,
// 6.8 to 6.3 TB/s, on different GPUs.
template <bool GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS)
    head_finish_kernel(HeadTargets tg, HeadRows rows, int V, float scale, float c, const float* __restrict__ grad,
                       float* __restrict__ out_scale, float* __restrict__ loss, float* __restrict__ lse_out,
                       uint16_t* __restrict__ e, int64_t lde, const __nv_bfloat16* __restrict__ x, int64_t ldx,
                       __nv_bfloat16* __restrict__ xs, int d, int* __restrict__ flags, int nflags) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int WARPS = THREADS / 32;
  __shared__ float red[3][WARPS];
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool lead = blockIdx.y == 0;
  if (row == 0 && lead)
    for (int i = threadIdx.x; i < nflags; i += THREADS) flags[i] = 0;
  const float2* part = rows.part + static_cast<int64_t>(row) * rows.groups;
  // gradient: this block's slice of e, in units of eight columns.  A thread has U
  // loads in flight: the first beside the row's statistics, then the next ones
  // beside the arithmetic and stores of the ones before (1024 x 50257 x 512 in
  // all: 182 us with U = 4 loads at the loop's head, 176 so; 180 / 183 with U =
  // 2 / 8)
  uint16_t* er = e + row * lde;
  uint4* e8 = reinterpret_cast<uint4*>(er);
  const int units = (V + 7) / 8, share = (units + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
  const int u0 = min(units, share * static_cast<int>(blockIdx.y)), u1 = min(units, u0 + share);
  constexpr int U = 4;
  uint4 v[U];
  float v_top[U];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * THREADS;
      if (i < u1) {
        v[u] = e8[i];
        v_top[u] = part[8 * i >> rows.group_shift].x;
      }
    }
  };
  if (GRAD) fetch(u0 + threadIdx.x);
  const float g32 = GRAD && lane < gridDim.x ? grad[lane] * scale : 0.0f;
  const float g_row = GRAD ? grad[row] * scale : 0.0f;
  // the row's targets, entry j (of k, at most kMaxK) with thread j: its column
  // (-1: none), weight, accumulator and its group's base
  static_assert(THREADS >= kMaxK, "an entry a thread");
  const int k = tg.k == 0 ? 1 : tg.k;
  int state;
  float Q = 1.0f, l = 0.0f, weight = 0.0f, acc = 0.0f, own = 0.0f;
  int64_t at = -1;
  int before = -1;  // the column of entry j - 1
  if (tg.k == 0) {
    const int64_t target = tg.index[row];
    state = target == tg.ignore_index ? 0 : target >= 0 && target < V ? 1 : -1;
    if (state == 1 && threadIdx.x == 0) {
      at = target;
      weight = 1.0f;
    }
  } else {
    const float4 sums = rows.sums[row];
    Q = sums.x;
    l = sums.y;
    state = static_cast<int>(sums.z);
    if (state == 1 && threadIdx.x < k) {
      const int64_t slot = static_cast<int64_t>(row) * k + threadIdx.x;
      const int col = rows.column[slot];
      at = col == kAbsent ? -1 : col;
      weight = rows.q[slot];
      if (threadIdx.x > 0) before = rows.column[slot - 1];
    }
  }
  if (at >= 0) {
    acc = rows.pick[static_cast<int64_t>(row) * k + threadIdx.x];
    own = part[at >> rows.group_shift].x;
  }
  float m = -INFINITY, s = 0.0f;
  for (int g = threadIdx.x; g < rows.groups; g += THREADS) {
    const float2 v = part[g];
    const float top = fmaxf(m, v.x);
    // a group without a maximum sums to zero, or to NaN
    s = top == -INFINITY ? s + v.y : s * exp2f(m - top) + v.y * exp2f(v.x - top);
    m = top;
  }
  const float wm = warp_max(m);
  s = warp_sum(wm == -INFINITY ? s : s * exp2f(m - wm));
  if (lane == 0) {
    red[0][warp] = wm;
    red[1][warp] = s;
  }
  __syncthreads();
  float base = red[0][0], S = 0.0f;
#pragma unroll
  for (int i = 1; i < WARPS; ++i) base = fmaxf(base, red[0][i]);
#pragma unroll
  for (int i = 0; i < WARPS; ++i) S += red[0][i] == -INFINITY ? red[1][i] : red[1][i] * exp2f(red[0][i] - base);
  S *= kUnshift;  // relative to 2^base
  const float log_S = log2f(S);

  // The entry's term is formed as the epilogue formed it, so that it is the very
  // number that S holds (but for a factor, 1 in the group of the row's maximum):
  // S - term is the sum of the others', never below zero, and a sure token's
  // loss and dz are what they leave.
  float term = 0.0f, short_of = 0.0f;  // 2^(y - base), and ((term - S) / S, p - 1)
  if (threadIdx.x < ((k + 31) & ~31)) {
    float t = 0.0f;
    if (at >= 0) {
      const float arg = head_argument(acc, c, own);
      term = ex2(arg) * (kUnshift * exp2f(own - base));
      short_of = (term - S) / S;
      // -log p, as -log(1 + (p - 1)) where p is large, else as log2 S - (y - base)
      if (weight != 0.0f)
        t = weight * (short_of > -0.5f ? -log1pf(short_of)
                                       : (log_S - ((arg - kHeadShift) + (own - base))) * kLn2);
    }
    t = warp_sum(t);
    if (lane == 0) red[2][warp] = t;
  }
  __syncthreads();
  if (threadIdx.x == 0 && lead) {
    float t = 0.0f;
    for (int w = 0; w < (k + 31) / 32; ++w) t += red[2][w];
    if (lse_out) lse_out[row] = (base + log_S) * kLn2;
    loss[row] = state < 0 ? NAN : state == 0 ? 0.0f : l + t;
  }
  if (!GRAD) return;

  const bool has = state == 1;
  const bool writes = row == 0 && lead;
  float common = common_significand(g32);
  // rows that need m and do not see it yet look for it, as far as themselves
  // where their own grad would do
  if (common == 0.0f && (writes || (has && g_row != 0.0f))) {
    __shared__ int found[WARPS];
    common = search_significand<THREADS>(grad, scale, is_normal(g_row) ? row + 1 : gridDim.x, found);
  }
  if (writes && threadIdx.x == 0) *out_scale = common;
  const float f = has && g_row != 0.0f ? __fdiv_rn(g_row, common) : 0.0f;
  const float fS = f * (Q / S);
  if (!has) {
    for (int i = u0 + threadIdx.x; i < u1; i += THREADS) e8[i] = make_uint4(0u, 0u, 0u, 0u);
  } else {
    for (int i0 = u0 + threadIdx.x; i0 < u1; i0 += U * THREADS) {
      uint4 now[U];
      float now_top[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        now[u] = v[u];
        now_top[u] = v_top[u];
      }
      fetch(i0 + U * THREADS);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * THREADS;
        if (i >= u1) break;
        const float a = fS * exp2f((now_top[u] - base) - kHeadShift);
        uint32_t* w = reinterpret_cast<uint32_t*>(&now[u]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 p2 = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          const __nv_bfloat162 b2 = __floats2bfloat162_rn(p2.x * a, p2.y * a);
          w[j] = *reinterpret_cast<const uint32_t*>(&b2);
        }
        e8[i] = now[u];
      }
    }
  }
  if (xs) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + row * ldx);
    uint4* xo = reinterpret_cast<uint4*>(xs + static_cast<int64_t>(row) * d);
    for (int i = threadIdx.x + blockIdx.y * THREADS; i < d / 8; i += THREADS * gridDim.y)
      xo[i] = has ? xr[i] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (!has) return;
  __syncthreads();
  // this thread's entry, if its column lies in this block's slice; entries of
  // one column are neighbours, and the first carries their weights
  if (at < static_cast<int64_t>(u0) * 8 || at >= static_cast<int64_t>(u1) * 8 || (tg.k != 0 && before == at)) return;
  float w = weight;
  if (tg.k != 0)
    for (int j = threadIdx.x + 1; j < k && rows.column[static_cast<int64_t>(row) * k + j] == at; ++j)
      w += rows.q[static_cast<int64_t>(row) * k + j];
  // Q p - w; of a likely token Q (p - 1) + (Q - w), the sums of the others
  const float dz = short_of > -0.5f ? f * fmaf(Q, short_of, Q - w) : f * (Q * (term / S) - w);
  er[at] = __bfloat16_as_ushort(__float2bfloat16(dz));
}

// dX from the fp32 sums of its ranges of the vocabulary, in order, so that the
// result does not depend on which finished first; a thread adds four columns of
// a row.  Bound by latency and L2: nine ranges of 1024 x 512 (19 MB) in 4.4 us.
__global__ void __launch_bounds__(256)
    head_join_kernel(const float* __restrict__ part, int64_t slab, int splits, __nv_bfloat16* __restrict__ out,
                     int64_t ldo, int rows, int cols) {
  griddep_wait();
  griddep_launch_dependents();  // dW loads its operands beside this (PDL_BATCH_NEXT)
  const int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x;
  if (i >= static_cast<int64_t>(rows) * (cols / 4)) return;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int k = 0; k < splits; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(part + k * slab + 4 * i);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  const __nv_bfloat162 o[2] = {__floats2bfloat162_rn(s.x, s.y), __floats2bfloat162_rn(s.z, s.w)};
  const int64_t r = i / (cols / 4), c = i % (cols / 4) * 4;
  *reinterpret_cast<uint2*>(out + r * ldo + c) = *reinterpret_cast<const uint2*>(o);
}

// Launch of a kernel that starts with griddep_wait.
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, unsigned threads, cudaStream_t stream,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// A bf16 dW from the fp32 sums of several chunks: 6 bytes an element, HBM-bound.
__global__ void head_to_bf16_kernel(const float* __restrict__ src, int64_t lds, __nv_bfloat16* __restrict__ dst,
                                    int64_t ldd, int64_t rows, int64_t cols) {
  const int64_t n = rows * (cols / 8);
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / (cols / 8), c = i % (cols / 8) * 8;
    const float4 a = *reinterpret_cast<const float4*>(src + r * lds + c);
    const float4 b = *reinterpret_cast<const float4*>(src + r * lds + c + 4);
    __nv_bfloat162 o[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w),
                           __floats2bfloat162_rn(b.x, b.y), __floats2bfloat162_rn(b.z, b.w)};
    *reinterpret_cast<uint4*>(dst + r * ldd + c) = *reinterpret_cast<uint4*>(o);
  }
}

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Chunk and workspace.  Rows of a chunk hold e (gradient), the prepared rows
// and the column groups' statistics; dX also needs the fp32 sums of its ranges or
// partial tiles, dW the rows of x and, when several chunks add up to a bf16 one,
// its fp32 sums.
struct HeadLayout {
  int64_t chunk = 0;  // tokens at a time (0: does not fit)
  int64_t lde = 0;    // row pitch of e, elements
  int64_t e = 0, xs = 0, pick = 0, part = 0, column = 0, q = 0, sums = 0, start = 0;
  int64_t split = 0, flags = 0, out_scale = 0, dw = 0;
  int64_t bytes = 0;
};

constexpr int64_t kChunkRows = 128;  // a chunk is a multiple of this
// The largest chunk: rows that fill every SM many times over, and with a
// gradient e of at most 1 GiB.  Each further chunk of a gradient reads and
// writes the fp32 sums of dW once more.
constexpr int64_t kChunkBytes = int64_t(1) << 30;
constexpr int64_t kChunkRowsMost = 32768;
constexpr int64_t kKeepBytes = int64_t(126) << 20;  // L2
constexpr int kSplitSlots = 160;  // partial tiles of 128 x 256: one per CTA

// Column groups of a row: halves of the logits' tiles.
int64_t head_groups(int64_t V, int tile_n) { return 2 * ((V + tile_n - 1) / tile_n); }

// The tile of the logits' product.  Up to 128 rows W's reads set the time: the
// narrower tile when it leaves the busiest SM fewer columns (V = 50257 on 152
// SMs, 3 x 128 against 2 x 256: 1 x 50257 x 2048 39.8 against 42.6 us; V = 32000,
// 2 x 128 against 1 x 256: 16 x 32000 x 4096 49.0 against 47.1).  Above, the cost
// model's cheaper of 128 x 256 tiles and 256 x 256 CTA pairs (333 rows: 3 row
// tiles against 2 of twice the height, 34 against 39 us).
constexpr int64_t kNarrowRows = 128;

int logits_tile_n(int64_t rows, int64_t V, int num_sms) {
  auto most = [&](int64_t cols) { return ((V + cols - 1) / cols + num_sms - 1) / num_sms * cols; };
  return rows <= kNarrowRows && most(128) < most(256) ? 128 : 256;
}

int logits_tile_m(int64_t rows, int64_t V, int64_t d, int num_sms) {
  if (rows <= kNarrowRows) return 128;
  double best = 0.0;
  int best_m = 0;
  for (int tile_m : {128, 256}) {
    double stage_us, tile_us;
    if (!tc_tile_cost(tile_m, 256, &stage_us, &tile_us)) continue;
    const int64_t units = num_sms / (tile_m == 256 ? 2 : 1);
    const int64_t tiles = ((rows + tile_m - 1) / tile_m) * ((V + 255) / 256);
    const double est = static_cast<double>((tiles + units - 1) / units) * ((d + 63) / 64 * stage_us + tile_us);
    if (best_m == 0 || est <= best) {
      best = est;
      best_m = tile_m;
    }
  }
  return best_m;
}

HeadLayout layout_for(const dgl_head_desc& h, int k, int64_t chunk) {
  HeadLayout l;
  l.lde = round_up(h.V, 64);
  l.chunk = chunk;
  const bool grad = h.grad != nullptr;
  const int64_t rows = std::min(chunk, round_up(std::max<int64_t>(h.T, 1), kChunkRows));
  // statistics of the chunk, or of one of few rows on the narrower tiles
  const int64_t groups = head_groups(h.V, 256);
  const int64_t narrow = std::min(rows, kNarrowRows) * head_groups(h.V, 128);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at = round_up(at + bytes, 256);
    return here;
  };
  if (grad) {
    l.e = take(rows * l.lde * 2);
    if (h.dW) l.xs = take(rows * h.d * 2);
    if (h.dX) {
      l.split = take(int64_t(kSplitSlots) * 128 * 256 * 4);
      l.flags = take(kSplitSlots * 4);
    }
    l.out_scale = take(4);
  }
  l.part = take(std::max(rows * groups, narrow) * 8);
  l.pick = take(rows * std::max(k, 1) * 4);
  if (k > 0) {
    l.column = take(rows * k * 4);
    l.q = take(rows * k * 4);
    l.sums = take(rows * 16);
    // one more than tiles of columns, which are half the groups
    l.start = take(std::max(rows * groups, narrow));
  }
  if (grad && h.dW && h.dw_dtype == DGL_OUT_BF16 && chunk < h.T) l.dw = take(h.V * h.d * 4);
  l.bytes = at;
  return l;
}

// The largest chunk whose layout fits `bytes` (chunk 0 if none does).
HeadLayout choose_layout(const dgl_head_desc& h, int k, int64_t bytes) {
  const int64_t fit = kChunkBytes / (round_up(h.V, 64) * 2) / kChunkRows * kChunkRows;
  const int64_t most = h.grad ? std::max(kChunkRows, std::min(fit, kChunkRowsMost)) : kChunkRowsMost;
  for (int64_t c = std::min(most, round_up(std::max<int64_t>(h.T, 1), kChunkRows)); c >= kChunkRows; c -= kChunkRows) {
    const HeadLayout l = layout_for(h, k, c);
    if (l.bytes <= bytes) return l;
  }
  return HeadLayout{};
}

dgl_status check_extents(const dgl_head_desc* h, int32_t k) {
  if (!h || k < 0 || k > kMaxK) return DGL_ERR_ARG;
  if (h->T < 0 || h->V <= 0 || h->d <= 0) return DGL_ERR_ARG;
  if (h->T > INT32_MAX || h->V > INT32_MAX - 512 || h->d > INT32_MAX) return DGL_ERR_SHAPE;
  if (h->d % 8 != 0) return DGL_ERR_ALIGN;
  if (h->d * 4 > INT32_MAX) return DGL_ERR_SHAPE;
  if (h->dw_dtype != DGL_OUT_BF16 && h->dw_dtype != DGL_OUT_F32) return DGL_ERR_ARG;
  return DGL_OK;
}

dgl_status check_matrix(const void* p, int64_t& ld, int64_t d) {
  if (ld == 0) ld = d;
  if (ld < d) return DGL_ERR_ARG;
  if (ld > INT32_MAX) return DGL_ERR_SHAPE;
  if (ld % 8 != 0 || !aligned(p, 16)) return DGL_ERR_ALIGN;
  return DGL_OK;
}

// dX's tile and schedule.  The sum runs over the vocabulary, so few tiles with
// a very long sum are the ordinary case.  With at most half as many tiles as
// workers, each tile's sum is cut into as many ranges as there are workers for
// and a further kernel adds their fp32 sums, all SMs at once; stream-K's tile
// owner would add them one after another (131 x 1024 over 11007: 63 us with
// stream-K, 18.6 us with ranges).  With more tiles, the tail's k-stages are
// shared by all workers where the cost model says so (stream-K): few ranges a
// tile.  Returns the number of ranges.
constexpr double kJoinUs = 3.0;           // the adding kernel's launch and latency
constexpr double kJoinBytesPerUs = 4.0e6;  // its reads, and the ranges' writes, mostly in L2

int choose_dx_plan(int64_t m, int64_t n, int64_t K, int num_sms, dgl_plan_info* out) {
  double best = 0.0;
  int best_splits = 0;
  const int nk = static_cast<int>((K + 63) / 64);
  for (int tile_m : {128, 256})
    for (int tile_n : {128, 256}) {
      const int units = num_sms / (tile_m == 256 ? 2 : 1);
      const int64_t tiles = ((m + tile_m - 1) / tile_m) * ((n + tile_n - 1) / tile_n);
      dgl_plan_info cand;
      fill_tc_plan(DGL_DTYPE_BF16, DGL_OUT_BF16, m, n, K, tile_m, tile_n, num_sms, &cand, 2 * tiles > units ? -1 : 0);
      if (best_splits == 0 || cand.est_us <= best) {
        *out = cand;
        best = cand.est_us;
        best_splits = 1;
      }
      const int splits = static_cast<int>(std::min<int64_t>(units / std::max<int64_t>(tiles, 1), nk / 4));
      if (splits < 2) continue;
      double stage_us, tile_us;
      if (!tc_tile_cost(tile_m, tile_n, &stage_us, &tile_us)) continue;
      const double est = 5.0 + (nk + splits - 1) / splits * stage_us + tile_us + kJoinUs +
                         8.0 * splits * static_cast<double>(m) * n / kJoinBytesPerUs;
      if (est < best) {
        fill_tc_plan(DGL_DTYPE_BF16, DGL_OUT_F32, m, n, K, tile_m, tile_n, num_sms, out, 0);
        out->split_tail = 0;
        best = est;
        best_splits = splits;
      }
    }
  return best_splits;
}

// dW's tile: the cost model's cheapest.
void choose_dw_plan(int64_t m, int64_t n, int64_t K, bool f32, int num_sms, dgl_plan_info* out) {
  bool have = false;
  for (int tile_m : {128, 256})
    for (int tile_n : {128, 256}) {
      dgl_plan_info cand;
      fill_tc_plan(DGL_DTYPE_BF16, f32 ? DGL_OUT_F32 : DGL_OUT_BF16, m, n, K, tile_m, tile_n, num_sms, &cand, 0);
      if (!have || cand.est_us <= out->est_us) *out = cand;
      have = true;
    }
}

dgl_status run_head(const dgl_head_desc* hp, const HeadTargets& targets, float scale, cudaStream_t stream) {
  HeadTargets tg = targets;
  dgl_status st = check_extents(hp, tg.k);
  if (st != DGL_OK) return st;
  dgl_head_desc h = *hp;
  if (!std::isfinite(scale)) return DGL_ERR_ARG;
  if (h.accumulate != 0 && (h.accumulate != 1 || !h.dW || h.dw_dtype != DGL_OUT_F32)) return DGL_ERR_ARG;
  if (h.T > 0 && (h.grad != nullptr) != (h.dX || h.dW)) return DGL_ERR_ARG;
  if (!h.W) return DGL_ERR_ARG;
  if (h.T > 0 && (!h.X || !h.loss || !tg.index || (tg.k > 0 && !tg.logits))) return DGL_ERR_ARG;
  if ((st = check_matrix(h.X, h.ldx, h.d)) != DGL_OK || (st = check_matrix(h.W, h.ldw, h.d)) != DGL_OK) return st;
  if (h.dX && (st = check_matrix(h.dX, h.lddx, h.d)) != DGL_OK) return st;
  if (h.dW && (st = check_matrix(h.dW, h.lddw, h.d)) != DGL_OK) return st;
  if (!aligned(h.loss, 4) || !aligned(h.lse, 4) || !aligned(h.grad, 4) || !aligned(tg.index, 8) ||
      !aligned(tg.logits, 4) || !aligned(tg.teacher_lse, 4))
    return DGL_ERR_ALIGN;
  const HeadLayout lay = choose_layout(h, tg.k, h.ws_bytes);
  if (h.T > 0) {
    if (lay.chunk == 0 || !h.ws) return DGL_ERR_ARG;
    if (!aligned(h.ws, 256)) return DGL_ERR_ALIGN;
  }
  int dev = 0;
  DeviceState* ds = nullptr;
  if ((st = get_device(&dev, &ds)) != DGL_OK) return st;
  if (ds->smem_optin < 232448) return DGL_ERR_UNSUPPORTED;  // every tile variant is sized for 227 KB
  if (h.T == 0) {
    if (!h.dW || h.accumulate) return DGL_OK;
    return launch_zero_fill(h.dw_dtype, h.dW, h.lddw, static_cast<int>(h.V), static_cast<int>(h.d), stream) ==
                   cudaSuccess
               ? DGL_OK
               : DGL_ERR_CUDA;
  }

  const bool grad = h.grad != nullptr;
  uint8_t* ws = static_cast<uint8_t*>(h.ws);
  uint16_t* e = grad ? reinterpret_cast<uint16_t*>(ws + lay.e) : nullptr;
  __nv_bfloat16* xs = h.dW ? reinterpret_cast<__nv_bfloat16*>(ws + lay.xs) : nullptr;
  SplitScratch scratch;
  scratch.ws = reinterpret_cast<float*>(ws + lay.split);
  scratch.ws_bytes = size_t(kSplitSlots) * 128 * 256 * 4;
  scratch.flags = reinterpret_cast<int*>(ws + lay.flags);
  scratch.nflags = kSplitSlots;
  float* out_scale = reinterpret_cast<float*>(ws + lay.out_scale);
  const int V = static_cast<int>(h.V), d = static_cast<int>(h.d);
  const int64_t V8 = round_up(h.V, 8);
  const float c = scale * kLog2e;
  // a bf16 dW of several chunks is summed in fp32 and rounded once at the end
  const bool dw_sums = h.dW && lay.chunk < h.T && h.dw_dtype == DGL_OUT_BF16;
  for (int64_t t0 = 0; t0 < h.T; t0 += lay.chunk) {
    const int n = static_cast<int>(std::min(lay.chunk, h.T - t0));
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(h.X) + t0 * h.ldx;
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(h.W);
    const int tile_m = logits_tile_m(n, h.V, h.d, ds->num_sms), tile_n = logits_tile_n(n, h.V, ds->num_sms);
    tg.index = targets.index + t0 * std::max(tg.k, 1);
    if (tg.k > 0) tg.logits = targets.logits + t0 * tg.k;
    if (tg.teacher_lse) tg.teacher_lse = targets.teacher_lse + t0;
    HeadRows rows = {};
    rows.pick = reinterpret_cast<float*>(ws + lay.pick);
    rows.part = reinterpret_cast<float2*>(ws + lay.part);
    rows.groups = static_cast<int>(head_groups(h.V, tile_n));
    rows.group_shift = tile_n == 256 ? 7 : 6;
    if (tg.k > 0) {
      rows.column = reinterpret_cast<int*>(ws + lay.column);
      rows.q = reinterpret_cast<float*>(ws + lay.q);
      rows.sums = reinterpret_cast<float4*>(ws + lay.sums);
      rows.start = ws + lay.start;
      rows.start_ld = rows.groups / 2 + 1;
    }

    if (tg.k > 0 && launch_dependent(tg.k <= 32   ? head_prepare_kernel<1>
                                     : tg.k <= 64 ? head_prepare_kernel<2>
                                                  : head_prepare_kernel<4>,
                                     static_cast<unsigned>((n + kPrepareWarps - 1) / kPrepareWarps), 32 * kPrepareWarps,
                                     stream, tg, rows, n, V) != cudaSuccess)
      return DGL_ERR_CUDA;

    // ---- logits
    const int cg = tile_m == 256 ? 2 : 1;
    CUtensorMap ta, tb, tc = {};
    const int a_box = static_cast<int>(std::min<int64_t>(round_up(n, 8), 128));
    if (!bf16_operand_map(&ta, x, h.d, n, a_box, h.ldx) || !bf16_operand_map(&tb, w, h.d, h.V, tile_n / cg, h.ldw) ||
        (grad && !bf16_output_map(&tc, e, V8, n, lay.lde)))
      return DGL_ERR_CUDA;
    TcParams p = {};
    p.m = n;
    p.n = V;
    p.K = d;
    p.tiles_m = (n + tile_m - 1) / tile_m;
    p.tiles_n = static_cast<int>((h.V + tile_n - 1) / tile_n);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (tiles > INT32_MAX) return DGL_ERR_SHAPE;
    p.num_tiles = static_cast<int>(tiles);
    p.num_kb = (d + 63) / 64;
    p.group_m = 16;
    p.c_tma = grad ? 1 : 0;
    p.a_box_rows = a_box < 128 ? a_box : 0;
    // W is swept once for up to 16 row tiles; with few of them it need not stay
    // in L2 (2047 x 50257 x 1024: 153 -> 144 us; at 16 row tiles no gain)
    p.b_once = p.tiles_m <= 8 ? 1 : 0;
    // e that fits L2 is kept there for the next kernels (1024 x 50257 x 512: 189
    // -> 185 us in all; 4095 x 32000, twice L2, 0.5% slower)
    p.c_keep = static_cast<int64_t>(n) * lay.lde * 2 <= kKeepBytes ? 1 : 0;
    p.status = ds->status;
    p.workers = std::min(p.num_tiles, ds->num_sms / cg);
    p.dp_tiles = p.num_tiles;
    p.sk_workers = p.workers;
    p.pdl_mode = tg.k > 0 ? PDL_BATCH_NEXT : PDL_SERIAL;
    p.head.c = c;
    p.head.part = rows.part;
    p.head.part_ld = rows.groups;
    p.head.target = tg.k > 0 ? nullptr : tg.index;
    p.head.column = rows.column;
    p.head.start = rows.start;
    p.head.start_ld = rows.start_ld;
    p.head.k = std::max(tg.k, 1);
    p.head.pick = rows.pick;
    if (launch_tc_head(grad, tile_m, tile_n, ta, tb, tc, p, p.workers * cg, stream) != cudaSuccess) return DGL_ERR_CUDA;

    // few rows: enough blocks for every SM to hold several, of at least 2048
    // columns (100 x 50257 x 512: 73 -> 66 us in all, 4 x 50257 x 2048: 155 -> 148)
    const int64_t slices = grad ? std::min<int64_t>(int64_t(8) * ds->num_sms / n, h.V / 2048) : 1;
    const dim3 finish(static_cast<unsigned>(n), static_cast<unsigned>(std::max<int64_t>(1, slices)));
    const bool small = grad && h.V / finish.y <= kFinishShort;
    if (launch_dependent(!grad   ? head_finish_kernel<false, 256>
                         : small ? head_finish_kernel<true, 128>
                                 : head_finish_kernel<true, 256>,
                         finish, small ? 128 : 256, stream, tg, rows, V, scale, c,
                         grad ? h.grad + t0 : nullptr, out_scale, h.loss + t0, h.lse ? h.lse + t0 : nullptr, e, lay.lde,
                         x, h.ldx, xs, d, scratch.flags, h.dX ? kSplitSlots : 0) != cudaSuccess)
      return DGL_ERR_CUDA;

    if (h.dX) {
      __nv_bfloat16* dx = static_cast<__nv_bfloat16*>(h.dX) + t0 * h.lddx;
      dgl_plan_info plan;
      const int splits = choose_dx_plan(n, h.d, V8, ds->num_sms, &plan);
      Problem px{DGL_DTYPE_BF16, splits > 1 ? DGL_OUT_F32 : DGL_OUT_BF16, e, w, nullptr, nullptr,
                 splits > 1 ? static_cast<void*>(scratch.ws) : dx, n, splits > 1 ? h.d : h.lddx, V8, n, h.d};
      px.b_mn = 1;
      px.lda = lay.lde;
      px.ldb = h.ldw;
      px.b_k = h.V;
      px.k_splits = splits;
      px.tight_a = 1;
      px.out_scale = out_scale;
      // dW needs nothing of dX: it loads its operands while dX's last tiles, or
      // the kernel that adds its ranges, run
      if (h.dW && splits == 1) px.pdl_mode = PDL_BATCH_HEAD;
      if ((st = run(px, &plan, stream, &scratch)) != DGL_OK) return st;
      const int64_t slab = round_up(n, plan.tile_m) * h.d;  // elements of a range's sums
      const int64_t quads = static_cast<int64_t>(n) * (h.d / 4);
      if (splits > 1 && launch_dependent(head_join_kernel, static_cast<unsigned>((quads + 255) / 256), 256, stream,
                                         scratch.ws, slab, splits, dx, h.lddx, n, d) != cudaSuccess)
        return DGL_ERR_CUDA;
    }
    if (h.dW) {
      const bool f32 = dw_sums || h.dw_dtype == DGL_OUT_F32;
      Problem pw{DGL_DTYPE_BF16, f32 ? DGL_OUT_F32 : DGL_OUT_BF16, e, xs, nullptr, nullptr,
                 dw_sums ? static_cast<void*>(ws + lay.dw) : h.dW, h.V, dw_sums ? h.d : h.lddw, n, h.V, h.d};
      pw.no_split = 1;
      pw.a_mn = pw.b_mn = 1;
      pw.lda = lay.lde;
      pw.ldb = h.d;
      pw.k_any = 1;
      pw.c_add = (t0 > 0 || h.accumulate) ? 1 : 0;
      if (h.dX) pw.pdl_mode = PDL_BATCH_NEXT;
      pw.out_scale = out_scale;
      dgl_plan_info plan;
      choose_dw_plan(h.V, h.d, n, f32, ds->num_sms, &plan);
      if ((st = run(pw, &plan, stream)) != DGL_OK) return st;
    }
  }
  if (dw_sums) {
    head_to_bf16_kernel<<<ds->num_sms * 8, 256, 0, stream>>>(reinterpret_cast<const float*>(ws + lay.dw), h.d,
                                                             static_cast<__nv_bfloat16*>(h.dW), h.lddw, h.V, h.d);
    if (cudaGetLastError() != cudaSuccess) return DGL_ERR_CUDA;
  }
  return DGL_OK;
}

}  // namespace
}  // namespace dgl

using namespace dgl;

extern "C" {

dgl_status dgl_head_workspace(const dgl_head_desc* head, int32_t k, int64_t* min_bytes, int64_t* best_bytes) {
  const dgl_status st = check_extents(head, k);
  if (st != DGL_OK) return st;
  if (!min_bytes || !best_bytes) return DGL_ERR_ARG;
  // (one chunk of all tokens needs no sums of dW, so it may be the smaller)
  *best_bytes = choose_layout(*head, k, INT64_MAX).bytes;
  *min_bytes = std::min(layout_for(*head, k, kChunkRows).bytes, *best_bytes);
  return DGL_OK;
}

dgl_status dgl_linear_xent(const dgl_head_desc* head, const int64_t* target, int64_t ignore_index, void* stream) {
  if (!head) return DGL_ERR_ARG;
  const HeadTargets tg{target, ignore_index, nullptr, nullptr, 1.0f, 0};
  return run_head(head, tg, head->logit_scale, static_cast<cudaStream_t>(stream));
}

dgl_status dgl_linear_distill(const dgl_head_desc* head, const int64_t* indices, const float* logits,
                              const float* teacher_lse, int32_t k, float temperature, void* stream) {
  const float inv_temp = 1.0f / temperature;
  if (!head || k < 1 || !(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(inv_temp))
    return DGL_ERR_ARG;
  const HeadTargets tg{indices, 0, logits, teacher_lse, inv_temp, k};
  return run_head(head, tg, head->logit_scale / temperature, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
