// Losses of a linear head (dgl_linear_xent, dgl_linear_distill): validation,
// workspace, the per-row kernels and the calls into the tile kernel.
//
// Tokens are taken in chunks.  A chunk's logits z = s X W^T are computed by
// the tile kernel, one block per row then reduces the row to its loss and
// writes dz, and two more products of the tile kernel give dX and dW.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dgl.h"
#include "host.h"
#include "launch.h"

namespace dgl {

namespace {

constexpr int kMaxK = DGL_DISTILL_MAX_K;
constexpr int kRowThreads = 256;

// What a row asks of the softmax: xent (k == 0) one target, distill k entries.
struct HeadTargets {
  const int64_t* index;      // [T] targets or [T][k] entries
  int64_t ignore_index;      // xent
  const float* logits;       // distill: [T][k]
  const float* teacher_lse;  // distill: [T] or null
  float inv_temp;            // distill
  int k;                     // 0: xent
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

// One row's entries: index (or -1), weight q and q log q, prepared by warp 0
// into shared memory.  state: 1 a row with a loss, 0 no entries, -1 an index
// out of range.
struct RowEntries {
  int index[kMaxK];
  float q[kMaxK];
  float qlogq, Q;
  int state;
};

__device__ __forceinline__ void load_entries(RowEntries& r, const HeadTargets& tg, int64_t t, int64_t V, int lane) {
  if (tg.k == 0) {
    if (lane == 0) {
      const int64_t y = tg.index[t];
      const bool in = y >= 0 && y < V;
      r.state = y == tg.ignore_index ? 0 : in ? 1 : -1;
      r.index[0] = r.state == 1 ? static_cast<int>(y) : -1;
      r.q[0] = r.state == 1 ? 1.0f : 0.0f;
      r.Q = r.q[0];
      r.qlogq = 0.0f;
    }
    return;
  }
  // the teacher's distribution, its maximum and sum in fp32
  float high = -INFINITY;
  int bad = 0;
  for (int j = lane; j < tg.k; j += 32) {
    const int64_t i = tg.index[t * tg.k + j];
    bad |= i >= V;
    const bool kept = i >= 0 && i < V;
    const float l = kept ? tg.logits[t * tg.k + j] * tg.inv_temp : -INFINITY;
    r.index[j] = kept ? static_cast<int>(i) : -1;
    r.q[j] = l;
    // a NaN logit of a kept entry has to reach the loss: fmaxf drops it, the
    // sum below does not
    high = fmaxf(high, l);
  }
  high = warp_max(high);
  bad = __any_sync(0xffffffffu, bad);
  const float base = tg.teacher_lse ? tg.teacher_lse[t] : high;
  float sum = 0.0f;
  bool some = false;
  for (int j = lane; j < tg.k; j += 32) {
    const float l = r.q[j];
    const bool here = r.index[j] >= 0 && !(l == -INFINITY);
    some |= here;
    sum += here ? expf(l - base) : 0.0f;
  }
  sum = warp_sum(sum);
  some = __any_sync(0xffffffffu, some);
  const float log_total = tg.teacher_lse ? base : base + logf(sum);
  float Q = 0.0f, qlogq = 0.0f;
  for (int j = lane; j < tg.k; j += 32) {
    const float l = r.q[j];
    const bool here = r.index[j] >= 0 && !(l == -INFINITY);
    const float lq = l - log_total;
    const float q = here ? expf(lq) : 0.0f;
    r.q[j] = q;
    Q += q;
    qlogq += q != 0.0f ? q * lq : 0.0f;
  }
  Q = warp_sum(Q);
  qlogq = warp_sum(qlogq);
  if (lane == 0) {
    r.state = bad ? -1 : some ? 1 : 0;
    r.Q = Q;
    r.qlogq = qlogq;
  }
}

// One block per row of a chunk: z (fp32, scaled here by `scale`) -> loss, lse
// and, with dz, the row of dz in bf16, zero from V to V8, and the row of X for
// dW = dz^T X, zero where the row has no gradient (0 x NaN would reach dW).
__global__ void __launch_bounds__(kRowThreads)
    head_row_kernel(const float* __restrict__ z, int64_t ldz, __nv_bfloat16* __restrict__ dz, int64_t lddz, int64_t t0,
                    int64_t V, float scale, HeadTargets tg, const float* __restrict__ grad, float* __restrict__ loss,
                    float* __restrict__ lse_out, const __nv_bfloat16* __restrict__ x, int64_t ldx,
                    __nv_bfloat16* __restrict__ xs, int64_t d) {
  __shared__ RowEntries ent;
  __shared__ float red[2][kRowThreads / 32];
  const int64_t t = t0 + blockIdx.x;
  const float* row = z + static_cast<int64_t>(blockIdx.x) * ldz;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) load_entries(ent, tg, t, V, lane);
  float m = -INFINITY, s = 0.0f;
  for (int64_t v = threadIdx.x; v < V; v += kRowThreads) {
    const float x = row[v] * scale;
    if (x > m) {
      s = s * expf(m - x) + 1.0f;
      m = x;
    } else {
      s += x == m ? 1.0f : expf(x - m);  // equal infinities count as one each
    }
  }
  const float wm = warp_max(m);
  s = warp_sum(m == wm ? s : s * expf(m - wm));
  if (lane == 0) {
    red[0][warp] = wm;
    red[1][warp] = s;
  }
  __syncthreads();
  float bm = red[0][0], bs = 0.0f;
  for (int w = 1; w < kRowThreads / 32; ++w) bm = fmaxf(bm, red[0][w]);
  for (int w = 0; w < kRowThreads / 32; ++w) bs += red[0][w] == bm ? red[1][w] : red[1][w] * expf(red[0][w] - bm);
  const float lse = bm + logf(bs);
  const int nk = tg.k == 0 ? 1 : tg.k;
  if (threadIdx.x == 0) {
    if (lse_out) lse_out[t] = lse;
    float l = 0.0f;
    if (ent.state == 1) {
      l = ent.qlogq;
      for (int j = 0; j < nk; ++j)
        if (ent.q[j] != 0.0f) l += ent.q[j] * (lse - row[ent.index[j]] * scale);
    }
    loss[t] = ent.state < 0 ? NAN : l;
  }
  if (!dz) return;
  __nv_bfloat16* out = dz + static_cast<int64_t>(blockIdx.x) * lddz;
  const bool live = ent.state == 1;
  const float g = live ? grad[t] * scale : 0.0f;
  const int64_t V8 = (V + 7) / 8 * 8;
  for (int64_t v = threadIdx.x; v < V8; v += kRowThreads)
    out[v] = __float2bfloat16(live && v < V ? g * ent.Q * expf(row[v] * scale - lse) : 0.0f);
  for (int64_t c = threadIdx.x; c < d / 8; c += kRowThreads)
    reinterpret_cast<uint4*>(xs + blockIdx.x * d)[c] =
        live ? reinterpret_cast<const uint4*>(x + blockIdx.x * ldx)[c] : make_uint4(0u, 0u, 0u, 0u);
  if (!live) return;
  // the entries' own values, one thread each; a repeated index is written by
  // its first occurrence, with the sum of its weights
  __syncthreads();
  for (int j = threadIdx.x; j < nk; j += kRowThreads) {
    const int i = ent.index[j];
    if (i < 0) continue;
    bool first = true;
    float q = 0.0f;
    for (int l = 0; l < nk; ++l) {
      if (ent.index[l] != i) continue;
      if (l < j) first = false;
      q += ent.q[l];
    }
    if (!first) continue;
    const float p = expf(row[i] * scale - lse);
    // xent: p - 1 as minus the sum of the others would need them; expm1 of
    // the log-probability is as exact
    out[i] = __float2bfloat16(g * (tg.k == 0 ? expm1f(row[i] * scale - lse) : ent.Q * p - q));
  }
}

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

// Chunk and workspace.  A chunk of c tokens needs c rows of fp32 logits and,
// with a gradient, c rows of bf16 dz; more than one chunk accumulating a bf16
// dW needs its fp32 sums.
struct HeadLayout {
  int64_t chunk = 0;    // tokens at a time
  int64_t ldz = 0;      // row pitch of the logits and of dz, elements
  int64_t z_off = 0, dz_off = 0, xs_off = 0, dw_off = 0, bytes = 0;
};

constexpr int64_t kChunkRows = 128;                // a chunk is a multiple of this
constexpr int64_t kChunkBytes = int64_t(1) << 30;  // dz of the largest chunk

HeadLayout layout_for(const dgl_head_desc& h, int64_t chunk) {
  HeadLayout l;
  l.ldz = round_up(h.V, 64);
  l.chunk = chunk;
  const bool grad = h.grad != nullptr;
  const int64_t rows = std::min(round_up(chunk, kChunkRows), round_up(std::max<int64_t>(h.T, 1), kChunkRows));
  int64_t at = 0;
  l.z_off = at;
  at = round_up(at + rows * l.ldz * 4, 256);
  l.dz_off = at;
  if (grad) at = round_up(at + rows * l.ldz * 2, 256);
  l.xs_off = at;
  if (grad) at = round_up(at + rows * h.d * 2, 256);
  l.dw_off = at;
  if (grad && h.dW && h.dw_dtype == DGL_OUT_BF16 && chunk < h.T) at = round_up(at + h.V * h.d * 4, 256);
  l.bytes = at;
  return l;
}

// The largest chunk whose layout fits `bytes` (0 if none does).
HeadLayout choose_layout(const dgl_head_desc& h, int64_t bytes) {
  const int64_t ldz = round_up(h.V, 64);
  const int64_t most = std::max<int64_t>(kChunkRows, kChunkBytes / (ldz * 2) / kChunkRows * kChunkRows);
  HeadLayout best;
  for (int64_t c = std::min(most, round_up(std::max<int64_t>(h.T, 1), kChunkRows)); c >= kChunkRows; c -= kChunkRows) {
    const HeadLayout l = layout_for(h, c);
    if (l.bytes <= bytes) return l;
  }
  return best;
}

dgl_status check_extents(const dgl_head_desc* h, int32_t k) {
  if (!h || k < 0 || k > kMaxK) return DGL_ERR_ARG;
  if (h->T < 0 || h->V <= 0 || h->d <= 0) return DGL_ERR_ARG;
  if (h->T > INT32_MAX || h->V > INT32_MAX - 64 || h->d > INT32_MAX) return DGL_ERR_SHAPE;
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

dgl_status run_head(const dgl_head_desc* hp, const HeadTargets& tg, float scale, cudaStream_t stream) {
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
  const HeadLayout lay = choose_layout(h, h.ws_bytes);
  if (h.T > 0) {
    if (lay.chunk == 0 || !h.ws) return DGL_ERR_ARG;
    if (!aligned(h.ws, 256)) return DGL_ERR_ALIGN;
  }
  int dev = 0;
  DeviceState* ds = nullptr;
  if ((st = get_device(&dev, &ds)) != DGL_OK) return st;
  if (h.T == 0) {
    if (!h.dW || h.accumulate) return DGL_OK;
    return launch_zero_fill(h.dw_dtype, h.dW, h.lddw, static_cast<int>(h.V), static_cast<int>(h.d), stream) ==
                   cudaSuccess
               ? DGL_OK
               : DGL_ERR_CUDA;
  }

  uint8_t* ws = static_cast<uint8_t*>(h.ws);
  float* z = reinterpret_cast<float*>(ws + lay.z_off);
  __nv_bfloat16* dz = h.grad ? reinterpret_cast<__nv_bfloat16*>(ws + lay.dz_off) : nullptr;
  __nv_bfloat16* xs = reinterpret_cast<__nv_bfloat16*>(ws + lay.xs_off);
  const int64_t V8 = round_up(h.V, 8);
  const bool chunked = lay.chunk < h.T;
  // a bf16 dW of several chunks is summed in fp32 and rounded once at the end
  const bool dw_sums = h.dW && chunked && h.dw_dtype == DGL_OUT_BF16;
  for (int64_t t0 = 0; t0 < h.T; t0 += lay.chunk) {
    const int64_t n = std::min(lay.chunk, h.T - t0);
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(h.X) + t0 * h.ldx;
    Problem pz{DGL_DTYPE_BF16, DGL_OUT_F32, x, h.W, nullptr, nullptr, z, n, lay.ldz, h.d, n, h.V};
    pz.no_split = 1;
    pz.lda = h.ldx;
    pz.ldb = h.ldw;
    if ((st = run(pz, nullptr, stream)) != DGL_OK) return st;
    head_row_kernel<<<static_cast<unsigned>(n), kRowThreads, 0, stream>>>(z, lay.ldz, dz, lay.ldz, t0, h.V, scale, tg,
                                                                         h.grad, h.loss, h.lse, x, h.ldx, xs, h.d);
    if (cudaGetLastError() != cudaSuccess) return DGL_ERR_CUDA;
    if (h.dX) {
      Problem px{DGL_DTYPE_BF16, DGL_OUT_BF16, dz, h.W, nullptr, nullptr,
                 static_cast<__nv_bfloat16*>(h.dX) + t0 * h.lddx, n, h.lddx, V8, n, h.d};
      px.no_split = 1;
      px.b_mn = 1;
      px.lda = lay.ldz;
      px.ldb = h.ldw;
      px.b_k = h.V;
      if ((st = run(px, nullptr, stream)) != DGL_OK) return st;
    }
    if (h.dW) {
      const bool f32 = dw_sums || h.dw_dtype == DGL_OUT_F32;
      Problem pw{DGL_DTYPE_BF16, f32 ? DGL_OUT_F32 : DGL_OUT_BF16, dz, xs, nullptr, nullptr,
                 dw_sums ? static_cast<void*>(ws + lay.dw_off) : h.dW, h.V, dw_sums ? h.d : h.lddw, n, h.V, h.d};
      pw.no_split = 1;
      pw.a_mn = pw.b_mn = 1;
      pw.lda = lay.ldz;
      pw.ldb = h.d;
      pw.k_any = 1;
      pw.c_add = (t0 > 0 || h.accumulate) ? 1 : 0;
      if ((st = run(pw, nullptr, stream)) != DGL_OK) return st;
    }
  }
  if (dw_sums) {
    head_to_bf16_kernel<<<ds->num_sms * 8, 256, 0, stream>>>(reinterpret_cast<const float*>(ws + lay.dw_off), h.d,
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
  *min_bytes = layout_for(*head, kChunkRows).bytes;
  *best_bytes = choose_layout(*head, INT64_MAX).bytes;
  return DGL_OK;
}

dgl_status dgl_linear_xent(const dgl_head_desc* head, const int64_t* target, int64_t ignore_index, void* stream) {
  if (!head) return DGL_ERR_ARG;
  const HeadTargets tg{target, ignore_index, nullptr, nullptr, 1.0f, 0};
  return run_head(head, tg, head->logit_scale, static_cast<cudaStream_t>(stream));
}

dgl_status dgl_linear_distill(const dgl_head_desc* head, const int64_t* indices, const float* logits,
                              const float* teacher_lse, int32_t k, float temperature, void* stream) {
  if (!head || k < 1 || !(temperature > 0.0f) || !std::isfinite(temperature)) return DGL_ERR_ARG;
  const HeadTargets tg{indices, 0, logits, teacher_lse, 1.0f / temperature, k};
  return run_head(head, tg, head->logit_scale / temperature, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
