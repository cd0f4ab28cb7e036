// Embedding lookup and its gradient (dgl_embedding, dgl_embedding_grad).
//
//   Y[t] = s W[token_t],   dW[v] = s sum_{t: token_t = v} dY[t]
//
// The lookup copies rows: bound by HBM.  The gradient sorts the positions by
// token, so that each row of dW is summed by one thread a column, in the order
// of the positions, and written once: no atomics, equal calls give equal bits.
//
//   sort   one cluster of up to 8 CTAs sorts up to 131072 tokens in its shared
//          memory (radix, stable).  The other CTAs of the launch write the rows
//          of a new dW that no token reaches: HBM is busy while the sort, which
//          latency bounds, runs.
//   sum    the sorted positions in chunks of equal length; a token's run inside
//          a chunk goes to dW at once, what crosses a chunk's border to fp32
//          partial sums.  Reads dY once.
//   join   the partial sums of runs over several chunks, in order.
// More tokens are taken 131072 at a time, each adding to the sums before.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
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

// ---- lookup

struct LookupArgs {
  const int64_t* tokens;
  int64_t ignore_index;
  const void* w;
  int64_t ldw;
  void* y;
  int64_t ldy;
  int64_t rows;
  int64_t vocab;
  int units;  // of a row
  float scale;
};

constexpr int kLookupThreads = 256, kLookupEach = 4;

// Four units a thread, all loads first.  A token that is ignored gives zeros, one
// outside the vocabulary NaN.
template <class WT, class YT, int VEC>
__global__ void __launch_bounds__(kLookupThreads) embed_lookup_kernel(const __grid_constant__ LookupArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kLookupThreads * kLookupEach);
  const int64_t row0 = first / a.units;
  const uint32_t rest = static_cast<uint32_t>(first - row0 * a.units);
  Unit<WT, VEC> u[kLookupEach];
  YT* to[kLookupEach];
  float fill[kLookupEach];
  bool found[kLookupEach];
#pragma unroll
  for (int i = 0; i < kLookupEach; ++i) {
    const uint32_t at = rest + i * kLookupThreads + threadIdx.x;
    const int64_t row = row0 + at / static_cast<uint32_t>(a.units);
    const int64_t col = static_cast<int64_t>(at % static_cast<uint32_t>(a.units)) * VEC;
    to[i] = nullptr;
    found[i] = false;
    if (row >= a.rows) continue;
    to[i] = static_cast<YT*>(a.y) + row * a.ldy + col;
    const int64_t token = a.tokens[row];
    found[i] = token != a.ignore_index && token >= 0 && token < a.vocab;
    fill[i] = token == a.ignore_index ? 0.0f : NAN;
    if (found[i]) u[i] = load_unit_once<WT, VEC>(static_cast<const WT*>(a.w) + token * a.ldw + col);
  }
#pragma unroll
  for (int i = 0; i < kLookupEach; ++i) {
    if (!to[i]) continue;
    float f[VEC];
    if (found[i]) unpack<WT, VEC>(u[i], f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = found[i] ? f[j] * a.scale : fill[i];
    store_unit<YT, VEC>(to[i], f);
  }
}

// ---- gradient: sort

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortMostEach = 16;   // tokens a thread holds
constexpr int kSortCtas = 8;        // of the cluster
constexpr int kSortFew = 2 * kSortThreads;  // tokens that one CTA sorts alone
constexpr int64_t kSortMost = static_cast<int64_t>(kSortCtas) * kSortThreads * kSortMostEach;
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits;
constexpr int kMapWords = 1024;     // rows that a CTA looks at together, 32 a word

struct SortArgs {
  const int64_t* tokens;
  int64_t ignore_index;
  int n;
  int64_t vocab;
  int passes, digit_bits;
  int* keys;       // [n] tokens in order; `vocab`, behind them, for those without a row
  int* positions;  // [n]
  // rows without a token are set to zero (null: not)
  void* dw;
  int64_t row_bytes, pitch_bytes;
  int store_bytes;  // 16, 4 or 2: of a store
};

struct SortShared {
  uint16_t hist[kSortWarps][kBins];  // tokens of a warp with a digit, then those of the warps before
  uint32_t total[kBins];             // of the CTA; other CTAs read it
  uint32_t base[kBins];              // where the CTA's tokens with a digit go
  uint32_t warp_sum[kSortWarps];
};

__device__ __forceinline__ uint32_t lanes_below() {
  uint32_t m;
  asm("mov.u32 %0, %%lanemask_lt;" : "=r"(m));
  return m;
}

__device__ __forceinline__ void store_cluster(uint32_t addr, uint2 v) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ uint32_t load_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// A stable radix sort.  Thread t of warp w holds items 32 EACH w + 32 i + lane
// of its CTA's EACH 1024; items past n have the highest key.  Of each digit: an
// item's place is the number of items with a lower digit, plus those with the
// same digit in CTAs, warps and lanes before it.
template <int EACH>
__device__ void sort_tokens(const SortArgs& a, SortShared& sh, uint2* items, int ctas, int rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kHeld = EACH * kSortThreads;
  uint32_t key[EACH], position[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int at = rank * kHeld + warp * 32 * EACH + i * 32 + lane;
    key[i] = 0xffffffffu;
    position[i] = at;
    if (at < a.n) {
      const int64_t t = a.tokens[at];
      key[i] = static_cast<uint32_t>(t == a.ignore_index || t < 0 || t >= a.vocab ? a.vocab : t);
    }
  }
  const uint32_t mask = (1u << a.digit_bits) - 1;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.digit_bits;
    uint4* clear = reinterpret_cast<uint4*>(&sh.hist[0][0]);
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(sh.hist) / sizeof(uint4)); i += kSortThreads)
      clear[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    uint32_t before[EACH];  // items of the warp before this one with its digit
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const uint32_t digit = key[i] >> shift & mask;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      const uint32_t lower = __popc(same & lanes_below());
      const uint32_t so_far = sh.hist[warp][digit];
      before[i] = so_far + lower;
      __syncwarp();
      if (lower == 0) sh.hist[warp][digit] = static_cast<uint16_t>(so_far + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    uint32_t all = 0;
    if (threadIdx.x < kBins) {
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = sh.hist[w][threadIdx.x];
        sh.hist[w][threadIdx.x] = static_cast<uint16_t>(all);
        all += c;
      }
      sh.total[threadIdx.x] = all;
    }
    uint32_t earlier = 0;  // with this thread's digit, in CTAs before this one
    if (ctas > 1) {
      cluster_sync();  // also: every CTA has taken its items of the last pass
      if (threadIdx.x < kBins) {
        all = 0;
        for (int r = 0; r < ctas; ++r) {
          const uint32_t c = load_cluster(mapa_shared(smem_u32(&sh.total[threadIdx.x]), r));
          if (r < rank) earlier += c;
          all += c;
        }
      }
    }
    // items with a lower digit
    uint32_t sum = all;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) sh.warp_sum[warp] = sum;
    __syncthreads();
    if (threadIdx.x < kBins) {
      uint32_t lower = sum - all + earlier;
      for (int w = 0; w < warp; ++w) lower += sh.warp_sum[w];
      sh.base[threadIdx.x] = lower;
    }
    __syncthreads();
    const bool last = pass == a.passes - 1;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const uint32_t digit = key[i] >> shift & mask;
      const uint32_t to = sh.base[digit] + sh.hist[warp][digit] + before[i];
      if (last) {
        if (to < static_cast<uint32_t>(a.n)) {
          a.keys[to] = static_cast<int>(key[i]);
          a.positions[to] = static_cast<int>(position[i]);
        }
      } else {
        store_cluster(mapa_shared(smem_u32(items + to % kHeld), to / kHeld), make_uint2(key[i], position[i]));
      }
    }
    // (after the last pass: no CTA leaves while another may read its totals)
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    if (last) break;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const uint2 v = items[warp * 32 * EACH + i * 32 + lane];
      key[i] = v.x;
      position[i] = v.y;
    }
    __syncthreads();
  }
}

template <class U>
__device__ __forceinline__ void zero_row(uint8_t* row, int64_t bytes, int lane) {
  U* to = reinterpret_cast<U*>(row);
  for (int64_t i = lane; i < bytes / static_cast<int64_t>(sizeof(U)); i += 32) to[i] = U{};
}

// Rows of dW that no token reaches: each CTA has a range of rows and looks
// through all tokens for those in it.
__device__ void zero_rows(const SortArgs& a, uint32_t* map, int cta, int ctas) {
  const int64_t share = (a.vocab + ctas - 1) / ctas;
  const int64_t end = min(a.vocab, share * (cta + 1));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t v0 = share * cta; v0 < end; v0 += kMapWords * 32) {
    const int64_t rows = min(end - v0, static_cast<int64_t>(kMapWords * 32));
    for (int i = threadIdx.x; i < kMapWords; i += kSortThreads) map[i] = 0;
    __syncthreads();
#pragma unroll 8
    for (int i = threadIdx.x; i < a.n; i += kSortThreads) {
      const int64_t t = a.tokens[i];
      if (t != a.ignore_index && t >= v0 && t < v0 + rows)
        atomicOr(&map[(t - v0) / 32], 1u << ((t - v0) % 32));
    }
    __syncthreads();
    for (int r = warp; r < rows; r += kSortWarps) {
      if (map[r / 32] >> (r % 32) & 1) continue;
      uint8_t* row = static_cast<uint8_t*>(a.dw) + (v0 + r) * a.pitch_bytes;
      if (a.store_bytes == 16) zero_row<uint4>(row, a.row_bytes, lane);
      else if (a.store_bytes == 4) zero_row<uint32_t>(row, a.row_bytes, lane);
      else zero_row<uint16_t>(row, a.row_bytes, lane);
    }
    __syncthreads();
  }
}

// The first `ctas` CTAs (one cluster) sort, the others write zeros.
template <int EACH>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const __grid_constant__ SortArgs a, int ctas) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(16) uint8_t raw[];
  SortShared& sh = *reinterpret_cast<SortShared*>(raw);
  if (static_cast<int>(blockIdx.x) < ctas)
    sort_tokens<EACH>(a, sh, reinterpret_cast<uint2*>(raw + sizeof(SortShared)), ctas, static_cast<int>(blockIdx.x));
  else
    zero_rows(a, reinterpret_cast<uint32_t*>(raw), static_cast<int>(blockIdx.x) - ctas,
              static_cast<int>(gridDim.x) - ctas);
}

// ---- gradient: sums

struct SumArgs {
  const int* keys;
  const int* positions;
  const void* dy;
  int64_t lddy;
  void* dw;
  int64_t lddw;
  float* part;  // [chunks][2][d]: a chunk's first run, when it began before; its last, when it goes on
  int n, vocab;
  int chunk;    // positions of a chunk
  int chunks;
  int d, units, lanes;  // units of a row, threads on a row's (part of the) units
  float scale;
  int add;
};

constexpr int kSumThreads = 256;
constexpr int kSumAhead = 8;  // rows of dY in flight

template <class DT, int VEC>
__device__ __forceinline__ void finish_row(const SumArgs& a, int key, int64_t col, float (&sum)[VEC]) {
  DT* to = static_cast<DT*>(a.dw) + key * a.lddw + col;
  if (a.add) {
    float old[VEC];
    unpack<DT, VEC>(load_unit<DT, VEC>(to), old);
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] = fmaf(sum[j], a.scale, old[j]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] *= a.scale;
  }
  store_unit<DT, VEC>(to, sum);
}

// A group of lanes takes a chunk of positions and lanes x VEC columns.
template <class GT, class DT, int VEC>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const __grid_constant__ SumArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int in_block = kSumThreads / a.lanes;
  const int chunk = blockIdx.x * in_block + threadIdx.x / a.lanes;
  const int unit = blockIdx.y * a.lanes + threadIdx.x % a.lanes;
  if (threadIdx.x / a.lanes >= in_block || chunk >= a.chunks || unit >= a.units) return;
  const int64_t col = static_cast<int64_t>(unit) * VEC;
  const GT* dy = static_cast<const GT*>(a.dy) + col;
  const int j0 = chunk * a.chunk, j1 = min(a.n, j0 + a.chunk);
  float* part = a.part + static_cast<int64_t>(chunk) * 2 * a.d + col;
  int run = a.keys[j0];  // the token being summed
  if (run >= a.vocab) return;
  bool began = j0 > 0 && a.keys[j0 - 1] == run;
  const int after = j1 < a.n ? a.keys[j1] : INT_MAX;
  float sum[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
  for (int j = j0; j < j1; j += kSumAhead) {
    int key[kSumAhead];
    Unit<GT, VEC> u[kSumAhead];
#pragma unroll
    for (int i = 0; i < kSumAhead; ++i) {
      key[i] = j + i < j1 ? a.keys[j + i] : INT_MAX;
      if (key[i] < a.vocab) u[i] = load_unit_once<GT, VEC>(dy + a.positions[j + i] * a.lddy);
    }
#pragma unroll
    for (int i = 0; i < kSumAhead; ++i) {
      if (key[i] != run) {
        if (run < a.vocab && j + i <= j1) {
          // the run ended before this position, which may be the chunk's end
          if (j + i == j1 && after == run) {  // goes on in the next chunk
            store_unit<float, VEC>(part + (began ? 0 : a.d), sum);
          } else if (began) {
            store_unit<float, VEC>(part, sum);
          } else {
            finish_row<DT, VEC>(a, run, col, sum);
          }
        }
        run = key[i];
        began = false;
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum[k] = 0.0f;
      }
      if (key[i] < a.vocab) {
        float f[VEC];
        unpack<GT, VEC>(u[i], f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum[k] += f[k];
      }
    }
  }
  if (run < a.vocab) {  // the chunk's length is a whole number of steps: its last run is open
    if (after == run) store_unit<float, VEC>(part + (began ? 0 : a.d), sum);
    else if (began) store_unit<float, VEC>(part, sum);
    else finish_row<DT, VEC>(a, run, col, sum);
  }
}

// A group of lanes for each chunk in which a run begins that goes on past it.
template <class DT, int VEC>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const __grid_constant__ SumArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int in_block = kSumThreads / a.lanes;
  const int chunk = blockIdx.x * in_block + threadIdx.x / a.lanes;
  const int unit = blockIdx.y * a.lanes + threadIdx.x % a.lanes;
  if (threadIdx.x / a.lanes >= in_block || chunk >= a.chunks - 1 || unit >= a.units) return;
  const int64_t col = static_cast<int64_t>(unit) * VEC;
  const int end = (chunk + 1) * a.chunk;  // below n: another chunk follows
  const int run = a.keys[end];
  if (run >= a.vocab || a.keys[end - 1] != run) return;
  const int begin = chunk * a.chunk;
  if (a.keys[begin] == run && begin > 0 && a.keys[begin - 1] == run) return;  // began before
  // the run's end: the first position with another token
  int lo = end, hi = a.n;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (a.keys[mid] > run) hi = mid;
    else lo = mid + 1;
  }
  const int last = (lo - 1) / a.chunk;  // the chunk that it ends in
  const int64_t pitch = 2 * static_cast<int64_t>(a.d);
  const float* part = a.part + chunk * pitch + col;
  float sum[VEC];
  unpack<float, VEC>(load_unit<float, VEC>(part + a.d), sum);
  part += pitch;
#pragma unroll 8
  for (int c = chunk + 1; c <= last; ++c, part += pitch) {
    float f[VEC];
    unpack<float, VEC>(load_unit<float, VEC>(part), f);
#pragma unroll
    for (int k = 0; k < VEC; ++k) sum[k] += f[k];
  }
  finish_row<DT, VEC>(a, run, col, sum);
}

// A bf16 dW from the fp32 sums of several calls' worth of tokens.
__global__ void __launch_bounds__(256) embed_round_kernel(const float* __restrict__ sums, bf16* __restrict__ dw,
                                                          int64_t lddw, int64_t rows, int d) {
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x; i < rows * d; i += gridDim.x * static_cast<int64_t>(256))
    dw[i / d * lddw + i % d] = __float2bfloat16_rn(sums[i]);
}

// ---- host

size_t size_of(int32_t dtype) { return dtype == DGL_OUT_F32 ? 4 : 2; }
bool is_type(int32_t t) { return t == DGL_OUT_BF16 || t == DGL_OUT_F32; }
int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// A matrix's pitch, and by how many elements at once its rows can be accessed
// (units of 16 bytes, or two of those).
dgl_status check_matrix(const void* p, int64_t& ld, int64_t rows, int64_t d, size_t size, int64_t& vec) {
  if (ld == 0) ld = d;
  if (ld < d) return DGL_ERR_ARG;
  if (ld > INT32_MAX) return DGL_ERR_SHAPE;
  if (!aligned(p, size)) return DGL_ERR_ALIGN;
  auto fits = [&](int64_t v) {
    const uintptr_t bytes = std::min<uintptr_t>(16, v * size);
    return aligned(p, bytes) && (rows <= 1 || ld * size % bytes == 0) && d % v == 0;
  };
  while (vec > 1 && !fits(vec)) vec /= 2;
  return DGL_OK;
}

template <class A, class B, class F>
cudaError_t with_vec(int64_t vec, F f) {
  constexpr int kMost = 16 / static_cast<int>(sizeof(A));
  if (vec >= kMost) return f(A{}, B{}, std::integral_constant<int, kMost>{});
  if (vec >= 2) return f(A{}, B{}, std::integral_constant<int, 2>{});
  return f(A{}, B{}, std::integral_constant<int, 1>{});
}

// Calls f with the type that is read, the type that is written and the access
// width (of the first's units) as template arguments.
template <class F>
cudaError_t with_types(int32_t from, int32_t to, int64_t vec, F f) {
  if (from == DGL_OUT_F32) return to == DGL_OUT_F32 ? with_vec<float, float>(vec, f) : with_vec<float, bf16>(vec, f);
  return to == DGL_OUT_F32 ? with_vec<bf16, float>(vec, f) : with_vec<bf16, bf16>(vec, f);
}

dgl_status check_extents(const dgl_embed_desc* e) {
  if (!e) return DGL_ERR_ARG;
  if (e->T < 0 || e->V <= 0 || e->d <= 0) return DGL_ERR_ARG;
  if (e->T > INT32_MAX || e->V > INT32_MAX - 512 || e->d > INT32_MAX / 8) return DGL_ERR_SHAPE;
  if (!is_type(e->w_dtype) || !is_type(e->y_dtype)) return DGL_ERR_ARG;
  return DGL_OK;
}

dgl_status run_lookup(dgl_embed_desc e, cudaStream_t stream) {
  if (!std::isfinite(e.scale)) return DGL_ERR_ARG;
  if (e.T > 0 && (!e.tokens || !e.W || !e.Y)) return DGL_ERR_ARG;
  if (!aligned(e.tokens, 8)) return DGL_ERR_ALIGN;
  int64_t vec = 16 / static_cast<int64_t>(size_of(e.w_dtype));
  dgl_status st;
  if ((st = check_matrix(e.W, e.ldw, e.V, e.d, size_of(e.w_dtype), vec)) != DGL_OK ||
      (st = check_matrix(e.Y, e.ldy, e.T, e.d, size_of(e.y_dtype), vec)) != DGL_OK)
    return st;
  int dev = 0;
  DeviceState* ds = nullptr;
  if ((st = get_device(&dev, &ds)) != DGL_OK) return st;
  if (e.T == 0) return DGL_OK;
  const cudaError_t err = with_types(e.w_dtype, e.y_dtype, vec, [&](auto w, auto y, auto v) {
    constexpr int kVec = decltype(v)::value;
    const int64_t units = e.d / kVec;
    const LookupArgs a{e.tokens, e.ignore_index, e.W, e.ldw, e.Y, e.ldy, e.T, e.V, static_cast<int>(units), e.scale};
    const int64_t each = kLookupThreads * kLookupEach;
    const int64_t blocks = (e.T * units + each - 1) / each;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    return launch_dependent(embed_lookup_kernel<decltype(w), decltype(y), kVec>, static_cast<unsigned>(blocks),
                            kLookupThreads, stream, a);
  });
  return err == cudaSuccess ? DGL_OK : DGL_ERR_CUDA;
}

struct GradLayout {
  int64_t keys = 0, positions = 0, part = 0, sums = 0, bytes = 0;
  int chunk = 0;  // positions that a group sums
};

// Positions of a chunk: 16, or as many more as leave about 2048 threads an SM.
// (units of 16 bytes; rows that are accessed in smaller ones have more threads)
int chunk_for(int64_t n, int64_t d, int64_t size) {
  const int64_t threads = n * round_up(d * size, 16) / 16;
  return static_cast<int>(std::min<int64_t>(256, std::max<int64_t>(16, round_up(threads / (152 * 2048), kSumAhead))));
}

GradLayout grad_layout(const dgl_embed_desc& e) {
  GradLayout l;
  const int64_t n = std::min(e.T, kSortMost);
  l.chunk = chunk_for(n, e.d, size_of(e.y_dtype));
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at = round_up(at + bytes, 256);
    return here;
  };
  l.keys = take(n * 4);
  l.positions = take(n * 4);
  l.part = take((n + l.chunk - 1) / l.chunk * 2 * e.d * 4);
  if (e.T > kSortMost && e.w_dtype == DGL_OUT_BF16) l.sums = take(e.V * e.d * 4);
  l.bytes = at;
  return l;
}

template <int EACH>
cudaError_t launch_sort(const SortArgs& a, int ctas, int zero_ctas, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int kBytes = static_cast<int>(sizeof(SortShared)) + EACH * kSortThreads * 8;
  const cudaError_t err = set_smem_attr_once(embed_sort_kernel<EACH>, kBytes, done);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas + (zero_ctas + ctas - 1) / ctas * ctas));
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, embed_sort_kernel<EACH>, a, ctas);
}

dgl_status run_grad(dgl_embed_desc e, cudaStream_t stream) {
  if (!std::isfinite(e.scale)) return DGL_ERR_ARG;
  if (e.accumulate != 0 && (e.accumulate != 1 || e.w_dtype != DGL_OUT_F32)) return DGL_ERR_ARG;
  if (!e.dW || (e.T > 0 && (!e.tokens || !e.dY))) return DGL_ERR_ARG;
  if (!aligned(e.tokens, 8)) return DGL_ERR_ALIGN;
  const int64_t size = size_of(e.w_dtype);
  int64_t vec = 16 / static_cast<int64_t>(size_of(e.y_dtype));
  dgl_status st;
  if ((st = check_matrix(e.dY, e.ldy, e.T, e.d, size_of(e.y_dtype), vec)) != DGL_OK ||
      (st = check_matrix(e.dW, e.ldw, e.V, e.d, size, vec)) != DGL_OK)
    return st;
  const GradLayout lay = grad_layout(e);
  if (e.T > 0) {
    if (!e.ws || e.ws_bytes < lay.bytes) return DGL_ERR_ARG;
    if (!aligned(e.ws, 256)) return DGL_ERR_ALIGN;
  }
  int dev = 0;
  DeviceState* ds = nullptr;
  if ((st = get_device(&dev, &ds)) != DGL_OK) return st;
  if (e.T == 0 && e.accumulate) return DGL_OK;
  uint8_t* ws = static_cast<uint8_t*>(e.ws);
  float* sums = lay.sums ? reinterpret_cast<float*>(ws + lay.sums) : nullptr;
  void* dw = sums ? sums : e.dW;
  const int64_t lddw = sums ? e.d : e.ldw, dw_size = sums ? 4 : size;
  const int32_t dw_type = sums ? DGL_OUT_F32 : e.w_dtype;

  SortArgs sort = {};
  sort.ignore_index = e.ignore_index;
  sort.vocab = e.V;
  int bits = 1;
  while (e.V >> bits) ++bits;
  sort.passes = (bits + kDigitBits - 1) / kDigitBits;
  sort.digit_bits = (bits + sort.passes - 1) / sort.passes;
  sort.row_bytes = e.d * dw_size;
  sort.pitch_bytes = lddw * dw_size;
  for (sort.store_bytes = 16; sort.store_bytes > dw_size; sort.store_bytes = sort.store_bytes == 16 ? 4 : 2)
    if (aligned(dw, sort.store_bytes) && sort.row_bytes % sort.store_bytes == 0 && sort.pitch_bytes % sort.store_bytes == 0)
      break;
  int64_t t0 = 0;
  do {
    const int n = static_cast<int>(std::min(kSortMost, e.T - t0));
    const bool dense = t0 == 0 && !e.accumulate;
    sort.tokens = e.tokens + t0;
    sort.n = n;
    sort.keys = reinterpret_cast<int*>(ws + lay.keys);
    sort.positions = reinterpret_cast<int*>(ws + lay.positions);
    sort.dw = dense ? dw : nullptr;
    const int ctas = n > kSortFew ? kSortCtas : 1;
    const int zero_ctas = dense ? std::max(1, ds->num_sms - ctas) : 0;
    const int each = (n + ctas * kSortThreads - 1) / (ctas * kSortThreads);
    const cudaError_t err = each <= 1   ? launch_sort<1>(sort, ctas, zero_ctas, stream)
                            : each <= 2 ? launch_sort<2>(sort, ctas, zero_ctas, stream)
                            : each <= 4 ? launch_sort<4>(sort, ctas, zero_ctas, stream)
                            : each <= 8 ? launch_sort<8>(sort, ctas, zero_ctas, stream)
                                        : launch_sort<kSortMostEach>(sort, ctas, zero_ctas, stream);
    if (err != cudaSuccess) return DGL_ERR_CUDA;
    if (n > 0) {
      const cudaError_t e2 = with_types(e.y_dtype, dw_type, vec, [&](auto g, auto w, auto v) {
        using G = decltype(g);
        using W = decltype(w);
        constexpr int kVec = decltype(v)::value;
        SumArgs a = {};
        a.keys = sort.keys;
        a.positions = sort.positions;
        a.dy = static_cast<const G*>(e.dY) + t0 * e.ldy;
        a.lddy = e.ldy;
        a.dw = dw;
        a.lddw = lddw;
        a.part = reinterpret_cast<float*>(ws + lay.part);
        a.n = n;
        a.vocab = static_cast<int>(e.V);
        a.chunk = lay.chunk;
        a.chunks = (n + lay.chunk - 1) / lay.chunk;
        a.d = static_cast<int>(e.d);
        a.units = static_cast<int>(e.d / kVec);
        a.lanes = static_cast<int>(std::min<int64_t>(kSumThreads, round_up(a.units, 32)));
        a.scale = e.scale;
        a.add = dense ? 0 : 1;
        const int in_block = kSumThreads / a.lanes;
        const dim3 grid(static_cast<unsigned>((a.chunks + in_block - 1) / in_block),
                        static_cast<unsigned>((a.units + a.lanes - 1) / a.lanes));
        if (grid.y > 65535) return cudaErrorInvalidValue;
        const cudaError_t e3 = launch_dependent(embed_sum_kernel<G, W, kVec>, grid, kSumThreads, stream, a);
        if (e3 != cudaSuccess || a.chunks < 2) return e3;
        return launch_dependent(embed_join_kernel<W, kVec>, grid, kSumThreads, stream, a);
      });
      if (e2 != cudaSuccess) return DGL_ERR_CUDA;
    }
    t0 += n;
  } while (t0 < e.T);
  if (sums && launch_dependent(embed_round_kernel, static_cast<unsigned>(ds->num_sms * 8), 256, stream, sums,
                               static_cast<bf16*>(e.dW), e.ldw, e.V, static_cast<int>(e.d)) != cudaSuccess)
    return DGL_ERR_CUDA;
  return DGL_OK;
}

}  // namespace
}  // namespace dgl

using namespace dgl;

extern "C" {

dgl_status dgl_embedding_workspace(const dgl_embed_desc* embed, int64_t* bytes) {
  const dgl_status st = check_extents(embed);
  if (st != DGL_OK) return st;
  if (!bytes) return DGL_ERR_ARG;
  *bytes = embed->T > 0 ? grad_layout(*embed).bytes : 0;
  return DGL_OK;
}

dgl_status dgl_embedding(const dgl_embed_desc* embed, void* stream) {
  const dgl_status st = check_extents(embed);
  return st != DGL_OK ? st : run_lookup(*embed, static_cast<cudaStream_t>(stream));
}

dgl_status dgl_embedding_grad(const dgl_embed_desc* embed, void* stream) {
  const dgl_status st = check_extents(embed);
  return st != DGL_OK ? st : run_grad(*embed, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
