// Embedding lookup and its gradient (dgl_embedding, dgl_embedding_grad).
//
//   Y[t] = s W[token_t],   dW[v] = s sum_{t: token_t = v} dY[t]
//
// The lookup copies rows: bound by HBM.  The gradient sorts the positions by
// token, so that each row of dW is summed by one thread a column, in the order
// of the positions, and written or added to once: equal calls give equal bits.
//
//   sort   one cluster of up to 8 CTAs sorts up to 131072 tokens in its shared
//          memory (radix, stable).  The other CTAs of the launch keep HBM busy
//          while the sort, which latency bounds, runs: with zeros for rows of a new dW
//          that no token reaches, or dY's rows on their way to L2.
//   sum    the sorted positions in chunks of equal length, a block each; a token's run
//          inside a chunk goes to dW at once, what crosses a chunk's border to
//          fp32 partial sums.  Reads dY once.
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
  int64_t vocab;
  int rows;
  int units;   // of a row
  int lanes;   // threads of a worker
  int slices;  // workers of a row
  float scale;
};

constexpr int kLookupThreads = 256;

// Units that a lane takes of a row: 64 bytes of W, in loads of what alignment allows.
template <class WT, int VEC>
constexpr int kLookupUnits = VEC == 1 ? 16 : 64 / (VEC * static_cast<int>(sizeof(WT)));

// A worker (a warp, or a part of one for narrow rows) takes a slice of a row, all
// loads first.  A token that is ignored gives zeros, one outside the vocabulary NaN.
template <class WT, class YT, int VEC>
__global__ void __launch_bounds__(kLookupThreads) embed_lookup_kernel(const __grid_constant__ LookupArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int U = kLookupUnits<WT, VEC>;
  const int lane = threadIdx.x % a.lanes;
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * (kLookupThreads / a.lanes) + threadIdx.x / a.lanes;
  const int64_t row = worker / a.slices;
  const int first = static_cast<int>(worker % a.slices) * a.lanes * U + lane;
  if (row >= a.rows || first >= a.units) return;
  const int64_t token = a.tokens[row];
  YT* y = static_cast<YT*>(a.y) + row * a.ldy;
  if (token == a.ignore_index || token < 0 || token >= a.vocab) {
    float f[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = token == a.ignore_index ? 0.0f : NAN;
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (first + i * a.lanes < a.units) store_unit<YT, VEC>(y + (first + i * a.lanes) * VEC, f);
    return;
  }
  const WT* w = static_cast<const WT*>(a.w) + token * a.ldw;
  Unit<WT, VEC> u[U];
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (first + i * a.lanes < a.units) u[i] = load_unit_once<WT, VEC>(w + (first + i * a.lanes) * VEC);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (first + i * a.lanes >= a.units) continue;
    float f[VEC];
    unpack<WT, VEC>(u[i], f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] *= a.scale;
    store_unit<YT, VEC>(y + (first + i * a.lanes) * VEC, f);
  }
}

// Threads of a worker: a warp, or fewer for rows of fewer units.
int lanes_for(int64_t units) {
  int lanes = 1;
  while (lanes < 32 && lanes < units) lanes *= 2;
  return lanes;
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
  int2* sorted;    // [n] tokens in order and their positions; behind them, as `vocab`, those without a row
  // what the other CTAs of the launch do meanwhile: a new dW's rows without a
  // token, or (null) dY's rows on their way to L2
  void* dw;
  int64_t row_bytes, pitch_bytes;
  int element;        // bytes
  uint32_t* present;  // bits of the rows of dW that a token reaches, where rows are left to the next kernel
  int share, quota;   // rows of a CTA's range, and of those that it sets to zero now; whole words
  const void* dy;
  int64_t dy_bytes;   // of a row that its CTA asks for (0: nothing to prefetch)
  int64_t dy_pitch;
};

struct SortShared {
  uint16_t hist[kSortWarps][kBins];  // tokens of a warp with a digit, then those of its half's warps before
  uint32_t half[2][kBins];           // of the CTA's lower and upper half of warps
  uint32_t total[kBins];             // of the CTA; other CTAs read it
  uint32_t base[kBins];              // where the CTA's tokens with a digit go
  uint32_t mine[kBins];              // and where among the CTA's own
  uint2 warp_sum[kBins / 32];
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
      // the lanes with this digit, by a vote on each of its bits (a match
      // instruction took longer: 131072 tokens 60 us with it, 55 so, and 50 with the
      // last pass below)
      uint32_t same = 0xffffffffu;
#pragma unroll
      for (int bit = 0; bit < kDigitBits; ++bit) {
        const uint32_t set = __ballot_sync(0xffffffffu, digit >> bit & 1);
        same &= digit >> bit & 1 ? set : ~set;
      }
      const uint32_t lower = __popc(same & lanes_below());
      const uint32_t so_far = sh.hist[warp][digit];
      before[i] = so_far + lower;
      __syncwarp();
      if (lower == 0) sh.hist[warp][digit] = static_cast<uint16_t>(so_far + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    // a digit's tokens in the warps before: two threads a digit, half of the warps each
    constexpr int kHalf = kSortWarps / 2;
    static_assert(kSortThreads == 2 * kBins, "two threads a digit");
    const int bin = threadIdx.x % kBins, half = threadIdx.x / kBins;
    uint32_t all = 0;
#pragma unroll
    for (int w = half * kHalf; w < (half + 1) * kHalf; ++w) {
      const uint32_t c = sh.hist[w][bin];
      sh.hist[w][bin] = static_cast<uint16_t>(all);
      all += c;
    }
    sh.half[half][bin] = all;
    __syncthreads();
    all = sh.half[0][bin] + sh.half[1][bin];
    if (half == 0) sh.total[bin] = all;
    uint32_t earlier = 0;  // with this thread's digit, in CTAs before this one
    if (ctas > 1) {
      cluster_sync();  // also: every CTA has taken its items of the last pass
      if (half == 0) {
        uint32_t c[kSortCtas];
#pragma unroll
        for (int r = 0; r < kSortCtas; ++r) c[r] = load_cluster(mapa_shared(smem_u32(&sh.total[bin]), r));
        all = 0;
#pragma unroll
        for (int r = 0; r < kSortCtas; ++r) {
          if (r < rank) earlier += c[r];
          all += c[r];
        }
      }
    }
    // items with a lower digit, in all CTAs and in this one
    const uint32_t own = sh.half[0][bin] + sh.half[1][bin];
    uint2 sum = make_uint2(all, own);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint2 v = make_uint2(__shfl_up_sync(0xffffffffu, sum.x, o), __shfl_up_sync(0xffffffffu, sum.y, o));
      if (lane >= o) sum.x += v.x, sum.y += v.y;
    }
    if (half == 0 && lane == 31) sh.warp_sum[warp] = sum;
    __syncthreads();
    if (half == 0) {
      uint2 before_warp = lane < warp ? sh.warp_sum[lane] : make_uint2(0, 0);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        before_warp.x += __shfl_xor_sync(0xffffffffu, before_warp.x, o);
        before_warp.y += __shfl_xor_sync(0xffffffffu, before_warp.y, o);
      }
      sh.base[bin] = sum.x - all + earlier + before_warp.x;
      sh.mine[bin] = sum.y - own + before_warp.y;
    }
    __syncthreads();
    const bool last = pass == a.passes - 1;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const uint32_t digit = key[i] >> shift & mask;
      // the items with this digit before it in the CTA
      const uint32_t nth = (warp < kHalf ? 0 : sh.half[0][digit]) + sh.hist[warp][digit] + before[i];
      if (last) {
        items[sh.mine[digit] + nth] = make_uint2(key[i], position[i]);
      } else {
        const uint32_t to = sh.base[digit] + nth;
        store_cluster(mapa_shared(smem_u32(items + to % kHeld), to / kHeld), make_uint2(key[i], position[i]));
      }
    }
    // (after the last pass: no CTA leaves while another may read its totals)
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    if (last) {
      // in order among the CTA's own, so that neighbours mostly go to neighbouring
      // places (131072 tokens: 55 us with each item written where it goes at once)
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        const uint32_t at = i * kSortThreads + threadIdx.x;
        const uint2 v = items[at];
        const uint32_t digit = v.x >> shift & mask, to = sh.base[digit] + at - sh.mine[digit];
        if (to < static_cast<uint32_t>(a.n)) a.sorted[to] = make_int2(static_cast<int>(v.x), static_cast<int>(v.y));
      }
    }
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

// Zeros in a row of any alignment: 16-byte stores, and single elements at its ends.
__device__ __forceinline__ void zero_row(uint8_t* row, int64_t bytes, int element, int lane) {
  const int64_t head = min(bytes, static_cast<int64_t>(-reinterpret_cast<uintptr_t>(row) & 15));
  const int64_t body = (bytes - head) / 16 * 16;
  for (int64_t i = lane * 16; i < body; i += 512) *reinterpret_cast<uint4*>(row + head + i) = make_uint4(0, 0, 0, 0);
  const int64_t edge = bytes - body;  // bytes that are left, at both ends
  for (int64_t i = lane * element; i < edge; i += 32 * element) {
    uint8_t* to = row + (i < head ? i : i + body);
    if (element == 4) *reinterpret_cast<uint32_t*>(to) = 0;
    else *reinterpret_cast<uint16_t*>(to) = 0;
  }
}

// Rows of dW that no token reaches: each CTA has a range of rows and looks through
// all tokens for those in it.  It writes zeros to the first of them, about as many
// as the sort takes time for, and leaves the others to the next kernel, whose sums
// wait on latency and not on HBM: 185 of 206 MB of zeros by these CTAs alone took
// 45 us, and the sums 18 us after them.
__device__ void zero_rows(const SortArgs& a, uint32_t* map, int cta) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t begin = static_cast<int64_t>(a.share) * cta, end = min(a.vocab, begin + a.share);
  for (int64_t v0 = begin; v0 < end; v0 += kMapWords * 32) {
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
    if (a.quota < a.share) {
      uint32_t* present = a.present + v0 / 32;  // (shares are whole words)
      for (int i = threadIdx.x; i < (rows + 31) / 32; i += kSortThreads) present[i] = map[i];
    }
    const int64_t now = min(rows, begin + a.quota - v0);
    for (int r = warp; r < now; r += kSortWarps)
      if (!(map[r / 32] >> (r % 32) & 1))
        zero_row(static_cast<uint8_t*>(a.dw) + (v0 + r) * a.pitch_bytes, a.row_bytes, a.element, lane);
    __syncthreads();
  }
}

// dY's rows into L2, where the sums then find them: nothing else reads HBM while the
// sort runs.
__device__ void prefetch_rows(const SortArgs& a, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  for (int t = cta * kSortWarps + (threadIdx.x >> 5); t < a.n; t += ctas * kSortWarps) {
    const int64_t token = a.tokens[t];
    if (token == a.ignore_index || token < 0 || token >= a.vocab) continue;
    const uint8_t* row = static_cast<const uint8_t*>(a.dy) + t * a.dy_pitch;
    for (int64_t i = lane * 128; i < a.dy_bytes; i += 32 * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row + i));
  }
}

// The first `ctas` CTAs (one cluster) sort; what the others do, see above.
template <int EACH>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const __grid_constant__ SortArgs a, int ctas) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(16) uint8_t raw[];
  SortShared& sh = *reinterpret_cast<SortShared*>(raw);
  const int cta = static_cast<int>(blockIdx.x) - ctas;
  if (cta < 0)
    sort_tokens<EACH>(a, sh, reinterpret_cast<uint2*>(raw + sizeof(SortShared)), ctas, static_cast<int>(blockIdx.x));
  else if (a.dw)
    zero_rows(a, reinterpret_cast<uint32_t*>(raw), cta);
  else
    prefetch_rows(a, cta, static_cast<int>(gridDim.x) - ctas);
}

// ---- gradient: sums

struct SumArgs {
  const int2* sorted;  // tokens and positions
  const void* dy;
  int64_t lddy;
  void* dw;
  int64_t lddw;
  float* part;  // [chunks][2][d]: a chunk's first run, when it began before; its last, when it goes on
  int n, vocab;
  int each;     // positions that a worker takes
  int chunk;    // and a block, all its workers together
  int chunks;
  int d, units;  // units of a row
  int lanes;    // threads of a worker
  int slices;   // blocks that share a chunk, each with some columns
  float scale;
  int add;
  // a new dW's rows without a token that are left to be set to zero
  int zero_blocks;
  int64_t words;       // of `present`, in all ranges together
  int words_each;      // that a block takes
  int range_words, quota_words;  // of a range, and of those that are done
  const uint32_t* present;
};

constexpr int kSumThreads = 256;
constexpr int kMostChunk = 2048;
// A lane's units of a row, 16 bytes of dY in all (their loads are smaller where
// alignment says so), and the rows that a worker has in flight.
template <class GT, int VEC>
constexpr int kSumUnits = 16 / (VEC * static_cast<int>(sizeof(GT)));
template <class GT, int VEC>
constexpr int kSumAhead = kSumUnits<GT, VEC> == 1 ? 8 : kSumUnits<GT, VEC> == 8 ? 2 : 4;

// sum: of a unit.  To an fp32 dW by a reduction in L2, which waits for no load;
// each element gets one, so that its order is fixed (subnormal sums count as zero
// there).
template <class DT, int VEC>
__device__ __forceinline__ void finish_unit(const SumArgs& a, int key, int64_t col, const float* sum) {
  DT* to = static_cast<DT*>(a.dw) + key * a.lddw + col;
  float f[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] = sum[j] * a.scale;
  if constexpr (sizeof(DT) == 4) {
    if (a.add) {
      if constexpr (VEC >= 4) {
#pragma unroll
        for (int j = 0; j < VEC; j += 4)
          asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to + j), "f"(f[j]), "f"(f[j + 1]),
                       "f"(f[j + 2]), "f"(f[j + 3])
                       : "memory");
      } else if constexpr (VEC == 2) {
        asm volatile("red.global.add.v2.f32 [%0], {%1, %2};" ::"l"(to), "f"(f[0]), "f"(f[1]) : "memory");
      } else {
        asm volatile("red.global.add.f32 [%0], %1;" ::"l"(to), "f"(f[0]) : "memory");
      }
      return;
    }
  }
  store_unit<DT, VEC>(to, f);
}

__device__ void zero_rest(const SumArgs& a, int64_t row_bytes, int64_t pitch_bytes, int element, int block) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int left = a.range_words - a.quota_words;
  const int64_t begin = static_cast<int64_t>(block) * a.words_each, end = min(a.words, begin + a.words_each);
  for (int64_t k = begin; k < end; ++k) {
    const int64_t word = k / left * a.range_words + a.quota_words + k % left;
    if (word * 32 >= a.vocab) continue;
    const uint32_t present = a.present[word];
    for (int r = warp; r < 32 && word * 32 + r < a.vocab; r += kSumThreads / 32)
      if (!(present >> r & 1))
        zero_row(static_cast<uint8_t*>(a.dw) + (word * 32 + r) * pitch_bytes, row_bytes, element, lane);
  }
}

// A block takes a chunk of the sorted positions and the columns of one worker. Its
// workers (a warp, or a part of one for narrow rows) take neighbouring pieces of
// the chunk and all the same columns.  A run of one token inside a piece goes to
// dW; a piece's first run that began before it, and its last that goes on, are left
// in shared memory, where the block adds up those of its workers in order.  What
// began before the chunk, or goes on after it, goes to `part`. Blocks that write
// the remaining zeros lie between them.
template <class GT, class DT, int VEC>
__global__ void __launch_bounds__(kSumThreads, 3) embed_sum_kernel(const __grid_constant__ SumArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int U = kSumUnits<GT, VEC>, E = U * VEC, AHEAD = kSumAhead<GT, VEC>;
  __shared__ __align__(16) float open[2][kSumThreads * E];  // first runs and last runs of the pieces
  __shared__ int keys_at[kMostChunk + 2];                   // the chunk's, one before and one behind
  __shared__ int positions[kMostChunk];
  // zero block `z` of all, spread evenly, or sum block `block`
  const int64_t all = gridDim.x;
  const int z = static_cast<int>(blockIdx.x * static_cast<int64_t>(a.zero_blocks) / all);
  if (static_cast<int>((blockIdx.x + 1) * static_cast<int64_t>(a.zero_blocks) / all) != z) {
    zero_rest(a, static_cast<int64_t>(a.d) * sizeof(DT), a.lddw * static_cast<int64_t>(sizeof(DT)), sizeof(DT), z);
    return;
  }
  const int block = blockIdx.x - z, chunk = block / a.slices, slice = block % a.slices;
  const int lane = threadIdx.x % a.lanes, worker = threadIdx.x / a.lanes, workers = kSumThreads / a.lanes;
  const int first_unit = slice * a.lanes * U + lane;
  const int c0 = chunk * a.chunk, c1 = min(a.n, c0 + a.chunk);
  const int* keys = keys_at + 1 - c0;
  for (int i = threadIdx.x; i < c1 - c0 + 2; i += kSumThreads) {
    const int at = c0 - 1 + i;
    const int2 v = at < 0 ? make_int2(-1, 0) : at < a.n ? a.sorted[at] : make_int2(INT_MAX, 0);
    keys_at[i] = v.x;
    if (at >= c0 && at < c1) positions[at - c0] = v.y;
  }
  __syncthreads();
  const int j0 = min(c0 + worker * a.each, c1), j1 = min(j0 + a.each, c1);
  float* first = &open[0][threadIdx.x * E];
  float* last = &open[1][threadIdx.x * E];
  float sum[E];
  auto clear = [&] {
#pragma unroll
    for (int k = 0; k < E; ++k) sum[k] = 0.0f;
  };
  auto finish = [&](int key) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int unit = first_unit + i * a.lanes;
      if (unit < a.units) finish_unit<DT, VEC>(a, key, static_cast<int64_t>(unit) * VEC, sum + i * VEC);
    }
  };
  auto keep = [&](float* to) {
#pragma unroll
    for (int k = 0; k < E; ++k) to[k] = sum[k];
  };
  if (j0 < j1 && first_unit < a.units) {
    const GT* dy = static_cast<const GT*>(a.dy) + static_cast<int64_t>(first_unit) * VEC;
    int run = keys[j0];  // the token being summed
    bool began = keys[j0 - 1] == run;
    clear();
    for (int j = j0; j < j1 && run < a.vocab; j += AHEAD) {
      Unit<GT, VEC> u[AHEAD][U];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (j + i >= j1 || keys[j + i] >= a.vocab) continue;
        const GT* row = dy + positions[j + i - c0] * a.lddy;
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (U == 1 || first_unit + k * a.lanes < a.units) u[i][k] = load_unit_once<GT, VEC>(row + k * a.lanes * VEC);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (j + i >= j1) continue;
        const int key = keys[j + i];
        if (key != run) {  // the run ended before this position
          if (began) keep(first);
          else finish(run);
          run = key;
          began = false;
          clear();
          if (run >= a.vocab) break;  // only tokens without a row follow
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          float f[VEC];
          unpack<GT, VEC>(u[i][k], f);
#pragma unroll
          for (int l = 0; l < VEC; ++l) sum[k * VEC + l] += f[l];
        }
      }
    }
    if (run < a.vocab) {
      if (began) keep(first);  // (and may go on)
      else if (keys[j1] == run) keep(last);
      else finish(run);
    }
  }
  __syncthreads();
  // the pieces' open runs, in order: a worker's threads again
  if (worker != 0 || first_unit >= a.units) return;
  auto leave = [&](float* part) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int unit = first_unit + i * a.lanes;
      if (unit >= a.units) continue;
      float f[VEC];
#pragma unroll
      for (int l = 0; l < VEC; ++l) f[l] = sum[i * VEC + l];
      store_unit<float, VEC>(part + static_cast<int64_t>(unit) * VEC, f);
    }
  };
  float* part = a.part + static_cast<int64_t>(chunk) * 2 * a.d;
  bool before = true;  // the run that is open began before the chunk
  clear();
  int p0 = c0;
  for (int w = 0; w < workers && p0 < c1; ++w) {
    const int p1 = min(p0 + a.each, c1);
    const int head = keys[p0], tail = keys[p1 - 1];
    if (head >= a.vocab) break;
    const bool began = keys[p0 - 1] == head, goes_on = keys[p1] == tail && tail < a.vocab;
    const int at = (w * a.lanes + lane) * E;
    if (began) {
#pragma unroll
      for (int k = 0; k < E; ++k) sum[k] += open[0][at + k];
      if (head != tail || !goes_on) {  // it ends here
        if (before) leave(part);
        else finish(head);
        before = false;
      }
    }
    if (goes_on && !(began && head == tail)) {  // a run begins that goes on
#pragma unroll
      for (int k = 0; k < E; ++k) sum[k] = open[1][at + k];
      before = false;
    } else if (!goes_on) {
      clear();
    }
    if (p1 == c1 && goes_on) leave(part + (before ? 0 : a.d));
    p0 = p1;
  }
}

// Runs over several chunks: a thread a unit for each chunk in which one begins
// that goes on past it.
template <class DT, int VEC>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const __grid_constant__ SumArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kSumThreads + threadIdx.x;
  const int chunk = static_cast<int>(at / a.units);
  if (chunk >= a.chunks - 1) return;
  const int64_t col = at % a.units * VEC;
  const int begin = chunk * a.chunk, end = begin + a.chunk;  // below n: another chunk follows
  const int run = a.sorted[end].x, tail = a.sorted[end - 1].x, head = a.sorted[begin].x;
  const int prior = begin > 0 ? a.sorted[begin - 1].x : -1;
  if (run >= a.vocab || tail != run) return;
  if (head == run && prior == run) return;  // began before
  const int64_t pitch = 2 * static_cast<int64_t>(a.d);
  const float* part = a.part + chunk * pitch + col;
  float sum[VEC];
  unpack<float, VEC>(load_unit<float, VEC>(part + a.d), sum);
  // each chunk whose first key is the run's adds its first run; keys and sums of
  // eight chunks at once
  for (int c = chunk + 1; c < a.chunks; c += 8) {
    int key[8];
    Unit<float, VEC> u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) key[i] = c + i < a.chunks ? a.sorted[(c + i) * a.chunk].x : INT_MAX;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (key[i] == run) u[i] = load_unit<float, VEC>(part + (c + i - chunk) * pitch);
    bool more = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      more = more && key[i] == run;
      if (!more) continue;
      float f[VEC];
      unpack<float, VEC>(u[i], f);
#pragma unroll
      for (int k = 0; k < VEC; ++k) sum[k] += f[k];
    }
    if (!more) break;
  }
  finish_unit<DT, VEC>(a, run, col, sum);
}

// A bf16 dW from the fp32 sums of several calls' worth of tokens.
__global__ void __launch_bounds__(256) embed_round_kernel(const float* __restrict__ sums, bf16* __restrict__ dw,
                                                          int64_t lddw, int64_t rows, int d) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t step = gridDim.x * static_cast<int64_t>(256);
  for (int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x; i < rows * d; i += step)
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
    const int lanes = lanes_for(units);
    const int64_t slice = static_cast<int64_t>(lanes) * kLookupUnits<decltype(w), kVec>;
    const int64_t slices = (units + slice - 1) / slice;
    const LookupArgs a{e.tokens, e.ignore_index,         e.W,   e.ldw,
                       e.Y,      e.ldy,                  e.V,   static_cast<int>(e.T),
                       static_cast<int>(units), lanes, static_cast<int>(slices), e.scale};
    const int64_t blocks = (e.T * slices + kLookupThreads / lanes - 1) / (kLookupThreads / lanes);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    return launch_dependent(embed_lookup_kernel<decltype(w), decltype(y), kVec>, static_cast<unsigned>(blocks),
                            kLookupThreads, stream, a);
  });
  return err == cudaSuccess ? DGL_OK : DGL_ERR_CUDA;
}

constexpr int kMostSms = 160;  // workspaces are sized for this many

struct GradLayout {
  int64_t sorted = 0, part = 0, present = 0, sums = 0, bytes = 0;
  int each = 0;  // positions that a worker sums
};

// Positions that a worker sums: 8, or as many more as leave about 1500 threads an SM.
int each_for(int64_t n, int64_t d, int64_t size) {
  const int64_t threads = n * round_up(d * size, 16) / 16;
  return static_cast<int>(std::min<int64_t>(64, std::max<int64_t>(8, round_up(threads / (152 * 1500), 8))));
}

GradLayout grad_layout(const dgl_embed_desc& e) {
  GradLayout l;
  const int64_t n = std::min(e.T, kSortMost);
  l.each = each_for(n, e.d, size_of(e.y_dtype));
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at = round_up(at + bytes, 256);
    return here;
  };
  l.sorted = take(n * 8);
  // (a block has the fewest workers when they are whole warps)
  const int64_t chunk = static_cast<int64_t>(l.each) * (kSumThreads / 32);
  l.part = take((n + chunk - 1) / chunk * 2 * e.d * 4);
  l.present = take((e.V + 32 * 32 * kMostSms) / 8);  // (ranges are whole words)
  if (e.T > kSortMost && e.w_dtype == DGL_OUT_BF16) l.sums = take(e.V * e.d * 4);
  l.bytes = at;
  return l;
}

constexpr int64_t kZeroBytes = int64_t(20) << 20;      // zeros written beside the sort (40 or 64 MB: 4% slower)
constexpr int64_t kZeroBlockBytes = int64_t(64) << 10;  // and by a block beside the sums
constexpr int64_t kPrefetchBytes = int64_t(80) << 20;  // of dY that L2 keeps until the sums

template <int EACH>
cudaError_t launch_sort(const SortArgs& a, int ctas, int helpers, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int kBytes = static_cast<int>(sizeof(SortShared)) + EACH * kSortThreads * 8;
  const cudaError_t err = set_smem_attr_once(embed_sort_kernel<EACH>, kBytes, done);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas + helpers));  // (whole clusters)
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
  const int64_t size = size_of(e.w_dtype), y_size = size_of(e.y_dtype);
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
  sort.element = static_cast<int>(dw_size);
  sort.present = reinterpret_cast<uint32_t*>(ws + lay.present);
  int64_t t0 = 0;
  do {
    const int n = static_cast<int>(std::min(kSortMost, e.T - t0));
    const bool dense = t0 == 0 && !e.accumulate;
    sort.tokens = e.tokens + t0;
    sort.n = n;
    sort.sorted = reinterpret_cast<int2*>(ws + lay.sorted);
    sort.dw = dense ? dw : nullptr;
    const int ctas = n > kSortFew ? kSortCtas : 1;
    const int others = std::max(1, (ds->num_sms - ctas) / ctas) * ctas;  // CTAs that do not sort
    sort.share = static_cast<int>(round_up((e.V + others - 1) / others, 32));
    // zeros for the time of the sort; without a next kernel, all of them
    const int64_t now = n > 0 ? kZeroBytes / (others * sort.row_bytes) : sort.share;
    sort.quota = static_cast<int>(std::min<int64_t>(sort.share, round_up(now, 32)));
    sort.dy = static_cast<const uint8_t*>(e.dY) + t0 * e.ldy * y_size;
    sort.dy_pitch = e.ldy * y_size;
    sort.dy_bytes = n * e.d * y_size <= kPrefetchBytes ? e.d * y_size : 0;
    const int helpers = dense || (sort.dy_bytes > 0 && n > kSortFew) ? others : 0;
    const int each = (n + ctas * kSortThreads - 1) / (ctas * kSortThreads);
    const cudaError_t err = each <= 1   ? launch_sort<1>(sort, ctas, helpers, stream)
                            : each <= 2 ? launch_sort<2>(sort, ctas, helpers, stream)
                            : each <= 4 ? launch_sort<4>(sort, ctas, helpers, stream)
                            : each <= 8 ? launch_sort<8>(sort, ctas, helpers, stream)
                                        : launch_sort<kSortMostEach>(sort, ctas, helpers, stream);
    if (err != cudaSuccess) return DGL_ERR_CUDA;
    if (n > 0) {
      const cudaError_t e2 = with_types(e.y_dtype, dw_type, vec, [&](auto g, auto w, auto v) {
        using G = decltype(g);
        using W = decltype(w);
        constexpr int kVec = decltype(v)::value;
        SumArgs a = {};
        a.sorted = sort.sorted;
        a.dy = static_cast<const G*>(e.dY) + t0 * e.ldy;
        a.lddy = e.ldy;
        a.dw = dw;
        a.lddw = lddw;
        a.part = reinterpret_cast<float*>(ws + lay.part);
        a.n = n;
        a.vocab = static_cast<int>(e.V);
        a.units = static_cast<int>(e.d / kVec);
        a.lanes = lanes_for(a.units);
        const int workers = kSumThreads / a.lanes;
        a.each = std::min(lay.each, kMostChunk / workers);
        a.chunk = a.each * workers;
        a.chunks = (n + a.chunk - 1) / a.chunk;
        a.d = static_cast<int>(e.d);
        const int slice = a.lanes * kSumUnits<G, kVec>;
        a.slices = (a.units + slice - 1) / slice;
        a.scale = e.scale;
        a.add = dense ? 0 : 1;
        if (dense && sort.quota < sort.share) {
          a.present = sort.present;
          a.range_words = sort.share / 32;
          a.quota_words = sort.quota / 32;
          a.words = static_cast<int64_t>(helpers) * (a.range_words - a.quota_words);
          a.words_each = static_cast<int>(std::max<int64_t>(1, kZeroBlockBytes / (32 * sort.row_bytes)));
          a.zero_blocks = static_cast<int>((a.words + a.words_each - 1) / a.words_each);
        }
        const int64_t grid = static_cast<int64_t>(a.chunks) * a.slices + a.zero_blocks;
        const int64_t join = (static_cast<int64_t>(a.chunks - 1) * a.units + kSumThreads - 1) / kSumThreads;
        if (grid > INT32_MAX || join > INT32_MAX) return cudaErrorInvalidValue;
        const cudaError_t e3 =
            launch_dependent(embed_sum_kernel<G, W, kVec>, static_cast<unsigned>(grid), kSumThreads, stream, a);
        if (e3 != cudaSuccess || a.chunks < 2) return e3;
        return launch_dependent(embed_join_kernel<W, kVec>, static_cast<unsigned>(join), kSumThreads, stream, a);
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
