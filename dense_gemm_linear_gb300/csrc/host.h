// Host-side state and helpers shared by the C entry points: per-device
// state, the GEMM problem and its dispatch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "dgl.h"

namespace dgl {

constexpr int kMaxDevices = 64;

struct DeviceState {
  bool ready = false;
  int num_sms = 0;
  int cc_major = 0, cc_minor = 0;
  int smem_optin = 0;
  int* status = nullptr;  // device address of the status word on this device
};

// The current device's state; DGL_ERR_UNSUPPORTED when it is not sm_103.
dgl_status get_device(int* dev_out, DeviceState** st_out);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Problem {
  int dtype, out;
  const void *A, *B;
  const float *sa, *sb;
  void* C;
  int64_t M, N, K, m, n;
  // linear-layer epilogue (dgl_linear): bias per column, activation, gated up projection
  const float* bias = nullptr;
  int act = 0;
  int gated = 0;
  // operand layouts (dgl_gemm_bf16_ex): MN-major A is [K][m], B is [K][n];
  // lda / ldb are row pitches in elements (0: the packed pitch)
  int a_mn = 0;
  int b_mn = 0;
  int64_t lda = 0;
  int64_t ldb = 0;
  // W4A8 (dgl_gemm_w4a8): dtype E4M3 for A, B holds packed E2M1 codes (K / 2
  // bytes a row)
  int w4 = 0;
  // programmatic dependent launch mode of the kernel (PDL_*; dgl_gemm_batch)
  int pdl_mode = PDL_SERIAL;
  // rows of an MN-major B that exist (0: K): K may be rounded up past them to
  // whole 16-byte units of A's rows, and the rows in between read as zeros
  int64_t b_k = 0;
  // 1: K need not be whole 16-byte units (both operands MN-major: K is their
  // outer extent, and rows past it read as zeros)
  int k_any = 0;
  // bf16 operands, a TMA-stored C on 128- or 256-wide tiles: factor of every
  // element (device scalar); else null
  const float* out_scale = nullptr;
  // (the next three with out_scale only)
  // 1: A's box holds only the rows that exist when those are fewer than the tile's
  int tight_a = 0;
  // > 1: the sum over K in this many ranges, each with an fp32 C of its own:
  // tile-aligned slabs of rows (ceil(m / tile_m) tile_m) one after another
  int k_splits = 0;
  // 1: no split schedule, whose workspace the library would allocate
  int no_split = 0;
  // 1: add the product to C instead of replacing it (fp32 C whose rows are
  // whole 16-byte units; the TMA stores do the addition)
  int c_add = 0;
};

// Partial tiles and flags of a split schedule: flags zero before a launch, and
// zero again after it.
struct SplitScratch {
  float* ws = nullptr;
  size_t ws_bytes = 0;
  int* flags = nullptr;
  int nflags = 0;
};

// Validates, plans and enqueues one bf16 / E4M3 / W4A8 GEMM.  scratch: where
// a split schedule keeps its partial tiles (null: the stream's own workspace).
dgl_status run(const Problem& pr, const dgl_plan_info* forced, cudaStream_t stream,
               const SplitScratch* scratch = nullptr);

// Tensor maps of a K-major bf16 operand (128-byte boxes of box_rows rows) and
// of a 16-bit output (32 x 32 boxes), from the cache.
bool bf16_operand_map(CUtensorMap* map, const void* base, int64_t inner, int64_t rows, int box_rows, int64_t pitch);
bool bf16_output_map(CUtensorMap* map, void* base, int64_t cols, int64_t rows, int64_t ldc);

}  // namespace dgl
