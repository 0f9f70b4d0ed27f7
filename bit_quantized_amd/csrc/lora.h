// Host-side interface of the adapter linear (lora.hip), for rows_abi.hip.
#pragma once

#include "rows.h"

namespace w4a8 {

struct LoraArgs {
  const void* x;
  int x_dtype;
  PackedView w;
  const uint16_t *A, *B;
  const float* scale;
  const int* ids;
  int64_t M, N, K;
  int L, R;
  uint16_t* y;
  uint8_t* ws;
};

// How a pass of at most `rows` rows runs, and its buffers in the workspace.
struct LoraPlan {
  int64_t rows = 0;
  int path = 0;       // RowPath of the shared product (one row: the M = 1 GEMV)
  bool gemv = false;
  int mt = 0;      // 16-row tiles of the streaming kernel; 0: the 256-row tile kernel
  int kw = 0;      // streaming kernel: log2 wavefronts per column
  int ksplit = 1;  // K slices across workgroups (float sums, then a reduction)
  bool sorted = false;  // rows taken in the order of their adapters
  int slots = 1;   // workgroups that share a 16-row fragment's adapters
  int slices = 1;  // K slices of x A^T
  int64_t qa = 0, sa = 0, hx = 0, order = 0, hi = 0, lo = 0, parts = 0;
  int64_t bytes = 0;
};

LoraPlan lora_plan(int64_t M, int64_t N, int64_t K, int L, int R);
// Bytes that the plans of every row count up to M fit in.
int64_t lora_workspace(int64_t M, int64_t N, int64_t K, int L, int R);
hipError_t launch_lora(const LoraArgs& l, const LoraPlan& p, hipStream_t st);

}  // namespace w4a8
