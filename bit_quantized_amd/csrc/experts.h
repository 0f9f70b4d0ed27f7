// Host-side interface of the expert MLP (experts.hip), for rows_abi.hip.
#pragma once

#include "rows.h"

namespace w4a8 {

constexpr int kMaxExperts = 1024;

struct MoeArgs {
  const void* x;
  int x_dtype;
  PackedView up, down;
  const int* ids;
  const float* weights;
  int64_t M;
  int k, E;
  int64_t I, K;
  uint16_t* y;
  uint8_t* ws;
};

// Tokens per pass and the byte offsets of a pass's buffers in the workspace.
struct MoePlan {
  int64_t tokens = 0;
  bool direct = false;
  int bm = 0;            // rows a tile holds
  int up = 0, down = 0;  // RowPath of the products
  bool raw = false;      // the down product quantises its rows itself
  int64_t qa = 0, sa = 0, count = 0, tiles = 0, list = 0, rank = 0, counts = 0, h = 0, hq = 0, hs = 0, parts = 0;
  int64_t bytes = 0;
};

MoePlan moe_plan(int64_t M, int k, int E, int64_t I, int64_t K);
// Consecutive columns that a wavefront of the down product takes in a pass of
// P pairs (not for the 256-row tiles).
int down_columns(const MoePlan& p, int64_t P, int E, int64_t I, int64_t K);
// One pass of at most p.tokens tokens.
hipError_t launch_moe(const MoeArgs& m, const MoePlan& p, hipStream_t st);

}  // namespace w4a8
