// The tensor-core forward (fwd_tc.cu) as attn_fwd and the long segments of
// attn_kv_fwd call it.
#pragma once

#include "common.cuh"

namespace attn {

// Segments given by first row and length instead of offsets (group mode): row
// arrays of `batch` entries on the device.  Their query tiles pack the heads of a
// group (rows = token x head), at most 128 of them, and the keys of a tile may be
// split over CTAs, whose parts a second kernel joins.
struct FwdSegments {
  const int* zeros;
  const int* len_q;
  const int* start_q;
  const int* len_k;
  const int* start_k;
  int nsplit;              // most splits of a tile's keys
  // where nsplit > 1: per split and part row, which is a row of q, or where slot_rows
  // is not 0 token + slot_rows x segment
  long long part_rows, slot_rows;
  float* part_o;           // [nsplit][part_rows][nhead_q][d_v]
  float2* part_ml;         // [nsplit][part_rows][nhead_q]: running maximum (log2 units) and sum
  int* status;             // ATTN_ERR_TIMEOUT where a wait ran out (its rows are NaN)
};
constexpr int FWD_TILE_ROWS = 128;   // query rows of a tile of the tensor-core forward, and keys
constexpr int FWD_MIN_SPLIT = 8;     // key tiles of a split at least
// Tensor-core forward (fwd_tc.cu); ATTN_ERR_UNSUPPORTED_HEADDIM for the
// dtypes, head dims and scales it is not built for.  `seg` replaces the cu_seqlens of p.
int launch_fwd_tc(const attn_fwd_params& p, const FwdLayout& L, cudaStream_t st, const FwdSegments* seg = nullptr);

}  // namespace attn
