// Argument blocks, launchers and device helpers of the paged KV cache: lsa_kv_append,
// lsa_attend and lsa_attend_topk.
#pragma once

#include "common.hpp"

namespace lsa {

// The cache as the kernels see it. Page p, key head h is one contiguous tile of page_tokens
// rows: row number (p * n_kv + h) * page_tokens + slot. Scales are per tile (FP8 only).
struct KvView {
  char* k;
  char* v;
  float* k_scale;
  float* v_scale;
  const int32_t* table;   // [B][table_stride]
  const int32_t* kv_len;  // [B]
  int64_t table_stride;
  int32_t n_pages, n_kv, pt_log2;
};

struct AppendArgs {
  KvView c;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const uint16_t* q;      // or null
  uint16_t* q_out;
  int64_t k_stride, v_stride, q_stride;
  const int64_t* off;     // [B+1]
  const int32_t* positions;
  const float* inv_freq;  // [rot / 2], or null: no rotation
  int64_t first_row, T;   // off[0] and the number of new tokens
  int64_t page_slots;     // see append_page_slots()
  int32_t B, n_q, rot;
};

// Sequence b's new tokens touch at most (n_b - 1) / pt + 2 pages. Page slots are numbered
// (off[b] - off[0]) / pt + 2 b + j, which leaves every sequence that many and lets a wave find
// its sequence from the offsets alone.
inline int64_t append_page_slots(int64_t T, int32_t B, int32_t pt) { return T / pt + 2 * (int64_t)B; }

// Work of one attention launch. Rows of a sequence are its (new token, query head of the group)
// pairs, row = token * G + head; a row block is M of them for one key head. The keys that a row
// block sees are numbered in tiles of 32 (first tokens, then the window; listed entries last) and
// split in runs of `run` tiles; partial results of several runs are joined by a second launch.
struct AttendArgs {
  KvView c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;             // or null
  int64_t q_stride, out_stride;
  const int64_t* off;     // [B+1], or null: one row each (lsa_attend_topk)
  const int32_t* idx;     // [B][k] listed entries, or null
  const int32_t* count;   // [B]
  float* part_o;          // [splits][T][n_q][D]
  float* part_ml;         // [splits][T][n_q][2]: running maximum (base 2) and sum
  int64_t first_row, T;
  int64_t blocks;         // row-block slots
  float scale_log2;       // softmax scale * log2(e)
  int32_t B, n_q, G, max_kv_len, window, sinks, k, r;
  int32_t splits, run;
};

// Tiles of 32 tokens that the rows at positions p_lo..p_hi see. Tile i < n_first is tile i of the
// sequence, tile i >= n_first is tile first_b + i - n_first.
struct TileRange {
  int32_t n_first, first_b, n;
  __device__ __forceinline__ int32_t tile(int32_t i) const { return i < n_first ? i : first_b + (i - n_first); }
};

__host__ __device__ __forceinline__ TileRange tile_range(int32_t p_lo, int32_t p_hi, int32_t window, int32_t sinks) {
  TileRange t{0, 0, 0};
  if (p_hi < 0) return t;
  const int32_t end = p_hi / 32 + 1;
  if (window > 0) {
    const int32_t s = sinks / 32 + (sinks % 32 != 0);
    t.n_first = s < end ? s : end;
    const int32_t lo = p_lo - window + 1;  // p_lo >= -2^31 + window fits: both are at most 2^31 - 1
    t.first_b = lo > 0 ? lo / 32 : 0;
    if (t.first_b < t.n_first) t.first_b = t.n_first;
  }
  t.n = t.n_first + (end > t.first_b ? end - t.first_b : 0);
  return t;
}

constexpr int ATTEND_MAX_RUN = 64;         // tiles of one split
constexpr int ATTEND_MAX_RUN_LISTED = 16;  // the same over listed keys, each with a place of its own in LDS

hipError_t launch_kv_append(const AppendArgs& a, bool fp8, int d, int style, hipStream_t s);
hipError_t launch_attend_split(const AttendArgs& a, bool fp8, int d, int row_tiles, bool listed, hipStream_t s);
hipError_t launch_attend_join(const AttendArgs& a, int d, int row_tiles, bool listed, hipStream_t s);

// Largest b in [0, B) with slot(b) <= x, for slot strictly increasing and slot(0) <= x: the lanes
// of a wave try 64 places at a time.
template <typename F>
__device__ __forceinline__ int wave_find(int B, int64_t x, F slot) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 63) >> 6;
    const int at = lane * step;
    const uint64_t le = __ballot(at < n && slot(lo + (at < n ? at : 0)) <= x);
    const int c = __popcll(le) - 1;
    lo += c * step;
    n = min(step, n - c * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Maximum and sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48 (one column of a 16x16 tile).
__device__ __forceinline__ float max_column(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_column(float x) {
  x = sum_halves(x);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
// Two floats to packed bf16, to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

}  // namespace lsa
