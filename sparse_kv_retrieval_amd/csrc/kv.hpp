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
// pairs, row = token * G + head; a row block is up to M of them for one key head. The keys that a row
// block sees are numbered in tiles (first tokens, then the window; listed entries last). A launch works
// on the sequences with more than rows_above and at most rows_to rows.
struct AttendArgs {
  KvView c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;             // or null
  int64_t q_stride, out_stride;
  const int64_t* off;     // [B+1], or null: one row each (lsa_attend_topk)
  const int32_t* idx;     // [B][k] listed entries, or null
  const int32_t* count;   // [B]
  int64_t first_row, T;
  float scale_log2;       // softmax scale * log2(e)
  int32_t B, n_q, G, max_kv_len, window, sinks, k, r;
  int64_t rows_above, rows_to;
  float* part_o;          // partial results of row blocks whose keys are split
  float* part_ml;         // and their running maximum (base 2) and sum
  // Tile kernel: a row block's keys are split in runs of `run` tiles; partials [splits][T][n_q][D].
  int64_t blocks;         // row-block slots
  int32_t splits, run;
  // Split kernel: the tiles of all row blocks of a key head, one after the other, are shared evenly by
  // `workers` blocks (0: each row block has a worker of its own). A worker's part of a row block goes to
  // partials [part_slot()][n_kv][M][D], and joins[row block][n_kv] says which workers took part.
  int32_t entries, per;   // row blocks, and how many of them a sequence has (LISTED)
  int32_t workers;
  int32_t* joins;         // pairs: first worker, number of parts (0: written whole)
};

// Where the part goes that `worker` has of row block `entry`, which worker `owner` begins. From a part to the next one the
// worker grows (the same row block), or the row block does, and with it the owner: only the last row block that a
// worker begins can have several parts. So neither sum is met twice; the one that needs less room is taken.
__device__ __forceinline__ int32_t part_slot(const AttendArgs& a, int32_t worker, int32_t entry, int32_t owner) {
  return worker + (a.entries < a.workers ? entry : owner);
}

// Tiles of `tile` tokens that the rows at positions p_lo..p_hi see. Tile i < n_first is tile i of the
// sequence, tile i >= n_first is tile first_b + i - n_first.
struct TileRange {
  int32_t n_first, first_b, n;
  __device__ __forceinline__ int32_t tile(int32_t i) const { return i < n_first ? i : first_b + (i - n_first); }
};

template <int tile>
__device__ __forceinline__ TileRange tile_range(int32_t p_lo, int32_t p_hi, int32_t window, int32_t sinks) {
  TileRange t{0, 0, 0};
  if (p_hi < 0) return t;
  const int32_t end = (int32_t)((uint32_t)p_hi / tile) + 1;
  if (window > 0) {
    const int32_t s = (int32_t)((uint32_t)sinks / tile) + (sinks % tile != 0);
    t.n_first = s < end ? s : end;
    const int32_t lo = max(p_lo, 0) - window + 1;  // a row before the first cached token sees none
    t.first_b = lo > 0 ? (int32_t)((uint32_t)lo / tile) : 0;
    if (t.first_b < t.n_first) t.first_b = t.n_first;
  }
  t.n = t.n_first + (end > t.first_b ? end - t.first_b : 0);
  return t;
}

constexpr int ATTEND_TILE_ROWS = 256;       // rows of a block of the tile kernel
constexpr int ATTEND_TILE_KEYS = 64;        // keys of its tiles
constexpr int ATTEND_RESOLVED = 64;         // tiles whose places a block of the split kernel holds at once
constexpr int ATTEND_RESOLVED_LISTED = 16;  // the same over listed keys, each with a place of its own

// Blocks of the split kernel that a compute unit holds: what a lane keeps of its rows grows with their number and with
// the dimensions, and from 32 rows of 128 dimensions (or 64 of 64) on a wave needs a SIMD's registers.
constexpr int attend_split_blocks(int rows, int d) { return rows * d >= 32 * 128 ? 1 : 2; }

hipError_t launch_kv_append(const AppendArgs& a, bool fp8, int d, int style, hipStream_t s);
hipError_t launch_attend_split(const AttendArgs& a, bool fp8, int d, int row_tiles, bool listed, hipStream_t s);
hipError_t launch_attend_split_join(const AttendArgs& a, int d, int rows, bool listed, hipStream_t s);
hipError_t launch_attend_tile_join(const AttendArgs& a, int d, hipStream_t s);
hipError_t launch_attend_tile(const AttendArgs& a, bool fp8, int d, hipStream_t s);

// Largest b in [0, B) with slot(b) <= x, for slot non-decreasing and slot(0) <= x: the lanes of a wave try
// 64 places at a time.
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

// Inclusive sum over the lanes of a wave (DPP: within rows of 16, then across them), and its last lane's.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast 15 into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast 31 into rows 2 and 3
  return x;
}
__device__ __forceinline__ int wave_last(int x) { return __builtin_amdgcn_readlane(x, 63); }

// As __syncthreads() for what waves share in LDS, but loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

constexpr float ATTEND_LAZY = 8.0f;
constexpr float ATTEND_LOWEST = -3.402823466e38f;  // running maximum of a row that has seen nothing
constexpr float LN2 = 0.6931471805599453f;

// One row block: rows r0 .. r0 + n - 1 of sequence b for key head h.
struct Rows {
  int32_t b, n, r0;
  int32_t p0;          // position of the sequence's first query token (negative: it has fewer cached tokens)
  int32_t p_lo, p_hi;  // positions of the block's first and last row
  int32_t w_lo, w_hi;  // positions beyond these are in their windows
  int64_t t0;          // row number of the sequence's first token in q
  TileRange near;      // tiles seen by position
  int32_t tiles;       // those and the listed ones
  int32_t listed;      // listed entries
};

// The row at position p sees s <= p where s > window_start(a, p) or s < a.sinks.
__device__ __forceinline__ int32_t window_start(const AttendArgs& a, int32_t p) {
  return a.window > 0 && p >= a.window ? p - a.window : -1;
}

// Whether a launch works on sequences of n_tok new tokens.
__device__ __forceinline__ bool of_class(const AttendArgs& a, int64_t n_tok) {
  const int64_t rows = n_tok * a.G;
  return rows > a.rows_above && rows <= a.rows_to;
}

// What a row block's sequence brings: its new tokens, its cached tokens and (LISTED) its listed entries.
struct Seq {
  int32_t n_tok, len, listed;
  int32_t row;  // its first row, after first_row
};

template <bool LISTED>
__device__ __forceinline__ Seq seq_of(const AttendArgs& a, int b, int64_t row, int64_t n_tok) {
  return {(int32_t)n_tok, min(max(a.c.kv_len[b], 0), a.max_kv_len), LISTED ? min(max(a.count[b], 0), a.k) : 0,
          (int32_t)(row - a.first_row)};
}

// Rows r0 .. r0 + n - 1 of a sequence, whose first and last belong to new tokens `lo` and `hi`, and the tiles of TILE keys
// that they see by position.
template <int TILE>
__device__ __forceinline__ void set_rows(const AttendArgs& a, Seq s, int32_t r0, int32_t n, int32_t lo, int32_t hi, Rows* w) {
  w->r0 = r0;
  w->n = n;
  w->p0 = s.len - s.n_tok;
  w->p_lo = w->p0 + lo;
  w->p_hi = w->p0 + hi;
  w->w_lo = window_start(a, w->p_lo);
  w->w_hi = window_start(a, w->p_hi);
  w->near = tile_range<TILE>(w->p_lo, w->p_hi, a.window, a.sinks);
  w->tiles = w->near.n;
  w->listed = s.listed;
}

// Tile kernel: row block j of a sequence.
__device__ __forceinline__ void set_block(const AttendArgs& a, Seq s, int32_t j, Rows* w) {
  const int32_t r0 = j * ATTEND_TILE_ROWS, n = min(ATTEND_TILE_ROWS, s.n_tok * a.G - r0);
  set_rows<ATTEND_TILE_KEYS>(a, s, r0, n, r0 / a.G, (r0 + n - 1) / a.G, w);
}

// The fields that a block agrees on, in scalar registers.
__device__ __forceinline__ void pin_rows(Rows* w) {
  w->b = uni(w->b); w->n = uni(w->n); w->r0 = uni(w->r0); w->p0 = uni(w->p0); w->p_lo = uni(w->p_lo); w->p_hi = uni(w->p_hi);
  w->w_lo = uni(w->w_lo); w->w_hi = uni(w->w_hi); w->t0 = uni(w->t0); w->tiles = uni(w->tiles); w->listed = uni(w->listed);
  w->near.n_first = uni(w->near.n_first); w->near.first_b = uni(w->near.first_b); w->near.n = uni(w->near.n);
}

// Tile kernel: the row block of a slot (see AttendArgs::blocks), if it has rows.
__device__ __forceinline__ bool find_rows(const AttendArgs& a, int64_t block, Rows* w) {
  constexpr int M = ATTEND_TILE_ROWS;
  auto slot_of = [&](int x) -> int64_t { return (a.off[x] - a.first_row) * a.G / M + x; };
  w->b = wave_find(a.B, block, slot_of);
  w->t0 = a.off[w->b];
  const int64_t n_tok = a.off[w->b + 1] - w->t0, j = block - slot_of(w->b);
  if (j * M >= n_tok * a.G || !of_class(a, n_tok)) return false;
  set_block(a, seq_of<false>(a, w->b, w->t0, n_tok), (int32_t)j, w);
  pin_rows(w);
  return true;
}

// Split kernel: row block e is block e % per of sequence e / per (only LISTED sequences have several).
// Whether it has rows; its sequence.
template <bool LISTED>
__device__ __forceinline__ bool entry_seq(const AttendArgs& a, int e, Seq* s) {
  const int b = LISTED && a.per > 1 ? e / a.per : e;
  const int64_t row = LISTED ? b : a.off[b], n_tok = LISTED ? 1 : a.off[b + 1] - row;
  *s = seq_of<LISTED>(a, b, row, n_tok);
  if (!LISTED && !of_class(a, n_tok)) return false;
  return true;
}
template <bool LISTED>
__device__ __forceinline__ void set_entry(const AttendArgs& a, int e, Seq s, int M, Rows* w) {
  if constexpr (LISTED) {
    w->b = a.per == 1 ? e : e / a.per;
    const int32_t r0 = (e - w->b * a.per) * M;
    set_rows<32>(a, s, r0, min(M, a.G - r0), 0, 0, w);
    if (a.window == 0) {  // here no window is none, not all
      const int32_t end = w->p_hi < 0 ? 0 : (int32_t)((uint32_t)w->p_hi / 32) + 1;
      w->near.n_first = w->near.n = min((int32_t)((uint32_t)a.sinks / 32) + (a.sinks % 32 != 0), end);
      w->near.first_b = 0;
    }
    w->tiles = w->p_hi < 0 ? 0 : w->near.n + (int32_t)(((int64_t)s.listed * a.r + 31) / 32);
  } else {
    w->b = e;
    set_rows<32>(a, s, 0, s.n_tok * a.G, 0, s.n_tok - 1, w);
  }
  w->t0 = a.first_row + s.row;
}

// The elements of a dword that are not finite, as a mask over its bits.
template <bool FP8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  if constexpr (FP8) {
    const uint32_t hit = (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;  // code 7F or FF
    return hit * 0xFFu;
  } else {
    return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
  }
}

// Dimension d of a cached row, in units of its scale.
template <bool FP8>
__device__ __forceinline__ float cached_value(const char* row, int d) {
  if constexpr (FP8) {
    return __builtin_amdgcn_cvt_f32_fp8((int)*(const uint8_t*)(row + d), 0);
  } else {
    return bf16_bits_to_f32(*(const uint16_t*)(row + 2 * d));
  }
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
