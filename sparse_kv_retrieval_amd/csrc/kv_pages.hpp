// Argument blocks and launchers of what moves pages and tokens of the paged KV cache: lsa_kv_kept, lsa_kv_compact,
// lsa_kv_extend, lsa_kv_fork and lsa_kv_free.
#pragma once

#include "kv.hpp"

namespace lsa {

constexpr int KV_LAYERS = 16;  // layers of one launch: their pointers are kernel arguments

// ---------------------------------------------------------------- compaction
struct CompactLayer {
  const char *k, *v;
  const float *k_scale, *v_scale;
  char *to_k, *to_v;
  float *to_k_scale, *to_v_scale;
};

// One side's places: see KvView.
struct PageMap {
  const int32_t* table;
  int64_t table_stride;
  int32_t n_pages, pt_log2;
};

// Which tokens are kept.
struct KeptArgs {
  PageMap from;
  const int32_t* kv_len;
  const int32_t* idx;
  const int64_t* idx_offsets;
  const int32_t* count;
  int32_t B, r, window, sinks;
};

struct CompactArgs {
  KeptArgs what;
  PageMap to;
  int32_t max_kept, n_kv;
  int32_t pages;             // destination pages of a sequence that the launch looks at
  int32_t groups, per_group; // blocks of a page, and the (layer, K or V, head) tiles of each
  int32_t tiles;             // L * 2 * n_kv
  CompactLayer layer[KV_LAYERS];
};

hipError_t launch_kv_kept(const KeptArgs& a, int32_t* kept, hipStream_t s);
hipError_t launch_kv_compact(const CompactArgs& a, bool fp8, int d, hipStream_t s);

// ---------------------------------------------------------------- the pool
struct PoolArgs {
  int32_t* refs;
  int32_t* table;
  int32_t* kv_len;
  int64_t table_stride;
  int32_t B, n_pages, pt_log2;
};

// What lsa_kv_fork's kernels tell one another about a pair.
struct ForkPair {
  int32_t tail;      // used slots of the last page that are to be copied; -1: the pair was refused
  int32_t src_page;  // from here
  int32_t dst_page;  // to here; -1: nothing is copied
  int32_t unused;
};

struct ForkLayer {
  char *k, *v;
  float *k_scale, *v_scale;
};
struct ForkCopyArgs {
  const ForkPair* pairs;
  int32_t n_kv, pt_log2, row_bytes;
  ForkLayer layer[KV_LAYERS];
};

constexpr int POOL_MAX = 4096;  // sequences of a pool, and pairs or sequences of one call

hipError_t launch_kv_extend(const PoolArgs& p, const int32_t* n_new, int32_t* missing, hipStream_t s);
hipError_t launch_kv_fork(const PoolArgs& p, int n, const int32_t* src, const int32_t* dst, int32_t* status, ForkPair* pairs,
                          hipStream_t s);
hipError_t launch_kv_fork_copy(const ForkCopyArgs& a, int n, int layers, hipStream_t s);
hipError_t launch_kv_free(const PoolArgs& p, int n, const int32_t* seqs, hipStream_t s);

}  // namespace lsa
