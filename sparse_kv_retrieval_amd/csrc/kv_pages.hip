// lsa_kv_extend, lsa_kv_fork and lsa_kv_free: pages of a pool taken, shared and given back.
//
// A page is free when no entry of the table holds it (refs <= 0), and the free pages with the lowest numbers are taken first.
// So refs, table and lengths are the whole state: there is no list of free pages to keep in order, counts are sums
// and do not depend on the order of their atomics, and the pages that a call takes depend on the state alone. The price is a
// search of refs, 4 bytes a page, by one block of 1024 threads: 16,384 pages a round trip to memory, and none where no
// sequence crosses the end of a page. It begins at page 0, so it grows with the pages in use: where only the last ones are free, extend
// takes 13, 29 and 96 us over 30,000, 120,000 and 500,000 pages.
//
// Everything here is bound by latency: launches and a few dependent reads (length, table, refs). Giving back and sharing have one
// block per sequence, so that no two threads look at one entry; taking has one block, which needs no order between blocks.
// Measured on MI355X, the kernels alone: 8 sequences of up to 4096 tokens free 2.5, extend 6.1, fork 3.2 + 4.4 + 2.5 us (share, take, copy); 64 sequences,
// 16 of them admitted, eight samples each, over 29,177 pages 4.0, 9.9 and 4.9 + 6.0 + 3.7. A fork
// in one launch of one block was slower (11.9 against 7.2 us): the pairs' entries then have one CU's latency after another.
#include "kv_pages.hpp"

namespace lsa {

static constexpr int PG_THREADS = 256;    // of a block that goes through one sequence's entries
static constexpr int TAKE_THREADS = 1024; // of the block that takes pages
static constexpr int TAKE_WAVES = TAKE_THREADS / 64;
static constexpr int TAKE_CHUNK = 16 * TAKE_THREADS;  // pages looked at together
static constexpr int PER_THREAD = POOL_MAX / TAKE_THREADS;
static constexpr int TAKE_HELD = 8192;    // pages found before they are given out

__device__ __forceinline__ bool is_page(const PoolArgs& p, int32_t page) { return page >= 0 && page < p.n_pages; }

__device__ __forceinline__ int32_t held_len(const PoolArgs& p, int b) { return max(p.kv_len[b], 0); }
__device__ __forceinline__ int64_t pages_of(const PoolArgs& p, int64_t len) { return (len + (1 << p.pt_log2) - 1) >> p.pt_log2; }
// Entries of a row that hold its pages.
__device__ __forceinline__ int32_t held_entries(const PoolArgs& p, int b) {
  return (int32_t)min(pages_of(p, held_len(p, b)), p.table_stride);
}

// Whether x is among list[0 .. n - 1], for a whole block.
__device__ __forceinline__ bool block_has(const int32_t* list, int n, int32_t x) {
  bool hit = false;
  for (int i = threadIdx.x; i < n; i += PG_THREADS) hit |= list[i] == x;
  return __syncthreads_or(hit) != 0;
}

__global__ __launch_bounds__(PG_THREADS) void free_kernel(const PoolArgs p, const int32_t* seqs) {
  const int i = blockIdx.x, b = seqs[i];
  if (b < 0 || b >= p.B || block_has(seqs, i, b)) return;
  const int held = held_entries(p, b);
  int32_t* row = p.table + b * p.table_stride;
  for (int j = threadIdx.x; j < held; j += PG_THREADS) {
    const int32_t page = row[j];
    if (is_page(p, page)) atomicSub(p.refs + page, 1);
    row[j] = -1;
  }
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) p.kv_len[b] = 0;
}

// One pair: dst's pages back, src's full pages shared. The last page is left to take_tails_kernel.
__global__ __launch_bounds__(PG_THREADS) void share_kernel(const PoolArgs p, int n, const int32_t* src, const int32_t* dst, ForkPair* pairs) {
  const int i = blockIdx.x, s = src[i], t = dst[i];
  const bool bad = s < 0 || s >= p.B || t < 0 || t >= p.B;
  if (bad || block_has(src, n, t) || block_has(dst, i, t)) {
    if (threadIdx.x == 0) pairs[i] = {-1, -1, -1, 0};
    return;
  }
  const int held = held_entries(p, t);
  const int32_t len = (int32_t)min((int64_t)held_len(p, s), p.table_stride << p.pt_log2);
  const int full = len >> p.pt_log2, tail = len & ((1 << p.pt_log2) - 1);
  const int32_t* from = p.table + s * p.table_stride;
  int32_t* to = p.table + t * p.table_stride;
  const int end = max(held, full + (tail > 0));
  for (int j = threadIdx.x; j < end; j += PG_THREADS) {
    if (j < held) {
      const int32_t old = to[j];
      if (is_page(p, old)) atomicSub(p.refs + old, 1);
    }
    int32_t page = -1;
    if (j < full) {
      page = from[j];
      if (is_page(p, page)) atomicAdd(p.refs + page, 1);
      else page = -1;
    }
    to[j] = page;
  }
  __syncthreads();  // every thread has read dst's length
  if (threadIdx.x == 0) {
    // where src's last entry holds no page there is nothing to copy
    const int32_t last = tail > 0 ? from[full] : -1;
    const bool copies = is_page(p, last);
    pairs[i] = {copies ? tail : 0, last, -1, 0};
    p.kv_len[t] = copies ? full << p.pt_log2 : len;
  }
}

struct Two {
  int32_t a, b;
};
// Inclusive sums over the threads of a block of TAKE_THREADS, and the whole sums. `s_sums` is read until the next barrier of
// the caller's.
__device__ __forceinline__ Two block_scan(Two x, Two* s_sums, Two* total) {
  const int wave = threadIdx.x >> 6;
  x = {wave_scan(x.a), wave_scan(x.b)};
  if ((threadIdx.x & 63) == 63) s_sums[wave] = x;
  __syncthreads();
  Two all = {0, 0};
#pragma unroll
  for (int w = 0; w < TAKE_WAVES; ++w) {
    const Two y = s_sums[w];
    if (w < wave) x = {x.a + y.a, x.b + y.b};
    all = {all.a + y.a, all.b + y.b};
  }
  *total = all;
  return x;
}

// A chunk of pages is four runs of 4 * TAKE_THREADS; a thread has four pages of each, so that its neighbours' lie beside them. Which of
// them are free, four bits a run.
__device__ __forceinline__ uint32_t free_bits(const PoolArgs& p, int64_t chunk) {
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t base = chunk + 4 * ((int64_t)i * TAKE_THREADS + threadIdx.x);
    if (base + 4 <= p.n_pages) {
      const u32x4 r = *(const u32x4*)(p.refs + base);
#pragma unroll
      for (int e = 0; e < 4; ++e) bits |= ((int32_t)r[e] <= 0 ? 1u : 0u) << (4 * i + e);
    } else {
      for (int e = 0; e < 4 && base + e < p.n_pages; ++e) bits |= (p.refs[base + e] <= 0 ? 1u : 0u) << (4 * i + e);
    }
  }
  return bits;
}

// Looks for free pages from page *at on, whose chunk's bits are `next`, until `want` are found or all were looked at; the first TAKE_HELD
// of them go to s_ids, in ascending order. Returns how many there are (at most `want`); *at becomes the first page of the last chunk,
// where a search that goes on after those pages were taken begins.
__device__ __forceinline__ int32_t find_free(const PoolArgs& p, int64_t* at, uint32_t next, int32_t want, int32_t* s_ids, Two (*s_sums)[TAKE_WAVES]) {
  int64_t found = 0, chunk = *at;
  int turn = 0;
  const int32_t most = min(want, TAKE_HELD);
  for (; found < want && chunk < p.n_pages; chunk += TAKE_CHUNK, turn ^= 1) {
    *at = chunk;
    const uint32_t bits = next;
    // the next chunk is on its way while this one is counted
    next = free_bits(p, chunk + TAKE_CHUNK);
    // the runs' counts, two to a number: none is above 4 * TAKE_THREADS
    auto count = [&](int i) -> int32_t { return __popc(bits >> (4 * i) & 15); };
    const Two mine = {count(0) | count(1) << 16, count(2) | count(3) << 16};
    Two all;
    const Two upto = block_scan(mine, s_sums[turn], &all);
    const Two before = {upto.a - mine.a, upto.b - mine.b};
    const int32_t ends[4] = {all.a & 0xFFFF, all.a >> 16, all.b & 0xFFFF, all.b >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int64_t rank = found + ((i < 2 ? before.a : before.b) >> (16 * (i & 1)) & 0xFFFF);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (bits >> (4 * i + e) & 1) {
          if (rank < most) s_ids[rank] = (int32_t)(chunk + 4 * (i * TAKE_THREADS + (int)threadIdx.x) + e);
          ++rank;
        }
      found += ends[i];
    }
  }
  __syncthreads();  // s_ids is whole
  return (int32_t)min(found, (int64_t)want);
}

// Sequence i * TAKE_THREADS + (thread) is the thread's i-th. What all of them have beyond the first is skipped where there are few.
__global__ __launch_bounds__(TAKE_THREADS) void extend_kernel(const PoolArgs p, const int32_t* n_new, int32_t* missing) {
  __shared__ int32_t s_ids[TAKE_HELD], s_upto[POOL_MAX], s_have[POOL_MAX];
  __shared__ Two s_sums[2][TAKE_WAVES];
  __shared__ int32_t s_limit;
  constexpr int LOW = 18;  // bits of a sum that are added apart: TAKE_THREADS times 2^18 fits 32 bits
  int64_t total = 0;
  int32_t need[PER_THREAD] = {}, upto[PER_THREAD], after[PER_THREAD];  // pages, their sum up to here, the length with the new tokens
  bool fits[PER_THREAD];
#pragma unroll
  for (int i = 0; i < PER_THREAD; ++i) {
    if (i * TAKE_THREADS >= p.B) break;
    const int b = i * TAKE_THREADS + threadIdx.x;
    if (b < p.B) {
      const int64_t len = held_len(p, b), more = max(n_new[b], 0), have = pages_of(p, len), want = pages_of(p, len + more);
      fits[i] = more == 0 || (want <= p.table_stride && len + more <= INT32_MAX);
      after[i] = (int32_t)(fits[i] ? len + more : len);
      need[i] = fits[i] ? (int32_t)(want - have) : 0;
      s_have[b] = (int32_t)have;
    }
    Two all;
    const Two sum = block_scan({need[i] & ((1 << LOW) - 1), need[i] >> LOW}, s_sums[i & 1], &all);
    upto[i] = (int32_t)min(total + ((int64_t)sum.b << LOW) + sum.a, (int64_t)INT32_MAX);
    if (b < p.B) s_upto[b] = upto[i];
    total += ((int64_t)all.b << LOW) + all.a;
  }
  if (threadIdx.x == 0) s_limit = 0;
  __syncthreads();
  int64_t at = 0;
  int32_t found = 0;
  // all that are asked for, or all that there are: the number decides who gets any
  if (total > 0) found = find_free(p, &at, free_bits(p, 0), (int32_t)min(total, (int64_t)p.n_pages), s_ids, s_sums);
#pragma unroll
  for (int i = 0; i < PER_THREAD; ++i) {
    if (i * TAKE_THREADS >= p.B) break;
    const int b = i * TAKE_THREADS + threadIdx.x;
    if (b >= p.B) continue;
    const bool granted = need[i] == 0 || upto[i] <= found;
    if (granted && need[i] > 0 && upto[i] > s_limit) atomicMax(&s_limit, upto[i]);
    if (missing) missing[b] = !fits[i] ? -1 : granted ? 0 : need[i];
    if (granted && fits[i]) p.kv_len[b] = after[i];
  }
  if (total == 0) return;
  __syncthreads();
  const int32_t limit = s_limit;
  // s_ids holds the first of them; where there are more, the search goes on behind those that are taken by now
  if (found > TAKE_HELD) at = 0;
  for (int32_t done = 0; done < limit;) {
    const int32_t n = min(limit - done, TAKE_HELD);
    if (done > 0) find_free(p, &at, free_bits(p, at), n, s_ids, s_sums);
    constexpr int UN = 4;  // pages of a thread whose sequences are looked for side by side
    for (int32_t x0 = 0; x0 < n; x0 += UN * TAKE_THREADS) {
      int32_t seq[UN] = {};  // how many sequences end at or before the page's rank
#pragma unroll 1
      for (int step = POOL_MAX / 2; step; step >>= 1) {
        if (step >= p.B) continue;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          const int32_t rank = done + x0 + u * TAKE_THREADS + (int32_t)threadIdx.x;
          if (seq[u] + step < p.B && s_upto[seq[u] + step - 1] <= rank) seq[u] += step;
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int32_t x = x0 + u * TAKE_THREADS + (int32_t)threadIdx.x;
        if (x >= n) break;
        const int32_t page = s_ids[x], before = seq[u] > 0 ? s_upto[seq[u] - 1] : 0;
        p.refs[page] = 1;
        p.table[seq[u] * p.table_stride + s_have[seq[u]] + (done + x - before)] = page;
      }
    }
    done += n;
    __syncthreads();  // the counts are written before they are looked at again, and s_ids is read
  }
}

// The last pages of a fork: one page for each pair that copies, lowest first. Pairs lie in the threads as sequences do above.
__global__ __launch_bounds__(TAKE_THREADS) void take_tails_kernel(const PoolArgs p, int n, const int32_t* dst, int32_t* status, ForkPair* pairs) {
  __shared__ int32_t s_ids[POOL_MAX];  // every pair's page is held at once
  __shared__ Two s_sums[2][TAKE_WAVES];
  static_assert(TAKE_HELD >= POOL_MAX, "find_free fills no more than are wanted");
  const uint32_t front = free_bits(p, 0);  // asked for beside the pairs
  int32_t total = 0, found = 0, tail[PER_THREAD] = {}, rank[PER_THREAD];
#pragma unroll
  for (int i = 0; i < PER_THREAD; ++i) {
    if (i * TAKE_THREADS >= n) break;
    const int x = i * TAKE_THREADS + threadIdx.x;
    if (x < n) tail[i] = pairs[x].tail;
    Two all;
    const Two sum = block_scan({tail[i] > 0, 0}, s_sums[i & 1], &all);
    rank[i] = total + sum.a - 1;
    total += all.a;
  }
  __syncthreads();
  int64_t at = 0;
  if (total > 0) found = find_free(p, &at, front, total, s_ids, s_sums);
#pragma unroll
  for (int i = 0; i < PER_THREAD; ++i) {
    const int x = i * TAKE_THREADS + threadIdx.x;
    if (i * TAKE_THREADS >= n) break;
    if (x >= n) continue;
    int32_t st = tail[i] < 0 ? -1 : 0;
    if (tail[i] > 0 && rank[i] < found) {
      const int32_t page = s_ids[rank[i]], t = dst[x], len = p.kv_len[t];
      p.refs[page] = 1;
      p.table[t * p.table_stride + (len >> p.pt_log2)] = page;
      p.kv_len[t] = len + tail[i];
      pairs[x].dst_page = page;
    } else if (tail[i] > 0) {
      st = 1;
    }
    status[x] = st;
  }
}

// One pair, layer, K or V and head: the used slots of the last page are one run of bytes.
__global__ __launch_bounds__(PG_THREADS) void copy_tails_kernel(const ForkCopyArgs a) {
  const ForkPair pair = a.pairs[blockIdx.x];
  if (pair.dst_page < 0) return;
  const int h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const ForkLayer& l = a.layer[blockIdx.z];
  char* base = is_v ? l.v : l.k;
  float* scale = is_v ? l.v_scale : l.k_scale;
  const int64_t from = (int64_t)pair.src_page * a.n_kv + h, to = (int64_t)pair.dst_page * a.n_kv + h;
  const u32x4* in = (const u32x4*)(base + (from << a.pt_log2) * a.row_bytes);
  u32x4* out = (u32x4*)(base + (to << a.pt_log2) * a.row_bytes);
  const int units = pair.tail * (a.row_bytes / 16);
  for (int i = threadIdx.x; i < units; i += PG_THREADS) out[i] = in[i];
  if (scale && threadIdx.x == 0) scale[to] = scale[from];
}

hipError_t launch_kv_extend(const PoolArgs& p, const int32_t* n_new, int32_t* missing, hipStream_t s) {
  extend_kernel<<<1, TAKE_THREADS, 0, s>>>(p, n_new, missing);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const PoolArgs& p, int n, const int32_t* src, const int32_t* dst, int32_t* status, ForkPair* pairs,
                          hipStream_t s) {
  share_kernel<<<n, PG_THREADS, 0, s>>>(p, n, src, dst, pairs);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  take_tails_kernel<<<1, TAKE_THREADS, 0, s>>>(p, n, dst, status, pairs);
  return hipGetLastError();
}

hipError_t launch_kv_fork_copy(const ForkCopyArgs& a, int n, int layers, hipStream_t s) {
  copy_tails_kernel<<<dim3(n, 2 * a.n_kv, layers), PG_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_free(const PoolArgs& p, int n, const int32_t* seqs, hipStream_t s) {
  free_kernel<<<n, PG_THREADS, 0, s>>>(p, seqs);
  return hipGetLastError();
}

}  // namespace lsa
