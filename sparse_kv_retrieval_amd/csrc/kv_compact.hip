// lsa_kv_kept and lsa_kv_compact: listed tokens, window and first tokens of a paged cache, dense in other pages.
//
// Where a token goes. The list is ascending, so of its entries those at or below the last first token and those that reach into the
// window are its two ends: two searches find them, and between them every entry has entry_tokens tokens. Source and
// place of a kept token are then arithmetic, with no sum over the list.
//
// e4m3. The new page's scale is the least power of two that holds its largest value, as in an append. A value is rounded anew
// only where its old page's scale differs and the result is subnormal in e4m3, for scales that are powers of two.
//
// Shape. A block has one destination page of one sequence. It finds the page's tokens once, for all layers, heads, K and V;
// then each wave takes tiles (layer, K or V, head) in turn, whole in its registers between the maximum and the
// store, so that a wave waits for no other one. Tiles of a page are shared among blocks until some 8192 are there: the last of fewer,
// longer ones end the call alone, and each block finds its tokens anew. With 2048, 4096, 8192 and 16,384 (us, kept 13.5 %):
//   8 x 125,000 tokens, three layers, eight heads of 128   bf16 678, 641, 626, 636    e4m3 364, 347, 343, 343
//   32 x 4096 to 131,071, one layer, bf16                  245, 245, 237, 248
//   64 x 4000, three layers, pages of 16, e4m3             115, 112, 109, 116
//   1 x 125,000, three layers, e4m3                        50, 49, 49, 49
//   1 x 125,000, one layer, bf16; 32 ragged, two heads of 64, e4m3; 1 x 8000, 16 layers, bf16    all four within 3 %
//
// Bound by HBM: each kept row is read and written once, and nothing reads either again soon, so both go past the caches
// (non-temporal stores: 360 against 378 us). Measured on MI355X: the first of these shapes, 3.34 GB read and written in bf16 626 us (5.3 TB/s) and
// 1.67 in e4m3 343 to 347 (4.8 to 4.9; a copy of 1 GiB 5.1). One short sequence is bound by latency: the two ends,
// list, page and row are four to five dependent reads, 8 us.
#include "kv_pages.hpp"

namespace lsa {

static constexpr int CP_WAVES = 4;
static constexpr int CP_THREADS = 64 * CP_WAVES;

// Kept tokens of one sequence: `first` first tokens, `far` tokens of list entries lo .. hi - 1 (the first of them without its `cut`
// first tokens), and those from `near` on.
struct Kept {
  int32_t len, first, near, lo, cut;
  int64_t far;
  const int32_t* list;
  __device__ __forceinline__ int64_t all() const { return first + far + (len - near); }
};

// For a whole wave, which agrees on the result.
__device__ __forceinline__ Kept find_kept(const KeptArgs& a, int b) {
  Kept k;
  const int64_t cap = a.from.table_stride << a.from.pt_log2;
  k.len = (int32_t)min((int64_t)max(a.kv_len[b], 0), cap);
  k.first = min(a.sinks, k.len);
  k.near = a.window < k.len ? k.len - a.window : 0;
  if (k.near < k.first) k.near = k.first;  // together they are everything
  k.list = a.idx + a.idx_offsets[b];
  k.lo = k.cut = 0;
  k.far = 0;
  const int n = max(a.count[b], 0);
  if (n == 0 || k.near == k.first) return k;
  // The numbers of entries <= x and <= y, with the lanes at 64 places of both ends' ranges at once.
  const int32_t x = k.first / a.r - 1, y = (k.near - 1) / a.r;
  const int lane = threadIdx.x & 63;
  int hi = 0;
  for (int nx = n + 1, ny = n + 1; nx > 1 || ny > 1;) {
    const int sx = (nx + 63) >> 6, sy = (ny + 63) >> 6, ax = lane * sx, ay = lane * sy;
    const int px = k.lo + (ax < nx ? ax : 0), py = hi + (ay < ny ? ay : 0);
    const int32_t ex = px > 0 ? k.list[px - 1] : INT32_MIN, ey = py > 0 ? k.list[py - 1] : INT32_MIN;
    const int cx = __popcll(__ballot(ax < nx && ex <= x)) - 1, cy = __popcll(__ballot(ay < ny && ey <= y)) - 1;
    k.lo += max(cx, 0) * sx; hi += max(cy, 0) * sy;
    nx = min(sx, nx - max(cx, 0) * sx); ny = min(sy, ny - max(cy, 0) * sy);
  }
  k.lo = uni(k.lo);
  hi = uni(hi);
  if (hi <= k.lo) return k;
  const int64_t begin = (int64_t)k.list[k.lo] * a.r, end = (int64_t)k.list[hi - 1] * a.r + a.r;
  k.cut = (int32_t)min(max((int64_t)k.first - begin, (int64_t)0), (int64_t)a.r - 1);
  const int64_t over = min(max(end - k.near, (int64_t)0), (int64_t)a.r - 1);
  k.far = max((int64_t)(hi - k.lo) * a.r - k.cut - over, (int64_t)0);
  return k;
}

// The position that the i-th kept token has, or -1 (a list that is not ascending may hold anything).
__device__ __forceinline__ int32_t kept_token(const KeptArgs& a, const Kept& k, int32_t i) {
  if (i < k.first) return i;
  const int64_t at = (int64_t)i - k.first;
  if (at >= k.far) return at - k.far < k.len - k.near ? (int32_t)(k.near + (at - k.far)) : -1;
  const uint32_t q = (uint32_t)(at + k.cut), e = q / (uint32_t)a.r;  // at < 2^31 and cut < 128
  const int64_t tok = (int64_t)k.list[k.lo + (int64_t)e] * a.r + (q - e * a.r);
  return tok >= 0 && tok < k.len ? (int32_t)tok : -1;
}

// The page that holds a position, or -1.
__device__ __forceinline__ int32_t page_at(const PageMap& m, int b, int32_t pos) {
  const int64_t j = pos >> m.pt_log2;
  if (j >= m.table_stride) return -1;
  const int32_t page = m.table[b * m.table_stride + j];
  return page >= 0 && page < m.n_pages ? page : -1;
}

__global__ __launch_bounds__(CP_THREADS) void kept_kernel(const KeptArgs a, int32_t* kept) {
  const int b = blockIdx.x * CP_WAVES + (threadIdx.x >> 6);
  if (b >= a.B) return;
  const Kept k = find_kept(a, b);
  if ((threadIdx.x & 63) == 0) kept[b] = (int32_t)min(k.all(), (int64_t)INT32_MAX);
}

// Four codes times `s`.
__device__ __forceinline__ void widen_codes(uint32_t w, float s, float (&x)[4]) {
  const auto p = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), q = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  x[0] = p[0] * s; x[1] = p[1] * s; x[2] = q[0] * s; x[3] = q[1] * s;
}

// NL: 16-byte units of a tile's rows per lane. A bf16 tile is copied in parts of at most 8.
template <bool FP8, int D, int NL>
__global__ __launch_bounds__(CP_THREADS) void compact_kernel(const CompactArgs a) {
  constexpr int ROW = D * (FP8 ? 1 : 2), U = ROW / 16;  // bytes and units of a row
  constexpr int PT = NL * 64 / U;
  static_assert(PT >= 16 && PT <= 128, "page sizes");
  __shared__ int64_t s_row[PT];   // source row of head 0, or -1
  __shared__ int32_t s_page[PT];  // and its page
  const int lane = threadIdx.x & 63, wave = uni((int)(threadIdx.x >> 6));
  const int64_t id = blockIdx.x;
  const int group = (int)(id % a.groups), page_i = (int)((id / a.groups) % a.pages), b = (int)(id / a.groups / a.pages);
  const int32_t to_page = page_at(a.to, b, page_i * PT);
  if (to_page < 0) return;
  const Kept k = find_kept(a.what, b);
  const int32_t i0 = page_i * PT, m = (int32_t)min(min(k.all(), (int64_t)a.max_kept) - i0, (int64_t)PT);
  if (m <= 0) return;
  for (int i = threadIdx.x; i < PT; i += CP_THREADS) {
    int32_t page = -1, tok = -1;
    if (i < m) {
      tok = kept_token(a.what, k, i0 + i);
      if (tok >= 0) page = page_at(a.what.from, b, tok);
    }
    s_page[i] = page;
    s_row[i] = page < 0 ? -1 : (((int64_t)page * a.n_kv) << a.what.from.pt_log2) + (tok & ((1 << a.what.from.pt_log2) - 1));
  }
  __syncthreads();
  const int end = min((group + 1) * a.per_group, a.tiles);
  for (int t = group * a.per_group + wave; t < end; t += CP_WAVES) {
    const int h = t % a.n_kv, kv = t / a.n_kv;
    const CompactLayer& l = a.layer[kv >> 1];
    const bool is_v = kv & 1;
    const char* src = is_v ? l.v : l.k;
    const int64_t to = (int64_t)to_page * a.n_kv + h;
    char* dst = (is_v ? l.to_v : l.to_k) + to * (PT * ROW);
    if constexpr (!FP8) {
      constexpr int P = NL < 8 ? NL : 8;
      for (int i = 0; i < NL; i += P) {
        u32x4 x[P];
        bool here[P];
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const int u = (i + e) * 64 + lane;
          const int64_t row = s_row[u / U];
          here[e] = row >= 0;
          if (here[e]) x[e] = __builtin_nontemporal_load((const u32x4*)(src + (row + ((int64_t)h << a.what.from.pt_log2)) * ROW + u % U * 16));
        }
#pragma unroll
        for (int e = 0; e < P; ++e)
          if (here[e]) __builtin_nontemporal_store(x[e], (u32x4*)(dst + ((i + e) * 64 + lane) * 16));
      }
    } else {
      const float* scales = is_v ? l.v_scale : l.k_scale;
      u32x4 x[NL];
      float s[NL];
      bool here[NL];
      float most = 0.f;
      bool any = false;
#pragma unroll
      for (int e = 0; e < NL; ++e) {
        const int u = e * 64 + lane;
        const int64_t row = s_row[u / U];
        here[e] = row >= 0;
        any |= here[e];
        x[e] = (u32x4){0, 0, 0, 0};
        s[e] = 0.f;
        if (here[e]) {
          x[e] = __builtin_nontemporal_load((const u32x4*)(src + (row + ((int64_t)h << a.what.from.pt_log2)) * ROW + u % U * 16));
          s[e] = scales[(int64_t)s_page[u / U] * a.n_kv + h];
        }
      }
#pragma unroll
      for (int e = 0; e < NL; ++e)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float y[4];
          widen_codes(x[e][w], s[e], y);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float z = fabsf(y[c]);
            most = fmaxf(most, z < __builtin_inff() ? z : 0.f);
          }
        }
#pragma unroll
      for (int o = 32; o; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
      const float scale = least_scale(most);
      if (!__any(any)) continue;  // nothing goes there: the scale stays
      if (lane == 0) (is_v ? l.to_v_scale : l.to_k_scale)[to] = scale;
      const float inv = 1.f / scale;  // a power of two: the product is the quotient
#pragma unroll
      for (int e = 0; e < NL; ++e) {
        if (!here[e]) continue;
        asm volatile("" : "+v"(x[e]));  // widened again: the values of the maximum would take four times the registers
        u32x4 z;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float y[4];
          widen_codes(x[e][w], s[e], y);
          z[w] = pack_e4m3(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
        }
        if (s[e] == scale) z = x[e];  // NaN keeps its sign there too
        __builtin_nontemporal_store(z, (u32x4*)(dst + (e * 64 + lane) * 16));
      }
    }
  }
}

hipError_t launch_kv_kept(const KeptArgs& a, int32_t* kept, hipStream_t s) {
  kept_kernel<<<(a.B + CP_WAVES - 1) / CP_WAVES, CP_THREADS, 0, s>>>(a, kept);
  return hipGetLastError();
}

template <bool FP8, int D>
static hipError_t launch_page(const CompactArgs& a, hipStream_t s) {
  constexpr int U = D * (FP8 ? 1 : 2) / 16;
  const dim3 grid((unsigned)((int64_t)a.what.B * a.pages * a.groups));
  switch (a.to.pt_log2) {
    case 4: compact_kernel<FP8, D, 16 * U / 64><<<grid, CP_THREADS, 0, s>>>(a); break;
    case 5: compact_kernel<FP8, D, 32 * U / 64><<<grid, CP_THREADS, 0, s>>>(a); break;
    case 6: compact_kernel<FP8, D, 64 * U / 64><<<grid, CP_THREADS, 0, s>>>(a); break;
    default: compact_kernel<FP8, D, 128 * U / 64><<<grid, CP_THREADS, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

hipError_t launch_kv_compact(const CompactArgs& a, bool fp8, int d, hipStream_t s) {
  if (d == 64) return fp8 ? launch_page<true, 64>(a, s) : launch_page<false, 64>(a, s);
  return fp8 ? launch_page<true, 128>(a, s) : launch_page<false, 128>(a, s);
}

}  // namespace lsa
