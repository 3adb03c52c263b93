// lsa_kv_append: new keys and values into the paged cache, keys (and queries) rotated by their
// positions on the way.
//
// Mathematics. Dimension pair j of a head at position p turns by the angle p * inv_freq[j]. The
// angle of a far position has no accurate fp32 form (p = 10^6 leaves 2^-4 of a turn), so the turns
// p * inv_freq / (2 pi) are formed and reduced to [-1/2, 1/2] in fp64, and only the remainder goes
// to fp32. The rotation is fp32 and each stored value is rounded once, to bf16 or to e4m3.
//
// 8-bit pages hold e4m3(x / s) with one scale s per (page, key head), a power of two: the least
// one that holds the page's largest value. While a page fills, its scale may have to grow; a
// power-of-two growth only lowers the exponents of the codes stored before, so they change by
// less than a step only where they become subnormal. Dividing by s is exact for the same reason.
//
// Shape. One block per (touched page, key head, K or V): it alone owns the tile and its scale, so
// the page's maximum needs no atomics and the result no order. A thread keeps its values in
// registers between the maximum and the store. Query rows are independent blocks of the same
// launch, each thread turning some heads with one set of angles.
//
// Measured on MI355X (64 query heads, 8 key heads, d_h 128): 13,612 new tokens of four prompts into e4m3 pages,
// 530 MB read and written, 108 us, the rate of a plain copy (4.9 TB/s against 5.1), into bf16 pages 111 us (5.0 TB/s);
// at d_h 64 54 us (4.9 TB/s) and 62 (4.5); one token of 32 sequences
// 6.1 us, which is launch and dependent reads (offsets, length, page, scale).
#include "kv.hpp"

namespace lsa {

static constexpr int KA_THREADS = 256;

// Query heads per thread. A launch that the device holds at once (one token per sequence) lasts as long as its longest
// chain: two heads, asked for before their position is known. A longer one is bound by the rate of its reads and
// writes, where four heads share one set of angles and the registers of a head at a time leave more waves.
// Measured, two against four: one token of 32 sequences (e4m3) 6.0 us against 6.6; 13,612 new tokens 119 us against 108.
template <bool SHORT>
constexpr int kQueryHeads = SHORT ? 2 : 4;
static constexpr int64_t KA_SHORT_GRID = 256 * (2048 / KA_THREADS);  // 256 compute units of 2048 threads

enum RopeStyle { ROPE_HALVES = 1, ROPE_PAIRS = 2 };

// Unit u of a head row: 16 dimensions in two vectors of 8, and the 8 pairs they form.
struct Unit {
  int a, b;  // first dimension of the two vectors
  bool turn;
};
__device__ __forceinline__ Unit unit_of(int u, int rot, int style) {
  const bool turn = 16 * u < rot;
  if (turn && style == ROPE_HALVES) return {8 * u, 8 * u + rot / 2, true};
  return {16 * u, 16 * u + 8, turn};
}

struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ Angles angles_of(const float* inv_freq, int u, int pos) {
  Angles t;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double turns = (double)pos * (double)inv_freq[8 * u + i] * 0.15915494309189533577;
    const float x = 2.0f * (float)(turns - __builtin_rint(turns));
    sincospif(x, &t.s[i], &t.c[i]);
  }
  return t;
}

__device__ __forceinline__ void widen_unit(u32x4 a, u32x4 b, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(a[i] << 16);
    x[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    x[8 + 2 * i] = __uint_as_float(b[i] << 16);
    x[9 + 2 * i] = __uint_as_float(b[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load_unit(const uint16_t* row, Unit w, float (&x)[16]) {
  widen_unit(*(const u32x4*)(row + w.a), *(const u32x4*)(row + w.b), x);
}

__device__ __forceinline__ void turn_unit(float (&x)[16], const Angles& t, int style) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = style == ROPE_HALVES ? i : 2 * i, b = style == ROPE_HALVES ? i + 8 : 2 * i + 1;
    const float p = x[a], q = x[b];
    x[a] = p * t.c[i] - q * t.s[i];
    x[b] = q * t.c[i] + p * t.s[i];
  }
}

__device__ __forceinline__ void store_bf16(uint16_t* row, Unit w, const float (&x)[16]) {
  u32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    b[i] = pack_bf16(x[8 + 2 * i], x[9 + 2 * i]);
  }
  *(u32x4*)(row + w.a) = a;
  *(u32x4*)(row + w.b) = b;
}

// x / s: s is a power of two wherever this library wrote it, and then the product with its
// reciprocal is exact and equal to the quotient.
struct Divide {
  float s, inv;
  bool pow2;
  __device__ __forceinline__ explicit Divide(float scale) : s(scale), inv(1.0f / scale) {
    pow2 = (__float_as_uint(scale) & 0x007FFFFFu) == 0;
  }
  __device__ __forceinline__ float operator()(float x) const { return pow2 ? x * inv : x / s; }
};

template <int D, bool SHORT>
__device__ __forceinline__ void append_queries(const AppendArgs& a, int style, int64_t block) {
  // a thread: one unit of one token, H heads; a block: 256 / (D/16) consecutive (token, head group) pairs
  constexpr int U = D / 16, H = kQueryHeads<SHORT>;
  const int groups = (a.n_q + H - 1) / H;
  const int64_t at = block * (KA_THREADS / U) + threadIdx.x / U;
  const int u = threadIdx.x % U;
  // every lane takes part in finding the sequence, so those without work go on with row 0 and store nothing
  const bool live = at < a.T * groups;
  const int64_t t = live ? at / groups : 0;
  const int h0 = (int)(live ? at % groups : 0) * H;
  const int64_t row = a.first_row + t;
  const Unit w = unit_of(u, a.inv_freq ? a.rot : 0, style);
  auto from = [&](int h) { return a.q + row * a.q_stride + (int64_t)h * D; };
  u32x4 raw[SHORT ? H : 1][2];
  if constexpr (SHORT) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const uint16_t* q = from(min(h0 + i, a.n_q - 1));
      raw[i][0] = *(const u32x4*)(q + w.a);
      raw[i][1] = *(const u32x4*)(q + w.b);
    }
  }
  Angles ang;
  if (a.inv_freq) {
    int32_t pos;
    if (a.positions) {
      pos = a.positions[row];
    } else {
      // the sequence of the wave's first row, and the next few from there
      const int64_t head = a.first_row + min((block * KA_THREADS + (int64_t)(threadIdx.x & ~63u)) / U / groups, a.T - 1);
      int b = wave_find(a.B, head, [&](int x) { return a.off[x]; });
      for (int i = 0; i < 4 && a.off[b + 1] <= row; ++i) ++b;
      if (row < a.off[b] || a.off[b + 1] <= row) b = upper_seq(a.off, a.B, row);
      pos = (int32_t)(a.c.kv_len[b] - (a.off[b + 1] - row));
    }
    if (w.turn) ang = angles_of(a.inv_freq, u, pos);
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const int h = h0 + i;
    if (h >= a.n_q) break;
    float x[16];
    if constexpr (SHORT) widen_unit(raw[i][0], raw[i][1], x);
    else load_unit(from(h), w, x);
    if (w.turn) turn_unit(x, ang, style);
    store_bf16(a.q_out + (row * a.n_q + h) * D, w, x);
  }
}

template <bool FP8, int D, int UN, bool SHORT>
__global__ __launch_bounds__(KA_THREADS) void append_kernel(const AppendArgs a, int style) {
  constexpr int U = D / 16;  // units per row
  const int64_t tiles = a.page_slots * a.c.n_kv * 2;
  if ((int64_t)blockIdx.x >= tiles) {
    append_queries<D, SHORT>(a, style, (int64_t)blockIdx.x - tiles);
    return;
  }
  const bool is_v = blockIdx.x & 1;
  const int64_t hs = blockIdx.x >> 1;
  const int h = (int)(hs % a.c.n_kv);
  const int64_t slot = hs / a.c.n_kv;
  const int ptl = a.c.pt_log2, pt = 1 << ptl;
  const int64_t off0 = a.first_row;
  auto slot_of = [&](int b) -> int64_t { return ((a.off[b] - off0) >> ptl) + 2 * (int64_t)b; };
  const int b = wave_find(a.B, slot, slot_of);
  const int64_t row0 = a.off[b], n = a.off[b + 1] - row0;
  const int64_t cap = a.c.table_stride << ptl;
  const int64_t len = min((int64_t)a.c.kv_len[b], cap);
  const int64_t first = (int64_t)a.c.kv_len[b] - n;  // position of the sequence's first new token
  const int64_t begin = first > 0 ? first : 0;
  const int64_t lp = (begin >> ptl) + (slot - slot_of(b));
  const int64_t lo = max(begin, lp << ptl), hi = min(len, (lp + 1) << ptl);
  if (lo >= hi) return;
  // The page is used only after the values are turned: its read, and that of the values, overlap.
  const int32_t page = a.c.table[b * a.c.table_stride + lp];
  const int s0 = (int)(lo - (lp << ptl)), m = (int)(hi - lo);
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const uint16_t* src = (is_v ? a.v_new : a.k_new) + (row0 + (lo - first)) * stride + (int64_t)h * D;
  const bool turns = !is_v && a.inv_freq;

  const bool there = page >= 0 && page < a.c.n_pages;
  const int64_t tile = (int64_t)page * a.c.n_kv + h;
  char* dst = (is_v ? a.c.v : a.c.k) + (tile << ptl) * (D * (FP8 ? 1 : 2));  // of a page that is there

  float x[FP8 ? UN : 1][16];  // in bf16 nothing waits for the page's maximum
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < UN; ++i) {
    const int at = threadIdx.x + i * KA_THREADS, t = at / U, u = at % U;
    if (t < m) {
      const Unit w = unit_of(u, turns ? a.rot : 0, style);
      float(&y)[16] = x[FP8 ? i : 0];
      load_unit(src + t * stride, w, y);
      if (w.turn) {
        const int32_t pos = a.positions ? a.positions[row0 + (lo - first) + t] : (int32_t)(lo + t);
        turn_unit(y, angles_of(a.inv_freq, u, pos), style);
      }
      if constexpr (FP8) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float z = fabsf(y[e]);
          most = fmaxf(most, z < __builtin_inff() ? z : 0.f);
        }
      } else if (there) {
        store_bf16((uint16_t*)dst + (int64_t)(s0 + t) * D, w, y);
      }
    }
  }
  if constexpr (FP8) {
    if (!there) return;
    float scale;
    __shared__ float wave_most[KA_THREADS / 64];
    float* scales = is_v ? a.c.v_scale : a.c.k_scale;
    const float was = s0 > 0 ? scales[tile] : 0.f;
#pragma unroll
    for (int o = 32; o; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
    if ((threadIdx.x & 63) == 0) wave_most[threadIdx.x >> 6] = most;
    __syncthreads();
    scale = least_scale(fmaxf(fmaxf(wave_most[0], wave_most[1]), fmaxf(wave_most[2], wave_most[3])));
    const bool keeps = was > 0.f && was < __builtin_inff();  // anything else is no scale: the earlier codes count as 0
    if (s0 > 0 && keeps && was >= scale) {
      scale = was;
    } else {
      if (threadIdx.x == 0) scales[tile] = scale;
      if (s0 > 0) {
        const Divide by(scale);
        uint32_t* codes = (uint32_t*)dst;
        for (int i = threadIdx.x; i < s0 * (D / 4); i += KA_THREADS) {
          const int c = (int)codes[i];
          float y[4];
          const auto p = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), q = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
          y[0] = p[0]; y[1] = p[1]; y[2] = q[0]; y[3] = q[1];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = keeps ? by(y[e] * was) : 0.f;
          codes[i] = pack_e4m3(y[0], y[1], y[2], y[3]);
        }
      }
    }
    const Divide by(scale);
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int at = threadIdx.x + i * KA_THREADS, t = at / U, u = at % U;
      if (t < m) {
        const Unit w = unit_of(u, turns ? a.rot : 0, style);
        uint32_t c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = pack_e4m3(by(x[i][4 * e]), by(x[i][4 * e + 1]), by(x[i][4 * e + 2]), by(x[i][4 * e + 3]));
        char* row = dst + (int64_t)(s0 + t) * D;
        *(u32x2*)(row + w.a) = (u32x2){c[0], c[1]};
        *(u32x2*)(row + w.b) = (u32x2){c[2], c[3]};
      }
    }
  }
}

static int64_t query_blocks(const AppendArgs& a, int d, int heads) {
  if (!a.q) return 0;
  const int64_t groups = (a.n_q + heads - 1) / heads, per = KA_THREADS / (d / 16);
  return (a.T * groups + per - 1) / per;
}

template <bool FP8, int D, bool SHORT>
static hipError_t launch_units(const AppendArgs& a, int style, hipStream_t s) {
  const dim3 grid((unsigned)(a.page_slots * a.c.n_kv * 2 + query_blocks(a, D, kQueryHeads<SHORT>)));
  const int units = (D / 16) << a.c.pt_log2;
  if (units <= KA_THREADS) append_kernel<FP8, D, 1, SHORT><<<grid, KA_THREADS, 0, s>>>(a, style);
  else if (units <= 2 * KA_THREADS) append_kernel<FP8, D, 2, SHORT><<<grid, KA_THREADS, 0, s>>>(a, style);
  else append_kernel<FP8, D, 4, SHORT><<<grid, KA_THREADS, 0, s>>>(a, style);
  return hipGetLastError();
}

template <bool FP8, int D>
static hipError_t launch_length(const AppendArgs& a, int style, hipStream_t s) {
  const int64_t blocks = a.page_slots * a.c.n_kv * 2 + query_blocks(a, D, kQueryHeads<true>);
  return blocks <= KA_SHORT_GRID ? launch_units<FP8, D, true>(a, style, s) : launch_units<FP8, D, false>(a, style, s);
}

hipError_t launch_kv_append(const AppendArgs& a, bool fp8, int d, int style, hipStream_t s) {
  if (d == 64) return fp8 ? launch_length<true, 64>(a, style, s) : launch_length<false, 64>(a, style, s);
  return fp8 ? launch_length<true, 128>(a, style, s) : launch_length<false, 128>(a, style, s);
}

}  // namespace lsa
