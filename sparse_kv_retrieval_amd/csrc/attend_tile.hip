// lsa_attend for many rows (prompts, chunks): the matrix cores bound it, so keys and values go
// through LDS once per block and serve its 256 rows.
//
// Mathematics and precision are those of the split kernel (attend.hip): one pass with a lazily
// raised maximum, S^T = K Q^T and O^T = V^T P^T, fp32 sums, probabilities rounded once to bf16.
//
// Layout. Eight waves of 32 rows each; a row is one lane column of 32x32x16 MFMA results, so a
// lane's 16 scores of a 32-key half tile belong to one row and become the second product's operand
// where they are (half h holds keys 8a + 4h + 0..3). Tiles of 64 keys go through three LDS buffers as
// bf16 rows, swizzled so that no read or write meets in a bank, and V's operand comes from the transposing
// LDS load. A wave fetches 16 rows of K or of V (one page) to registers one tile ahead of their LDS store and
// two ahead of their use: one barrier per tile.
//
// Schedule. Three steps are in work at once: the scores of the next 32 keys, the exponentials of these and
// the second product of the ones before, one matrix instruction of each product and two exponentials
// a group, in a fixed order. Left to itself the compiler sank the exponentials behind the products (954
// against 865 us for two prompts of 4981 and 4888 tokens).
//
// e4m3 codes are widened on the way to LDS, once per block. The power-of-two part of the page's scale
// goes in there, exactly; what is left of a scale that is no power of two rides in the exponentials'
// argument and costs nothing.
//
// Measured on MI355X (64 query heads, 8 key heads, d_h 128; torch's bf16 matrix product of 8192^3 reaches
// 1269 TFLOP/s there; the kernel's time in a trace): 2048 tokens on top of 30,720 in e4m3 2.1 ms (1.01 PFLOP/s); prompts of
// 4981 and 4888 tokens in bf16 850 us (0.94 PFLOP/s); of 7203 and 6711 tokens with a window of 1024 593 us (0.73 PFLOP/s of
// visible pairs). The matrix
// pipes are busy 42 % of the time in the first, the vector ALUs about as long; without exponentials, LDS
// reads, staging and maxima the second still takes 617 us. A block's first tile, its queries and its output
// cost some 6 us that nothing overlaps, as one block fills a CU's registers and LDS: they are what
// short and windowed prompts pay. Blocks of four waves and two buffers, two to a CU, were slower (2428 and 925 us
// against 2190 and 865).
#include <type_traits>

#include "kv.hpp"

namespace lsa {

static constexpr int TL_WAVES = 8;
static constexpr int TL_THREADS = 64 * TL_WAVES;
static constexpr int TL_M = ATTEND_TILE_ROWS, TL_N = ATTEND_TILE_KEYS;
static_assert(TL_M == 32 * TL_WAVES, "a wave has 32 rows");
static constexpr int TL_BUFS = 3;
static constexpr int TL_SUBS = TL_N / 16;
static_assert(TL_WAVES == 2 * TL_SUBS, "one wave fetches 16 rows of K or of V");

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Swizzles of 16-byte chunks. A read of K takes one chunk of consecutive rows: 16 of them (or 8 rows of two
// lines) meet all banks once. A transposing read of V takes four chunks of four rows.
template <int CPR>
__device__ __forceinline__ int k_swizzle(int r) {
  return (r * CPR / 16) % CPR;
}
template <int CPR>
__device__ __forceinline__ int v_swizzle(int r) {
  return 4 * ((r * CPR / 16) % (CPR / 4));
}

// e4m3 to bf16 times a power of two.
__device__ __forceinline__ u32x2 widen4(uint32_t four, float pow2) {
  u32x2 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, pow2, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, pow2, true));
  return r;
}

// The lowest n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// A scale as a power of two within bf16's middle range, times what is left (1, or beyond that range).
__device__ __forceinline__ void split_scale(float s, float* pow2, float* rest) {
  int e = (int)((__float_as_uint(s) >> 23) & 255) - 127;
  e = e < -100 ? -100 : e > 100 ? 100 : e;
  *pow2 = __uint_as_float((uint32_t)(e + 127) << 23);
  *rest = s * __uint_as_float((uint32_t)(127 - e) << 23);
}

template <bool FP8, int D>
__global__ __launch_bounds__(TL_THREADS, 2) void attend_tile_kernel(const AttendArgs a) {
  constexpr int CPR = D / 8;                  // 16-byte chunks of a row in LDS
  constexpr int SRC = FP8 ? D / 16 : D / 8;   // and of a cached row
  constexpr int LOADS = SRC / 4;              // 16-byte loads per lane of 16 rows
  constexpr int ROWB = 2 * D;                 // bytes of a row in LDS
  constexpr int KS = D / 16, DT = D / 32;
  __shared__ __attribute__((aligned(16))) char s_k[TL_BUFS][TL_N * ROWB], s_v[TL_BUFS][TL_N * ROWB];
  // what is left of the scales of 16 keys: of K times c, of V as log2 and reciprocal
  __shared__ __attribute__((aligned(16))) float s_kc[TL_BUFS][TL_SUBS], s_vlog[TL_BUFS][TL_SUBS], s_vinv[TL_BUFS][TL_SUBS];
  __shared__ __attribute__((aligned(16))) int32_t s_here[TL_BUFS][TL_SUBS];  // whether the 16 keys are there
  __shared__ __attribute__((aligned(16))) int32_t s_odd[TL_BUFS][TL_SUBS];   // whether values were taken out

  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), col = lane & 31, h = lane >> 5;
  const int sub = wave % TL_SUBS;        // the wave fetches this 16 tokens' keys, or values
  const bool is_v = wave >= TL_SUBS;
  const int64_t id = blockIdx.x;
  const int kv = (int)(id % a.c.n_kv);
  const int split = (int)((id / a.c.n_kv) % a.splits);
  // the last row blocks see the most keys: they go first
  Rows w;
  if (!find_rows(a, a.blocks - 1 - id / ((int64_t)a.c.n_kv * a.splits), &w)) return;
  const int parts = (w.tiles + a.run - 1) / a.run;
  if (split > 0 && split >= parts) return;
  const int first = split * a.run, count = min(a.run, w.tiles - first);

  // scores in units of |scale|: its sign goes into the queries
  const float c = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
  const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u, keep = a.scale_log2 == 0.f ? 0u : ~0u;
  const int r = wave * 32 + col;
  const int row = w.r0 + min(r, w.n - 1), tok = row / a.G, head = kv * a.G + (row - tok * a.G);
  const int p_row = w.p0 + tok, w_row = window_start(a, p_row);
  bf16x8 q[KS];
  {
    const uint16_t* from = a.q + (w.t0 + tok) * a.q_stride + (int64_t)head * D + 8 * h;
#pragma unroll
    for (int s = 0; s < KS; ++s) q[s] = as_bf16x8((*(const u32x4*)(from + 16 * s) & keep) ^ flip);
  }

  // The 16 tokens of tile i that this wave fetches: the first one's position, or -1 where no row sees
  // any of them, and the page that holds them. The page is asked for one tile ahead of its use, so
  // that reading it never waits for the tile's own loads.
  auto tokens = [&](int i) __attribute__((always_inline)) -> int {
    if (i >= count) return -1;
    const int t = w.near.tile(first + i) * TL_N + sub * 16;
    return t > w.p_hi || (t + 15 <= w.w_lo && t >= a.sinks) ? -1 : t;
  };
  const int32_t* table = a.c.table + w.b * a.c.table_stride;
  auto page_of = [&](int t) __attribute__((always_inline)) -> int32_t { return table[max(t, 0) >> a.c.pt_log2]; };
  auto place = [&](int t, int32_t page) __attribute__((always_inline)) -> int64_t {
    page = uni(page);
    if (t < 0 || page < 0 || page >= a.c.n_pages) return -1;
    return (((int64_t)page * a.c.n_kv + kv) << a.c.pt_log2) + (t & ((1 << a.c.pt_log2) - 1));
  };

  u32x4 in[LOADS];
  float in_scale = 1.f;
  const char* src = is_v ? a.c.v : a.c.k;
  const float* src_scale = is_v ? a.c.v_scale : a.c.k_scale;
  auto fetch = [&](int64_t at) __attribute__((always_inline)) {
    const int64_t row0 = at < 0 ? 0 : at;  // nothing there: any row, its values are cleared below
#pragma unroll
    for (int i = 0; i < LOADS; ++i) in[i] = *(const u32x4*)(src + row0 * (SRC * 16) + (uint32_t)((i * 64 + lane) * 16));
    if constexpr (FP8) in_scale = src_scale[row0 >> a.c.pt_log2];
  };
  auto whole_tile = [&](int t0) __attribute__((always_inline)) { return t0 + TL_N - 1 <= w.p_lo && (t0 > w.w_hi || t0 + TL_N - 1 < a.sinks); };
  // Values that no row of the block sees become 0: a probability of 0 would not clear an infinity. (Keys
  // may stay, their scores are masked.) Where some rows see a value and others do not, one that is not
  // finite becomes 0 as well, and the tile is marked: rescue() brings it to the rows that see it.
  auto store = [&](int buf, int i, int64_t at) __attribute__((always_inline)) {
    const int t0 = w.near.tile(first + i) * TL_N + sub * 16;
    if (is_v) {
      uint32_t odd = 0;
      if (at < 0 || !whole_tile(t0 - sub * 16)) {
#pragma unroll
        for (int e = 0; e < LOADS; ++e) {
          const int t = t0 + (e * 64 + lane) / SRC;
          const bool some = at >= 0 && t <= w.p_hi && (t > w.w_lo || t < a.sinks);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const uint32_t x = some ? in[e][z] : 0u, bad = not_finite<FP8>(x);
            odd |= bad;
            in[e][z] = x & ~bad;
          }
        }
      }
      const bool any = __any(odd != 0);
      if (lane == 0) s_odd[buf][sub] = any;
    } else if (lane == 0) {
      s_here[buf][sub] = at >= 0;
    }
    float pow2 = 1.f, rest = 1.f;
    if constexpr (FP8) {
      if (at >= 0) split_scale(in_scale, &pow2, &rest);
      if (lane == 0) {
        if (is_v) {
          s_vlog[buf][sub] = __log2f(rest);
          s_vinv[buf][sub] = 1.f / rest;
        } else {
          s_kc[buf][sub] = rest * c;
        }
      }
    }
    char* dst = is_v ? s_v[buf] : s_k[buf];
#pragma unroll
    for (int e = 0; e < LOADS; ++e) {
      const int at_row = (e * 64 + lane) / SRC, ch = (e * 64 + lane) % SRC, rr = sub * 16 + at_row;
      char* d = dst + rr * ROWB;
      const int sw = is_v ? v_swizzle<CPR>(rr) : k_swizzle<CPR>(rr);
      if constexpr (FP8) {
        // Eight lanes write at once and meet 32 banks: half of them begin with the upper eight codes, or they would
        // all write even chunks, two to a bank.
        const bool turn = lane & 4;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bool upper = turn != (x == 1);
          const uint32_t c0 = upper ? in[e][2] : in[e][0], c1 = upper ? in[e][3] : in[e][1];
          const u32x2 lo = widen4(c0, pow2), hi = widen4(c1, pow2);
          *(u32x4*)(d + ((2 * ch + upper) ^ sw) * 16) = (u32x4){lo[0], lo[1], hi[0], hi[1]};
        }
      } else {
        *(u32x4*)(d + (ch ^ sw) * 16) = in[e];
      }
    }
  };

  f32x16 acc[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) acc[i] = (f32x16)(0.f);
  float m = ATTEND_LOWEST, l = 0.f;

  // LDS addresses of the operands: K row `col`, chunk 2 s + h; V rows 4 h + (lane % 16) / 4, 8 bytes of
  // the 32 that the lane's group of 16 reads per row
  const int k_at = col * ROWB + (k_swizzle<CPR>(col) ^ h) * 16;
  const int vrow = 4 * h + (lane & 15) / 4;
  const int v_at = vrow * ROWB + ((2 * ((lane >> 4) & 1) + (lane & 3) / 2) ^ v_swizzle<CPR>(vrow)) * 16 + (lane & 1) * 8;
  auto k_operand = [&](int buf, int u, int x) __attribute__((always_inline)) { return *(const u32x4*)(s_k[buf] + u * 32 * ROWB + (k_at ^ (32 * x))); };
  // operand e of key step x: dimensions 32 e + lane % 32, keys 16 x + 8 z + 4 h + 0..3 for z = 0, 1
  auto v_operand = [&](int buf, int u, int x, int e) __attribute__((always_inline)) {
    typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
    u32x4 v;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(s_v[buf] + (u * 32 + 16 * x + 8 * z) * ROWB + (v_at ^ (64 * e))));
      const u32x2 t2 = __builtin_bit_cast(u32x2, t);
      v[2 * z] = t2[0];
      v[2 * z + 1] = t2[1];
    }
    return v;
  };
  auto seen = [&](int t) __attribute__((always_inline)) { return t <= p_row && (t > w_row || t < a.sinks); };

  // Scores of 32 keys before their softmax: register i of a lane is key 8 (i / 4) + 4 h + i % 4. Applies the mask and
  // raises the maximum; returns whether it rose for some row of the wave, and then what to scale by in `fall`.
  auto settle = [&](int buf, int t0, int u, bool whole, bool here0, bool here1, f32x16& s, float& fall) __attribute__((always_inline)) -> bool {
    if (!whole) {
      // a bit for each of the 32 keys from the lane's first on: x <= hi, and x > lo or x < few
      const int base = t0 + 32 * u + 4 * h;
      const uint32_t in = low_bits(p_row - base + 1) & (~low_bits(w_row - base + 1) | low_bits(a.sinks - base)) &
                          ((here0 ? 0x0000FFFFu : 0u) | (here1 ? 0xFFFF0000u : 0u));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t see = __builtin_amdgcn_sbfe((int)in, 8 * (i / 4) + i % 4, 1);  // all ones or none
        s[i] = __uint_as_float((__float_as_uint(s[i]) & see) | (0xFF800000u & ~see));
      }
    }
    float top = s[0], top1 = s[8];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      top = fmaxf(top, s[i]);
      top1 = fmaxf(top1, s[8 + i]);
    }
    top = FP8 ? fmaxf(top * s_kc[buf][2 * u], top1 * s_kc[buf][2 * u + 1]) : fmaxf(top, top1) * c;
    if (!__any(top > m + ATTEND_LAZY)) return false;
    const auto o = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
    const float high = fmaxf(m, fmaxf(__uint_as_float(o[0]), __uint_as_float(o[1])));
    fall = __builtin_amdgcn_exp2f(m - high);
    m = high;
    l *= fall;
    return true;
  };

  // One step over 32 keys (buf, u) does three things side by side: the scores of the next 32 keys, this
  // one's probabilities, and the second product of the ones before. The order is fixed group by group: one matrix
  // instruction of each product (they do not wait for each other), the LDS reads of the group after the
  // next, and a share of the exponentials. What is left of V's scale rides in the exponent, and leaves
  // the sum again by its reciprocal.
  bf16x8 p[2] = {as_bf16x8((u32x4){0, 0, 0, 0}), as_bf16x8((u32x4){0, 0, 0, 0})};
  u32x4 kf[3], vf[3];
  // a step's first operands, asked for before the scores are settled
  auto ahead = [&](int next_buf, int next_u, int old_buf, int old_u) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      kf[x] = k_operand(next_buf, next_u, x);
      vf[x] = v_operand(old_buf, old_u, x / DT, x % DT);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](int buf, int u, const f32x16& s, int next_buf, int next_u, f32x16& s_next, int old_buf, int old_u) __attribute__((always_inline)) {
    constexpr int E = 16 / KS;  // exponentials of a group
    static_assert(KS == 2 * DT, "as many key steps as value operands");
    float c2[2] = {c, c}, add[2] = {-m, -m}, inv[2] = {1.f, 1.f};
    if constexpr (FP8) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        c2[x] = s_kc[buf][2 * u + x];
        add[x] = s_vlog[buf][2 * u + x] - m;
        inv[x] = s_vinv[buf][2 * u + x];
      }
    }
    uint32_t packed[8];
    s_next = (f32x16)(0.f);
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      if (x + 2 < KS) {
        kf[(x + 2) % 3] = k_operand(next_buf, next_u, x + 2);
        vf[(x + 2) % 3] = v_operand(old_buf, old_u, (x + 2) / DT, (x + 2) % DT);
      }
      s_next = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(kf[x % 3]), q[x], s_next, 0, 0, 0);
      acc[x % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(vf[x % 3]), p[x / DT], acc[x % DT], 0, 0, 0);
#pragma unroll
      for (int i = E * x; i < E * (x + 1); i += 2) {
        const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c2[i / 8], add[i / 8]));
        const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i + 1], c2[i / 8], add[i / 8]));
        if constexpr (FP8) {
          l = __builtin_fmaf(e0, inv[i / 8], l);
          l = __builtin_fmaf(e1, inv[i / 8], l);
        } else {
          l += e0;
          l += e1;
        }
        packed[i / 2] = pack_bf16(e0, e1);
        asm volatile("" : "+v"(packed[i / 2]), "+v"(l));  // here, and not sunk to where they are used
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) p[x] = as_bf16x8((u32x4){packed[4 * x], packed[4 * x + 1], packed[4 * x + 2], packed[4 * x + 3]});
  };
  auto scale_out = [&](float f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < DT; ++i) acc[i] *= f;
  };
  // Values that are not finite, taken out of a tile on its way to LDS, reach the rows that see them.
  auto rescue = [&](int t0) __attribute__((always_inline)) {
#pragma unroll 1
    for (int j = 0; j < TL_N; ++j) {
      const int t = t0 + j;
      if (t > w.p_hi || !(t > w.w_lo || t < a.sinks)) continue;
      const int64_t row = place(t, page_of(t));
      if (row < 0) continue;
      const char* from = a.c.v + row * (SRC * 16);
      const bool sees = seen(t);
#pragma unroll
      for (int e = 0; e < DT; ++e) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float z = cached_value<FP8>(from, 32 * e + 8 * (i / 4) + 4 * h + i % 4);
          if (sees && !(fabsf(z) < __builtin_inff())) acc[e][i] += z;
        }
        __builtin_amdgcn_sched_barrier(0);  // rare: keep its registers few
      }
    }
  };

  int t_next = tokens(0);
  int32_t page = page_of(t_next);
  int64_t at = place(t_next, page);
  t_next = tokens(1);
  page = page_of(t_next);
  f32x16 s0 = (f32x16)(0.f), s1;
  float fall = 1.f;
  if (count > 0) {
    fetch(at);
    store(0, 0, at);
    at = place(t_next, page);
    t_next = tokens(2);
    page = page_of(t_next);
    fetch(at);  // beyond the run: row 0, not used
    // the first step's second product is of no probabilities and these values
    for (int i = tid; i < TL_N * ROWB / 16; i += TL_THREADS) *(u32x4*)(s_v[TL_BUFS - 1] + 16 * i) = (u32x4){0, 0, 0, 0};
    __syncthreads();
#pragma unroll
    for (int x = 0; x < KS; ++x) s0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(k_operand(0, 0, x)), q[x], s0, 0, 0, 0);
  }
  // tile i, in a buffer known when compiled: its operands' LDS addresses are constants beside the lane's
  auto tile = [&](int i, auto which) __attribute__((always_inline)) {
    constexpr int buf = decltype(which)::value, nb = (buf + 1) % TL_BUFS, old = (buf + TL_BUFS - 1) % TL_BUFS;
    const int t0 = w.near.tile(first + i) * TL_N;
    const u32x4 here = *(const u32x4*)s_here[buf];
    const bool h0 = uni((int)here[0]), h1 = uni((int)here[1]), h2 = uni((int)here[2]), h3 = uni((int)here[3]);
    const bool whole = h0 && h1 && h2 && h3 && whole_tile(t0);
    // The probabilities before this step's belong to the maximum before it: the output is scaled after them.
    ahead(buf, 1, old, 1);
    bool rose = settle(buf, t0, 0, whole, h0, h1, s0, fall);
    step(buf, 0, s0, buf, 1, s1, old, 1);
    if (rose) scale_out(fall);
    // The next tile: its buffer was last read two barriers ago.
    if (i + 1 < count) {
      store(nb, i + 1, at);
      at = place(t_next, page);
      t_next = tokens(i + 3);
      page = page_of(t_next);
      fetch(at);
    }
    lds_barrier();  // the loads of the tile after next stay in flight
    ahead(nb, 0, buf, 0);
    rose = settle(buf, t0, 1, whole, h2, h3, s1, fall);
    // after the last tile the next scores are those of an old buffer, and not used
    step(buf, 1, s1, nb, 0, s0, buf, 0);
    if (rose) scale_out(fall);
    if (!whole) {
      const u32x4 odd = *(const u32x4*)s_odd[buf];
      if (uni((int)(odd[0] | odd[1] | odd[2] | odd[3]))) rescue(t0);
    }
  };
  auto last = [&](auto which) __attribute__((always_inline)) {
    constexpr int buf = decltype(which)::value;
#pragma unroll
    for (int x = 0; x < KS; ++x)
      acc[x % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(v_operand(buf, 1, x / DT, x % DT)), p[x / DT], acc[x % DT], 0, 0, 0);
  };
  static_assert(TL_BUFS == 3, "the loop goes through the buffers");
  typedef std::integral_constant<int, 0> B0;
  typedef std::integral_constant<int, 1> B1;
  typedef std::integral_constant<int, 2> B2;
  for (int i = 0; i < count; i += 3) {
    tile(i, B0{});
    if (i + 1 < count) tile(i + 1, B1{});
    if (i + 2 < count) tile(i + 2, B2{});
  }
  if (count > 0) {
    if (count % 3 == 1) last(B0{});
    else if (count % 3 == 2) last(B1{});
    else last(B2{});
  }

  const float sum = sum_halves(l);
  if (r >= w.n) return;
  if (parts <= 1) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* dst = a.out + (w.t0 + tok) * a.out_stride + (int64_t)head * D + 4 * h;
#pragma unroll
    for (int e = 0; e < DT; ++e)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *(u32x2*)(dst + 32 * e + 2 * i) = (u32x2){pack_bf16(acc[e][i] * inv, acc[e][i + 1] * inv),
                                                  pack_bf16(acc[e][i + 2] * inv, acc[e][i + 3] * inv)};
    if (a.lse && h == 0) a.lse[(w.t0 + tok) * a.n_q + head] = sum == 0.f ? -__builtin_inff() : (m + __log2f(sum)) * LN2;
  } else {
    const int64_t to = ((int64_t)split * a.T + (w.t0 - a.first_row + tok)) * a.n_q + head;
#pragma unroll
    for (int e = 0; e < DT; ++e)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *(f32x4*)(a.part_o + to * D + 4 * h + 32 * e + 2 * i) = (f32x4){acc[e][i], acc[e][i + 1], acc[e][i + 2], acc[e][i + 3]};
    if (h == 0) *(f32x2*)(a.part_ml + 2 * to) = (f32x2){m, sum};
  }
}

hipError_t launch_attend_tile(const AttendArgs& a, bool fp8, int d, hipStream_t s) {
  const dim3 grid((unsigned)(a.blocks * a.splits * a.c.n_kv));
  if (d == 64) {
    if (fp8) attend_tile_kernel<true, 64><<<grid, TL_THREADS, 0, s>>>(a);
    else attend_tile_kernel<false, 64><<<grid, TL_THREADS, 0, s>>>(a);
  } else {
    if (fp8) attend_tile_kernel<true, 128><<<grid, TL_THREADS, 0, s>>>(a);
    else attend_tile_kernel<false, 128><<<grid, TL_THREADS, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace lsa
