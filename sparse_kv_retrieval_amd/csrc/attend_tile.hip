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
// LDS load. A wave fetches 16 rows of K or of V (one page) to registers; beside a tile's first step the next tile goes
// from there to LDS and the one after it is asked for: one barrier per tile. Where 16 rows lie, and whether all rows
// see them all, is found for 96 tiles at once and waits in LDS, so that a tile begins with one LDS read instead of a chain of
// two dependent reads of memory (two prompts of 4981 and 4888 tokens 831 against 858 us). Queries come and outputs
// leave through LDS in whole rows: a lane's own pieces are 16 and 32 bytes of a line (799 against 815 us).
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
// Forms (kv.hpp has the mathematics). Each is an instance of its own, so the plain one pays for none. Only tiles that
// FLAG_WHOLE does not name look at masks. A cap adds an exponential and a reciprocal a score; masked scores are NaN
// there, which the last exponential's clamp turns into 0. A bias is linear in the position up to the row itself, so it is one more
// addend of the exponential's argument, and the maximum of 32 keys is bounded by the greatest score plus the greatest bias.
// With a bias tiles go from the nearest to the farthest: the maximum then hardly ever rises (2107 against 2565 us for 2048
// tokens on top of 30,720). Documents and prefixes shorten the range of tiles a block goes through.
//
// Measured on MI355X (64 query heads, 8 key heads, d_h 128; torch's bf16 matrix product of 8192^3 reaches
// 1397 TFLOP/s there, warmed in the same way; whole calls in turn): 2048 tokens on top of 30,720 in e4m3 1.94 ms (1.10 PFLOP/s), with a bias 2.02;
// prompts of 4981 and 4888 tokens in bf16 788 us (1.01 PFLOP/s), with a cap 1019; of 7203 and 6711 tokens with a window of 1024
// 561 us (0.77 PFLOP/s of visible pairs); 8192 tokens of packed documents of 89 to 1519 215 us. The matrix
// pipes are busy 50 % of the time in a plain prompt and 35 % in a capped one, the vector ALUs 51 and 67: together some 100 %, so the two
// hardly work at once, although a wave's own groups have work for both. Without
// the exponentials a prompt takes 5 % less, without transposing reads 2, fetches 3, LDS stores 2, half of the first product 11: no
// single one bounds it. A block's rows, places, queries, first tile and output cost some 14 us that nothing overlaps, as one block fills a
// CU's registers and LDS: they are what documents and short or windowed prompts pay. Slower were blocks of four waves and two
// buffers, two to a CU (2428 and 925 us against 2190 and 865); 64 rows a wave in four waves (1005 against 857); masks by
// branches inside the groups (capped 1140 against 1076); exponentials before the maximum is known, and again where it rose
// (biased 3311 against 2597).
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
// Tiles whose places a block finds at once: a multiple of the buffers, and with those that are fetched ahead a thread for each 16 rows.
static constexpr int TL_RUN = 96, TL_AHEAD = 3;
static_assert(TL_RUN % TL_BUFS == 0 && (TL_RUN + TL_AHEAD) * TL_SUBS <= TL_THREADS, "places");

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

// Of a tile: bit i says that its i-th 16 keys are there, FLAG_WHOLE that all are and every row sees them.
static constexpr uint32_t FLAG_WHOLE = 1u << TL_SUBS;

template <bool FP8, int D, int FORM>
__global__ __launch_bounds__(TL_THREADS, 2) void attend_tile_kernel(const AttendArgs a) {
  constexpr int CPR = D / 8;                  // 16-byte chunks of a row in LDS
  constexpr int SRC = FP8 ? D / 16 : D / 8;   // and of a cached row
  constexpr int LOADS = SRC / 4;              // 16-byte loads per lane of 16 rows
  constexpr int ROWB = 2 * D;                 // bytes of a row in LDS
  constexpr int KS = D / 16, DT = D / 32;
  constexpr bool SEEN = (FORM & FORM_SEEN) != 0, CAP = (FORM & FORM_CAP) != 0, BIAS = (FORM & FORM_BIAS) != 0;
  __shared__ __attribute__((aligned(16))) char s_k[TL_BUFS][TL_N * ROWB], s_v[TL_BUFS][TL_N * ROWB];
  // what is left of the scales of 16 keys: of K times c, of V as log2 and reciprocal
  __shared__ __attribute__((aligned(16))) float s_kc[TL_BUFS][TL_SUBS], s_vlog[TL_BUFS][TL_SUBS], s_vinv[TL_BUFS][TL_SUBS];
  // Of 16 keys of a tile: where they lie, in rows (negative: nowhere), what the tile's subs and rows have (see FLAG_WHOLE), and its position.
  __shared__ __attribute__((aligned(16))) u32x4 s_place[TL_RUN + TL_AHEAD][TL_SUBS];
  __shared__ __attribute__((aligned(16))) int32_t s_odd[TL_BUFS][TL_SUBS];   // whether values were taken out

  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), col = lane & 31, h = lane >> 5;
  const int sub = wave % TL_SUBS;        // the wave fetches this 16 tokens' keys, or values
  const bool is_v = wave >= TL_SUBS;
  const int64_t id = blockIdx.x;
  const int kv = (int)(id % a.c.n_kv);
  const int split = (int)((id / a.c.n_kv) % a.splits);
  // the last row blocks see the most keys: they go first
  Rows w;
  if (!find_rows<FORM>(a, a.blocks - 1 - id / ((int64_t)a.c.n_kv * a.splits), &w)) return;
  const int parts = (w.tiles + a.run - 1) / a.run;
  if (split > 0 && split >= parts) return;
  const int first = split * a.run, count = min(a.run, w.tiles - first);

  // scores in units of |scale|: its sign goes into the queries
  const float c = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
  const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u, keep = a.scale_log2 == 0.f ? 0u : ~0u;
  const int r = wave * 32 + col;
  const int row = w.r0 + min(r, w.n - 1), tok = row / a.G, head = kv * a.G + (row - tok * a.G);
  const int p_row = w.p0 + tok, w_row = window_start(a, p_row);
  const int f_row = SEEN ? first_seen(a, w.t0 + tok) : 0;
  const int e_row = SEEN ? last_seen(a, w.t0 + tok, p_row, w.len) : p_row;
  const float slope = BIAS ? slope_log2(a, head) : 0.f;
  // The wave's queries come, and its output leaves, in whole rows, through LDS that no tile is in: a lane's own pieces of its row are 32 bytes
  // of a line here and 16 there. mine(row, chunk): where the wave's 32 rows lie, swizzled like keys.
  static_assert(TL_WAVES / 2 * 32 <= TL_BUFS * TL_N, "half the waves' rows fit the keys' buffers");
  constexpr int UNITS = 32 * CPR / 64;
  auto mine = [&](int row, int chunk) __attribute__((always_inline)) {
    return (wave < TL_WAVES / 2 ? s_k[0] : s_v[0]) + (wave % (TL_WAVES / 2) * 32 + row) * ROWB + (chunk ^ k_swizzle<CPR>(row)) * 16;
  };
  // what row `row` of the wave has of x
  auto of_row = [&](int64_t x, int row) __attribute__((always_inline)) {
    const uint32_t lo = __shfl((int)(uint32_t)x, row), hi = __shfl((int)(uint32_t)((uint64_t)x >> 32), row);
    return (int64_t)(((uint64_t)hi << 32) | lo);
  };
  bf16x8 q[KS];
  {
    const int64_t from = (w.t0 + tok) * a.q_stride + (int64_t)head * D;
    u32x4 x[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) x[i] = *(const u32x4*)(a.q + of_row(from, i * (64 / CPR) + lane / CPR) + lane % CPR * 8);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) *(u32x4*)mine(i * (64 / CPR) + lane / CPR, lane % CPR) = x[i];
    // a wave's LDS accesses are in order, and no other wave's touch these rows before the barrier behind the places
#pragma unroll
    for (int s = 0; s < KS; ++s) q[s] = as_bf16x8((*(const u32x4*)mine(col, 2 * s + h) & keep) ^ flip);
  }

  const int32_t* table = a.c.table + w.b * a.c.table_stride;
  // The cached row of a position that some row sees, or -1.
  auto row_of = [&](int t) __attribute__((always_inline)) -> int64_t {
    const int32_t page = table[t >> a.c.pt_log2];
    if (page < 0 || page >= a.c.n_pages) return -1;
    return (((int64_t)page * a.c.n_kv + kv) << a.c.pt_log2) + (t & ((1 << a.c.pt_log2) - 1));
  };
  auto whole_tile = [&](int t0) __attribute__((always_inline)) { return t0 + TL_N - 1 <= end_lo<FORM>(w) && all_begin<FORM>(a, w, t0, t0 + TL_N - 1); };
  // Finds the places of the tiles from `base` on, a thread for each 16 keys, so that the loop over the tiles has no page to wait for and
  // few scalar instructions: two waves a SIMD hide little of either.
  auto resolve = [&](int base) __attribute__((always_inline)) {
    const int x = tid / TL_SUBS;  // its tile
    if (x >= TL_RUN + TL_AHEAD) return;
    // With a bias the near keys go first: far ones hardly ever raise a maximum.
    const int i = base + x, t0 = i < count ? w.near.tile(first + (BIAS ? count - 1 - i : i)) * TL_N : 0, t = t0 + tid % TL_SUBS * 16;
    int64_t row = -1;
    if (i < count && t <= end_hi<FORM>(w) && some_begin<FORM>(a, w, t, t + 15)) row = row_of(t);
    const uint32_t here = (uint32_t)(__ballot(row >= 0) >> (lane & ~(TL_SUBS - 1))) & ((1u << TL_SUBS) - 1);
    const uint32_t flags = here | (i < count && here == (1u << TL_SUBS) - 1 && whole_tile(t0) ? FLAG_WHOLE : 0u);
    s_place[x][tid % TL_SUBS] = (u32x4){(uint32_t)row, (uint32_t)((uint64_t)row >> 32), flags, (uint32_t)t0};
  };
  struct Place {
    int64_t row;
    uint32_t flags;
    int32_t t0;
  };
  auto place_of = [&](int x) __attribute__((always_inline)) -> Place {
    const u32x4 y = s_place[x][sub];
    return {uni((int64_t)(((uint64_t)y[1] << 32) | y[0])), (uint32_t)uni((int32_t)y[2]), uni((int32_t)y[3])};
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
  // Values that no row of the block sees become 0: a probability of 0 would not clear an infinity. (Keys
  // may stay, their scores are masked.) Where some rows see a value and others do not, one that is not
  // finite becomes 0 as well, and the tile is marked: rescue() brings it to the rows that see it.
  float pow2 = 1.f;
  auto clean = [&](int buf, const Place& of) __attribute__((always_inline)) {
    if (is_v && !(of.flags & FLAG_WHOLE)) {
      uint32_t odd = 0;
#pragma unroll
      for (int e = 0; e < LOADS; ++e) {
        const int t = of.t0 + sub * 16 + (e * 64 + lane) / SRC;
        const bool some = of.row >= 0 && t <= end_hi<FORM>(w) && some_begin<FORM>(a, w, t, t);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint32_t x = some ? in[e][z] : 0u, bad = not_finite<FP8>(x);
          odd |= bad;
          in[e][z] = x & ~bad;
        }
      }
      const bool any = __any(odd != 0);
      if (lane == 0) s_odd[buf][sub] = any;
    }
    if constexpr (FP8) {
      float rest = 1.f;
      pow2 = 1.f;
      if (of.row >= 0) split_scale(in_scale, &pow2, &rest);
      if (lane == 0) {
        if (is_v) {
          s_vlog[buf][sub] = __log2f(rest);
          s_vinv[buf][sub] = 1.f / rest;
        } else {
          s_kc[buf][sub] = rest * c;
        }
      }
    }
  };
  // the e-th 16 bytes of each lane
  auto store = [&](int buf, int e) __attribute__((always_inline)) {
    char* dst = is_v ? s_v[buf] : s_k[buf];
    const int at_row = (e * 64 + lane) / SRC, ch = (e * 64 + lane) % SRC, rr = sub * 16 + at_row;
    char* d = dst + rr * ROWB;
    const int sw = is_v ? v_swizzle<CPR>(rr) : k_swizzle<CPR>(rr);
    if constexpr (FP8) {
      // Eight lanes write at once and meet 32 banks: half of them begin with the upper eight codes, or they would
      // all write even chunks, two to a bank.
      const bool turn = lane & 4;
      const uint32_t y0 = in[e][0], y1 = in[e][1], y2 = in[e][2], y3 = in[e][3];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool upper = turn != (x == 1);
        const uint32_t c0 = upper ? y2 : y0, c1 = upper ? y3 : y1;
        const u32x2 lo = widen4(c0, pow2), hi = widen4(c1, pow2);
        *(u32x4*)(d + ((2 * ch + upper) ^ sw) * 16) = (u32x4){lo[0], lo[1], hi[0], hi[1]};
      }
    } else {
      *(u32x4*)(d + (ch ^ sw) * 16) = in[e];
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
  auto seen = [&](int t) __attribute__((always_inline)) { return t <= e_row && (t > w_row || t < a.sinks) && (!SEEN || t >= f_row); };

  // The maximum is raised by the greatest score that a row sees among 32 keys and the greatest bias of the 32, which may not meet. Where it
  // sees one of them it is then up to 31 slope log2(e) too high: 2^45 for a slope of 1, for which fp32 and bf16 have room. Where it sees none
  // they must not raise it at all: their biases may be any distance away from those of the keys that it does see. Waves with
  // steeper heads look at each key. (So do those of so small a scale that a bias in units of the products would overflow.)
  const bool steep = BIAS && ((!CAP && c < 0x1p-96f) || __any(!(fabsf(slope) <= LOG2E)));
  // There, without a cap, settle() makes the scores whole, in base 2 and with their biases. A line through 32 keys is off by some 2^-24 of 31
  // slopes, which is much beside a near key's own bias; and far keys' scores have to be the numbers that their maximum is one of.
  const bool made = !CAP && steep;
  const float line_slope = made ? 0.f : slope;
  // A cap makes a score of minus infinity finite, so masked places hold NaN instead. In bf16 the probabilities are then held below
  // 1, where the clamp changes no other one.
  constexpr float SHIFT = CAP && !FP8 ? ATTEND_LAZY : 0.f;
  // Scores of 32 keys before their softmax: register i of a lane is key 8 (i / 4) + 4 h + i % 4. Applies the mask and
  // raises the maximum; returns whether it rose for some row of the wave, and then what to scale by in `fall`.
  auto settle = [&](int buf, int t0, int u, bool whole, bool here0, bool here1, f32x16& s, float& fall) __attribute__((always_inline)) -> bool {
    uint32_t visible = ~0u;
    if (!whole) {
      // a bit for each of the 32 keys from the lane's first on: x <= hi, and x > lo or x < few
      const int base = t0 + 32 * u + 4 * h;
      visible = low_bits(e_row - base + 1) & (~low_bits(w_row - base + 1) | low_bits(a.sinks - base)) &
                          (SEEN ? ~low_bits(f_row - base) : ~0u) &
                          ((here0 ? 0x0000FFFFu : 0u) | (here1 ? 0xFFFF0000u : 0u));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t see = __builtin_amdgcn_sbfe((int)visible, 8 * (i / 4) + i % 4, 1);  // all ones or none
        s[i] = __uint_as_float((__float_as_uint(s[i]) & see) | (0xFF800000u & ~see));
      }
    }
    // Without a cap the bias is taken as linear in the position, slope * (t - p). Beyond the row, where only a prefix is seen, the scores
    // make up for it.
    const bool bent = BIAS && !CAP && !made && a.prefix_end && t0 + 32 * u + 31 > w.p_lo;
    if (bent) {
      const int beyond = t0 + 32 * u + 4 * h - p_row;
      float back[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) back[x] = -2.f * slope / (FP8 ? s_kc[buf][2 * u + x] : c);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_fmaf(back[i / 8], (float)max(beyond + 8 * (i / 4) + i % 4, 0), s[i]);
    }
    // where NaN stands for what is masked, a maximum that passes it on shows the others
    auto greater = [](float x, float y) __attribute__((always_inline)) { return CAP ? __builtin_elementwise_maximum(x, y) : fmaxf(x, y); };
    float top = s[0], top1 = s[8];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      top = greater(top, s[i]);
      top1 = greater(top1, s[8 + i]);
    }
    top = FP8 ? greater(top * s_kc[buf][2 * u], top1 * s_kc[buf][2 * u + 1]) : greater(top, top1) * c;
    if constexpr (CAP) {
      top = cap_score(a, top);
      l = __builtin_fmaf(top, 0.f, l);
      // The cap of minus infinity is finite. By the mask and not by the score, as a score of minus infinity that is seen counts as -cap; and
      // without a bias no score lies below -cap, so there it does no harm.
      if (BIAS && !whole) top = visible & 0x0F0F0F0Fu ? top : -__builtin_inff();
    }
    if constexpr (BIAS) {
      if (!steep) {
        // the greatest bias of the 32 keys: the nearest one's, or with a negative slope the farthest one's
        const int lo = p_row - (t0 + 32 * u + 31), hi = lo + 31;
        const int by = slope < 0.f ? (CAP ? max(-lo, hi) : hi) : bent ? lo : max(CAP ? max(lo, -hi) : lo, 0);
        top = __builtin_fmaf(-slope, (float)by, top);
      } else {
        const float d0 = (float)(p_row - (t0 + 32 * u + 4 * h));
        top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = 8 * (i / 4) + i % 4;
          float y = s[i] * (FP8 ? s_kc[buf][2 * u + i / 8] : c);
          if constexpr (CAP) y = visible >> at & 1 ? cap_score(a, y) : y;
          y = __builtin_fmaf(-slope, fabsf(d0 - (float)at), y);
          if constexpr (!CAP) s[i] = y = visible >> at & 1 ? y : -__builtin_inff();
          top = fmaxf(top, y);
        }
      }
    }
    if (CAP && !whole) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t see = __builtin_amdgcn_sbfe((int)visible, 8 * (i / 4) + i % 4, 1);
        s[i] = __uint_as_float((__float_as_uint(s[i]) & see) | (0x7FC00000u & ~see));
      }
    }
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
  // next, a share of the exponentials, and what `beside` does. What is left of V's scale rides in the exponent, and leaves
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
  auto step = [&](int t0, int buf, int u, const f32x16& s, int next_buf, int next_u, f32x16& s_next, int old_buf, int old_u, auto beside) __attribute__((always_inline)) {
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
    if (made) c2[0] = c2[1] = 1.f;
    const float d0 = BIAS ? (float)(p_row - (t0 + 32 * u + 4 * h)) : 0.f;
    float line[2] = {add[0], add[1]};
    if constexpr (CAP) {
      c2[0] *= a.two_over_cap; c2[1] *= a.two_over_cap;
      add[0] += a.cap_log2 - SHIFT; add[1] += a.cap_log2 - SHIFT;
      line[0] = add[0]; line[1] = add[1];
    }
    if constexpr (BIAS) {
      line[0] = __builtin_fmaf(-line_slope, d0, add[0]);
      line[1] = __builtin_fmaf(-line_slope, d0, add[1]);
    }
    auto prob = [&](int i) __attribute__((always_inline)) {
      const float at = (float)(8 * (i / 4) + i % 4);
      float y = line[i / 8];
      if constexpr (BIAS && CAP) y = __builtin_fmaf(-slope, fabsf(d0 - at), add[i / 8]);
      else if constexpr (BIAS) y = __builtin_fmaf(line_slope, at, y);
      if constexpr (!CAP) return __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c2[i / 8], y));
      const float r = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(s[i] * c2[i / 8]));
      const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(-2.f * a.cap_log2, r, y));
      // NaN in a masked place becomes 0: in bf16 by the clamp of the exponential itself, which costs nothing. A steep bias of far keys alone is
      // rounded otherwise than in their maximum; the upper end keeps what that may make of it from being an infinity, which a later
      // maximum's factor of 0 would not clear. (e4m3: 2^8, times the most that is left of a scale, 2^28.)
      return FP8 && !BIAS ? fmaxf(e, 0.f) : __builtin_amdgcn_fmed3f(e, 0.f, FP8 ? 0x1p36f : 1.f);
    };
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
        const float e0 = prob(i), e1 = prob(i + 1);
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
      beside(x);
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
      if (t > end_hi<FORM>(w) || !some_begin<FORM>(a, w, t, t)) continue;
      const int64_t row = row_of(t);
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

  f32x16 s0 = (f32x16)(0.f), s1;
  float fall = 1.f;
  Place now{}, next{};  // of the tile that is worked on, and of the one after it
  if (count > 0) {
    resolve(0);
    __syncthreads();
    now = place_of(0);
    next = place_of(1);
    fetch(now.row);
    clean(0, now);
#pragma unroll
    for (int e = 0; e < LOADS; ++e) store(0, e);
    fetch(next.row);  // beyond the run: row 0, not used
    // the first step's second product is of no probabilities and these values
    for (int i = tid; i < TL_N * ROWB / 16; i += TL_THREADS) *(u32x4*)(s_v[TL_BUFS - 1] + 16 * i) = (u32x4){0, 0, 0, 0};
    __syncthreads();
#pragma unroll
    for (int x = 0; x < KS; ++x) s0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(k_operand(0, 0, x)), q[x], s0, 0, 0, 0);
  }
  // tile i, in a buffer known when compiled: its operands' LDS addresses are constants beside the lane's
  auto tile = [&](int i, int base, auto which) __attribute__((always_inline)) {
    constexpr int buf = decltype(which)::value, nb = (buf + 1) % TL_BUFS, old = (buf + TL_BUFS - 1) % TL_BUFS;
    const int t0 = now.t0;
    const bool whole = now.flags & FLAG_WHOLE, h0 = now.flags & 1, h1 = now.flags & 2, h2 = now.flags & 4, h3 = now.flags & 8;
    // The probabilities before this step's belong to the maximum before it: the output is scaled after them.
    ahead(buf, 1, old, 1);
    bool rose = settle(buf, t0, 0, whole, h0, h1, s0, fall);
    // Beside this step the next tile goes to its buffer, which was last read two barriers ago, and the one after it is asked for. Beyond
    // the run it is row 0, and not used.
    clean(nb, next);
    step(t0, buf, 0, s0, buf, 1, s1, old, 1, [&](int x) __attribute__((always_inline)) {
      constexpr int PER = (LOADS + KS - 3) / (KS - 2);  // stores of a group, from the second one to the last but one
#pragma unroll
      for (int e = 0; e < LOADS; ++e)
        if (x == 1 + e / PER) store(nb, e);
      if (x == KS - 1) {
        now = next;
        next = place_of(i - base + 2);
        fetch(next.row);
      }
    });
    if (rose) scale_out(fall);
    lds_barrier();  // the loads of the tile after next stay in flight
    ahead(nb, 0, buf, 0);
    rose = settle(buf, t0, 1, whole, h2, h3, s1, fall);
    // after the last tile the next scores are those of an old buffer, and not used
    step(t0, buf, 1, s1, nb, 0, s0, buf, 0, [](int) {});
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
  for (int base = 0; base < count; base += TL_RUN) {
    if (base > 0) {
      __syncthreads();
      resolve(base);
      __syncthreads();
    }
    for (int i = base, end = min(base + TL_RUN, count); i < end; i += 3) {
      tile(i, base, B0{});
      if (i + 1 < end) tile(i + 1, base, B1{});
      if (i + 2 < end) tile(i + 2, base, B2{});
    }
  }
  if (count > 0) {
    if (count % 3 == 1) last(B0{});
    else if (count % 3 == 2) last(B1{});
    else last(B2{});
  }

  const float sum = sum_halves(l);
  m += SHIFT;
  if (parts <= 1) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __syncthreads();  // no wave reads keys or values any more
    int l2 = lane;
    asm volatile("" : "+v"(l2));  // or the addresses of the beginning stay in registers until here
    const int c2 = l2 & 31, h2 = l2 >> 5;
#pragma unroll
    for (int e = 0; e < DT; ++e)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *(u32x2*)(mine(c2, 4 * e + i / 4) + 8 * h2) = (u32x2){pack_bf16(acc[e][i] * inv, acc[e][i + 1] * inv),
                                                              pack_bf16(acc[e][i + 2] * inv, acc[e][i + 3] * inv)};
    const int64_t to = (w.t0 + tok) * a.out_stride + (int64_t)head * D;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int unit_row = i * (64 / CPR) + l2 / CPR;
      const int64_t at = of_row(to, unit_row);
      const u32x4 y = *(const u32x4*)mine(unit_row, l2 % CPR);
      if (wave * 32 + unit_row < w.n) *(u32x4*)(a.out + at + l2 % CPR * 8) = y;
    }
    if (a.lse && h == 0 && r < w.n) a.lse[(w.t0 + tok) * a.n_q + head] = sum == 0.f ? -__builtin_inff() : (m + __log2f(sum)) * LN2;
  } else if (r < w.n) {
    const int64_t to = ((int64_t)split * a.T + (w.t0 - a.first_row + tok)) * a.n_q + head;
#pragma unroll
    for (int e = 0; e < DT; ++e)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *(f32x4*)(a.part_o + to * D + 4 * h + 32 * e + 2 * i) = (f32x4){acc[e][i], acc[e][i + 1], acc[e][i + 2], acc[e][i + 3]};
    if (h == 0) *(f32x2*)(a.part_ml + 2 * to) = (f32x2){m, sum};
  }
}

template <int FORM>
hipError_t launch_attend_tile(const AttendArgs& a, bool fp8, int d, hipStream_t s) {
  constexpr int F = FORM ? FORM | FORM_SEEN : FORM_PLAIN;
  const dim3 grid((unsigned)(a.blocks * a.splits * a.c.n_kv));
  if (d == 64) {
    if (fp8) attend_tile_kernel<true, 64, F><<<grid, TL_THREADS, 0, s>>>(a);
    else attend_tile_kernel<false, 64, F><<<grid, TL_THREADS, 0, s>>>(a);
  } else {
    if (fp8) attend_tile_kernel<true, 128, F><<<grid, TL_THREADS, 0, s>>>(a);
    else attend_tile_kernel<false, 128, F><<<grid, TL_THREADS, 0, s>>>(a);
  }
  return hipGetLastError();
}

// One object of this file for each form.
#ifndef ATTEND_FORM
#define ATTEND_FORM 0
#endif
template hipError_t launch_attend_tile<ATTEND_FORM>(const AttendArgs&, bool, int, hipStream_t);

}  // namespace lsa
