// lsa_attend and lsa_attend_topk: attention over the paged cache, keys split among waves.
//
// Mathematics. For a row (one query head of one token) and the keys it sees,
//   out = sum_s 2^(x_s - m) V_s / sum_s 2^(x_s - m),  x_s = scale * log2(e) * q . K_s,
// with a running maximum m, so one pass over the keys is enough and any split of the keys can be
// joined: partial (m, l, o) triples add after scaling by 2^(m - m').
//
// Layout. Both products are formed transposed. S^T = K Q^T puts one row per lane (column
// lane % 16 of the 16x16 result) and four keys of it in the lane's registers, so the softmax needs
// no lane exchange except for a new maximum, and the four + four probabilities of a 32-key tile are
// already the operand of O^T = V^T P^T: the contraction may number its keys in any order, and the
// one that the registers hold is used. V^T's operand then wants, for each dimension, those eight
// keys of a lane group: every lane loads the same D/16 dimensions of its group's eight rows and
// transposes the small block in registers. Keys and values go from HBM to registers with no
// exchange through LDS, and no row block reads one twice (of listed entries with more than 64 query heads a key
// head, each row block of 64 heads reads the rows again).
//
// Precision. q and bf16 keys enter the matrix cores as they are, e4m3 codes widen to bf16 exactly;
// page scales multiply the fp32 score (keys) and the probability (values). The probability is
// rounded once, to bf16, for the second product; sums and accumulators are fp32. bf16 because the values' operand is
// bf16, and an fp32 probability would take a second product with what the rounding left. It costs as much as the output's own
// rounding at most: outputs are off by 1.9 to 2.3e-3 of their norm against 64 bits, where the output's rounding alone
// is 1.6 to 1.7e-3.
//
// The maximum follows the scores lazily: it is raised (and the accumulators rescaled) only when
// some score exceeds it by 2^8. Probabilities then stay below 2^8, and no bit is lost in fp32 or
// bf16, whose exponents have room.
//
// Split. HBM bounds it: G query heads share each row read. The 32-key tiles of all sequences are
// numbered through and cut on the device into equal shares for as many blocks as fit the device at once,
// so ragged lengths balance; a second launch joins the parts of a row (see AttendArgs). A block's four
// waves take its tiles in turn, with two or three of them in registers, and join through LDS.
//
// Measured on MI355X (64 query heads, 8 key heads, d_h 128; the kernel's time in a trace): 8 x 125,000 tokens in bf16,
// 4.10 GB, 602 us (6.8 TB/s); 32 ragged sequences of 4K to 128K in e4m3, 2.32 GB, 375 us (6.2 TB/s). Short calls are
// bound by latency: finding the share, the page table, the rows and the queries are four dependent
// reads, about 8 us with the launch, and the join 4 to 5 us (one sequence of 4096 tokens: 8.2 + 5.1 us).
// 33 to 64 rows (17 to 64 at d_h 128) take all registers, one wave a SIMD, and the bf16 instance of 64 at d_h 128 spills ten
// (44 bytes of scratch a lane): 64 rows over 131,072 tokens in bf16 take 108 us (5.0 TB/s) where 16 rows take 93 (5.8).
//
// Forms (kv.hpp). Caps and biases are instances of their own: the plain ones are as they were. What they add hides behind the
// reads with 16 rows: 8 x 125,000 tokens take 609 us plain, 612 capped, 623 with a bias and 626 with both (bf16; 333, 336, 336 and 342 in
// e4m3). Registers are what they are short of: a row's window, document and prefix lie in LDS, and a tile's distances are one number a row
// and lane (without these bf16 spilled 8 and 19 registers instead of 2 and 8: 624, 639 and 639 us). With 64 rows, where one
// wave a SIMD has to do it all, 8 x 40,000 tokens in bf16 take 45, 47, 47 and 52 us (45, 52, 56 and 57 before).
#include "kv.hpp"

namespace lsa {

static constexpr int AT_WAVES = 4;
static constexpr int AT_THREADS = 64 * AT_WAVES;

// One wave's tile of 32 keys in registers.
template <bool FP8, int D>
struct Tile {
  static constexpr int ROW = D * (FP8 ? 1 : 2);            // bytes of a cached row
  static constexpr int KL = ROW / 64;                      // 16-byte loads per lane and 16 keys
  static constexpr int VPL = D / 16;                       // dimensions a lane loads of each of its 8 value rows
  static constexpr int VB = VPL * (FP8 ? 1 : 2);           // bytes of them
  u32x4 k[2][KL];
  uint32_t v[8][VB / 4];
  // FP8, the scales: of the two 16 keys of K and of V; LISTED, of key lane % 32, of K in lanes 0-31 and of V above
  float scale[FP8 ? 4 : 1];
};

// The cached rows of a row block are read once in all, by non-temporal loads: 8 x 125,000 tokens in bf16 take 602 us with
// them (6.8 TB/s) and 677 us without. Listed rows, scattered and few, gain nothing from it.
template <bool NT, typename V>
__device__ __forceinline__ V load_once(const char* p) {
  if constexpr (NT) return __builtin_nontemporal_load((const V*)p);
  else return *(const V*)p;
}
template <bool NT, int N>
__device__ __forceinline__ void load_words(const char* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const u32x4 x = load_once<NT, u32x4>(p);
    w[0] = x[0]; w[1] = x[1]; w[2] = x[2]; w[3] = x[3];
  } else if constexpr (N == 2) {
    const u32x2 x = load_once<NT, u32x2>(p);
    w[0] = x[0]; w[1] = x[1];
  } else {
    w[0] = load_once<NT, uint32_t>(p);
  }
}

// Operand of contraction step s for the lane's key. The dimensions are numbered as the loads bring
// them: FP8 step 2c + e holds 64 c + 16 g + 8 e + j, bf16 step s holds 32 s + 8 g + j (j = 0..7).
template <bool FP8, int D>
__device__ __forceinline__ bf16x8 k_operand(const Tile<FP8, D>& t, int sub, int s) {
  if constexpr (FP8) {
    const u32x4 x = t.k[sub][s >> 1];
    const u32x2 lo = e4m3x4_to_bf16x4(x[2 * (s & 1)]), hi = e4m3x4_to_bf16x4(x[2 * (s & 1) + 1]);
    return as_bf16x8((u32x4){lo[0], lo[1], hi[0], hi[1]});
  } else {
    return as_bf16x8(t.k[sub][s]);
  }
}
template <bool FP8>
__device__ __forceinline__ int q_dim(int s, int g) {
  return FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
}

// Operand of the second product, dimension VPL * (lane % 16) + i: the lane group's 8 keys, in the
// order of the probabilities (4g .. 4g+3 of the first 16 keys, then of the second 16).
template <bool FP8, int D>
__device__ __forceinline__ bf16x8 v_operand(const Tile<FP8, D>& t, int i) {
  if constexpr (FP8) {
    const int w = i / 4, c = i % 4;
    const uint32_t sel = 0x0C0C0000u | ((uint32_t)c << 8) | (uint32_t)(c + 4);  // byte c of two dwords
    u32x4 r;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t lo = __builtin_amdgcn_perm(t.v[4 * x][w], t.v[4 * x + 1][w], sel);
      const uint32_t hi = __builtin_amdgcn_perm(t.v[4 * x + 2][w], t.v[4 * x + 3][w], sel);
      const u32x2 y = e4m3x4_to_bf16x4(lo | (hi << 16));
      r[2 * x] = y[0];
      r[2 * x + 1] = y[1];
    }
    return as_bf16x8(r);
  } else {
    const int w = i / 2;
    const uint32_t sel = i % 2 ? 0x07060302u : 0x05040100u;  // upper or lower halves of two dwords
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = __builtin_amdgcn_perm(t.v[2 * j + 1][w], t.v[2 * j][w], sel);
    return as_bf16x8(r);
  }
}

template <bool FP8, int D, int RT, bool LISTED, int FORM>
__global__ __launch_bounds__(AT_THREADS, attend_split_blocks(16 * RT, D)) void attend_split_kernel(const AttendArgs a) {
  using TileT = Tile<FP8, D>;
  constexpr int KS = D / 32, VPL = TileT::VPL, ROW = TileT::ROW, M = 16 * RT;
  constexpr int RUN = LISTED ? ATTEND_RESOLVED_LISTED : ATTEND_RESOLVED;
  constexpr int DEPTH = (FP8 || D == 64) && RT <= 2 && !LISTED ? 3 : 2;
  constexpr int PLACES = LISTED ? 32 : 2;  // places resolved per tile: single keys, or 16 in a row
  constexpr bool SEEN = (FORM & FORM_SEEN) != 0, CAP = (FORM & FORM_CAP) != 0, BIAS = (FORM & FORM_BIAS) != 0;
  __shared__ int64_t s_row[RUN * PLACES];  // cached row of the place, or -1: nothing there
  __shared__ int32_t s_tok[LISTED && BIAS ? RUN * PLACES : 1];  // position of the place
  // SEEN: what the rows' window, document and prefix let them see; only tiles at an edge ask, and registers are short
  __shared__ int32_t s_edge[SEEN ? 3 : 1][SEEN ? M : 1];
  __shared__ float s_o[AT_WAVES][M][D + 4];
  __shared__ float s_m[AT_WAVES][M], s_l[AT_WAVES][M];

  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), col = lane & 15, g = lane >> 4;
  const int h = (int)(blockIdx.x % a.c.n_kv);
  const int worker = (int)(blockIdx.x / a.c.n_kv);

  // The worker's share. The tiles of all row blocks are cut into `workers` equal runs of `share`; where it
  // takes no more workers, no run crosses into another row block, and each row block's runs are equal instead
  // (whole: units are runs, otherwise tiles). 64 row blocks are looked at at a time: `upto` is the sum of the units of
  // row blocks chunk .. chunk + lane, `before` that of the ones before the chunk. A row block with rows counts at
  // least one tile, so that someone writes the rows that see nothing.
  int chunk = 0, upto = 0, before = 0, at = 0, end = 0, share = 1, mine_tiles = 0;
  bool whole = false;
  Seq mine{};  // row block chunk + lane
  auto look = [&]() {
    const int e = chunk + lane;
    mine_tiles = 0;
    if (e < a.entries && entry_seq<LISTED, FORM>(a, e, &mine)) {
      Rows w;
      set_entry<LISTED, FORM>(a, e, mine, M, &w);
      mine_tiles = max(w.tiles, 1);
    }
  };
  auto units = [&]() { return whole ? (mine_tiles + share - 1) / share : mine_tiles; };
  if (a.workers > 0) {
    // several chunks are gone through three times; one is looked at once
    const bool one = a.entries <= 64;
    int total = 0, runs = 0;
    for (; chunk < a.entries; chunk += 64) {
      look();
      total += wave_last(wave_scan(mine_tiles));
    }
    share = max((total - 1) / a.workers + 1, AT_WAVES);
    if (!one) chunk = 0;
    for (whole = true; one ? runs == 0 && total > 0 : chunk < a.entries; chunk += 64) {
      if (!one) look();
      runs += wave_last(wave_scan(units()));
    }
    whole = runs <= a.workers;
    chunk = 0;
    if (!one) look();
    upto = wave_scan(units());
    at = whole ? worker : (int)min((int64_t)worker * share, (int64_t)total);
    end = whole ? min(worker + 1, runs) : (int)min((int64_t)at + share, (int64_t)total);
  }

  for (bool again = false;; again = true) {
  Rows w;
  int first = 0, count, slot = -1, entry = worker;  // slot: where the worker's part goes; negative: it is the whole
  if (a.workers > 0) {
    if (at >= end) return;
    while (at >= before + wave_last(upto)) {
      before += wave_last(upto);
      chunk += 64;
      look();
      upto = wave_scan(units());
    }
    const int which = __ffsll((unsigned long long)__ballot(before + upto > at)) - 1;
    entry = uni(chunk + which);
    auto of = [&](int x) { return __builtin_amdgcn_readlane(x, which); };
    Seq s{of(mine.n_tok), of(mine.len), of(mine.listed), of(mine.row), 0, 0, 0, 0};
    if constexpr (SEEN) {
      s.f_lo = of(mine.f_lo); s.f_hi = of(mine.f_hi); s.e_lo = of(mine.e_lo); s.e_hi = of(mine.e_hi);
    }
    set_entry<LISTED, FORM>(a, entry, s, M, &w);
    pin_rows<FORM>(&w);
    const int last = before + __builtin_amdgcn_readlane(upto, which), n = max(w.tiles, 1);
    int owner, parts;  // owner: the worker that begins this row block
    if (whole) {
      parts = (n + share - 1) / share;
      owner = last - parts;
      const int per = (n + parts - 1) / parts;
      first = (at - owner) * per;
      count = min(per, n - first);
      at = end;
    } else {
      const int begins = last - n;
      owner = begins / share;
      parts = (last - 1) / share - owner + 1;
      first = at - begins;
      count = min(end - at, n - first);
      at += count;
    }
    if (owner == worker && tid == 0) {
      a.joins[2 * (entry * a.c.n_kv + h)] = worker;
      a.joins[2 * (entry * a.c.n_kv + h) + 1] = parts > 1 ? parts : 0;
    }
    slot = uni(parts > 1 ? part_slot(a, worker, entry, owner) : -1);
    count = min(count, w.tiles - first);  // 0 where nothing is seen
  } else {
    Seq s;
    if (again || !entry_seq<LISTED, FORM>(a, entry, &s)) return;
    set_entry<LISTED, FORM>(a, entry, s, M, &w);
    pin_rows<FORM>(&w);
    count = w.tiles;
  }
  if (again) __syncthreads();

  f32x4 acc[RT][VPL];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = ATTEND_LOWEST;
    l[rt] = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[rt][i] = (f32x4){0.f, 0.f, 0.f, 0.f};
  }

  int base = first;  // first of the resolved tiles
  // where the keys of tiles tile0 .. tile0 + n - 1 lie
  auto resolve = [&](int tile0, int n) {
    for (int i = tid; i < n * PLACES; i += AT_THREADS) {
      const int tile = tile0 + i / PLACES;
      int tok = -1;
      if constexpr (LISTED) {
        if (tile < w.near.n) {
          tok = w.near.tile(tile) * 32 + i % 32;
          const bool seen = tok <= w.p_hi && ((a.window > 0 && tok > w.w_hi) || tok < a.sinks);
          tok = seen ? tok : -1;
        } else {
          const uint32_t at = (uint32_t)(tile - w.near.n) * 32 + i % 32, e = a.r == 1 ? at : at / (uint32_t)a.r;
          if ((int)e < w.listed) {
            const int32_t* list = a.idx + (int64_t)w.b * a.k;
            const int32_t entry = list[e];
            const int64_t far = (int64_t)entry * a.r + (at - e * a.r);
            const bool near = (a.window > 0 && far > w.w_hi) || far < a.sinks;
            if (entry >= 0 && far <= w.p_hi && !near && !(e > 0 && list[e - 1] == entry)) tok = (int)far;
          }
        }
      } else {
        tok = w.near.tile(tile) * 32 + (i % 2) * 16;
        // no row sees any of the 16: the page may not be the sequence's any more
        if (tok > end_hi<FORM>(w) || !some_begin<FORM>(a, w, tok, tok + 15)) tok = -1;
      }
      int64_t row = -1;
      if (tok >= 0) {
        const int32_t page = a.c.table[w.b * a.c.table_stride + (tok >> a.c.pt_log2)];
        if (page >= 0 && page < a.c.n_pages) {
          const int64_t t = (int64_t)page * a.c.n_kv + h;
          row = (t << a.c.pt_log2) + (tok & ((1 << a.c.pt_log2) - 1));
        }
      }
      s_row[i] = row;
      if constexpr (LISTED && BIAS) s_tok[i] = tok;
    }
  };

  // the first places are asked for before the queries: loads return in order, and the keys' wait for the places
  resolve(first, min(RUN, count));
  // the block's queries: lane column = row
  bf16x8 q[RT][KS];
  int32_t p_row[RT], w_row[SEEN ? 1 : RT];
  float slope[BIAS ? RT : 1];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = rt * 16 + col;
    const bool live = r < w.n;
    const int row = w.r0 + (live ? r : w.n - 1);
    const int tok = row / a.G;
    p_row[rt] = w.p0 + tok;
    if constexpr (!SEEN) {
      w_row[rt] = window_start(a, p_row[rt]);
    } else if (tid < 16) {  // for all waves, behind the places' barrier
      s_edge[0][r] = window_start(a, p_row[rt]);
      s_edge[1][r] = first_seen(a, w.t0 + tok);
      s_edge[2][r] = last_seen(a, w.t0 + tok, p_row[rt], w.len);
    }
    if constexpr (BIAS) slope[rt] = slope_log2(a, h * a.G + (row - tok * a.G));
    const uint16_t* src = a.q + (w.t0 + tok) * a.q_stride + (int64_t)(h * a.G + (row - tok * a.G)) * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4 x = *(const u32x4*)(src + q_dim<FP8>(s, g));
      if (!live) x = (u32x4){0, 0, 0, 0};
      q[rt][s] = as_bf16x8(x);
    }
  }

  // Loads of the resolved tile i. A place with nothing reads row 0 of the cache; what it brings is masked.
  auto load = [&](int i, TileT& t) {
    if constexpr (LISTED) {
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int64_t row = max(s_row[32 * i + 16 * sub + col], (int64_t)0);
#pragma unroll
        for (int c = 0; c < TileT::KL; ++c) t.k[sub][c] = load_once<false, u32x4>(a.c.k + row * ROW + 64 * c + 16 * g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t row = max(s_row[32 * i + 16 * (j / 4) + 4 * g + j % 4], (int64_t)0);
        load_words<false>(a.c.v + row * ROW + col * TileT::VB, t.v[j]);
      }
      if constexpr (FP8) {
        const int64_t row = max(s_row[32 * i + lane % 32], (int64_t)0);
        t.scale[0] = (lane < 32 ? a.c.k_scale : a.c.v_scale)[row >> a.c.pt_log2];
      }
    } else {
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int64_t row = max(uni(s_row[2 * i + sub]), (int64_t)0);
        const char* kb = a.c.k + row * ROW;
        const char* vb = a.c.v + row * ROW;
#pragma unroll
        for (int c = 0; c < TileT::KL; ++c) t.k[sub][c] = load_once<true, u32x4>(kb + (uint32_t)(col * ROW + 64 * c + 16 * g));
#pragma unroll
        for (int j = 0; j < 4; ++j) load_words<true>(vb + (uint32_t)((4 * g + j) * ROW + col * TileT::VB), t.v[4 * sub + j]);
        if constexpr (FP8) {
          t.scale[sub] = a.c.k_scale[row >> a.c.pt_log2];
          t.scale[2 + sub] = a.c.v_scale[row >> a.c.pt_log2];
        }
      }
    }
  };

  auto compute = [&](int i, TileT& t) {
    float ks[FP8 && LISTED ? 8 : 1], vs[FP8 && LISTED ? 8 : 1];
    if constexpr (FP8 && LISTED) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ks[j] = __shfl(t.scale[0], 16 * (j / 4) + 4 * g + j % 4);
        vs[j] = __shfl(t.scale[0], 32 + 16 * (j / 4) + 4 * g + j % 4);
      }
    }
    // x[rt][j]: score, base 2, of key 16 (j / 4) + 4 g + j % 4
    float x[RT][8];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      f32x4 s[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        const bf16x8 kk = k_operand<FP8, D>(t, sub, c);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, q[rt][c], s[rt], 0, 0, 0);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f = a.scale_log2;
          if constexpr (FP8) f *= LISTED ? ks[4 * sub + j] : t.scale[sub];
          float y = s[rt][j] * f;
          if constexpr (CAP) y = cap_score(a, y);
          x[rt][4 * sub + j] = y;
        }
    }
    if constexpr (BIAS) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        // the distance to the lane's first key, and from there on
        const float d = LISTED ? 0.f : (float)(p_row[rt] - (w.near.tile(base + i) * 32 + 4 * g));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = 16 * (j / 4) + j % 4;
          const float far = LISTED ? (float)(p_row[rt] - s_tok[32 * i + at + 4 * g]) : d - (float)at;
          x[rt][j] = __builtin_fmaf(-slope[rt], fabsf(far), x[rt][j]);
        }
      }
    }
    auto sees = [&](int rt, int tok) {
      if constexpr (SEEN) {
        const int r = rt * 16 + col;
        return tok <= s_edge[2][r] && tok >= s_edge[1][r] && (tok > s_edge[0][r] || tok < a.sinks);
      }
      else return tok <= p_row[rt] && (tok > w_row[rt] || tok < a.sinks);
    };
    // masks
    bool rescue = false;
    if constexpr (LISTED) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool gone = s_row[32 * i + 16 * (j / 4) + 4 * g + j % 4] < 0;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) x[rt][j] = gone ? -__builtin_inff() : x[rt][j];
#pragma unroll
        for (int e = 0; e < TileT::VB / 4; ++e) t.v[j][e] = gone ? 0u : t.v[j][e];
      }
    } else {
      const int t0 = w.near.tile(base + i) * 32;
      const bool here0 = uni(s_row[2 * i]) >= 0, here1 = uni(s_row[2 * i + 1]) >= 0;
      const bool whole = here0 && here1 && t0 + 31 <= end_lo<FORM>(w) && all_begin<FORM>(a, w, t0, t0 + 31);
      if (!whole) {
        uint32_t odd = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int tok = t0 + 16 * (j / 4) + 4 * g + j % 4;
          const bool here = j < 4 ? here0 : here1;
          const bool some = here && tok <= end_hi<FORM>(w) && some_begin<FORM>(a, w, tok, tok);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            x[rt][j] = here && sees(rt, tok) ? x[rt][j] : -__builtin_inff();
          }
#pragma unroll
          for (int e = 0; e < TileT::VB / 4; ++e) {
            t.v[j][e] = some ? t.v[j][e] : 0u;
            odd |= not_finite<FP8>(t.v[j][e]);
          }
        }
        // A value that is not finite would reach rows that do not see it as 0 * inf. Such values are
        // taken out of the product and added below to the rows that see them.
        if (w.p_lo != w.p_hi && __any(odd != 0)) {
          rescue = true;
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < TileT::VB / 4; ++e) t.v[j][e] &= ~not_finite<FP8>(t.v[j][e]);
        }
      }
    }
    // softmax
    bf16x8 p[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float top = x[rt][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = fmaxf(top, x[rt][j]);
      if (__any(top > m[rt] + ATTEND_LAZY)) {
        const float up = fmaxf(m[rt], max_column(top));
        const float f = __builtin_amdgcn_exp2f(m[rt] - up);
        m[rt] = up;
        l[rt] *= f;
#pragma unroll
        for (int e = 0; e < VPL; ++e) acc[rt][e] *= f;
      }
      u32x4 packed;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float y0 = __builtin_amdgcn_exp2f(x[rt][j] - m[rt]), y1 = __builtin_amdgcn_exp2f(x[rt][j + 1] - m[rt]);
        l[rt] += y0 + y1;
        if constexpr (FP8) {
          // where nothing is seen the scale may be anything: 0 stays 0
          const float v0 = LISTED ? vs[j] : t.scale[2 + j / 4], v1 = LISTED ? vs[j + 1] : v0;
          y0 = y0 == 0.f ? 0.f : y0 * v0;
          y1 = y1 == 0.f ? 0.f : y1 * v1;
        }
        packed[j / 2] = pack_bf16(y0, y1);
      }
      p[rt] = as_bf16x8(packed);
    }
#pragma unroll
    for (int e = 0; e < VPL; ++e) {
      const bf16x8 vv = v_operand<FP8, D>(t, e);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) acc[rt][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, p[rt], acc[rt][e], 0, 0, 0);
    }
    if constexpr (!LISTED) {
      if (rescue) {
        const int t0 = w.near.tile(base + i) * 32;
#pragma unroll 1
        for (int j = 0; j < 32; ++j) {
          const int64_t row = uni(s_row[2 * i + j / 16]);
          if (row < 0) continue;
          const char* src = a.c.v + (row + j % 16) * ROW;
          const int tok = t0 + j;
#pragma unroll
          for (int e = 0; e < VPL; ++e) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float y = cached_value<FP8>(src, VPL * (4 * g + c) + e);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt)
                if (sees(rt, tok) && !(fabsf(y) < __builtin_inff())) acc[rt][e][c] += y;
            }
            __builtin_amdgcn_sched_barrier(0);  // rare: keep its registers few
          }
        }
      }
    }
  };

  for (int done = 0; done < count; done += RUN) {
    const int n = min(RUN, count - done);
    base = first + done;
    if (done) {
      __syncthreads();
      resolve(base, n);
    }
    lds_barrier();
    if (wave >= n) continue;
    // DEPTH tiles in registers: the loads of the next ones are in flight while one is worked on
    TileT t[DEPTH];
#pragma unroll
    for (int x = 0; x < DEPTH - 1; ++x)
      if (wave + x * AT_WAVES < n) load(wave + x * AT_WAVES, t[x]);
    for (int i = wave; i < n; i += DEPTH * AT_WAVES) {
#pragma unroll
      for (int x = 0; x < DEPTH; ++x) {
        const int now = i + x * AT_WAVES, then = now + (DEPTH - 1) * AT_WAVES;
        if (then < n) load(then, t[(x + DEPTH - 1) % DEPTH]);
        if (now < n) compute(now, t[x]);
      }
    }
  }

  // join the waves' partial results
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float sum = sum_column(l[rt]);
    if (g == 0) {
      s_m[wave][rt * 16 + col] = m[rt];
      s_l[wave][rt * 16 + col] = sum;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < VPL; e += 4)
        *(f32x4*)&s_o[wave][rt * 16 + col][VPL * (4 * g + c) + e] = (f32x4){acc[rt][e][c], acc[rt][e + 1][c], acc[rt][e + 2][c], acc[rt][e + 3][c]};
  }
  __syncthreads();
  const int d0 = (tid % 16) * VPL;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = rt * 16 + tid / 16;
    if (r < w.n) {
      float top = s_m[0][r], sum = 0.f, o[VPL];
#pragma unroll
      for (int v = 1; v < AT_WAVES; ++v) top = fmaxf(top, s_m[v][r]);
#pragma unroll
      for (int e = 0; e < VPL; ++e) o[e] = 0.f;
#pragma unroll
      for (int v = 0; v < AT_WAVES; ++v) {
        const float f = __builtin_amdgcn_exp2f(s_m[v][r] - top);
        sum += s_l[v][r] * f;
#pragma unroll
        for (int e = 0; e < VPL; ++e) o[e] += s_o[v][r][d0 + e] * f;
      }
      const int row = w.r0 + r, tok = row / a.G, head = h * a.G + (row - tok * a.G);
      if (slot < 0) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint16_t* dst = a.out + (w.t0 + tok) * a.out_stride + (int64_t)head * D + d0;
#pragma unroll
        for (int e = 0; e < VPL; e += 4)
          *(u32x2*)(dst + e) = (u32x2){pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv)};
        if (a.lse && tid % 16 == 0)
          a.lse[(w.t0 + tok) * a.n_q + head] = sum == 0.f ? -__builtin_inff() : (top + __log2f(sum)) * LN2;
      } else {
        const int64_t to = ((int64_t)slot * a.c.n_kv + h) * M + r;
#pragma unroll
        for (int e = 0; e < VPL; e += 4) *(f32x4*)(a.part_o + to * D + d0 + e) = (f32x4){o[e], o[e + 1], o[e + 2], o[e + 3]};
        if (tid % 16 == 0) *(f32x2*)(a.part_ml + 2 * to) = (f32x2){top, sum};
      }
    }
  }
  }
}

// Joins `parts` partial results of one row, at first, first + step, ...: one wave per row.
template <int D>
__device__ __forceinline__ void join_row(const AttendArgs& a, int64_t first, int64_t step, int parts, int64_t row, int head) {
  constexpr int LP = D / 4, GP = 64 / LP, UN = 8;  // lanes of a part, parts at once, and of those in flight
  const int lane = threadIdx.x & 63, d0 = lane % LP * 4;
  f32x4 o[UN];
  auto fetch = [&](int s0, int s) {
    const int n = min(64, parts - s0);
#pragma unroll
    for (int u = 0; u < UN; ++u)
      o[u] = *(const f32x4*)(a.part_o + (first + (s0 + min(s + u * GP + lane / LP, n - 1)) * step) * D + d0);
  };
  fetch(0, 0);  // in flight beside the statistics
  float top = ATTEND_LOWEST;
  for (int s = lane; s < parts; s += 64) top = fmaxf(top, a.part_ml[2 * (first + s * step)]);
#pragma unroll
  for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
  float sum = 0.f;
  f32x4 acc = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < parts; s0 += 64) {
    const int n = min(64, parts - s0);
    float f = 0.f;
    if (lane < n) {
      const f32x2 ml = *(const f32x2*)(a.part_ml + 2 * (first + (s0 + lane) * step));
      f = __builtin_amdgcn_exp2f(ml[0] - top);
      sum += ml[1] * f;
    }
    for (int s = 0; s < n; s += GP * UN) {
      if (s0 + s > 0) fetch(s0, s);
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int at = s + u * GP + lane / LP;
        const float w = __shfl(f, at);
        // beyond the last part that one was read again: a factor of 0 would not clear an infinity
        if (at < n) acc += o[u] * w;
      }
    }
  }
#pragma unroll
  for (int o = LP; o < 64; o <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], o);
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (lane < LP)
    *(u32x2*)(a.out + row * a.out_stride + (int64_t)head * D + d0) =
        (u32x2){pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
  if (a.lse && lane == 0) a.lse[row * a.n_q + head] = sum == 0.f ? -__builtin_inff() : (top + __log2f(sum)) * LN2;
}

template <int D, bool LISTED>
__global__ __launch_bounds__(AT_THREADS) void split_join_kernel(const AttendArgs a, int M, int64_t from) {
  const int64_t id = from + (int64_t)blockIdx.x * AT_WAVES + (threadIdx.x >> 6);
  if (id >= a.T * a.n_q) return;
  const int64_t t = id / a.n_q;
  const int head = (int)(id - t * a.n_q), h = head / a.G;
  int entry, r = head - h * a.G;
  if constexpr (LISTED) {
    entry = (int)t * a.per + r / M;
    r %= M;
  } else {
    if (t + a.first_row >= a.off[a.B]) return;
    entry = wave_find(a.B, t + a.first_row, [&](int b) { return a.off[b]; });
    if (!of_class(a, a.off[entry + 1] - a.off[entry])) return;
    r += (int)(t + a.first_row - a.off[entry]) * a.G;
  }
  const int worker = a.joins[2 * ((int64_t)entry * a.c.n_kv + h)], parts = a.joins[2 * ((int64_t)entry * a.c.n_kv + h) + 1];
  if (parts == 0) return;
  join_row<D>(a, ((int64_t)part_slot(a, worker, entry, worker) * a.c.n_kv + h) * M + r, (int64_t)a.c.n_kv * M, parts, t + a.first_row, head);
}

template <int D, int FORM>
__global__ __launch_bounds__(AT_THREADS) void tile_join_kernel(const AttendArgs a, int64_t from) {
  const int64_t id = from + (int64_t)blockIdx.x * AT_WAVES + (threadIdx.x >> 6);
  if (id >= a.T * a.n_q) return;
  const int64_t t = id / a.n_q;
  const int head = (int)(id - t * a.n_q);
  if (t + a.first_row >= a.off[a.B]) return;
  Rows w;
  w.b = wave_find(a.B, t + a.first_row, [&](int b) { return a.off[b]; });
  w.t0 = a.off[w.b];
  const int64_t n_tok = a.off[w.b + 1] - w.t0;
  if (!of_class(a, n_tok)) return;
  const int64_t row = (t + a.first_row - w.t0) * a.G + head % a.G;
  set_block<FORM>(a, seq_of<false>(a, w.b, w.t0, n_tok), (int32_t)(row / ATTEND_TILE_ROWS), &w);
  const int parts = (w.tiles + a.run - 1) / a.run;
  if (parts > 1) join_row<D>(a, id, a.T * a.n_q, parts, t + a.first_row, head);
}

template <bool FP8, int D, bool LISTED, int FORM>
static hipError_t launch_rows(const AttendArgs& a, int row_tiles, hipStream_t s) {
  const dim3 grid((unsigned)((a.workers > 0 ? a.workers : a.entries) * (int64_t)a.c.n_kv));
  if (row_tiles == 1) attend_split_kernel<FP8, D, 1, LISTED, FORM><<<grid, AT_THREADS, 0, s>>>(a);
  else if (row_tiles == 2) attend_split_kernel<FP8, D, 2, LISTED, FORM><<<grid, AT_THREADS, 0, s>>>(a);
  else attend_split_kernel<FP8, D, 4, LISTED, FORM><<<grid, AT_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

template <bool LISTED, int FORM>
static hipError_t launch_dim(const AttendArgs& a, bool fp8, int d, int row_tiles, hipStream_t s) {
  if (d == 64) return fp8 ? launch_rows<true, 64, LISTED, FORM>(a, row_tiles, s) : launch_rows<false, 64, LISTED, FORM>(a, row_tiles, s);
  return fp8 ? launch_rows<true, 128, LISTED, FORM>(a, row_tiles, s) : launch_rows<false, 128, LISTED, FORM>(a, row_tiles, s);
}

// Listed positions are seen for what they are: there, forms with SEEN alone do not exist, and the others go without it.
template <int FORM>
hipError_t launch_attend_split(const AttendArgs& a, bool fp8, int d, int row_tiles, bool listed, hipStream_t s) {
  if (!listed) return launch_dim<false, FORM ? FORM | FORM_SEEN : FORM_PLAIN>(a, fp8, d, row_tiles, s);
  if constexpr (FORM == FORM_SEEN) return hipErrorInvalidValue;
  else return launch_dim<true, FORM>(a, fp8, d, row_tiles, s);
}

// One object of this file for each form, so that they are compiled side by side; the first has the joins.
#ifndef ATTEND_FORM
#define ATTEND_FORM 0
#endif
template hipError_t launch_attend_split<ATTEND_FORM>(const AttendArgs&, bool, int, int, bool, hipStream_t);

#if ATTEND_FORM == 0
// One wave per row and head, in launches of at most `most` blocks each: a launch has fewer than 2^32 threads.
template <typename F>
static hipError_t launch_joins(const AttendArgs& a, F launch) {
  constexpr int64_t most = (int64_t)(UINT32_MAX / AT_THREADS);
  const int64_t blocks = (a.T * a.n_q + AT_WAVES - 1) / AT_WAVES;
  hipError_t e = hipSuccess;
  for (int64_t at = 0; at < blocks && e == hipSuccess; at += most) {
    launch(dim3((unsigned)(blocks - at < most ? blocks - at : most)), at * AT_WAVES);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_attend_split_join(const AttendArgs& a, int d, int M, bool listed, hipStream_t s) {
  return launch_joins(a, [&](dim3 grid, int64_t from) {
    if (listed) {
      if (d == 64) split_join_kernel<64, true><<<grid, AT_THREADS, 0, s>>>(a, M, from);
      else split_join_kernel<128, true><<<grid, AT_THREADS, 0, s>>>(a, M, from);
    } else {
      if (d == 64) split_join_kernel<64, false><<<grid, AT_THREADS, 0, s>>>(a, M, from);
      else split_join_kernel<128, false><<<grid, AT_THREADS, 0, s>>>(a, M, from);
    }
  });
}

hipError_t launch_attend_tile_join(const AttendArgs& a, int d, bool seen, hipStream_t s) {
  return launch_joins(a, [&](dim3 grid, int64_t from) {
    if (seen) {
      if (d == 64) tile_join_kernel<64, FORM_SEEN><<<grid, AT_THREADS, 0, s>>>(a, from);
      else tile_join_kernel<128, FORM_SEEN><<<grid, AT_THREADS, 0, s>>>(a, from);
    } else {
      if (d == 64) tile_join_kernel<64, FORM_PLAIN><<<grid, AT_THREADS, 0, s>>>(a, from);
      else tile_join_kernel<128, FORM_PLAIN><<<grid, AT_THREADS, 0, s>>>(a, from);
    }
  });
}
#endif

}  // namespace lsa
