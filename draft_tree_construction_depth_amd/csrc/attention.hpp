// Attention of a verified block over a paged key/value cache.
//
// Row i of request b's block (0 the root, then the tree's nodes) sees the
// past_len[b] committed cache rows and, of the block's own rows past + j,
// those whose bit is set in row i of the ancestor mask (without a mask:
// j <= i, a chain). out_i = sum_n a_in V_n with a_i the softmax of
// scale * q_i . K_n over the rows seen; lse_i is that softmax's log-sum-exp.
// Query heads share key/value heads in groups of G = q_heads / kv_heads.
//
// One pass over the cache with the running maximum and sum of the softmax.
// The T * G query rows that share a key/value head form the columns of the
// products: a wave owns NQ = 32 of them (or 16) and forms S^T = K Q^T
// (32x32x16 MFMA, or 16x16x32; K fragments from LDS, Q fragments in
// registers), so that a lane holds scores of one query only: maximum, sum and
// rescaling need no reduction across lanes beyond an exchange between the
// wave's halves (quarters), and the weights leave the accumulator layout as
// the B operand of O^T += V^T P^T as they are. The accumulator's row order
// (4-row pieces dealt to the halves or quarters in turn) is the order in
// which V^T's columns are read; V's fragments come transposed out of
// row-major LDS (ds_read_b64_tr_b16).
//
// A workgroup is four waves: QW of them side by side over NQ QW queries, NG =
// 4 / QW groups of those over different cache rows, merged at the end. Few
// queries (plain decoding, short chains) are bound by the cache's bytes: up to
// 64 rows share a key/value head's pass, 16 to a wave (half the registers of
// 32), and as many waves as are left take other rows. More (trees) are bound
// by the products and the LDS reads that feed them, so all four waves share
// one staged tile, and 32 queries to a wave halve the LDS reads per product.
//
// The next tile's rows are in flight while the present one is worked on:
// straight into a second LDS buffer where there is one (64 trees of the sizes
// below 291 -> 280 us, on one box, against registers on the way; 32 blocks of 32 rows, heads
// of 256, 357 -> 330), else into registers. Work is cut evenly: all steps of
// all units (a unit: one request's, key/value head's and query tile's pass over
// the cache) lie on one axis, and each of the workgroups that the card holds at
// once takes an equal stretch of it, from the lengths on the device
// (attn_plan). A unit cut by a stretch's end leaves partial results in the
// workspace for attn_merge_kernel.
//
// Measured per call, by box and day (bf16, 32 query and 8 key/value heads of
// 128, unless said otherwise). 64 single tokens over 4 to 8 k rows: 297 to 314
// us, 1.61 GB at 5.1 to 5.4 TB/s, bound by HBM reads. 64 trees of 129 rows over
// 1 to 2 k: 272 to 294 us (f16 286 to 302), 166 GFLOP at 0.56 to 0.61 PFLOP/s;
// two waves on each SIMD (the accumulators, the queries and the scores fill
// the registers) leave the matrix units busy 26%, the vector units 35% and the
// LDS 24% of the time, and wait 38% of theirs; tiles of 32 rows with three
// workgroups to a CU spill (499 us), workgroups of eight waves take 335. 3
// chains of 17 rows over 50 to 100 k (f16, heads of 64, 40 and 8): 110 to 122 us,
// 461 MB at 3.8 to 4.2 TB/s. One tree of 65 rows over 1 k: 20 to 21 us, of which
// the merge is 4 and the steps are 6: a chain of waits. 32 blocks of 32 rows
// with 16 heads of 256 on 4 over 2 to 4 k: 194 us; 2 pieces of a prompt of 513
// rows over 4 to 8 k: 180 us.
//
// Caches of 8-bit rows (CACHE) go the same way: codes are loaded to registers
// and become values of the queries' type, which all of them have exactly, on
// their way into LDS; a row's scale multiplies its scores, or its weight. They
// halve the bytes and leave the products as they are. The same sizes: 64 single
// tokens 166 to 174 us (806 MB and 25 of scales at 4.9 TB/s), 64 trees 264 to
// 280, 3 chains 105 to 122 (bound by the vector units: exponentials, scales and
// masks; bf16 92 to 98), one tree 19. Heads of 256, one workgroup to a CU: 32
// blocks of 32 rows 186, 64 single tokens of 4 heads 229.
//
// Rows that all requests share (EXT, kAtPrefix and kAtRest): one pass over them
// with the query rows of the whole batch, whose maxima, sums and rows go to the
// workspace, then each request's own rows, which begin from those. 64 single
// tokens behind 8 k shared rows of 16 bits: 82 us, 270 without; 24 chains of 5
// rows (f16) behind 30 k of 8 bits: 123 to 132 us, 311 without.
#pragma once

#include "paged.hpp"

namespace ddt {

constexpr int kAtThreads = 256;
constexpr int kAtWaves = kAtThreads / kWave;
constexpr int kAtMerge = 2;       // 4-float pieces per lane of a merging wave

// Weights are 2^kBias at the maximum in use, which a score may pass by kSlack
// (log2): up to 2^8 in bf16, whose relative precision is the same at any size.
// A float16 weight loses bits below 2^-14 and is 0 below 2^-25, so its weights
// use the type's whole range: 2^14 at the maximum, 2^15 at most (65504 is the
// largest), full precision down to 2^-28 of the maximum in use and steps of
// 2^-38 of it below (n keys there put the output off by at most n 2^-39 |V|).
// The factor stays in the running sum and leaves with it.
template <typename H>
struct AttnWeight {
  static constexpr float kBias = __is_same(H, __bf16) ? 0.0f : 14.0f;
  static constexpr float kSlack = __is_same(H, __bf16) ? 8.0f : 1.0f;
};

typedef unsigned int at_u32x4 __attribute__((ext_vector_type(4)));
typedef short at_s16x4 __attribute__((ext_vector_type(4)));
typedef float at_f32x4 __attribute__((ext_vector_type(4)));
typedef float at_f32x16 __attribute__((ext_vector_type(16)));

// What a cache holds: elements of the queries' type, or 8-bit codes and a
// float32 scale for each row of a head.
enum { kAtSame, kAtE4M3, kAtI8 };

template <int DH_, int NQ_, int QW_, int CACHE_ = kAtSame>
struct AttnTile {
  static constexpr int DH = DH_, NQ = NQ_, QW = QW_, CACHE = CACHE_;
  static constexpr bool CODES = CACHE != kAtSame;
  static constexpr int NG = kAtWaves / QW;                 // groups over cache rows
  static constexpr int SK = QW == 4 && DH <= 128 ? 64 : 32;  // rows that a wave works on at once
  // Workgroups of a CU. Codes of heads of 64 leave LDS and registers for three,
  // with shorter tiles and some registers spilled. us with two / three, bf16, 8
  // key/value heads: 85 query rows, 3 requests over 50 to 100 k rows 117 / 110, 16
  // over 4 to 8 k 57 / 56, 64 over 1 to 2 k 54 / 60; 516 query rows 382 / 363, 180 /
  // 164, 185 / 169; f16 127 / 122, 65 / 65, 65 / 70; 429 / 413, 208 / 190, 221 / 202.
  static constexpr int PER_CU = DH == 256 ? 1 : (CODES && DH == 64 && NQ == 32 ? 3 : 2);
  static constexpr int KT = CODES && QW == 4 && DH == 64 && PER_CU == 2 ? 2 * SK : SK;  // rows of a group's tile
  static constexpr int TR = NG * KT;                       // rows of a workgroup's step
  static constexpr int ROW = DH * 2;                       // bytes of a row in LDS
  static constexpr int KROW = CODES ? ROW + 16 : ROW;      // ... of K's there, padded
  static constexpr int CROW = CODES ? DH : ROW;            // ... in the cache
  static constexpr int CPR = CROW / 16;                    // 16-byte chunks of a row there
  static constexpr int LOADS = KT * CPR / (QW * kWave);    // chunks per thread, K and V each
  static constexpr int NBUF = QW == 1 ? 1 : 2;             // one wave needs no second buffer
  static constexpr int KTILE = KT * KROW;                  // bytes of K of a tile
  static constexpr int TILE = KT * ROW;                    // ... of V (and of K unpadded)
  static constexpr int LDS = NG * NBUF * (KTILE + TILE);
  static constexpr int SCALES = CODES ? NG * NBUF * 2 * KT : 0;  // floats in LDS
  static constexpr int PIECES = DH * NQ / (4 * kWave);     // 4-float pieces of O per lane
  // tiles of codes in flight: two where the registers hold them
  static constexpr int PREFETCH = DH == 64 && NQ == 16 ? 2 : 1;
};

// What a workgroup's stretch leaves to merge: the unit that it begins and does
// not end (pieces 0: none), whose first piece is in slot 2 w + 1 and the others
// in 2 (w + 1), 2 (w + 2), ..., the continuations with which the next stretches
// begin.
struct AttnPlace {
  int32_t pieces, b, u;
  int32_t rows, waves, tiles;  // of AttnReq
  int32_t k;  // EXT: the stretch that begins it
  int32_t pad;
};

struct AttnParams {
  const void* q;  // [batch][T][q_heads][head_dim]
  const void* k_cache;
  const void* v_cache;
  int64_t batch;
  int32_t T, q_heads, kv_heads, G;
  int32_t groups;  // workgroups that share the work
  int32_t least;   // fewest steps for a workgroup of its own
  PagedRows rows;
  const int32_t* past_len;
  const int32_t* num_nodes;  // [batch], may be null: T - 1
  const uint64_t* mask;      // [batch][T][W], may be null: a chain
  int32_t W;
  float scale2;  // scale * log2(e)
  void* out;     // [batch][T][q_heads][head_dim]
  float* lse;    // [batch][T][q_heads], may be null
  AttnPlace* place;  // [groups]
  float* part;       // [slot][QW] of PIECES x 64 lanes x 4 floats, two slots a workgroup
  float* part_ml;    // [slot][QW][64 lanes][2]: running maximum (log2) and sum
  const float* k_scale;  // [pages][kv_heads][page_size], of caches of codes
  const float* v_scale;
  // A batch that shares its first rows (EXT kernels): kAtPrefix forms all
  // requests' block rows' state over those, as one request of batch * T rows;
  // kAtRest each request's over the rows behind, joined with that state.
  int32_t mode;
  int32_t requests;           // of the batch, for kAtPrefix (batch is 1 there)
  const int32_t* shared_len;  // [1]
  int32_t* prefix;            // [1], the shared rows in use: written by kAtPrefix
  float* pre_o;               // [batch][T][q_heads][head_dim], divided by the sums
  float* pre_ml;              // [batch][T][q_heads][2]: maximum (log2) and sum
  int32_t shared;             // *prefix, in the kernel
  int32_t few;  // EXT: at most kAtThreads requests, all their steps counted in 31 bits
  // EXT: `place` has an entry for each unit if by_unit (of as many as
  // place[places].pieces says), else for each workgroup
  int32_t places, by_unit;
};

enum { kAtAlone, kAtPrefix, kAtRest };
constexpr int kAtShare = 128;  // shared rows are used in multiples of every tile's TR

// Shared rows get a pass of their own where that keeps so many bytes from being
// read again, by as many requests as there are beyond one: the pass and its
// merge are 25 to 30 us, of which the reading that they save has to be more. us
// without / with, 8 key/value heads of 128, 4 query rows to each, own rows of
// 512: 16 bits, 2 requests x 8 k (34 MB saved) 33 / 36, 32 x 1 k (130 MB) 36 /
// 42, 8 x 8 k (235 MB) 58 / 40, 32 x 8 k (1 GB) 152 / 54; e4m3, 8 x 8 k (117 MB)
// 38 / 37, at 64 query rows 56 / 61, 16 x 8 k (252 MB) at 64 rows 92 / 83, 32 x 8 k
// 87 / 50.
constexpr int64_t kAtShareBytes = (int64_t)192 << 20;

// One request's work: rows [0, rows) of its block see anything (0: the
// request is taken out); its waves of NQ query rows per key/value head are
// dealt evenly to `tiles` query tiles.
struct AttnReq {
  int past, rows, len, steps, waves, tiles;
};

// The rest of a request, from its past and rows.
template <class C, bool EXT>
__host__ __device__ __forceinline__ void attn_request_sizes(const AttnParams& p, AttnReq& r) {
  const int64_t n = (int64_t)r.past + (EXT && p.mode == kAtPrefix ? 0 : r.rows);
  r.len = r.past < 0 ? 0 : (int)(n < p.rows.cap ? n : p.rows.cap);
  // one step for an empty request: its rows are cleared
  r.steps = r.len > C::TR ? (r.len + C::TR - 1) / C::TR : 1;
  if (EXT && p.mode == kAtRest) {  // (len >= shared where a request has rows)
    r.steps -= p.shared / C::TR;
    r.steps = r.steps > 1 ? r.steps : 1;
  }
  r.waves = (r.rows * p.G + C::NQ - 1) / C::NQ;
  r.tiles = r.waves > C::QW ? (r.waves + C::QW - 1) / C::QW : 1;
}

template <class C, bool EXT>
__device__ __forceinline__ AttnReq attn_request(const AttnParams& p, int64_t b) {
  static_assert(kAtShare % C::TR == 0, "shared rows are whole steps");
  AttnReq r;
  if (EXT && p.mode == kAtPrefix) {
    r.past = p.shared;
    r.rows = p.T;
    attn_request_sizes<C, EXT>(p, r);
    return r;
  }
  r.past = p.past_len[b];
  int nodes = p.num_nodes ? p.num_nodes[b] : p.T - 1;
  nodes = nodes < 0 ? 0 : (nodes > p.T - 1 ? p.T - 1 : nodes);
  r.rows = r.past < 0 ? 0 : nodes + 1;
  attn_request_sizes<C, EXT>(p, r);
  return r;
}

// Inclusive scan of one 64-bit number per lane.
__device__ __forceinline__ int64_t attn_wave_scan(int64_t x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Which of n stretches or units is workgroup w's (n or more: none, each number
// once). Consecutive workgroups of one XCD (ids 8 apart) take consecutive ones:
// query tiles of one key/value head read its rows from one L2, and no XCD has
// more than an eighth of all.
__host__ __device__ __forceinline__ int attn_nth(int w, int n) {
  const int per = (n + 7) >> 3;
  return (w >> 3) < per ? (w & 7) * per + (w >> 3) : w;
}

// A position on the axis of steps: request, unit of the request (key/value
// head, then query tile) and step.
struct AttnPos {
  int64_t x;  // steps before it
  int b, u, s;
};

// attn_plan's shared memory.
struct AttnScratch {
  int64_t part[kAtWaves][2];
  int longest[kAtWaves];
  AttnPos pos[2];
};

// attn_plan_few's.
struct AttnFew {
  int part[2][kAtWaves][2];
  int longest[kAtWaves];
  alignas(16) int steps[kAtThreads];
  int past[kAtThreads], rows[kAtThreads], order[kAtThreads], units[kAtThreads];
  AttnPos pos[2];
  int b, i;
  int unit;  // units of requests before the first position's
};

// A workgroup's shared memory, all of it in one object, so that the tiles lie
// at its start: loads straight into LDS go to the 64 KiB that m0's 16 bits
// reach, which the tiles may fill.
template <class C, bool EXT>
struct AttnLds {
  alignas(256) unsigned char tiles[C::LDS];
  int any[kAtWaves];
  AttnScratch plan;
  alignas(16) unsigned char few[EXT ? sizeof(AttnFew) : 1];
  alignas(16) float scale[C::SCALES ? C::SCALES : 1];  // [NG][NBUF]: K's times scale2, then V's
  // [NG][NBUF][QW]: of what a wave staged, the largest scale of V; NaN codes of V
  alignas(16) float most[C::CODES ? kAtWaves * C::NBUF : 1];
  int flag[C::CODES ? kAtWaves * C::NBUF : 1];
};

// The cut of the axis: end e of n stretches lies at total * e / n.
struct AttnCut {
  int64_t n, total, range, extra, slack;
};

__device__ __forceinline__ AttnPos attn_uniform(const AttnPos& a) {
  const uint64_t x = (uint64_t)a.x;
  return AttnPos{
      (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 |
                (uint32_t)__builtin_amdgcn_readfirstlane((int)x)),
      __builtin_amdgcn_readfirstlane(a.b), __builtin_amdgcn_readfirstlane(a.u),
      __builtin_amdgcn_readfirstlane(a.s)};
}

// a / b for a >= 0, b > 0: a 64-bit division is some 130 instructions and
// hardly ever needed.
__device__ __forceinline__ int64_t attn_div(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

__device__ __forceinline__ int64_t attn_end(const AttnCut& c, int64_t e) {
  return c.range * e + attn_div(c.extra * e, c.n);
}

// Step s of a unit's `steps` as the end of a stretch: 0 or `steps` where that
// is near.
__device__ __forceinline__ int64_t attn_near(const AttnCut& c, int64_t s, int steps) {
  if (s <= c.slack && s <= steps - s) return 0;
  return steps - s <= c.slack ? steps : s;
}

// The stretch [from, to) of workgroup w; false: none. The axis is request
// after request, each tiles * kv_heads units of `steps`, cut evenly for the
// p.groups workgroups that the card holds at once. An end that falls close to
// a unit's is moved there: by up to an eighth of a stretch, so that short
// units are not cut at all, or, where a stretch is a few steps, by up to half
// of one, so that no stretch has the start of two units to wait for.
//
// With many units, none of them long, each workgroup takes a whole one (to.x
// < 0): the units' cache rows are then read by a key/value head's query tiles
// at the same time, and the hardware deals the units out as they end.
template <class C, bool EXT>
__device__ bool attn_plan(const AttnParams& p, AttnScratch& sh, int w, int& k, AttnCut& cut,
                          AttnPos& from, AttnPos& to) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto axis = [&](int64_t b, int64_t& units, int& steps) {
    units = 0;
    steps = 0;
    if (b >= p.batch) return;
    const AttnReq r = attn_request<C, EXT>(p, b);
    units = (int64_t)r.tiles * p.kv_heads;
    steps = r.steps;
  };
  int64_t total = 0, all_units = 0, units;
  int longest = 0, steps;
  if (p.batch == 1) {
    axis(0, all_units, longest);
    total = all_units * longest;
  } else {
    for (int64_t b = tid; b < p.batch; b += kAtThreads) {
      axis(b, units, steps);
      total += units * steps;
      all_units += units;
      longest = steps > longest ? steps : longest;
    }
    total = attn_wave_scan(total);
    all_units = attn_wave_scan(all_units);
    longest = wave_max(longest);
    if (lane == 63) {
      sh.part[wave][0] = total;
      sh.part[wave][1] = all_units;
      sh.longest[wave] = longest;
    }
    __syncthreads();
    total = all_units = 0;
#pragma unroll
    for (int i = 0; i < kAtWaves; ++i) {
      total += sh.part[i][0];
      all_units += sh.part[i][1];
      longest = sh.longest[i] > longest ? sh.longest[i] : longest;
    }
  }
  const bool whole = all_units >= 2 * p.groups && longest * (int64_t)p.groups <= total;
  const int64_t want = attn_div(total + p.least - 1, p.least);
  const int64_t n = whole ? all_units : (want < p.groups ? want : p.groups);
  // consecutive workgroups of one XCD (ids 8 apart) take consecutive
  // stretches: query tiles of one unit read its rows from one L2
  const int64_t per = (n + 7) >> 3;
  k = w;
  if ((w >> 3) >= per) return false;  // (these keep their numbers: those from 8 per on)
  k = (int)((w & 7) * per) + (w >> 3);
  if (k >= n) return false;
  cut.n = n;
  cut.total = total;
  cut.range = attn_div(total, n);
  cut.extra = total - cut.range * n;
  cut.slack = cut.range < 8 ? cut.range >> 1 : cut.range >> 3;
  // end number e of the stretches, as a position in the request that holds it
  auto place = [&](int64_t e, int64_t before, int b, AttnPos& at) {
    if (whole) {
      at = AttnPos{-1, b, (int)(e - before), 0};
      return;
    }
    const AttnReq r = attn_request<C, EXT>(p, b);
    const int64_t x = attn_end(cut, e) - before;
    int64_t u = attn_div(x, r.steps), s = x - u * r.steps;
    if (e > 0 && e < n) s = attn_near(cut, s, r.steps);
    at.x = before + u * r.steps + s;
    at.b = b;
    at.u = (int)u + (s == r.steps);
    at.s = s == r.steps ? 0 : (int)s;
  };
  if (p.batch == 1) {
    place(k, 0, 0, from);
    place(k + 1, 0, 0, to);
  } else {
    const int64_t x0 = whole ? k : attn_end(cut, k),
                  x1 = whole ? k + 1 : attn_end(cut, k + 1);
    int64_t base = 0;
    for (int64_t b0 = 0; b0 < p.batch; b0 += kAtThreads) {
      const int64_t b = b0 + tid;
      axis(b, units, steps);
      const int64_t mine = whole ? units : units * steps;
      int64_t incl = attn_wave_scan(mine);
      __syncthreads();  // sh.part's readers before this round
      if (lane == 63) sh.part[wave][0] = incl;
      __syncthreads();
      int64_t all = 0;
#pragma unroll
      for (int i = 0; i < kAtWaves; ++i) {
        incl += i < wave ? sh.part[i][0] : 0;
        all += sh.part[i][0];
      }
      const int64_t before = base + incl - mine;
      if (x0 >= before && x0 < before + mine) place(k, before, (int)b, sh.pos[0]);
      // (the axis' own end belongs to the last request)
      if (x1 > before && x1 <= before + mine) place(k + 1, before, (int)b, sh.pos[1]);
      base += all;
      if (base >= x1) break;  // uniform
    }
    __syncthreads();
    from = attn_uniform(sh.pos[0]);
    to = attn_uniform(sh.pos[1]);
  }
  return true;
}

// Inclusive sum over the wave of one 32-bit number per lane, by DPP moves.
__device__ __forceinline__ int attn_wave_sum(int x) {
  x += (int)dpp_u32<0x111>((uint32_t)x);  // row_shr:1, 2, 4, 8
  x += (int)dpp_u32<0x112>((uint32_t)x);
  x += (int)dpp_u32<0x114>((uint32_t)x);
  x += (int)dpp_u32<0x118>((uint32_t)x);
  // the rows' totals: lane 15 to row 1 and lane 47 to row 3, lane 31 to rows 2 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return x;
}

// attn_plan for at most kAtThreads requests whose steps are counted in 31 bits:
// a thread holds a request, whose lengths are read once.
//
// The cut is attn_plan's. Whole units go to the workgroups of one XCD after the
// other: key/value head h of request b is the work of XCD (b * kv_heads + h) % 8,
// which reads its rows once for all its query tiles, and each XCD's longest
// requests come first, so that the card runs dry at once. (64 trees of 129
// rows over 1 to 2 k rows, a request's heads on one XCD and in the requests'
// order: of 334 us a fifth passed with workgroups ending one by one.) One
// request's units, and those of few heads in many query tiles, of which some
// XCDs would get more than others, are dealt as attn_plan deals them (us by head
// / as here: 32832 query rows of one head of 256 over 2 k rows of int8 2228 / 407,
// three requests of 12312 918 / 411; behind 8 k shared rows of 16 bits, heads of
// 128, 163840 query rows of one 4764 / 907, 40960 of each of four 1448 / 865, of
// twelve 3221 / 2440, of eight 1612 / 1612).
template <class C>
__device__ bool attn_plan_few(const AttnParams& p, AttnFew& sh, int w, int& k, AttnCut& cut,
                              AttnPos& from, AttnPos& to, AttnReq& rq, int& unit, int& all_units) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, batch = (int)p.batch;
  auto stretches = [&](int total) -> int {
    const int want = __builtin_amdgcn_readfirstlane(
        (int)(((uint32_t)total + (uint32_t)p.least - 1) / (uint32_t)p.least));
    return want < p.groups ? want : p.groups;
  };
  auto dealt_whole = [&](int total, int longest) -> bool {
    if (!p.by_unit) return all_units >= 2 * p.groups && longest * (int64_t)p.groups <= total;
    // One round: whole units spare the second start of most stretches and the
    // merge, and workgroups of long and short units share a CU; cut ones fill the
    // card. us cut / whole over 0.5 to 1 k rows, 2 to 4 k: 64 single tokens (128 rows
    // to a step) 34 / 30, 93 / 90, 52 of them 32 / 28, 71 / 74, 33 of them 25 /
    // 26, 48 / 67; 64 requests of 128 query rows (64 to a step) 65 / 53, 156 /
    // 151, 46 of them 53 / 50, 123 / 141; 64 of 64 query rows over 8 to 16 k 430 / 461.
    // (Two workgroups to a CU keep it nearly as busy as three.) Too little work for
    // that is cut into stretches of p.least steps, which end sooner than units of
    // more than twice that: a call over 150 rows, 64-row steps, one tree of 65 16 /
    // 17, 16 of them 30 / 24; heads of 256, 32-row steps, 16 query rows 15.5 / 19.6.
    constexpr int kFull = C::PER_CU == 1 ? 256 : 512;
    int g = stretches(total);
    const int spare = g < kFull ? 2 : 4;
    g = g < kFull ? g : kFull;
    const int64_t even = total;  // steps of an even stretch, in 1 / g
    return 2 * (int64_t)longest * g <= 3 * even + 8 * g && longest * (int64_t)g <= even + 20 * g &&
           even * g < (even + spare * g) * all_units;
  };
  // the cut, and whether workgroup w has stretch k of it
  auto stretch = [&](int total) -> bool {
    const int n = stretches(total);
    k = attn_nth(w, n);
    if (k >= n) return false;
    const int range = __builtin_amdgcn_readfirstlane((int)((uint32_t)total / (uint32_t)n));
    cut.n = n;
    cut.total = total;
    cut.range = range;
    cut.extra = total - range * n;
    // (a step at least: 64 requests of 4 to 9 steps behind shared rows, 6.5 to a
    // stretch, 66 us with half a stretch to either side and 60 with one step)
    cut.slack = range < 4 ? range >> 1 : (range < 8 ? 1 : range >> 3);
    return true;
  };
  auto end = [&](int e) -> int {  // attn_end: extra * e is below 2^20
    const uint32_t more = (uint32_t)((int)cut.extra * e) / (uint32_t)(int)cut.n;
    return (int)cut.range * e + __builtin_amdgcn_readfirstlane((int)more);
  };
  if (batch == 1) {
    // One request (and a batch's shared rows): nothing to add up, so all of it is
    // in scalars, without the LDS (one tree of 65 rows over 1 k: 19.9 -> 19.1 us).
    rq = attn_request<C, true>(p, 0);
    rq.past = __builtin_amdgcn_readfirstlane(rq.past);
    rq.rows = __builtin_amdgcn_readfirstlane(rq.rows);
    attn_request_sizes<C, true>(p, rq);
    all_units = rq.tiles * p.kv_heads;
    unit = 0;
    const int total = all_units * rq.steps;
    k = w;
    if (dealt_whole(total, rq.steps)) {
      const int u = attn_nth(w, all_units);
      if (u >= all_units) return false;
      from = AttnPos{-1, 0, u, 0};
      to = AttnPos{-1, 0, u + 1, 0};
      return true;
    }
    if (!stretch(total)) return false;
    auto place = [&](int e) -> AttnPos {
      const int x = end(e);
      const int u = __builtin_amdgcn_readfirstlane((int)((uint32_t)x / (uint32_t)rq.steps));
      int step = x - u * rq.steps;
      if (e > 0 && e < (int)cut.n) step = (int)attn_near(cut, step, rq.steps);
      const bool past = step == rq.steps;
      return attn_uniform(AttnPos{(int64_t)u * rq.steps + step, 0, u + past, past ? 0 : step});
    };
    from = place(k);
    to = place(k + 1);
    return true;
  }
  AttnReq r;
  r.past = r.rows = r.steps = 0;
  r.tiles = 1;
  int units = 0;
  if (tid < batch) {
    r = attn_request<C, true>(p, tid);
    units = r.tiles * p.kv_heads;
  }
  const int mine = units * r.steps;
  const int steps_to = attn_wave_sum(mine), units_to = attn_wave_sum(units);
  const int longest_here = wave_max(r.steps);
  sh.steps[tid] = r.steps;
  sh.past[tid] = r.past;
  sh.rows[tid] = r.rows;
  if (lane == 63) {
    sh.part[0][wave][0] = steps_to;
    sh.part[0][wave][1] = units_to;
    sh.longest[wave] = longest_here;
  }
  __syncthreads();
  int total = 0, longest = 0, before = steps_to - mine;
  all_units = 0;
  int units_before = units_to - units;
#pragma unroll
  for (int i = 0; i < kAtWaves; ++i) {
    before += i < wave ? sh.part[0][i][0] : 0;
    units_before += i < wave ? sh.part[0][i][1] : 0;
    total += sh.part[0][i][0];
    all_units += sh.part[0][i][1];
    longest = sh.longest[i] > longest ? sh.longest[i] : longest;
  }
  total = __builtin_amdgcn_readfirstlane(total);
  longest = __builtin_amdgcn_readfirstlane(longest);
  all_units = __builtin_amdgcn_readfirstlane(all_units);
  if (!dealt_whole(total, longest)) {
    if (!stretch(total)) return false;
    const int x0 = end(k), x1 = end(k + 1), n = (int)cut.n;
    auto place = [&](int e, int x, AttnPos& at) {
      x -= before;
      int u = (int)((uint32_t)x / (uint32_t)r.steps), s = x - u * r.steps;
      if (e > 0 && e < n) s = (int)attn_near(cut, s, r.steps);
      at.x = (int64_t)before + u * r.steps + s;
      at.b = tid;
      at.u = u + (s == r.steps);
      at.s = s == r.steps ? 0 : s;
    };
    if (x0 >= before && x0 < before + mine) {
      place(k, x0, sh.pos[0]);
      sh.unit = units_before;
    }
    if (x1 > before && x1 <= before + mine) place(k + 1, x1, sh.pos[1]);
    __syncthreads();
    from = attn_uniform(sh.pos[0]);
    to = attn_uniform(sh.pos[1]);
    unit = __builtin_amdgcn_readfirstlane(sh.unit);
  } else if (!p.by_unit && batch * p.kv_heads < 64 && (batch * p.kv_heads & 7)) {
    // heads that do not fill the XCDs alike, in query tiles that fill the card
    const int n = attn_nth(w, all_units);
    k = w;
    if (n >= all_units) return false;
    if (n >= units_before && n < units_before + units)
      sh.pos[0] = AttnPos{-1, tid, n - units_before, 0};
    __syncthreads();
    from = attn_uniform(sh.pos[0]);
    to = AttnPos{-1, from.b, from.u + 1, 0};
  } else {
    // requests by their steps, the longest first
    int rank = 0;
    for (int j = 0; j < batch; j += 4) {
      const int4 other = *(const int4*)(sh.steps + j);
      rank += (other.x > r.steps) | ((other.x == r.steps) & (j < tid));
      rank += (other.y > r.steps) | ((other.y == r.steps) & (j + 1 < tid));
      rank += (other.z > r.steps) | ((other.z == r.steps) & (j + 2 < tid));
      rank += (other.w > r.steps) | ((other.w == r.steps) & (j + 3 < tid));
    }
    // (threads without a request have no steps, requests one at least)
    const int xcd = w & 7, h0 = (xcd - tid * p.kv_heads) & 7;
    sh.order[rank] = tid;
    sh.units[rank] =
        tid < batch && h0 < p.kv_heads ? ((p.kv_heads - 1 - h0) / 8 + 1) * r.tiles : 0;
    if (tid == 0) sh.b = -1;
    __syncthreads();
    const int have = tid < batch ? sh.units[tid] : 0, to_here = attn_wave_sum(have);
    if (lane == 63) sh.part[1][wave][0] = to_here;
    __syncthreads();
    int first = to_here - have;
#pragma unroll
    for (int i = 0; i < kAtWaves; ++i) first += i < wave ? sh.part[1][i][0] : 0;
    const int i = w >> 3;
    if (i >= first && i < first + have) {
      sh.b = sh.order[tid];
      sh.i = i - first;
    }
    __syncthreads();
    k = w;
    const int b = __builtin_amdgcn_readfirstlane(sh.b);
    if (b < 0) return false;
    rq.past = sh.past[b];
    rq.rows = sh.rows[b];
    attn_request_sizes<C, true>(p, rq);
    const int at = __builtin_amdgcn_readfirstlane(sh.i), group = at / rq.tiles;
    const int head = ((xcd - b * p.kv_heads) & 7) + 8 * group;
    from = AttnPos{-1, b, head * rq.tiles + (at - group * rq.tiles), 0};
    to = AttnPos{-1, b, from.u + 1, 0};
  }
  rq.past = __builtin_amdgcn_readfirstlane(sh.past[from.b]);
  rq.rows = __builtin_amdgcn_readfirstlane(sh.rows[from.b]);
  attn_request_sizes<C, true>(p, rq);
  return true;
}

template <typename H>
__device__ __forceinline__ at_f32x16 attn_mfma(at_u32x4 a, at_u32x4 b, at_f32x16 c) {
  typedef H v8 __attribute__((ext_vector_type(8)));
  if constexpr (__is_same(H, __bf16))
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a),
                                                   __builtin_bit_cast(v8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a),
                                                  __builtin_bit_cast(v8, b), c, 0, 0, 0);
}
template <typename H>
__device__ __forceinline__ at_f32x4 attn_mfma(at_u32x4 a, at_u32x4 b, at_f32x4 c) {
  typedef H v8 __attribute__((ext_vector_type(8)));
  if constexpr (__is_same(H, __bf16))
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a),
                                                   __builtin_bit_cast(v8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a),
                                                  __builtin_bit_cast(v8, b), c, 0, 0, 0);
}

// Over the lanes that hold the same query: l and l + 32, or l % 16 in all
// four quarters.
template <int NQ, typename Op>
__device__ __forceinline__ float attn_across(float x, Op op) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  if constexpr (NQ == 16) {
    const auto t =
        __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = op(__uint_as_float(t[0]), __uint_as_float(t[1]));
  }
  return x;
}
template <int NQ>
__device__ __forceinline__ float attn_max_across(float x) {
  return attn_across<NQ>(x, [](float a, float b) { return fmaxf(a, b); });
}
template <int NQ>
__device__ __forceinline__ float attn_sum_across(float x) {
  return attn_across<NQ>(x, [](float a, float b) { return a + b; });
}

// Places of a 16-byte chunk in a staged tile. K is read 32 rows at a time at
// one chunk, V four rows at a time at two neighbouring chunks; both orders
// spread such a read over the 64 banks.
template <int DH>
__device__ __forceinline__ int attn_k_chunk(int row, int c) {
  return c ^ (DH == 64 ? (row >> 1) & 7 : row & 15);
}
template <int DH>
__device__ __forceinline__ int attn_v_chunk(int row, int c) {
  return c ^ (DH == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2);
}

template <typename H>
__device__ __forceinline__ bool attn_not_finite(uint32_t two) {
  constexpr uint32_t e = __is_same(H, __bf16) ? 0x7F80u : 0x7C00u;
  return (two & e) == e || (two >> 16 & e) == e;
}
template <typename H>
__device__ __forceinline__ uint32_t attn_finite_only(uint32_t two) {
  constexpr uint32_t e = __is_same(H, __bf16) ? 0x7F80u : 0x7C00u;
  two = (two & e) == e ? two & 0xFFFF0000u : two;
  return (two >> 16 & e) == e ? two & 0xFFFFu : two;
}

// The values of 16 codes, in order: all of them have exact values in H.
template <typename H, int CACHE>
__device__ __forceinline__ void attn_values(at_u32x4 codes, at_u32x4 (&x)[2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    if constexpr (CACHE == kAtE4M3) {
      if constexpr (__is_same(H, __bf16)) {
        lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], 1.0f, false));
        hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], 1.0f, true));
      } else {
        lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes[i], 1.0f, false));
        hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes[i], 1.0f, true));
      }
    } else {
      typedef float f2 __attribute__((ext_vector_type(2)));
      typedef H h2 __attribute__((ext_vector_type(2)));
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = (float)(int8_t)(codes[i] >> (8 * e));
      lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{f[0], f[1]}, h2));
      hi = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{f[2], f[3]}, h2));
    }
    x[i >> 1][2 * (i & 1)] = lo;
    x[i >> 1][2 * (i & 1) + 1] = hi;
  }
}

template <int N>
struct AttnNumber {
  static constexpr int value = N;
};
struct AttnFalse {
  static constexpr bool value = false;
};
struct AttnTrue {
  static constexpr bool value = true;
};

// A wave's running softmax over its NQ queries: lane l has query l % NQ; the
// lanes with one query hold different rows of S^T and O^T.
template <int DH, int NQ>
struct AttnState;

template <int DH>
struct AttnState<DH, 32> {
  static constexpr int PIECES = DH / 8, R = 16;  // registers of an accumulator
  float m, mref, l;  // maximum in use (log2), the same less kBias or 0 while it is -inf, sum of weights
  float unit;  // of float16 weights for caches of codes: o and l are in units of 2^unit
  at_f32x16 o[DH / 32];
  __device__ __forceinline__ at_f32x4 get(int j) const {
    const at_f32x16& x = o[j >> 2];
    const int r = 4 * (j & 3);
    return at_f32x4{x[r], x[r + 1], x[r + 2], x[r + 3]};
  }
  __device__ __forceinline__ void set(int j, at_f32x4 v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j >> 2][4 * (j & 3) + e] = v[e];
  }
  // first of the four head elements of piece j
  static __device__ __forceinline__ int element(int j, int lane) {
    return 32 * (j >> 2) + 8 * (j & 3) + 4 * (lane >> 5);
  }
};

template <int DH>
struct AttnState<DH, 16> {
  static constexpr int PIECES = DH / 16, R = 4;
  float m, mref, l;
  float unit;
  at_f32x4 o[DH / 16];
  __device__ __forceinline__ at_f32x4 get(int j) const { return o[j]; }
  __device__ __forceinline__ void set(int j, at_f32x4 v) { o[j] = v; }
  static __device__ __forceinline__ int element(int j, int lane) { return 16 * j + 4 * (lane >> 4); }
};

// Rows of the group's tile that this lane's query sees, as bits.
template <int KT>
__device__ __forceinline__ uint64_t attn_visible(const AttnParams& p, int64_t b, int past, int r0,
                                                 int i, bool live, uint64_t held) {
  if (!live) return 0;
  const int a = past - r0;  // rows of the tile before the block
  uint64_t v = a >= 64 ? ~0ull : (a > 0 ? (1ull << a) - 1 : 0ull);
  if (a < 64) {
    if (p.mask) {
      const uint64_t* words = p.mask + (b * p.T + i) * p.W;
      if (a >= 0) {
        v |= words[0] << a;
      } else {
        const int k = -a >> 6, s = -a & 63;
        if (k < p.W) v |= words[k] >> s;
        if (s && k + 1 < p.W) v |= words[k + 1] << (64 - s);
      }
    } else {
      const int n = i + 1 + a;  // rows up to the query's own
      v |= n >= 64 ? ~0ull : (n > 0 ? (1ull << n) - 1 : 0ull);
    }
  }
  return v & held;
}

// One staged tile. k, v: its rows in LDS; MASKED: vis says which are seen.
template <typename H, int DH, int NQ, int KT, bool MASKED>
__device__ __forceinline__ void attn_tile(const unsigned char* k, const unsigned char* v,
                                          const at_u32x4 (&q)[DH * NQ / 512], float scale2,
                                          uint64_t vis, AttnState<DH, NQ>& st, int lane) {
  typedef AttnState<DH, NQ> State;
  constexpr int NB = KT / NQ, R = State::R, ROW = DH * 2, CPR = DH / 8;
  constexpr int Z = kWave / NQ;  // lanes with one query
  const int z = lane / NQ;
  decltype(st.o[0] + st.o[0]) s[NB];
#pragma unroll
  for (int t = 0; t < NB; ++t) {
#pragma unroll
    for (int r = 0; r < R; ++r) s[t][r] = 0.0f;
    const int row = NQ * t + lane % NQ;
    at_u32x4 a[CPR / Z];
#pragma unroll
    for (int c = 0; c < CPR / Z; ++c)
      a[c] = *(const at_u32x4*)(k + row * ROW + attn_k_chunk<DH>(row, Z * c + z) * 16);
#pragma unroll
    for (int c = 0; c < CPR / Z; ++c) s[t] = attn_mfma<H>(a[c], q[c], s[t]);
  }
  // four fragments' reads ahead of the products
  constexpr int kF = NB * CPR / Z, kAhead = 4;
  __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
  for (int c = 0; c < kF; ++c) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (c + kAhead < kF) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  // s[t][r] is row NQ t + 4 Z (r / 4) + 4 z + r % 4
  if (MASKED) {
#pragma unroll
    for (int t = 0; t < NB; ++t) {
      const uint32_t bits = (uint32_t)(vis >> (NQ * t)) >> (4 * z);
#pragma unroll
      for (int r = 0; r < R; ++r) {  // a clear bit: -inf
        const int b = (r >> 2) * 4 * Z + (r & 3);
        const uint32_t on = (uint32_t)((int32_t)(bits << (31 - b)) >> 31);
        s[t][r] = __uint_as_float((on & __float_as_uint(s[t][r])) | (~on & 0xFF800000u));
      }
    }
  }
  // V^T fragments: product c = D u + d takes rows [8 Z u, 8 Z u + 8 Z), in
  // two 4-row pieces of each lane, 4 Z rows apart, and head elements [NQ d,
  // NQ d + NQ). Two are read ahead of the products, the first two here.
  constexpr int U = KT / (8 * Z), D = DH / NQ;
  const int ls = lane & 15, vrow = 4 * z + (ls >> 2);
  const int vc = (NQ == 32 ? ((lane >> 4) & 1) * 2 : 0) + ((ls & 3) >> 1);
  auto fragment = [&](int c) -> at_u32x4 {
    typedef __attribute__((address_space(3))) at_s16x4 lds_s16x4;
    const int u = c / D, d = c % D;
    const int at = vrow * ROW + attn_v_chunk<DH>(vrow, NQ / 8 * d + vc) * 16 + (ls & 1) * 8;
    struct {
      at_s16x4 lo, hi;
    } f;
    f.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + (8 * Z * u) * ROW + at));
    f.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + (8 * Z * u + 4 * Z) * ROW + at));
    return __builtin_bit_cast(at_u32x4, f);
  };
  at_u32x4 f[3] = {fragment(0), fragment(1), {0, 0, 0, 0}};
  float top = s[0][0];
#pragma unroll
  for (int t = 0; t < NB; ++t)
#pragma unroll
    for (int r = 0; r < R; ++r) top = fmaxf(top, s[t][r]);
  top = attn_max_across<NQ>(top) * scale2;
  // The maximum moves only when a score passes it by more than kSlack.
  typedef AttnWeight<H> Weight;
  if (__ballot(top > st.m + Weight::kSlack) != 0) {
    const float m = top > st.m + Weight::kSlack ? top : st.m;
    const float keep = m > st.m ? __builtin_amdgcn_exp2f(st.m - m) : 1.0f;
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int r = 0; r < R; ++r) st.o[d][r] *= keep;
    st.l *= keep;
    st.m = m;
    st.mref = m > -INFINITY ? m - Weight::kBias : 0.0f;
  }
  // The weights' exponents score * scale2 - maximum are formed by an FMA, whose
  // product is not rounded, while the maximum's was: a factor that all weights
  // share, below 2^0.5 up to a maximum of 2^24. Beyond, where it (and the
  // rounding of maximum less kBias) could take them out of range, the products
  // are rounded first, as the maximum's was, and kBias comes last.
  float factor = scale2, ref = st.mref;
  if (__ballot(fabsf(st.mref) > 0x1p24f - 16.0f) != 0) {
#pragma clang fp contract(off)
    const float m = st.m > -INFINITY ? st.m : 0.0f;
#pragma unroll
    for (int t = 0; t < NB; ++t)
#pragma unroll
      for (int r = 0; r < R; ++r) s[t][r] = s[t][r] * scale2 - m;
    factor = 1.0f;
    ref = -Weight::kBias;
  }
  // Rows that a query does not see have weight 0, but 0 times a NaN or an
  // infinity among their values is no 0: such values (garbage behind the
  // block, on unmapped pages, or in other nodes' rows) are taken out of the
  // product and added by themselves for the queries that do see them.
  uint64_t dirty = 0;
  if (MASKED) {
    bool bad = false;
    if (lane < KT)
      for (int c = 0; c < CPR; ++c) {
        const at_u32x4 x = *(const at_u32x4*)(v + lane * ROW + c * 16);
        bad |= attn_not_finite<H>(x[0]) || attn_not_finite<H>(x[1]) || attn_not_finite<H>(x[2]) ||
               attn_not_finite<H>(x[3]);
      }
    dirty = __ballot(bad);
  }
  // weight i (0..7) of the rows of product group u
  auto score = [&](int u, int i) -> float {
    return NQ == 32 ? s[u >> 1][(8 * (u & 1) + i) % R] : s[NQ == 32 ? 0 : 2 * u + (i >> 2)][i & 3];
  };
  float sum[2] = {0.0f, 0.0f};
  auto weigh = [&](int u, int i) {
    const float w = __builtin_amdgcn_exp2f(fmaf(score(u, i), factor, -ref));
    if (NQ == 32)
      s[u >> 1][(8 * (u & 1) + i) % R] = w;
    else
      s[NQ == 32 ? 0 : 2 * u + (i >> 2)][i & 3] = w;
    sum[i & 1] += w;
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) weigh(0, i);
  at_u32x4 pb;
#pragma unroll
  for (int c = 0; c < U * D; ++c) {
    const int u = c / D, d = c % D;
    if (d == 0) {
      H w8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w8[i] = (H)score(u, i);
      pb = __builtin_bit_cast(at_u32x4, w8);
    }
    if (MASKED && dirty)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[c % 3][i] = attn_finite_only<H>(f[c % 3][i]);
    st.o[d] = attn_mfma<H>(f[c % 3], pb, st.o[d]);
    if (c + 2 < U * D) f[(c + 2) % 3] = fragment(c + 2);
    // between the products: the exponentials of the next group
    if (u + 1 < U)
#pragma unroll
      for (int i = 8 * d / D; i < 8 * (d + 1) / D; ++i) weigh(u + 1, i);
    __builtin_amdgcn_sched_barrier(0);
  }
  st.l += sum[0] + sum[1];
  while (MASKED && dirty) {  // uniform
    const int row = __builtin_ctzll(dirty);
    dirty &= dirty - 1;
    if (vis >> row & 1) {
#pragma unroll
      for (int j = 0; j < State::PIECES; ++j) {
        const int e = State::element(j, lane);
        const uint2 x =
            *(const uint2*)(v + row * ROW + attn_v_chunk<DH>(row, e >> 3) * 16 + (e & 7) * 2);
        // what is not finite, times any weight; 0 elsewhere
        const uint32_t two[2] = {x.x ^ attn_finite_only<H>(x.x), x.y ^ attn_finite_only<H>(x.y)};
        at_f32x4 o = st.get(j);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] += (float)__builtin_bit_cast(H, (uint16_t)(two[i >> 1] >> (16 * (i & 1))));
        st.set(j, o);
        if (j & 1) asm volatile("" ::: "memory");  // a few elements at a time
      }
    }
  }
}

// One staged tile of a cache of codes. k, v hold the codes' values; ks, vs the
// rows' scales (K's times scale * log2(e)): a score takes its key's, a weight
// its value's before it is rounded, so that the codes enter the products as
// they are. most: the largest finite scale of the tile's values (of an unmasked
// tile, for float16); scan: V may hold NaNs. The rest is attn_tile's.
constexpr float kAtLeastUnit = -60.0f;  // log2: values of smaller scales are 0 in a float16 output

template <typename H, int DH, int NQ, int KT, bool MASKED>
__device__ __forceinline__ void attn_tile_codes(const unsigned char* k, const unsigned char* v,
                                                const float* ks, const float* vs, float most,
                                                bool scan, const at_u32x4 (&q)[DH * NQ / 512],
                                                uint64_t vis, AttnState<DH, NQ>& st, int lane) {
  typedef AttnState<DH, NQ> State;
  typedef AttnWeight<H> Weight;
  constexpr bool kUnits = !__is_same(H, __bf16);
  constexpr int NB = KT / NQ, R = State::R, ROW = DH * 2, KROW = ROW + 16, CPR = DH / 8;
  constexpr int Z = kWave / NQ;  // lanes with one query
  const int z = lane / NQ;
  decltype(st.o[0] + st.o[0]) s[NB];
#pragma unroll
  for (int t = 0; t < NB; ++t) {
#pragma unroll
    for (int r = 0; r < R; ++r) s[t][r] = 0.0f;
    const int row = NQ * t + lane % NQ;
    at_u32x4 a[CPR / Z];
#pragma unroll
    for (int c = 0; c < CPR / Z; ++c)
      a[c] = *(const at_u32x4*)(k + row * KROW + (Z * c + z) * 16);
#pragma unroll
    for (int c = 0; c < CPR / Z; ++c) s[t] = attn_mfma<H>(a[c], q[c], s[t]);
  }
  // four fragments' reads ahead of the products
  constexpr int kF = NB * CPR / Z, kAhead = 4;
  __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
  for (int c = 0; c < kF; ++c) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (c + kAhead < kF) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  // s[t][r] is row NQ t + 4 Z (r / 4) + 4 z + r % 4
  // Weights for float16 are in units of 2^unit, above all scales of values that
  // the query has seen.
  if constexpr (kUnits) {
    if (MASKED) {
      uint32_t top = 0;
#pragma unroll
      for (int r = 0; r < KT; r += 4 * Z) {
        const at_u32x4 a = *(const at_u32x4*)(vs + r + 4 * z);
        const uint32_t bits = (uint32_t)(vis >> (r + 4 * z));
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // magnitudes as numbers, those seen and finite
          const uint32_t x = a[e] & (uint32_t)((int32_t)(bits << (31 - e)) >> 31) & 0x7FFFFFFFu;
          const uint32_t y = x < 0x7F800000u ? x : 0;
          top = y > top ? y : top;
        }
      }
      most = __uint_as_float(top);
      most = attn_max_across<NQ>(most);
    }
    // (the unit is a float16 step or two above the scale, so it seldom moves)
    const float need = fminf((float)(__builtin_amdgcn_frexp_expf(most) + 1), -kAtLeastUnit);
    const bool more = (most > 0.0f) & (need > st.unit + 1.0f);
    if (__ballot(more) != 0) {
      const float to = more ? need : st.unit, keep = __builtin_amdgcn_exp2f(st.unit - to);
#pragma unroll
      for (int d = 0; d < DH / NQ; ++d)
#pragma unroll
        for (int r = 0; r < R; ++r) st.o[d][r] *= keep;
      st.l *= keep;
      st.mref += st.m > -INFINITY ? to - st.unit : 0.0f;
      st.unit = to;
    }
  }
  // A weight's exponent is score * ks - mref, in one FMA. Past 2^24 the product
  // is rounded first and the maximum taken off it, mref's bias last.
  const bool big = __ballot(fabsf(st.mref) > 0x1p24f - 256.0f) != 0;
  const float from = big ? 0.0f : st.mref;
#pragma unroll
  for (int t = 0; t < NB; ++t) {
    const uint32_t bits = (uint32_t)(vis >> (NQ * t)) >> (4 * z);
#pragma unroll
    for (int r = 0; r < R; r += 4) {
      const at_f32x4 a = *(const at_f32x4*)(ks + NQ * t + Z * r + 4 * z);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = fmaf(s[t][r + e], a[e], -from);
        if (MASKED) {  // a clear bit: -inf
          const uint32_t on = (uint32_t)((int32_t)(bits << (31 - (Z * r + e))) >> 31);
          x = __uint_as_float((on & __float_as_uint(x)) | (~on & 0xFF800000u));
        }
        s[t][r + e] = x;
      }
    }
  }
  // V^T fragments: product c = D u + d takes rows [8 Z u, 8 Z u + 8 Z), in
  // two 4-row pieces of each lane, 4 Z rows apart, and head elements [NQ d,
  // NQ d + NQ). Two are read ahead of the products, the first two here.
  constexpr int U = KT / (8 * Z), D = DH / NQ;
  const int ls = lane & 15, vrow = 4 * z + (ls >> 2);
  const int vc = (NQ == 32 ? ((lane >> 4) & 1) * 2 : 0) + ((ls & 3) >> 1);
  auto fragment = [&](int c) -> at_u32x4 {
    typedef __attribute__((address_space(3))) at_s16x4 lds_s16x4;
    const int u = c / D, d = c % D;
    const int at = vrow * ROW + attn_v_chunk<DH>(vrow, NQ / 8 * d + vc) * 16 + (ls & 1) * 8;
    struct {
      at_s16x4 lo, hi;
    } f;
    f.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + (8 * Z * u) * ROW + at));
    f.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + (8 * Z * u + 4 * Z) * ROW + at));
    return __builtin_bit_cast(at_u32x4, f);
  };
  at_u32x4 f[3] = {fragment(0), fragment(1), {0, 0, 0, 0}};
  float top = s[0][0];
#pragma unroll
  for (int t = 0; t < NB; ++t)
#pragma unroll
    for (int r = 0; r < R; ++r) top = fmaxf(top, s[t][r]);
  top = attn_max_across<NQ>(top) + from;
  // The maximum moves only when a score passes it by more than kSlack.
  const bool more = top > st.m + Weight::kSlack;
  if (big || __ballot(more) != 0) {
    const float m = more ? top : st.m, keep = more ? __builtin_amdgcn_exp2f(st.m - m) : 1.0f;
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int r = 0; r < R; ++r) st.o[d][r] *= keep;
    st.l *= keep;
    st.m = m;
    const float bias = Weight::kBias - st.unit, ref = m > -INFINITY ? m : 0.0f;
    st.mref = m > -INFINITY ? m - bias : 0.0f;
#pragma unroll
    for (int t = 0; t < NB; ++t)
#pragma unroll
      for (int r = 0; r < R; ++r) s[t][r] = (s[t][r] + (from - ref)) + bias;
  }
  // Rows that a query does not see have weight 0, but 0 times a NaN or an
  // infinity among their values is no 0: such values (garbage behind the
  // block, on unmapped pages, or in other nodes' rows) are taken out of the
  // product and added by themselves for the queries that do see them.
  uint64_t dirty = 0;
  if (MASKED && scan) {  // uniform
    bool bad = false;
    const unsigned char* const mine = v + (lane & (KT - 1)) * ROW;
    for (int c = 0; c < CPR; ++c) {
      const at_u32x4 x = *(const at_u32x4*)(mine + c * 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) bad |= attn_not_finite<H>(x[e]);
    }
    bad &= lane < KT;
    dirty = __ballot(bad);
  }
  // weight i (0..7) of the rows of product group u
  auto score = [&](int u, int i) -> float {
    return NQ == 32 ? s[u >> 1][(8 * (u & 1) + i) % R] : s[NQ == 32 ? 0 : 2 * u + (i >> 2)][i & 3];
  };
  float sum[2] = {0.0f, 0.0f};
  auto weigh = [&](int u, int i) {
    const float w = __builtin_amdgcn_exp2f(score(u, i));
    if (NQ == 32)
      s[u >> 1][(8 * (u & 1) + i) % R] = w;
    else
      s[NQ == 32 ? 0 : 2 * u + (i >> 2)][i & 3] = w;
    sum[i & 1] += w;
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) weigh(0, i);
  at_u32x4 pb;
#pragma unroll
  for (int c = 0; c < U * D; ++c) {
    const int u = c / D, d = c % D;
    if (d == 0) {
      H w8[8];
      const uint32_t bits = (uint32_t)(vis >> (8 * Z * u + 4 * z));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const at_f32x4 a = *(const at_f32x4*)(vs + 8 * Z * u + 4 * Z * h + 4 * z);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float w = score(u, 4 * h + e) * a[e];
          if (MASKED)  // 0 where the scale of a row that is not seen may be NaN
            w = __uint_as_float(__float_as_uint(w) &
                                (uint32_t)((int32_t)(bits << (31 - (4 * Z * h + e))) >> 31));
          w8[4 * h + e] = (H)w;
        }
      }
      pb = __builtin_bit_cast(at_u32x4, w8);
    }
    if (MASKED && dirty)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[c % 3][i] = attn_finite_only<H>(f[c % 3][i]);
    st.o[d] = attn_mfma<H>(f[c % 3], pb, st.o[d]);
    if (c + 2 < U * D) f[(c + 2) % 3] = fragment(c + 2);
    // between the products: the exponentials of the next group
    if (u + 1 < U)
#pragma unroll
      for (int i = 8 * d / D; i < 8 * (d + 1) / D; ++i) weigh(u + 1, i);
    __builtin_amdgcn_sched_barrier(0);
  }
  st.l += sum[0] + sum[1];
  while (MASKED && dirty) {  // uniform
    const int row = __builtin_ctzll(dirty);
    dirty &= dirty - 1;
    const bool seen = vis >> row & 1;
#pragma unroll
    for (int j = 0; j < State::PIECES; ++j) {
      const int e = State::element(j, lane);
      const uint2 x =
          *(const uint2*)(v + row * ROW + attn_v_chunk<DH>(row, e >> 3) * 16 + (e & 7) * 2);
      // what is not finite, times any weight; 0 elsewhere
      const uint32_t two[2] = {x.x ^ attn_finite_only<H>(x.x), x.y ^ attn_finite_only<H>(x.y)};
      at_f32x4 o = st.get(j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = (float)__builtin_bit_cast(H, (uint16_t)(two[i >> 1] >> (16 * (i & 1))));
        o[i] += seen ? y : 0.0f;
      }
      st.set(j, o);
      if (j & 1) asm volatile("" ::: "memory");  // a few elements at a time
    }
  }
}

// Takes another state of the same queries into this one.
template <int DH, int NQ>
__device__ __forceinline__ void attn_join(AttnState<DH, NQ>& st, float m, float l,
                                          const at_f32x4* o, int stride) {
  const float top = fmaxf(st.m, m);
  const float a = st.m > -INFINITY ? __builtin_amdgcn_exp2f(st.m - top) : 0.0f;
  const float b = m > -INFINITY ? __builtin_amdgcn_exp2f(m - top) : 0.0f;
  st.m = top;
  st.l = st.l * a + l * b;
#pragma unroll
  for (int j = 0; j < AttnState<DH, NQ>::PIECES; ++j) st.set(j, st.get(j) * a + o[j * stride] * b);
}

// The thread's number, not known to the compiler as one value: what is derived
// from it for a piece's start or end is formed there, and not kept in
// registers over the steps.
__device__ __forceinline__ int attn_tid() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// A lane's query: a wave of unit u's query tile holds NQ consecutive query
// rows of the unit's key/value head, query head by query head for each block row.
struct AttnQuery {
  int i, hq;  // block row and query head
  bool live;  // it takes part
};

// A request's waves are dealt evenly to its query tiles: this is the first of
// tile `tile`, floor(tile * waves / tiles). That product leaves 32 bits from
// 1.5 M query rows on, which a batch's shared rows may have; the waves that the
// tiles are short of, fewer than QW for all of them together (QW for a request
// without rows), give the same number.
template <int QW>
__host__ __device__ __forceinline__ int attn_first_wave(const AttnReq& r, int tile) {
  const int spare = QW * r.tiles - r.waves;
  return QW * tile - (tile * spare + r.tiles - 1) / r.tiles;
}

template <int NQ, int QW>
__host__ __device__ __forceinline__ AttnQuery attn_query(const AttnParams& p, const AttnReq& r, int u,
                                                         int wq, int lane) {
  const int head = u / r.tiles, tile = u - head * r.tiles;
  const int w0 = attn_first_wave<QW>(r, tile), w1 = attn_first_wave<QW>(r, tile + 1);
  const int col = (w0 + wq) * NQ + lane % NQ;
  AttnQuery q;
  q.i = col / p.G;
  q.hq = head * p.G + (col - q.i * p.G);
  q.live = w0 + wq < w1 && q.i < r.rows;
  return q;
}

// Pieces [j0, j0 + NP) of an output row.
template <typename H, int DH, int NQ, int NP, bool EXT>
__device__ __forceinline__ void attn_store(const AttnParams& p, int64_t row, int j0, float m,
                                           float l, at_f32x4 (&o)[NP], int lane) {
  if (EXT && p.mode == kAtPrefix) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int j = 0; j < NP; ++j)
      *(at_f32x4*)(p.pre_o + row * DH + AttnState<DH, NQ>::element(j0 + j, lane)) = o[j] * inv;
    if (lane < NQ && j0 == 0) *(float2*)(p.pre_ml + row * 2) = float2{m, l};
    return;
  }
  if (EXT && p.mode == kAtRest && p.shared > 0) {
    const float2 ml = *(const float2*)(p.pre_ml + row * 2);
    const float top = fmaxf(m, ml.x);
    const float a = (ml.x > -INFINITY ? __builtin_amdgcn_exp2f(ml.x - top) : 0.0f) * ml.y;
    const float b = m > -INFINITY ? __builtin_amdgcn_exp2f(m - top) : 0.0f;
    m = top;
    l = a + l * b;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const at_f32x4 x =
          *(const at_f32x4*)(p.pre_o + row * DH + AttnState<DH, NQ>::element(j0 + j, lane));
      o[j] = x * a + o[j] * b;
    }
  }
  const bool none = l == 0.0f;  // (a NaN stays one)
  const float inv = none ? 0.0f : 1.0f / l;
  H* out = (H*)p.out + row * DH;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    H x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = none ? (H)0.0f : (H)(o[j][e] * inv);
    *(uint64_t*)(out + AttnState<DH, NQ>::element(j0 + j, lane)) = __builtin_bit_cast(uint64_t, x);
  }
  if (p.lse && lane < NQ && j0 == 0)
    p.lse[row] =
        none ? -INFINITY : (m + (log2f(l) - AttnWeight<H>::kBias)) * 0.6931471805599453f;
}

// Whether cache rows [r0, r1) of request b lie on pages of the pool; every
// thread calls it.
__device__ __forceinline__ bool attn_mapped(const PagedRows& p, int b, int r0, int r1, int* s_any) {
  if (!p.table) return true;
  bool bad = false;
  for (int g = (r0 >> p.shift) + (int)threadIdx.x; g <= (r1 - 1) >> p.shift; g += kAtThreads)
    bad |= page_of(p, b, g << p.shift) < 0;
  const uint64_t any = __ballot(bad);
  if ((threadIdx.x & 63) == 0) s_any[threadIdx.x >> 6] = any != 0;
  __syncthreads();
  return !(s_any[0] | s_any[1] | s_any[2] | s_any[3]);
}

// Row of the output that is query row k of block rows [rows, T) of a key/value
// head, k < (T - rows) * G.
__host__ __device__ __forceinline__ int64_t attn_row_behind(const AttnParams& p, int64_t b, int rows,
                                                            int head, int k) {
  const int row = k / p.G;
  return (b * p.T + rows + row) * p.q_heads + head * p.G + (k - row * p.G);
}

// Clears the rows of request b that see nothing, for one key/value head. (Rows
// are counted, which stay below 2^29, and not their pieces of 16 bytes.)
template <typename H, int DH>
__device__ __forceinline__ void attn_clear(const AttnParams& p, int64_t b, int rows, int head) {
  constexpr int PIECES = DH / 8;
  const int tid = attn_tid(), n = (p.T - rows) * p.G, c = tid % PIECES;
  for (int k = tid / PIECES; k < n; k += kAtThreads / PIECES)
    *(at_u32x4*)((H*)p.out + attn_row_behind(p, b, rows, head, k) * DH + c * 8) =
        at_u32x4{0, 0, 0, 0};
  if (p.lse)
    for (int k = tid; k < n; k += kAtThreads)
      p.lse[attn_row_behind(p, b, rows, head, k)] = -INFINITY;
}

// 64 lanes' 16-byte pieces from global memory straight into 1 KiB of LDS at
// `to` (whole KiB below 64 KiB: m0 has 16 bits for it), lane by lane. The
// compiler does not know of the load: the step that reads the tile waits for it.
__device__ __forceinline__ void attn_to_lds(const char* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(to), "v"(from)
               : "memory", "m0");
}

// Steps [t0, t1) of one key/value head's pass over a 16-bit cache.
template <typename H, class C>
__device__ __forceinline__ void attn_steps(const AttnParams& p, unsigned char* lds, int* s_any,
                                           int b, const AttnReq& rq, int head, int t0, int t1,
                                           int g, int wq, int lane, int i, bool live, bool busy,
                                           const at_u32x4 (&q)[C::DH * C::NQ / 512],
                                           AttnState<C::DH, C::NQ>& st) {
  constexpr int DH = C::DH, NQ = C::NQ, QW = C::QW;
  // this thread's chunks of a tile: row ld_row + k * STEP, chunk ld_c
  constexpr int STEP = QW * kWave / C::CPR;
  const int gt = wq * kWave + lane, ld_row = gt / C::CPR, ld_c = gt % C::CPR;
  unsigned char* const tiles = lds + g * C::NBUF * 2 * C::TILE;
  typedef __attribute__((address_space(3))) unsigned char lds_byte;
  const uint32_t tiles_at = (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)((uint32_t)(uintptr_t)(lds_byte*)lds + g * C::NBUF * 2 * C::TILE + wq * kWave * 16));
  // With two buffers (in the first 64 KiB) a tile goes straight into
  // LDS, its chunks' order made by the lanes' addresses; otherwise it waits in
  // registers.
  constexpr bool DIRECT = C::NBUF == 2 && C::LDS <= 65536;
  at_u32x4 kr[DIRECT ? 1 : C::LOADS], vr[DIRECT ? 1 : C::LOADS];
  // the entries of the next tile's pages, as read: a test here would wait for
  // them, and with them for the tile in flight
  int page[C::LOADS];
  const bool paged = p.rows.table != nullptr;
  const int32_t* const table = p.rows.table + (int64_t)b * p.rows.width;
  const uint32_t page_bytes = (uint32_t)p.kv_heads * (uint32_t)p.rows.page_size * C::ROW;
  const int row_mask = paged ? p.rows.page_size - 1 : 0x7FFFFFFF;
  const int64_t base =
      ((paged ? 0 : (int64_t)b * p.kv_heads) + head) * p.rows.page_size * C::ROW;
  const char* const kh = (const char*)p.k_cache + base;
  const char* const vh = (const char*)p.v_cache + base;
  auto row_of = [&](int t, int k) {  // the cache row that chunk k is of, clamped into the request
    const int r = t * C::TR + g * C::KT + ld_row + k * STEP;
    return r < rq.len ? r : rq.len - 1;
  };
  // Pages of STEP rows or more: the STEP rows that a group's waves load at
  // once lie on one page, so its address is scalar. (The entry still comes by
  // a vector load: a scalar one would make every LDS wait a full one.)
  const bool wide = paged && p.rows.page_size >= STEP;
  const uint32_t lane_at = (uint32_t)(ld_row * C::ROW + ld_c * 16);
  int zero = 0;
  asm volatile("" : "+v"(zero));
  auto find = [&](int t) {
    if (wide) {
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) {
        const int r = t * C::TR + g * C::KT + k * STEP;
        page[k] = table[((r < rq.len ? r : rq.len - 1) >> p.rows.shift) + zero];
      }
    } else if (paged) {
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) page[k] = table[row_of(t, k) >> p.rows.shift];
    } else {
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) page[k] = 0;
    }
  };
  auto fetch = [&](int t) {
    if constexpr (DIRECT) {
      const uint32_t kt = tiles_at + (t & 1) * 2 * C::TILE;
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) {
        const int row = ld_row + k * STEP;
        const uint32_t ck = attn_k_chunk<DH>(row, ld_c) * 16, cv = attn_v_chunk<DH>(row, ld_c) * 16;
        uint64_t at;
        if (wide) {  // (rows behind the request's last are on the page too)
          uint32_t pg = (uint32_t)__builtin_amdgcn_readfirstlane(page[k]);
          pg = pg < (uint32_t)p.rows.pages ? pg : 0;
          at = (uint64_t)pg * page_bytes +
               (uint64_t)(uint32_t)((t * C::TR + g * C::KT + k * STEP) & row_mask) * C::ROW;
          attn_to_lds(kh + at + (uint32_t)(ld_row * C::ROW + ck), kt + k * STEP * C::ROW);
          attn_to_lds(vh + at + (uint32_t)(ld_row * C::ROW + cv), kt + C::TILE + k * STEP * C::ROW);
        } else {  // rows on no page: some row's values, taken out by the mask
          const uint32_t pg = (uint32_t)page[k] < (uint32_t)p.rows.pages ? page[k] : 0;
          at = (uint64_t)pg * page_bytes + (uint64_t)(uint32_t)(row_of(t, k) & row_mask) * C::ROW;
          attn_to_lds(kh + at + ck, kt + k * STEP * C::ROW);
          attn_to_lds(vh + at + cv, kt + C::TILE + k * STEP * C::ROW);
        }
      }
    } else if (wide) {
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) {
        uint32_t pg = (uint32_t)__builtin_amdgcn_readfirstlane(page[k]);
        pg = pg < (uint32_t)p.rows.pages ? pg : 0;
        // (rows behind the request's last are on the page too)
        const uint64_t at =
            (uint64_t)pg * page_bytes +
            (uint64_t)(uint32_t)((t * C::TR + g * C::KT + k * STEP) & row_mask) * C::ROW;
        kr[k] = *(const at_u32x4*)(kh + at + lane_at);
        vr[k] = *(const at_u32x4*)(vh + at + lane_at);
      }
    } else {
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) {
        // rows on no page: some row's values, taken out by the mask
        const uint32_t pg = (uint32_t)page[k] < (uint32_t)p.rows.pages ? page[k] : 0;
        const uint64_t at = (uint64_t)pg * page_bytes +
                            (uint64_t)(uint32_t)(row_of(t, k) & row_mask) * C::ROW + ld_c * 16;
        kr[k] = *(const at_u32x4*)(kh + at);
        vr[k] = *(const at_u32x4*)(vh + at);
      }
    }
  };
  // steps before tm see every row they hold
  int tm = t0;
  if (DIRECT) __syncthreads();  // the piece before is done with the LDS
  if (t0 < t1) {
    find(t0);
    fetch(t0);
    if (t0 + 1 < t1) find(t0 + 1);
    const int end = t1 * C::TR < rq.len ? t1 * C::TR : rq.len;
    if (attn_mapped(p.rows, b, t0 * C::TR, end, s_any)) {
      tm = (rq.past < rq.len ? rq.past : rq.len) / C::TR;
      tm = tm < t0 ? t0 : (tm > t1 ? t1 : tm);
    }
  }
  if (!DIRECT) __syncthreads();
  auto step = [&](int t, auto is_masked) {
    constexpr bool MASKED = decltype(is_masked)::value;
    unsigned char* const kt = tiles + (C::NBUF == 2 ? (t & 1) * 2 * C::TILE : 0);
    unsigned char* const vt = kt + C::TILE;
    if constexpr (DIRECT) {  // the tile, and the next one's pages
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) asm volatile("" : "+v"(page[k]));
    }
#pragma unroll
    for (int k = 0; k < (DIRECT ? 0 : C::LOADS); ++k) {
      const int row = ld_row + k * STEP;
      *(at_u32x4*)(kt + row * C::ROW + attn_k_chunk<DH>(row, ld_c) * 16) = kr[k];
      *(at_u32x4*)(vt + row * C::ROW + attn_v_chunk<DH>(row, ld_c) * 16) = vr[k];
    }
    if (QW > 1) {
      __syncthreads();
    } else {  // the tile is the wave's own: its LDS operations take effect in order
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    if (t + 1 < t1) {
      fetch(t + 1);
      if (t + 2 < t1) find(t + 2);
    }
    const int r0 = t * C::TR + g * C::KT;
    if (busy && (!MASKED || r0 < rq.len)) {
      uint64_t vis = 0;
      if (MASKED) {
        const int r = r0 + lane;
        const bool held = lane < C::KT && r < rq.len && page_of(p.rows, b, r) >= 0;
        vis = attn_visible<C::KT>(p, b, rq.past, r0, i, live, __ballot(held));
      }
      attn_tile<H, DH, NQ, C::KT, MASKED>(kt, vt, q, p.scale2, vis, st, lane);
    }
    if (QW == 1) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  };
  int t = t0;
  for (; t < tm; ++t) step(t, AttnFalse{});
  for (; t < t1; ++t) step(t, AttnTrue{});
}

// Rows of the tile that this lane's query sees, as bits: attn_visible's, for all
// lanes alike.
__device__ __forceinline__ uint64_t attn_visible_codes(const AttnParams& p, int64_t b, int past,
                                                       int r0, int i, bool live, uint64_t held) {
  const int a = past - r0;  // rows of the tile before the block
  uint64_t v = a >= 64 ? ~0ull : (a > 0 ? (1ull << a) - 1 : 0ull);
  if (a < 64) {  // (a is uniform)
    if (p.mask) {
      const uint64_t* words = p.mask + (b * p.T + (live ? i : 0)) * p.W;
      if (a >= 0) {
        v |= words[0] << a;
      } else {
        const int k = -a >> 6, s = -a & 63;
        if (k < p.W) v |= words[k] >> s;
        if (s && k + 1 < p.W) v |= words[k + 1] << (64 - s);
      }
    } else {
      const int n = i + 1 + a;  // rows up to the query's own
      v |= n >= 64 ? ~0ull : (n > 0 ? (1ull << (n & 63)) - 1 : 0ull);
    }
  }
  return live ? v & held : 0;
}

// The same over a cache of codes. A step's codes wait in registers, two steps
// ahead of their use where those suffice, and become values of H on their way
// into LDS. Masks are bit operations and addresses are clamped: a branch of a
// step that depends on the lane holds one store of one number (the largest scale,
// the flag of NaN codes). With nearly all registers in use the compiler has moved
// values across the end of longer ones for the lanes inside them alone (zeros to
// be stored later came out as other numbers).
template <typename H, class C>
__device__ __forceinline__ void attn_steps_codes(const AttnParams& p, unsigned char* lds,
                                                 float* s_scale, float* s_most, int* s_flag,
                                                 int* s_any, int b,
                                                 const AttnReq& rq, int head, int t0, int t1, int g,
                                                 int wq, int lane, int i, bool live, bool busy,
                                                 const at_u32x4 (&q)[C::DH * C::NQ / 512],
                                                 AttnState<C::DH, C::NQ>& st) {
  constexpr int DH = C::DH, NQ = C::NQ, QW = C::QW;
  // this thread's chunks of a tile: row ld_row + k * STEP, chunk ld_c
  constexpr int STEP = QW * kWave / C::CPR;
  const int gt = wq * kWave + lane, ld_row = gt / C::CPR, ld_c = gt % C::CPR;
  unsigned char* const tiles = lds + g * C::NBUF * (C::KTILE + C::TILE);
  constexpr int DEEP = C::PREFETCH;  // tiles in flight
  constexpr bool kUnits = !__is_same(H, __bf16);
  at_u32x4 kr[DEEP][C::LOADS], vr[DEEP][C::LOADS];
  // the entries of a tile's pages, read before the loads of the tile before it:
  // waiting for them waits for nothing else
  int page[DEEP][C::LOADS];
  const bool paged = p.rows.table != nullptr;
  const int32_t* const table = p.rows.table + (int64_t)b * p.rows.width;
  const uint32_t page_rows = (uint32_t)p.kv_heads * (uint32_t)p.rows.page_size;
  const uint32_t page_bytes = page_rows * C::CROW;
  const int row_mask = paged ? p.rows.page_size - 1 : 0x7FFFFFFF;
  const int64_t first = ((paged ? 0 : (int64_t)b * p.kv_heads) + head) * p.rows.page_size;
  const char* const kh = (const char*)p.k_cache + first * C::CROW;
  const char* const vh = (const char*)p.v_cache + first * C::CROW;
  auto clamped = [&](int r) { return r < rq.len ? r : rq.len - 1; };
  // (as above) pages of STEP rows or more: a load's address is scalar
  const bool wide = paged && p.rows.page_size >= STEP;
  const uint32_t lane_at = (uint32_t)(ld_row * C::CROW + ld_c * 16);
  int zero = 0;
  asm volatile("" : "+v"(zero));
  // scales of a tile: the group's thread gt has that of K's row gt, or of V's row gt - KT
  const bool scaler = wq * kWave < 2 * C::KT;  // whole waves
  const int s_row = gt % C::KT;
  const float* const scales = (gt < C::KT ? p.k_scale : p.v_scale) + first;
  int s_page[DEEP];
  float s_value[DEEP];
  auto find = [&](int t, int d) {
    const int r0 = t * C::TR + g * C::KT;
    if (!paged) {
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) page[d][k] = 0;
      s_page[d] = 0;
      return;
    }
#pragma unroll
    for (int k = 0; k < C::LOADS; ++k)
      page[d][k] = wide ? table[(clamped(r0 + k * STEP) >> p.rows.shift) + zero]
                        : table[clamped(r0 + ld_row + k * STEP) >> p.rows.shift];
    s_page[d] = table[clamped(r0 + s_row) >> p.rows.shift];
  };
  auto fetch = [&](int t, int d) {
    const int r0 = t * C::TR + g * C::KT;
#pragma unroll
    for (int k = 0; k < C::LOADS; ++k) {
      // rows on no page: some row's values, taken out by the mask
      uint64_t at;
      if (wide) {  // (rows behind the request's last are on the page too)
        uint32_t pg = (uint32_t)__builtin_amdgcn_readfirstlane(page[d][k]);
        pg = pg < (uint32_t)p.rows.pages ? pg : 0;
        at = (uint64_t)pg * page_bytes +
             (uint64_t)(uint32_t)((r0 + k * STEP) & row_mask) * C::CROW + lane_at;
      } else {
        const uint32_t pg = (uint32_t)page[d][k] < (uint32_t)p.rows.pages ? page[d][k] : 0;
        at = (uint64_t)pg * page_bytes +
             (uint64_t)(uint32_t)(clamped(r0 + ld_row + k * STEP) & row_mask) * C::CROW + ld_c * 16;
      }
      kr[d][k] = *(const at_u32x4*)(kh + at);
      vr[d][k] = *(const at_u32x4*)(vh + at);
    }
    if (scaler) {
      const uint32_t pg = (uint32_t)s_page[d] < (uint32_t)p.rows.pages ? s_page[d] : 0;
      s_value[d] =
          scales[(uint64_t)pg * page_rows + (uint32_t)(clamped(r0 + s_row) & row_mask)];
    }
  };
  // steps before tm see every row they hold
  int tm = t0;
  const int last = t1 - 1;
  if (t0 < t1) {
    // whether all rows' pages are the pool's: the entries are read before the
    // first tile's, so that nothing waits for them alone
    const int end = t1 * C::TR < rq.len ? t1 * C::TR : rq.len;
    const int pages = ((end - 1) >> p.rows.shift) - (t0 * C::TR >> p.rows.shift) + 1;
    const int32_t* const entries = table + (t0 * C::TR >> p.rows.shift);
    const int at = (int)threadIdx.x < pages ? (int)threadIdx.x : pages - 1;
    const int entry = paged && pages > 0 ? entries[at] : 0;
    find(t0, 0);
    if (DEEP == 2) find(t0 < last ? t0 + 1 : last, DEEP - 1);
    fetch(t0, 0);
    find(t0 + DEEP < last ? t0 + DEEP : last, 0);
    if (DEEP == 2) fetch(t0 < last ? t0 + 1 : last, DEEP - 1);
    bool hole = (uint32_t)entry >= (uint32_t)p.rows.pages;
    if (paged)
      for (int e = kAtThreads; e < pages; e += kAtThreads) {  // uniform
        const int next = e + (int)threadIdx.x;
        hole |= (uint32_t)entries[next < pages ? next : pages - 1] >= (uint32_t)p.rows.pages;
      }
    const uint64_t any = __ballot(hole);
    if (lane == 0) s_any[threadIdx.x >> 6] = any != 0;
    __syncthreads();
    if (!(s_any[0] | s_any[1] | s_any[2] | s_any[3])) {
      tm = (rq.past < rq.len ? rq.past : rq.len) / C::TR;
      tm = tm < t0 ? t0 : (tm > t1 ? t1 : tm);
    }
  }
  __syncthreads();  // the piece before is done with the LDS
  // A CU's older workgroup comes before its younger one wherever both could go
  // on, and ends a fifth earlier: they take turns (long chains 118 -> 114 us,
  // chains behind shared rows 132 -> 126).
  const int turn = (int)(blockIdx.x >> 8);
  auto step = [&](int t, auto number, auto is_masked) {
    constexpr int d = decltype(number)::value;  // the step's registers
    constexpr bool masked = decltype(is_masked)::value;
    if ((t ^ turn) & 1)
      __builtin_amdgcn_s_setprio(1);
    else
      __builtin_amdgcn_s_setprio(0);
    const int buf = C::NBUF == 1 ? 0 : (DEEP == 2 ? d : (t - t0) & 1);
    unsigned char* const kt = tiles + buf * (C::KTILE + C::TILE);
    unsigned char* const vt = kt + C::KTILE;
    float* const sc = s_scale + (g * C::NBUF + buf) * 2 * C::KT;
    int* const flag = s_flag + (g * C::NBUF + buf) * QW;
    bool nan = false;
#pragma unroll
    for (int k = 0; k < C::LOADS; ++k) {
      const int row = ld_row + k * STEP;
      at_u32x4 x[2];
      attn_values<H, C::CACHE>(kr[d][k], x);
      unsigned char* const kx = kt + row * C::KROW + ld_c * 32;
      *(at_u32x4*)kx = x[0];
      *(at_u32x4*)(kx + 16) = x[1];
      attn_values<H, C::CACHE>(vr[d][k], x);
      *(at_u32x4*)(vt + row * C::ROW + attn_v_chunk<DH>(row, 2 * ld_c) * 16) = x[0];
      *(at_u32x4*)(vt + row * C::ROW + attn_v_chunk<DH>(row, 2 * ld_c + 1) * 16) = x[1];
      if (C::CACHE == kAtE4M3 && masked) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          nan |= (((vr[d][k][e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
      }
      __builtin_amdgcn_sched_barrier(0);  // one chunk's values at a time
    }
    if (scaler) sc[gt] = gt < C::KT ? s_value[d] * p.scale2 : s_value[d];
    float* const most = s_most + (g * C::NBUF + buf) * QW;
    if (kUnits && !masked) {
      const float x = fabsf(s_value[d]);
      const float top = wave_max(scaler && gt >= C::KT && x < INFINITY ? x : 0.0f);
      if (lane == 0) most[wq] = top;
    }
    if (C::CACHE == kAtE4M3 && masked) {
      const uint64_t any = __ballot(nan);
      if (lane == 0) flag[wq] = any != 0;
    }
    if (QW > 1) {
      __syncthreads();
    } else {  // the tile is the wave's own: its LDS operations take effect in order
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    // Behind the last step its tile comes again: a load that is always made
    // leaves the compiler certain what is in flight.
    if constexpr (DEEP == 2) {
      find(t + 3 < last ? t + 3 : last, 1 - d);
      fetch(t + 2 < last ? t + 2 : last, d);
    } else if (t < last) {
      fetch(t + 1, 0);
      if (t + 1 < last) find(t + 2, 0);
    }
    if (busy) {
      float top = 0.0f;
      if (kUnits && !masked)
#pragma unroll
        for (int w = 0; w < QW; ++w) top = fmaxf(top, most[w]);
#pragma unroll
      for (int h = 0; h < C::KT; h += C::SK) {
        const int r0 = t * C::TR + g * C::KT + h;
        const unsigned char* const kh = kt + h * C::KROW;
        const unsigned char* const vh = vt + h * C::ROW;
        if constexpr (!masked) {
          attn_tile_codes<H, DH, NQ, C::SK, false>(kh, vh, sc + h, sc + C::KT + h, top, false, q, 0,
                                                   st, lane);
        } else if (r0 < rq.len) {
          const int r = r0 + lane;
          bool held = (lane < C::SK) & (r < rq.len);
          if (paged)
            held &= (uint32_t)table[clamped(r) >> p.rows.shift] < (uint32_t)p.rows.pages;
          const uint64_t vis =
              attn_visible_codes(p, b, rq.past, r0, i, live, __ballot(held));
          int scan = 0;
          if (C::CACHE == kAtE4M3)
#pragma unroll
            for (int w = 0; w < QW; ++w) scan |= flag[w];
          attn_tile_codes<H, DH, NQ, C::SK, true>(kh, vh, sc + h, sc + C::KT + h, 0.0f,
                                                  __builtin_amdgcn_readfirstlane(scan) != 0, q, vis,
                                                  st, lane);
        }
      }
    }
    if (QW == 1) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  };
  int t = t0;
  while (t < tm) {
    step(t++, AttnNumber<0>{}, AttnFalse{});
    if constexpr (DEEP == 2) {
      if (t == tm) break;
      step(t++, AttnNumber<1>{}, AttnFalse{});
    }
  }
  for (; t < t1; ++t) {
    if (DEEP == 1 || !((t - t0) & 1))
      step(t, AttnNumber<0>{}, AttnTrue{});
    else if constexpr (DEEP == 2)
      step(t, AttnNumber<1>{}, AttnTrue{});
  }
}

// Steps [t0, t1) of unit u of request b, into the output or workspace slot
// `slot` (-1: the output).
template <typename H, class C, bool EXT>
__device__ __forceinline__ void attn_piece(const AttnParams& p, unsigned char* lds, float* s_scale,
                                           float* s_most, int* s_flag, int* s_any, int b, int u,
                                           const AttnReq& rq, int t0, int t1, int slot) {
  constexpr int DH = C::DH, NQ = C::NQ, QW = C::QW;
  const int tid = attn_tid(), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = wave / QW, wq = wave % QW;
  const int head = u / rq.tiles;
  const AttnQuery me = attn_query<NQ, QW>(p, rq, u, wq, lane);
  const int i = me.i;
  const bool live = me.live;
  const bool busy = __ballot(live) != 0;  // a wave without queries only carries rows
  if (EXT && p.mode == kAtRest) {  // steps behind the shared rows
    t0 += p.shared / C::TR;
    t1 += p.shared / C::TR;
  }
  if (rq.len == 0) t1 = t0;
  constexpr int NF = DH * NQ / 512;  // Q fragments of 16 bytes
  at_u32x4 q[NF];
  {
    const H* src =
        (const H*)p.q + (((int64_t)b * p.T + i) * p.q_heads + me.hq) * DH + lane / NQ * 8;
#pragma unroll
    for (int c = 0; c < NF; ++c)
      q[c] = live ? *(const at_u32x4*)(src + DH / NF * c) : at_u32x4{0, 0, 0, 0};
  }
  AttnState<DH, NQ> st;
  st.m = -INFINITY;
  st.mref = st.l = 0.0f;
  st.unit = C::CODES && !__is_same(H, __bf16) ? kAtLeastUnit : 0.0f;
#pragma unroll
  for (int j = 0; j < C::PIECES; ++j) st.set(j, at_f32x4{0.0f, 0.0f, 0.0f, 0.0f});

  if constexpr (C::CODES)
    attn_steps_codes<H, C>(p, lds, s_scale, s_most, s_flag, s_any, b, rq, head, t0, t1, g, wq, lane, i,
                           live, busy, q, st);
  else
    attn_steps<H, C>(p, lds, s_any, b, rq, head, t0, t1, g, wq, lane, i, live, busy, q, st);
  st.l = attn_sum_across<NQ>(st.l);
  if constexpr (C::CODES && !__is_same(H, __bf16)) {
    const float unit = __builtin_amdgcn_exp2f(st.unit);
    st.l *= unit;
#pragma unroll
    for (int j = 0; j < C::PIECES; ++j) st.set(j, st.get(j) * unit);
  }
  const int out_lane = attn_tid() & 63;

  // merge the groups
  if constexpr (C::NG > 1) {
    constexpr int BLOCK = C::PIECES * kWave * 16 + kWave * 8;  // bytes of a wave's state
    static_assert(C::NG / 2 * QW * BLOCK <= C::LDS, "states fit the tiles' LDS");
#pragma unroll
    for (int half = C::NG / 2; half >= 1; half /= 2) {
      __syncthreads();
      unsigned char* at = lds + ((g >= half ? g - half : g) * QW + wq) * BLOCK;
      at_f32x4* o = (at_f32x4*)at + out_lane;
      float* ml = (float*)(at + C::PIECES * kWave * 16) + 2 * out_lane;
      if (g >= half && g < 2 * half) {
#pragma unroll
        for (int j = 0; j < C::PIECES; ++j) o[j * kWave] = st.get(j);
        ml[0] = st.m;
        ml[1] = st.l;
      }
      __syncthreads();
      if (g < half) attn_join<DH, NQ>(st, ml[0], ml[1], o, kWave);
    }
    if (g > 0) return;
  }
  at_f32x4 o[C::PIECES];
#pragma unroll
  for (int j = 0; j < C::PIECES; ++j) o[j] = st.get(j);
  if (slot < 0) {
    const AttnQuery to = attn_query<NQ, QW>(p, rq, u, wq, out_lane);
    if (to.live)
      attn_store<H, DH, NQ, C::PIECES, EXT>(p, ((int64_t)b * p.T + to.i) * p.q_heads + to.hq, 0,
                                            st.m, st.l, o, out_lane);
    return;
  }
  at_f32x4* part = (at_f32x4*)p.part + ((int64_t)slot * QW + wq) * C::PIECES * kWave + out_lane;
#pragma unroll
  for (int j = 0; j < C::PIECES; ++j) part[j * kWave] = o[j];
  float* ml = p.part_ml + (((int64_t)slot * QW + wq) * kWave + out_lane) * 2;
  ml[0] = st.m;
  ml[1] = st.l;
}

// The rows that all requests taken part share, in whole steps of every tile, for
// a batch whose first shared_len rows lie on the same pages: no more than any
// request has committed, and none where that saves too little. row_bytes: of all
// heads' keys and values. from: a request whose page table maps them.
__device__ __forceinline__ int attn_shared(const AttnParams& p, AttnScratch& sh, int row_bytes,
                                           int& from) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int least = 0x7FFFFFFF, first = 0x7FFFFFFF, count = 0;
  for (int b0 = 0; b0 < p.requests; b0 += kAtThreads) {  // uniform
    const int b = b0 + tid;
    const int past = b < p.requests ? p.past_len[b] : -1;
    least = past >= 0 && past < least ? past : least;
    first = past >= 0 && b < first ? b : first;
    count += __popcll(__ballot(past >= 0));
  }
  least = -wave_max(-least);
  first = -wave_max(-first);
  if (lane == 0) {
    sh.part[wave][0] = least;
    sh.part[wave][1] = first;
    sh.longest[wave] = count;
  }
  __syncthreads();
  count = 0;
  for (int i = 0; i < kAtWaves; ++i) {
    least = sh.part[i][0] < least ? (int)sh.part[i][0] : least;
    first = sh.part[i][1] < first ? (int)sh.part[i][1] : first;
    count += sh.longest[i];
  }
  __syncthreads();  // before the plan takes sh
  from = __builtin_amdgcn_readfirstlane(first);
  int n = *p.shared_len;
  n = n < least ? n : least;
  n = n < p.rows.cap ? n : (int)p.rows.cap;
  n = n > 0 ? n / kAtShare * kAtShare : 0;
  n = (int64_t)(count - 1) * n < (kAtShareBytes + row_bytes - 1) / row_bytes ? 0 : n;
  return __builtin_amdgcn_readfirstlane(n);
}

template <typename H, int DH, int NQ, int QW, int CACHE = kAtSame, bool EXT = false>
__global__ __launch_bounds__(
    kAtThreads, (AttnTile<DH, NQ, QW, CACHE>::PER_CU)) void attn_kernel(AttnParams p) {
  using C = AttnTile<DH, NQ, QW, CACHE>;
  using Lds = AttnLds<C, EXT>;
  __shared__ Lds sh;
  static_assert(offsetof(Lds, tiles) == 0, "the tiles at LDS address 0");
  AttnPos at, to;
  const int id = (int)blockIdx.x;
  AttnPlace mark{};
  AttnCut cut;
  int k = id;
  bool some = true;
  if (EXT) {
    p.shared = 0;
    if (p.mode == kAtPrefix) {
      int from;
      p.shared = attn_shared(p, sh.plan, 2 * p.kv_heads * C::CROW, from);
      if (id == 0 && threadIdx.x == 0) *p.prefix = p.shared;
      some = p.shared > 0;
      if (some) p.rows.table += (int64_t)from * p.rows.width;
    } else if (p.mode == kAtRest) {
      p.shared = __builtin_amdgcn_readfirstlane(*p.prefix);
    }
  }
  AttnReq rq;
  bool mine = some;
  int unit = 0, units = 0;  // of the requests before at.b, of all
  if (EXT && p.few) {
    mine = some && attn_plan_few<C>(p, *(AttnFew*)sh.few, id, k, cut, at, to, rq, unit,
                                         units);
  } else if (some) {
    mine = attn_plan<C, EXT>(p, sh.plan, id, k, cut, at, to);
    if (mine) rq = attn_request<C, EXT>(p, at.b);
  }
  if (mine) {
    const bool whole = to.x < 0;
    do {  // uniform; no stretch is empty but for ends moved onto one another
      if (!whole && at.x >= to.x) break;
      if (at.u == rq.tiles * p.kv_heads) {  // on to the next request
        unit += at.u;
        ++at.b;
        at.u = 0;
        rq = attn_request<C, EXT>(p, at.b);
      }
      const int64_t left = whole ? rq.steps : to.x - at.x;
      const int t1 = at.s + left < rq.steps ? at.s + (int)left : rq.steps;
      const bool ends = t1 == rq.steps, begins = at.s == 0;
      if (begins && !ends) {
        // the first end of a stretch at or behind the unit's
        const int64_t x1 = at.x + rq.steps;
        int64_t e = attn_div((x1 - cut.slack) * cut.n, cut.total);
        e = e > k + 1 ? e : k + 1;
        while (e < cut.n) {
          const int64_t s = attn_end(cut, e) - at.x;
          if (s >= rq.steps || attn_near(cut, s, rq.steps) == rq.steps) break;
          ++e;
        }
        mark = AttnPlace{(int)(e - k), at.b, at.u, rq.rows, rq.waves, rq.tiles, k, 0};
      }
      if (EXT && p.by_unit && begins && !whole && threadIdx.x == 0)
        p.place[unit + at.u] = ends ? AttnPlace{} : mark;
      attn_piece<H, C, EXT>(p, sh.tiles, sh.scale, sh.most, sh.flag, sh.any, at.b, at.u, rq, at.s, t1,
                            begins && ends ? -1 : 2 * k + (begins ? 1 : 0));
      if (ends && (at.u + 1) % rq.tiles == 0 && rq.rows < p.T)
        attn_clear<H, DH>(p, at.b, rq.rows, at.u / rq.tiles);
      at.x += t1 - at.s;
      at.s = 0;
      ++at.u;
    } while (!whole);
  }
  if (EXT && p.by_unit) {
    // (without shared rows to attend to, or dealt out whole, no unit is cut)
    if (id == 0 && threadIdx.x == 0) p.place[p.places].pieces = mine && to.x >= 0 ? units : 0;
  } else if (threadIdx.x == 0 && k < p.groups) {
    p.place[k] = mark;
  }
}

// Merges the pieces of the unit that a workgroup's stretch began and did not
// end: a wave per stretch, query wave and kAtMerge pieces of its state, as a
// workgroup of its own (with few units cut, the pieces' bytes have to come in
// through as many CUs as there are; four pieces to a wave against two: 5.0 and
// 4.0 us for one tree, 11.3 and 8.9 for 24 units in 512 pieces, 5.0 and 5.9 for
// the 64 trees, where it finds nothing to merge).
template <typename H, int DH, int NQ, int QW>
__global__ __launch_bounds__(kWave) void attn_merge_kernel(AttnParams p) {
  using C = AttnTile<DH, NQ, QW>;
  constexpr int PP = kAtMerge, PER = C::PIECES / PP;  // waves of a state
  const int k = (int)(blockIdx.x / (QW * PER)), r = (int)(blockIdx.x % (QW * PER));
  const AttnPlace pl = p.place[k];
  if (pl.pieces == 0) return;
  const int lane = threadIdx.x, wq = r / PER, j0 = PP * (r % PER);
  AttnReq rq;
  rq.rows = pl.rows;
  rq.waves = pl.waves;
  rq.tiles = pl.tiles;
  const AttnQuery me = attn_query<NQ, QW>(p, rq, pl.u, wq, lane);
  if (!__ballot(me.live)) return;
  float m = -INFINITY, l = 0.0f;
  at_f32x4 o[PP];
#pragma unroll
  for (int j = 0; j < PP; ++j) o[j] = at_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < pl.pieces; ++s) {
    const int64_t at = (int64_t)(s == 0 ? 2 * k + 1 : 2 * (k + s)) * QW + wq;
    const float2 ml = *(const float2*)(p.part_ml + (at * kWave + lane) * 2);
    const at_f32x4* part = (const at_f32x4*)p.part + (at * C::PIECES + j0) * kWave + lane;
    const float top = fmaxf(m, ml.x);
    const float a = m > -INFINITY ? __builtin_amdgcn_exp2f(m - top) : 0.0f;
    const float b = ml.x > -INFINITY ? __builtin_amdgcn_exp2f(ml.x - top) : 0.0f;
    m = top;
    l = l * a + ml.y * b;
#pragma unroll
    for (int j = 0; j < PP; ++j) o[j] = o[j] * a + part[j * kWave] * b;
  }
  if (me.live)
    attn_store<H, DH, NQ, PP, false>(p, ((int64_t)pl.b * p.T + me.i) * p.q_heads + me.hq, j0, m, l,
                                     o, lane);
}

// The same with four waves to a state's part, each of every fourth piece, whose
// results are joined in LDS: shared rows leave few units in many pieces (16
// units of 128 queries in 512 pieces: 20.2 us with one wave, 10.6 with four).
template <typename H, int DH, int NQ, int QW, int CACHE>
__global__ __launch_bounds__(kAtThreads) void attn_merge_many_kernel(AttnParams p) {
  using C = AttnTile<DH, NQ, QW, CACHE>;
  constexpr int PP = kAtMerge, PER = C::PIECES / PP;  // workgroups of a state
  __shared__ at_f32x4 s_o[kAtWaves][PP][kWave];
  __shared__ float2 s_ml[kAtWaves][kWave];
  const int id = (int)(blockIdx.x / (QW * PER)), r = (int)(blockIdx.x % (QW * PER));
  if (p.by_unit && id >= p.place[p.places].pieces) return;
  const AttnPlace pl = p.place[id];
  if (pl.pieces == 0) return;
  const int k = pl.k;
  if (p.mode == kAtRest) p.shared = *p.prefix;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wq = r / PER, j0 = PP * (r % PER);
  AttnReq rq;
  rq.rows = pl.rows;
  rq.waves = pl.waves;
  rq.tiles = pl.tiles;
  const AttnQuery me = attn_query<NQ, QW>(p, rq, pl.u, wq, lane);
  if (!__ballot(me.live)) return;  // all waves alike
  float m = -INFINITY, l = 0.0f;
  at_f32x4 o[PP];
#pragma unroll
  for (int j = 0; j < PP; ++j) o[j] = at_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto join = [&](float2 ml, const at_f32x4* part, int step) {
    const float top = fmaxf(m, ml.x);
    const float a = m > -INFINITY ? __builtin_amdgcn_exp2f(m - top) : 0.0f;
    const float b = ml.x > -INFINITY ? __builtin_amdgcn_exp2f(ml.x - top) : 0.0f;
    m = top;
    l = l * a + ml.y * b;
#pragma unroll
    for (int j = 0; j < PP; ++j) o[j] = o[j] * a + part[j * step] * b;
  };
#pragma unroll 4
  for (int s = wave; s < pl.pieces; s += kAtWaves) {
    const int64_t at = (int64_t)(s == 0 ? 2 * k + 1 : 2 * (k + s)) * QW + wq;
    join(*(const float2*)(p.part_ml + (at * kWave + lane) * 2),
         (const at_f32x4*)p.part + (at * C::PIECES + j0) * kWave + lane, kWave);
  }
  if (pl.pieces > 1) {
    s_ml[wave][lane] = float2{m, l};
#pragma unroll
    for (int j = 0; j < PP; ++j) s_o[wave][j][lane] = o[j];
    __syncthreads();
    if (wave > 0) return;
    for (int s = 1; s < kAtWaves && s < pl.pieces; ++s) join(s_ml[s][lane], &s_o[s][0][lane], kWave);
  } else if (wave > 0) {
    return;
  }
  if (me.live)
    attn_store<H, DH, NQ, PP, true>(p, ((int64_t)pl.b * p.T + me.i) * p.q_heads + me.hq, j0, m, l,
                                    o, lane);
}

}  // namespace ddt
