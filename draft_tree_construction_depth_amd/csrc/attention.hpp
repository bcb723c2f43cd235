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
// 128, unless said otherwise). 64 single tokens over 4 to 8 k rows: 304 to 314
// us, 1.61 GB at 5.1 to 5.3 TB/s, bound by HBM reads. 64 trees of 129 rows over
// 1 to 2 k: 272 to 294 us (f16 286 to 302), 166 GFLOP at 0.56 to 0.61 PFLOP/s;
// two waves on each SIMD (the accumulators, the queries and the scores fill
// the registers) leave the matrix units busy 26%, the vector units 35% and the
// LDS 24% of the time, and wait 38% of theirs; tiles of 32 rows with three
// workgroups to a CU spill (499 us), workgroups of eight waves take 335. 3
// chains of 17 rows over 50 to 100 k (f16, heads of 64, 40 and 8): 115 to 122 us,
// 461 MB at 3.8 to 4 TB/s. One tree of 65 rows over 1 k: 20 to 21 us, of which
// the merge is 4 and the steps are 6: a chain of waits. 32 blocks of 32 rows
// with 16 heads of 256 on 4 over 2 to 4 k: 194 us; 2 pieces of a prompt of 513
// rows over 4 to 8 k: 180 us.
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

template <int DH_, int NQ_, int QW_>
struct AttnTile {
  static constexpr int DH = DH_, NQ = NQ_, QW = QW_;
  static constexpr int NG = kAtWaves / QW;                 // groups over cache rows
  static constexpr int KT = QW == 4 && DH <= 128 ? 64 : 32;  // rows of a group's tile
  static constexpr int TR = NG * KT;                       // rows of a workgroup's step
  static constexpr int ROW = DH * 2;                       // bytes of a row
  static constexpr int CPR = DH / 8;                       // 16-byte chunks of a row
  static constexpr int LOADS = KT * CPR / (QW * kWave);    // chunks per thread, K and V each
  static constexpr int NBUF = QW == 1 ? 1 : 2;             // one wave needs no second buffer
  static constexpr int TILE = KT * ROW;                    // bytes of K (or V) of a tile
  static constexpr int LDS = NG * NBUF * 2 * TILE;
  static constexpr int PIECES = DH * NQ / (4 * kWave);     // 4-float pieces of O per lane
};

// What a workgroup's stretch leaves to merge: the unit that it begins and does
// not end (pieces 0: none), whose first piece is in slot 2 w + 1 and the others
// in 2 (w + 1), 2 (w + 2), ..., the continuations with which the next stretches
// begin.
struct AttnPlace {
  int32_t pieces, b, u;
  int32_t rows, waves, tiles;  // of AttnReq
  int32_t pad[2];
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
};

// One request's work: rows [0, rows) of its block see anything (0: the
// request is taken out); its waves of NQ query rows per key/value head are
// dealt evenly to `tiles` query tiles.
struct AttnReq {
  int past, rows, len, steps, waves, tiles;
};

template <class C>
__device__ __forceinline__ AttnReq attn_request(const AttnParams& p, int64_t b) {
  AttnReq r;
  r.past = p.past_len[b];
  int nodes = p.num_nodes ? p.num_nodes[b] : p.T - 1;
  nodes = nodes < 0 ? 0 : (nodes > p.T - 1 ? p.T - 1 : nodes);
  r.rows = r.past < 0 ? 0 : nodes + 1;
  const int64_t n = (int64_t)r.past + r.rows;
  r.len = r.past < 0 ? 0 : (int)(n < p.rows.cap ? n : p.rows.cap);
  // one step for an empty request: its rows are cleared
  r.steps = r.len > C::TR ? (r.len + C::TR - 1) / C::TR : 1;
  r.waves = (r.rows * p.G + C::NQ - 1) / C::NQ;
  r.tiles = r.waves > C::QW ? (r.waves + C::QW - 1) / C::QW : 1;
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

// A workgroup's shared memory, all of it in one object, so that the tiles lie
// at its start: loads straight into LDS go to the 64 KiB that m0's 16 bits
// reach, which the tiles may fill.
template <class C>
struct AttnLds {
  alignas(256) unsigned char tiles[C::LDS];
  int any[kAtWaves];
  AttnScratch plan;
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
template <class C>
__device__ bool attn_plan(const AttnParams& p, AttnScratch& sh, int w, int& k, AttnCut& cut,
                          AttnPos& from, AttnPos& to) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto axis = [&](int64_t b, int64_t& units, int& steps) {
    units = 0;
    steps = 0;
    if (b >= p.batch) return;
    const AttnReq r = attn_request<C>(p, b);
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
    const AttnReq r = attn_request<C>(p, b);
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

template <int NQ>
__device__ __forceinline__ AttnQuery attn_query(const AttnParams& p, const AttnReq& r, int u, int wq,
                                                int lane) {
  const int head = u / r.tiles, tile = u - head * r.tiles;
  const int w0 = tile * r.waves / r.tiles, w1 = (tile + 1) * r.waves / r.tiles;
  const int col = (w0 + wq) * NQ + lane % NQ;
  AttnQuery q;
  q.i = col / p.G;
  q.hq = head * p.G + (col - q.i * p.G);
  q.live = w0 + wq < w1 && q.i < r.rows;
  return q;
}

// Pieces [j0, j0 + NP) of an output row.
template <typename H, int DH, int NQ, int NP>
__device__ __forceinline__ void attn_store(const AttnParams& p, int64_t row, int j0, float m,
                                           float l, const at_f32x4 (&o)[NP], int lane) {
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

// Clears the rows of request b that see nothing, for one key/value head.
template <typename H, int DH>
__device__ __forceinline__ void attn_clear(const AttnParams& p, int64_t b, int rows, int head) {
  const int per = p.G * DH / 8;  // 16-byte pieces of a block row's heads
  for (int k = threadIdx.x; k < (p.T - rows) * per; k += kAtThreads) {
    const int row = k / per, c = k - row * per;
    const int64_t at = ((b * p.T + rows + row) * p.q_heads + (int64_t)head * p.G) * DH + c * 8;
    *(at_u32x4*)((H*)p.out + at) = at_u32x4{0, 0, 0, 0};
  }
  if (p.lse)
    for (int k = threadIdx.x; k < (p.T - rows) * p.G; k += kAtThreads) {
      const int row = k / p.G;
      p.lse[(b * p.T + rows + row) * p.q_heads + head * p.G + (k - row * p.G)] = -INFINITY;
    }
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

// Steps [t0, t1) of unit u of request b, into the output or workspace slot
// `slot` (-1: the output).
template <typename H, class C>
__device__ __forceinline__ void attn_piece(const AttnParams& p, unsigned char* lds, int* s_any,
                                           int b, int u, const AttnReq& rq, int t0, int t1,
                                           int slot) {
  constexpr int DH = C::DH, NQ = C::NQ, QW = C::QW;
  const int tid = attn_tid(), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = wave / QW, wq = wave % QW;
  const int head = u / rq.tiles;
  const AttnQuery me = attn_query<NQ>(p, rq, u, wq, lane);
  const int i = me.i;
  const bool live = me.live;
  const bool busy = __ballot(live) != 0;  // a wave without queries only carries rows
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
#pragma unroll
  for (int j = 0; j < C::PIECES; ++j) st.set(j, at_f32x4{0.0f, 0.0f, 0.0f, 0.0f});

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
  st.l = attn_sum_across<NQ>(st.l);
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
    const AttnQuery to = attn_query<NQ>(p, rq, u, wq, out_lane);
    if (to.live)
      attn_store<H, DH, NQ>(p, ((int64_t)b * p.T + to.i) * p.q_heads + to.hq, 0, st.m, st.l, o,
                            out_lane);
    return;
  }
  at_f32x4* part = (at_f32x4*)p.part + ((int64_t)slot * QW + wq) * C::PIECES * kWave + out_lane;
#pragma unroll
  for (int j = 0; j < C::PIECES; ++j) part[j * kWave] = o[j];
  float* ml = p.part_ml + (((int64_t)slot * QW + wq) * kWave + out_lane) * 2;
  ml[0] = st.m;
  ml[1] = st.l;
}

template <typename H, int DH, int NQ, int QW>
__global__ __launch_bounds__(kAtThreads, DH == 256 ? 1 : 2) void attn_kernel(AttnParams p) {
  using C = AttnTile<DH, NQ, QW>;
  __shared__ AttnLds<C> sh;
  static_assert(offsetof(AttnLds<C>, tiles) == 0, "the tiles at LDS address 0");
  AttnPos at, to;
  const int id = (int)blockIdx.x;
  AttnPlace mark{};
  AttnCut cut;
  int k = id;
  if (attn_plan<C>(p, sh.plan, id, k, cut, at, to)) {
    const bool whole = to.x < 0;
    AttnReq rq = attn_request<C>(p, at.b);
    do {  // uniform; no stretch is empty but for ends moved onto one another
      if (!whole && at.x >= to.x) break;
      if (at.u == rq.tiles * p.kv_heads) {  // on to the next request
        ++at.b;
        at.u = 0;
        rq = attn_request<C>(p, at.b);
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
        mark = AttnPlace{(int)(e - k), at.b, at.u, rq.rows, rq.waves, rq.tiles, {0, 0}};
      }
      attn_piece<H, C>(p, sh.tiles, sh.any, at.b, at.u, rq, at.s, t1,
                       begins && ends ? -1 : 2 * k + (begins ? 1 : 0));
      if (ends && (at.u + 1) % rq.tiles == 0 && rq.rows < p.T)
        attn_clear<H, DH>(p, at.b, rq.rows, at.u / rq.tiles);
      at.x += t1 - at.s;
      at.s = 0;
      ++at.u;
    } while (!whole);
  }
  if (threadIdx.x == 0 && k < p.groups) p.place[k] = mark;
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
  const AttnQuery me = attn_query<NQ>(p, rq, pl.u, wq, lane);
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
    attn_store<H, DH, NQ>(p, ((int64_t)pl.b * p.T + me.i) * p.q_heads + me.hq, j0, m, l, o, lane);
}

}  // namespace ddt
