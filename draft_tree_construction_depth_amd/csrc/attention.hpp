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
// products: a wave owns 32 of them and forms S^T = K Q^T (32x32x16 MFMA, K
// fragments from LDS, Q fragments in registers), so that a lane holds scores
// of one query only: maximum, sum and rescaling need no reduction across
// lanes beyond one exchange between the wave's halves, and the weights leave
// the accumulator layout as the B operand of O^T += V^T P^T as they are. The
// accumulator's row order (4-row pieces alternating between the halves) is
// the order in which V^T's columns are read; V's fragments come transposed
// out of row-major LDS (ds_read_b64_tr_b16).
//
// A workgroup is four waves: QW of them side by side over 32 QW queries, NG =
// 4 / QW groups of those over different cache rows, merged at the end. Few
// queries (plain decoding, short chains) are bound by the cache's bytes, so
// all four waves take rows (QW = 1); many (trees) by the products and the
// LDS reads that feed them, so all four share one staged tile (QW = 4).
//
// The next tile's rows are in flight (global to registers) while the present
// one is worked on. The cache's rows are split over workgroups in pieces of
// about one size for all requests, from the lengths on the device (attn_plan);
// the pieces' results go through the workspace and attn_merge_kernel.
#pragma once

#include "paged.hpp"

namespace ddt {

constexpr int kAtThreads = 256;
constexpr int kAtWaves = kAtThreads / kWave;
constexpr float kAtSlack = 8.0f;  // log2 by which a score may pass the maximum in use

typedef unsigned int at_u32x4 __attribute__((ext_vector_type(4)));
typedef short at_s16x4 __attribute__((ext_vector_type(4)));
typedef float at_f32x4 __attribute__((ext_vector_type(4)));
typedef float at_f32x16 __attribute__((ext_vector_type(16)));

template <int DH_, int QW_>
struct AttnTile {
  static constexpr int DH = DH_, QW = QW_;
  static constexpr int NG = kAtWaves / QW;                 // groups over cache rows
  static constexpr int KT = QW == 4 && DH <= 128 ? 64 : 32;  // rows of a group's tile
  static constexpr int TR = NG * KT;                       // rows of a workgroup's step
  static constexpr int ROW = DH * 2;                       // bytes of a row
  static constexpr int CPR = DH / 8;                       // 16-byte chunks of a row
  static constexpr int LOADS = KT * CPR / (QW * kWave);    // chunks per thread, K and V each
  static constexpr int NBUF = QW == 1 ? 1 : 2;             // one wave needs no second buffer
  static constexpr int TILE = KT * ROW;                    // bytes of K (or V) of a tile
  static constexpr int LDS = NG * NBUF * 2 * TILE;
  static constexpr int OQ = DH / 8;                        // 4-float pieces of O per lane
};

struct AttnPlace {
  int32_t b, slot, splits;  // a split request, its first workspace slot, its pieces
  int32_t count;            // entry 0: split requests
};

struct AttnParams {
  const void* q;  // [batch][T][q_heads][head_dim]
  const void* k_cache;
  const void* v_cache;
  int64_t batch;
  int32_t T, q_heads, kv_heads, G;
  int32_t MT;       // query tiles of a (request, key/value head)
  int32_t target;   // workgroups to split the rows over
  int32_t least;    // fewest steps of a piece
  PagedRows rows;
  const int32_t* past_len;
  const int32_t* num_nodes;  // [batch], may be null: T - 1
  const uint64_t* mask;      // [batch][T][W], may be null: a chain
  int32_t W;
  float scale2;  // scale * log2(e)
  void* out;     // [batch][T][q_heads][head_dim]
  float* lse;    // [batch][T][q_heads], may be null
  AttnPlace* place;  // split requests, in order
  float* part;       // [slot][QW] of OQ x 64 lanes x 4 floats
  float* part_ml;    // [slot][QW][64 lanes][2]: running maximum (log2) and sum
};

struct AttnWork {
  int b, u, piece, splits, slot;  // slot: of this workgroup, -1 for the only piece
  int len, past, nodes, steps;
};

__device__ __forceinline__ void attn_lengths(const AttnParams& p, int b, int& past, int& nodes,
                                             int& len) {
  past = p.past_len[b];
  nodes = p.num_nodes ? p.num_nodes[b] : p.T - 1;
  nodes = nodes < 0 ? 0 : (nodes > p.T - 1 ? p.T - 1 : nodes);
  int64_t n = past < 0 ? 0 : (int64_t)past + nodes + 1;
  len = (int)(n < p.rows.cap ? n : p.rows.cap);
}

template <int TR>
__device__ __forceinline__ int attn_steps(int len) {
  return len > TR ? (len + TR - 1) / TR : 1;  // one for an empty request: its rows are cleared
}

// Which piece of which request this workgroup takes; false: none. Every
// request's rows are cut into pieces of at most c steps, c the same for all,
// such that about p.target pieces result; logical order is request, piece,
// unit (key/value head, then query tile), and consecutive workgroups of one
// XCD (ids 8 apart) take consecutive ones, so that a piece's query tiles read
// its rows from one L2.
template <int TR>
__device__ bool attn_plan(const AttnParams& p, AttnWork& w) {
  __shared__ __align__(16) int s_sum[kAtWaves];
  __shared__ __align__(16) int s_sum2[kAtWaves];
  __shared__ int s_hit[4];
  const int tid = threadIdx.x;
  const int units = p.kv_heads * p.MT;
  const int id = (int)blockIdx.x;
  int past, nodes, len;
  if (p.batch == 1) {
    attn_lengths(p, 0, past, nodes, len);
    const int steps = attn_steps<TR>(len);
    int64_t c = ((int64_t)steps * units + p.target - 1) / p.target;
    c = c < p.least ? p.least : c;
    const int splits = (int)((steps + c - 1) / c), total = splits * units;
    const int per = (total + 7) >> 3, l = (id & 7) * per + (id >> 3);
    if ((id >> 3) >= per || l >= total) return false;
    w = AttnWork{0, l % units, l / units, splits, splits > 1 ? l : -1, len, past, nodes, steps};
    if (l == 0 && tid == 0) p.place[0] = AttnPlace{0, 0, splits, splits > 1};
    return true;
  }
  int64_t sum = 0;
  for (int64_t b0 = 0; b0 < p.batch; b0 += kAtThreads) {
    int x = 0, t;
    if (b0 + tid < p.batch) {
      attn_lengths(p, (int)(b0 + tid), past, nodes, len);
      x = attn_steps<TR>(len);
    }
    block_excl_scan_reg<kAtThreads>(x, s_sum, t);
    sum += t;
    __syncthreads();
  }
  int64_t c = (sum * units + p.target - 1) / p.target;
  c = c < p.least ? p.least : c;
  // split requests and their workspace slots are counted in one number: slots
  // are fewer than 2^20, split requests fewer than half the slots
  constexpr int kOne = 1 << 20;
  int total = 0, split = 0;
  for (int64_t b0 = 0; b0 < p.batch; b0 += kAtThreads) {
    int x = 0, t;
    if (b0 + tid < p.batch) {
      attn_lengths(p, (int)(b0 + tid), past, nodes, len);
      x = (int)((attn_steps<TR>(len) + c - 1) / c) * units;
    }
    block_excl_scan_reg<kAtThreads>(x, s_sum, t);
    total += t;
    if (blockIdx.x == 0) {
      block_excl_scan_reg<kAtThreads>(x > units ? 1 : 0, s_sum2, t);
      split += t;
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) p.place[0].count = split;
  const int per = (total + 7) >> 3, l = (id & 7) * per + (id >> 3);
  if ((id >> 3) >= per || l >= total) return false;
  int at = 0, slots = 0;
  for (int64_t b0 = 0; b0 < p.batch; b0 += kAtThreads) {
    int x = 0, t, t2;
    if (b0 + tid < p.batch) {
      attn_lengths(p, (int)(b0 + tid), past, nodes, len);
      x = (int)((attn_steps<TR>(len) + c - 1) / c) * units;
    }
    const int y = x > units ? x + kOne : 0;  // only split requests use the workspace
    const int first = at + block_excl_scan_reg<kAtThreads>(x, s_sum, t);
    const int slot = slots + block_excl_scan_reg<kAtThreads>(y, s_sum2, t2);
    if (l >= first && l < first + x) {
      s_hit[0] = (int)b0 + tid;
      s_hit[1] = first;
      s_hit[2] = slot;
      s_hit[3] = x / units;
    }
    __syncthreads();
    at += t;
    slots += t2;
    if (at > l) break;  // uniform
  }
  w.b = s_hit[0];
  w.splits = s_hit[3];
  const int r = l - s_hit[1];
  w.piece = r / units;
  w.u = r - w.piece * units;
  w.slot = w.splits > 1 ? (s_hit[2] & (kOne - 1)) + r : -1;
  attn_lengths(p, w.b, w.past, w.nodes, w.len);
  w.steps = attn_steps<TR>(w.len);
  if (r == 0 && tid == 0 && w.splits > 1) {
    AttnPlace* e = p.place + s_hit[2] / kOne;
    e->b = w.b;
    e->slot = s_hit[2] & (kOne - 1);
    e->splits = w.splits;
  }
  return true;
}

template <typename H>
__device__ __forceinline__ at_f32x16 attn_mfma(at_u32x4 a, at_u32x4 b, at_f32x16 c) {
  if constexpr (__is_same(H, __bf16)) {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a),
                                                   __builtin_bit_cast(v8, b), c, 0, 0, 0);
  } else {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a),
                                                  __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
}

// The other half's value of this lane's query, with this one's.
__device__ __forceinline__ float attn_max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float attn_sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
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

// A wave's running softmax over its 32 queries: lane l has query l % 32; the
// halves hold different rows of S^T and O^T.
template <int DH>
struct AttnState {
  float m, mref, l;  // maximum in use (log2), the same or 0 while it is -inf, sum of weights
  at_f32x16 o[DH / 32];
};

// Rows of the group's tile that this lane's query sees, as bits.
template <int KT>
__device__ __forceinline__ uint64_t attn_visible(const AttnParams& p, const AttnWork& w, int r0,
                                                 int i, bool live, uint64_t held) {
  if (!live) return 0;
  const int a = w.past - r0;  // rows of the tile before the block
  uint64_t v = a >= 64 ? ~0ull : (a > 0 ? (1ull << a) - 1 : 0ull);
  if (a < 64) {
    if (p.mask) {
      const uint64_t* words = p.mask + ((int64_t)w.b * p.T + i) * p.W;
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
template <typename H, int DH, int KT, bool MASKED>
__device__ __forceinline__ void attn_tile(const unsigned char* k, const unsigned char* v,
                                          const at_u32x4 (&q)[DH / 16], float scale2, uint64_t vis,
                                          AttnState<DH>& st) {
  constexpr int NB = KT / 32, ROW = DH * 2, CPR = DH / 8;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  at_f32x16 s[NB];
#pragma unroll
  for (int t = 0; t < NB; ++t) {
#pragma unroll
    for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
    const int row = 32 * t + (lane & 31);
#pragma unroll
    for (int c = 0; c < DH / 16; ++c) {
      const at_u32x4 a =
          *(const at_u32x4*)(k + row * ROW + attn_k_chunk<DH>(row, 2 * c + h) * 16);
      s[t] = attn_mfma<H>(a, q[c], s[t]);
    }
  }
  if (MASKED) {
#pragma unroll
    for (int t = 0; t < NB; ++t) {
      const uint32_t bits = (uint32_t)(vis >> (32 * t)) >> (4 * h);
#pragma unroll
      for (int r = 0; r < 16; ++r) {  // a clear bit: -inf
        const int k = (r >> 2) * 8 + (r & 3);
        const uint32_t on = (uint32_t)((int32_t)(bits << (31 - k)) >> 31);
        s[t][r] = __uint_as_float((on & __float_as_uint(s[t][r])) | (~on & 0xFF800000u));
      }
    }
  }
  float top = s[0][0];
#pragma unroll
  for (int t = 0; t < NB; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
  top = attn_max_halves(top) * scale2;
  // The maximum moves only when a score passes it by 2^8: weights up to 256
  // keep their relative precision in either type.
  if (__ballot(top > st.m + kAtSlack) != 0) {
    const float m = top > st.m + kAtSlack ? top : st.m;
    const float keep = m > st.m ? __builtin_amdgcn_exp2f(st.m - m) : 1.0f;
#pragma unroll
    for (int d = 0; d < DH / 32; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[d][r] *= keep;
    st.l *= keep;
    st.m = m;
    st.mref = m > -INFINITY ? m : 0.0f;
  }
  float sum = 0.0f;
#pragma unroll
  for (int t = 0; t < NB; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[t][r] = __builtin_amdgcn_exp2f(fmaf(s[t][r], scale2, -st.mref));
      sum += s[t][r];
    }
  st.l += sum;
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
  const int ls = lane & 15, vrow = 4 * h + (ls >> 2), vc = ((lane >> 4) & 1) * 2 + ((ls & 3) >> 1);
  typedef __attribute__((address_space(3))) at_s16x4 lds_s16x4;
#pragma unroll
  for (int u = 0; u < KT / 16; ++u) {
    H w8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w8[i] = (H)s[u >> 1][8 * (u & 1) + i];
    const at_u32x4 pb = __builtin_bit_cast(at_u32x4, w8);
#pragma unroll
    for (int d = 0; d < DH / 32; ++d) {
      const int at = vrow * ROW + attn_v_chunk<DH>(vrow, 4 * d + vc) * 16 + (ls & 1) * 8;
      struct {
        at_s16x4 lo, hi;
      } f;
      f.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + (16 * u) * ROW + at));
      f.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + (16 * u + 8) * ROW + at));
      at_u32x4 a = __builtin_bit_cast(at_u32x4, f);
      if (MASKED && dirty)
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = attn_finite_only<H>(a[i]);
      st.o[d] = attn_mfma<H>(a, pb, st.o[d]);
    }
  }
  while (MASKED && dirty) {  // uniform
    const int row = __builtin_ctzll(dirty);
    dirty &= dirty - 1;
    if (vis >> row & 1) {
#pragma unroll
      for (int d = 0; d < DH / 32; ++d) {
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int e = 32 * d + 2 * r + 4 * h;
          const uint2 x =
              *(const uint2*)(v + row * ROW + attn_v_chunk<DH>(row, e >> 3) * 16 + (e & 7) * 2);
          // what is not finite, times any weight; 0 elsewhere
          const uint32_t two[2] = {x.x ^ attn_finite_only<H>(x.x), x.y ^ attn_finite_only<H>(x.y)};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            st.o[d][r + k] +=
                (float)__builtin_bit_cast(H, (uint16_t)(two[k >> 1] >> (16 * (k & 1))));
        }
        asm volatile("" ::: "memory");  // a few elements at a time
      }
    }
  }
}

// Takes another state of the same queries into this one.
template <int DH>
__device__ __forceinline__ void attn_join(AttnState<DH>& st, float m, float l,
                                          const at_f32x4* o, int stride) {
  const float top = fmaxf(st.m, m);
  const float a = st.m > -INFINITY ? __builtin_amdgcn_exp2f(st.m - top) : 0.0f;
  const float b = m > -INFINITY ? __builtin_amdgcn_exp2f(m - top) : 0.0f;
  st.m = top;
  st.l = st.l * a + l * b;
#pragma unroll
  for (int d = 0; d < DH / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const at_f32x4 x = o[(d * 4 + (r >> 2)) * stride];
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[d][r + e] = st.o[d][r + e] * a + x[e] * b;
    }
}

// Query row `col` of unit u of request b: block row i and query head; false
// past the last.
__device__ __forceinline__ bool attn_query(const AttnParams& p, int u, int col, int& i, int& hq) {
  const int head = u / p.MT;
  i = col / p.G;
  hq = head * p.G + (col - i * p.G);
  return i < p.T;
}

template <typename H, int ND>
__device__ __forceinline__ void attn_store(const AttnParams& p, int64_t row, int d0, float m,
                                           float l, bool seen, const at_f32x16 (&o)[ND], int DH) {
  const int h = (threadIdx.x & 63) >> 5;
  const float inv = seen && l > 0.0f ? 1.0f / l : 0.0f;
  const bool none = !seen || l == 0.0f;
  H* out = (H*)p.out + row * DH;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      H x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = none ? (H)0.0f : (H)(o[d][r + e] * inv);
      *(uint64_t*)(out + 32 * (d0 + d) + (r >> 2) * 8 + 4 * h) = __builtin_bit_cast(uint64_t, x);
    }
  if (p.lse && h == 0 && d0 == 0)
    p.lse[row] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
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

template <typename H, int DH, int QW>
__global__ __launch_bounds__(kAtThreads, DH == 256 ? 1 : 2) void attn_kernel(AttnParams p) {
  using C = AttnTile<DH, QW>;
  __shared__ __align__(256) unsigned char lds[C::LDS];
  __shared__ int s_any[kAtWaves];
  AttnWork w;
  if (!attn_plan<C::TR>(p, w)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = wave / QW, wq = wave % QW;
  const int head = w.u / p.MT;
  // this lane's query
  const int col = ((w.u - head * p.MT) * QW + wq) * 32 + (lane & 31);
  int i, hq;
  const bool in = attn_query(p, w.u, col, i, hq);
  const bool live = in && i <= w.nodes && w.past >= 0;
  const bool busy = __ballot(live) != 0;  // waves past the last node only carry rows
  at_u32x4 q[DH / 16];
  {
    const H* src = (const H*)p.q + (((int64_t)w.b * p.T + i) * p.q_heads + hq) * DH + (lane >> 5) * 8;
#pragma unroll
    for (int c = 0; c < DH / 16; ++c)
      q[c] = live ? *(const at_u32x4*)(src + 16 * c) : at_u32x4{0, 0, 0, 0};
  }
  AttnState<DH> st;
  st.m = -INFINITY;
  st.mref = st.l = 0.0f;
#pragma unroll
  for (int d = 0; d < DH / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) st.o[d][r] = 0.0f;

  // the piece's steps [t0, t1); those before tm see every row they hold
  const int each = (w.steps + w.splits - 1) / w.splits;
  const int t0 = w.piece * each;
  const int t1 = w.len == 0 ? t0 : (t0 + each < w.steps ? t0 + each : w.steps);
  // this thread's chunks of a tile: row ld_row + k * STEP, chunk ld_c
  constexpr int STEP = QW * kWave / C::CPR;
  const int gt = wq * kWave + lane, ld_row = gt / C::CPR, ld_c = gt % C::CPR;
  unsigned char* const tiles = lds + g * C::NBUF * 2 * C::TILE;
  at_u32x4 kr[C::LOADS], vr[C::LOADS];
  int page[C::LOADS];
  const int64_t page_rows = (int64_t)p.kv_heads * p.rows.page_size;
  const H* const k0 = (const H*)p.k_cache + (int64_t)head * p.rows.page_size * DH + ld_c * 8;
  const H* const v0 = (const H*)p.v_cache + (int64_t)head * p.rows.page_size * DH + ld_c * 8;
  auto row_of = [&](int t, int k) {  // the cache row that chunk k is of, clamped into the request
    const int r = t * C::TR + g * C::KT + ld_row + k * STEP;
    return r < w.len ? r : w.len - 1;
  };
  auto find = [&](int t) {
#pragma unroll
    for (int k = 0; k < C::LOADS; ++k) page[k] = page_of(p.rows, w.b, row_of(t, k));
  };
  auto fetch = [&](int t) {
#pragma unroll
    for (int k = 0; k < C::LOADS; ++k) {
      // rows on no page: some row's values, taken out by the mask
      const int64_t pg = page[k] < 0 ? 0 : page[k];
      const int rp = page[k] < 0 ? 0 : row_in_page(p.rows, row_of(t, k));
      const int64_t at = (pg * page_rows + rp) * DH;
      kr[k] = *(const at_u32x4*)(k0 + at);
      vr[k] = *(const at_u32x4*)(v0 + at);
    }
  };
  int tm = t0;
  if (t0 < t1) {
    find(t0);
    fetch(t0);
    if (t0 + 1 < t1) find(t0 + 1);
    const int end = t1 * C::TR < w.len ? t1 * C::TR : w.len;
    if (attn_mapped(p.rows, w.b, t0 * C::TR, end, s_any)) {
      tm = w.past / C::TR;
      tm = tm < t0 ? t0 : (tm > t1 ? t1 : tm);
    }
  }
  auto step = [&](int t, auto is_masked) {
    constexpr bool MASKED = decltype(is_masked)::value;
    unsigned char* const kt = tiles + (C::NBUF == 2 ? (t & 1) * 2 * C::TILE : 0);
    unsigned char* const vt = kt + C::TILE;
#pragma unroll
    for (int k = 0; k < C::LOADS; ++k) {
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
    if (busy && (!MASKED || r0 < w.len)) {
      uint64_t vis = 0;
      if (MASKED) {
        const int r = r0 + lane;
        const bool held = lane < C::KT && r < w.len && page_of(p.rows, w.b, r) >= 0;
        vis = attn_visible<C::KT>(p, w, r0, i, live, __ballot(held));
      }
      attn_tile<H, DH, C::KT, MASKED>(kt, vt, q, p.scale2, vis, st);
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
  st.l = attn_sum_halves(st.l);

  // merge the groups
  if constexpr (C::NG > 1) {
    constexpr int BLOCK = C::OQ * kWave * 16 + kWave * 8;  // bytes of a wave's state
    static_assert(C::NG / 2 * QW * BLOCK <= C::LDS, "states fit the tiles' LDS");
#pragma unroll
    for (int half = C::NG / 2; half >= 1; half /= 2) {
      __syncthreads();
      unsigned char* at = lds + ((g >= half ? g - half : g) * QW + wq) * BLOCK;
      at_f32x4* o = (at_f32x4*)at + lane;
      float* ml = (float*)(at + C::OQ * kWave * 16) + 2 * lane;
      if (g >= half && g < 2 * half) {
#pragma unroll
        for (int d = 0; d < DH / 32; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4)
            o[(d * 4 + (r >> 2)) * kWave] =
                at_f32x4{st.o[d][r], st.o[d][r + 1], st.o[d][r + 2], st.o[d][r + 3]};
        ml[0] = st.m;
        ml[1] = st.l;
      }
      __syncthreads();
      if (g < half) attn_join<DH>(st, ml[0], ml[1], o, kWave);
    }
    if (g > 0) return;
  }
  if (w.slot < 0) {
    if (in)
      attn_store<H, DH / 32>(p, ((int64_t)w.b * p.T + i) * p.q_heads + hq, 0, st.m, st.l, live, st.o,
                             DH);
    return;
  }
  at_f32x4* o = (at_f32x4*)p.part + ((int64_t)w.slot * QW + wq) * C::OQ * kWave + lane;
#pragma unroll
  for (int d = 0; d < DH / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      o[(d * 4 + (r >> 2)) * kWave] =
          at_f32x4{st.o[d][r], st.o[d][r + 1], st.o[d][r + 2], st.o[d][r + 3]};
  float* ml = p.part_ml + (((int64_t)w.slot * QW + wq) * kWave + lane) * 2;
  ml[0] = st.m;
  ml[1] = st.l;
}

// Merges the pieces of split requests: a wave per 32 queries and 32 elements
// of the head.
template <typename H, int DH, int QW>
__global__ __launch_bounds__(DH * 2) void attn_merge_kernel(AttnParams p) {
  const int units = p.kv_heads * p.MT;
  const int id = (int)blockIdx.x;  // split request, unit, query wave
  const int wq = id % QW, k = id / QW / units, u = id / QW - k * units;
  if (k >= p.place[0].count) return;
  const AttnPlace pl = p.place[k];
  const int b = pl.b;
  int past, nodes, len;
  attn_lengths(p, b, past, nodes, len);
  const int lane = threadIdx.x & 63, d = threadIdx.x >> 6;
  const int col = ((u - u / p.MT * p.MT) * QW + wq) * 32 + (lane & 31);
  int i, hq;
  const bool in = attn_query(p, u, col, i, hq);
  const bool live = in && i <= nodes;
  constexpr int OQ = AttnTile<DH, QW>::OQ;
  AttnState<32> st;
  st.m = -INFINITY;
  st.mref = st.l = 0.0f;
#pragma unroll
  for (int r = 0; r < 16; ++r) st.o[0][r] = 0.0f;
  if (__ballot(live))
    for (int s = 0; s < pl.splits; ++s) {
      const int64_t at = ((int64_t)pl.slot + (int64_t)s * units + u) * QW + wq;
      const float* ml = p.part_ml + (at * kWave + lane) * 2;
      attn_join<32>(st, ml[0], ml[1], (const at_f32x4*)p.part + (at * OQ + d * 4) * kWave + lane,
                    kWave);
    }
  if (in)
    attn_store<H, 1>(p, ((int64_t)b * p.T + i) * p.q_heads + hq, d, st.m, st.l, live, st.o, DH);
}

}  // namespace ddt
