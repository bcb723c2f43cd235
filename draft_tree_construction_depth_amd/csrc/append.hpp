// Appending a verified block's keys and values to a paged cache, with the
// position rotation applied on the way.
//
// The rows of the root and of the tree's nodes go to cache rows past + j
// (j = 0 the root), where the attention under the ancestor mask and the
// compaction look for them, but a node's position in the text is that of its
// depth: past + depth(j), since the nodes of one depth are alternatives for
// one place. A pair (a, b) of a query or key head turns by its angle at that
// position: (a cos - b sin, b cos + a sin), formed in float32 and rounded
// once. Pairs are (i, i + rot/2) or, interleaved, (2i, 2i+1); elements from
// rot on and the values are copied.
//
// HBM-bound: q, k and v are read once and written once. One workgroup per
// row of the block, whose past length, depth, page and angles are the same
// for all its heads; a thread takes eight pairs (two 16-byte vectors and 64
// bytes of angles, which stay in L1 for the row's other heads) or one
// 16-byte vector to copy. 64 blocks of 129 rows (32 query and 8 key/value heads
// of 128, bf16): 28 us, 153 MB at 5.5 TB/s (a large copy: 4.7). One token: 2.6 us, the launch.
#pragma once

#include "paged.hpp"

namespace ddt {

constexpr int kApThreads = 256;

struct AppendParams {
  const void* q;  // [batch][T] rows of q_heads * head_dim, q_stride apart (elements); may be null
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;
  int32_t T, q_heads, kv_heads, head_dim;
  const float* rope;  // [rope_len][rot]: rot/2 cosines, then rot/2 sines
  int64_t rope_len;
  int32_t rot;        // rotated elements of a head, a multiple of 16; 0: none
  const int32_t* past_len;
  const int32_t* depths;     // [batch][T-1], may be null: row j is at depth j
  const int32_t* num_nodes;  // [batch], may be null: T - 1
  PagedRows rows;
  void* k_cache;
  void* v_cache;
  void* q_out;  // [batch][T][q_heads][head_dim]
};

typedef unsigned int ap_u32x4 __attribute__((ext_vector_type(4)));
typedef float ap_f32x4 __attribute__((ext_vector_type(4)));

template <typename H>
struct ApVec {
  H h[8];
};

template <typename H>
__device__ __forceinline__ ApVec<H> ap_load(const H* p) {
  return __builtin_bit_cast(ApVec<H>, *(const ap_u32x4*)p);
}

template <typename H>
__device__ __forceinline__ void ap_store(H* p, const ApVec<H>& x) {
  *(ap_u32x4*)p = __builtin_bit_cast(ap_u32x4, x);
}

// Eight pairs of one head: pairs first .. first + 7, from src to dst.
template <typename H, bool INTER>
__device__ __forceinline__ void ap_rotate(const H* src, H* dst, const float* turn, int first,
                                          int half) {
  const int at0 = INTER ? 2 * first : first, at1 = INTER ? 2 * first + 8 : first + half;
  ApVec<H> x = ap_load(src + at0), y = ap_load(src + at1);
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const ap_f32x4 ci = *(const ap_f32x4*)(turn + first + i);
    const ap_f32x4 si = *(const ap_f32x4*)(turn + half + first + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[i + e] = ci[e];
      s[i + e] = si[e];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    H& ha = INTER ? (i < 4 ? x.h[2 * i] : y.h[2 * i - 8]) : x.h[i];
    H& hb = INTER ? (i < 4 ? x.h[2 * i + 1] : y.h[2 * i - 7]) : y.h[i];
    const float a = (float)ha, b = (float)hb;
    ha = (H)(a * c[i] - b * s[i]);
    hb = (H)(b * c[i] + a * s[i]);
  }
  ap_store(dst + at0, x);
  ap_store(dst + at1, y);
}

template <typename H, bool INTER>
__global__ __launch_bounds__(kApThreads) void append_kernel(AppendParams p) {
  const int64_t row = blockIdx.x;
  const int64_t b = row / p.T;
  const int j = (int)(row - b * p.T);
  const int past = p.past_len[b];
  if (past < 0) return;
  if (j > 0 && p.num_nodes && j > p.num_nodes[b]) return;
  const int depth = j == 0 || !p.depths ? j : p.depths[b * (p.T - 1) + j - 1];
  const int64_t pos = (int64_t)past + depth;
  const float* turn = nullptr;
  if (p.rot > 0) {
    if (pos < 0 || pos >= p.rope_len) return;  // no angle: the row is left out
    turn = p.rope + pos * p.rot;
  }
  const int64_t slot = (int64_t)past + j;
  const int page = slot < p.rows.cap ? page_of(p.rows, b, (int)slot) : -1;
  const int dh = p.head_dim, half = p.rot >> 1;
  const int pairs = half >> 3, items = pairs + ((dh - p.rot) >> 3), vecs = dh >> 3;
  const int nq = p.q_heads * items, nk = p.kv_heads * items, nv = p.kv_heads * vecs;
  const H* q = (const H*)p.q + row * p.q_stride;
  const H* k = (const H*)p.k + row * p.k_stride;
  const H* v = (const H*)p.v + row * p.v_stride;
  H* qo = (H*)p.q_out + row * ((int64_t)p.q_heads * dh);
  // this row of head 0 on its page; heads are page_size rows apart
  const int64_t at =
      page < 0 ? 0
               : ((int64_t)page * p.kv_heads * p.rows.page_size + row_in_page(p.rows, (int)slot)) * dh;
  const int64_t head_step = (int64_t)p.rows.page_size * dh;
  H* ko = (H*)p.k_cache + at;
  H* vo = (H*)p.v_cache + at;
  const int end = page < 0 ? nq : nq + nk + nv;
  for (int t = threadIdx.x; t < end; t += kApThreads) {
    if (t < nq + nk) {
      const bool is_q = t < nq;
      const int u = is_q ? t : t - nq;
      const int head = u / items, i = u - head * items;
      const H* src = (is_q ? q : k) + (int64_t)head * dh;
      H* dst = is_q ? qo + (int64_t)head * dh : ko + head * head_step;
      if (i < pairs) {
        ap_rotate<H, INTER>(src, dst, turn, 8 * i, half);
      } else {
        const int e = p.rot + 8 * (i - pairs);
        ap_store(dst + e, ap_load(src + e));
      }
    } else {
      const int u = t - nq - nk;
      const int head = u / vecs, e = 8 * (u - head * vecs);
      ap_store(vo + head * head_step + e, ap_load(v + (int64_t)head * dh + e));
    }
  }
}

}  // namespace ddt
