// Attention of a verified block over a paged key/value cache.
//
// Row i of request b's block (0 the root, then the tree's nodes) sees the
// past_len[b] committed cache rows and, of the block's own rows past + j,
// those whose bit is set in row i of the ancestor mask (without a mask:
// j <= i, a chain). out_i = sum_n a_in V_n with a_i the softmax of
// scale * q_i . K_n over the rows seen; lse_i is that softmax's log-sum-exp.
// Query heads share key/value heads in groups of q_heads / kv_heads.
//
// One wavefront per query head's row, one pass over the cache with the
// running maximum and sum of the softmax: per tile of 64 cache rows each
// lane scores one row, the tile's weights go through LDS, and each lane
// accumulates its elements of the head.
#pragma once

#include "paged.hpp"

namespace ddt {

struct AttnParams {
  const void* q;  // [batch][T][q_heads][head_dim]
  const void* k_cache;
  const void* v_cache;
  int64_t batch;
  int32_t T, q_heads, kv_heads;
  PagedRows rows;
  const int32_t* past_len;
  const int32_t* num_nodes;  // [batch], may be null: T - 1
  const uint64_t* mask;      // [batch][T][W], may be null: a chain
  int32_t W;
  float scale2;  // scale * log2(e)
  void* out;     // [batch][T][q_heads][head_dim]
  float* lse;    // [batch][T][q_heads], may be null
};

template <typename H, int DH>
__global__ __launch_bounds__(kWave) void attn_row_kernel(AttnParams p) {
  constexpr int E = DH / kWave;  // elements of the head per lane
  __shared__ float s_p[kWave];
  __shared__ int64_t s_at[kWave];
  const int64_t id = blockIdx.x;
  const int hq = (int)(id % p.q_heads);
  const int64_t row = id / p.q_heads;
  const int64_t b = row / p.T;
  const int i = (int)(row - b * p.T), lane = threadIdx.x;
  const int h = hq / (p.q_heads / p.kv_heads);
  int past = p.past_len[b];
  int nodes = p.num_nodes ? p.num_nodes[b] : p.T - 1;
  nodes = nodes < 0 ? 0 : (nodes > p.T - 1 ? p.T - 1 : nodes);
  H* out = (H*)p.out + id * DH;
  const bool off = past < 0 || i > nodes;
  int64_t len = off ? 0 : (int64_t)past + nodes + 1;
  if (len > p.rows.cap) len = p.rows.cap;
  const H* q = (const H*)p.q + id * DH;
  const uint64_t* words = p.mask ? p.mask + (b * p.T + i) * p.W : nullptr;
  float m = -INFINITY, l = 0.0f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int64_t n0 = 0; n0 < len; n0 += kWave) {
    const int64_t n = n0 + lane;
    bool seen = n < len;
    if (seen && n >= past) {
      const int j = (int)(n - past);
      seen = words ? (words[j >> 6] >> (j & 63)) & 1 : j <= i;
    }
    const int page = seen ? page_of(p.rows, b, (int)n) : -1;
    seen = page >= 0;
    int64_t at = 0;
    float x = -INFINITY;
    if (seen) {
      at = (((int64_t)page * p.kv_heads + h) * p.rows.page_size + row_in_page(p.rows, (int)n)) * DH;
      const H* k = (const H*)p.k_cache + at;
      float dot = 0.0f;
      for (int d = 0; d < DH; ++d) dot = fmaf((float)q[d], (float)k[d], dot);
      x = dot * p.scale2;
    }
    const float top = fmaxf(m, wave_max(x));
    const float w = seen && top > -INFINITY ? exp2f(x - top) : 0.0f;
    const float keep = top > -INFINITY ? exp2f(m - top) : 1.0f;
    l = l * keep + wave_sum(w);
    m = top;
    __syncthreads();
    s_p[lane] = w;
    s_at[lane] = seen ? at : -1;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= keep;
    for (int t = 0; t < kWave; ++t) {
      if (s_at[t] < 0) continue;
      const H* v = (const H*)p.v_cache + s_at[t];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(s_p[t], (float)v[lane + e * kWave], acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + e * kWave] = (H)(l > 0.0f ? acc[e] / l : 0.0f);
  if (p.lse && lane == 0)
    p.lse[id] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace ddt
