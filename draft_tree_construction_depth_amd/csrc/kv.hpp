// KV-cache compaction to the accepted path.
//
// DDTree explainer, section 5 ("KV cache management"): after each round only
// the accepted path's cache is kept. The verification pass wrote the key and
// value rows of the tree's nodes at positions past + j (j = 0 the root, the
// bonus token; j = 1..B the nodes in output order). After the walk accepted
// nodes a_1..a_n, rows past + i (i = 1..n) take the rows of node a_i and the
// cache's length becomes past + n + 1; every other row is left as it was.
//
// MI355X design: the work is a scattered copy of n rows per (layer, request,
// KV head), HBM-bound. One wavefront per such slice moves its K and V rows:
// a row of R bytes (R <= 1024, a multiple of 16) is R/16 lanes of 16-byte
// loads, so a wave moves 64*16/R rows per instruction. In place is safe
// without a barrier: node numbers increase along a path (a_i >= i), so a
// destination row past + i is never the source of a later row, and a wave's
// stores of a batch are issued after that batch's loads and all earlier ones
// have returned.
#pragma once

#include "paged.hpp"

namespace ddt {

constexpr int kKvThreads = 256;
constexpr int kKvBatch = 8;  // load groups held in registers per batch

struct KvParams {
  unsigned char* k;  // [layers][batch][heads][cap][row_bytes]
  unsigned char* v;
  int64_t layers, batch, cap;
  int32_t heads;
  int32_t row_bytes;   // multiple of 16, <= 1024
  const int32_t* past_len;    // [batch]
  const int32_t* accepted;    // [batch][L] node numbers, -1 padded
  const int32_t* accept_len;  // [batch]
  int32_t L;
  int32_t* new_len;  // [batch], may be null
};

typedef unsigned int kv_u32x4 __attribute__((ext_vector_type(4)));

__global__ __launch_bounds__(kKvThreads) void kv_compact_kernel(KvParams p) {
  const int64_t slices = p.layers * p.batch * p.heads;
  const int64_t slice = (int64_t)blockIdx.x * (kKvThreads / kWave) + (threadIdx.x >> 6);
  if (slice >= slices) return;  // whole wave
  const int lane = threadIdx.x & 63;
  const int64_t b = (slice / p.heads) % p.batch;
  const int head = (int)(slice % p.heads);
  const int64_t layer = slice / (p.heads * p.batch);
  const int past = p.past_len[b];
  int n = p.accept_len[b];
  n = n < 0 ? 0 : (n > p.L ? p.L : n);
  if (layer == 0 && head == 0 && lane == 0 && p.new_len) p.new_len[b] = past + n + 1;
  const int lpr = p.row_bytes >> 4;  // lanes per row
  const int rpi = kWave / lpr;       // rows per load instruction
  const int q = lane / lpr, ch = lane - q * lpr;
  const bool lane_on = q < rpi;      // lanes past rpi * lpr idle
  const size_t slice_off = (size_t)slice * (size_t)p.cap * (size_t)p.row_bytes;
  const int32_t* acc = p.accepted + b * p.L;
  for (int i0 = 1; i0 <= n; i0 += kKvBatch * rpi) {  // uniform
    kv_u32x4 kr[kKvBatch], vr[kKvBatch];
    int64_t dst[kKvBatch];
#pragma unroll
    for (int g = 0; g < kKvBatch; ++g) {
      const int i = i0 + g * rpi + q;  // this lane's row: slot past + i
      dst[g] = -1;
      if (lane_on && i <= n) {
        const int node = acc[i - 1];
        const int64_t src = (int64_t)past + node, d = (int64_t)past + i;
        if (node >= 0 && src < p.cap && d < p.cap && past >= 0) {
          const size_t so = slice_off + (size_t)src * p.row_bytes + 16 * ch;
          kr[g] = *(const kv_u32x4*)(p.k + so);
          vr[g] = *(const kv_u32x4*)(p.v + so);
          dst[g] = d;
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kKvBatch; ++g) {
      if (dst[g] >= 0) {
        const size_t dof = slice_off + (size_t)dst[g] * p.row_bytes + 16 * ch;
        *(kv_u32x4*)(p.k + dof) = kr[g];
        *(kv_u32x4*)(p.v + dof) = vr[g];
      }
    }
  }
}

struct KvPagedParams {
  unsigned char* k;  // [layers][pages][heads][page_size][row_bytes]
  unsigned char* v;
  int64_t layers, batch;
  int32_t heads;
  int32_t row_bytes;    // multiple of 16, <= 1024
  int32_t waves, each;  // waves of a request, slices (layer and head) of a wave
  PagedRows rows;
  const int32_t* past_len;
  const int32_t* accepted;
  const int32_t* accept_len;
  int32_t L;
  int32_t* new_len;  // [batch], may be null
};

constexpr int kKvMaxRows = 32;  // DDT_MAX_L

// The same compaction through a page table. A request's rows lie at the same
// places of its pages in every layer and head, so a wave finds them once (into
// LDS) and copies them for several slices: 16-byte pieces of 64 * 16 /
// row_bytes rows per instruction, kKvBatch instructions for K and for V in
// flight, whatever slices they are of. The argument for doing it in place is
// the same as above, slice by slice: rows go in increasing order, and a
// batch's loads come before its stores. With one slice to a wave the four
// dependent lookups (lengths, nodes, pages, rows) were most of its time: 64
// requests x 36 layers x 8 heads of 256-byte rows took 47.9 us, now 27 (142 MB at
// 5.2 TB/s). One request: 5 us, the lookups.
__global__ __launch_bounds__(kKvThreads) void kv_compact_paged_kernel(KvPagedParams p) {
  __shared__ int64_t s_from[kKvThreads / kWave][kKvMaxRows];
  __shared__ int64_t s_to[kKvThreads / kWave][kKvMaxRows];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * (kKvThreads / kWave) + w;
  const int64_t b = id / p.waves;
  if (b >= p.batch) return;  // whole wave
  const int part = (int)(id - b * p.waves);
  const int past = p.past_len[b];
  int n = p.accept_len[b];
  n = n < 0 ? 0 : (n > p.L ? p.L : n);
  // (a request taken out stays out)
  if (part == 0 && lane == 0 && p.new_len) p.new_len[b] = past < 0 ? past : past + n + 1;
  if (past < 0 || n == 0) return;
  const int64_t head_bytes = (int64_t)p.rows.page_size * p.row_bytes;
  // byte offset of cache row r in a layer's head 0, -1 where no page holds it
  auto offset = [&](int64_t r) -> int64_t {
    if (r >= p.rows.cap) return -1;
    const int page = page_of(p.rows, b, (int)r);
    if (page < 0) return -1;
    return (int64_t)page * p.heads * head_bytes + (int64_t)row_in_page(p.rows, (int)r) * p.row_bytes;
  };
  if (lane < n) {
    const int node = p.accepted[b * p.L + lane];
    s_from[w][lane] = node >= 0 ? offset((int64_t)past + node) : -1;
    s_to[w][lane] = offset((int64_t)past + lane + 1);
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const int lpr = p.row_bytes >> 4;  // lanes per row
  const int rpi = kWave / lpr;       // rows per load instruction
  const int q = lane / lpr, ch = lane - q * lpr;
  const bool lane_on = q < rpi;      // lanes past rpi * lpr idle
  const int groups = (n + rpi - 1) / rpi;
  const int64_t all = p.layers * p.heads;
  const int64_t first = (int64_t)part * p.each;
  const int slices = (int)(first + p.each < all ? p.each : all - first);
  const int64_t layer_bytes = p.rows.pages * p.heads * head_bytes;
  int64_t layer = first / p.heads;
  int head = (int)(first - layer * p.heads), g = 0;
  const int items = slices * groups;
  for (int k0 = 0; k0 < items; k0 += kKvBatch) {  // uniform
    kv_u32x4 kr[kKvBatch], vr[kKvBatch];
    int64_t dst[kKvBatch];
#pragma unroll
    for (int k = 0; k < kKvBatch; ++k) {
      dst[k] = -1;
      const int i = g * rpi + q;
      if (k0 + k < items && lane_on && i < n) {
        const int64_t from = s_from[w][i], to = s_to[w][i];
        if (from >= 0 && to >= 0) {
          const int64_t at = layer * layer_bytes + head * head_bytes + 16 * ch;
          kr[k] = *(const kv_u32x4*)(p.k + at + from);
          vr[k] = *(const kv_u32x4*)(p.v + at + from);
          dst[k] = at + to;
        }
      }
      if (++g == groups) {  // on to the next slice
        g = 0;
        if (++head == p.heads) {
          head = 0;
          ++layer;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kKvBatch; ++k) {
      if (dst[k] >= 0) {
        *(kv_u32x4*)(p.k + dst[k]) = kr[k];
        *(kv_u32x4*)(p.v + dst[k]) = vr[k];
      }
    }
  }
}

}  // namespace ddt
