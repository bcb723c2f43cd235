// Paged caches of 8-bit rows: written as they are quantised, compacted, read
// back.
//
// A row x of one head (its key rotated in float32, not rounded to 16 bits on
// the way, or its value) is held as codes and one float32 scale:
//   s = max(max |x| / M, 2^-126), r = 1 / s, code = x r to the nearest
// (ties to even), M = 448 for e4m3 codes, 127 for int8 ones; it stands for
// code * s. The division by M is a product with 1 / M rounded to float32, and
// nothing is contracted, so that the codes are a function of the inputs that
// any IEEE float32 arithmetic gives. A row that holds a NaN or an infinity has
// the scale NaN and codes 0: all of it reads as NaN.
//
// Append: one workgroup per row of the block, as in append.hpp. A key or value
// head is the work of a group of lanes, a power of two of them inside a wave,
// that find the row's largest magnitude by exchanges and then quantise what
// they hold in registers: the inputs are read once. 64 blocks of 129 rows, 32
// and 8 heads of 128: 27 us, 140 MB at 5.2 TB/s (HBM); one row: 3.1 us, two
// dependent reads (length, page) and the exchanges.
#pragma once

#include "append.hpp"

namespace ddt {

enum { kCodeE4M3, kCodeI8 };

struct Append8Params {
  AppendParams a;  // k_cache, v_cache: codes
  float* k_scale;  // [pages][kv_heads][page_size]
  float* v_scale;
};

constexpr float kTiniestScale = 0x1p-126f;

template <int CODE>
struct Code8;
template <>
struct Code8<kCodeE4M3> {
  static constexpr float kMost = 448.0f, kInverse = (float)(1.0 / 448.0);
  static __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) {
    const int two = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, two, true);
  }
  static __device__ __forceinline__ void wide(uint32_t x, float (&y)[4]) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, true);
    y[0] = lo[0];
    y[1] = lo[1];
    y[2] = hi[0];
    y[3] = hi[1];
  }
};
template <>
struct Code8<kCodeI8> {
  static constexpr float kMost = 127.0f, kInverse = (float)(1.0 / 127.0);
  static __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) {
    const auto one = [](float x) { return (uint32_t)(int)__builtin_rintf(x) & 0xFFu; };
    return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
  }
  static __device__ __forceinline__ void wide(uint32_t x, float (&y)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (float)(int8_t)(x >> (8 * e));
  }
};

// The largest magnitude of a lane's values, infinity where one is not finite.
template <int N>
__device__ __forceinline__ float k8_most(const float (&x)[N]) {
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float a = fabsf(x[i]);
    most = fmaxf(most, a < INFINITY ? a : INFINITY);  // (a NaN too)
  }
  return most;
}

// Eight codes of x.
template <int CODE>
__device__ __forceinline__ uint2 k8_codes(const float* x, float r) {
  typedef Code8<CODE> Q;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = fminf(fmaxf(x[i] * r, -Q::kMost), Q::kMost);
  return uint2{Q::four(y[0], y[1], y[2], y[3]), Q::four(y[4], y[5], y[6], y[7])};
}

// Pairs of eight: the first and the second elements, unrounded.
template <typename H, bool INTER>
__device__ __forceinline__ void k8_rotate(const H* src, const float* turn, int first, int half,
                                          float (&out)[16]) {
#pragma clang fp contract(off)
  const int at0 = INTER ? 2 * first : first, at1 = INTER ? 2 * first + 8 : first + half;
  const ApVec<H> x = ap_load(src + at0), y = ap_load(src + at1);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = turn[first + i], s = turn[half + first + i];
    const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + 8;
    const float a = (float)(ia < 8 ? x.h[ia & 7] : y.h[ia & 7]);
    const float b = (float)(ib < 8 ? x.h[ib & 7] : y.h[ib & 7]);
    const float ac = a * c, bs = b * s, bc = b * c, as = a * s;
    out[ia] = ac - bs;
    out[ib] = bc + as;
  }
}

// Smallest power of two with at least n (n <= 64).
__host__ __device__ inline int k8_lanes(int n) {
  int g = 1;
  while (g < n) g *= 2;
  return g;
}

template <typename H, bool INTER, int CODE>
__global__ __launch_bounds__(kApThreads) void append8_kernel(Append8Params pp) {
  typedef Code8<CODE> Q;
  const AppendParams& p = pp.a;
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
  const int lk = k8_lanes(items), lv = k8_lanes(vecs);  // lanes of a key's, a value's head
  // queries, then keys, then values, each from a wave's first lane on
  const int nq = p.q_heads * items, q_end = (nq + 63) & ~63;
  const int k_end = q_end + ((p.kv_heads * lk + 63) & ~63);
  const int v_end = k_end + ((p.kv_heads * lv + 63) & ~63);
  const H* q = (const H*)p.q + row * p.q_stride;
  const H* k = (const H*)p.k + row * p.k_stride;
  const H* v = (const H*)p.v + row * p.v_stride;
  H* qo = (H*)p.q_out + row * ((int64_t)p.q_heads * dh);
  // this row of head 0 on its page; heads are page_size rows apart
  const int64_t at =
      page < 0 ? 0 : (int64_t)page * p.kv_heads * p.rows.page_size + row_in_page(p.rows, (int)slot);
  const int end = page < 0 ? q_end : v_end;
  for (int t = threadIdx.x; t < end; t += kApThreads) {  // whole waves
    if (t < q_end) {
      if (t >= nq) continue;
      const int head = t / items, i = t - head * items;
      const H* src = q + (int64_t)head * dh;
      H* dst = qo + (int64_t)head * dh;
      if (i < pairs) {
        ap_rotate<H, INTER>(src, dst, turn, 8 * i, half);
      } else {
        const int e = p.rot + 8 * (i - pairs);
        ap_store(dst + e, ap_load(src + e));
      }
      continue;
    }
    const bool is_k = t < k_end;
    const int u = is_k ? t - q_end : t - k_end, lanes = is_k ? lk : lv;
    const int head = u / lanes, i = u - head * lanes;
    const bool on = head < p.kv_heads && i < (is_k ? items : vecs);
    const bool two = is_k && i < pairs;  // sixteen elements, not eight
    const H* src = (is_k ? k : v) + (int64_t)head * dh;
    // places of a lane's two vectors of eight
    const int e0 = !is_k ? 8 * i : (!two ? p.rot + 8 * (i - pairs) : (INTER ? 16 * i : 8 * i));
    const int e1 = INTER ? e0 + 8 : e0 + half;
    float x[16];
#pragma unroll
    for (int n = 0; n < 16; ++n) x[n] = 0.0f;
    if (on) {
      if (two) {
        k8_rotate<H, INTER>(src, turn, 8 * i, half, x);
      } else {
        const ApVec<H> y = ap_load(src + e0);
#pragma unroll
        for (int n = 0; n < 8; ++n) x[n] = (float)y.h[n];
      }
    }
    float most = k8_most(x);
    for (int d = 1; d < lanes; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
    const bool finite = most < INFINITY;
    const float scale = finite ? fmaxf(most * Q::kInverse, kTiniestScale) : __builtin_nanf("");
    const float r = 1.0f / scale;
    if (!on) continue;
    const int64_t to = at + (int64_t)head * p.rows.page_size;
    unsigned char* codes = (unsigned char*)(is_k ? p.k_cache : p.v_cache) + to * dh;
    uint2 c = k8_codes<CODE>(x, r);
    *(uint2*)(codes + e0) = finite ? c : uint2{0, 0};
    if (two) {
      c = k8_codes<CODE>(x + 8, r);
      *(uint2*)(codes + e1) = finite ? c : uint2{0, 0};
    }
    if (i == 0) (is_k ? pp.k_scale : pp.v_scale)[to] = scale;
  }
}

// ---- compaction -----------------------------------------------------------------
struct Kv8CompactParams {
  unsigned char* k;  // [layers][pages][heads][page_size][row_bytes]
  unsigned char* v;
  float* k_scale;  // [layers][pages][heads][page_size]
  float* v_scale;
  int64_t layers, batch;
  int32_t heads;
  int32_t row_bytes;    // a multiple of the pieces' size, <= 512
  int32_t waves, each;  // waves of a request, slices (layer and head) of a wave
  PagedRows rows;
  const int32_t* past_len;
  const int32_t* accepted;
  const int32_t* accept_len;
  int32_t L;
  int32_t* new_len;  // [batch], may be null
};

typedef unsigned int k8_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int k8_u32x2 __attribute__((ext_vector_type(2)));

constexpr int kK8Threads = 256;
constexpr int kK8Batch = 8;     // load groups held in registers per batch
constexpr int kK8MaxRows = 32;  // DDT_MAX_L

// The accepted path's rows take the places behind the root's, codes and scales
// (csrc/kv.hpp has the 16-bit caches' and why it can be done in place: node
// numbers increase along a path, and of one slice loads come before the stores
// of the same or of later rows). A wave finds its request's rows once and moves
// them for `each` slices; V is the piece that a lane moves at once. All of a
// batch's loads are in flight before its first store, scales among them (64
// requests of 15 rows in 36 layers of 8 heads of 128, 73 MB: 37.5 -> 20 us), at
// 3.6 TB/s: single rows of 128 bytes, and of 4 for the scales, at random places.
template <typename V>
__global__ __launch_bounds__(kK8Threads) void compact8_kernel(Kv8CompactParams p) {
  __shared__ int64_t s_from[kK8Threads / kWave][kK8MaxRows];
  __shared__ int64_t s_to[kK8Threads / kWave][kK8MaxRows];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * (kK8Threads / kWave) + w;
  const int64_t b = id / p.waves;
  if (b >= p.batch) return;  // whole wave
  const int part = (int)(id - b * p.waves);
  const int past = p.past_len[b];
  int n = p.accept_len[b];
  n = n < 0 ? 0 : (n > p.L ? p.L : n);
  // (a request taken out stays out)
  if (part == 0 && lane == 0 && p.new_len) p.new_len[b] = past < 0 ? past : past + n + 1;
  if (past < 0 || n == 0) return;
  // number of cache row r in a layer's head 0, -1 where no page holds it
  auto place = [&](int64_t r) -> int64_t {
    if (r >= p.rows.cap) return -1;
    const int page = page_of(p.rows, b, (int)r);
    if (page < 0) return -1;
    return (int64_t)page * p.heads * p.rows.page_size + row_in_page(p.rows, (int)r);
  };
  if (lane < n) {
    const int node = p.accepted[b * p.L + lane];
    const int64_t from = node >= 0 ? place((int64_t)past + node) : -1;
    const int64_t to = place((int64_t)past + lane + 1);
    s_from[w][lane] = to < 0 ? -1 : from;  // both or none
    s_to[w][lane] = to;
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const int64_t all = p.layers * p.heads;
  const int64_t first = (int64_t)part * p.each;
  const int slices = (int)(first + p.each < all ? p.each : all - first);
  const int64_t layer_rows = p.rows.pages * p.heads * p.rows.page_size;
  int head = (int)(first % p.heads);
  int64_t at = first / p.heads * layer_rows + (int64_t)head * p.rows.page_size;  // the slice's row 0
  // scales: lane l moves row l % 32 of K or, from lane 32 on, of V
  float* const scale = lane < 32 ? p.k_scale : p.v_scale;
  const int si = lane & 31;
  const int64_t s_src = si < n ? s_from[w][si] : -1, s_dst = s_to[w][si < n ? si : 0];
  const int lpr = p.row_bytes / (int)sizeof(V);  // lanes per row
  const int rpi = kWave / lpr;                   // rows per load instruction
  const int q = lane / lpr, ch = lane - q * lpr;
  const bool lane_on = q < rpi;  // lanes past rpi * lpr idle
  const int groups = (n + rpi - 1) / rpi, items = slices * groups;
  int g = 0;
  for (int k0 = 0; k0 < items; k0 += kK8Batch) {  // uniform
    V kr[kK8Batch], vr[kK8Batch];
    float sr[kK8Batch];
    int64_t dst[kK8Batch], place[kK8Batch];
#pragma unroll
    for (int k = 0; k < kK8Batch; ++k) {
      dst[k] = place[k] = -1;
      const int i = g * rpi + q;
      if (k0 + k < items) {
        if (g == 0 && s_src >= 0) {
          sr[k] = scale[at + s_src];
          place[k] = at + s_dst;
        }
        if (lane_on && i < n) {
          const int64_t from = s_from[w][i];
          if (from >= 0) {
            const int64_t src = (at + from) * p.row_bytes + (int)sizeof(V) * ch;
            kr[k] = *(const V*)(p.k + src);
            vr[k] = *(const V*)(p.v + src);
            dst[k] = (at + s_to[w][i]) * p.row_bytes + (int)sizeof(V) * ch;
          }
        }
      }
      if (++g == groups) {  // on to the next slice
        g = 0;
        at += p.rows.page_size;
        if (++head == p.heads) {
          head = 0;
          at += layer_rows - (int64_t)p.heads * p.rows.page_size;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kK8Batch; ++k) {
      if (place[k] >= 0) scale[place[k]] = sr[k];
      if (dst[k] >= 0) {
        *(V*)(p.k + dst[k]) = kr[k];
        *(V*)(p.v + dst[k]) = vr[k];
      }
    }
  }
}

// ---- reading back -----------------------------------------------------------------
struct Read8Params {
  const unsigned char* k;  // [pages][heads][page_size][head_dim] codes
  const unsigned char* v;
  const float* k_scale;  // [pages][heads][page_size]
  const float* v_scale;
  int32_t heads, head_dim;
  PagedRows rows;
  const int32_t* first;  // [batch]
  const int32_t* count;  // [batch], may be null: n
  int32_t n;
  int32_t per;    // output rows of a workgroup
  int64_t parts;  // workgroups of a request
  void* k_out;    // [batch][n][heads][head_dim]
  void* v_out;
};

constexpr int kR8Threads = 256;

// code * scale in float32, rounded once: a thread takes eight codes of K and of
// V. Rows that no page holds, and those from count on, are cleared. Bound by
// HBM writes: 16 requests of 8 k rows, 8 heads of 128, int8 to bf16, 744 MB in
// 146 us (5.1 TB/s); 129 rows 3.7 us.
template <typename O, int CODE>
__global__ __launch_bounds__(kR8Threads) void read8_kernel(Read8Params p) {
  const int64_t b = blockIdx.x / p.parts;
  const int part = (int)(blockIdx.x - b * p.parts);
  const int i0 = part * p.per;
  const int rows = p.n - i0 < p.per ? p.n - i0 : p.per;
  int count = p.count ? p.count[b] : p.n;
  const int64_t first = p.first[b];
  const int vecs = p.head_dim >> 3, width = p.heads * vecs;  // pieces of a head, of a row
  for (int t = threadIdx.x; t < rows * width; t += kR8Threads) {
    const int i = t / width, h = (t - i * width) / vecs, c = t - i * width - h * vecs;
    const int64_t r = first + i0 + i;
    const bool some = i0 + i < count && r >= 0 && r < p.rows.cap;
    const int page = some ? page_of(p.rows, b, (int)r) : -1;
    O ko[8], vo[8];
    if (page >= 0) {
      const int64_t at = ((int64_t)page * p.heads + h) * p.rows.page_size + row_in_page(p.rows, (int)r);
      const uint2 kc = *(const uint2*)(p.k + at * p.head_dim + 8 * c);
      const uint2 vc = *(const uint2*)(p.v + at * p.head_dim + 8 * c);
      const float ks = p.k_scale[at], vs = p.v_scale[at];
      float x[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e % 4 == 0) Code8<CODE>::wide(e ? kc.y : kc.x, x);
        ko[e] = (O)(x[e % 4] * ks);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e % 4 == 0) Code8<CODE>::wide(e ? vc.y : vc.x, x);
        vo[e] = (O)(x[e % 4] * vs);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) ko[e] = vo[e] = (O)0.0f;
    }
    const int64_t to = ((b * p.n + i0 + i) * p.heads + h) * p.head_dim + 8 * c;
    __builtin_memcpy(__builtin_assume_aligned((O*)p.k_out + to, 16), ko, sizeof ko);
    __builtin_memcpy(__builtin_assume_aligned((O*)p.v_out + to, 16), vo, sizeof vo);
  }
}

}  // namespace ddt
