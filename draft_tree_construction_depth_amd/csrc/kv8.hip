// C ABI of caches of 8-bit rows and of the attention of batches that share
// their first rows (declared in include/ddtree.h): argument checks, workspace,
// launch geometry.
#include "ddtree.h"

#include "kv8.hpp"
#include "verify.hpp"

namespace {

using ddt::align_up;
using ddt::attn_check;
using ddt::attn_plan_host;
using ddt::AttnPlan;
using ddt::launchable;
using ddt::paged_rows;
using ddt::valid_half;

bool valid_codes(int cache_dtype) { return cache_dtype == DDT_E4M3 || cache_dtype == DDT_I8; }

template <typename H, int CODE>
void launch_append8(const ddt::Append8Params& ap, int64_t blocks, int interleaved, hipStream_t st) {
  if (interleaved)
    hipLaunchKernelGGL((ddt::append8_kernel<H, true, CODE>), dim3((unsigned)blocks),
                       dim3(ddt::kApThreads), 0, st, ap);
  else
    hipLaunchKernelGGL((ddt::append8_kernel<H, false, CODE>), dim3((unsigned)blocks),
                       dim3(ddt::kApThreads), 0, st, ap);
}

template <typename O>
void launch_read8(const ddt::Read8Params& rp, int64_t blocks, int cache_dtype, hipStream_t st) {
  if (cache_dtype == DDT_E4M3)
    hipLaunchKernelGGL((ddt::read8_kernel<O, ddt::kCodeE4M3>), dim3((unsigned)blocks),
                       dim3(ddt::kR8Threads), 0, st, rp);
  else
    hipLaunchKernelGGL((ddt::read8_kernel<O, ddt::kCodeI8>), dim3((unsigned)blocks),
                       dim3(ddt::kR8Threads), 0, st, rp);
}

// Whether a batch's shared rows can be worth a pass of their own, of `cap` rows
// of `elem` bytes an element (attn_shared decides, by the lengths). Up to 80 query
// rows to a key/value head reading the rows again takes longer than the pass over
// them; with more the pass takes longer, at half the rate of a large product: 32
// requests x 8 k shared rows of 16 bits, 64 / 80 / 96 / 112 / 128 query rows,
// without 154 / 170 / 170 / 173 / 182 us, with 123 / 150 / 168 / 187 / 200.
bool shares(int64_t batch, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
            int64_t cap, int elem) {
  return batch > 1 && (int64_t)T * (q_heads / kv_heads) <= 80 &&
         (double)(batch - 1) * (double)cap * 2.0 * kv_heads * head_dim * elem >=
             (double)ddt::kAtShareBytes;
}

// The attention of a batch that shares rows: the pass over them, with all
// requests' block rows as one request's, then the requests' own. (attn_check
// leaves fewer than 2^29 query rows to a key/value head: they are counted in 31
// bits.)
struct SharePlan {
  AttnPlan shared, own;
  size_t ml, o, work, end;  // workspace; *prefix lies at its start
};

SharePlan share_plan(int64_t batch, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                     int64_t cap, bool codes) {
  SharePlan pl;
  pl.shared = attn_plan_host(1, (int32_t)(batch * T), q_heads, kv_heads, head_dim, cap, codes);
  // a stretch's start and its pieces' way to the merge are worth steps, too long
  // ones leave CUs idle. us in stretches of 4 / 8 / 16 steps at least, 8 heads of
  // 128, 16 bits: 64 single tokens behind 8 k rows 88 / 84 / 89, of e4m3 68 / 65 /
  // 74, behind 30 k 117 / 116 / 120, 8 of them behind 16 k 46 / 44 / 49; heads of
  // 64 54 / 53 / 58, 32 of 4 heads of 256 75 / 75 / 80; chains of 5 and 16 alike
  pl.shared.least = 8;
  pl.own = attn_plan_host(batch, T, q_heads, kv_heads, head_dim, cap, codes);
  const size_t rows = (size_t)batch * T * q_heads;
  pl.ml = align_up(sizeof(int32_t));
  pl.o = align_up(pl.ml + rows * 2 * sizeof(float));
  pl.work = align_up(pl.o + rows * head_dim * sizeof(float));
  pl.end = pl.work + (pl.shared.end > pl.own.end ? pl.shared.end : pl.own.end);
  return pl;
}

bool launchable(const AttnPlan& pl) { return launchable(pl.grid, ddt::kAtThreads); }

// elem: bytes of an element of the cache, one if it holds codes
size_t attention_workspace(int64_t batch, int32_t T, int32_t q_heads, int32_t kv_heads,
                           int32_t head_dim, int64_t pages_per_request, int32_t page_size,
                           int elem, bool shared) {
  if (batch <= 0 || pages_per_request <= 0 || page_size <= 0 ||
      attn_check(DDT_BF16, batch, T, q_heads, kv_heads, head_dim) != DDT_OK)
    return 0;
  const int64_t cap = pages_per_request > 0x7FFFFFFFLL / page_size
                          ? 0x7FFFFFFFLL
                          : pages_per_request * page_size;
  if (shared && shares(batch, T, q_heads, kv_heads, head_dim, cap, elem)) {
    const SharePlan pl = share_plan(batch, T, q_heads, kv_heads, head_dim, cap, elem == 1);
    return launchable(pl.shared) && launchable(pl.own) ? pl.end : 0;
  }
  const AttnPlan pl = attn_plan_host(batch, T, q_heads, kv_heads, head_dim, cap, elem == 1);
  return launchable(pl) ? pl.end : 0;
}

void set_work(ddt::AttnParams& ap, const AttnPlan& pl, char* at) {
  ap.groups = (int32_t)pl.groups;
  ap.least = (int32_t)pl.least;
  ap.place = (ddt::AttnPlace*)at;
  ap.part = (float*)(at + pl.part);
  ap.part_ml = (float*)(at + pl.ml);
  // every tile has 32 rows or more to a step
  const int64_t most = ap.rows.cap / 32 + 1, M = (int64_t)ap.T * ap.G / 16 + 1;
  ap.few = ap.batch <= ddt::kAtThreads && ap.batch * ap.kv_heads <= 0x7FFFFFFFLL / M / most;
  ap.by_unit = ap.few && pl.units <= pl.groups;
  ap.places = (int32_t)(ap.by_unit ? pl.units : pl.groups);
}

typedef int (*AttnLaunch)(const ddt::AttnParams&, const AttnPlan&, int, int, hipStream_t);

// Attention over a cache of row_elem bytes an element (one: codes); shared_len
// null: no shared rows.
int attention(const void* q, int dtype, int64_t batch, int32_t T, int32_t q_heads,
              int32_t kv_heads, int32_t head_dim, int row_elem, AttnLaunch launch,
              const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
              const int32_t* page_table, int64_t table_width, int64_t pages, int32_t page_size,
              const int32_t* past_len, const int32_t* num_nodes, const uint64_t* mask,
              const int32_t* shared_len, float scale, void* out, float* lse, void* workspace,
              size_t workspace_bytes, hipStream_t stream) {
  const int chk = attn_check(dtype, batch, T, q_heads, kv_heads, head_dim);
  if (chk == DDT_EINVAL) return chk;
  if (batch == 0) return DDT_OK;
  if (!q || !k_cache || !v_cache || !past_len || !out || !workspace) return DDT_EINVAL;
  if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out |
       (uintptr_t)workspace) & 15)
    return DDT_EINVAL;
  if (!(scale > 0.0f && scale * ddt::kLog2e < INFINITY)) return DDT_EINVAL;
  if (shared_len && !page_table) return DDT_EINVAL;
  ddt::AttnParams ap{};
  const int chk2 = paged_rows(page_table, table_width, batch, pages, page_size, ap.rows);
  if (chk2 == DDT_EINVAL) return chk2;
  if (chk != DDT_OK || chk2 != DDT_OK) return DDT_ENOTSUP;
  if (ap.rows.cap > (1 << 27) ||  // the plan counts steps in 32 bits
      (page_table && (int64_t)kv_heads * page_size > (((int64_t)1 << 32) - 1) / (row_elem * head_dim)))
    return DDT_ENOTSUP;  // ... and a page's bytes are addressed in 32
  ap.q = q;
  ap.k_cache = k_cache;
  ap.v_cache = v_cache;
  ap.k_scale = k_scale;
  ap.v_scale = v_scale;
  ap.batch = batch;
  ap.T = T;
  ap.q_heads = q_heads;
  ap.kv_heads = kv_heads;
  ap.G = q_heads / kv_heads;
  ap.past_len = past_len;
  ap.num_nodes = num_nodes;
  ap.mask = mask;
  ap.W = (T + 63) / 64;
  ap.scale2 = scale * ddt::kLog2e;
  ap.out = out;
  ap.lse = lse;
  ap.mode = ddt::kAtAlone;
  if (!shared_len || !shares(batch, T, q_heads, kv_heads, head_dim, ap.rows.cap, row_elem)) {
    const AttnPlan pl =
        attn_plan_host(batch, T, q_heads, kv_heads, head_dim, ap.rows.cap, row_elem == 1);
    if (!launchable(pl)) return DDT_ENOTSUP;
    if (workspace_bytes < pl.end) return DDT_EWORKSPACE;
    set_work(ap, pl, (char*)workspace);
    return launch(ap, pl, dtype, head_dim, stream);
  }
  const SharePlan pl =
      share_plan(batch, T, q_heads, kv_heads, head_dim, ap.rows.cap, row_elem == 1);
  if (!launchable(pl.shared) || !launchable(pl.own)) return DDT_ENOTSUP;
  if (workspace_bytes < pl.end) return DDT_EWORKSPACE;
  char* const ws = (char*)workspace;
  ap.shared_len = shared_len;
  ap.prefix = (int32_t*)ws;
  ap.pre_ml = (float*)(ws + pl.ml);
  ap.pre_o = (float*)(ws + pl.o);
  ddt::AttnParams pre = ap;
  pre.mode = ddt::kAtPrefix;
  pre.requests = (int32_t)batch;
  pre.batch = 1;
  pre.T = (int32_t)(batch * T);
  pre.num_nodes = nullptr;
  pre.mask = nullptr;
  set_work(pre, pl.shared, ws + pl.work);
  const int rc = launch(pre, pl.shared, dtype, head_dim, stream);
  if (rc != DDT_OK) return rc;
  ap.mode = ddt::kAtRest;
  set_work(ap, pl.own, ws + pl.work);
  return launch(ap, pl.own, dtype, head_dim, stream);
}

}  // namespace

extern "C" {

int ddtree_append_kv8(const void* q, const void* k, const void* v, int dtype, int64_t batch,
                      int32_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                      int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* rope,
                      int64_t rope_len, int32_t rope_dim, int32_t interleaved,
                      const int32_t* past_len, const int32_t* depths, const int32_t* num_nodes,
                      const int32_t* page_table, int64_t table_width, int64_t pages,
                      int32_t page_size, int cache_dtype, void* k_cache, void* v_cache,
                      float* k_scale, float* v_scale, void* q_out, hipStream_t stream) {
  if (!valid_half(dtype) || !valid_codes(cache_dtype) || batch < 0 || T <= 0 || q_heads < 0 ||
      kv_heads <= 0 || head_dim <= 0 || rope_dim < 0 || rope_dim > head_dim || rope_len < 0 ||
      (interleaved != 0 && interleaved != 1))
    return DDT_EINVAL;
  if (q_heads > 0 && q_heads % kv_heads != 0) return DDT_EINVAL;
  if (batch == 0) return DDT_OK;
  if (!k || !v || !past_len || !k_cache || !v_cache || !k_scale || !v_scale ||
      (rope_dim > 0 && !rope))
    return DDT_EINVAL;
  if (q_heads > 0 && (!q || !q_out)) return DDT_EINVAL;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)rope | (uintptr_t)k_cache |
       (uintptr_t)v_cache | (uintptr_t)q_out) & 15 ||
      ((uintptr_t)k_scale | (uintptr_t)v_scale) & 3)
    return DDT_EINVAL;
  if ((q_heads > 0 && q_stride < (int64_t)q_heads * head_dim) ||
      k_stride < (int64_t)kv_heads * head_dim || v_stride < (int64_t)kv_heads * head_dim)
    return DDT_EINVAL;
  ddt::Append8Params pp;
  ddt::AppendParams& ap = pp.a;
  const int chk = paged_rows(page_table, table_width, batch, pages, page_size, ap.rows);
  if (chk != DDT_OK) return chk;
  if (T > DDT_MAX_B + 1 || head_dim % 8 != 0 || head_dim > 512 || rope_dim % 16 != 0 ||
      q_heads > 0xFFFF || kv_heads > 0xFFFF)
    return DDT_ENOTSUP;
  if ((q_heads > 0 && q_stride % 8 != 0) || k_stride % 8 != 0 || v_stride % 8 != 0)
    return DDT_ENOTSUP;
  if (batch > 0x7FFFFFFFLL / T || !launchable(batch * T, ddt::kApThreads)) return DDT_ENOTSUP;
  ap.q = q;
  ap.k = k;
  ap.v = v;
  ap.q_stride = q_stride;
  ap.k_stride = k_stride;
  ap.v_stride = v_stride;
  ap.T = T;
  ap.q_heads = q_heads;
  ap.kv_heads = kv_heads;
  ap.head_dim = head_dim;
  ap.rope = rope;
  ap.rope_len = rope_len;
  ap.rot = rope_dim;
  ap.past_len = past_len;
  ap.depths = depths;
  ap.num_nodes = num_nodes;
  ap.k_cache = k_cache;
  ap.v_cache = v_cache;
  ap.q_out = q_out;
  pp.k_scale = k_scale;
  pp.v_scale = v_scale;
  const int64_t blocks = batch * T;
  if (cache_dtype == DDT_E4M3) {
    if (dtype == DDT_BF16)
      launch_append8<__bf16, ddt::kCodeE4M3>(pp, blocks, interleaved, stream);
    else
      launch_append8<_Float16, ddt::kCodeE4M3>(pp, blocks, interleaved, stream);
  } else {
    if (dtype == DDT_BF16)
      launch_append8<__bf16, ddt::kCodeI8>(pp, blocks, interleaved, stream);
    else
      launch_append8<_Float16, ddt::kCodeI8>(pp, blocks, interleaved, stream);
  }
  return hipGetLastError() == hipSuccess ? DDT_OK : DDT_EHIP;
}

int ddtree_compact_kv8(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                       int64_t layers, int64_t pages, int32_t heads, int32_t page_size,
                       int32_t head_dim, const int32_t* page_table, int64_t table_width,
                       int64_t batch, const int32_t* past_len, const int32_t* accepted_nodes,
                       const int32_t* accept_len, int32_t L, int32_t* new_len,
                       hipStream_t stream) {
  if (layers < 0 || batch < 0 || heads < 0 || head_dim <= 0 || L <= 0) return DDT_EINVAL;
  if (layers == 0 || batch == 0 || heads == 0) return DDT_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !past_len || !accepted_nodes || !accept_len)
    return DDT_EINVAL;
  if (((uintptr_t)k_cache | (uintptr_t)v_cache) & 15 ||
      ((uintptr_t)k_scale | (uintptr_t)v_scale) & 3)
    return DDT_EINVAL;
  ddt::Kv8CompactParams kp;
  const int chk = paged_rows(page_table, table_width, batch, pages, page_size, kp.rows);
  if (chk != DDT_OK) return chk;
  if (head_dim % 8 != 0 || head_dim > 512 || L > DDT_MAX_L) return DDT_ENOTSUP;
  const int64_t per_block = ddt::kK8Threads / ddt::kWave;
  if (batch > 0x7FFFFFFFLL || layers > 0x7FFFFFFFLL / heads) return DDT_ENOTSUP;
  const int64_t slices = layers * heads;
  // one wave for each slice (layer and head) of a request until they fill the
  // card, then up to 16 slices to a wave, which find the rows' pages once (64
  // requests, 36 layers of 8 heads: a call with two slices to a wave 18.0 us, with
  // one 20.8; 4 and 64 at most as 16)
  int64_t each = slices * batch / 8192;
  each = each < 1 ? 1 : (each > 16 ? 16 : each);
  kp.waves = (int32_t)((slices + each - 1) / each);
  kp.each = (int32_t)each;
  if (batch > 0x7FFFFFFFLL / kp.waves) return DDT_ENOTSUP;
  const int64_t blocks = (batch * kp.waves + per_block - 1) / per_block;
  if (!launchable(blocks, ddt::kK8Threads)) return DDT_ENOTSUP;
  kp.k = (unsigned char*)k_cache;
  kp.v = (unsigned char*)v_cache;
  kp.k_scale = k_scale;
  kp.v_scale = v_scale;
  kp.layers = layers;
  kp.batch = batch;
  kp.heads = heads;
  kp.row_bytes = head_dim;
  kp.past_len = past_len;
  kp.accepted = accepted_nodes;
  kp.accept_len = accept_len;
  kp.L = L;
  kp.new_len = new_len;
  if (head_dim % 16 == 0)
    hipLaunchKernelGGL(ddt::compact8_kernel<ddt::k8_u32x4>, dim3((unsigned)blocks), dim3(ddt::kK8Threads),
                       0, stream, kp);
  else
    hipLaunchKernelGGL(ddt::compact8_kernel<ddt::k8_u32x2>, dim3((unsigned)blocks), dim3(ddt::kK8Threads),
                       0, stream, kp);
  return hipGetLastError() == hipSuccess ? DDT_OK : DDT_EHIP;
}

int ddtree_read_kv8(int cache_dtype, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, int32_t kv_heads, int32_t head_dim,
                    const int32_t* page_table, int64_t table_width, int64_t pages,
                    int32_t page_size, int64_t batch, const int32_t* first, const int32_t* count,
                    int32_t n, int dtype, void* k_out, void* v_out, hipStream_t stream) {
  if (!valid_codes(cache_dtype) || (!valid_half(dtype) && dtype != DDT_F32) || batch < 0 ||
      kv_heads <= 0 || head_dim <= 0 || n < 0)
    return DDT_EINVAL;
  if (batch == 0 || n == 0) return DDT_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !first || !k_out || !v_out)
    return DDT_EINVAL;
  if (((uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)k_out | (uintptr_t)v_out) & 15 ||
      ((uintptr_t)k_scale | (uintptr_t)v_scale) & 3)
    return DDT_EINVAL;
  ddt::Read8Params rp;
  const int chk = paged_rows(page_table, table_width, batch, pages, page_size, rp.rows);
  if (chk != DDT_OK) return chk;
  if (head_dim % 8 != 0 || head_dim > 512 || kv_heads > 0xFFFF) return DDT_ENOTSUP;
  const int64_t width = (int64_t)kv_heads * (head_dim / 8);  // < 2^22
  // two pieces to a thread, or a row (16 requests of 8 k rows: one, two, four
  // pieces 135.6, 136.2, 140.6 us; few rows alike)
  int64_t per = 2 * ddt::kR8Threads / width;
  per = per < 1 ? 1 : per;
  rp.per = (int32_t)per;
  rp.parts = (n + per - 1) / per;
  if (batch > 0x7FFFFFFFLL / rp.parts || !launchable(batch * rp.parts, ddt::kR8Threads))
    return DDT_ENOTSUP;
  rp.k = (const unsigned char*)k_cache;
  rp.v = (const unsigned char*)v_cache;
  rp.k_scale = k_scale;
  rp.v_scale = v_scale;
  rp.heads = kv_heads;
  rp.head_dim = head_dim;
  rp.first = first;
  rp.count = count;
  rp.n = n;
  rp.k_out = k_out;
  rp.v_out = v_out;
  const int64_t blocks = batch * rp.parts;
  if (dtype == DDT_BF16)
    launch_read8<__bf16>(rp, blocks, cache_dtype, stream);
  else if (dtype == DDT_F16)
    launch_read8<_Float16>(rp, blocks, cache_dtype, stream);
  else
    launch_read8<float>(rp, blocks, cache_dtype, stream);
  return hipGetLastError() == hipSuccess ? DDT_OK : DDT_EHIP;
}

size_t ddtree_attention_kv8_workspace_size(int64_t batch, int32_t T, int32_t q_heads,
                                           int32_t kv_heads, int32_t head_dim,
                                           int64_t pages_per_request, int32_t page_size,
                                           int32_t shared) {
  return attention_workspace(batch, T, q_heads, kv_heads, head_dim, pages_per_request, page_size,
                             1, shared != 0);
}

int ddtree_attention_kv8(const void* q, int dtype, int64_t batch, int32_t T, int32_t q_heads,
                         int32_t kv_heads, int32_t head_dim, int cache_dtype, const void* k_cache,
                         const void* v_cache, const float* k_scale, const float* v_scale,
                         const int32_t* page_table, int64_t table_width, int64_t pages,
                         int32_t page_size, const int32_t* past_len, const int32_t* num_nodes,
                         const uint64_t* mask, const int32_t* shared_len, float scale, void* out,
                         float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!valid_codes(cache_dtype)) return DDT_EINVAL;
  if (batch > 0 && (!k_scale || !v_scale || ((uintptr_t)k_scale | (uintptr_t)v_scale) & 3))
    return DDT_EINVAL;
  return attention(q, dtype, batch, T, q_heads, kv_heads, head_dim, 1,
                   cache_dtype == DDT_E4M3 ? ddt::launch_attn_e4m3 : ddt::launch_attn_i8, k_cache,
                   v_cache, k_scale, v_scale, page_table, table_width, pages, page_size, past_len,
                   num_nodes, mask, shared_len, scale, out, lse, workspace, workspace_bytes, stream);
}

size_t ddtree_attention_shared_workspace_size(int64_t batch, int32_t T, int32_t q_heads,
                                              int32_t kv_heads, int32_t head_dim,
                                              int64_t pages_per_request, int32_t page_size) {
  return attention_workspace(batch, T, q_heads, kv_heads, head_dim, pages_per_request, page_size,
                             2, true);
}

int ddtree_attention_shared(const void* q, int dtype, int64_t batch, int32_t T, int32_t q_heads,
                            int32_t kv_heads, int32_t head_dim, const void* k_cache,
                            const void* v_cache, const int32_t* page_table, int64_t table_width,
                            int64_t pages, int32_t page_size, const int32_t* past_len,
                            const int32_t* num_nodes, const uint64_t* mask,
                            const int32_t* shared_len, float scale, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (batch > 0 && (!shared_len || !page_table)) return DDT_EINVAL;
  const bool apart =
      attn_check(dtype, batch, T, q_heads, kv_heads, head_dim) == DDT_OK && batch > 0 &&
      table_width > 0 && page_size > 0 &&
      shares(batch, T, q_heads, kv_heads, head_dim,
             table_width > 0x7FFFFFFFLL / page_size ? 0x7FFFFFFFLL : table_width * page_size, 2);
  if (!apart)
    return ddtree_attention(q, dtype, batch, T, q_heads, kv_heads, head_dim, k_cache, v_cache,
                            page_table, table_width, pages, page_size, past_len, num_nodes, mask,
                            scale, out, lse, workspace, workspace_bytes, stream);
  return attention(q, dtype, batch, T, q_heads, kv_heads, head_dim, 2, ddt::launch_attn_shared,
                   k_cache, v_cache, nullptr, nullptr, page_table, table_width, pages, page_size,
                   past_len, num_nodes, mask, shared_len, scale, out, lse, workspace,
                   workspace_bytes, stream);
}

}  // extern "C"
