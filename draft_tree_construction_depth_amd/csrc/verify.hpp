// Host side of the paged caches and of the attention over them: argument
// checks, launch geometry and workspace, shared by the sources that hold the
// entry points and the kernels' variants.
#pragma once

#include "ddtree.h"

#include "attention.hpp"

namespace ddt {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

// ---- paged caches -------------------------------------------------------------
// A layer's cache of `pages` pages and the table that maps `batch` requests'
// rows onto it (null: page b is request b's). Page sizes behind a table are
// powers of two, so that no row needs a division.
inline int paged_rows(const int32_t* table, int64_t width, int64_t batch, int64_t pages,
               int64_t page_size, PagedRows& r) {
  if (pages <= 0 || page_size <= 0 || (table && width <= 0)) return DDT_EINVAL;
  if (!table && pages != batch) return DDT_EINVAL;
  if (pages > 0x7FFFFFFFLL || page_size > 0x7FFFFFFFLL || width > 0x7FFFFFFFLL) return DDT_ENOTSUP;
  if (table && (page_size & (page_size - 1))) return DDT_ENOTSUP;
  r.table = table;
  r.width = table ? width : 1;
  r.pages = pages;
  r.page_size = (int32_t)page_size;
  r.shift = 31;
  if (table)
    for (r.shift = 0; ((int64_t)1 << r.shift) < page_size; ++r.shift) {
    }
  r.cap = r.width * page_size;
  if (r.cap > 0x7FFFFFFFLL) r.cap = 0x7FFFFFFFLL;  // lengths are 32-bit
  return DDT_OK;
}

// Whether one launch takes `blocks` workgroups: it has fewer than 2^32 threads.
inline bool launchable(int64_t blocks, int threads) { return blocks <= 0xFFFFFFFFLL / threads; }

inline bool valid_half(int dtype) { return dtype == DDT_BF16 || dtype == DDT_F16; }

// ---- attention: waves along the queries, workgroups, workspace -------------------
struct AttnPlan {
  int NQ, QW;  // queries of a wave, waves side by side
  int64_t groups, least, grid;
  int64_t units;  // no call has more
  bool merge;  // a unit can be cut
  size_t part, ml, end;
};

inline AttnPlan attn_plan_host(int64_t batch, int32_t T, int32_t q_heads, int32_t kv_heads,
                        int32_t head_dim, int64_t cap, bool codes = false) {
  AttnPlan pl;
  const int G = q_heads / kv_heads;
  // M query rows share a key/value head's pass. Up to 64: 16 to a wave, as many
  // waves side by side as they fill; more: 32 to a wave (at head_dim 256 always
  // 16, and two waves or more: 32 queries' state or four groups' tiles would
  // not leave registers for the next tile). 32 requests x 4 heads over 4096
  // rows, us at 16x1 / 16x2 / 16x4 / 32x4 queries x waves:
  //   head_dim 128  M = 16: 62 / 64 / 71 / 77   32: 65 / 63 / 67 / 75
  //                 64: 87 / 74 / 69 / 77       256: 239 / 165 / 117 / 104
  //   head_dim 64   M = 16: 36 / 37 / 39 / 42   64: 53 / 46 / 41 / 44
  //                 128: 83 / 67 / 50 / 53      256: 129 / 85 / 77 / 66
  //   head_dim 256  M = 16: - / 114 / 125 / 276 128: - / 289 / 180 / 323
  // (the last column of 256 with tiles that went through registers)
  const int64_t M = (int64_t)T * G;
  pl.NQ = M <= 64 || head_dim == 256 ? 16 : 32;
  pl.QW = M <= 16 && head_dim < 256 ? 1 : (M <= 32 ? 2 : 4);
  const int rows = pl.QW == 4 ? (head_dim <= 128 ? 64 : 32) : 32 * (4 / pl.QW);  // AttnTile::TR
  const int64_t steps = (cap + rows - 1) / rows;
  const int64_t tiles = (M + pl.NQ * pl.QW - 1) / (pl.NQ * pl.QW);
  pl.least = 2;
  // two workgroups on each of 256 CUs (one where a tile fills the LDS or the
  // registers, or AttnTile::PER_CU), fewer for little work
  pl.groups = head_dim == 256 ? 256 : (codes && head_dim == 64 && pl.NQ == 32 ? 768 : 512);
  const int64_t axis = steps > ((int64_t)1 << 31) / (kv_heads * tiles) / batch
                           ? (int64_t)1 << 31
                           : batch * kv_heads * tiles * steps;
  const int64_t want = ((axis + pl.least - 1) / pl.least + 7) & ~(int64_t)7;
  if (want < pl.groups) pl.groups = want;
  // or one for each unit, where there are many (attn_plan decides); the XCDs
  // may have one unit of one request more or less, or one key/value head of
  // several requests
  const int64_t units = batch == 1 ? (kv_heads * tiles + 7) & ~(int64_t)7
                                   : ((batch * kv_heads + 7) & ~(int64_t)7) * tiles;
  pl.units = units;
  pl.grid = units >= 2 * pl.groups ? units : pl.groups;
  pl.merge = steps > 1;
  const int64_t slots = pl.merge ? 2 * pl.groups : 0;
  size_t o = align_up((size_t)(pl.groups + 1) * sizeof(AttnPlace));
  pl.part = o;
  o = align_up(o + (size_t)slots * pl.QW * pl.NQ * head_dim * sizeof(float));
  pl.ml = o;
  o = align_up(o + (size_t)slots * pl.QW * 64 * 2 * sizeof(float));
  pl.end = o;
  return pl;
}

template <typename H, int DH, int NQ, int QW, int CACHE, bool EXT>
int launch_attn_tile(const AttnParams& ap, const AttnPlan& pl, hipStream_t st) {
  hipLaunchKernelGGL((attn_kernel<H, DH, NQ, QW, CACHE, EXT>), dim3((unsigned)pl.grid),
                     dim3(kAtThreads), 0, st, ap);
  if (hipGetLastError() != hipSuccess) return DDT_EHIP;
  if (!pl.merge) return DDT_OK;
  const int64_t merges = (EXT ? ap.places : pl.groups) * QW * AttnTile<DH, NQ, QW>::PIECES / kAtMerge;
  if constexpr (EXT)
    hipLaunchKernelGGL((attn_merge_many_kernel<H, DH, NQ, QW, CACHE>), dim3((unsigned)merges),
                       dim3(kAtThreads), 0, st, ap);
  else
    hipLaunchKernelGGL((attn_merge_kernel<H, DH, NQ, QW>), dim3((unsigned)merges), dim3(kWave), 0,
                       st, ap);
  return hipGetLastError() == hipSuccess ? DDT_OK : DDT_EHIP;
}

template <typename H, int DH, int CACHE, bool EXT>
int launch_attn_waves(const AttnParams& ap, const AttnPlan& pl, hipStream_t st) {
  if constexpr (DH < 256) {
    if (pl.NQ == 32) return launch_attn_tile<H, DH, 32, 4, CACHE, EXT>(ap, pl, st);
    if (pl.QW == 1) return launch_attn_tile<H, DH, 16, 1, CACHE, EXT>(ap, pl, st);
  }
  if (pl.QW == 4) return launch_attn_tile<H, DH, 16, 4, CACHE, EXT>(ap, pl, st);
  return launch_attn_tile<H, DH, 16, 2, CACHE, EXT>(ap, pl, st);
}

template <typename H, int CACHE = kAtSame, bool EXT = false>
int launch_attn(const AttnParams& ap, const AttnPlan& pl, int head_dim, hipStream_t st) {
  switch (head_dim) {
    case 64: return launch_attn_waves<H, 64, CACHE, EXT>(ap, pl, st);
    case 128: return launch_attn_waves<H, 128, CACHE, EXT>(ap, pl, st);
    default: return launch_attn_waves<H, 256, CACHE, EXT>(ap, pl, st);
  }
}

inline int attn_check(int dtype, int64_t batch, int32_t T, int32_t q_heads, int32_t kv_heads,
               int32_t head_dim) {
  if (!valid_half(dtype) || batch < 0 || T <= 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0)
    return DDT_EINVAL;
  if (q_heads % kv_heads != 0) return DDT_EINVAL;
  if (T > DDT_MAX_B + 1 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return DDT_ENOTSUP;
  // keeps the plan's counts far below 63 bits; the launch itself is tested with the plan
  if (batch > 0x1FFFFFFFLL || batch * T > 0x1FFFFFFFLL / q_heads) return DDT_ENOTSUP;
  return DDT_OK;
}

// The variants for caches of codes and for shared rows, in sources of their own.
int launch_attn_e4m3(const AttnParams& ap, const AttnPlan& pl, int dtype, int head_dim,
                     hipStream_t st);
int launch_attn_i8(const AttnParams& ap, const AttnPlan& pl, int dtype, int head_dim,
                   hipStream_t st);
int launch_attn_shared(const AttnParams& ap, const AttnPlan& pl, int dtype, int head_dim,
                       hipStream_t st);

}  // namespace ddt
