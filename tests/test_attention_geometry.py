"""The attention kernels' arithmetic of query rows, waves and tiles (csrc/attention.hpp), run on
the host: the functions themselves, compiled with the undefined-behaviour sanitizer, at the sizes
where a product leaves 32 bits. Calls of that size are tested on the GPU in
tests/test_gpu_shared_rows.py."""

import os
import subprocess

import pytest

from draft_tree_construction_depth_amd import _build

PROGRAM = r"""
#include <cstddef>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "attention.hpp"

using namespace ddt;

#define CHECK(x) \
  if (!(x)) printf("%s: DH %d NQ %d QW %d T %d G %d tile %d\n", #x, C::DH, C::NQ, C::QW, p.T, p.G, tile), exit(1)

// One request of T block rows, all of them live: its query tiles hold each query row once.
template <int DH, int NQ, int QW>
void dealt(int T, int G, int kv_heads) {
  using C = AttnTile<DH, NQ, QW>;
  AttnParams p{};
  p.T = T;
  p.G = G;
  p.kv_heads = kv_heads;
  p.q_heads = G * kv_heads;
  p.rows.cap = 4096;
  AttnReq r{};
  r.past = 1000;
  r.rows = T;
  attn_request_sizes<C, false>(p, r);
  const int64_t N = (int64_t)T * G;
  int tile = 0;
  CHECK(r.waves == (N + NQ - 1) / NQ && r.tiles == (r.waves + QW - 1) / QW);
  const int64_t around[] = {0, r.tiles / 2, ((int64_t)1 << 31) / r.waves, r.tiles - 4};  // the third: the border
  for (int64_t at : around)
    for (tile = at < 3 ? 0 : at > r.tiles ? r.tiles : (int)at - 3; tile < at + 4 && tile < r.tiles; ++tile) {
      const int64_t first = (int64_t)tile * r.waves / r.tiles, next = (int64_t)(tile + 1) * r.waves / r.tiles;
      CHECK(attn_first_wave<QW>(r, tile) == first && attn_first_wave<QW>(r, tile + 1) == next);
      CHECK(next > first && next - first <= QW);
      for (int head = 0; head < kv_heads; ++head)
        for (int wq = 0; wq < QW; ++wq)
          for (int lane = 0; lane < kWave; ++lane) {
            const AttnQuery q = attn_query<NQ, QW>(p, r, head * r.tiles + tile, wq, lane);
            const int64_t row = (first + wq) * NQ + lane % NQ;
            CHECK(q.live == (first + wq < next && row < N));
            if (q.live) CHECK(q.i == row / G && q.hq == head * G + row % G);
          }
    }
  tile = r.tiles;
  CHECK(attn_first_wave<QW>(r, 0) == 0 && attn_first_wave<QW>(r, r.tiles) == r.waves);
}

// A request without rows (taken out): one tile that holds none.
template <int DH, int NQ, int QW>
void none(int G) {
  using C = AttnTile<DH, NQ, QW>;
  AttnParams p{};
  p.T = 5;
  p.G = G;
  p.kv_heads = 2;
  p.q_heads = 2 * G;
  p.rows.cap = 4096;
  AttnReq r{};
  r.past = -1;
  attn_request_sizes<C, false>(p, r);
  int tile = 0;
  CHECK(r.tiles == 1 && r.len == 0);
  for (int u = 0; u < 2; ++u)
    for (int wq = 0; wq < QW; ++wq)
      for (int lane = 0; lane < kWave; ++lane) CHECK((!attn_query<NQ, QW>(p, r, u, wq, lane).live));
}

// Query rows of block rows [rows, T) of a head lie one behind the other, block row by block row.
void behind(int T, int rows, int G, int kv_heads) {
  using C = AttnTile<64, 16, 2>;
  AttnParams p{};
  p.T = T;
  p.G = G;
  p.kv_heads = kv_heads;
  p.q_heads = G * kv_heads;
  int tile = 0;
  const int64_t all = (int64_t)(T - rows) * G;
  const int64_t around[] = {0, G, 2 * (int64_t)G, all / 2, all, 1 << 26, 1 << 28};
  const int head = kv_heads - 1;
  for (int64_t at : around)
    for (int64_t k = at < 2 ? 0 : at - 2; k < at + 3 && k < all; ++k)
      CHECK(attn_row_behind(p, 3, rows, head, (int)k) ==
            (3 * (int64_t)T + rows + k / G) * p.q_heads + (int64_t)head * G + k % G);
}

// Each of n stretches or units is one workgroup's, and no XCD (id % 8) has more than an eighth.
void nth(int n) {
  using C = AttnTile<64, 16, 2>;
  AttnParams p{};
  int tile = n;
  const int grid = (n + 7) / 8 * 8 + 24;
  std::vector<int> had(grid), per(8);
  for (int w = 0; w < grid; ++w) {
    const int k = attn_nth(w, n);
    CHECK(k >= 0 && k < grid && !had[k]);
    had[k] = 1;
    if (k < n) ++per[w % 8];
  }
  for (int k = 0; k < n; ++k) CHECK(had[k]);
  for (int x = 0; x < 8; ++x) CHECK(per[x] <= (n + 7) / 8);
}

template <int DH, int NQ, int QW>
void all() {
  const int rows[] = {1, 2, 7, 16, 17, 63, 64, 65, 129, 1000, 513 * 80, 1480000, 1490000, 1500001, 2960000, 2980000,
                      3000001, 6000000, 1 << 25, (1 << 26) + 5, (1 << 29) - 1};
  for (int T : rows) {
    dealt<DH, NQ, QW>(T, 1, 1);
    if (T <= (1 << 29) / 6) dealt<DH, NQ, QW>(T, 3, 2);
    if (T <= (1 << 29) / 80) dealt<DH, NQ, QW>(T, 80, 1);
  }
  dealt<DH, NQ, QW>(513, (1 << 29) / 513, 1);
  none<DH, NQ, QW>(1);
  none<DH, NQ, QW>(80);
}

int main() {
  all<64, 16, 1>();
  all<64, 16, 2>();
  all<64, 16, 4>();
  all<64, 32, 4>();
  all<256, 16, 2>();
  all<256, 16, 4>();
  for (int G : {1, 5, 128, 100000, (1 << 29) / 513}) {
    behind(513, 1, G, 1);
    behind(513, 0, G, 1);
    if (G < 1000) behind(9, 5, G, 7);
  }
  behind(1, 0, (1 << 29) - 1, 1);
  for (int n : {1, 2, 7, 8, 9, 63, 64, 100, 511, 512, 513, 579, 1024, 3 * 257, 12 * 86, 8388607}) nth(n);
  puts("fine");
}
"""


def test_query_rows_of_any_count(tmp_path):
    source, program = tmp_path / "geometry.hip", tmp_path / "geometry"
    source.write_text(PROGRAM)
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("no hipcc")
    made = subprocess.run([hipcc, "--offload-host-only", "-std=c++17", "-O1", "-Xarch_host",
                           "-fsanitize=signed-integer-overflow", "-Xarch_host", "-fno-sanitize-recover=all",
                           "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC, str(source), "-o", str(program)],
                          capture_output=True, text=True)
    assert made.returncode == 0, made.stderr[-4000:]
    ran = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    assert ran.returncode == 0 and ran.stdout == "fine\n", (ran.stdout + ran.stderr)[-2000:]
