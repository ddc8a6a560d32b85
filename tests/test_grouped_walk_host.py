"""The tile indices of the grouped products on the host, compiled from the
kernels' headers and run on the CPU: at the largest sizes that the calls take,
the band of row tiles that each form asks for maps every tile index to a tile
of the grid, without leaving 32 bits."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_epilogue_fusion_gb300", "csrc")

PROGRAM = r"""
#include "grouped_skinny.cuh"
#include "grouped_wgrad.cuh"
#include <cstdio>
#include <cstdlib>
#include <cstring>
using namespace coda;
// the sizes that the calls take (check_grouped)
static bool taken(long long T, long long E, long long N, long long K) {
  return N < (1ll << 30) && K < (1ll << 30) && N * K < (1ll << 37) &&
         (T / 32 + E) * ((N + 63) / 64) < (1ll << 30) && E * ((N + 127) / 128) * ((K + 127) / 128) < (1ll << 30);
}
// tile_coord in 64 bits
static bool right(long long t, long long m_tiles, long long n_tiles, long long group) {
  const long long per = group * n_tiles, g = t / per, first = g * group;
  const long long gm = group < m_tiles - first ? group : m_tiles - first, local = t - g * per;
  if (per > 2147483647ll || static_cast<int>(per) == 0) {  // the 32-bit product would wrap
    printf("band of %lld row tiles x %lld column tiles\n", group, n_tiles);
    return false;
  }
  const TileCoord c = tile_coord(static_cast<int>(t), static_cast<int>(m_tiles), static_cast<int>(n_tiles),
                                 static_cast<int>(group));
  return c.m == first + local % gm && c.n == local / gm && c.m >= 0 && c.m < m_tiles && c.n >= 0 && c.n < n_tiles;
}
template <class C>
static void form(const char* name, long long T, long long E, long long N, long long K) {
  if (!taken(T, E, N, K)) { printf("FAIL size %lld %lld %lld %lld\n", T, E, N, K); exit(1); }
  GroupProblem p = {};
  p.T = static_cast<int>(T), p.E = static_cast<int>(E), p.N = static_cast<int>(N), p.K = static_cast<int>(K);
  const GroupArgs a = group_args<C>(p);
  // an expert with all rows, and one with a single row
  for (long long rows : {T, 1ll}) {
    const long long m = C::WGRAD ? a.m_tiles : (rows + C::TILE_M - 1) / C::TILE_M, tiles = m * a.n_tiles;
    for (long long t : {0ll, 1ll, tiles / 3, tiles / 2, tiles - 2, tiles - 1})
      if (t >= 0 && t < tiles && !right(t, m, a.n_tiles, a.group)) {
        printf("FAIL %s T=%lld E=%lld N=%lld K=%lld tile %lld of %lld x %d\n", name, T, E, N, K, t, m, a.n_tiles);
        exit(1);
      }
  }
}
template <int PROG>
static void forms(long long T, long long E, long long N, long long K) {
  form<SkinnyCfg<kKindBF16, PROG, 1>>("32 rows", T, E, N, K);
  form<SkinnyCfg<kKindBF16, PROG, 8>>("32 rows, split", T, E, N, K);
  form<GroupCfg<kKindBF16, PROG, 4, 2>>("lone", T, E, N, K);
  form<WideCfg<kKindBF16, PROG>>("pairs", T, E, N, K);
}
int main() {
  const long long sizes[][4] = {{1, 1, (1 << 24), 256},        {64, 1, (1 << 24), 256},      {1, 1, (1 << 23), 256},
                                {64, 2, (1 << 23), 256},       {100, 1, (1 << 24) - 8, 256}, {96, 3, (1 << 23) - 8, 512},
                                {1, 1, (1 << 30) - 8, 120},    {1900, 4, (1 << 30) - 8, 120}, {2147482000, 1, 960, 64},
                                {2147482000, 1024, 896, 64},   {500, 1024, 1 << 25, 8},      {33, 1, (1 << 24) + 64, 256}};
  for (const auto& s : sizes) {
    if (!taken(s[0], s[1], s[2], s[3])) { printf("skip %lld %lld %lld %lld\n", s[0], s[1], s[2], s[3]); continue; }
    forms<kGroupPlain>(s[0], s[1], s[2], s[3]);
    forms<kGroupSwiGLU>(s[0], s[1], s[2], s[3]);
    form<GroupCfg<kKindBF16, kGroupWgrad, 3, 4>>("weight gradient", s[0], s[1], s[2], s[3]);
    form<WgradCfg>("weight gradient, pairs", s[0], s[1], s[2], s[3]);
    printf("size %lld %lld %lld %lld\n", s[0], s[1], s[2], s[3]);
  }
  printf("all ok\n");
  return 0;
}
"""


def test_bands_of_row_tiles_stay_within_32_bits(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "walk.cu", tmp_path / "walk"
    src.write_text(PROGRAM)
    # the host's side alone
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                        "--expt-relaxed-constexpr", "-gencode", "arch=compute_103a,code=sm_103a", str(src),
                        "-o", str(exe), "-lcuda"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "all ok" in out.stdout, out.stdout[-2000:]
    assert out.stdout.count("size ") >= 10, out.stdout
