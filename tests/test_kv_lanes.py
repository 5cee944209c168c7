"""The single-token attention kernel on the host, lane by lane: its loads of a
cache row lie inside the row, and together they are the whole row; its join's
sums are of the workgroup's own threads, each of them added once."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_decode_mat_amd", "csrc")

SOURCE = r"""
#include <cstdio>
#include <cstring>
#include "kv_lanes.h"

static int bad = 0;
static void load(const char* what, int dim, int bytes, int first, int n, char* seen) {
  if (first < 0 || first + n > dim) {
    std::printf("%s, %d dims of %d bytes: reads %d..%d\n", what, dim, bytes, first, first + n - 1);
    ++bad;
  } else {
    std::memset(seen + first, 1, n);
  }
}

template <int DP, bool FULL>
static void check(int dim) {
  for (int bytes = 1; bytes <= 2; ++bytes) {
    char k[256] = {}, v[256] = {};
    for (int s = 0; s < xq::decode_k_loads(DP, bytes); ++s)
      for (int g = 0; g < 4; ++g) load("k", dim, bytes, xq::decode_k_dim<DP, FULL>(s, g, bytes, dim), 16 / bytes, k);
    for (int c = 0; c < xq::decode_v_loads(DP); ++c)
      for (int l = 0; l < 16; ++l) load("v", dim, bytes, xq::decode_v_dim<DP, FULL>(c, l, dim), xq::decode_v_dims(DP), v);
    for (int d = 0; d < dim; ++d)
      if (!k[d] || !v[d]) std::printf("dim %d of %d is not read\n", d, dim), ++bad;
  }
}

template <int DP>
static void check_pad(int dim) {
  if (dim == DP) check<DP, true>(dim);
  check<DP, false>(dim);
}

static void join(int heads, int dp) {
  const int threads = 256, quads = heads * dp / 4, teams = xq::join_teams(threads, quads);
  int outputs = 0;
  for (int q0 = 0; q0 < quads; q0 += threads / teams) {
    char added[256] = {};
    for (int t = 0; t < threads; ++t) {
      if (!xq::join_adds(t, teams, quads - q0)) continue;
      ++outputs;
      for (int i = 0; i < teams; ++i)
        if (t + i >= threads || added[t + i]++) std::printf("%d heads of %d: thread %d adds %d\n", heads, dp, t, t + i), ++bad;
    }
  }
  if (outputs != quads) std::printf("%d heads of %d: %d of %d outputs\n", heads, dp, outputs, quads), ++bad;
}

int main() {
  for (int heads = 1; heads <= 16; ++heads)
    for (int dp = 64; dp <= 256; dp += 64) join(heads, dp);
  for (int dim = 16; dim <= 256; dim += 16) switch (xq::decode_dim_pad(dim)) {
      case 64: check_pad<64>(dim); break;
      case 128: check_pad<128>(dim); break;
      case 192: check_pad<192>(dim); break;
      case 256: check_pad<256>(dim); break;
      default: std::printf("dim %d has no padded size\n", dim), ++bad;
    }
  return bad != 0;
}
"""


def test_every_load_lies_in_its_row(tmp_path):
    src, exe = tmp_path / "lanes.cpp", tmp_path / "lanes"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
