"""Which bytes the kernel of attention over the cache fetches of a token: compiled from its own header for the host."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "walsh_hadamard_sparse_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

PROGRAM = r"""
#include <cstdio>
#include "attention_mma.cuh"
using namespace qwha;
using namespace qwha::attn;

// Of a pool's last token, every block of cached heads: the pieces of each array end where the array ends, cover what the
// block has, and lie within the stage. Returns the number of pieces that break this.
static long check(int D, int bits_k, int bits_v, int group_k, int group_v, int heads, int warps, int nt, int pieces) {
  const int dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  const int blocks = (heads + warps - 1) / warps, hb = (heads + blocks - 1) / blocks, per_head = warps / hb > 0 ? warps / hb : 1;
  const MmaShape sh(D, dp, bits_k, bits_v, group_k, group_v, nt, pieces, heads, hb, per_head, hb * per_head);
  long bad = 0;
  const int bits[2] = {bits_k, bits_v}, group[2] = {group_k, group_v};
  for (int kv0 = 0; kv0 < heads; kv0 += hb) {
    const int here = heads - kv0 < hb ? heads - kv0 : hb;
    for (int i = 0; i < 2; ++i) {
      const int head[3] = {D / 8 * bits[i], D / group[i] * 4, D / group[i]};
      const Part *parts[3] = {&sh.codes[i], &sh.scales[i], &sh.zeros[i]};
      for (int w = 0; w < 3; ++w) {
        const Part &p = *parts[w];
        bad += p.head != head[w] || p.stride != heads * head[w];
        // wide 0 is bounded by the array's end as it is fetched, whatever the number of pieces
        if (p.wide) bad += kv0 * head[w] + p.pieces(here) * p.wide != (kv0 + here) * head[w];
        else bad += p.pieces(here) * 4 < here * head[w] + 3;
        bad += p.pieces(hb) != p.per || p.pieces(here) > p.per || p.per * (p.wide ? p.wide : 4) > p.pitch;
      }
      // whole blocks in 16-byte pieces: as many of the codes for every head
      if (sh.fast && here == hb) bad += sh.codes[i].wide != 16 || sh.codes[i].per != hb * (sh.row[i] >> 4);
    }
  }
  return bad;
}

int main() {
  const int dims[][2] = {{8, 8}, {24, 8}, {40, 8}, {64, 64}, {64, 32}, {80, 40}, {96, 32}, {96, 96}, {128, 128}, {128, 64},
                         {128, 8}, {256, 256}, {256, 64}};
  const int bits[] = {2, 3, 4, 8};
  long bad = 0, partial = 0;
  for (auto &d : dims)
    for (int bk : bits)
      for (int bv : bits) {
        if ((bk == 2 || bv == 2) && d[0] % 16) continue;
        for (int heads = 1; heads <= 64; ++heads)
          for (int warps = 8; warps; warps /= 2)
            for (int pieces = 1; pieces <= 2; ++pieces) {
              const long b = check(d[0], bk, bv, d[1], d[1], heads, warps, 1, pieces);
              if (b && !bad) printf("first: D %d bits %d %d group %d heads %d warps %d: %ld\n", d[0], bk, bv, d[1], heads, warps, b);
              bad += b;
              const int blocks = (heads + warps - 1) / warps, hb = (heads + blocks - 1) / blocks;
              partial += heads % hb != 0;
            }
      }
  printf("partial %ld bad %ld\n", partial, bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(not shutil.which(NVCC), reason="needs nvcc")
def test_pieces_end_where_the_cache_ends(tmp_path):
    """Every number of cached heads up to 64, blocks of 1 to 8 of them, the last block with fewer among them."""
    src, exe = tmp_path / "reads.cu", tmp_path / "reads"
    src.write_text(PROGRAM)
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-O1", "-std=c++17", "--expt-relaxed-constexpr", f"-I{CSRC}",
                    f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split("partial ")[1].split()[0]) > 1000
