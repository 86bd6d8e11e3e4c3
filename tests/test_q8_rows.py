"""Which cache rows the tcgen05 attention over the 8-bit cache reads (CPU): the
kernel's own rule, compiled for the host, walked over every tile, converter
thread and pass.  Every row lies inside the cache and below the context, and
every token of the context whose page is there is read exactly once."""
import subprocess

import pytest

from block_draft_tree_b200 import build

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "attn_q8.cuh"

// args: rule (0: the kernel's, 1: every row of a group, 2: the same, row 0 for a group
// that is not there), rows of the cache, base row, T, page size (0: dense), page ids ...
// (paged), -1: no page.  Prints the rows read outside [0, rows), tokens read at or past T,
// and tokens of the context not read exactly once.
int main(int argc, char** argv) {
  const int rule = atoi(argv[1]), T = atoi(argv[4]), page = atoi(argv[5]);
  const long rows = atol(argv[2]), base = atol(argv[3]);
  long outside = 0, past = 0;
  std::vector<int> seen(T + 256, 0);
  std::vector<char> there(T + 256, 0);
  for (int tile = 0; tile * 128 < T; ++tile)
    for (int tok = 0; tok < 32; ++tok)
      for (int q = 0; q < 8; q += 2) {
        const int t = tile * 128 + (q >> 1) * 32 + tok, t0 = t / 16 * 16;
        long row = -1;                         // the group's first, as the look-up finds it
        if (t0 < T) {
          const int id = page ? atoi(argv[6 + t0 / page]) : 0;
          row = !page ? base + t0 : id < 0 ? -1 : (long)id * page + t0 % page;
        }
        if (t < T && row >= 0) there[t] = 1;
        if (rule == 2 && row < 0) row = 0;
        const bool reads = rule ? row >= 0 : ddt::q8_wide_reads((int)row, q, ddt::q8_wide_left(T, tile, tok));
        if (!reads) continue;
        const long at = row + t % 16;
        outside += at < 0 || at >= rows;
        past += t >= T;
        seen[t]++;
      }
  long wrong = 0;
  for (int t = 0; t < T; ++t) wrong += seen[t] != there[t];
  printf("%ld %ld %ld\n", outside, past, wrong);
}
"""


@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "rows.cu").write_text(SOURCE)
    subprocess.run([build.NVCC] + [f for f in build.FLAGS if f not in ("-shared", "-O3", "-lineinfo")]
                   + ["-o", str(d / "rows"), str(d / "rows.cu")], check=True)

    def run(rule, n, base, T, page=0, ids=()):
        out = subprocess.run([str(d / "rows")] + [str(x) for x in (rule, n, base, T, page, *ids)],
                             check=True, capture_output=True, text=True).stdout
        return tuple(int(x) for x in out.split())
    return run


@pytest.mark.parametrize("t_max", [1, 5, 15, 16, 17, 100, 127, 128, 129, 300])
def test_dense_caches_of_any_length(rows, t_max):
    """The last sequence of a dense cache of two, at every kind of length."""
    for T in {0, 1, t_max // 2, t_max - 1, t_max}:
        assert rows(0, 2 * t_max, t_max, T) == (0, 0, 0)
    if t_max % 16:
        # a rule by whole groups leaves the cache, and this check sees it
        assert rows(1, 2 * t_max, t_max, t_max)[0] > 0


def test_pages_that_are_not_there(rows):
    for page in (16, 48, 64):
        n = -(-300 // page)
        ids = [(3 * i + 1) % n if i % 3 else -1 for i in range(n)]
        assert rows(0, n * page, 0, 300, page, ids) == (0, 0, 0)
        assert rows(2, n * page, 0, 300, page, ids)[2] > 0
