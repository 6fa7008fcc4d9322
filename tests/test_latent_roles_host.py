"""Host logic of the latent kernels' roles, compiled from the kernels' own headers into a host program (no GPU).

  * The barrier and parity that a role waits on for the queries of a segment: a role that is up to one segment late must
    still find them complete, one that is early must not.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_decode_attention_b200", "csrc")

PROG = r'''
#include <cstdio>
#include "k_latent.cuh"
using namespace s4r;
int main() {
  for (int i = 0; i < 64; ++i) printf("query %d %d %u\n", i, la_query_bar(i), la_query_parity(i));
  return 0;
}
'''


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("roles")
    src, out = d / "roles.cu", d / "roles"
    src.write_text(PROG)
    subprocess.run(["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O1", "--expt-relaxed-constexpr",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(out)], check=True)
    rows = [line.split() for line in subprocess.run([str(out)], capture_output=True, text=True, check=True).stdout.splitlines()]
    return lambda key: [[int(x) for x in r[1:]] for r in rows if r[0] == key]


def test_queries_are_found_by_a_late_role(lines):
    """The queries of segments 0 .. done are complete.  A softmax warp that waits for segment i has not handled its first
    tile, so the queries of i + 2 cannot be (they need q_empty of i + 1, and the products behind it need this warp):
    done is i - 1 (not yet there), i, or i + 1.  A wait for the phase of parity P on a barrier returns when the phase in
    progress has the other parity."""
    place = {i: (bar, parity) for i, bar, parity in lines("query")}
    for i in range(62):
        for done in (i - 1, i, i + 1):
            phases = {bar: sum(1 for k in range(done + 1) if place[k][0] == bar) for bar in (0, 1)}
            bar, parity = place[i]
            assert (phases[bar] % 2 != parity) == (done >= i), (i, done)
