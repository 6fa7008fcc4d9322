"""Host logic of the latent kernels' roles, compiled from the kernels' own headers into a host program (no GPU).

  * The barrier and parity that a role waits on for the queries of a segment: a role that is up to one segment late must
    still find them complete, one that is early must not.
  * Which requests of a page plan are served, when the pages they ask for exceed 31 and 32 bits.
  * The slots that a unit's record of its parts may name, whatever the record holds.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_decode_attention_b200", "csrc")

PROG = r'''
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "k_latent.cuh"
using namespace s4r;
int main(int argc, char **argv) {
  if (argc == 1) {
    for (int i = 0; i < 64; ++i) printf("query %d %d %u\n", i, la_query_bar(i), la_query_parity(i));
    return 0;
  }
  if (argc == 5 && argv[1][0] == 'p') {   // p groups row_blocks seed: every legal record, then random ones
    const int groups = atoi(argv[2]), blocks = atoi(argv[3]);
    const long long slots = 2LL * groups * blocks;
    srand(atoi(argv[4]));
    for (int c = 0; c < groups * blocks; ++c)
      for (int second = 0; second < 2; ++second)
        for (int n = 1; c / blocks + n <= groups; ++n)
          if (!la_parts_ok(2 * c + second, n, groups, blocks)) printf("refused %d %d\n", 2 * c + second, n);
    for (int i = 0; i < 2000000; ++i) {
      const int mask = 1 << (rand() % 31);
      int first = (int)((unsigned)rand() * 3u) % mask, n = (int)((unsigned)rand() * 5u) % mask;
      if (rand() % 4 == 0) first = -first;
      if (rand() % 4 == 0) n = -n;
      if (i < 4) first = i & 1 ? INT32_MAX : INT32_MIN, n = i & 2 ? INT32_MAX : 1;
      if (!la_parts_ok(first, n, groups, blocks)) continue;
      for (int k = 0; k < n; ++k)
        if (la_part_slot(first, k, blocks) < 0 || la_part_slot(first, k, blocks) >= slots) printf("outside %d %d\n", first, n);
    }
    return 0;
  }
  const int32_t free_pages = atoi(argv[1]);   // then the pages that each request needs
  std::vector<uint32_t> demand(1, 0u);
  long long sum = 0;
  for (int i = 2; i < argc; ++i) demand.push_back(plan_hold_pages(sum += atoll(argv[i])));
  for (int i = 2; i < argc; ++i)   // need pages of 16 tokens, 5 tokens of a page held already
    printf("served %d\n", plan_served(5, atoi(argv[i]) ? 16 * atoi(argv[i]) : 11, 1 << 27, 4, demand[i - 1], free_pages) ? 1 : 0);
  printf("taken %u\n", demand[plan_find(demand.data(), argc - 2, (uint32_t)free_pages)]);
  return 0;
}
'''


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("roles")
    src, out = d / "roles.cu", d / "roles"
    src.write_text(PROG)
    subprocess.run(["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O1", "--expt-relaxed-constexpr",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(out)], check=True)

    def run(key, *args):
        text = subprocess.run([str(out), *map(str, args)], capture_output=True, text=True, check=True).stdout
        return [[int(x) for x in line.split()[1:]] for line in text.splitlines() if line.split()[0] == key]
    return run


def test_queries_are_found_by_a_late_role(host):
    """The queries of segments 0 .. done are complete.  A softmax warp that waits for segment i has not handled its first
    tile, so the queries of i + 2 cannot be (they need q_empty of i + 1, and the products behind it need this warp):
    done is i - 1 (not yet there), i, or i + 1.  A wait for the phase of parity P on a barrier returns when the phase in
    progress has the other parity."""
    place = {i: (bar, parity) for i, bar, parity in host("query")}
    for i in range(62):
        for done in (i - 1, i, i + 1):
            phases = {bar: sum(1 for k in range(done + 1) if place[k][0] == bar) for bar in (0, 1)}
            bar, parity = place[i]
            assert (phases[bar] % 2 != parity) == (done >= i), (i, done)


@pytest.mark.parametrize("free", [0, 3, 2 ** 27, 2 ** 31 - 1])
@pytest.mark.parametrize("needs", [[2 ** 27 - 1] * 17 + [1, 0, 2], [1, 2, 0, 1], [2 ** 27 - 1] * 16 + [15, 1, 0, 1],
                                   [2 ** 27 - 1] * 40 + [1, 0]])
def test_the_plan_serves_while_the_demand_fits(host, needs, free):
    demand, want, taken = 0, [], 0
    for need in needs:
        demand += need
        want.append([int(need == 0 or demand <= free)])
        if demand <= free:
            taken = demand
    assert host("served", free, *needs) == want
    assert host("taken", free, *needs) == [[taken]]


@pytest.mark.parametrize("groups,blocks", [(148, 1), (74, 2), (1, 1024), (5, 3), (1, 1)])
def test_records_of_parts(host, groups, blocks):
    assert host("refused", "p", groups, blocks, 1) == []
    assert host("outside", "p", groups, blocks, 1) == []
