"""The paged latent operators and prefill attention at rare inputs: where their roles, roundings and special cases meet."""
import pytest

import rank_decode_attention_b200 as s4r
from test_gpu_latent import check_latent, latent_problem, run_latent

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- segments of one tile

@pytest.mark.parametrize("dt", ["fp4", "bf16"])
@pytest.mark.parametrize("name,lens,H", [
    ("one row each", [1] * 2000, 16),
    ("behind a long one", [20000] + [1 + 7 * i % 64 for i in range(700)], 64),
    ("long and short by turns", [(3000 if i % 40 == 20 else 1 + i % 64) for i in range(400)], 64),
    ("many empty", [(1 if i % 3 == 0 else 0) for i in range(6000)], 3)])
def test_segments_of_one_tile(name, lens, H, dt):
    """Many requests of one tile a CTA: the softmax warps come to a request while the queries of the next one are
    already there."""
    p = latent_problem(dt, lens, 1, H, 96, 16, seed=len(lens), waste=0)
    d = run_latent(p, 64, 0.1)
    assert d["status"] == s4r.S4R_OK
    check_latent(p, d, 64, 0.1)
