"""The paged latent operators and prefill attention at rare inputs: where their roles, roundings and special cases meet."""
import math

import pytest
import torch

import rank_decode_attention_b200 as s4r
from latent_reference import HALF_STEP, assert_within, cdiv, latent_attend, pack_page, quantise
from test_gpu_latent import (check_latent, check_prefill, check_project, i32, latent_problem, prefill_problem, run_latent,
                             run_prefill, status_words)

pytestmark = pytest.mark.gpu
BF, DEV = torch.bfloat16, "cuda"


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


# ---------------------------------------------------------------- probabilities in 16 bits

def fp16_steps(rows, rank):
    """What the smallest probabilities of a 4-bit cache may be off by, beside their relative rounding (2^-11, counted in
    latent_attend): the largest one is kept in fp16 as 2^7 at least, so the sum that divides them is 2^7 at least, and
    none is off by more than half of fp16's smallest step, 2^-25: 2^-32 of the sum, times the values (and 2^-7 of it
    again for the other roundings on the way)."""
    return 2.0 ** -32 * (1 + 2.0 ** -7) * rows[:, :rank].abs().sum(0)

@pytest.mark.parametrize("at", [5, 32760])
def test_fp4_small_probabilities_behind_a_dominant_row(at):
    """One row takes nearly all of the weight and is 0 in the columns looked at; the 2^15 others weigh 2^-X of it each.
    All requests name the same pages, one request a multiprocessor, so that no part has a maximum of its own.

    Looked at: the error that fp16_steps allows, which is small beside what the others weigh together."""
    n, width, rank, page, H = 1 << 15, 64, 64, 1024, 10
    g = torch.Generator().manual_seed(at)
    rows = torch.randn(n, width, generator=g).abs().to(BF)
    rows[:, 0] = 0.0
    rows[at] = 0.0
    rows[at, 0] = 6.0                                         # a scale of 1: exact
    q = torch.zeros(1, 1, H, width)
    q[0, 0, :, 0] = torch.tensor([0.0, 14, 18, 20, 22, 24, 24.5, 25, 25.5, 26]) / 6   # X, with logits in powers of two
    codes, scales, exact = quantise(rows)
    cache = torch.stack([pack_page(codes[i:i + page], scales[i:i + page]) for i in range(0, n, page)])
    B = torch.cuda.get_device_properties(0).multi_processor_count
    p = dict(q=q.to(BF).expand(B, 1, H, width).contiguous(), cache=cache, page=page, dt="fp4", lens=[n] * B,
             table=torch.arange(n // page, dtype=torch.int32).expand(B, -1).contiguous())
    scale = math.log(2)
    d = run_latent(p, rank, scale)
    assert d["status"] == s4r.S4R_OK
    exact = exact.to(DEV)
    out, lse, ob, lb = latent_attend(p["q"][0, 0].double().to(DEV), exact, n, rank, scale, HALF_STEP[torch.float16])
    ob = ob + fp16_steps(exact, rank)
    for b in (0, 1, B // 2, B - 1):
        assert_within(d["out"][b, 0], out, ob, f"request {b}")
        assert_within(d["lse"][b, 0], lse, lb, f"request {b}")


def test_fp4_growing_logits():
    """4-bit rows whose logits rise by far more than the reference is allowed to lag, so that it moves again and again."""
    lens, H, width, rank, page = [700, 2500], 40, 192, 128, 32
    p = latent_problem("fp4", lens, 1, H, width, page, seed=3)
    g = torch.Generator().manual_seed(4)
    for b, n in enumerate(lens):
        rows = (torch.randn(n, width, generator=g) * torch.linspace(0.1, 8, n)[:, None]).to(BF)
        codes, scales, p["rows"][b] = quantise(rows)
        for k in range(cdiv(n, page)):
            c, s = torch.zeros(page, width, dtype=torch.uint8), torch.zeros(page, width // 16, dtype=torch.uint8)
            m = min(page, n - k * page)
            c[:m], s[:m] = codes[k * page:k * page + m], scales[k * page:k * page + m]
            c[m:], s[m:] = 15, 0x7e                           # the largest values behind the length
            p["cache"][int(p["table"][b, k])] = pack_page(c, s)
    for scale in (1.0, -0.7):
        d = run_latent(p, rank, scale)
        assert d["status"] == s4r.S4R_OK
        for b, n in enumerate(lens):
            rows = p["rows"][b].to(DEV)
            out, lse, ob, lb = latent_attend(p["q"][b, 0].double().to(DEV), rows, n, rank, scale, HALF_STEP[torch.float16])
            assert_within(d["out"][b, 0], out, ob + fp16_steps(rows, rank), f"out of request {b}")
            assert_within(d["lse"][b, 0], lse, lb, f"lse of request {b}")


# ---------------------------------------------------------------- logits of minus infinity

@pytest.mark.parametrize("n", [2, 3, 5, 40, 3000, 30000])
def test_latent_keys_of_weight_zero_in_rows_computed_again(n):
    """Row 0 has a logit of minus infinity for every query, and so has the newest row, whose infinity lies beside value
    columns that only the last query may see: its rows are computed again one by one, and both rows weigh nothing."""
    H, width, rank = 5, 192, 160
    p = latent_problem("bf16", [n, 100], 2, H, width, 32, seed=n)
    p["q"][..., 170], p["q"][..., 180] = -0.5, 0.5
    flat = p["cache"].view(-1, width)
    for at, col, bad in ((0, 180, -math.inf), (n - 1, 170, math.inf)):
        flat[int(p["table"][0, at // 32]) * 32 + at % 32, col] = bad
    live = p["rows"][0][1:n - 1]
    d = run_latent(p, rank, 0.05)
    assert d["status"] == s4r.S4R_OK
    for t in range(2):        # both queries see rows 1 .. n - 2, and rows that weigh nothing
        out, lse, ob, lb = latent_attend(p["q"][0, t].double(), live, n - 2, rank, 0.05, HALF_STEP[BF])
        assert_within(d["out"][0, t].cpu(), out, ob, f"out of token {t}")
        assert_within(d["lse"][0, t].cpu(), lse, lb, f"lse of token {t}")
    for t in range(2):
        out, lse, ob, lb = latent_attend(p["q"][1, t].double(), p["rows"][1], 99 + t, rank, 0.05, HALF_STEP[BF])
        assert_within(d["out"][1, t].cpu(), out, ob, "the other request")


@pytest.mark.parametrize("n", [1, 2, 40])
def test_latent_rows_without_any_weight(n):
    """Every row has an infinity, so that no logit of the even heads is above minus infinity: they get 0 and minus infinity,
    infinite values or not.  The odd heads' logits are NaN or infinite, and so are they; the other request stays exact."""
    H, width = 6, 64
    p = latent_problem("bf16", [n, 90], 1, H, width, 16, seed=n)
    p["q"][0, 0, 0::2, 11], p["q"][0, 0, 1::2, 11] = -0.5, 0.5
    flat = p["cache"].view(-1, width)
    for at in range(n):
        flat[int(p["table"][0, at // 16]) * 16 + at % 16, 11] = math.inf
    d = run_latent(p, width, 0.2)
    assert d["status"] == s4r.S4R_OK
    assert (d["out"][0, 0, 0::2] == 0).all() and (d["lse"][0, 0, 0::2] == -math.inf).all()
    assert torch.isnan(d["out"][0, 0, 1::2]).all()
    out, lse, ob, lb = latent_attend(p["q"][1, 0].double(), p["rows"][1], 90, width, 0.2, HALF_STEP[BF])
    assert_within(d["out"][1, 0].cpu(), out, ob)


@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("n", [40, 300])
def test_prefill_keys_of_weight_zero_in_rows_computed_again(n, rope):
    """Key 0 has a logit of minus infinity for every query; a value on the diagonal is infinite, so the queries that see
    it are computed again one by one.  Only the column of the infinity is infinite."""
    p = prefill_problem([n, 70], [n, 70], 4, 2, 64, rope, 64, seed=n + rope)
    p["q"][..., 9] = 0.5
    p["k"][0, :, 9] = -math.inf
    late = n - 7
    p["v"][late, :, 3] = math.inf
    d = run_prefill(p, 0.1)
    assert s4r.s4r_read_device_status(None) == s4r.S4R_OK
    assert (d["out"][0] == 0).all() and (d["lse"][0] == -math.inf).all()        # sees key 0 only
    clean = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    clean["k"][0], clean["v"][late, :, 3] = 0.0, 0.0
    clean["q"] = clean["q"][1:]                                                  # queries 1 .. with keys 1 ..
    clean["k"], clean["v"] = clean["k"][1:], clean["v"][1:]
    if rope:
        clean["k_rope"] = clean["k_rope"][1:]
    clean["cu_q"] = clean["cu_k"] = [0, n - 1, n + 69]
    got = dict(out=d["out"][1:].clone(), lse=d["lse"][1:])
    assert (got["out"][late - 1:n - 1, :, 3] == math.inf).all()
    got["out"][late - 1:n - 1, :, 3] = 0.0
    # the column of the infinity: compared where no query sees it
    keep = got["out"].clone()
    want = run_prefill(clean, 0.1)
    got["out"][late - 1:n - 1, :, 3] = want["out"][late - 1:n - 1, :, 3]
    check_prefill(clean, got, 0.1)
    assert torch.isfinite(keep).all()


# ---------------------------------------------------------------- page plan

def test_page_plan_demand_beyond_32_bits():
    """17 requests ask for 2^27 - 1 pages each; behind them one page is not there either, though the sum of the pages
    no longer fits 31 bits.  A request that opens no page is served all the same."""
    page, cols = 16, 2 ** 27 - 1
    B = 19
    old, new = [0] * B, [page * cols] * 17 + [5, 3]
    old[18] = 1
    table = torch.empty(B, cols, dtype=torch.int32, device=DEV)
    table[18, 0] = 6
    lengths, free = i32(old), i32([3])
    cu, slots, w = i32([0] * (B + 1)), torch.zeros(20, dtype=torch.int64, device=DEV), status_words()
    s4r.s4r_page_plan(lengths=lengths, new_tokens=i32(new), block_table=table, free_pages=i32([7, 8, 9]), free_count=free,
                      lengths_out=lengths, free_count_out=free, cu_tokens=cu, slots=slots, page_size=page, status_workspace=w)
    assert s4r.s4r_read_device_status(w) == s4r.S4R_ERR_DEVICE
    assert lengths.tolist() == [0] * 18 + [4] and int(free) == 3
    assert (slots == -1).all()


# ---------------------------------------------------------------- waits that give up

@pytest.fixture
def waits():
    yield s4r.s4r_debug_waits
    torch.cuda.synchronize()
    s4r.s4r_debug_waits(0, False)
    s4r.s4r_clear_device_status(None)


@pytest.mark.parametrize("limit,unreachable", [(2_000_000, True), (1, True), (1, False), (2000, False)])
@pytest.mark.parametrize("dt", ["bf16", "fp4"])
@pytest.mark.parametrize("lens,T,H", [([5000, 20, 0, 300], 1, 20), ([9000, 70] + [1] * 400, 2, 64)])
def test_latent_attend_waits_that_give_up(waits, lens, T, H, dt, limit, unreachable):
    """The call ends and reports it, on a workspace that held another call's sums; the next call is right again."""
    p = latent_problem(dt, lens, T, H, 192, 32, seed=len(lens))
    good = run_latent(p, 160, 0.1)
    check_latent(p, good, 160, 0.1)
    g = torch.Generator(device=DEV).manual_seed(1)
    ws = good["ws"].view(torch.int32)
    for fill in ("sums", "whole numbers"):
        ws[64:] = (torch.randn(ws.numel() - 64, generator=g, device=DEV).view(torch.int32) if fill == "sums" else
                   torch.randint(-2 ** 31, 2 ** 31, (ws.numel() - 64,), generator=g, device=DEV).int())
        waits(limit, unreachable)
        s4r.s4r_latent_attend(good["args"])
        status = s4r.s4r_read_device_status(good["ws"])
        waits(0, False)
        assert status == s4r.S4R_ERR_TIMEOUT or (status == s4r.S4R_OK and not unreachable)
        s4r.s4r_clear_device_status(good["ws"])
        s4r.s4r_latent_attend(good["args"])
        assert s4r.s4r_read_device_status(good["ws"]) == s4r.S4R_OK
        check_latent(p, good, 160, 0.1)


@pytest.mark.parametrize("limit,unreachable", [(2_000_000, True), (1, True), (1, False), (2000, False)])
@pytest.mark.parametrize("dim,rope,vdim", [(128, 64, 128), (64, 0, 64), (128, 0, 128), (64, 0, 128)])
def test_prefill_waits_that_give_up(waits, dim, rope, vdim, limit, unreachable):
    p = prefill_problem([700, 40, 1], [900, 40, 3000], 4, 2, dim, rope, vdim, seed=dim + rope + vdim)
    good = run_prefill(p, 0.1)
    check_prefill(p, good, 0.1)
    waits(limit, unreachable)
    s4r.s4r_prefill_attend(good["args"])
    status = s4r.s4r_read_device_status(None)
    waits(0, False)
    assert status == s4r.S4R_ERR_TIMEOUT or (status == s4r.S4R_OK and not unreachable)
    s4r.s4r_clear_device_status(None)
    s4r.s4r_prefill_attend(good["args"])
    assert s4r.s4r_read_device_status(None) == s4r.S4R_OK
    check_prefill(p, good, 0.1)


@pytest.mark.parametrize("limit,unreachable", [(2_000_000, True), (1, True), (1, False), (2000, False)])
@pytest.mark.parametrize("n,H,dim,rank,to_latent", [(1, 2, 64, 128, True), (3000, 24, 128, 512, False), (700, 100, 64, 256, True)])
def test_project_waits_that_give_up(waits, n, H, dim, rank, to_latent, limit, unreachable):
    g = torch.Generator().manual_seed(n)
    n_in, n_out = (dim, rank) if to_latent else (rank, dim)
    x = torch.randn(n, H, n_in, generator=g).to(BF)
    basis = (torch.randn(H * dim, rank, generator=g) / math.sqrt(n_in)).to(BF)
    xd, bd, out = x.to(DEV), basis.to(DEV), torch.empty(n, H, n_out, dtype=BF, device=DEV)
    waits(limit, unreachable)
    s4r.s4r_latent_project(xd, bd, out, to_latent=to_latent)
    status = s4r.s4r_read_device_status(None)
    waits(0, False)
    assert status == s4r.S4R_ERR_TIMEOUT or (status == s4r.S4R_OK and not unreachable)
    s4r.s4r_clear_device_status(None)
    s4r.s4r_latent_project(xd, bd, out, to_latent=to_latent)
    assert s4r.s4r_read_device_status(None) == s4r.S4R_OK
    check_project(x, basis, out, H, dim, rank, to_latent)


# ---------------------------------------------------------------- every kernel instance

def project_width(n, H, dim, rank, to_latent, shared, sms=148):
    """Columns a tile that the projection's rule chooses: rounds of the grid times (column groups a tile + 1)."""
    out = rank if to_latent else dim
    groups, cost = cdiv(out, 64), {}
    for width in (256, 128, 64):
        k = width // 64
        tiles = cdiv(H * groups, k) if shared else H * cdiv(groups, k)
        cost[width] = cdiv(tiles * cdiv(n, 128), sms) * (min(k, H * groups if shared else groups) + 1)
    return min(cost, key=lambda w: (cost[w], -w))


@pytest.mark.parametrize("n,H,dim,rank,to_latent,shared,width", [
    (64, 128, 128, 512, True, False, 256), (64, 128, 128, 512, False, False, 256), (64, 128, 96, 512, True, False, 256),
    (64, 128, 96, 512, False, False, 256), (3001, 32, 128, 512, False, True, 256), (3001, 32, 96, 512, False, True, 256),
    (1500, 33, 256, 136, False, False, 256), (200, 100, 128, 448, True, True, 256), (1500, 33, 72, 136, False, True, 128),
    (2500, 5, 96, 320, False, True, 128), (2000, 12, 128, 320, True, False, 128), (100, 74, 256, 512, False, False, 128)])
def test_project_tiles_of_several_column_groups(n, H, dim, rank, to_latent, shared, width):
    assert project_width(n, H, dim, rank, to_latent, shared) == width      # on a GPU of 148 multiprocessors
    g = torch.Generator().manual_seed(n + dim)
    n_in, n_out = (dim, rank) if to_latent else (rank, dim)
    x = torch.randn(*((n, n_in) if shared else (n, H, n_in)), generator=g).to(BF)
    basis = (torch.randn(H * dim, rank, generator=g) / math.sqrt(n_in)).to(BF)
    wide = torch.full((n + 2, H, n_out + 16), 5.0, dtype=BF, device=DEV)
    out = wide[1:n + 1, :, 8:8 + n_out]
    s4r.s4r_latent_project(x.to(DEV), basis.to(DEV), out, to_latent=to_latent)
    check_project(x, basis, out, H, dim, rank, to_latent)
    assert (wide[0] == 5).all() and (wide[-1] == 5).all() and (wide[..., :8] == 5).all() and (wide[..., 8 + n_out:] == 5).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,vdim", [(64, 128), (40, 72), (8, 96)])
def test_prefill_wide_values_beside_short_keys(dim, vdim, causal):
    p = prefill_problem([1, 5, 0, 130, 257, 64], [1, 5, 3, 130, 1100, 65], 6, 2, dim, 0, vdim, seed=dim + vdim, pad=3)
    d = run_prefill(p, 1.5 / math.sqrt(dim), causal)
    check_prefill(p, d, 1.5 / math.sqrt(dim), causal)
    assert (d["out"][-3:] == 77).all() and (d["lse"][-3:] == 77).all()
    assert s4r.s4r_read_device_status(None) == s4r.S4R_OK


# ---------------------------------------------------------------- 4-bit rows

@pytest.mark.parametrize("change", ["page", "negative page", "length", "negative length"])
def test_fp4_other_requests_beside_a_bad_one(change):
    """The requests beside one with a bad length or page keep fp16's precision."""
    p = latent_problem("fp4", [100, 50, 20, 64], 1, 4, 64, 16, seed=10)
    q = dict(p, table=p["table"].clone(), lens=list(p["lens"]))
    if change == "page":
        q["table"][1, 2] = p["cache"].shape[0]
    elif change == "negative page":
        q["table"][1, 0] = -1
    else:
        q["lens"][1] = 16 * p["table"].shape[1] + 1 if change == "length" else -3
    d = run_latent(q, 64, 0.2)
    assert d["status"] == s4r.S4R_ERR_DEVICE
    for b in (0, 2, 3):
        out, lse, ob, lb = latent_attend(p["q"][b, 0].double(), p["rows"][b], p["lens"][b], 64, 0.2, HALF_STEP[torch.float16])
        assert_within(d["out"][b, 0].cpu(), out, ob, f"request {b}")
        assert_within(d["lse"][b, 0].cpu(), lse, lb, f"request {b}")


@pytest.mark.parametrize("H", [5, 40])
@pytest.mark.parametrize("n", [3, 64, 65, 20033])
def test_fp4_rows_without_a_value_that_only_later_queries_see(n, H):
    """The newest row has a group whose scale is NaN: queries that do not see it stay exact, the last one gets NaN."""
    width, rank, page = 192, 160, 32
    p = latent_problem("fp4", [n, 100], 3, H, width, page, seed=n)
    at = n - 1
    p["cache"][int(p["table"][0, at // page]), page * width // 2 + (at % page) * (width // 16) + 4] = 0x7f
    d = run_latent(p, rank, 0.05)
    assert d["status"] == s4r.S4R_OK
    assert torch.isnan(d["out"][0, 2]).all() and torch.isnan(d["lse"][0, 2]).all()
    for b, t, sees in ((0, 0, n - 2), (0, 1, n - 1), (1, 0, 98), (1, 1, 99), (1, 2, 100)):
        out, lse, ob, lb = latent_attend(p["q"][b, t].double(), p["rows"][b], sees, rank, 0.05, HALF_STEP[torch.float16])
        assert_within(d["out"][b, t].cpu(), out, ob, f"request {b} token {t}")
        assert_within(d["lse"][b, t].cpu(), lse, lb, f"request {b} token {t}")


# ---------------------------------------------------------------- a captured step

@pytest.mark.parametrize("dt", ["bf16", "fp4"])
@pytest.mark.parametrize("B,T", [(5, 1), (1100, 1), (40, 3)])
def test_captured_decode_steps(B, T, dt):
    """Plan, write, absorb, attend and expand captured as one graph and replayed step by step: each step equals the same
    calls made one by one, and the last one 64-bit attention over the rows written."""
    H, dim, rope, rank, page, steps = 6, 64, 32, 160, 16, 4
    width, n = rank + rope, B * T
    g = torch.Generator().manual_seed(B + T)
    bk = (torch.randn(H * dim, rank, generator=g) / 8).to(BF).to(DEV)
    old = torch.randint(0, 90, (B,), generator=g).int()
    cols = cdiv(90 + steps * T, page)
    pages = B * cols
    pool = torch.randperm(pages, generator=g).int()
    new_rows = torch.randn(steps, n, width, generator=g).to(BF)
    new_q = torch.randn(steps, n, H, dim + rope, generator=g).to(BF)
    first = torch.randn(pages * page, width, generator=g).to(BF)

    def state():
        table = torch.full((B, cols), -1, dtype=torch.int32)
        have = [cdiv(int(x), page) for x in old]
        at = pages
        for b in range(B):
            table[b, :have[b]] = pool[at - have[b]:at]
            at -= have[b]
        cache = (torch.zeros(pages, page, width, dtype=BF, device=DEV) if dt == "bf16"
                 else torch.zeros(pages, page * width * 9 // 16, dtype=torch.uint8, device=DEV))
        s4r.s4r_latent_write(latents=first.to(DEV), slots=torch.arange(pages * page, device=DEV), cache=cache, page_size=page)
        s = dict(table=table.to(DEV), cache=cache, pool=pool.to(DEV), free=i32([at]), held=old.to(DEV), new=i32([T] * B),
                 cu=i32([0] * (B + 1)), slots=torch.zeros(n, dtype=torch.int64, device=DEV), rows=new_rows[0].to(DEV),
                 q=new_q[0].to(DEV), ql=torch.zeros(B, T, H, width, dtype=BF, device=DEV), w=status_words(),
                 ol=torch.zeros(B, T, H, rank, dtype=BF, device=DEV), out=torch.zeros(n, H, dim, dtype=BF, device=DEV))
        args = dict(q=s["ql"], cache=cache, block_table=s["table"], lengths=s["held"], out=s["ol"], page_size=page, scale=0.1)
        s["ws"] = torch.empty(s4r.s4r_latent_attend_workspace_bytes(s4r.latent_attend_args(**args)), dtype=torch.uint8, device=DEV)
        s4r.s4r_workspace_init(s["ws"])
        s["args"] = s4r.latent_attend_args(**args, workspace=s["ws"])
        return s

    def step(s, wait=lambda: None):
        s4r.s4r_page_plan(lengths=s["held"], new_tokens=s["new"], block_table=s["table"], free_pages=s["pool"],
                          free_count=s["free"], lengths_out=s["held"], free_count_out=s["free"], cu_tokens=s["cu"],
                          slots=s["slots"], page_size=page, status_workspace=s["w"])
        wait()
        s4r.s4r_latent_write(latents=s["rows"], slots=s["slots"], cache=s["cache"], page_size=page, status_workspace=s["w"])
        wait()
        ql = s["ql"].view(n, H, width)
        ql[..., rank:] = s["q"][..., dim:]
        s4r.s4r_latent_project(s["q"][..., :dim], bk, ql[..., :rank], to_latent=True)
        wait()
        s4r.s4r_latent_attend(s["args"])
        wait()
        s4r.s4r_latent_project(s["ol"].view(n, H, rank), bk, s["out"], to_latent=False)
        wait()

    a, b = state(), state()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(a)
    for k in range(steps):
        for s in (a, b):
            s["rows"].copy_(new_rows[k])
            s["q"].copy_(new_q[k])
        graph.replay()
        step(b, torch.cuda.synchronize)
        torch.cuda.synchronize()
        for key in ("table", "free", "held", "cu", "slots", "cache", "ql", "ol", "out"):
            assert torch.equal(a[key], b[key]), (k, key)
    for s in (a, b):
        assert s4r.s4r_read_device_status(s["w"]) == s4r.S4R_OK and s4r.s4r_read_device_status(s["ws"]) == s4r.S4R_OK
    exact = (first if dt == "bf16" else quantise(first)[2]).double()
    fresh = [(new_rows[k] if dt == "bf16" else quantise(new_rows[k])[2]).double() for k in range(steps)]
    table, half = a["table"].cpu().long(), HALF_STEP[BF if dt == "bf16" else torch.float16]
    for r in range(0, B, max(1, B // 20)):
        pos = torch.arange(int(old[r]))
        rows = torch.cat([exact[table[r, pos // page] * page + pos % page]] + [f[r * T:(r + 1) * T] for f in fresh]).to(DEV)
        for t in range(T):
            out, _, ob, _ = latent_attend(a["ql"][r, t].double(), rows, len(rows) - T + 1 + t, rank, 0.1, half)
            assert_within(a["ol"][r, t], out, ob, f"request {r} token {t}")


def test_prefill_reports_rows_that_a_limit_of_zero_leaves_out():
    p = prefill_problem([3, 0], [3, 4], 2, 1, 64, 0, 64, seed=1)
    d = run_prefill(p, 0.1, max_q=0)
    assert s4r.s4r_read_device_status(None) == s4r.S4R_ERR_DEVICE
    s4r.s4r_clear_device_status(None)
    assert (d["out"] == 77).all() and (d["lse"] == 77).all()
    p = prefill_problem([0, 0], [5, 0], 2, 1, 64, 0, 64, seed=1, pad=4)         # rows, but none of a sequence
    d = run_prefill(p, 0.1, max_q=0)
    assert s4r.s4r_read_device_status(None) == s4r.S4R_OK
    assert (d["out"] == 77).all() and (d["lse"] == 77).all()


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
@pytest.mark.parametrize("case", ["a part of nothing else", "a part that weighs nothing"])
def test_latent_nan_logits_reach_the_joined_result(case, dt):
    """Logits of NaN make a query's result NaN, wherever the request is cut: also where one CTA saw nothing else, and
    where all else that it saw weighs nothing beside another part's."""
    n, H, width, page = 30000, 5, 64, 64
    p = latent_problem(dt, [n, 100], 1, H, width, page, seed=7)
    if case == "a part that weighs nothing":            # 256 above the others
        p["q"][0, 0, :, 16:32], p["q"][0, 0, :, 40] = 0.0, 0.0
        p["q"][0, 0, :, 16] = 8.0
        top, bad = torch.zeros(1, width), [20000]
        top[0, 16] = 6.0 * 16
        codes, scales, _ = quantise(top.to(BF))
        at = 100
        if dt == "bf16":
            p["cache"][int(p["table"][0, at // page]), at % page] = top[0].to(BF)
        else:
            pg = p["cache"][int(p["table"][0, at // page])]
            pg[at % page * (width // 2):(at % page + 1) * (width // 2)] = codes[0, 0::2] | (codes[0, 1::2] << 4)
            first = page * width // 2 + at % page * (width // 16)
            pg[first:first + width // 16] = scales[0]
    else:
        bad = range(12032, 12288)         # on 148 multiprocessors: the four tiles of one CTA
    for at in bad:
        pg = p["cache"][int(p["table"][0, at // page])]
        if dt == "bf16":
            pg[at % page, 35] = math.nan
        else:
            pg[page * width // 2 + at % page * (width // 16) + 2] = 0x7f
    d = run_latent(p, width, 0.35)
    assert d["status"] == s4r.S4R_OK
    assert torch.isnan(d["out"][0]).all() and torch.isnan(d["lse"][0]).all()
    step = HALF_STEP[BF if dt == "bf16" else torch.float16]
    out, lse, ob, lb = latent_attend(p["q"][1, 0].double(), p["rows"][1], 100, width, 0.35, step)
    assert_within(d["out"][1, 0].cpu(), out, ob)
    assert_within(d["lse"][1, 0].cpu(), lse, lb)


@pytest.mark.parametrize("n,at", [(30000, 20000), (30000, 29990), (200, 150)])
def test_latent_infinite_values_of_weight_zero(n, at):
    """A row whose infinity makes its logit minus infinity has weight 0: its column is 0 times infinity, the others are
    exact, also where the rest of its part weighs nothing beside another part's."""
    H, width, page = 5, 64, 64
    p = latent_problem("bf16", [n, 100], 1, H, width, page, seed=8)
    p["q"][0, 0, :, 16], p["q"][0, 0, :, 35] = 8.0, -0.5
    flat = p["cache"].view(-1, width)
    row = lambda i: int(p["table"][0, i // page]) * page + i % page  # noqa: E731
    flat[row(100)] = 0.0
    flat[row(100), 16] = 96.0
    flat[row(at), 35] = math.inf
    rows = p["rows"][0].clone()
    rows[100] = flat[row(100)].double()
    live = torch.cat([rows[:at], rows[at + 1:]])
    d = run_latent(p, width, 0.35)
    assert d["status"] == s4r.S4R_OK
    assert torch.isnan(d["out"][0, 0, :, 35]).all()
    out, lse, ob, lb = latent_attend(p["q"][0, 0].double(), live, n - 1, width, 0.35, HALF_STEP[BF])
    keep = [c for c in range(width) if c != 35]
    assert_within(d["out"][0, 0][:, keep].cpu(), out[:, keep], ob[:, keep])
    assert_within(d["lse"][0, 0].cpu(), lse, lb)
