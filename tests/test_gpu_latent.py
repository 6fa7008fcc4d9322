"""Paged latent cache, latent attention, per-head projection and prefill attention against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import rank_decode_attention_b200 as s4r
from latent_reference import assert_within, attend, cdiv, latent_attend, pack_page, plan, quantise

pytestmark = pytest.mark.gpu
BF, DEV = torch.bfloat16, "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def status_words():
    w = torch.empty(256, dtype=torch.uint8, device=DEV)
    s4r.s4r_workspace_init(w)
    return w


# ---------------------------------------------------------------- page plan

def plan_state(B, page, low, high, new_low, new_high, spare, seed, extra_cols=0, pad=7):
    rng = np.random.default_rng(seed)
    old, new = rng.integers(low, high + 1, B), rng.integers(new_low, new_high + 1, B)
    have, full = -(-old // page), -(-(old + new) // page)
    width = int(full.max(initial=0)) + extra_cols or 1
    free = max(0, int((full - have).sum()) + spare)
    ids = rng.permutation(int(have.sum()) + free + 3)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    return dict(old=old, new=new, table=table, free_pages=ids[at:at + free], free=free, page=page,
                max_tokens=int(new.sum()) + pad)


def run_plan(st, in_place=False, optional=True, max_tokens=None):
    n = st["max_tokens"] if max_tokens is None else max_tokens
    d = dict(lengths=i32(st["old"]), new_tokens=i32(st["new"]), block_table=i32(st["table"]),
             free_pages=i32(st["free_pages"]), free_count=i32([st["free"]]))
    d["lengths_out"] = d["lengths"] if in_place else torch.full_like(d["lengths"], -9)
    d["free_count_out"] = d["free_count"] if in_place else i32([-9])
    d["cu_tokens"] = i32([-9] * (len(st["old"]) + 1))
    d["slots"] = torch.full((n,), -9, dtype=torch.int64, device=DEV)
    if optional:
        d["positions"], d["requests"] = i32([-9] * n), i32([-9] * n)
    w = status_words()
    s4r.s4r_page_plan(**d, page_size=st["page"], status_workspace=w)
    return d, s4r.s4r_read_device_status(w)


def check_plan(st, d, status, max_tokens=None):
    want = plan(st["old"], st["new"], st["table"], st["free_pages"], st["free"], st["page"],
                st["max_tokens"] if max_tokens is None else max_tokens)
    for key, got in (("table", "block_table"), ("lengths", "lengths_out"), ("cu", "cu_tokens"), ("slots", "slots"),
                     ("positions", "positions"), ("requests", "requests")):
        if got in d:
            np.testing.assert_array_equal(d[got].cpu().numpy(), want[key], err_msg=key)
    assert int(d["free_count_out"]) == want["free"]
    assert status == (s4r.S4R_OK if want["ok"] else s4r.S4R_ERR_DEVICE)
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,low,high,new_low,new_high,spare", [
    (1, 16, 0, 0, 1, 1, 0), (1, 64, 100, 100, 0, 0, 0), (3, 16, 0, 40, 0, 40, 5), (256, 64, 1, 8000, 1, 1, 100),
    (1001, 16, 0, 500, 0, 60, -400), (8192, 128, 0, 300, 0, 2, 3), (7, 1024, 0, 9000, 0, 7000, 0),
    (1, 32, 12345, 12345, 200001, 200001, 1), (1500, 16, 0, 16, 0, 17, 0)])
def test_page_plan(B, page, low, high, new_low, new_high, spare, in_place):
    st = plan_state(B, page, low, high, new_low, new_high, spare, seed=B + page, extra_cols=B % 3)
    check_plan(st, *run_plan(st, in_place))


@pytest.mark.parametrize("tokens", [50, 6000])
def test_page_plan_refuses_requests_one_by_one(tokens):
    st = plan_state(40, 16, 0, 100, 0, 2 * tokens // 40, -3, seed=4)
    st["new"][3], st["new"][4], st["old"][7] = -5, 16 * st["table"].shape[1] + 1, -1
    d, status = run_plan(st, max_tokens=9000)
    check_plan(st, d, status, 9000)
    assert status == s4r.S4R_ERR_DEVICE


def test_page_plan_too_few_token_entries_and_a_bad_free_count():
    st = plan_state(9, 16, 0, 100, 5, 40, 3, seed=5)
    check_plan(st, *run_plan(st, max_tokens=31), 31)
    check_plan(st, *run_plan(st, optional=False, max_tokens=0), 0)
    st["free"] = len(st["free_pages"]) + 2
    check_plan(st, *run_plan(st))
    st["free"] = -1
    check_plan(st, *run_plan(st))


def test_page_plan_without_requests():
    st = dict(old=np.zeros(0, dtype=int), new=np.zeros(0, dtype=int), table=np.zeros((0, 3), dtype=int), page=16,
              free_pages=np.array([4, 5]), free=2, max_tokens=5)
    for n in (5, 0, 9000):
        check_plan(st, *run_plan(st, max_tokens=n), n)


def test_page_plan_sums_beyond_32_bits():
    st = dict(old=np.array([5, 2 ** 31 - 1, 0]), new=np.array([3, 2 ** 31 - 1, 4]), table=np.full((3, 2), -1), page=16,
              free_pages=np.array([8, 9]), free=2, max_tokens=20)
    st["table"][0, 0] = 1
    d, status = run_plan(st)
    assert status == s4r.S4R_ERR_DEVICE
    assert d["slots"].tolist() == [21, 22, 23] + [-1] * 17 and d["lengths_out"].tolist() == [8, 2 ** 31 - 1, 4]
    assert d["cu_tokens"].tolist() == [0, 3, 2 ** 31 - 1, 2 ** 31 - 1] and int(d["free_count_out"]) == 1


def test_page_plan_captured_steps():
    """A serving loop: one captured call, lengths and free count updated in place, replayed."""
    st = plan_state(33, 16, 0, 40, 1, 1, 200, seed=6, extra_cols=6, pad=0)
    d = dict(lengths=i32(st["old"]), new_tokens=i32(st["new"]), block_table=i32(st["table"]),
             free_pages=i32(st["free_pages"]), free_count=i32([st["free"]]), cu_tokens=i32([0] * 34),
             slots=torch.zeros(33, dtype=torch.int64, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s4r.s4r_page_plan(**d, lengths_out=d["lengths"], free_count_out=d["free_count"], page_size=16)
    for _ in range(20):
        want = plan(st["old"], st["new"], st["table"], st["free_pages"], st["free"], 16, 33)
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(d["slots"].cpu().numpy(), want["slots"])
        np.testing.assert_array_equal(d["block_table"].cpu().numpy(), want["table"])
        assert int(d["free_count"]) == want["free"]
        st["old"], st["table"], st["free"] = want["lengths"], want["table"], want["free"]


# ---------------------------------------------------------------- latent write

@pytest.mark.parametrize("n,width,page,ld", [(1, 8, 16, 8), (5, 576, 64, 576), (130, 200, 32, 208), (3000, 320, 1024, 640)])
def test_write_bf16(n, width, page, ld):
    g = torch.Generator().manual_seed(n)
    src = torch.randn(n, ld, generator=g).to(BF)
    pages = cdiv(n, page) + 2
    slots = torch.randperm(pages * page, generator=g)[:n]
    if n > 1:
        slots[n // 2], slots[0] = -1, -2 ** 40
    cache = torch.full((pages, page, width), 7.0, dtype=BF)
    want = cache.clone().view(-1, width)
    for t in range(n):
        if slots[t] >= 0:
            want[slots[t]] = src[t, :width]
    got = cache.to(DEV)
    s4r.s4r_latent_write(latents=src.to(DEV)[:, :width], slots=slots.to(DEV), cache=got, page_size=page)
    assert torch.equal(got.cpu().view(-1, width), want)


@pytest.mark.parametrize("n,width,page,cache_scale", [(1, 32, 16, 1.0), (77, 576, 16, 1.0), (300, 224, 64, 0.3),
                                                      (2000, 64, 1024, 4.0)])
def test_write_fp4_is_the_definition_bit_by_bit(n, width, page, cache_scale):
    g = torch.Generator().manual_seed(n)
    src = (torch.randn(n, width, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))).to(BF)
    src[0, :16] = 0.0
    if n > 20:
        src[1, :16] = torch.linspace(-6, 6, 16).to(BF)                    # ties of the 4-bit grid, scale 1
        src[2, 0], src[2, 17], src[3, 5], src[4, :16] = math.inf, -math.inf, math.nan, math.nan
        src[5, :16] = 2.0 ** -30                                          # a scale that rounds to zero
        src[6, :16] = 3e38
        src[7, :16] = torch.tensor([0.25, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.75, -5, 6, -0.0, 0.1, -0.1, 4.9, 5.1])
    pages = cdiv(n, page) + 1
    slots = torch.randperm(pages * page, generator=g)[:n]
    if n > 1:
        slots[n // 2] = -1
    codes, scales, values = quantise(src, cache_scale)
    all_codes = torch.zeros(pages * page, width, dtype=torch.uint8)
    all_scales = torch.zeros(pages * page, width // 16, dtype=torch.uint8)
    for t in range(n):
        if slots[t] >= 0:
            all_codes[slots[t]], all_scales[slots[t]] = codes[t], scales[t]
    want = torch.stack([pack_page(all_codes[i * page:(i + 1) * page], all_scales[i * page:(i + 1) * page]) for i in range(pages)])
    got = torch.zeros(pages, page * width * 9 // 16, dtype=torch.uint8, device=DEV)
    stored = torch.zeros(n, width, dtype=BF, device=DEV)
    s4r.s4r_latent_write(latents=src.to(DEV), slots=slots.to(DEV), cache=got, page_size=page, cache_scale=cache_scale,
                         stored=stored)
    assert torch.equal(got.cpu(), want)
    # code * scale is exact in 6 bits; the product with cache_scale is one fp32 rounding before the bf16 one
    assert_within(stored.cpu(), values, values.abs() * (2.0 ** -8 + 2.0 ** -23 if math.log2(cache_scale) % 1 else 0.0), "stored")


def test_write_beyond_the_cache_is_skipped_and_reported():
    for dt in (BF, torch.uint8):
        shape = (3, 16, 64) if dt is BF else (3, 16 * 64 * 9 // 16)
        cache = torch.zeros(shape, dtype=dt, device=DEV)
        w = status_words()
        src = torch.ones(2, 64, dtype=BF, device=DEV)
        s4r.s4r_latent_write(latents=src, slots=torch.tensor([48, 2 ** 40], device=DEV), cache=cache, page_size=16,
                             status_workspace=w)
        assert s4r.s4r_read_device_status(w) == s4r.S4R_ERR_DEVICE
        assert not cache.any()


# ---------------------------------------------------------------- latent attention

def latent_problem(dt, lens, T, H, width, page, seed, spread=1.0, waste=2, shuffle=True):
    """A paged cache whose unseen rows hold NaN (bf16) or the largest values (4-bit), and the rows in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    B, cols = len(lens), max(1, max(cdiv(n, page) for n in lens)) + waste
    need = sum(cdiv(n, page) for n in lens)
    pages = need + 2
    order = torch.randperm(pages, generator=g) if shuffle else torch.arange(pages)
    table = torch.full((B, cols), -1, dtype=torch.int32)
    rows = (torch.randn(pages * page, width, generator=g) * spread).to(BF)
    if dt == "bf16":
        exact, unseen = rows.double(), math.nan
    else:
        codes, scales, exact = quantise(rows)
        unseen = 0x7e
    seen = torch.zeros(pages * page, dtype=torch.bool)
    at, per = 0, []
    for b, n in enumerate(lens):
        k = cdiv(n, page)
        table[b, :k] = order[at:at + k].int()
        idx = (order[at:at + k, None] * page + torch.arange(page)[None]).reshape(-1)[:n]
        seen[idx] = True
        per.append(exact[idx])
        at += k
    if dt == "bf16":
        rows[~seen] = math.nan
        cache = rows.view(pages, page, width)
    else:
        codes[~seen] = 15
        scales[~seen] = unseen
        cache = torch.stack([pack_page(codes[i * page:(i + 1) * page], scales[i * page:(i + 1) * page]) for i in range(pages)])
    q = torch.randn(B, T, H, width, generator=g).to(BF)
    return dict(q=q, cache=cache.contiguous(), table=table, lens=lens, rows=per, page=page, dt=dt)


def run_latent(p, rank, scale, lse=True, stream=None, workspace=None):
    B, T, H, width = p["q"].shape
    d = dict(q=p["q"].to(DEV), cache=p["cache"].to(DEV), block_table=p["table"].to(DEV), lengths=i32(p["lens"]),
             out=torch.full((B, T, H, rank), 77.0, dtype=BF, device=DEV),
             lse=torch.full((B, T, H), 77.0, device=DEV) if lse else None)
    a = s4r.latent_attend_args(**d, page_size=p["page"], scale=scale)
    ws = torch.empty(s4r.s4r_latent_attend_workspace_bytes(a), dtype=torch.uint8, device=DEV) if workspace is None else workspace
    s4r.s4r_workspace_init(ws)
    a = s4r.latent_attend_args(**d, page_size=p["page"], scale=scale, workspace=ws)
    s4r.s4r_latent_attend(a)
    d.update(args=a, ws=ws, status=s4r.s4r_read_device_status(ws))
    return d


def check_latent(p, d, rank, scale):
    T = p["q"].shape[1]
    step = 2.0 ** -8 if p["dt"] == "bf16" else 2.0 ** -11
    for b, n in enumerate(p["lens"]):
        rows = p["rows"][b].to(DEV)
        for t in range(T):
            out, lse, ob, lb = latent_attend(p["q"][b, t].double().to(DEV), rows, n - T + 1 + t, rank, scale, step)
            assert_within(d["out"][b, t], out, ob, f"out of request {b} token {t}")
            if d["lse"] is not None:
                assert_within(d["lse"][b, t], lse, lb, f"lse of request {b} token {t}")


SHAPES = [  # heads, queries, width, rank
    (16, 1, 576, 512), (64, 1, 576, 512), (128, 2, 576, 512), (20, 1, 224, 192), (1, 1, 64, 64), (3, 3, 320, 256),
    (130, 1, 192, 128), (33, 2, 512, 512), (8, 1, 96, 32), (5, 4, 544, 480), (7, 1, 160, 160)]


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
@pytest.mark.parametrize("H,T,width,rank", SHAPES)
def test_latent_attend_shapes(H, T, width, rank, dt):
    p = latent_problem(dt, [0, 1, 63, 64, 65, 200, 1031], T, H, width, [16, 32, 64, 128][H % 4], seed=H + width)
    d = run_latent(p, rank, 1.5 / math.sqrt(width))
    assert d["status"] == s4r.S4R_OK
    check_latent(p, d, rank, 1.5 / math.sqrt(width))


@pytest.mark.parametrize("width,rank", [(8, 8), (24, 16), (40, 40), (136, 8), (568, 504)])
def test_latent_attend_odd_widths(width, rank):
    p = latent_problem("bf16", [5, 77, 500], 2, 6, width, 16, seed=width)
    check_latent(p, run_latent(p, rank, 0.3), rank, 0.3)


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_latent_attend_pages(page, dt):
    p = latent_problem(dt, [page - 1, page, page + 1, 3 * page + 5], 1, 12, 160, page, seed=page)
    check_latent(p, run_latent(p, 128, 0.1, lse=False), 128, 0.1)


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
@pytest.mark.parametrize("lens", [[30000], [9000, 3, 0, 4097], [64 * 148 * 2] * 2, [130] * 300, [0], [0] * 200, [1] * 149])
def test_latent_attend_lengths(lens, dt):
    p = latent_problem(dt, lens, 1, 16, 320, 64, seed=len(lens))
    check_latent(p, run_latent(p, 256, 0.05), 256, 0.05)


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
def test_latent_attend_growing_logits(dt):
    """Logits that rise by far more than e^8 along the cache, so that the running maximum moves again and again."""
    p = latent_problem(dt, [700, 2500], 1, 40, 192, 32, seed=3)
    for b, n in enumerate(p["lens"]):
        pages = p["table"][b, :cdiv(n, 32)].long()
        if dt == "bf16":
            ramp = torch.linspace(0.1, 8, n)
            flat = p["cache"].view(-1, 192)
            idx = (pages[:, None] * 32 + torch.arange(32)[None]).reshape(-1)[:n]
            flat[idx] = (flat[idx].float() * ramp[:, None]).to(BF)
            p["rows"][b] = flat[idx].double()
    check_latent(p, run_latent(p, 128, 1.0), 128, 1.0)
    check_latent(p, run_latent(p, 128, -0.7), 128, -0.7)
    check_latent(p, run_latent(p, 128, 0.0), 128, 0.0)


def test_latent_attend_cache_scale():
    p = latent_problem("fp4", [100, 333], 1, 9, 96, 16, seed=8)
    d = dict(q=p["q"].to(DEV), cache=p["cache"].to(DEV), block_table=p["table"].to(DEV), lengths=i32(p["lens"]),
             out=torch.empty(2, 1, 9, 64, dtype=BF, device=DEV), lse=torch.empty(2, 1, 9, device=DEV))
    a = s4r.latent_attend_args(**d, page_size=16, scale=0.2, cache_scale=0.37)
    ws = torch.empty(s4r.s4r_latent_attend_workspace_bytes(a), dtype=torch.uint8, device=DEV)
    s4r.s4r_workspace_init(ws)
    s4r.s4r_latent_attend(s4r.latent_attend_args(**d, page_size=16, scale=0.2, cache_scale=0.37, workspace=ws))
    scale = float(np.float32(0.37))
    p["rows"] = [r * scale for r in p["rows"]]
    check_latent(p, d, 64, float(np.float32(0.2)))


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
def test_latent_attend_infinite_values_in_seen_rows(dt):
    """A query whose row overflows gets what the formula gives; the other requests stay exact."""
    if dt == "fp4":
        pytest.skip("a 4-bit row holds no infinities")
    p = latent_problem(dt, [90, 200], 1, 4, 64, 16, seed=9)
    flat = p["cache"].view(-1, 64)
    flat[int(p["table"][0, 0]) * 16 + 3, 5] = math.nan
    d = run_latent(p, 64, 0.2)
    assert torch.isnan(d["out"][0]).all()
    out, lse, ob, lb = latent_attend(p["q"][1, 0].double(), p["rows"][1], 200, 64, 0.2, 2.0 ** -8)
    assert_within(d["out"][1, 0].cpu(), out, ob)
    assert_within(d["lse"][1, 0].cpu(), lse, lb)


@pytest.mark.parametrize("H", [5, 40])
@pytest.mark.parametrize("n", [3, 64, 65, 66, 20000, 20033])
def test_latent_attend_infinities_that_only_later_queries_see(n, H):
    """The newest row holds an infinity and the one before it a NaN in a value column: the queries that do not see them
    stay exact."""
    p = latent_problem("bf16", [n, 100], 3, H, 192, 32, seed=n)
    flat = p["cache"].view(-1, 192)
    for back, bad in ((1, math.inf), (2, math.nan)):
        at = n - back
        flat[int(p["table"][0, at // 32]) * 32 + at % 32, 7 * back] = bad
    d = run_latent(p, 160, 0.05)
    assert d["status"] == s4r.S4R_OK
    out, lse, ob, lb = latent_attend(p["q"][0, 0].double(), p["rows"][0], n - 2, 160, 0.05, 2.0 ** -8)
    assert_within(d["out"][0, 0].cpu(), out, ob)
    assert_within(d["lse"][0, 0].cpu(), lse, lb)
    assert torch.isnan(d["out"][0, 1]).all() and torch.isnan(d["out"][0, 2]).all()
    for t in range(3):
        out, lse, ob, lb = latent_attend(p["q"][1, t].double(), p["rows"][1], 98 + t, 160, 0.05, 2.0 ** -8)
        assert_within(d["out"][1, t].cpu(), out, ob)


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
def test_latent_attend_many_query_tokens(dt):
    """More query tokens than a tile has rows, some of them with nothing to see, and values that only the later ones may
    see spread over several tiles and parts."""
    T, H = 150, 3
    p = latent_problem(dt, [140, 149, 400, 30000], T, H, 96, 16, seed=31)
    first = {}
    if dt == "bf16":
        flat = p["cache"].view(-1, 96)
        for b, at in ((2, 300), (3, 29900), (3, 29990)):
            flat[int(p["table"][b, at // 16]) * 16 + at % 16, 20] = math.inf
            first.setdefault(b, at)
    d = run_latent(p, 64, 0.1)
    assert d["status"] == s4r.S4R_OK
    step = 2.0 ** -8 if dt == "bf16" else 2.0 ** -11
    for b, n in enumerate(p["lens"]):
        rows = p["rows"][b].to(DEV)
        for t in list(range(0, T, 7)) + [T - 1]:
            sees = n - T + 1 + t
            if sees > first.get(b, n):
                assert not torch.isfinite(d["out"][b, t].float()).all(1).any()
                continue
            out, lse, ob, lb = latent_attend(p["q"][b, t].double().to(DEV), rows, sees, 64, 0.1, step)
            assert_within(d["out"][b, t], out, ob, f"request {b} token {t}")
            assert_within(d["lse"][b, t], lse, lb, f"request {b} token {t}")


def test_latent_attend_more_row_blocks_than_multiprocessors():
    p = latent_problem("bf16", [130, 64], 1, 9601, 64, 16, seed=32)
    d = run_latent(p, 40, 0.1)
    assert d["status"] == s4r.S4R_OK
    check_latent(p, d, 40, 0.1)


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
def test_cache_beyond_32_bit_offsets(dt):
    """Rows written to and read from pages behind 2^32 bytes (and 2^32 values in bf16)."""
    width, page = 576, 64
    pages = 120000 if dt == "bf16" else 210000
    shape, kind = ((pages, page, width), BF) if dt == "bf16" else ((pages, page * width * 9 // 16), torch.uint8)
    cache = torch.empty(shape, dtype=kind, device=DEV)
    g = torch.Generator().manual_seed(33)
    n = 200
    src = torch.randn(n, width, generator=g).to(BF)
    ids = [pages - 1, 3, pages - 7, pages // 2]
    slots = torch.tensor([ids[t // page] * page + t % page for t in range(n)], device=DEV)
    s4r.s4r_latent_write(latents=src.to(DEV), slots=slots, cache=cache, page_size=page)
    rows = src.double() if dt == "bf16" else quantise(src)[2]
    q = torch.randn(1, 1, 20, width, generator=g).to(BF)
    d = dict(q=q.to(DEV), cache=cache, block_table=i32([ids]), lengths=i32([n]), out=torch.empty(1, 1, 20, 512, dtype=BF, device=DEV),
             lse=torch.empty(1, 1, 20, device=DEV))
    a = s4r.latent_attend_args(**d, page_size=page, scale=0.05)
    ws = torch.empty(s4r.s4r_latent_attend_workspace_bytes(a), dtype=torch.uint8, device=DEV)
    s4r.s4r_workspace_init(ws)
    s4r.s4r_latent_attend(s4r.latent_attend_args(**d, page_size=page, scale=0.05, workspace=ws))
    assert s4r.s4r_read_device_status(ws) == s4r.S4R_OK
    check_latent(dict(q=q, rows=[rows], lens=[n], dt=dt), d, 512, 0.05)


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
def test_latent_attend_reports_bad_lengths_and_pages(dt):
    p = latent_problem(dt, [100, 50, 20, 64], 1, 4, 64, 16, seed=10)
    good = run_latent(p, 64, 0.2)
    assert good["status"] == s4r.S4R_OK
    for change in ("page", "negative page", "length", "negative length"):
        q = dict(p, table=p["table"].clone(), lens=list(p["lens"]))
        if change == "page":
            q["table"][1, 2] = p["cache"].shape[0]
        elif change == "negative page":
            q["table"][1, 0] = -1
        elif change == "length":
            q["lens"][1] = 16 * p["table"].shape[1] + 1
        else:
            q["lens"][1] = -3
        d = run_latent(q, 64, 0.2)
        assert d["status"] == s4r.S4R_ERR_DEVICE, change
        for b in (0, 2, 3):
            out, lse, ob, lb = latent_attend(p["q"][b, 0].double(), p["rows"][b], p["lens"][b], 64, 0.2, 2.0 ** -8)
            assert_within(d["out"][b, 0].cpu(), out, ob, change)


@pytest.mark.parametrize("dt", ["bf16", "fp4"])
def test_latent_attend_two_streams_capture_and_replay(dt):
    probs = [latent_problem(dt, [3000, 10], 1, 16, 320, 64, seed=s) for s in (11, 12)]
    first = [run_latent(p, 256, 0.06) for p in probs]
    want = [d["out"].clone() for d in first]
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s in zip(first, streams):
            s4r.s4r_latent_attend(d["args"], s)
    torch.cuda.synchronize()
    graphs = []
    for d, s in zip(first, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            s4r.s4r_latent_attend(d["args"])
        graphs.append(g)
        d["out"].zero_()
    # other lengths than at capture, then the old ones again
    keep = first[0]["lengths"].clone()
    first[0]["lengths"].copy_(i32([100, 3]))
    graphs[0].replay()
    torch.cuda.synchronize()
    short = dict(probs[0], lens=[100, 3], rows=[r[:n] for r, n in zip(probs[0]["rows"], (100, 3))])
    check_latent(short, first[0], 256, 0.06)
    first[0]["lengths"].copy_(keep)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for d, w in zip(first, want):
        assert torch.equal(d["out"], w)            # no order of arrival in any sum
        assert s4r.s4r_read_device_status(d["ws"]) == s4r.S4R_OK


# ---------------------------------------------------------------- projection

@pytest.mark.parametrize("to_latent", [True, False])
@pytest.mark.parametrize("n,H,dim,rank", [(1, 1, 8, 8), (1, 16, 128, 512), (3, 5, 96, 192), (64, 32, 128, 512),
                                          (129, 3, 64, 136), (1000, 4, 40, 320), (300, 2, 256, 64)])
def test_project(n, H, dim, rank, to_latent):
    g = torch.Generator().manual_seed(n + dim)
    n_in, n_out = (dim, rank) if to_latent else (rank, dim)
    x = torch.randn(n, H, n_in, generator=g).to(BF)
    basis = (torch.randn(H * dim, rank, generator=g) / math.sqrt(n_in)).to(BF)
    wide = torch.full((n, H, n_out + 16), 5.0, dtype=BF, device=DEV)
    out = wide[:, :, 8:8 + n_out]
    s4r.s4r_latent_project(x.to(DEV), basis.to(DEV), out, to_latent=to_latent)
    check_project(x, basis, out, H, dim, rank, to_latent)
    assert (wide[:, :, :8] == 5).all() and (wide[:, :, 8 + n_out:] == 5).all()


def check_project(x, basis, out, H, dim, rank, to_latent):
    """`n_in` products in fp32 with 2^-23 an addition, then one rounding to bf16."""
    b = basis.double().view(H, dim, rank)
    form = "nhd,hdr->nhr" if to_latent else "nhr,hdr->nhd"
    xd = x.double() if x.dim() == 3 else x.double()[:, None].expand(-1, H, -1)
    exact = torch.einsum(form, xd, b)
    acc = (x.shape[-1] + 2) * 2.0 ** -23 * torch.einsum(form, xd.abs(), b.abs())
    assert_within(out.cpu(), exact, 2.0 ** -8 * (exact.abs() + acc) + acc + 2.0 ** -133, "project")


@pytest.mark.parametrize("n", [1, 70, 515])
def test_project_views(n):
    """A slice of a wider query, one latent for all heads, heads outside tokens."""
    g = torch.Generator().manual_seed(n)
    H, dim, rank = 6, 64, 192
    basis = (torch.randn(H * dim, rank, generator=g) / 14).to(BF).to(DEV)
    q = torch.randn(n, H, dim + 64, generator=g).to(BF).to(DEV)
    latent = torch.zeros(n, H, rank + 64, dtype=BF, device=DEV)
    s4r.s4r_latent_project(q[..., :dim], basis, latent[..., :rank], to_latent=True)
    check_project(q[..., :dim].cpu(), basis.cpu(), latent[..., :rank], H, dim, rank, True)
    assert not latent[..., rank:].any()
    rows = torch.randn(n, rank + 64, generator=g).to(BF).to(DEV)
    out = torch.empty(n, H, dim, dtype=BF, device=DEV)
    s4r.s4r_latent_project(rows[:, :rank], basis, out, to_latent=False)
    check_project(rows[:, :rank].cpu(), basis.cpu(), out, H, dim, rank, False)
    heads_first = torch.randn(H, n, rank, generator=g).to(BF).to(DEV).transpose(0, 1)
    out = torch.empty(H, n, dim, dtype=BF, device=DEV).transpose(0, 1)
    s4r.s4r_latent_project(heads_first, basis, out, to_latent=False)
    check_project(heads_first.cpu(), basis.cpu(), out, H, dim, rank, False)


# ---------------------------------------------------------------- prefill attention

def prefill_problem(nq, nk, Hq, Hkv, dim, rope, vdim, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    cq, ck = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    tq, tk = int(cq[-1]) + pad, int(ck[-1]) + pad
    p = dict(q=torch.randn(tq, Hq, dim + rope, generator=g).to(BF), k=torch.randn(tk, Hkv, dim, generator=g).to(BF),
             v=torch.randn(tk, Hkv, vdim, generator=g).to(BF), k_rope=torch.randn(tk, rope, generator=g).to(BF) if rope else None,
             cu_q=cq, cu_k=ck)
    if pad:                                   # rows of no sequence
        for key in ("k", "v"):
            p[key][-pad:] = math.nan
    return p


def run_prefill(p, scale, causal=True, lse=True, max_q=None):
    tq, Hq, vdim = p["q"].shape[0], p["q"].shape[1], p["v"].shape[2]
    d = {k: (None if p[k] is None else p[k].to(DEV)) for k in ("q", "k", "v", "k_rope")}
    d.update(cu_q=i32(p["cu_q"]), cu_k=i32(p["cu_k"]), out=torch.full((tq, Hq, vdim), 77.0, dtype=BF, device=DEV),
             lse=torch.full((tq, Hq), 77.0, device=DEV) if lse else None)
    a = s4r.prefill_attend_args(**d, max_q=int(np.diff(p["cu_q"]).max()) if max_q is None else max_q, scale=scale, causal=causal)
    s4r.s4r_prefill_attend(a)
    d["args"] = a
    return d


def check_prefill(p, d, scale, causal=True, only=None):
    Hq, Hkv, dim = p["q"].shape[1], p["k"].shape[1], p["k"].shape[2]
    for b in range(len(p["cu_q"]) - 1):
        if only is not None and b not in only:
            continue
        q0, q1, k0, k1 = (int(x) for x in (p["cu_q"][b], p["cu_q"][b + 1], p["cu_k"][b], p["cu_k"][b + 1]))
        nq, nk = q1 - q0, k1 - k0
        if nq == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            q = p["q"][q0:q1, h].double().to(DEV)
            k, v = p["k"][k0:k1, g].double().to(DEV), p["v"][k0:k1, g].double().to(DEV)
            if p["k_rope"] is not None:
                k = torch.cat([k, p["k_rope"][k0:k1].double().to(DEV)], 1)
            sees = torch.arange(nq, device=DEV) + nk - nq if causal else torch.full((nq,), nk - 1, device=DEV)
            hid = torch.arange(nk, device=DEV)[None] > sees[:, None]
            live = sees >= 0
            if nk and live.any():
                z = (q @ k.T * scale).masked_fill(hid, -math.inf)[live]
                za = (q.abs() @ k.abs().T * abs(scale)).masked_fill(hid, 0.0)[live]
                out, lse, ob, lb = attend(z, za, v, q.shape[1], 2.0 ** -8)
                assert_within(d["out"][q0:q1, h][live], out, ob, f"out of sequence {b} head {h}")
                if d["lse"] is not None:
                    assert_within(d["lse"][q0:q1, h][live], lse, lb, f"lse of sequence {b} head {h}")
            if (~live).any():
                assert (d["out"][q0:q1, h][~live] == 0).all()
                if d["lse"] is not None:
                    assert (d["lse"][q0:q1, h][~live] == -math.inf).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,dim,rope,vdim", [(4, 4, 128, 64, 128), (8, 2, 128, 0, 128), (3, 1, 64, 0, 64), (2, 2, 64, 64, 128),
                                                  (5, 5, 40, 24, 72), (6, 3, 8, 8, 8), (2, 1, 128, 64, 64), (4, 1, 96, 0, 96)])
def test_prefill_shapes(Hq, Hkv, dim, rope, vdim, causal):
    p = prefill_problem([1, 5, 0, 130, 257, 64], [1, 5, 3, 130, 600, 65], Hq, Hkv, dim, rope, vdim, seed=dim + Hq, pad=3)
    d = run_prefill(p, 1.5 / math.sqrt(dim + rope), causal)
    check_prefill(p, d, 1.5 / math.sqrt(dim + rope), causal)
    assert (d["out"][-3:] == 77).all() and (d["lse"][-3:] == 77).all()
    assert s4r.s4r_read_device_status(None) == s4r.S4R_OK


@pytest.mark.parametrize("nq,nk", [([127, 128, 129], [127, 128, 129]), ([255, 256, 257], [255, 256, 257]), ([1], [5000]),
                                   ([1100], [1100]), ([300, 2], [7, 900]), ([10, 4], [0, 4]), ([513], [2049])])
def test_prefill_lengths(nq, nk):
    p = prefill_problem(nq, nk, 2, 1, 128, 64, 128, seed=nq[0])
    check_prefill(p, run_prefill(p, 0.1, lse=nq[0] % 2 == 0), 0.1)
    check_prefill(p, run_prefill(p, -0.2, max_q=5000), -0.2)


def test_prefill_growing_logits():
    p = prefill_problem([700], [700], 2, 2, 64, 0, 64, seed=2)
    p["k"] = (p["k"].float() * torch.linspace(0.1, 10, 700)[:, None, None]).to(BF)
    check_prefill(p, run_prefill(p, 1.0), 1.0)
    check_prefill(p, run_prefill(p, 0.0), 0.0)


@pytest.mark.parametrize("scale", [1.0, -0.5])
def test_prefill_growing_logits_with_rotary_keys(scale):
    """The reference maximum is exceeded again and again in tiles that every query sees whole."""
    p = prefill_problem([300], [1500], 3, 1, 128, 64, 128, seed=22)
    p["k"] = (p["k"].float() * torch.linspace(0.05, 12, 1500)[:, None, None]).to(BF)
    check_prefill(p, run_prefill(p, scale), scale)
    check_prefill(p, run_prefill(p, scale, causal=False), scale, causal=False)


def test_prefill_unseen_keys_have_no_influence():
    p = prefill_problem([200, 90], [200, 90], 2, 1, 64, 64, 64, seed=3)
    d = run_prefill(p, 0.1)
    q = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    for key in ("k", "v", "k_rope"):            # keys 150 .. of the first sequence
        q[key][150:200] = math.nan
    e = run_prefill(q, 0.1)
    assert torch.equal(d["out"][:150], e["out"][:150]) and torch.equal(d["out"][200:], e["out"][200:])
    assert torch.equal(d["lse"][:150], e["lse"][:150])


def test_prefill_without_any_key():
    p = prefill_problem([3, 200], [0, 0], 4, 2, 128, 64, 128, seed=23)
    for causal in (True, False):
        d = run_prefill(p, 0.1, causal)
        assert not d["out"].any() and (d["lse"] == -math.inf).all()


def test_prefill_strided_keys():
    p = prefill_problem([150], [333], 4, 2, 64, 32, 64, seed=4)
    kv = torch.cat([p["k"].flatten(1), p["v"].flatten(1), p["k_rope"]], 1).to(DEV)        # one row a token
    k, v = kv[:, :128].view(333, 2, 64), kv[:, 128:256].view(333, 2, 64)
    out = torch.empty(150, 4, 64, dtype=BF, device=DEV)
    s4r.s4r_prefill_attend(s4r.prefill_attend_args(q=p["q"].to(DEV), k=k, v=v, k_rope=kv[:, 256:], cu_q=i32([0, 150]),
                                                   cu_k=i32([0, 333]), max_q=150, scale=0.1, out=out))
    check_prefill(p, dict(out=out, lse=None), 0.1)


def test_prefill_bad_offsets_are_reported():
    p = prefill_problem([40, 50, 60], [40, 50, 60], 2, 2, 64, 0, 64, seed=5)
    good = dict(p)
    for key, at, value in (("cu_q", 3, 151), ("cu_k", 3, 151), ("cu_k", 3, 80), ("cu_q", 0, -1)):
        p[key] = good[key].copy()
        p[key][at] = value
        d = run_prefill(p, 0.1, max_q=60)
        assert s4r.s4r_read_device_status(None) == s4r.S4R_ERR_DEVICE
        s4r.s4r_clear_device_status(None)
        check_prefill(good, d, 0.1, only=[1])
        p[key] = good[key]
    d = run_prefill(p, 0.1, max_q=55)           # the last sequence is longer
    assert s4r.s4r_read_device_status(None) == s4r.S4R_ERR_DEVICE
    s4r.s4r_clear_device_status(None)
    check_prefill(p, d, 0.1, only=[0, 1])
    assert (d["out"][150 - 5:] == 77).all()


def test_prefill_captured():
    p = prefill_problem([200, 100], [200, 300], 4, 2, 128, 64, 128, seed=6)
    d = run_prefill(p, 0.1)
    want = d["out"].clone()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        s4r.s4r_prefill_attend(d["args"])
    d["out"].zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(d["out"], want)


def test_calls_on_two_streams_at_once():
    """Projection and prefill have no workspace: calls on two streams do not meet."""
    probs = [prefill_problem([300, 40], [300, 500], 4, 2, 128, 64, 128, seed=k) for k in (7, 8)]
    runs = [run_prefill(p, 0.1) for p in probs]
    want = [d["out"].clone() for d in runs]
    g = torch.Generator().manual_seed(9)
    x = [torch.randn(400, 8, 128, generator=g).to(BF).to(DEV) for _ in probs]
    basis = [(torch.randn(8 * 128, 256, generator=g) / 11).to(BF).to(DEV) for _ in probs]
    out = [torch.empty(400, 8, 256, dtype=BF, device=DEV) for _ in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    for _ in range(10):
        for d, s, a, b, o in zip(runs, streams, x, basis, out):
            s4r.s4r_prefill_attend(d["args"], s)
            s4r.s4r_latent_project(a, b, o, to_latent=True, stream=s)
    torch.cuda.synchronize()
    for d, w, a, b, o in zip(runs, want, x, basis, out):
        assert torch.equal(d["out"], w)
        check_project(a.cpu(), b.cpu(), o, 8, 128, 256, True)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dt", ["bf16", "fp4"])
def test_prompt_then_decode(dt):
    """A prompt is encoded, planned, written and attended in the expanded form; then two tokens are decoded in the
    absorbed form.  Both agree with 64-bit attention over keys and values expanded from what the cache holds."""
    g = torch.Generator().manual_seed(21)
    H, dim, rope, vdim, rank, page, D = 8, 64, 32, 64, 192, 32, 256
    lens, width, T = [90, 200], rank + rope, 2
    down = (torch.randn(D, rank, generator=g) / 16).to(BF).to(DEV)
    bk = (torch.randn(H * dim, rank, generator=g) / 14).to(BF).to(DEV)
    bv = (torch.randn(H * vdim, rank, generator=g) / 14).to(BF).to(DEV)
    total = sum(lens)
    latents = torch.randn(total, width, generator=g).to(BF).to(DEV)
    states = torch.randn(total, D, generator=g).to(BF).to(DEV)
    coeffs = torch.empty(total, rank, dtype=BF, device=DEV)
    s4r.s4r_encode(states, down, coeffs)
    latents[:, :rank] = coeffs
    pages = 20
    cache = (torch.zeros(pages, page, width, dtype=BF, device=DEV) if dt == "bf16"
             else torch.zeros(pages, page * width * 9 // 16, dtype=torch.uint8, device=DEV))
    table, held, free = i32(-np.ones((2, 10), dtype=int)), i32([0, 0]), i32([pages])
    pool = i32(np.random.default_rng(1).permutation(pages))
    cu, slots = i32([0, 0, 0]), torch.empty(total, dtype=torch.int64, device=DEV)
    stored = torch.empty(total, width, dtype=BF, device=DEV) if dt == "fp4" else None

    def admit(new, n):
        s4r.s4r_page_plan(lengths=held, new_tokens=i32(new), block_table=table, free_pages=pool, free_count=free,
                          lengths_out=held, free_count_out=free, cu_tokens=cu, slots=slots[:n], page_size=page)

    admit(lens, total)
    s4r.s4r_latent_write(latents=latents, slots=slots, cache=cache, page_size=page, stored=stored)
    kept = latents if stored is None else stored
    # expanded form of the prompt
    k, v = torch.empty(total, H, dim, dtype=BF, device=DEV), torch.empty(total, H, vdim, dtype=BF, device=DEV)
    s4r.s4r_latent_project(kept[:, :rank], bk, k, to_latent=False)
    s4r.s4r_latent_project(kept[:, :rank], bv, v, to_latent=False)
    q = torch.randn(total, H, dim + rope, generator=g).to(BF).to(DEV)
    out = torch.empty(total, H, vdim, dtype=BF, device=DEV)
    s4r.s4r_prefill_attend(s4r.prefill_attend_args(q=q, k=k, v=v, k_rope=kept[:, rank:], cu_q=cu, cu_k=cu, max_q=200,
                                                   scale=0.1, out=out))
    check_prefill(dict(q=q.cpu(), k=k.cpu(), v=v.cpu(), k_rope=kept[:, rank:].cpu(), cu_q=[0, 90, 290], cu_k=[0, 90, 290]),
                  dict(out=out, lse=None), 0.1)
    # two more tokens a request, absorbed form
    fresh = torch.randn(4, width, generator=g).to(BF).to(DEV)
    fresh_stored = torch.empty(4, width, dtype=BF, device=DEV) if dt == "fp4" else None
    admit([T, T], 4)
    s4r.s4r_latent_write(latents=fresh, slots=slots[:4], cache=cache, page_size=page, stored=fresh_stored)
    q = torch.randn(2, T, H, dim + rope, generator=g).to(BF).to(DEV)
    ql = torch.empty(2, T, H, width, dtype=BF, device=DEV)
    s4r.s4r_latent_project(q.view(4, H, -1)[..., :dim], bk, ql.view(4, H, -1)[..., :rank], to_latent=True)
    ql[..., rank:] = q[..., dim:]
    ol = torch.empty(2, T, H, rank, dtype=BF, device=DEV)
    a = s4r.latent_attend_args(q=ql, cache=cache, block_table=table, lengths=held, out=ol, page_size=page, scale=0.1)
    ws = torch.empty(s4r.s4r_latent_attend_workspace_bytes(a), dtype=torch.uint8, device=DEV)
    s4r.s4r_workspace_init(ws)
    s4r.s4r_latent_attend(s4r.latent_attend_args(q=ql, cache=cache, block_table=table, lengths=held, out=ol, page_size=page,
                                                 scale=0.1, workspace=ws))
    o = torch.empty(4, H, vdim, dtype=BF, device=DEV)
    s4r.s4r_latent_project(ol.view(4, H, rank), bv, o, to_latent=False)
    assert s4r.s4r_read_device_status(ws) == s4r.S4R_OK
    new = (fresh if fresh_stored is None else fresh_stored).double()
    at = [0, 90, 290]
    for b in range(2):
        rows = torch.cat([kept[at[b]:at[b + 1]].double(), new[2 * b:2 * b + 2]])
        for t in range(T):
            seen = rows[:lens[b] + 1 + t]
            for h in range(H):
                keys = torch.cat([seen[:, :rank] @ bk[h * dim:(h + 1) * dim].double().T, seen[:, rank:]], 1)
                p = torch.softmax(keys @ q[b, t, h].double() * 0.1, 0)
                want = (p @ seen[:, :rank]) @ bv[h * vdim:(h + 1) * vdim].double().T
                # bf16 roundings on the way: absorbed queries (2^-8 of sum |q B| |c| in the logits), probabilities,
                # attended latents, the result; each bounded by 2^-8 of its absolute sums
                qa = q[b, t, h, :dim].double().abs() @ bk[h * dim:(h + 1) * dim].double().abs()
                ez = (qa @ seen[:, :rank].abs().T * 0.1 * 2.0 ** -8).max()
                mass = (p @ seen[:, :rank].abs()) @ bv[h * vdim:(h + 1) * vdim].double().abs().T
                assert_within(o[2 * b + t, h], want, mass * (2 * torch.expm1(ez) + 3 * 2.0 ** -8 + 2.0 ** -9))
