"""Plain 64-bit forms of the paged latent operators and of prefill attention, with the error bounds that their 16-bit
roundings allow."""
import math

import numpy as np
import torch

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def cdiv(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- page plan

def plan(lengths, new, table, free_pages, free_count, page_size, max_tokens):
    """The plan, one request after another.  Returns table, lengths, free count, cu, slots, positions, requests, ok."""
    B, width = table.shape
    table = table.copy()
    free = min(max(int(free_count), 0), len(free_pages))
    ok = free == int(free_count)
    demand, taken = 0, 0
    out = list(map(int, lengths))
    cu, slots, positions, requests = [0], [], [], []
    for b in range(B):
        old, add = int(lengths[b]), int(new[b])
        fits = old >= 0 and add >= 0 and old + add <= width * page_size
        have = cdiv(old, page_size)
        need = cdiv(old + add, page_size) - have if fits else 0
        demand += need
        served = fits and (need == 0 or demand <= free)
        ok &= served
        if served:
            for i in range(need):
                table[b, have + i] = free_pages[free - 1 - (demand - need + i)]
            if need:
                taken = demand
            out[b] = old + add
        count = max(add, 0)
        for j in range(min(count, max(0, max_tokens - cu[-1]))):
            p = old + j
            slots.append(int(table[b, p // page_size]) * page_size + p % page_size if served else -1)
            positions.append(p)
            requests.append(b)
        cu.append(cu[-1] + count)
    ok &= cu[-1] <= max_tokens
    pad = max_tokens - len(slots)
    return dict(table=table, lengths=np.array(out, dtype=np.int64), free=free - taken, cu=np.array(cu),
                slots=np.array(slots + [-1] * pad), positions=np.array(positions + [-1] * pad),
                requests=np.array(requests + [-1] * pad), ok=bool(ok))


# ---------------------------------------------------------------- 4-bit rows

def quantise(rows, cache_scale=1.0):
    """(codes [n][w] uint8, scale bytes [n][w/16] uint8, values [n][w] float64) of bf16 rows on the CPU, finite or not."""
    n, w = rows.shape
    x = rows.float()
    if cache_scale != 1.0:
        x = x / torch.tensor(cache_scale, dtype=torch.float32)
    x = x.view(n, w // 16, 16)
    top = torch.nan_to_num(x.abs(), nan=0.0, posinf=math.inf).amax(2)
    scale8 = (top / torch.tensor(6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale8.float()[..., None]
    t = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x)).double()
    mag = torch.nan_to_num(t.abs(), nan=6.0, posinf=6.0).clamp(max=6.0)
    dist = (mag[..., None] - E2M1).abs()
    best = dist.amin(-1, keepdim=True)
    even = (torch.arange(8) % 2 == 0)
    # of two nearest codes the even one
    code = torch.where((dist == best) & even, torch.zeros(8), torch.where(dist == best, torch.ones(8), torch.full((8,), 9.0))).argmin(-1)
    neg = torch.signbit(t) & ~torch.isnan(t) & (s > 0)
    value = E2M1[code] * torch.where(neg, -1.0, 1.0) * s.double() * cache_scale
    code = torch.where(s > 0, code + 8 * neg.long(), torch.zeros_like(code))
    return code.view(n, w).to(torch.uint8), scale8.view(torch.uint8), value.view(n, w)


def pack_page(codes, scales):
    """Bytes of a page from its rows' codes [page][w] and scales [page][w/16]."""
    return torch.cat([(codes[:, 0::2] | (codes[:, 1::2] << 4)).reshape(-1), scales.reshape(-1)])


# ---------------------------------------------------------------- attention

def latent_attend(q, rows, sees, rank, scale, p_half_step):
    """One query token: q [H][w], rows [n][w] float64; the first `sees` rows.  (out, lse, out bound, lse bound)."""
    H, w = q.shape
    if sees <= 0:
        z = torch.zeros(H, rank, dtype=torch.float64, device=q.device)
        inf = torch.full((H,), -math.inf, dtype=torch.float64, device=q.device)
        return z, inf, z + 1e-300, torch.zeros_like(inf)
    return attend(q @ rows[:sees].T * scale, (q.abs() @ rows[:sees].abs().T) * abs(scale), rows[:sees, :rank], w, p_half_step)


def attend(z, z_abs, v, width, p_half_step):
    """softmax(z) v with bounds.  z [H][n] exact logits, z_abs their sums of absolute products.

    Logits: `width` products summed in fp32 in some order, each addition within 2^-23 of its partial sum (a tensor core
    may cut instead of rounding): off by at most ez = (width + 2) 2^-23 z_abs.  Then e^(z - reference) is off by a factor
    e^(ez) and the 2^-21 of exp itself; the sum of n of them in fp32, in pieces, adds less than 2^-14.  Numerator and
    denominator: twice that.  Probabilities are rounded to 16 bits for the value product only (p_half_step), which is
    summed with 2^-23 an addition (together under 2^-12 for the lengths tested, as they are split).  At last the result
    is rounded to bf16."""
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    out = p @ v
    ez = ((width + 2) * 2.0 ** -23 * z_abs).amax(1)
    rel = 2 * (torch.expm1(ez) + 2.0 ** -14) + 2.0 ** -12 + p_half_step
    bound = rel[:, None] * (p @ v.abs())
    bound = bound + 2.0 ** -8 * (out.abs() + bound) + 2.0 ** -133
    return out, lse, bound, 2 * ez + 2.0 ** -14 + 2.0 ** -22 * lse.abs()


def assert_within(got, exact, bound, what=""):
    got = got.double().to(exact.device)
    same = (got == exact)                      # infinities
    off = (got - exact).abs()
    bad = ~(same | (off <= bound))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {off[bad].max().item():.3e} "
                           f"with a bound of {bound.expand_as(off)[bad].min().item():.3e}, first at {bad.nonzero()[0].tolist()}")
