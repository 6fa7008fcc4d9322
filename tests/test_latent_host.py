"""Host-side checks of the paged latent operators and prefill attention that need no GPU: structure layouts, workspace
sizes, and argument errors that are reported before anything is enqueued."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import rank_decode_attention_b200 as s4r
from latent_reference import plan
from rank_decode_attention_b200 import build as s4r_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = s4r.S4R_OK, s4r.S4R_ERR_INVALID_ARG, s4r.S4R_ERR_UNSUPPORTED, s4r.S4R_ERR_WORKSPACE
STRUCTS = {"s4r_page_plan_args": s4r.PagePlanArgs, "s4r_latent_write_args": s4r.LatentWriteArgs,
           "s4r_latent_attend_args": s4r.LatentAttendArgs, "s4r_latent_project_args": s4r.LatentProjectArgs,
           "s4r_prefill_attend_args": s4r.PrefillAttendArgs}


@pytest.fixture(scope="module", autouse=True)
def built():
    s4r_build.build()


def test_struct_layouts_match_c():
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "s4r.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(src, "w").write(prog)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        name, field, off = line.split()
        cls = STRUCTS[name]
        assert int(off) == (ctypes.sizeof(cls) if field == "size" else getattr(cls, field).offset), line


GOOD = {
    "s4r_page_plan": dict(batch=0, page_size=64, max_pages=10, free_capacity=5, max_tokens=3, lengths=0x1000, new_tokens=0x2000,
                          block_table=0x3000, free_pages=0x4000, free_count=0x5000, lengths_out=0x6000, free_count_out=0x7000,
                          cu_tokens=0x8000, slots=0x9000, positions=0xa000, requests=0xb000, status_workspace=None),
    "s4r_latent_write": dict(n_tokens=0, width=576, page_size=64, n_pages=10, cache_dtype=1, cache_scale=1.0, latents=0x1000,
                             latents_ld=576, slots=0x2000, cache=0x3000, stored=None, status_workspace=None),
    "s4r_latent_attend": dict(batch=0, n_query=1, n_heads=16, width=576, rank=512, page_size=64, max_pages=10, cache_dtype=1,
                              n_pages=100, scale=0.1, cache_scale=1.0, q=0x1000, cache=0x2000, block_table=0x3000,
                              lengths=0x4000, out=0x5000, lse=None, workspace=0x6000, workspace_bytes=1 << 40),
    "s4r_latent_project": dict(n_tokens=0, n_heads=4, head_dim=64, rank=192, to_latent=1, x=0x1000, x_ts=256, x_hs=64,
                               basis=0x2000, out=0x3000, out_ts=768, out_hs=192),
    "s4r_prefill_attend": dict(batch=0, n_heads_q=8, n_heads_kv=2, head_dim=128, rope_dim=64, value_dim=128, causal=1, max_q=10,
                               total_q=20, total_k=20, scale=0.1, q=0x1000, k=0x2000, v=0x3000, k_rope=0x4000, k_ts=256,
                               v_ts=256, k_rope_ts=64, cu_q=0x5000, cu_k=0x6000, out=0x7000, lse=None),
}


def call(name, **over):
    cls = STRUCTS[name + "_args"]
    a = cls(**dict(GOOD[name], **over))
    return getattr(s4r.lib(), name)(ctypes.byref(a), None)


@pytest.mark.parametrize("name", [n for n in GOOD if n != "s4r_page_plan"])
def test_empty_calls_are_no_ops(name):
    assert call(name) == OK
    assert getattr(s4r.lib(), name)(None, None) == INVALID


# every refusal with some work to do, so that nothing but the check keeps the call from the GPU
REFUSALS = {
    "s4r_page_plan": (dict(batch=4), [
        (INVALID, dict(batch=-1)), (INVALID, dict(max_pages=0)), (INVALID, dict(free_capacity=-1)), (INVALID, dict(max_tokens=-1)),
        (INVALID, dict(page_size=0)), (UNSUPPORTED, dict(page_size=48)), (UNSUPPORTED, dict(page_size=8)),
        (UNSUPPORTED, dict(page_size=2048)), (UNSUPPORTED, dict(batch=8193)), (UNSUPPORTED, dict(max_tokens=1 << 31)),
        (UNSUPPORTED, dict(max_pages=1 << 26)), (INVALID, dict(lengths=None)), (INVALID, dict(new_tokens=0x2004)),
        (INVALID, dict(block_table=None)), (INVALID, dict(free_pages=None)), (INVALID, dict(free_count=None)),
        (INVALID, dict(lengths_out=None)), (INVALID, dict(free_count_out=0x7004)), (INVALID, dict(cu_tokens=None)),
        (INVALID, dict(slots=None)), (INVALID, dict(positions=0xa004)), (INVALID, dict(requests=0xb008)),
        (INVALID, dict(status_workspace=0x10001))]),
    "s4r_latent_write": (dict(n_tokens=4), [
        (INVALID, dict(n_tokens=-1)), (INVALID, dict(cache_dtype=3)), (UNSUPPORTED, dict(cache_dtype=0)), (INVALID, dict(width=0)),
        (UNSUPPORTED, dict(width=584, latents_ld=584)), (UNSUPPORTED, dict(width=12)), (UNSUPPORTED, dict(width=72, cache_dtype=2)),
        (UNSUPPORTED, dict(page_size=100)), (INVALID, dict(latents_ld=568)), (INVALID, dict(latents_ld=577)),
        (INVALID, dict(latents=None)), (INVALID, dict(slots=0x2004)), (INVALID, dict(cache=None)), (INVALID, dict(cache=0x3008)),
        (INVALID, dict(stored=0x4000)), (INVALID, dict(cache_dtype=2, stored=0x4004)), (INVALID, dict(cache_dtype=2, cache_scale=0.0)),
        (INVALID, dict(cache_dtype=2, cache_scale=-1.0)), (INVALID, dict(cache_dtype=2, cache_scale=float("nan"))),
        (INVALID, dict(cache_dtype=2, cache_scale=float("inf"))), (INVALID, dict(n_pages=-1)), (UNSUPPORTED, dict(n_pages=1 << 31))]),
    "s4r_latent_attend": (dict(batch=2), [
        (INVALID, dict(batch=-1)), (INVALID, dict(n_query=0)), (INVALID, dict(n_heads=0)), (INVALID, dict(rank=0)),
        (INVALID, dict(rank=584)), (UNSUPPORTED, dict(rank=520)), (UNSUPPORTED, dict(rank=500)), (UNSUPPORTED, dict(width=580)),
        (UNSUPPORTED, dict(width=640)), (UNSUPPORTED, dict(cache_dtype=0)), (UNSUPPORTED, dict(cache_dtype=2, width=568)),
        (INVALID, dict(cache_dtype=2, cache_scale=0.0)), (INVALID, dict(scale=float("inf"))), (INVALID, dict(scale=float("nan"))),
        (INVALID, dict(max_pages=0)), (UNSUPPORTED, dict(max_pages=1 << 26)), (UNSUPPORTED, dict(batch=8193)),
        (UNSUPPORTED, dict(n_query=1 << 20, n_heads=1 << 10)), (UNSUPPORTED, dict(n_query=1 << 10, n_heads=65)),
        (UNSUPPORTED, dict(max_pages=(1 << 31) // 64 - 1)), (INVALID, dict(n_pages=0)), (INVALID, dict(q=None)), (INVALID, dict(q=0x1002)),
        (INVALID, dict(cache=None)), (INVALID, dict(block_table=None)), (INVALID, dict(lengths=0x4004)), (INVALID, dict(out=None)),
        (INVALID, dict(lse=0x7004)), (WORKSPACE, dict(workspace=None)), (WORKSPACE, dict(workspace_bytes=8)),
        (WORKSPACE, dict(workspace=0x6008))]),
    "s4r_latent_project": (dict(n_tokens=4), [
        (INVALID, dict(n_tokens=-1)), (INVALID, dict(n_heads=0)), (INVALID, dict(head_dim=0)), (INVALID, dict(rank=0)),
        (UNSUPPORTED, dict(head_dim=60)), (UNSUPPORTED, dict(head_dim=264)), (UNSUPPORTED, dict(rank=520)), (UNSUPPORTED, dict(rank=100)),
        (UNSUPPORTED, dict(n_heads=70000)), (UNSUPPORTED, dict(n_tokens=1 << 31)), (UNSUPPORTED, dict(n_tokens=(1 << 31) - 100)), (INVALID, dict(x=None)), (INVALID, dict(x=0x1008)),
        (INVALID, dict(basis=None)), (INVALID, dict(out=0x3004)), (INVALID, dict(x_ts=260)), (INVALID, dict(x_hs=-64)),
        (INVALID, dict(x_hs=32)), (INVALID, dict(x_ts=0)), (INVALID, dict(out_hs=0)), (INVALID, dict(out_ts=760)),
        (INVALID, dict(out_hs=184)), (INVALID, dict(out_ts=4))]),
    "s4r_prefill_attend": (dict(batch=2), [
        (INVALID, dict(batch=-1)), (INVALID, dict(n_heads_q=7)), (INVALID, dict(n_heads_kv=0)), (INVALID, dict(head_dim=0)),
        (INVALID, dict(rope_dim=-8)), (INVALID, dict(value_dim=0)), (INVALID, dict(max_q=-1)), (INVALID, dict(total_k=-1)),
        (UNSUPPORTED, dict(head_dim=136)), (UNSUPPORTED, dict(head_dim=100)), (UNSUPPORTED, dict(value_dim=256)),
        (UNSUPPORTED, dict(rope_dim=72)), (UNSUPPORTED, dict(rope_dim=4)), (UNSUPPORTED, dict(batch=65536)),
        (UNSUPPORTED, dict(total_q=1 << 31)), (UNSUPPORTED, dict(total_k=(1 << 31) - 200)), (UNSUPPORTED, dict(max_q=1 << 25)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(q=None)), (INVALID, dict(k=None)),
        (INVALID, dict(v=0x3008)), (INVALID, dict(k_rope=None)), (INVALID, dict(cu_q=None)), (INVALID, dict(cu_k=0x6004)),
        (INVALID, dict(out=None)), (INVALID, dict(lse=0x9004)), (INVALID, dict(k_ts=248)), (INVALID, dict(v_ts=260)),
        (INVALID, dict(k_rope_ts=56))]),
}


@pytest.mark.parametrize("name,status,over", [(n, s, o) for n, (base, cases) in REFUSALS.items() for s, o in cases])
def test_refusals(name, status, over):
    assert call(name, **dict(REFUSALS[name][0], **over)) == status


def test_latent_attend_workspace_bytes():
    def size(**over):
        return s4r.s4r_latent_attend_workspace_bytes(s4r.LatentAttendArgs(**dict(GOOD["s4r_latent_attend"], **over)))
    assert size() >= 256 and size() % 256 == 0
    for bad in (dict(width=640), dict(rank=0), dict(page_size=17), dict(cache_dtype=0), dict(n_heads=0)):
        assert size(**bad) == 0, bad


def test_the_binding_refuses_wrong_tensors():
    """Types, shapes and devices, before any pointer is taken (CPU tensors are never on the current CUDA device)."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="current CUDA device|No CUDA|NVIDIA"):
        try:
            s4r.s4r_latent_write(latents=z(2, 64), slots=z(2, dt=torch.int64), cache=z(3, 16, 64), page_size=16)
        except (RuntimeError, AssertionError) as e:
            raise ValueError(str(e))
    with pytest.raises(ValueError, match="slots must be torch.int64|latents|cache"):
        s4r.s4r_latent_write(latents=z(2, 64), slots=z(2, dt=torch.int32), cache=z(3, 16, 64), page_size=16)
    with pytest.raises(ValueError, match="cache must have shape"):
        s4r.s4r_latent_write(latents=z(2, 64), slots=z(2, dt=torch.int64), cache=z(3, 16, 72), page_size=16)
    with pytest.raises(ValueError, match="cache must have 2 dimensions"):
        s4r.s4r_latent_write(latents=z(2, 64), slots=z(2, dt=torch.int64), cache=z(3, 16, 36, dt=torch.uint8), page_size=16)
    with pytest.raises(ValueError, match="lengths must be torch.int32"):
        i = lambda *s: z(*s, dt=torch.int32)  # noqa: E731
        s4r.s4r_page_plan(lengths=z(2, dt=torch.int64), new_tokens=i(2), block_table=i(2, 3), free_pages=i(4), free_count=i(1),
                          lengths_out=i(2), free_count_out=i(1), cu_tokens=i(3), slots=z(4, dt=torch.int64), page_size=16)
    with pytest.raises(ValueError, match="contiguous from dimension 2"):
        s4r.s4r_latent_project(z(4, 2, 64).transpose(1, 2).contiguous().transpose(1, 2), z(128, 32), z(4, 2, 32), to_latent=True)


def test_the_plain_plan():
    """The reference plan on a small example, by hand: request 0 opens a page inside its tokens, request 1 does not fit."""
    import numpy as np
    table = np.array([[7, -1, -1], [-1, -1, -1], [3, -1, -1]])
    r = plan([15, 0, 10], [3, 40, 6], table, [1, 2, 4], 3, 16, 50)
    assert r["table"].tolist() == [[7, 4, -1], [-1, -1, -1], [3, -1, -1]]
    assert r["slots"][:3].tolist() == [7 * 16 + 15, 4 * 16, 4 * 16 + 1]
    assert (r["slots"][3:43] == -1).all() and r["slots"][43:49].tolist() == [58, 59, 60, 61, 62, 63] and r["slots"][49] == -1
    assert r["lengths"].tolist() == [18, 0, 16] and r["free"] == 2 and r["cu"].tolist() == [0, 3, 43, 49] and not r["ok"]
