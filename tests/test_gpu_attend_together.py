"""kvfix_shared_attend and kvfix_tree_attend beside another stream's calls: the bits that they give alone.

Two streams run at once, each with a workspace of its own and two rounds in turn in it, so that nothing
that an earlier call left (plans, parts, tiles in shared memory) could pass for what a call has to make.
Rows enough that blocks take both softmax groups, and singles beside them; every pair of stored forms.
"""
import pytest
import torch

from test_gpu_attend import Round
from test_gpu_tree import Trees

gpu = pytest.mark.gpu
AGENTS = 12
SHAPES = {"short": dict(heads=8, T=30, group=4, dim=128), "long": dict(heads=4, T=64, group=5, dim=128),
          "narrow": dict(heads=8, T=30, group=4, dim=64), "few": dict(heads=2, T=4, group=2, dim=128)}


@pytest.fixture(scope="module")
def kvfix():
    from cross_context_kv_gb300 import build
    build.build()
    from cross_context_kv_gb300 import kvfix
    return kvfix


def make(kvfix, call, fmt, seed, heads, T, group, dim):
    before = [(53 + 11 * seed) * a % 300 for a in range(AGENTS)]
    args = (heads, group, dim, 16, T, [(900, 400, 650, 130)[seed]], [0, AGENTS])
    if call == "tree":
        return Trees(kvfix, fmt, *args, before, [T - (a + seed) % 3 for a in range(AGENTS)], seed=seed)
    return Round(kvfix, fmt, *args, [n + T for n in before], seed=seed)


def differences(got, want):
    """What differs of a call's (out, lse), in words, or nothing."""
    out = (got[0].view(torch.int16) != want[0].view(torch.int16)).any(-1)
    lse = got[1].view(torch.int32) != want[1].view(torch.int32)
    if not out.any() and not lse.any():
        return ""
    at = (out | lse).nonzero().tolist()
    away = (got[0].float() - want[0].float()).abs().nan_to_num(nan=float("inf")).max().item()
    return (f"{int(out.sum())} rows of out (largest difference {away:.3g}) and {int(lse.sum())} of lse, NaN: "
            f"{bool(torch.isnan(got[0].float()).any())}; agents {sorted({a for a, _, _ in at})}, heads "
            f"{sorted({h for _, _, h in at})}, first (agent, token, head) {at[0]}")


@gpu
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("forms", ("bf16 e4m3", "e4m3 int4", "int4 bf16", "e4m3 e4m3", "bf16 bf16", "int4 int4"))
@pytest.mark.parametrize("call", ("tree", "shared"))
def test_beside_another_stream(kvfix, call, forms, shape):
    rounds = [[make(kvfix, call, fmt, 2 * i + k, **SHAPES[shape]) for k in range(2)] for i, fmt in enumerate(forms.split())]
    alone = [[r.call() for r in mine] for mine in rounds]
    size = kvfix.shared_attend_workspace_bytes(rounds[0][0].q, rounds[0][0].pool, 1)
    works = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in rounds]
    calls = 20
    outs = [[torch.zeros_like(rounds[0][0].q) for _ in range(calls)] for _ in rounds]
    streams = [torch.cuda.Stream() for _ in rounds]
    for again in range(10):
        lses = [[] for _ in rounds]
        torch.cuda.synchronize()
        for n in range(calls):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    lses[i].append(rounds[i][n % 2].call(out=outs[i][n], workspace=works[i])[1])
        torch.cuda.synchronize()
        kvfix.check_status()
        for i, fmt in enumerate(forms.split()):
            for n in range(calls):
                said = differences((outs[i][n], lses[i][n]), alone[i][n % 2])
                assert not said, f"pass {again}, stream {i} ({fmt}), call {n}: {said}"
