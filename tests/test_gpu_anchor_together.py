"""The anchor pool's gate and correction beside another stream's calls: the bits that they give alone.

Two streams run at once, each with two inputs in turn, so that what an earlier call left in shared memory
could not pass for what a call has to read.  Units enough that a CTA walks several.
"""
import pytest
import torch

from cross_context_kv_gb300 import synth
from test_gpu_anchor import compose, factors

DEV = "cuda"


@pytest.fixture(scope="module")
def kvfix():
    from cross_context_kv_gb300 import build
    build.build()
    from cross_context_kv_gb300 import kvfix
    return kvfix


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("fused", (False, True))
@pytest.mark.parametrize("anchors,rank,dim", ((4, 16, 128), (10, 32, 128), (5, 64, 64)))
def test_beside_another_stream(kvfix, anchors, rank, dim, fused):
    cases = []
    for seed in range(4):
        cfg = synth.ANCHOR_8B.with_(name="together", segments=2, anchors=anchors, layers=3, tokens=1500, kv_heads=4, head_dim=dim,
                                    rank=rank, seed=70 + seed)
        inp = synth.anchor_inputs(cfg, DEV)
        cases.append((cfg, inp, compose(cfg, inp), factors(inp)))

    def call(i):
        cfg, inp, src, fac = cases[i]
        if not fused:
            return kvfix.anchor_gate(src["v"], inp["a_c_v"], inp["b_ct_v"], cfg.tokens, tau=cfg.tau)
        # (a threshold that every segment passes, so that all outputs are written)
        return kvfix.anchor_gate_correct(src["k"], src["v"], fac, cfg.tokens, inp["delta"], cfg.rope_base, tau=1.0)

    alone = [call(i) for i in range(4)]
    kvfix.check_status()
    assert all(a[-1].all() for a in alone) or not fused
    streams = [torch.cuda.Stream() for _ in range(2)]
    for again in range(5):
        got = [[], []]
        torch.cuda.synchronize()
        for n in range(8):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[i].append(call(2 * i + n % 2))
        torch.cuda.synchronize()
        kvfix.check_status()
        for i in range(2):
            for n in range(8):
                for k, (x, y) in enumerate(zip(got[i][n], alone[2 * i + n % 2])):
                    assert torch.equal(bits(x), bits(y)), f"pass {again}, stream {i}, call {n}, output {k}: " \
                        f"{int((bits(x) != bits(y)).sum())} bytes or words"
