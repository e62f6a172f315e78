"""The operators of a decoder layer one after the other, as a serving loop runs
them: quantized projections, the step's keys and values into the 8-bit cache,
attention over it, the quantized output projection, the router and the routed
block. A prompt of two sequences, then single tokens; every stage is compared
with its own 64-bit reference on the inputs that it was given."""
import pytest
import torch

import group_wise_affine_dequant_b200 as nvq
import oracle as O
from group_wise_affine_dequant_b200 import workloads as W
from tests import kv_reference as R
from tests import parity as P

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
def test_prompt_then_tokens(mode):
    K, H, G, D, E, I, topk, block = 512, 2, 4, 64, 8, 512, 2, 16
    wide = (H * G + 2 * H) * D
    qkv = O.quantize_affine(W.normal((wide, K), 0.06, 1, "bf16"), 64, 4)
    proj = O.quantize_affine(W.normal((K, H * G * D), 0.06, 2, "bf16"), 64, 8)
    gate = O.quantize_affine(W.normal((E, I, K), 0.04, 3, "bf16"), 64, 4)
    up = O.quantize_affine(W.normal((E, I, K), 0.04, 4, "bf16"), 64, 4)
    down = O.quantize_affine(W.normal((E, K, I), 0.04, 5, "bf16"), 64, 4)
    router = W.normal((E, K), 0.05, 6, "bf16").cuda()
    dev = lambda q: tuple(t.cuda() for t in q)  # noqa: E731
    qkv_d, proj_d, gate_d, up_d, down_d = dev(qkv), dev(proj), dev(gate), dev(up), dev(down)
    pages = torch.arange(12, dtype=torch.int32).view(2, 6)
    kc = torch.zeros(12, H, block, D, dtype=R.MODES[mode], device="cuda")
    vc = torch.zeros(12, H, block, D, dtype=R.MODES[mode], device="cuda")
    ks, vs = torch.zeros(12, H, device="cuda"), torch.zeros(12, H, device="cuda")
    kraw, vraw = (torch.zeros(12, H, block, D, dtype=torch.uint8) for _ in range(2))
    ksr, vsr = torch.zeros(12, H), torch.zeros(12, H)
    lens = [0, 0]
    for step_no, news in enumerate([(37, 50), (1, 1), (1, 1), (1, 0), (3, 1)]):
        lens = [a + b for a, b in zip(lens, news)]
        step = R.Step(lens, news, block)
        step.pages, step.P = pages, 12
        T = sum(news)
        x = W.normal((T, K), 1.0, 10 + step_no, "bf16").cuda()
        rows = nvq.nv_qmm(x, *qkv_d, 64, 4, True).view(T, H * G + 2 * H, D)
        q, k, v = rows[:, : H * G], rows[:, H * G: H * G + H], rows[:, H * G + H:]
        nvq.nv_kv_quantize(k, v, kc, ks, vc, vs, *step.dev())
        att = nvq.nv_kv_attention(q, kc, ks, vc, vs, *step.dev(), max_q=max(news))
        o = nvq.nv_qmm(att.view(T, H * G * D), *proj_d, 64, 8, True)
        ids, rw = nvq.nv_moe_route((o @ router.t()).float(), topk, "sigmoid")
        y = nvq.nv_moe_swiglu(o, gate_d, up_d, down_d, ids, rw, 64, 4)
        torch.cuda.synchronize()
        kraw, ksr = R.write(k.cpu(), kraw, ksr, step, mode)
        vraw, vsr = R.write(v.cpu(), vraw, vsr, step, mode)
        for got, want in ((kc, kraw), (vc, vraw)):
            assert torch.equal(got.cpu().view(torch.uint8), want), step_no
        assert torch.equal(ks.cpu(), ksr) and torch.equal(vs.cpu(), vsr)
        want, *terms = R.attention(q.cpu(), kraw, ksr, vraw, vsr, step, mode, D ** -0.5)
        room = R.attention_tolerance(want, terms, BF16, D, max(lens))
        assert bool(((att.cpu().double() - want).abs() <= room).all()), step_no
        yr, ya = O.qmm(att.cpu().view(T, -1), *proj, 64, 8, True)
        P.assert_within(o, yr, ya, BF16, "output projection")
        yr, ya = O.moe_swiglu(o.cpu(), gate, up, down, ids.cpu().long(), rw.cpu(), 64, 4)
        P.assert_within(y, yr, ya, BF16, "routed block")
        assert bool((rw.sum(1) - 1).abs().max() < 1e-6)
    assert nvq.nv_pipeline_error() == 0
