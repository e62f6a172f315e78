"""Argument errors of the router and the key/value cache calls (CPU only: every
call here is refused, or has nothing to do, before anything is launched)."""
import pytest
import torch

import group_wise_affine_dequant_b200 as nvq
from group_wise_affine_dequant_b200 import binding as B

INVALID, UNSUPPORTED, WORKSPACE, OK = B.NV_ERR_INVALID_ARG, B.NV_ERR_UNSUPPORTED, B.NV_ERR_WORKSPACE, B.NV_OK


def _route(**kw):
    a = dict(z=16, dt=1, T=4, E=64, bias=0, score=0, groups=1, topk_groups=1, group_top=1, topk=4, renorm=1,
             scale=1.0, ids=16, w=16)
    a.update(kw)
    return nvq.lib().nv_moe_route(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), UNSUPPORTED), (dict(E=1024), UNSUPPORTED), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(E=0), INVALID), (dict(score=2), INVALID), (dict(groups=0), INVALID), (dict(groups=5), INVALID),
    (dict(groups=8, topk_groups=9), INVALID), (dict(groups=8, topk_groups=0), INVALID), (dict(group_top=0), INVALID),
    (dict(group_top=3), INVALID), (dict(topk=0), INVALID), (dict(topk=65, E=128), INVALID), (dict(topk=33, E=32), INVALID),
    (dict(groups=8, topk_groups=1, topk=9), INVALID), (dict(z=0), INVALID), (dict(z=8), INVALID), (dict(ids=0), INVALID),
    (dict(w=0), INVALID), (dict(w=18), INVALID), (dict(bias=17), INVALID), (dict(T=0), OK), (dict(T=0, z=0), OK)])
def test_route(kw, status):
    assert _route(**kw) == status


CACHE = dict(kc=16, ks=16, vc=16, vs=16, mode=1, P=8, H=2, block=64, D=128)
STEPS = dict(pages=16, max_pages=4, starts=16, lens=16, S=2)
SHARED = [
    (dict(dt=2), UNSUPPORTED), (dict(mode=0), INVALID), (dict(mode=3), INVALID), (dict(P=-1), INVALID),
    (dict(P=1 << 31), INVALID), (dict(H=0), INVALID), (dict(H=1025, Hq=1025, k_stride=1 << 18, v_stride=1 << 18), INVALID),
    (dict(block=48), UNSUPPORTED), (dict(block=256), UNSUPPORTED), (dict(block=0), INVALID), (dict(D=8), UNSUPPORTED),
    (dict(D=272), UNSUPPORTED), (dict(D=0), INVALID), (dict(rows=-1), INVALID), (dict(S=-1), INVALID),
    (dict(S=1 << 25), INVALID), (dict(max_pages=-1), INVALID), (dict(kc=0), INVALID), (dict(vc=8), INVALID),
    (dict(ks=0), INVALID), (dict(vs=18), INVALID), (dict(pages=0), INVALID), (dict(pages=18), INVALID),
    (dict(starts=0), INVALID), (dict(lens=0), INVALID), (dict(flags=18), INVALID), (dict(rows=0), OK), (dict(S=0), OK)]


def _fill(order, kw):
    a = dict(order)
    a.update({k: v for k, v in kw.items() if k in a})
    return list(a.values())


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k=8), INVALID), (dict(k_stride=255), INVALID),
    (dict(v_stride=260), INVALID), (dict(k_stride=128), INVALID), (dict(dt=0, k_stride=258), INVALID)])
def test_quantize(kw, status):
    order = dict(k=16, v=16, k_stride=256, v_stride=256, dt=1, rows=3, **CACHE, **STEPS, flags=0)
    assert nvq.lib().nv_kv_quantize(*_fill(order, kw), None) == status


@pytest.mark.parametrize("kw,status", SHARED + [(dict(k=0), INVALID), (dict(v=0), INVALID), (dict(v=24), INVALID)])
def test_dequantize(kw, status):
    order = dict(**CACHE, **STEPS, dt=1, rows=3, k=16, v=16, flags=0)
    assert nvq.lib().nv_kv_dequantize(*_fill(order, kw), None) == status


def _attention(**kw):
    order = dict(q=16, q_stride=1024, dt=1, rows=3, Hq=8, **CACHE, **STEPS, scale=0.1, causal=1, window=0, max_q=1,
                 ws=16, ws_bytes=None, out=16, flags=0)
    a = dict(order)
    a.update({k: v for k, v in kw.items() if k in a})
    if a["ws_bytes"] is None:
        a["ws_bytes"] = _workspace(**kw)
    return nvq.lib().nv_kv_attention(*a.values(), None)


def _workspace(**kw):
    a = dict(dt=1, rows=3, Hq=8, H=2, block=64, D=128, max_pages=4, S=2, max_q=1)
    a.update({k: v for k, v in kw.items() if k in a})
    return nvq.lib().nv_kv_attention_workspace_size(*a.values())


@pytest.mark.parametrize("kw,status", [x for x in SHARED if x[0] != dict(H=0)] + [
    (dict(H=0, ws_bytes=1 << 30), INVALID), (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(q=8), INVALID),
    (dict(out=24), INVALID), (dict(q_stride=1000), INVALID), (dict(q_stride=1028), INVALID), (dict(Hq=0), INVALID),
    (dict(Hq=7), INVALID), (dict(window=-1), INVALID), (dict(window=5, causal=0), INVALID), (dict(max_q=-1), INVALID),
    (dict(rows=1 << 30), INVALID)])
def test_attention(kw, status):
    assert _attention(**kw) == status


def test_attention_workspace():
    """Sizes are a function of the arguments; what is needed is asked for, a byte less refused."""
    for kw in (dict(), dict(max_pages=4000), dict(rows=2000, max_q=1000, max_pages=400), dict(max_q=0, max_pages=400),
               dict(dt=0, max_pages=4000), dict(D=80, max_pages=4000)):
        need = _workspace(**kw)
        assert need == _workspace(**kw) and need >= 0
        if need:
            assert _attention(**kw, ws_bytes=need - 1) == WORKSPACE
            assert _attention(**kw, ws=0) == WORKSPACE
            assert _attention(**kw, ws=24) == WORKSPACE
    for bad in (dict(H=0), dict(Hq=0), dict(D=0), dict(block=0), dict(rows=-1), dict(S=-1), dict(max_pages=-1)):
        assert _workspace(**bad) == 0


def test_attention_of_sizes_that_no_memory_holds():
    """Products of the largest sizes neither wrap around in the workspace's bytes nor in a grid."""
    huge = dict(rows=(1 << 31) // 8 - 1, S=(1 << 24) - 1, H=8, max_pages=(1 << 31) - 1, block=128, P=8, max_q=0)
    assert _workspace(**huge) >= 1 << 50
    assert _attention(**huge, ws_bytes=1 << 49) == WORKSPACE
    wide = dict(rows=4, S=(1 << 24) - 1, H=64, Hq=64, q_stride=64 * 128, max_q=0, max_pages=1)
    assert _attention(**wide, ws_bytes=1 << 62) == INVALID
    assert _attention(**{**wide, "S": 1 << 20}, q=8, ws_bytes=1 << 62) == INVALID  # the queries' alignment, past the sizes


def test_tensors_that_do_not_fit():
    """The Python calls refuse what is not on a GPU, or no tensor, before anything is launched."""
    z = torch.zeros(4, 8)
    cache = [torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2)] * 2
    steps = [torch.zeros(1, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)]
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for bad in (lambda: nvq.nv_moe_route(z, 2), lambda: nvq.nv_moe_route(None, 2), lambda: nvq.nv_moe_route(z, 2, "relu"),
                lambda: nvq.nv_kv_quantize(x, x, *cache, *steps), lambda: nvq.nv_kv_quantize(x, None, *cache, *steps),
                lambda: nvq.nv_kv_dequantize(*cache, *steps, rows=4), lambda: nvq.nv_kv_attention(x, *cache, *steps),
                lambda: nvq.nv_kv_attention(x, 5, *cache[1:], *steps)):
        with pytest.raises(ValueError):
            bad()
