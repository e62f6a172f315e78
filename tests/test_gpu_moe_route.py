"""The router (nv_moe_route) against the definition in 64 bits: the chosen ids
equal, at ties, next to ties, under masks and with odd group sizes, the weights
to fp32 rounding."""
import numpy as np
import pytest
import torch

import group_wise_affine_dequant_b200 as nvq
from group_wise_affine_dequant_b200 import workloads as W

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LOWEST = torch.finfo(BF16).min


def _reference(z, topk, score, bias, groups, topk_groups, group_top, renormalize, scale):
    """ids, weights in float64. z: float64 [T, E]; masked: NaN or at most the lowest bf16."""
    T, E = z.shape
    per = E // groups
    ids, weights = np.zeros((T, topk), np.int64), np.zeros((T, topk))
    for t in range(T):
        open_ = z[t] > LOWEST
        row = np.where(open_, np.minimum(z[t], np.finfo(np.float32).max), -np.inf)
        if score == "softmax":
            e = np.exp(row - (row.max() if open_.any() else 0.0))
            s = e / e.sum() if open_.any() else e
        else:
            with np.errstate(over="ignore"):
                s = np.where(open_, 1 / (1 + np.exp(-row)), 0.0)
        c = np.where(open_, s + (0.0 if bias is None else bias), -np.inf)
        by_logit = row  # without a bias the logits give the order, also where scores are equal in 64 bits
        rank = by_logit if bias is None else c
        can = np.ones(E, bool)
        if groups > 1:
            key = rank if group_top == 1 else c
            best = []
            for g in range(groups):
                top = np.sort(key[g * per:(g + 1) * per])[::-1][:group_top]
                top = top[top > -np.inf]
                best.append(top.sum() if len(top) else -np.inf)
            kept = np.argsort(-np.array(best), kind="stable")[:topk_groups]
            can = np.isin(np.arange(E) // per, kept)
        order = np.lexsort((np.arange(E), -rank, ~can))
        ids[t] = order[:topk]
        w = s[ids[t]]
        if renormalize:
            # ratios: from the logits, where single scores would underflow
            if score == "softmax":
                zz = row[ids[t]]
                w = np.exp(zz - zz.max()) if zz.max() > -np.inf else np.zeros(topk)
            w = w / w.sum() if w.sum() > 0 else w * 0
        weights[t] = w * scale
    return ids, weights


def _check(z, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renormalize=True, scale=1.0, reach=32.0):
    ids, w = nvq.nv_moe_route(z.cuda(), topk, score, bias=None if bias is None else bias.cuda(), groups=groups,
                              topk_groups=topk_groups, group_top=group_top, renormalize=renormalize, scale=scale)
    torch.cuda.synchronize()
    want, ww = _reference(z.double().numpy(), topk, score, None if bias is None else bias.double().numpy(), groups, topk_groups,
                          group_top, renormalize, scale)
    bad = (ids.cpu().numpy() != want).any(1).nonzero()[0]
    assert len(bad) == 0, f"{len(bad)} tokens, first {bad[0]}: {ids[bad[0]].tolist()} want {want[bad[0]].tolist()}"
    # exponent arguments up to `reach` are rounded to 2^-24 of themselves, the exponential, the
    # sum over E (1/32 of it one after the other) and a few products and quotients to 2^-23 each
    room = (reach + z.shape[1] / 32 + 24) * 2.0 ** -23
    err = np.abs(w.cpu().double().numpy() - ww)
    assert (err <= room * ww + 1e-37).all(), float((err / np.maximum(ww, 1e-37)).max())
    return ids.cpu(), w.cpu()


def _logits(T, E, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(T, E, generator=g)).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,topk", [(1, 1), (2, 2), (7, 3), (32, 32), (33, 4), (64, 4), (100, 6), (256, 8), (300, 64), (1023, 10)])
def test_plain_choice(E, topk, score, dtype):
    for T in (1, 5, 130):
        z = _logits(T, E, dtype, E + T)
        _check(z, topk, score)
        _check(z, topk, score, renormalize=False, scale=2.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups,group_top,topk", [
    (256, 8, 4, 2, 8), (64, 8, 3, 1, 6), (160, 8, 3, 1, 6), (64, 4, 4, 2, 4), (60, 5, 2, 2, 7), (256, 256, 5, 2, 5),
    (512, 2, 1, 2, 20), (39, 3, 2, 1, 3), (1000, 40, 7, 2, 8)])
def test_bias_and_groups(E, groups, topk_groups, group_top, topk, score, dtype):
    g = torch.Generator().manual_seed(E)
    bias = 0.1 * torch.randn(E, generator=g)
    z = _logits(70, E, dtype, E + 1)
    for b in (None, bias):
        for renormalize in (True, False):
            _check(z, topk, score, b, groups, topk_groups, group_top, renormalize, 1.7)
    _check(z, topk, score, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4, 6])
def test_scores_that_fp32_cannot_tell_apart(score, groups):
    """Biases that bring every choice score to about the same number: the order is decided
    between 1e-7 and 1e-9 of each other, and by exact ties."""
    E, T = 96, 40
    z = _logits(1, E, F32, 5, std=0.7).repeat(T, 1)
    zd = z[0].double()
    s = torch.softmax(zd, 0) if score == "softmax" else torch.sigmoid(zd)
    bias = (0.5 - s).float()
    noise = torch.randn(E, generator=torch.Generator().manual_seed(6)) * 2.0 ** -26
    for t in range(T):
        z[t] += noise.roll(t) * (t % 5)
    _check(z, 9, score, bias, groups, max(1, groups // 2), 2 if groups > 1 else 1)
    # repeated logits and biases: real ties, which go to the lower id
    z2 = torch.tensor([1.0, 2.0, 2.0, -1.0]).repeat(10, 24)
    b2 = torch.tensor([0.25, 0.0, 0.0, 0.5]).repeat(24)
    _check(z2, 30, score, b2, groups, max(1, groups // 2), 2 if groups > 1 else 1)
    _check(z2, 30, score, None, groups, max(1, groups // 2), 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_saturated_scores_keep_the_logits_order(score, dtype):
    z = torch.tensor([[30.0, 60.0, 45.0, 61.0, -300.0, -200.0, 0.0, 90.0]] * 3).to(dtype)
    ids, _ = _check(z, 8, score, reach=400.0)
    assert ids[0].tolist() == [7, 3, 1, 2, 0, 6, 5, 4]
    _check(z, 3, score, groups=2, topk_groups=1, reach=400.0)
    _check(torch.tensor([[-500.0, -501.0, -502.5, -499.0]]).to(dtype), 2, "softmax", reach=600.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,bias", [(1, False), (1, True), (4, False), (4, True)])
def test_masked_experts(score, dtype, groups, bias):
    """-infinity, NaN and the lowest value of either type mask; rows masked to fewer than topk, and whole rows."""
    E, topk = 48, 6
    z = _logits(12, E, dtype, 9)
    lowest = torch.finfo(dtype).min
    marks = [-float("inf"), float("nan"), lowest, LOWEST]
    for t in range(12):
        z[t, torch.randperm(E, generator=torch.Generator().manual_seed(t))[: [0, 10, 40, 44, 47, 48][t % 6]]] = marks[t % 4]
    b = torch.randn(E, generator=torch.Generator().manual_seed(3)) if bias else None
    for top in (1, 2):
        ids, w = _check(z, topk, score, b, groups, max(1, groups // 2), top if groups > 1 else 1)
        assert bool(torch.isfinite(w).all()) and bool((w[5] == 0).all()) and bool((w[11] == 0).all())
        assert all(len(set(r)) == topk for r in ids.tolist())


def test_infinite_logits_share_the_weight():
    z = torch.zeros(2, 16)
    z[0, 3] = z[0, 9] = float("inf")
    z[1, 2] = torch.finfo(F32).max
    ids, w = nvq.nv_moe_route(z.cuda(), 3)
    assert ids[0, :2].tolist() == [3, 9] and w[0].tolist() == [0.5, 0.5, 0.0]
    assert ids[1, 0].item() == 2 and w[1].tolist() == [1.0, 0.0, 0.0]


def test_a_bias_that_is_not_a_number_ranks_last():
    z = _logits(4, 20, F32, 2)
    b = torch.zeros(20)
    b[5] = float("nan")
    ids, w = nvq.nv_moe_route(z.cuda(), 19, "sigmoid", bias=b.cuda())
    assert not bool((ids == 5).any()) and bool(torch.isfinite(w).all())


def test_many_tokens_outputs_given_and_capture():
    z = _logits(3000, 64, BF16, 3).cuda()
    ids = torch.full((3000, 4), -1, dtype=torch.int32, device="cuda")
    w = torch.full((3000, 4), -1.0, device="cuda")
    a, b = nvq.nv_moe_route(z, 4, ids=ids, weights=w)
    assert a.data_ptr() == ids.data_ptr() and b.data_ptr() == w.data_ptr()
    _check(z.cpu(), 4)
    again, wagain = nvq.nv_moe_route(z, 4)
    assert torch.equal(again, ids) and torch.equal(wagain, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids2, w2 = nvq.nv_moe_route(z, 4)
    z.copy_(_logits(3000, 64, BF16, 4))
    graph.replay()
    torch.cuda.synchronize()
    want, ww = nvq.nv_moe_route(z, 4)
    assert torch.equal(ids2, want) and torch.equal(w2, ww)
    del graph


def test_refusals():
    z = torch.zeros(3, 24, dtype=BF16, device="cuda")
    for kw in (dict(topk=0), dict(topk=25), dict(topk=65), dict(topk=2, groups=5), dict(topk=2, groups=4, topk_groups=5),
               dict(topk=13, groups=4, topk_groups=2), dict(topk=2, group_top=3), dict(topk=2, groups=0)):
        with pytest.raises(nvq.NvqError):
            nvq.nv_moe_route(z, **kw)
    with pytest.raises(nvq.NvqError):
        nvq.nv_moe_route(z.half(), 2)
    with pytest.raises(nvq.NvqError):
        nvq.nv_moe_route(torch.zeros(2, 1024, device="cuda"), 2)
    for bad in (lambda: nvq.nv_moe_route(z, 2, "relu"), lambda: nvq.nv_moe_route(z[0], 2), lambda: nvq.nv_moe_route(z.cpu(), 2),
                lambda: nvq.nv_moe_route(z[:, ::2], 2), lambda: nvq.nv_moe_route(z, 2, bias=torch.zeros(24, device="cuda").half()),
                lambda: nvq.nv_moe_route(z, 2, ids=torch.zeros(3, 2, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    assert nvq.nv_moe_route(z[:0], 2)[0].shape == (0, 2)


def test_feeds_the_routed_block():
    """Router and routed block as a mixture-of-experts layer runs them."""
    import oracle as O
    E, I, K, T, topk = 8, 1024, 1024, 24, 2
    gate = O.quantize_affine(W.normal((E, I, K), 0.02, 1, "bf16"), 64, 4)
    up = O.quantize_affine(W.normal((E, I, K), 0.02, 2, "bf16"), 64, 4)
    down = O.quantize_affine(W.normal((E, K, I), 0.02, 3, "bf16"), 64, 4)
    x, wr = W.normal((T, K), 1.0, 4, "bf16"), W.normal((E, K), 0.05, 5, "bf16")
    z = x.cuda() @ wr.cuda().t()
    ids, rw = nvq.nv_moe_route(z, topk)
    y = nvq.nv_moe_swiglu(x.cuda(), *[tuple(t.cuda() for t in q) for q in (gate, up, down)], ids, rw, 64, 4)
    want, _ = _reference(z.cpu().double().numpy(), topk, "softmax", None, 1, 1, 1, True, 1.0)
    assert (ids.cpu().numpy() == want).all()
    yr, a = O.moe_swiglu(x, gate, up, down, ids.cpu().long(), rw.cpu(), 64, 4)
    assert bool(O.within_tolerance(y.cpu(), yr, a, BF16).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups,group_top", [
    (15, 3, 2, 1), (160, 8, 3, 2), (66, 11, 4, 2), (96, 32, 9, 1), (33, 33, 5, 1), (372, 3, 1, 2), (21, 7, 7, 2), (1023, 3, 2, 1)])
def test_groups_of_odd_sizes_to_the_last_expert(E, groups, topk_groups, group_top, score, dtype):
    """Every expert of the open groups is chosen (or 64 of them), masked ones last: none that does not exist."""
    topk = min(64, topk_groups * (E // groups))
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))
    z = _logits(50, E, dtype, E + 2)
    z[10:20, ::3] = -float("inf")
    z[20:30, : E // 2] = torch.finfo(torch.bfloat16).min
    z[30:35] = -float("inf")
    z[35:40] = 0.25  # ties everywhere
    for b in (None, bias):
        ids, _ = _check(z, topk, score, b, groups, topk_groups, group_top)
        assert bool((ids.sort(1).values.diff(dim=1) > 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("E,groups,group_top", [(1023, 1023, 1), (1008, 504, 2), (768, 768, 2), (752, 752, 1), (753, 753, 1), (1020, 510, 1)])
def test_hundreds_of_groups(E, groups, group_top, dtype):
    """The ranking of many groups keeps E + groups doubles a token: more than 48 KB of shared memory a block here."""
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))
    z = _logits(9, E, dtype, E + 3)
    for b in (None, bias):
        _check(z, 8, "sigmoid", b, groups, 20, group_top)
