"""Attention over the paged 8-bit cache (nv_kv_attention) against the 64-bit
reference, at the lengths, groups, masks and descriptors where it can go wrong."""
import pytest
import torch

import group_wise_affine_dequant_b200 as nvq
from tests import kv_reference as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _cache(P, H, block, D, mode, seed):
    """Codes that fill their range roughly normally, scales a few times apart from block to block."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(P, H, block, D, generator=g).double() * (R.LARGEST[mode] / 4)
    scales = (torch.exp(0.5 * torch.randn(P, H, generator=g)) * (4 / R.LARGEST[mode])).float()
    return R.nearest_codes(x, mode), scales


def _run(step, q, caches, mode, **kw):
    kraw, ks, vraw, vs = caches
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    want_flags = kw.pop("expect_flags", 0)
    qd = kw.pop("qd", None)
    got = nvq.nv_kv_attention(q.cuda() if qd is None else qd, kraw.view(R.MODES[mode]).cuda(), ks.cuda(),
                              vraw.view(R.MODES[mode]).cuda(), vs.cuda(), *step.dev(), out=out, flags=flags, **kw)
    torch.cuda.synchronize()
    assert int(flags) == want_flags and nvq.nv_pipeline_error() == 0
    return got.cpu()


def _check(step, H, G, D, mode, dtype, seed, causal=True, window=0, q_scale=1.0, scale=None, max_q=None, caches=None):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(step.rows, H * G, D, generator=g) * q_scale).to(dtype)
    if caches is None:
        caches = (*_cache(step.P, H, step.block, D, mode, seed + 1), *_cache(step.P, H, step.block, D, mode, seed + 2))
    got = _run(step, q, caches, mode, causal=causal, window=window, scale=scale,
               max_q=step.max_q if max_q is None else max_q)
    sc = D ** -0.5 if scale is None else scale
    out, *terms = R.attention(q, *caches, step, mode, sc, causal, window)
    room = R.attention_tolerance(out, terms, dtype, D, max(step.lens + [1]))
    lo, hi = int(step.starts[0]), int(step.starts[-1])
    err = (got.double() - out).abs()[lo:hi]
    bad = (~(err <= room[lo:hi])).nonzero()
    assert len(bad) == 0, (f"{len(bad)} of {err.numel()} off, first {bad[0].tolist()}: got {got[lo:hi][tuple(bad[0])]} want "
                           f"{out[lo:hi][tuple(bad[0])]} room {room[lo:hi][tuple(bad[0])]}")
    # rows of no sequence are left as they were
    assert bool((got[:lo] == 9.0).all()) and bool((got[hi:] == 9.0).all())
    return got


DECODE = [  # lens, block, H, G
    ([1], 16, 1, 1),
    ([17, 1, 300], 16, 2, 4),
    ([63, 64, 65, 128, 129], 64, 2, 8),
    ([1000, 0, 5], 32, 3, 7),
    ([2500, 130], 128, 1, 16),
    ([777], 64, 2, 2),
]


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (BF16, 80)])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_one_token(case, dtype, D, mode):
    lens, block, H, G = DECODE[case]
    news = [min(1, n) for n in lens]
    _check(R.Step(lens, news, block, seed=case, lead=case % 2, behind=case % 3), H, G, D, mode, dtype, 100 + case)


STEPS = [  # lens, news, block, H, G, window
    ([5], [5], 16, 1, 1, 0),
    ([40, 300, 7], [33, 2, 7], 16, 2, 4, 0),
    ([130, 0, 64, 260], [130, 0, 1, 70], 64, 2, 3, 0),
    ([300, 290], [300, 17], 128, 1, 8, 100),
    ([513], [400], 32, 2, 1, 33),
    ([257, 130, 129], [256, 129, 128], 64, 1, 5, 1),
    ([600, 1, 2], [3, 1, 2], 64, 2, 4, 0),
    ([200, 450], [2, 2], 32, 1, 24, 64),
]


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128), (BF16, 16)])
@pytest.mark.parametrize("case", range(len(STEPS)))
def test_steps_of_many_tokens(case, dtype, D, mode):
    lens, news, block, H, G, window = STEPS[case]
    _check(R.Step(lens, news, block, seed=case, lead=case % 3, behind=case % 2), H, G, D, mode, dtype, 200 + case,
           window=window)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("hint", [0, 1, 5, 10 ** 6])
def test_the_hint_changes_no_result_beyond_rounding(dtype, D, hint):
    _check(R.Step([300, 70, 9], [140, 5, 1], 64, seed=1), 2, 4, D, "int8", dtype, 300, max_q=hint)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("news", [[1, 1, 1], [40, 150, 3]])
def test_every_token_of_another_sequence(dtype, D, news):
    """causal = 0: queries of any number over an encoder's states, more than there are states among them."""
    _check(R.Step([100, 149, 3], [min(a, b) for a, b in zip(news, [100, 149, 3])], 32, seed=2), 2, 2, D, "e4m3", dtype, 310,
           causal=False)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64)])
@pytest.mark.parametrize("q_scale", [1e-20, 30.0, 3000.0])
def test_flat_and_peaked_rows(dtype, D, q_scale):
    """Scores from all alike to one that takes all the weight, tiny and large queries."""
    step = R.Step([700, 300], [1, 200], 64, seed=3)
    _check(step, 2, 4, D, "int8", dtype, 320, q_scale=q_scale)


@pytest.mark.parametrize("dtype,D,news", [(BF16, 128, 1), (BF16, 128, 300), (BF16, 64, 1), (BF16, 64, 300), (F32, 64, 9)])
def test_blocks_of_very_different_scales(dtype, D, news):
    """Value scales from 1e-12 to 1e6 and blocks of zeros, key scales of zero: a block that
    is large but hardly attended to hides nothing."""
    H, G, mode = 2, 4, "int8"
    step = R.Step([640], [news], 64, seed=4)
    kraw, ks = _cache(step.P, H, 64, D, mode, 1)
    vraw, vs = _cache(step.P, H, 64, D, mode, 2)
    ids = step.pages[0, :10].long()
    vs[ids] = torch.tensor([1e-3, 0.0, 1e-12, 1e6, 1e-3, 1e-8, 0.0, 1e2, 1e-4, 1e-2])[:, None].float()
    vraw[ids[1]] = 0
    vraw[ids[6]] = 0
    ks[ids[2]] = 0
    # keys against which every query scores far below the rest, where the values are huge
    kraw[ids[3]] = 0
    kraw[ids[3], :, :, 0] = 129  # -127
    g = torch.Generator().manual_seed(7)
    q = torch.randn(step.rows, H * G, D, generator=g)
    q[:, :, 0] = 60.0
    q = q.to(dtype)
    ks[ids[3]] = 0.05
    caches = (kraw, ks, vraw, vs)
    got = _run(step, q, caches, mode, max_q=news)
    out, *terms = R.attention(q, *caches, step, mode, D ** -0.5)
    room = R.attention_tolerance(out, terms, dtype, D, 640)
    err = (got.double() - out).abs()
    assert bool((err <= room).all()), float((err / room).max())


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("news", [1, 100])
def test_nothing_visible_and_garbage_out_of_sight(dtype, D, news):
    """Slots behind the last token and unused pages hold NaN codes and NaN scales, table
    entries behind the length are nonsense: nothing of it is seen."""
    H, G, mode = 1, 4, "e4m3"
    step = R.Step([201, 0, 130], [news, 0, min(news, 130)], 64, seed=5)
    caches = [*_cache(step.P, H, 64, D, mode, 1), *_cache(step.P, H, 64, D, mode, 2)]
    used = {int(p) for s in range(3) for p in step.pages[s, : -(-step.lens[s] // 64)]}
    for raw, sc in ((caches[0], caches[1]), (caches[2], caches[3])):
        for p in range(step.P):
            if p not in used:
                raw[p] = 0x7F
                sc[p] = float("nan")
        for s in (0, 2):
            raw[int(step.pages[s, step.lens[s] // 64]), :, step.lens[s] % 64:] = 0x7F
    _check(step, H, G, D, mode, dtype, 330, caches=tuple(caches))
    # queries for which nothing is left: a length of zero, or shorter than the step's rows
    q = torch.randn(50, G, D).to(dtype)
    short = R.Step([64, 64], [30, 20], 64, seed=6)
    for lens in ([0, 64], [10, 64], [0, 0]):
        short.lens_t = torch.tensor(lens, dtype=torch.int32)
        c = (*_cache(short.P, H, 64, D, mode, 1), *_cache(short.P, H, 64, D, mode, 2))
        got = _run(short, q, c, mode, max_q=30, expect_flags=R.LENGTH_FLAG)
        assert bool((got[: 30 - lens[0]] == 0).all()) and bool(torch.isfinite(got.float()).all())
        if lens[0]:
            assert bool((got[30 - lens[0]: 30].abs().sum((1, 2)) > 0).all())
        assert bool((got[30:].abs().sum((1, 2)) > 0).all()) == (lens[1] == 64)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("news", [1, 90])
def test_pages_out_of_range_are_not_seen(dtype, D, news):
    H, G, mode = 2, 2, "int8"
    step = R.Step([200, 100], [news, 1], 32, seed=7)
    caches = (*_cache(step.P, H, 32, D, mode, 1), *_cache(step.P, H, 32, D, mode, 2))
    good = step.pages.clone()
    q = torch.randn(step.rows, H * G, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    for bad in (-1, step.P, 2 ** 31 - 1):
        step.pages = good.clone()
        step.pages[0, 2] = bad
        got = _run(step, q, caches, mode, max_q=news, expect_flags=R.PAGE_FLAG)
        step.pages = good
        out, *terms = R.attention(q, *caches, step, mode, D ** -0.5, drop=lambda s, j: s == 0 and j // 32 == 2)
        room = R.attention_tolerance(out, terms, dtype, D, 200)
        assert bool(((got.double() - out).abs() <= room).all())
    for starts in ([0, 70, 60], [-3, 40, 60], [50, 10, 60], [0, 2 ** 31 - 1, -2 ** 31]):
        other = R.Step([200, 100], [news, 1], 32, seed=7)
        other.starts = torch.tensor(starts, dtype=torch.int32)
        _run(other, q, caches, mode, max_q=0, expect_flags=R.LENGTH_FLAG)


@pytest.mark.parametrize("dtype,D,news", [(BF16, 128, 1), (BF16, 128, 140), (BF16, 64, 140), (F32, 64, 3)])
def test_a_row_that_is_not_finite_stays_alone(dtype, D, news):
    H, G, mode = 1, 4, "int8"
    step = R.Step([300, 200], [news, 1], 64, seed=8)
    caches = (*_cache(step.P, H, 64, D, mode, 1), *_cache(step.P, H, 64, D, mode, 2))
    q = torch.randn(step.rows, G, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    clean = _run(step, q, caches, mode, max_q=news)
    q[0, 1, 5] = float("nan")
    q[0, 2, 6] = float("inf")
    got = _run(step, q, caches, mode, max_q=news)
    assert not bool(torch.isfinite(got[0, 1].float()).any())
    keep = torch.ones(step.rows, G, dtype=torch.bool)
    keep[0, 1] = keep[0, 2] = False
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("news", [1, 200])
def test_deterministic_strided_and_on_a_side_stream(news):
    H, G, D, mode = 2, 4, 128, "int8"
    step = R.Step([3000, 500], [news, min(news, 70)], 64, seed=9)
    caches = (*_cache(step.P, H, 64, D, mode, 1), *_cache(step.P, H, 64, D, mode, 2))
    wide = torch.randn(step.rows, H * G + 2 * H, D, generator=torch.Generator().manual_seed(1)).to(BF16)
    q = wide[:, : H * G]
    first = _run(step, q.contiguous(), caches, mode, max_q=news)
    assert torch.equal(_run(step, q, caches, mode, max_q=news, qd=wide.cuda()[:, : H * G]), first)
    need = nvq.nv_kv_attention_workspace_size(step.rows, H * G, H, 64, D, step.pages.shape[1], 2, news)
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dev = [t.cuda() for t in (q.contiguous(), caches[0].view(torch.int8), caches[1], caches[2].view(torch.int8), caches[3], *step.dev())]
    torch.cuda.synchronize()
    for _ in range(3):
        got = nvq.nv_kv_attention(*dev, max_q=news, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(got.cpu(), first)
    assert bool((ws[need:] == 255).all())


@pytest.mark.parametrize("news", [1, 150])
def test_capture_and_replay_with_new_lengths(news):
    H, G, D, mode = 2, 4, 128, "e4m3"
    step = R.Step([1500, 900], [news, 1], 64, seed=10)
    caches = (*_cache(step.P, H, 64, D, mode, 1), *_cache(step.P, H, 64, D, mode, 2))
    q = torch.randn(step.rows, H * G, D, generator=torch.Generator().manual_seed(1)).to(BF16)
    dev = [q.cuda(), caches[0].view(R.MODES[mode]).cuda(), caches[1].cuda(), caches[2].view(R.MODES[mode]).cuda(),
           caches[3].cuda(), *step.dev()]
    nvq.nv_kv_attention(*dev, max_q=news)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nvq.nv_kv_attention(*dev, max_q=news)
    for lens in ([1500, 900], [news, 1], [700, 64], [1111, 899]):
        dev[7].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        step.lens = lens
        want, *terms = R.attention(q, *caches, step, mode, D ** -0.5)
        room = R.attention_tolerance(want, terms, BF16, D, 1500)
        assert bool(((out.cpu().double() - want).abs() <= room).all()), lens
    assert nvq.nv_pipeline_error() == 0
    del graph


@pytest.mark.parametrize("news,D", [(1, 128), (60, 128), (1, 64), (60, 64)])
def test_offsets_past_32_bits(news, D):
    """Pages at the far end of a pool of more than 2^32 bytes of codes (K and V the same array)."""
    H, G, block = 8, 4, 128
    P = (1 << 32) // (H * D * block) + 40
    codes = torch.zeros(P, H, block, D, dtype=torch.int8, device="cuda")
    scales = torch.zeros(P, H, device="cuda")
    step = R.Step([300], [news], block)
    raw, sc = _cache(3, H, block, D, "int8", 3)
    small = R.Step([300], [news], block)
    small.pages = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    step.pages = torch.tensor([[P - 1, P - 3, P - 8]], dtype=torch.int32)
    codes[step.pages[0].long().cuda()] = raw.view(torch.int8).cuda()
    scales[step.pages[0].long().cuda()] = sc.cuda()
    q = torch.randn(news, H * G, D, generator=torch.Generator().manual_seed(1)).to(BF16)
    got = nvq.nv_kv_attention(q.cuda(), codes, scales, codes, scales, *step.dev(), max_q=news).cpu()
    out, *terms = R.attention(q, raw, sc, raw, sc, small, "int8", D ** -0.5)
    assert bool(((got.double() - out).abs() <= R.attention_tolerance(out, terms, BF16, D, 300)).all())


def test_refusals():
    step = R.Step([4], [4], 16)
    q = torch.zeros(4, 4, 64, dtype=BF16, device="cuda")
    kc = torch.zeros(step.P, 2, 16, 64, dtype=torch.int8, device="cuda")
    ks = torch.zeros(step.P, 2, device="cuda")
    d = step.dev()
    assert nvq.nv_kv_attention(q, kc, ks, kc, ks, *d).shape == (4, 4, 64)
    for bad in (dict(q=q.half()), dict(q=q[:, :3]), dict(window=-1), dict(window=4, causal=False), dict(max_q=-1)):
        a = dict(q=q, causal=True, window=0, max_q=0)
        a.update(bad)
        with pytest.raises(nvq.NvqError):
            nvq.nv_kv_attention(a["q"], kc, ks, kc, ks, *d, causal=a["causal"], window=a["window"], max_q=a["max_q"])
    for bad in (dict(q=q[:, :, :32]), dict(q=q.cpu()), dict(q=q[0]), dict(out=q.float()), dict(kc=kc.float())):
        a = dict(q=q, out=None, kc=kc)
        a.update(bad)
        with pytest.raises(ValueError):
            nvq.nv_kv_attention(a["q"], a["kc"], ks, a["kc"], ks, *d, out=a["out"])
    assert nvq.nv_kv_attention(q[:0], kc, ks, kc, ks, *d).shape == (0, 4, 64)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("news", [1, 70])
@pytest.mark.parametrize("block", [16, 128])
def test_pages_in_front_of_a_window_are_free(dtype, D, news, block):
    """A sliding window's pages in front of every row's first visible token may be given back: their
    entries are not asked for, nor is what they point to read."""
    H, G, window, mode = 2, 4, 100, "e4m3"
    lens = [700, 333]
    step = R.Step(lens, [news, 1], block, seed=11)
    caches = (*_cache(step.P, H, block, D, mode, 1), *_cache(step.P, H, block, D, mode, 2))
    q = torch.randn(step.rows, H * G, D, generator=torch.Generator().manual_seed(3)).to(dtype)
    out, *terms = R.attention(q, *caches, step, mode, D ** -0.5, True, window)
    room = R.attention_tolerance(out, terms, dtype, D, max(lens))
    free = [max(n - m + 1 - window, 0) // block for n, m in zip(lens, step.news)]
    dead = torch.cat([step.pages[s, : free[s]] for s in range(2)]).long()
    assert len(dead) > 0
    for raw, sc in ((caches[0], caches[1]), (caches[2], caches[3])):
        raw[dead] = 0x7F
        sc[dead] = float("nan")
    got = _run(step, q, caches, mode, causal=True, window=window, max_q=news)
    assert bool(((got.double() - out).abs() <= room).all())
    for s in range(2):
        step.pages[s, : free[s]] = -1
    got = _run(step, q, caches, mode, causal=True, window=window, max_q=news)
    assert bool(((got.double() - out).abs() <= room).all())


@pytest.mark.parametrize("news", [1, 17])
def test_the_longest_sequence(news):
    """2^31 - 2^16 tokens in two pages that the table repeats, the second from three quarters on: a
    softmax over two blocks whose weights carry counts. A longer length is cut and flagged.
    Tolerance: sums take 64 additions a chunk of 1024 tokens and 2^31 / 2^14 joins (few rows), or
    2^31 / 16 / 148 (many: 148 parts of the tokens, 16 a product); a product's sum may be cut, not rounded
    (2^-23 a step where a rounded one costs 2^-24), so half as many steps are added."""
    H, D, block, mode = 1, 64, 128, "int8"
    most = 2 ** 31 - 2 ** 16
    raw, sc = _cache(2, H, block, D, mode, 5)
    vraw, vs = _cache(2, H, block, D, mode, 6)
    blocks = most // block
    border = blocks * 3 // 4
    pages = torch.zeros(1, blocks + 1, dtype=torch.int32)
    pages[0, border:] = 1
    q = torch.randn(news, 1, D, generator=torch.Generator().manual_seed(1)).to(BF16)
    values = R.code_values(mode)
    k, v = (values[r.long()][:, 0] * s.double()[:, :, None] for r, s in ((raw, sc), (vraw, vs)))  # [2, block, D]
    z = torch.einsum("nd,pjd->npj", q[:, 0].double(), k) * D ** -0.5
    e = torch.exp(z - z.amax((1, 2), keepdim=True)) * torch.tensor([border, blocks - border], dtype=torch.float64)[:, None]
    p = e / e.sum((1, 2), keepdim=True)
    want, a = torch.einsum("npj,pjd->nd", p, v), torch.einsum("npj,pjd->nd", p, v.abs())
    dz = torch.einsum("nd,pjd->npj", q[:, 0].double().abs(), k.abs()).amax((1, 2))[:, None] * D ** -0.5
    steps = 64 + 2 ** 31 / 2 ** 14 if news == 1 else 2 ** 31 / 16 / 148
    room = R.attention_tolerance(want, (a, dz, torch.zeros(())), BF16, D, 16 * 1.5 * steps)
    dev = [raw.view(torch.int8).cuda(), sc.cuda(), vraw.view(torch.int8).cuda(), vs.cuda(), pages.cuda(),
           torch.tensor([0, news], dtype=torch.int32, device="cuda")]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for length, flag in ((most, 0), (2 ** 31 - 1, R.LENGTH_FLAG)):
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        got = nvq.nv_kv_attention(q.cuda(), *dev, lens, causal=False, max_q=news, flags=flags).cpu()[:, 0]
        assert int(flags) == flag and nvq.nv_pipeline_error() == 0
        err = (got.double() - want).abs()
        assert bool((err <= room).all()), float((err / room).max())


@pytest.mark.parametrize("news", [1, 40])
def test_a_given_stream_owns_the_memory_of_its_call(news):
    """While a call waits on a side stream, memory that the current stream allocates is not the call's workspace."""
    H, G, D, mode = 2, 4, 128, "int8"
    step = R.Step([30000], [news], 64, seed=12)
    caches = (*_cache(step.P, H, 64, D, mode, 1), *_cache(step.P, H, 64, D, mode, 2))
    q = torch.randn(step.rows, H * G, D, generator=torch.Generator().manual_seed(1)).to(BF16)
    want = _run(step, q, caches, mode, max_q=news)
    dev = [t.cuda() for t in (q, caches[0].view(torch.int8), caches[1], caches[2].view(torch.int8), caches[3], *step.dev())]
    need = nvq.nv_kv_attention_workspace_size(step.rows, H * G, H, 64, D, step.pages.shape[1], 1, news)
    assert need > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    got = nvq.nv_kv_attention(*dev, max_q=news, stream=side)
    mine = [torch.full((need,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((m == 7).all()) for m in mine) and torch.equal(got.cpu(), want)
    ids = nvq.nv_moe_route(torch.randn(64, 16, device="cuda"), 2, stream=side)[0]
    back = nvq.nv_kv_dequantize(*dev[1:], rows=step.rows, stream=side.cuda_stream)
    side.synchronize()
    assert ids.shape == (64, 2) and torch.equal(back[0], nvq.nv_kv_dequantize(*dev[1:], rows=step.rows)[0])


ONE_SUBTILE = [  # lens, news, block, H, G: items of at most 128 rows, with tokens for 0, 1, 2 and many tiles
    ([40, 128, 129, 300], [17, 20, 33, 64], 16, 2, 1),
    ([1000, 257, 5000], [5, 9, 16], 64, 2, 8),
    ([700, 2000], [40, 75], 128, 1, 7),  # 280 and 525 rows: a last tile of 24 and 13
    ([6000], [128], 32, 1, 1),
]


@pytest.mark.parametrize("dtype,D,mode", [(BF16, 128, "int8"), (BF16, 64, "e4m3"), (BF16, 128, "e4m3"), (BF16, 64, "int8")])
@pytest.mark.parametrize("case", range(len(ONE_SUBTILE)))
def test_items_of_one_subtile(case, dtype, D, mode):
    lens, news, block, H, G = ONE_SUBTILE[case]
    step = R.Step(lens, news, block, seed=case, lead=1, behind=2)
    _check(step, H, G, D, mode, dtype, 700 + case)
    _check(step, H, G, D, mode, dtype, 720 + case, causal=False)
    _check(step, H, G, D, mode, dtype, 740 + case, window=130)
    _check(step, H, G, D, mode, dtype, 760 + case, q_scale=30.0, max_q=0)


@pytest.mark.parametrize("D,mode", [(128, "int8"), (64, "e4m3")])
def test_both_kernels_in_a_row_of_calls(D, mode):
    """Calls of many-row and single-token sequences, cut into parts that are joined, one behind the other
    with one workspace, one cache and no gap: each gives what it gives alone."""
    H, G, block = 1, 4, 64
    cases = [([5000, 3000, 9000], [40, 1, 3]), ([9000, 700, 40, 4100], [1, 300, 1, 70]), ([2000, 2000], [4, 5])]
    steps = [R.Step(lens, news, block, seed=20 + i) for i, (lens, news) in enumerate(cases)]
    P = max(s.P for s in steps)
    caches = (*_cache(P, H, block, D, mode, 1), *_cache(P, H, block, D, mode, 2))
    dev = [t.cuda() for t in (caches[0].view(R.MODES[mode]), caches[1], caches[2].view(R.MODES[mode]), caches[3])]
    calls, want, need = [], [], 0
    for i, s in enumerate(steps):
        q = torch.randn(s.rows, H * G, D, generator=torch.Generator().manual_seed(30 + i)).to(BF16)
        out, *terms = R.attention(q, *caches, s, mode, D ** -0.5)
        calls.append((q.cuda(), s.dev(), s.max_q))
        alone = nvq.nv_kv_attention(calls[-1][0], *dev, *calls[-1][1], max_q=s.max_q)
        torch.cuda.synchronize()
        room = R.attention_tolerance(out, terms, BF16, D, max(s.lens))
        assert bool(((alone.cpu().double() - out).abs() <= room).all())
        want.append(alone)
        need = max(need, nvq.nv_kv_attention_workspace_size(s.rows, H * G, H, block, D, s.pages.shape[1], len(s.lens), s.max_q))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def row():
        return [nvq.nv_kv_attention(q, *dev, *d, max_q=m, workspace=ws) for _ in range(6) for q, d, m in calls]

    for got in (row(), None):
        if got is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = row()
            for _ in range(3):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))
    assert nvq.nv_pipeline_error() == 0
    del graph


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("news", [1, 60])
@pytest.mark.parametrize("size", [2.0 ** 112, 2.0 ** 116, 1e36, 3e37, 2.0 ** -112, 2.0 ** -118, 1e-36, 1e-38, 1e-39])
def test_queries_at_the_ends_of_the_range(size, news, D, mode):
    """Queries up to the largest bf16 and down to its subnormals, against keys that bring the scores back
    to about 1. (Queries become fp16 times a power of two exactly here: no room is added for them.)"""
    H, G = 1, 4
    step = R.Step([300], [news], 64, seed=13)
    kraw, ks = _cache(step.P, H, 64, D, mode, 1)
    caches = (kraw, (ks.double() / size).clamp_max(1e36).float(), *_cache(step.P, H, 64, D, mode, 2))
    q = (torch.randn(step.rows, H * G, D, generator=torch.Generator().manual_seed(3)).double() * size).to(BF16)
    if size > 1:
        q[0, 0, 0] = torch.finfo(BF16).max
    for scale in (D ** -0.5, -D ** -0.5):
        got = _run(step, q, caches, mode, scale=scale, max_q=news)
        out, *terms = R.attention(q, *caches, step, mode, scale)
        room = R.attention_tolerance(out, terms, BF16, D, 300)
        err = (got.double() - out).abs()
        assert bool((err <= room).all()), float((err / room).max())


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 256), (BF16, 80), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("news", [1, 40])
@pytest.mark.parametrize("size", [2.0 ** 114, 3e37, 2.0 ** -112, 1e-38, 1e-39])
def test_queries_and_values_at_the_ends_of_the_range(size, news, dtype, D, mode):
    """Every kernel: queries as above, and values up to the largest number or down to the smallest normal
    ones, whose sum over the tokens would leave the range. Results below 1e-30 only have to be finite."""
    H, G = 1, 2
    step = R.Step([300], [news], 64, seed=14)
    kraw, ks = _cache(step.P, H, 64, D, mode, 1)
    vraw, vs = _cache(step.P, H, 64, D, mode, 2)
    vs = vs * (3e38 / R.LARGEST[mode] / float(vs.max()) if size > 1 else 2.0 ** -110)
    caches = (kraw, (ks.double() / size).clamp_max(1e36).float(), vraw, vs)
    q = (torch.randn(step.rows, H * G, D, generator=torch.Generator().manual_seed(3)).double() * size).to(dtype)
    if size > 1:
        q[0, 0, 0] = 3.3e38
    got = _run(step, q, caches, mode, max_q=news)
    out, *terms = R.attention(q, *caches, step, mode, D ** -0.5)
    room = R.attention_tolerance(out, terms, dtype, D, 300)
    err = (got.double() - out).abs()
    assert bool((err <= room).all()), float((err / room).max())


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("news,H,G,block,causal,window", [
    (1, 2, 4, 64, True, 0), (3, 1, 4, 16, True, 0), (2, 2, 8, 32, True, 300), (1, 1, 16, 128, False, 0),  # few rows
    (200, 1, 4, 64, True, 0), (90, 2, 1, 16, True, 250), (40, 1, 2, 128, False, 0), (700, 8, 8, 64, True, 0)])  # many; parts and one
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 27, 2.0 ** 60, 2.0 ** 110, 2.0 ** 124, 2.0 ** -20, 2.0 ** -60, 2.0 ** -110])
def test_values_of_another_size(size, news, H, G, block, causal, window, D, mode):
    """A cache written from values of about 1, but for a block of zeros, a token (or, where they are smaller,
    a block) in the middle that weighs next to nothing, and the last token, which only the last row
    sees. A large value leaves the other codes of its block 0. Rows that do not see it, or see another block's values
    beside it, are as exact as ever: no room is left for the size of a block's scale, but what the
    weights' 2^-33 of it are where it is at most 2^24 times another's."""
    n = 700
    whole, step = R.Step([n], [n], block, seed=15), R.Step([n], [news], block, seed=15)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(n, H, D, generator=g).double() for _ in range(2))
    q = torch.randn(step.rows, H * G, D, generator=g).to(BF16)
    mid = n // 2 + 5
    v[block * 2: block * 3] = 0
    if size > 1:
        v[mid] *= size
        k[:, :, 0], q[:, :, 0] = 0, 30
        k[mid, :, 0] = -60
    else:
        v[mid // block * block: (mid // block + 1) * block] *= size
    v[n - 1] *= size
    zeros = torch.zeros(step.P, H, block, D, dtype=torch.uint8), torch.zeros(step.P, H)
    caches = (*R.write(k.float(), *zeros, whole, mode), *R.write(v.float(), *zeros, whole, mode))
    got = _run(step, q, caches, mode, causal=causal, window=window, max_q=news)
    out, a, dz, small = R.attention(q, *caches, step, mode, D ** -0.5, causal, window)
    near = 2.0 ** -24 <= size <= 2.0 ** 24
    room = R.attention_tolerance(out, (a, dz, small if near else small * 0), BF16, D, n)
    err = (got.double() - out).abs()
    assert bool((err <= room).all()), float((err / room).max())


@pytest.mark.parametrize("D,mode", [(128, "int8"), (64, "e4m3"), (80, "int8")])
@pytest.mark.parametrize("news", [[1, 1, 1], [40, 3, 20], [2, 300, 1]])
def test_a_sequence_does_not_depend_on_its_neighbours(news, D, mode):
    """In calls of the same sizes a sequence's rows are the same bits whatever the other sequences' lengths, contents
    and places are. (Alone, or beside more or fewer, it may be cut into other parts.)"""
    H, G, block, n = 2, 4, 64, 5000
    first = R.Step([n, 300, 900], news, block, seed=16)
    P, width = 400, first.pages.shape[1]
    caches = [*_cache(P, H, block, D, mode, 1), *_cache(P, H, block, D, mode, 2)]
    q = torch.randn(first.rows, H * G, D, generator=torch.Generator().manual_seed(1)).to(BF16)
    want = _run(first, q, caches, mode, max_q=max(news))
    spare = [p for p in range(P) if p not in set(first.pages[0].tolist())]
    for place, others in ((0, [4000, 25]), (1, [700, 4900]), (2, [300, 64])):
        order = [1, 2]
        order.insert(place, 0)
        lens = list(others)
        lens.insert(place, n)
        step = R.Step([max(a, news[b]) for a, b in zip(lens, order)], [news[b] for b in order], block, seed=17)
        table = torch.full((3, width), -7, dtype=torch.int32)
        table[place] = first.pages[0]
        at = 0
        for s in range(3):
            if s != place:
                k = -(-step.lens[s] // block)
                table[s, :k] = torch.tensor(spare[at: at + k], dtype=torch.int32)
                at += k
        step.pages = table
        rows = torch.randn(step.rows, H * G, D, generator=torch.Generator().manual_seed(20 + place)).to(BF16)
        r0 = int(step.starts[place])
        rows[r0: r0 + news[0]] = q[: news[0]]
        got = _run(step, rows, caches, mode, max_q=max(news))
        assert torch.equal(got[r0: r0 + news[0]], want[: news[0]]), place


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (BF16, 80)])
@pytest.mark.parametrize("news", [1, 70])
@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("far", [False, True])
def test_an_infinite_query_gives_no_number(what, news, dtype, D, far):
    """Also where every score becomes -infinity, as if nothing were seen; in every kernel, and where value scales are far apart."""
    H, G, mode = 1, 4, "int8"
    step = R.Step([150], [news], 64, seed=18)
    caches = [*_cache(step.P, H, 64, D, mode, 1), *_cache(step.P, H, 64, D, mode, 2)]
    caches[0][..., 3] = 5 if what < 0 else 251  # keys of the other sign there
    if far:
        caches[3][step.pages[0, 0]] *= 2.0 ** 60
    q = torch.randn(step.rows, G, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    clean = _run(step, q, caches, mode, max_q=news)
    assert bool(torch.isfinite(clean.float()).all())
    q[0, 2, 3] = what
    got = _run(step, q, caches, mode, max_q=news)
    assert not bool(torch.isfinite(got[0, 2].float()).any())
    got[0, 2] = clean[0, 2]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64), (BF16, 80)])
@pytest.mark.parametrize("mode", ["int8", "e4m3"])
@pytest.mark.parametrize("news", [2, 70])
@pytest.mark.parametrize("size", [1.0, 500.0, 4000.0, 5e5])
def test_a_key_of_the_largest_size_out_of_sight(size, news, mode, dtype, D):
    """The last token's key is near the largest number, which leaves the other codes of its block 0: to the rows in
    front of it, of queries large and small, those are scores of 0."""
    H, G, n = 1, 4, 150
    step = R.Step([n], [news], 64, seed=19)
    caches = [*_cache(step.P, H, 64, D, mode, 1), *_cache(step.P, H, 64, D, mode, 2)]
    last = int(step.pages[0, (n - 1) // 64])
    caches[0][last] = 0
    caches[0][last, :, (n - 1) % 64] = 100
    caches[1][last] = 3.38e38 / R.LARGEST[mode]
    caches[1][step.pages[0, :2].long()] /= size
    q = (torch.randn(step.rows, G, D, generator=torch.Generator().manual_seed(1)) * size).to(dtype)
    got = _run(step, q, caches, mode, max_q=news)[:-1]
    out, *terms = R.attention(q, *caches, step, mode, D ** -0.5)
    room = R.attention_tolerance(out, terms, dtype, D, n)[:-1]
    err = (got.double() - out[:-1]).abs()
    assert bool((err <= room).all()), float((err / room).max())
