"""The paged 8-bit key/value cache on the GPU against the 64-bit reference:
nv_kv_quantize byte for byte over the whole pool (what a step must not touch
included), nv_kv_dequantize to one rounding."""
import pytest
import torch

import group_wise_affine_dequant_b200 as nvq
from tests import kv_reference as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _rows(step, H, D, dtype, seed, spread=1.0):
    """k and v as slices of one wider tensor, values over several binades."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(max(step.rows, 1), 3 * H, D, generator=g)
    x = x * torch.exp(spread * torch.randn(max(step.rows, 1), 3 * H, 1, generator=g))
    return x.to(dtype)[: step.rows]


def _write_case(step, H, D, mode, dtype, seed, x=None, expect_flags=0):
    x = _rows(step, H, D, dtype, seed) if x is None else x
    xd = x.cuda()
    kraw, ks = R.empty_cache(step.P, H, step.block, D, mode, seed + 1)
    vraw, vs = R.empty_cache(step.P, H, step.block, D, mode, seed + 2)
    kc, vc = (t.view(R.MODES[mode]).cuda() for t in (kraw, vraw))
    ksd, vsd = ks.cuda(), vs.cuda()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    nvq.nv_kv_quantize(xd[:, H:2 * H], xd[:, 2 * H:], kc, ksd, vc, vsd, *step.dev(), flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == expect_flags
    for name, x1, raw, sc, got, gs in (("k", x[:, H:2 * H], kraw, ks, kc, ksd), ("v", x[:, 2 * H:], vraw, vs, vc, vsd)):
        want, wants = R.write(x1, raw, sc, step, mode)
        assert torch.equal(gs.cpu(), wants), f"{name} scales: {(gs.cpu() != wants).nonzero()[:3].tolist()}"
        bad = (got.cpu().view(torch.uint8) != want).nonzero()
        assert len(bad) == 0, f"{name} codes: {len(bad)} differ, first {bad[0].tolist()}"
    return kc, ksd, vc, vsd


CASES = [  # lens, news, block, H, D
    ([1], [1], 16, 1, 16),
    ([5, 17, 33], [5, 1, 2], 16, 2, 64),
    ([64, 65, 63, 128], [1, 1, 1, 1], 64, 2, 128),
    ([200, 0, 7, 129, 50], [130, 0, 7, 129, 0], 64, 3, 128),
    ([300], [300], 128, 1, 256),
    ([257, 40], [255, 33], 128, 2, 48),
    ([31, 95], [30, 70], 32, 8, 80),
]


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_write_is_exact(case, dtype, mode):
    lens, news, block, H, D = CASES[case]
    _write_case(R.Step(lens, news, block, seed=case, lead=case % 2, behind=case % 3), H, D, mode, dtype, 10 * case)


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
def test_token_by_token_follows_the_rule(mode):
    """Forty single-token steps into two sequences: scales only grow, held codes
    are rounded again, every step byte for byte."""
    H, D, block = 2, 32, 16
    kraw = ks = None
    for t in range(1, 41):
        step = R.Step([t, t + 3], [1, 1], block, seed=5, spare_pages=40)
        step.pages = torch.arange(2 * 4, dtype=torch.int32).view(2, 4)  # the same pages every step
        x = _rows(step, H, D, F32, 100 + t, spread=1.5)
        if kraw is None:
            kraw, ks = R.empty_cache(step.P, H, block, D, mode, 1)
            kraw[4:5] = 0  # the second sequence starts three tokens in: zeros with scale 0
            ks[4:5] = 0
            P = step.P
            kc, vc = kraw.view(R.MODES[mode]).cuda(), kraw.view(R.MODES[mode]).cuda()
            ksd, vsd = ks.cuda(), ks.cuda()
        k = x[:, :H].cuda()
        nvq.nv_kv_quantize(k, k, kc, ksd, vc, vsd, *step.dev())
        kraw, ks = R.write(x[:, :H], kraw, ks, step, mode)
        assert kraw.shape[0] == P
        assert torch.equal(ksd.cpu(), ks) and torch.equal(kc.cpu().view(torch.uint8), kraw), t
        assert torch.equal(vsd.cpu(), ks) and torch.equal(vc.cpu().view(torch.uint8), kraw), t


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
def test_ties_extremes_and_non_finite_values(mode):
    """Quotients on and next to ties, zeros, subnormal and huge blocks, NaN and infinities."""
    D, H, block = 64, 1, 16
    step = R.Step([16 * 9], [16 * 9], block, seed=3)
    x = torch.zeros(step.rows, 3 * H, D)
    top = R.LARGEST[mode]
    half = torch.arange(D) + 0.5 if mode == "int8" else torch.arange(1, D + 1) * 2.0 ** -10
    scale = torch.tensor(0.37, dtype=F32)
    up = (half.float() * scale)
    for i, y in enumerate((half.float(), up, torch.nextafter(up, torch.tensor(9e9)), torch.nextafter(up, torch.zeros(())),
                           half.float() * 1e-38, half.float() * 2.0 ** -140, half.float() * 1e36, half.float(), torch.zeros(D))):
        x[16 * i, :] = y.clamp_max(3e38)
        x[16 * i + 1, :] = -y
        x[16 * i + 2, :, 0] = {0: top, 1: float(top * scale), 2: float(top * scale), 3: float(top * scale)}.get(i, 0.0)
    if mode == "e4m3":  # every tie between neighbouring codes
        values = R.code_values(mode)[:127]
        ties = ((values[1:] + values[:-1]) / 2).float()
        x[3, :, : 64] = ties[:64]
        x[4, :, : 62] = ties[64:126]
    x[16 * 7 + 3, :, 1] = float("inf")
    x[16 * 7 + 4, :, 2] = float("-inf")
    x[16 * 7 + 5, :, 3] = float("nan")
    x[16 * 8 + 1, :, 3] = float("nan")
    x[16 * 8 + 2, :, 3] = float("inf")
    want_inf = x.clone()
    # the reference saturates an infinity; a block without finite values has scale 0 and codes 0
    _write_case(step, H, D, mode, F32, 40, x=want_inf)


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_read_back(mode, dtype):
    H, D, block = 3, 80, 32
    lens = [1, 0, 77, 200]
    for news in (lens, [1, 0, 5, 170]):
        step = R.Step(lens, news, block, seed=8, lead=2, behind=3)
        kraw, ks = R.empty_cache(step.P, H, block, D, mode, 1)
        vraw, vs = R.empty_cache(step.P, H, block, D, mode, 2)
        out = [torch.full((step.rows, H, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        k, v = nvq.nv_kv_dequantize(kraw.view(R.MODES[mode]).cuda(), ks.cuda(), vraw.view(R.MODES[mode]).cuda(), vs.cuda(),
                                    *step.dev(), rows=step.rows, dtype=dtype, out=out, flags=flags)
        torch.cuda.synchronize()
        assert int(flags) == 0
        for got, raw, sc in ((k, kraw, ks), (v, vraw, vs)):
            want = torch.full((step.rows, H, D), 7.0, dtype=torch.float64)
            for s in range(len(lens)):
                a, b = int(step.starts[s]), int(step.starts[s + 1])
                want[a:b] = R.read(raw, sc, step, mode, s)[lens[s] - news[s]:]
            want32 = want.to(F32)  # the fp32 product is the exact one rounded once
            assert torch.equal(got.cpu(), want32.to(dtype))


def test_written_tokens_come_back_within_half_a_step():
    H, D, block = 2, 128, 64
    step = R.Step([130, 64, 1], [130, 64, 1], block, seed=4)
    x = _rows(step, H, D, F32, 50, spread=0.0)
    for mode in ("int8", "e4m3"):
        cache = _write_case(step, H, D, mode, F32, 60, x=x)
        k, v = nvq.nv_kv_dequantize(*cache, *step.dev(), rows=step.rows, dtype=F32)
        for got, want, sc in ((k, x[:, H:2 * H], cache[1]), (v, x[:, 2 * H:], cache[3])):
            for s in range(3):
                for row, page, _ in step.tokens(s):
                    scale = sc[page].cpu()[:, None]
                    # int8: half a step; E4M3: 2^-4 of the value, or half its smallest step
                    err, w = (got[row].cpu() - want[row]).abs(), want[row].abs()
                    room = scale * 0.5 if mode == "int8" else torch.maximum(w * 2.0 ** -4, scale * 2.0 ** -10)
                    assert bool((err <= room * (1 + 2.0 ** -20)).all()), (mode, row)


def test_bad_descriptors_are_flagged_and_stay_inside():
    """Pages out of range, lengths that do not fit, starts that do not ascend:
    the rest of the pool keeps its bytes, rows read back as zeros."""
    H, D, block, mode = 2, 64, 16, "int8"
    step = R.Step([40, 20], [40, 20], block, seed=2)
    good = step.pages.clone()
    x = _rows(step, H, D, BF16, 7)
    for bad in (-1, step.P, 2 ** 31 - 1, -2 ** 31):
        step.pages = good.clone()
        step.pages[0, 1] = bad
        kraw, ks = R.empty_cache(step.P, H, block, D, mode, 1)
        kc, ksd = kraw.view(torch.int8).cuda(), ks.cuda()
        vc, vsd = kc.clone(), ksd.clone()
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        xd = x.cuda()
        nvq.nv_kv_quantize(xd[:, :H], xd[:, :H], kc, ksd, vc, vsd, *step.dev(), flags=flags)
        assert int(flags) == R.PAGE_FLAG
        touched = {int(p) for s in range(2) for _, p, _ in step.tokens(s) if 0 <= p < step.P}
        for p in range(step.P):
            if p not in touched:
                assert torch.equal(kc[p].cpu().view(torch.uint8), kraw[p])
        k, _ = nvq.nv_kv_dequantize(kc, ksd, vc, vsd, *step.dev(), rows=step.rows, flags=flags)
        assert bool((k[16:32] == 0).all()) and bool((k[:16] != 0).any()) and bool((k[32:] != 0).any())
    # a length shorter than the step's rows: the rows that fit are its last ones
    pages, starts, _ = good.cuda(), step.starts.cuda(), None
    for lens in ([30, 20], [-5, 20], [0, 20], [2 ** 31 - 1, 20]):
        flags.zero_()
        before = kc.clone()
        lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        nvq.nv_kv_quantize(xd[:, :H], xd[:, :H], kc, ksd, vc, vsd, pages, starts, lens_t, flags=flags)
        assert int(flags) & R.LENGTH_FLAG
        unused = [p for p in range(step.P) if p not in set(good[:, :3].flatten().tolist())]
        assert all(torch.equal(kc[p], before[p]) for p in unused)
        k, _ = nvq.nv_kv_dequantize(kc, ksd, vc, vsd, pages, starts, lens_t, rows=step.rows, flags=flags)
        if 0 <= lens[0] < 40:
            assert bool((k[: 40 - lens[0]] == 0).all())
    lens_t = torch.tensor([40, 20], dtype=torch.int32, device="cuda")
    for starts in ([0, 70, 60], [-3, 40, 60], [50, 10, 60], [0, 2 ** 31 - 1, -2 ** 31]):
        flags.zero_()
        starts_t = torch.tensor(starts, dtype=torch.int32, device="cuda")
        nvq.nv_kv_quantize(xd[:, :H], xd[:, :H], kc, ksd, vc, vsd, pages, starts_t, lens_t, flags=flags)
        nvq.nv_kv_dequantize(kc, ksd, vc, vsd, pages, starts_t, lens_t, rows=step.rows, flags=flags)
        assert int(flags) & R.LENGTH_FLAG
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes of codes, written and read at its far end."""
    H, D, block = 8, 128, 128
    P = (1 << 32) // (H * D * block) + 40
    kc = torch.zeros(P, H, block, D, dtype=torch.int8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = (torch.zeros(P, H, device="cuda") for _ in range(2))
    step = R.Step([200], [200], block)
    step.pages = torch.tensor([[P - 1, P - 3]], dtype=torch.int32)
    x = _rows(step, H, D, BF16, 70).cuda()
    nvq.nv_kv_quantize(x[:, :H], x[:, H:2 * H], kc, ks, vc, vs, *step.dev())
    k, v = nvq.nv_kv_dequantize(kc, ks, vc, vs, *step.dev(), rows=200, dtype=F32)
    small = R.Step([200], [200], block)
    raw, sc = R.empty_cache(small.P, H, block, D, "int8", 3)
    raw, sc = R.write(x[:, :H].cpu(), raw, sc, small, "int8")
    assert torch.equal(k.cpu(), R.read(raw, sc, small, "int8", 0).to(F32))
    assert int((kc[: P - 3] != 0).sum()) == 0 and int((kc[P - 2] != 0).sum()) == 0
    assert bool((v != 0).any())


def test_capture_replay_and_a_side_stream():
    """A captured step of a growing sequence: the same graph, new lengths and values."""
    H, D, block = 2, 64, 16
    kc = torch.zeros(8, H, block, D, dtype=torch.int8, device="cuda")
    vc, ks = torch.zeros_like(kc), torch.zeros(8, H, device="cuda")
    vs = torch.zeros_like(ks)
    pages = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1], dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 2 * H, D, dtype=BF16, device="cuda")
    nvq.lib()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        nvq.nv_kv_quantize(x[:, :H], x[:, H:], kc, ks, vc, vs, pages, starts, lens)
        k, v = nvq.nv_kv_dequantize(kc, ks, vc, vs, pages, starts, lens, rows=1, dtype=F32)
    g = torch.Generator().manual_seed(0)
    raw, sc = torch.zeros(8, H, block, D, dtype=torch.uint8), torch.zeros(8, H)
    for n in range(1, 40):
        value = torch.randn(1, 2 * H, D, generator=g).to(BF16)
        x.copy_(value)
        lens.fill_(n)
        graph.replay()
        step = R.Step([n], [1], block)
        step.pages = pages.cpu()
        raw, sc = R.write(value[:, :H], raw, sc, step, "int8")
        assert torch.equal(kc.cpu().view(torch.uint8), raw) and torch.equal(ks.cpu(), sc)
        assert torch.equal(k.cpu(), R.read(raw, sc, step, "int8", 0)[n - 1:].to(F32))
    del graph


def test_refusals():
    step = R.Step([4], [4], 16)
    x = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    kc = torch.zeros(step.P, 2, 16, 64, dtype=torch.int8, device="cuda")
    ks = torch.zeros(step.P, 2, device="cuda")
    d = step.dev()
    nvq.nv_kv_quantize(x, x, kc, ks, kc.clone(), ks.clone(), *d)
    for bad in (dict(kc=kc.float()), dict(kc=kc[:, :1]), dict(ks=ks[:, :1]), dict(ks=ks.double()), dict(x=x[:, :1]),
                dict(x=x.transpose(0, 1)), dict(d=(d[0].long(), d[1], d[2])), dict(d=(d[0], d[1][:1], d[2])),
                dict(x=x.cpu()), dict(x=x[:, :, ::2])):
        a = dict(x=x, kc=kc, ks=ks, d=d)
        a.update(bad)
        with pytest.raises(ValueError):
            nvq.nv_kv_quantize(a["x"], a["x"], a["kc"], a["ks"], a["kc"], a["ks"], *a["d"])
    with pytest.raises(nvq.NvqError):  # fp16 values
        nvq.nv_kv_quantize(x.half(), x.half(), kc, ks, kc, ks, *d)
    odd = torch.zeros(4 * 130 + 1, dtype=BF16, device="cuda")
    with pytest.raises(nvq.NvqError):  # rows not 16 bytes apart
        nvq.nv_kv_quantize(*[odd[: 4 * 130].view(4, 130)[:, :128].unflatten(1, (2, 64))] * 2, kc, ks, kc, ks, *d)
    with pytest.raises(nvq.NvqError):  # base not on 16 bytes
        nvq.nv_kv_quantize(*[odd[1:513].view(4, 2, 64)] * 2, kc, ks, kc, ks, *d)
    with pytest.raises(nvq.NvqError):
        nvq.nv_kv_dequantize(kc, ks, kc, ks, *d, rows=4, dtype=torch.float16)
    assert nvq.nv_kv_dequantize(kc, ks, kc, ks, *d, rows=0)[0].shape == (0, 2, 64)


@pytest.mark.parametrize("mode", ["int8", "e4m3"])
def test_the_ends_of_the_fp32_range(mode):
    """Blocks whose scale is a subnormal of a few bits, so that their largest value lies above the
    largest code times it, and an infinity beside the largest float, whose code times scale overflows."""
    D, H, block = 32, 1, 16
    units = [1, 63, 64, 127, 190, 191, 254, 300, 700, 1000, 5000, 16065, 40000, 100000]
    step = R.Step([16 * (len(units) + 2)], [16 * (len(units) + 2)], block, seed=4)
    x = torch.zeros(step.rows, 3 * H, D)
    g = torch.Generator().manual_seed(2)
    for i, n in enumerate(units):
        share = torch.randint(-n, n + 1, (16, 3 * H, D), generator=g)
        share[3, :, 5], share[4, :, 6] = n, -n
        x[16 * i: 16 * i + 16] = (share.double() * 2.0 ** -149).float()
    most = torch.finfo(F32).max
    x[-32:] = torch.randn(32, 3 * H, D, generator=g) * 1e37
    x[-30, :, 3], x[-29, :, 4] = most, float("inf")
    x[-12, :, 3], x[-11, :, 4] = -most, float("-inf")
    _write_case(step, H, D, mode, F32, 50, x=x)
