"""Plain 64-bit counterparts of the key/value cache and attention calls, on the
CPU, and the step descriptors their tests share. Nothing here is taken from the
kernels: codes come from a search over all representable values."""
from __future__ import annotations

import math

import torch

MODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
LARGEST = {"int8": 127.0, "e4m3": 448.0}
PAGE_FLAG, LENGTH_FLAG = 0x8, 0x10


def code_values(mode: str) -> torch.Tensor:
    """The value of each of the 256 byte codes (float64; NaN codes are NaN)."""
    raw = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    return raw.view(MODES[mode]).to(torch.float64)


def nearest_codes(x: torch.Tensor, mode: str) -> torch.Tensor:
    """uint8 code nearest to each float64 x: ties to the even code, saturated, NaN -> 0."""
    x = torch.where(torch.isnan(x), torch.zeros_like(x), x)
    values = code_values(mode)[:128]  # non-negative codes ascend with the byte
    top = int(LARGEST[mode]) if mode == "int8" else 126
    values = values[: top + 1]
    size = x.abs().clamp_max(LARGEST[mode])
    above = torch.searchsorted(values, size).clamp_max(top)
    below = (above - 1).clamp_min(0)
    d_above, d_below = values[above] - size, size - values[below]
    up = (d_above < d_below) | ((d_above == d_below) & (above % 2 == 0))
    code = torch.where(up, above, below)
    if mode == "int8":
        return torch.where(x < 0, -code, code).to(torch.int8).view(torch.uint8)
    return (code + torch.where(torch.signbit(x), 128, 0)).to(torch.uint8)


class Step:
    """Lengths, rows and a shuffled page table (spare entries hold nonsense)."""

    def __init__(self, lens, news, block, seed=0, spare_pages=2, spare_columns=2, lead=0, behind=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.news, self.block = list(lens), list(news), block
        counts = [-(-n // block) for n in lens]
        self.P = sum(counts) + spare_pages
        order = torch.randperm(self.P, generator=g).tolist()
        width = max(counts + [0]) + spare_columns
        self.pages = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for i, n in enumerate(counts):
            self.pages[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        starts = [lead]
        for n in news:
            starts.append(starts[-1] + n)
        self.starts = torch.tensor(starts, dtype=torch.int32)
        self.rows = starts[-1] + behind
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32)
        self.max_q = max(list(news) + [0])

    def dev(self):
        return self.pages.cuda(), self.starts.cuda(), self.lens_t.cuda()

    def tokens(self, s):
        """(row, page, slot) of each of sequence s's rows of this step."""
        first = self.lens[s] - self.news[s]
        for i in range(self.news[s]):
            p = first + i
            if p >= 0:
                yield int(self.starts[s]) + i, int(self.pages[s, p // self.block]), p % self.block


def empty_cache(P, H, block, D, mode, seed):
    """A cache of random codes and scales (bytes that a write must leave or overwrite exactly)."""
    g = torch.Generator().manual_seed(seed)
    raw = torch.randint(0, 256, (P, H, block, D), generator=g, dtype=torch.int32)
    if mode == "e4m3":
        raw = torch.where(raw % 128 == 127, raw - 1, raw)  # the writer makes no NaN codes
    else:
        raw = torch.where(raw == 128, torch.full_like(raw, 127), raw)  # nor -128
    scales = torch.exp(torch.randn(P, H, generator=g)) * 0.01
    return raw.to(torch.uint8), scales.to(torch.float32)


def write(x, raw, scales, step: Step, mode: str):
    """nv_kv_quantize of one of K and V, on copies: (codes uint8, scales)."""
    raw, scales = raw.clone(), scales.clone()
    values, top = code_values(mode), torch.tensor(LARGEST[mode], dtype=torch.float32)
    for s in range(len(step.lens)):
        blocks = {}
        for row, page, slot in step.tokens(s):
            blocks.setdefault(page, []).append((row, slot))
        for page, items in blocks.items():
            rows, slots = [r for r, _ in items], [t for _, t in items]
            new = x[rows].to(torch.float32)  # [n, H, D]
            size = torch.where(torch.isfinite(new), new.abs(), torch.zeros_like(new))
            need = size.amax((0, 2)) / top
            held = slots[0]
            scale = torch.maximum(scales[page], need) if held else need
            if held:
                old = values[raw[page, :, :held].long()] * scales[page].double()[:, None, None]
                grown = scale > scales[page]
                again = nearest_codes(old / scale.double().clamp_min(1e-300)[:, None, None], mode)
                raw[page, :, :held] = torch.where(grown[:, None, None], again, raw[page, :, :held])
            scales[page] = scale
            divisor = scale.double()[None, :, None]
            q = torch.where(divisor > 0, new.double() / divisor.clamp_min(1e-300), torch.zeros(()).double())
            raw[page][:, slots] = nearest_codes(q, mode).transpose(0, 1)
    return raw, scales


def read(raw, scales, step: Step, mode: str, s: int, upto=None):
    """float64 [tokens, H, D] of the whole of sequence s (pages in table order)."""
    n = step.lens[s] if upto is None else upto
    values = code_values(mode)
    ids = step.pages[s, : -(-n // step.block)].long()
    dense = values[raw[ids].long()] * scales[ids].double()[..., None, None]  # [blocks, H, block, D]
    return dense.transpose(1, 2).reshape(-1, raw.shape[1], raw.shape[3])[:n]


def attention(q, kraw, ks, vraw, vs, step: Step, mode: str, scale, causal=True, window=0, drop=None):
    """float64 (out, a, dz, small): a = sum_j p_j |v_j|, dz the largest sum_d |scale q_d k_jd| a row
    sees (what fp32 rounding of its scores is a share of), small = max_j (p_j * value scale) *
    sum_j |value code_j| over what it sees. drop(s, j): tokens not seen."""
    T, Hq, D = q.shape
    H = kraw.shape[1]
    out, a, small = (torch.zeros(T, Hq, D, dtype=torch.float64) for _ in range(3))
    dz = torch.zeros(T, Hq, 1, dtype=torch.float64)
    for s, (n, m) in enumerate(zip(step.lens, step.news)):
        if m == 0:
            continue
        r0 = int(step.starts[s])
        if n == 0:
            continue
        k, v = read(kraw, ks, step, mode, s), read(vraw, vs, step, mode, s)
        codes = read(vraw, torch.ones_like(vs), step, mode, s).abs()
        ids = step.pages[s, : -(-n // step.block)].long()
        v_scale = vs[ids].double().repeat_interleave(step.block, 0)[:n]
        place = torch.arange(n)[None]
        rows = torch.arange(n - m, n)[:, None]
        seen = place <= rows if causal else torch.ones(m, n, dtype=torch.bool)
        if window:
            seen = seen & (place > rows - window)
        seen = seen & (rows >= 0) if causal else seen
        if drop is not None:
            seen = seen & ~torch.tensor([bool(drop(s, j)) for j in range(n)])[None]
        for h in range(Hq):
            kv = h // (Hq // H)
            qd = q[r0:r0 + m, h].double() * scale
            z = (qd @ k[:, kv].T).masked_fill(~seen, -math.inf)
            size = (qd.abs() @ k[:, kv].abs().T).masked_fill(~seen, 0)
            top = z.amax(1, keepdim=True)
            e = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
            p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
            out[r0:r0 + m, h] = p @ v[:, kv]
            a[r0:r0 + m, h] = p @ v[:, kv].abs()
            dz[r0:r0 + m, h, 0] = size.amax(1)
            small[r0:r0 + m, h] = (p * v_scale[:, kv]).amax(1, keepdim=True) * (seen.double() @ codes[:, kv])
    return out, a, dz, small


def attention_tolerance(out, terms, dtype, D, tokens):
    """|got - out| allowed, from the arithmetic alone; terms as attention() gives them.

    A score is a sum of D products in fp32 (any order: at most D + 4 roundings of
    2^-24 of its terms' sum, with the scale, the base-2 factor and the
    exponential's argument among them), so each weight is off by a share of
    2 (D + 8) 2^-24 dz at most, numerator and denominator alike; the
    exponential costs 2^-22, the sums over tokens (tokens + 64) 2^-24 each, by
    pieces of 16 and more at a time: no more than 64 + tokens / 16 steps. bf16 calls round
    the weights to 11 bits (2^-12 each, in the numerator) and the result to bf16 (2^-8).
    A weight times its value scale is rounded as an fp16 number that is at least 2^8 for
    the row's largest, so where it is subnormal its error is 2^-25 instead, 2^-33 of
    that largest: in all 2^-33 of `small`."""
    a, dz, small = terms
    share = 2 * 2 * (D + 8) * 2.0 ** -24 * dz + 2.0 ** -21 + 2 * (64 + tokens / 16) * 2.0 ** -24
    if dtype == torch.float32:
        return a * share + out.abs() * 2.0 ** -24 + 1e-30
    return a * (share + 2.0 ** -11) + out.abs() * 2.0 ** -8 + small * 2.0 ** -33 + 1e-30
