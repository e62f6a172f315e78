"""Cases of the serving operators that stand between the quantized products of
a decoder layer: the router in front of the routed experts, the write of new
keys and values into a paged 8-bit cache and their read-back, and attention
over that cache.

`run` computes each operator in its plain form (elementary torch operations)
or, where `own` is true, through the package's entry points.

Shared notation of the cache cases: pages hold `block` tokens of `heads`
key/value heads of `dim` values in 8 bits, one fp32 scale per (page, head);
sequence i has `lens[i]` tokens, of which the last starts[i + 1] - starts[i]
are this step's rows; its j-th block of tokens lives in page `pages[i, j]`.
"""
import math

import torch

own = False

INT8_MAX, E4M3_MAX = 127.0, 448.0


# ---------------------------------------------------------------------- cases
def listed():
    attend = {"op": "attend", "heads": 8, "group": 4, "dim": 128, "block": 64, "mode": "int8", "window": 0}
    cache = {"op": "cache", "heads": 8, "dim": 128, "block": 64, "mode": "int8", "type": "bf16"}
    return [
        # the router of one decoded token: nothing but latency
        {"name": "route_1x64", "op": "route", "tokens": 1, "experts": 64, "topk": 4, "score": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "group_top": 1, "type": "bf16"},
        # the mixture-of-experts layer of the benchmark: 512 tokens, 64 experts, 4 of them a token
        {"name": "route_512x64", "op": "route", "tokens": 512, "experts": 64, "topk": 4, "score": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "group_top": 1, "type": "bf16"},
        # a prompt through a router of many experts with a balancing bias and limited groups
        {"name": "route_16384x256", "op": "route", "tokens": 16384, "experts": 256, "topk": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "group_top": 2, "type": "f32"},
        # a decoding step appends one token to each of 128 sequences, most blocks partly filled
        {"name": "cache_append_128", **cache, "seqs": 128, "new": 1, "kv": 2048, "write": True},
        # a prompt of 8192 tokens is written
        {"name": "cache_prompt_8192", **cache, "seqs": 1, "new": 8192, "kv": 8192, "write": True},
        # ragged chunks into small pages, floating-point codes, fp32 values
        {"name": "cache_chunks_e4m3", **cache, "dim": 64, "block": 16, "mode": "e4m3", "type": "f32",
         "seqs": 7, "new": 611, "kv": 1500, "write": True},
        # whole sequences read back, as for moving them to a host or to another precision
        {"name": "cache_read_32", **cache, "seqs": 32, "new": 2048, "kv": 2048, "write": False},
        # one sequence decodes: latency, and few rows to fill the GPU with
        {"name": "attend_decode_1x4096", **attend, "seqs": 1, "new": 1, "kv": 4096},
        # a batch decodes over ragged lengths
        {"name": "attend_decode_64x8192", **attend, "seqs": 64, "new": 1, "kv": 8192},
        # two long contexts, floating-point codes, large pages
        {"name": "attend_decode_2x131072", **attend, "block": 128, "mode": "e4m3", "seqs": 2, "new": 1, "kv": 131072},
        # chunks of several prompts behind their earlier tokens, with a sliding window
        {"name": "attend_chunks_4x8192", **attend, "seqs": 4, "new": 1024, "kv": 8192, "window": 4096},
        # a whole prompt
        {"name": "attend_prompt_8192", **attend, "seqs": 1, "new": 8192, "kv": 8192},
    ]


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49))))))


def draw(rng):
    op = rng.choice(["route", "cache", "attend", "attend"])
    if op == "route":
        tokens, groups = _log(rng, 1, 16384), rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, max(2, 8 // groups), 384 // groups)
        topk_groups = rng.randint(1, groups)
        return {"op": op, "tokens": tokens, "experts": experts,
                "topk": rng.randint(1, min(10, topk_groups * (experts // groups))),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "topk_groups": topk_groups, "group_top": rng.choice([1, 2]) if groups > 1 else 1,
                "type": rng.choice(["bf16", "f32"])}
    shape = {"op": op, "heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]),
             "block": rng.choice([16, 32, 64, 128]), "mode": rng.choice(["int8", "e4m3"])}
    if op == "cache":
        seqs = _log(rng, 1, 128)
        kv = _log(rng, 8, 32768 // seqs)
        write = rng.random() < 0.75
        return {**shape, "type": rng.choice(["bf16", "bf16", "f32"]), "seqs": seqs,
                "new": _log(rng, 1, kv) if write else kv, "kv": kv, "write": write}
    group = rng.choice([1, 2, 3, 4, 7, 8])
    if rng.random() < 0.5:  # decoding: one new token, or a few to be verified
        seqs = _log(rng, 1, 64)
        new, kv = rng.choice([1, 1, 1, 2, 5]), _log(rng, 16, 262144 // seqs)
    else:
        seqs = _log(rng, 1, 6)
        new = _log(rng, 6, 4096 // seqs)
        kv = _log(rng, new, 16384 // seqs)
    return {**shape, "group": group, "seqs": seqs, "new": new, "kv": max(kv, new),
            "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)])}


def _lengths(case):
    """New tokens and length of each sequence: the first has the case's, the others are spread below."""
    seqs, new, kv = case["seqs"], case["new"], case["kv"]
    news, lens = [], []
    for i in range(seqs):
        part = 1.0 if i == 0 else 0.25 + 0.75 * ((i * 0.6180339887498949) % 1.0)
        lens.append(max(1, math.ceil(kv * part)))
        whole = case["op"] == "cache" and not case["write"]
        news.append(lens[i] if whole else min(lens[i], new if i == 0 else max(1, math.ceil(new * part))))
    return news, lens


def _types(case):
    return torch.float32 if case.get("type") == "f32" else torch.bfloat16


# --------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] == "route":
        s["logits"] = (1.5 * normal(case["tokens"], case["experts"])).to(_types(case))
        s["bias"] = 0.1 * normal(case["experts"]) if case["bias"] else None
        return s
    news, lens = _lengths(case)
    heads, dim, block = case["heads"], case["dim"], case["block"]
    counts = [-(-n // block) for n in lens]
    width, total = max(counts), sum(counts) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table, used = torch.zeros(case["seqs"], width, dtype=torch.int32, device="cuda"), 0
    for i, n in enumerate(counts):
        table[i, :n] = order[used:used + n]
        used += n
    s["pages"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor([0] + news, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
    s["rows"], s["max_q"] = sum(news), max(news)
    largest = INT8_MAX if case["mode"] == "int8" else E4M3_MAX
    for name in ("k", "v"):
        # values of one block and head fill its range, as the writer leaves them
        values = (normal(total, heads, block, dim) * (largest / 4)).clamp_(-largest, largest)
        s[name + "_codes"] = values.round().to(torch.int8) if case["mode"] == "int8" else values.to(torch.float8_e4m3fn)
        s[name + "_scales"] = torch.exp(0.3 * normal(total, heads)) * (4 / largest)
        del values
    # rows of one tensor hold the queries, keys and values of a token side by side, as a fused projection leaves them
    hq = heads * case.get("group", 0)
    rows = normal(s["rows"], hq + 2 * heads, dim).to(_types(case))
    s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:hq + heads], rows[:, hq + heads:]
    return s


# ---------------------------------------------------------------- plain forms
def _route_plain(s):
    case, logits = s["case"], s["logits"].double()  # 64 bits: scores next to one another decide who is chosen
    score = torch.softmax(logits, 1) if case["score"] == "softmax" else torch.sigmoid(logits)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if case["groups"] > 1:
        grouped = choice.view(len(choice), case["groups"], -1)
        of_group = grouped.sort(dim=2, descending=True).values[:, :, : case["group_top"]].sum(2)
        kept = of_group.sort(dim=1, descending=True, stable=True).indices[:, : case["topk_groups"]]
        open_ = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, kept, True)
        choice = grouped.masked_fill(~open_[:, :, None], -math.inf).view_as(choice)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, : case["topk"]]
    weights = score.gather(1, ids)
    weights = weights / weights.sum(1, keepdim=True)
    return ids.to(torch.int32), weights.float()


def _places(s):
    """Page and slot of every row of the step, and the sequence that it belongs to."""
    row = torch.arange(s["rows"], device="cuda")
    starts = s["starts"].long()
    seq = torch.searchsorted(starts[1:], row, right=True)
    pos = s["lens"].long()[seq] - (starts[seq + 1] - row)
    block = s["k_codes"].shape[2]
    return s["pages"].long()[seq, pos // block], pos % block, seq


def _round_e4m3(x):
    """float64 to the nearest E4M3 value, ties to even, saturated."""
    exponent = torch.frexp(x).exponent - 1
    step = torch.exp2((exponent.clamp_min(-6) - 3).double())
    return ((x / step).round() * step).clamp(-E4M3_MAX, E4M3_MAX)


def _encode(quotient, codes):
    if codes.dtype == torch.int8:
        return quotient.round().clamp(-INT8_MAX, INT8_MAX).to(torch.int8)
    return _round_e4m3(quotient).float().to(codes.dtype)


def _raw(codes):
    return codes.view(torch.uint8)


def _write_plain(s, name, page, slot):
    x, codes, scales = s[name], s[name + "_codes"], s[name + "_scales"]
    block = codes.shape[2]
    largest = torch.tensor(INT8_MAX if codes.dtype == torch.int8 else E4M3_MAX, device="cuda")
    most = torch.zeros_like(scales).index_reduce_(0, page, x.float().abs().amax(2), "amax")
    # the only block of a sequence that may hold earlier tokens is the first one it writes to
    first = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long()
    held = s["pages"].long().gather(1, (first // block)[:, None])[:, 0]
    older = (first % block > 0)[:, None]
    before = scales[held]
    needed = most / largest
    now = torch.where(older, torch.maximum(before, needed[held]), needed[held])
    touched = torch.zeros_like(scales, dtype=torch.bool).index_fill_(0, page, True)
    scales.copy_(torch.where(touched, needed, scales))
    scales.index_copy_(0, held, now)
    old = _raw(codes)[held].view(codes.dtype).double()
    ratio = old * before[:, :, None, None].double() / now[:, :, None, None].double()
    grown = (older & (now > before))[:, :, None, None]
    again = torch.where(grown, ratio, old)
    _raw(codes)[held] = _raw(_encode(torch.where(now[:, :, None, None] > 0, again, 0.0), codes))
    divisor = scales[page][:, :, None].double()
    quotient = torch.where(divisor > 0, x.double() / divisor, 0.0)
    _raw(codes)[page, :, slot] = _raw(_encode(quotient, codes))


def _read_plain(s, name, page, slot):
    codes = s[name + "_codes"]
    values = _raw(codes)[page, :, slot].view(codes.dtype).float() * s[name + "_scales"][page][:, :, None]
    return values.to(s[name].dtype)


def _cache_plain(s):
    page, slot, _ = _places(s)
    if s["case"]["write"]:
        _write_plain(s, "k", page, slot)
        _write_plain(s, "v", page, slot)
    return {"k": _read_plain(s, "k", page, slot), "v": _read_plain(s, "v", page, slot),
            "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _attend_plain(s):
    case = s["case"]
    seqs, heads, group, dim, block = (case[n] for n in ("seqs", "heads", "group", "dim", "block"))
    width, new = s["pages"].shape[1], s["max_q"]
    pages, starts, lens = s["pages"].long(), s["starts"].long(), s["lens"].long()

    def dense(name):
        codes = s[name + "_codes"]
        values = _raw(codes)[pages].view(codes.dtype).float() * s[name + "_scales"][pages][..., None, None]
        return values.transpose(1, 2).reshape(seqs, heads, width * block, dim)

    step = torch.arange(new, device="cuda")
    rows = (starts[:-1, None] + step).clamp_max(s["rows"] - 1)
    q = s["q"][rows].float().view(seqs, new, heads, group, dim).permute(0, 2, 3, 1, 4)
    scores = q.reshape(seqs, heads, group * new, dim) @ dense("k").transpose(2, 3) / math.sqrt(dim)
    last = (lens - (starts[1:] - starts[:-1]))[:, None] + step  # place of each row in its sequence
    place = torch.arange(width * block, device="cuda")
    seen = (place <= last[..., None]) & (place < lens[:, None, None])
    if case["window"]:
        seen &= place > last[..., None] - case["window"]
    scores = scores.view(seqs, heads, group, new, -1).masked_fill_(~seen[:, None, None], -math.inf)
    scores = scores - scores.amax(4, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    weights = scores.exp_()
    total = weights.sum(4, keepdim=True)
    out = weights.view(seqs, heads, group * new, -1) @ dense("v")
    out = out.view(seqs, heads, group, new, dim) / total.clamp_min(torch.finfo(torch.float32).tiny)
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(starts[1:], row, right=True)
    out = out.permute(0, 3, 1, 2, 4)[seq, row - starts[seq]]
    return out.reshape(s["rows"], heads * group, dim).to(s["q"].dtype)


def run(state):
    case = state["case"]
    if own:
        return _run_own(state)
    return {"route": _route_plain, "cache": _cache_plain, "attend": _attend_plain}[case["op"]](state)


def _run_own(s):
    import group_wise_affine_dequant_b200 as nvq

    case = s["case"]
    if case["op"] == "route":
        return nvq.nv_moe_route(s["logits"], case["topk"], case["score"], bias=s["bias"], groups=case["groups"],
                                topk_groups=case["topk_groups"], group_top=case["group_top"])
    cache = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    where = (s["pages"], s["starts"], s["lens"])
    if case["op"] == "cache":
        if case["write"]:
            nvq.nv_kv_quantize(s["k"], s["v"], *cache, *where)
        k, v = nvq.nv_kv_dequantize(*cache, *where, rows=s["rows"], dtype=s["k"].dtype)
        return {"k": k, "v": v, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    return nvq.nv_kv_attention(s["q"], *cache, *where, causal=True, window=case["window"], max_q=s["max_q"])


# ----------------------------------------------------------------------- work
def work(case):
    size = 4 if case.get("type") == "f32" else 2
    if case["op"] == "route":
        entries = case["tokens"] * case["experts"]
        return {"bytes": entries * size + case["tokens"] * case["topk"] * 8 + 4 * case["experts"] * case["bias"],
                "flops": 4 * entries}
    news, lens = _lengths(case)
    heads, dim, block = case["heads"], case["dim"], case["block"]
    if case["op"] == "cache":
        rows = sum(news)
        touched = sum(-(-n // block) - (n - m) // block for m, n in zip(news, lens))
        scales = 2 * touched * heads * 4
        once = 2 * rows * heads * dim
        # a write reads the values and writes the codes; the read-back reads the codes and writes the values
        each = once * (size + 1) + scales + 4 * touched
        return {"bytes": each * (2 if case["write"] else 1), "flops": once * (4 if case["write"] else 1)}
    hq, window = heads * case["group"], case["window"]
    pairs = spanned = 0
    for m, n in zip(news, lens):
        first = n - m
        low = max(0, first - window + 1) if window else 0
        spanned += n - low
        if window:
            pairs += sum(min(p + 1, window) for p in range(first, n))
        else:
            pairs += m * first + m * (m + 1) // 2
    return {"bytes": 2 * spanned * heads * (dim + 4 / block) + 4 * sum(hq * dim * m for m in news),
            "flops": 4 * dim * hq * pairs}


# -------------------------------------------------------- definition, 64 bits
def _code_value(x, mode):
    """Nearest storable code of x, as a float64 value."""
    if mode == "int8":
        return torch.clamp(torch.round(x), -INT8_MAX, INT8_MAX)
    size = x.abs()
    power = torch.floor(torch.log2(torch.where(size > 0, size, torch.ones_like(size))))
    power = torch.where(size < torch.exp2(power), power - 1, power)
    power = torch.where(size >= torch.exp2(power + 1), power + 1, power)
    ulp = torch.exp2(torch.clamp(power, min=-6.0) - 3)
    return torch.sign(x) * torch.clamp(torch.round(size / ulp) * ulp, max=E4M3_MAX)


def _exact_route(s):
    case = s["case"]
    z = s["logits"].cpu().numpy() if case["type"] == "f32" else s["logits"].float().cpu().numpy()
    import numpy as np
    z = z.astype(np.float64)
    if case["score"] == "softmax":
        e = np.exp(z - z.max(1, keepdims=True))
        score = e / e.sum(1, keepdims=True)
    else:
        score = 1.0 / (1.0 + np.exp(-z))
    choice = score + (s["bias"].cpu().numpy().astype(np.float64) if case["bias"] else 0.0)
    per = case["experts"] // case["groups"]
    weights = np.zeros((len(z), case["topk"]))
    for t in range(len(z)):
        c = choice[t]
        if case["groups"] > 1:
            best = np.sort(c.reshape(-1, per), 1)[:, ::-1][:, : case["group_top"]].sum(1)
            groups = np.argsort(-best, kind="stable")[: case["topk_groups"]]
            c = np.where(np.isin(np.arange(len(c)) // per, groups), c, -np.inf)
        chosen = score[t][np.argsort(-c, kind="stable")[: case["topk"]]]
        weights[t] = chosen / chosen.sum()
    return [None, torch.from_numpy(weights)]


def _exact_cache(s):
    case = s["case"]
    news, lens = _lengths(case)
    block, mode = case["block"], case["mode"]
    largest = INT8_MAX if mode == "int8" else E4M3_MAX
    pages = s["pages"].tolist()
    got = {}
    for name in ("k", "v"):
        x, scales = s[name].double(), s[name + "_scales"].clone()
        codes = s[name + "_codes"].float()
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        row = 0
        for i, (m, n) in enumerate(zip(news, lens)):
            pos = n - m
            while pos < n:
                page, slot = pages[i][pos // block], pos % block
                count = min(block - slot, n - pos)
                part = x[row:row + count]
                if case["write"]:
                    needed = (part.abs().amax((0, 2)) / largest).float()  # a stored scale is a 32-bit number
                    scales[page] = torch.maximum(scales[page], needed) if slot else needed
                    divisor = scales[page].double()[None, :, None]
                    stored = _code_value(torch.where(divisor > 0, part / divisor, 0.0), mode)
                else:
                    stored = codes[page, :, slot:slot + count].double().transpose(0, 1)
                out[row:row + count] = stored * scales[page].double()[None, :, None]
                row, pos = row + count, pos + count
        got[name], got[name + "_scales"] = out, scales.double()
    return got


def _exact_attend(s):
    case = s["case"]
    news, lens = _lengths(case)
    heads, group, dim, block = (case[n] for n in ("heads", "group", "dim", "block"))
    out = torch.zeros(s["rows"], heads * group, dim, dtype=torch.float64, device="cuda")
    row = 0
    for i, (m, n) in enumerate(zip(news, lens)):
        ids = s["pages"][i, : -(-n // block)].long()
        place, rows = torch.arange(n, device="cuda")[None], torch.arange(n - m, n, device="cuda")[:, None]
        hidden = place > rows
        if case["window"]:
            hidden |= rows - place >= case["window"]
        for h in range(heads):
            def sequence(name):
                raw = s[name + "_codes"].view(torch.uint8)[ids, h].view(s[name + "_codes"].dtype)
                return (raw.double() * s[name + "_scales"][ids, h, None, None].double()).reshape(-1, dim)[:n]

            keys, values = sequence("k"), sequence("v")
            for j in range(h * group, (h + 1) * group):
                z = torch.einsum("rd,kd->rk", s["q"][row:row + m, j].double(), keys) * dim ** -0.5
                z.masked_fill_(hidden, -math.inf)
                out[row:row + m, j] = torch.softmax(z, 1) @ values
        row += m
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "cache": _exact_cache, "attend": _exact_attend}[case["op"]](s)
