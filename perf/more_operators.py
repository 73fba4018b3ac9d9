"""A token's way through a block with its weights and its cache in four bits, as cases to time and compare: the norms
around a block with their gate and residual, the linear of a few rows over NVFP4 weights, the write of new keys and
values into a paged 4-bit cache (and their way back), and the attention that reads that cache.

``run`` computes a case either with elementary torch operations in fp32 (``own`` false) or with the package's calls
(``own`` true) on what ``prepare`` made.  Widths come from the repository's workloads or are generic.

Cases are dicts: ``op`` ("norm", "rows", "store", "attn") and sizes.  Ragged lengths follow from the case's ``split``
number alone, so ``work`` knows them without a GPU.
"""
import math
import random

import numpy as np
import torch

own = False

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------------- sizes of a case

def _lengths(total, n, split):
    """``n`` lengths of at least one that add up to ``total`` >= n: equal ones for split 0, else ragged."""
    if split == 0 or n == 1:
        return [total // n + (i < total % n) for i in range(n)]
    r = random.Random(split)
    w = [r.uniform(0.2, 1.8) for _ in range(n)]
    out = [1 + int((total - n) * x / sum(w)) for x in w]
    out[0] += total - sum(out)
    return out


def _offsets(lengths):
    return [0] + [int(v) for v in np.cumsum(lengths)]


def _new_rows(c):
    """New rows of each sequence, and the lengths of the sequences with them."""
    rows = _lengths(c["rows"], c["seqs"], c["split"] and c["split"] + 1)
    before = _lengths(c["keys"] + c["seqs"], c["seqs"], c["split"])      # each one longer than what is there before
    return rows, [a + b - 1 for a, b in zip(rows, before)]


# ---------------------------------------------------------------------------------------------------- listed and drawn

def listed():
    return [
        # one token between two blocks: nothing but latency
        dict(name="norm_one_token", op="norm", rows=1, width=3072, segments=1, split=0, y=True, post=True, layer=False,
             weight=True, mod=False, amax=False, x_scale=1.0),
        # the packed video + audio rows of the attn_out workload: gated residual, layer norm, modulation, and the
        # largest value for the quantisation that follows
        dict(name="norm_video_audio", op="norm", rows=31744, width=3072, segments=2, split=5, y=True, post=False,
             layer=True, weight=False, mod=True, amax=True, x_scale=1.0),
        # an odd number of rows of an odd width, norms before and after the block, a scaled residual
        dict(name="norm_odd", op="norm", rows=4099, width=5192, segments=3, split=9, y=True, post=True, layer=False,
             weight=True, mod=True, amax=False, x_scale=0.7),
        # one token's QKV projection
        dict(name="rows_one_qkv", op="rows", rows=1, width=3072, out=9216, swiglu=False, gated=False),
        # one token's gate and up projection of a wide block
        dict(name="rows_one_swiglu", op="rows", rows=1, width=8192, out=57344, swiglu=True, gated=False),
        # the down projection of sixteen sequences' tokens, with each row's own gate
        dict(name="rows_16_down", op="rows", rows=16, width=14336, out=4096, swiglu=False, gated=True),
        # an odd number of rows against odd sizes
        dict(name="rows_61_odd", op="rows", rows=61, width=4160, out=6152, swiglu=False, gated=True),
        # one token of each of 64 sequences goes into the cache, and comes back as the values that it holds
        dict(name="store_tokens", op="store", rows=64, keys=64 * 500, seqs=64, split=3, hk=8, d=128, page=64,
             whole=False),
        # a chunk of four prompts goes into the cache, and the whole sequences come back for attention on bf16 rows
        dict(name="store_prompts", op="store", rows=16384, keys=9001, seqs=4, split=6, hk=8, d=128, page=64,
             whole=True),
        # one token of a long sequence
        dict(name="attn_one_long", op="attn", rows=1, keys=131071, seqs=1, split=0, hq=32, hk=8, d=128, page=64,
             causal=True, lse=False),
        # one token for each of 64 sequences of different lengths
        dict(name="attn_batch", op="attn", rows=64, keys=64 * 8192, seqs=64, split=14, hq=32, hk=8, d=128, page=64,
             causal=True, lse=False),
        # a few rows each for six sequences, small heads, an odd number of query heads to a kv head, small pages
        dict(name="attn_rows_odd", op="attn", rows=31, keys=4433, seqs=6, split=27, hq=28, hk=4, d=64, page=16,
             causal=True, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rows", "store", "attn"])
    split = rng.choice([0, rng.randrange(1, 1000)])
    if op == "norm":
        width = 8 * _log(rng, 8, 2048)
        segments = rng.choice([1, 1, 2, 8])
        y = rng.random() < 0.8
        return dict(op=op, rows=_log(rng, segments, max(segments, 90000000 // width)), width=width,
                    segments=segments, split=split, y=y, post=y and rng.random() < 0.5, layer=rng.random() < 0.5,
                    weight=rng.random() < 0.5, mod=rng.random() < 0.5, amax=rng.random() < 0.3,
                    x_scale=rng.choice([1.0, 1.0, 0.5]))
    if op == "rows":
        swiglu = rng.random() < 0.3
        width = 64 * _log(rng, 1, 256)
        out = 8 * _log(rng, 1, min(16384, 8192 * 57344 // width // 8))
        out = max(256, out // 256 * 256) if swiglu else out
        return dict(op=op, rows=_log(rng, 1, 64), width=width, out=out, swiglu=swiglu,
                    gated=not swiglu and rng.random() < 0.5)
    d = rng.choice([64, 128, 128, 256, 16 * rng.randrange(1, 17)])
    hk = rng.choice([1, 2, 4, 8, 8])
    seqs = _log(rng, 1, 64)
    page = rng.choice([16, 32, 64, 64, 128])
    room = 64 * 8192 * 8 * 128 // 2 // hk // d
    if op == "store":
        return dict(op=op, rows=_log(rng, seqs, max(seqs, min(16384, room // 8))), keys=_log(rng, 1, min(32768, room // 8)),
                    seqs=seqs, split=split, hk=hk, d=d, page=page, whole=rng.random() < 0.5)
    group = rng.choice([1, 2, 4, 4, 7, 8, 16])
    rows = seqs * rng.choice([1, 1, 1, 2, 5])
    return dict(op=op, rows=rows, keys=_log(rng, seqs, max(seqs, min(131072 * seqs, room // (rows // seqs)))), seqs=seqs,
                split=split, hq=hk * group, hk=hk, d=d, page=page, causal=rng.random() < 0.7, lse=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------------- four bits

# E2M1's magnitudes, and the points between them: a tie goes to the code that is even
_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(m, s):
    """(codes uint8 [..., d/2], block scales E4M3 [..., d/16]) of bf16-valued fp32 ``m`` under the global scale ``s``
    (broadcast over the blocks): the format of the package's quantiser, each step one fp32 operation."""
    b = m.unflatten(-1, (-1, 16))
    sf = (b.abs().amax(-1) / 6.0 / s).clamp(max=448.0).to(F8)
    eff = sf.float() * s
    r = torch.where(eff == 0, torch.zeros_like(eff), (1.0 / eff).clamp(max=torch.finfo(torch.float32).max))
    q = b * r[..., None]
    a = q.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code = (code | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf


def _decode(codes, sf):
    """fp32 [..., d] of codes and block scales, without the global scale."""
    table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return (v.unflatten(-1, (-1, 16)) * sf.float()[..., None]).flatten(-2)


def _tiled(sf):
    """Block scales [rows, d/16] in tiles of 128 rows x 4 (the order that the matrix instruction reads)."""
    n, c = sf.shape
    t = torch.zeros((n + 127) // 128 * 128, c, dtype=torch.uint8, device=sf.device)
    t[:n] = sf.view(torch.uint8)
    return t.view(-1, 4, 32, c // 4, 4).permute(0, 3, 2, 1, 4).contiguous().flatten()


def _untiled(t, n, c):
    return t.view(-1, c // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, c)[:n].view(F8)


# ---------------------------------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _heads(g, rows, h, d):
    """bf16 [rows, h, d], normal, each channel with a gain of its own."""
    return (_normal(g, rows, h, d) * torch.exp(0.3 * _normal(g, h, d))).to(BF16)


def _cache(s, g, before):
    """Pages in the order in which a pool hands them out, and the keys and values of the first ``before`` rows of each
    sequence in them."""
    c, hk, d, page = s["case"], s["hk"], s["d"], s["page"]
    rows, total = s["rows"], s["total"]
    pages = [(n + page - 1) // page for n in total]
    n_pages = sum(pages) + 3
    most = max(pages)
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(pages), most), -1, dtype=torch.int32)
    at = _offsets(pages)
    seq_of = torch.repeat_interleave(torch.arange(len(pages)), torch.tensor(pages))
    table[seq_of, torch.arange(at[-1]) - torch.tensor(at)[seq_of]] = order[:at[-1]].cpu()
    s["table"] = table.cuda()
    s["length"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["row_off"] = torch.tensor(_offsets(rows), dtype=torch.int32, device="cuda")
    s["pages"] = n_pages
    # the keys and values that are there already, as the projections of earlier steps left them
    k, v = _heads(g, sum(before), hk, d), _heads(g, sum(before), hk, d)
    top = lambda t: t.float().abs().amax((0, 2)) / 2688.0 if len(t) else torch.ones(hk, device="cuda")  # noqa: E731
    s["k_gscale"], s["v_gscale"] = top(k) * 1.25, top(v) * 1.25
    off = torch.tensor(_offsets(before), dtype=torch.int32, device="cuda")
    length = torch.tensor(before, dtype=torch.int32, device="cuda")
    if own:
        import audio_dit_gb300 as A
        s["cache"] = A.alloc_kv_cache(n_pages, hk, d, page)
        if sum(before):
            A.h3fp4_cache_append(k, v, s["cache"], s["table"], length, off, k_gscale=s["k_gscale"],
                                 v_gscale=s["v_gscale"])
        return
    for name in ("k", "v"):
        s[name + "_codes"] = torch.zeros(n_pages, page, hk, d // 2, dtype=torch.uint8, device="cuda")
        s[name + "_sf"] = torch.zeros(n_pages, page, hk, d // 16, dtype=torch.uint8, device="cuda").view(F8)
    _put(s, k, v, *_places(before, before))


def _places(rows, total):
    """The sequence and the position of each of the packed rows that end their sequences."""
    seq = torch.repeat_interleave(torch.arange(len(rows), device="cuda"), torch.tensor(rows, device="cuda"),
                                  output_size=sum(rows))
    start = torch.tensor([t - n - o for t, n, o in zip(total, rows, _offsets(rows))], device="cuda")
    return seq, torch.arange(sum(rows), device="cuda") + start[seq]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    s = dict(case=c)
    if c["op"] == "norm":
        rows, width, n = c["rows"], c["width"], c["segments"]
        s["x"] = (_normal(g, rows, width) * torch.exp(0.5 * _normal(g, width)) * 2).to(BF16)
        s["y"] = _normal(g, rows, width).to(BF16) if c["y"] else None
        lengths = _lengths(rows, n, c["split"])
        s["off"] = _offsets(lengths)
        s["seg"] = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(lengths, device="cuda"),
                                           output_size=rows)
        vec = lambda on, mean, std: mean + std * _normal(g, n, width) if on else None  # noqa: E731
        s["y_weight"], s["gate"] = vec(c["post"], 1.0, 0.2), vec(c["y"], 0.5, 0.3)
        s["weight"] = vec(c["weight"], 1.0, 0.2)
        s["shift"], s["scale"] = vec(c["mod"], 0.0, 0.1), vec(c["mod"], 0.0, 0.1)
        s["out"] = torch.empty(rows, width, dtype=BF16, device="cuda")
        s["x_out"] = torch.empty(rows, width, dtype=BF16, device="cuda") if c["y"] else None
        s["amax"] = torch.empty(1, device="cuda") if c["amax"] else None
        s["eps"] = 1e-6
        return s
    if c["op"] == "rows":
        rows, width, n = c["rows"], c["width"], c["out"]
        w = (_normal(g, n, width) * 0.02).to(BF16).float()
        s["w_gscale"] = (w.abs().amax() / 2688.0).reshape(1)
        s["w_codes"], sf = _encode(w, s["w_gscale"])
        s["w_sf"] = _tiled(sf)
        del w, sf
        # activations with a few large channels
        gain = torch.where(torch.rand(width, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        s["x"] = (_normal(g, rows, width) * gain).to(BF16)
        s["bias"] = (_normal(g, n) * 0.1).to(BF16)
        s["gate"] = torch.rand(rows, n, generator=g, device="cuda") if c["gated"] else None
        s["resid"] = _normal(g, rows, n).to(BF16) if c["gated"] else None
        s["out"] = torch.empty(rows, n // 2 if c["swiglu"] else n, dtype=BF16, device="cuda")
        if own:
            import audio_dit_gb300 as A
            s["ws"] = A.alloc_rows_workspace(rows, n, width)
        return s
    hk, d = c["hk"], c["d"]
    s.update(hk=hk, d=d, page=c["page"])
    s["rows"], s["total"] = _new_rows(c)
    if c["op"] == "store":
        _cache(s, g, [t - n for t, n in zip(s["total"], s["rows"])])
        kv = _heads(g, c["rows"], 2 * hk, d)                  # K and V as one projection leaves them
        s["k"], s["v"] = kv[:, :hk], kv[:, hk:]
        back = s["total"] if c["whole"] else s["rows"]
        s["back"] = back
        s["back_off"] = torch.tensor(_offsets(back), dtype=torch.int32, device="cuda")
        s["k_out"], s["v_out"] = (torch.empty(sum(back), hk, d, dtype=BF16, device="cuda") for _ in range(2))
        return s
    _cache(s, g, s["total"])
    s["hq"] = c["hq"]
    s["q"] = _heads(g, c["rows"], c["hq"], d)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty(c["rows"], c["hq"], d, dtype=BF16, device="cuda")
    s["lse"] = torch.empty(c["rows"], c["hq"], device="cuda") if c["lse"] else None
    if own:
        import audio_dit_gb300 as A
        s["ws"] = A.alloc_cache_attn_workspace(c["rows"], c["seqs"], c["hq"], hk, d)
    return s


# ---------------------------------------------------------------------------------------------------- the plain forms

def _norm(s):
    c = s["case"]
    at = lambda v: v[s["seg"]]  # noqa: E731
    r = s["x"].float()
    if c["y"]:
        y = s["y"].float()
        if c["post"]:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * at(s["y_weight"])
        r = c["x_scale"] * r + at(s["gate"]) * y
    m = r - r.mean(-1, keepdim=True) if c["layer"] else r
    m = m * torch.rsqrt((m * m).mean(-1, keepdim=True) + s["eps"])
    if c["weight"]:
        m = m * at(s["weight"])
    if c["mod"]:
        m = m * (1 + at(s["scale"])) + at(s["shift"])
    m = m.to(BF16)
    got = dict(out=m)
    if c["y"]:
        got["x_out"] = r.to(BF16)
    if c["amax"]:
        got["amax"] = m.float().abs().amax().reshape(1)
    return got


def _rows(s):
    c = s["case"]
    w = _decode(s["w_codes"], _untiled(s["w_sf"], c["out"], c["width"] // 16))
    y = (s["x"].float() @ w.T) * s["w_gscale"] + s["bias"].float()
    if c["swiglu"]:
        # rows of the weight in groups of 128 gate rows and their 128 up rows, each rounded as a linear's output is
        g, u = y.to(BF16).float().unflatten(-1, (-1, 2, 128)).unbind(-2)
        return (g / (1 + torch.exp(-g)) * u).flatten(-2).to(BF16)
    if c["gated"]:
        y = s["resid"].float() + s["gate"] * y
    return y.to(BF16)


def _put(s, k, v, seq, pos):
    page, slot = s["table"][seq, pos // s["page"]].long(), pos % s["page"]
    s["k_codes"][page, slot], k_sf = _encode(k.float(), s["k_gscale"][:, None])
    s["v_codes"][page, slot], v_sf = _encode(v.float(), s["v_gscale"][:, None])
    s["k_sf"].view(torch.uint8)[page, slot] = k_sf.view(torch.uint8)
    s["v_sf"].view(torch.uint8)[page, slot] = v_sf.view(torch.uint8)


def _get(s, name, page, slot):
    sf = s[name + "_sf"].view(torch.uint8)[page, slot].view(F8)
    return _decode(s[name + "_codes"][page, slot], sf) * s[name + "_gscale"][:, None]


def _store(s):
    _put(s, s["k"], s["v"], *_places(s["rows"], s["total"]))
    seq, pos = _places(s["back"], s["total"])
    page, slot = s["table"][seq, pos // s["page"]].long(), pos % s["page"]
    return _get(s, "k", page, slot).to(BF16), _get(s, "v", page, slot).to(BF16)


def _attend(s):
    c, hk = s["case"], s["hk"]
    seqs, group = c["seqs"], s["hq"] // s["hk"]
    most_q, most_k = max(s["rows"]), max(s["total"])
    seq, pos = _places(s["rows"], s["total"])
    i = torch.arange(c["rows"], device="cuda") - s["row_off"].long()[seq]
    q = torch.zeros(seqs, most_q, s["hq"], s["d"], device="cuda")
    q[seq, i] = s["q"].float() * s["scale"]
    q = q.unflatten(2, (hk, group))
    at = torch.full((seqs, most_q), -1, device="cuda")
    at[seq, i] = pos if c["causal"] else s["length"].long()[seq] - 1
    # every place of the padded batch; those behind a sequence's end read some page and are left out
    j = torch.arange(most_k, device="cuda")
    page, slot = s["table"][:, j // s["page"]].clamp(min=0).long(), (j % s["page"]).expand(seqs, -1)
    keep = (j <= at[..., None]) & (j < s["length"][:, None, None])
    score = torch.einsum("bqhgd,bkhd->bhgqk", q, _get(s, "k", page, slot))
    score = score.masked_fill(~keep[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)   # places without a row
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    y = torch.einsum("bhgqk,bkhd->bhgqd", p, _get(s, "v", page, slot)) / total
    out = y.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, i].to(BF16)
    if s["lse"] is None:
        return out
    lse = (top + torch.log(total)).squeeze(-1)
    return out, lse.permute(0, 3, 1, 2).flatten(2, 3)[seq, i]


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"norm": _norm, "rows": _rows, "store": _store, "attn": _attend}[c["op"]](s)
    import audio_dit_gb300 as A
    if c["op"] == "norm":
        A.h3fp4_block_norm(s["x"], s["out"], y=s["y"], x_out=s["x_out"], gate=s["gate"], y_weight=s["y_weight"],
                           x_scale=c["x_scale"], weight=s["weight"], shift=s["shift"], scale=s["scale"],
                           seg_off=s["off"], eps=s["eps"], post_norm=c["post"], layer_norm=c["layer"],
                           out_amax=s["amax"])
        got = dict(out=s["out"])
        if c["y"]:
            got["x_out"] = s["x_out"]
        if c["amax"]:
            got["amax"] = s["amax"]
        return got
    if c["op"] == "rows":
        A.h3fp4_linear_rows(s["x"], s["w_codes"], s["w_sf"], s["w_gscale"], s["out"], s["ws"], bias=s["bias"],
                            gate=s["gate"], resid=s["resid"], swiglu=c["swiglu"])
        return s["out"]
    if c["op"] == "store":
        A.h3fp4_cache_append(s["k"], s["v"], s["cache"], s["table"], s["length"], s["row_off"], k_gscale=s["k_gscale"],
                             v_gscale=s["v_gscale"])
        A.h3fp4_cache_read(s["k_out"], s["v_out"], s["cache"], s["table"], s["length"], s["back_off"],
                           k_gscale=s["k_gscale"], v_gscale=s["v_gscale"])
        return s["k_out"], s["v_out"]
    A.h3fp4_cache_attn(s["q"], s["cache"], s["table"], s["length"], s["out"], s["ws"], row_off=s["row_off"],
                       k_gscale=s["k_gscale"], v_gscale=s["v_gscale"], causal=c["causal"], scale=s["scale"],
                       lse=s["lse"])
    return s["out"] if s["lse"] is None else (s["out"], s["lse"])


# ---------------------------------------------------------------------------------------------------- work and truth

def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["width"]
        vectors = c["post"] + c["y"] + c["weight"] + 2 * c["mod"]
        return {"bytes": (8 if c["y"] else 4) * n + 4 * vectors * c["segments"] * c["width"], "flops": 12 * n}
    if c["op"] == "rows":
        n, m, k = c["out"], c["rows"], c["width"]
        outs = m * (n // 2 if c["swiglu"] else n)
        return {"bytes": n * k * 9 // 16 + 2 * m * k + 2 * n + 2 * outs + (6 * m * n if c["gated"] else 0),
                "flops": 2 * m * n * k}
    rows, total = _new_rows(c)
    token = c["hk"] * c["d"] * 9 // 8                           # K and V of one position, 4.5 bits an element
    if c["op"] == "store":
        back = sum(total if c["whole"] else rows)
        return {"bytes": c["rows"] * (4 * c["hk"] * c["d"] + token) + back * (token + 4 * c["hk"] * c["d"]),
                "flops": 8 * c["rows"] * c["hk"] * c["d"]}
    pairs = sum(n * t - (n * (n - 1) // 2 if c["causal"] else 0) for n, t in zip(rows, total))
    return {"bytes": sum(total) * token + 4 * c["rows"] * c["hq"] * c["d"] + (4 * c["rows"] * c["hq"] if c["lse"] else 0),
            "flops": 4 * pairs * c["hq"] * c["d"]}


def _held(codes, sf, s):
    """Float64 of what codes and block scales stand for, by a table of bytes and the bits of E4M3."""
    lut = torch.tensor([[(-1.0 if x & 8 else 1.0) * _VALUES[x & 7] for x in (b & 15, b >> 4)] for b in range(256)],
                       dtype=torch.float64, device=codes.device)
    b = sf.view(torch.uint8).int()
    e, m = b >> 3 & 15, (b & 7).double()
    block = torch.where(e == 0, m / 512.0, (1 + m / 8) * torch.exp2(e.double() - 7))
    v = lut[codes.int()].flatten(-2)
    return v * torch.repeat_interleave(block, 16, -1) * s


def _nearest(m, s):
    """Float64 of what bf16 ``m`` is held as under the global scale ``s``: of E4M3's values the one nearest to the
    block's largest over 6 s, then of E2M1's the nearest, each found in a list (a tie goes to the even code)."""
    f32 = lambda v: v.float().double()  # noqa: E731  (a step of the format is rounded to fp32)
    e4m3 = torch.tensor([(x & 7) / 512.0 if x < 8 else (1 + (x & 7) / 8) * 2.0 ** ((x >> 3) - 7) for x in range(127)],
                        dtype=torch.float64, device=m.device)
    e2m1 = torch.tensor(_VALUES, dtype=torch.float64, device=m.device)

    def pick(values, x):
        hi = torch.bucketize(x, values).clamp(1, len(values) - 1)
        lo = hi - 1
        a, b = x - values[lo], values[hi] - x
        return values[torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)]

    b = m.double().unflatten(-1, (-1, 16))
    s = s.double()
    sf = pick(e4m3, f32(f32(b.abs().amax(-1) / 6) / s))
    eff = f32(sf * s)
    r = torch.where(eff == 0, eff, f32(1 / eff).clamp(max=torch.finfo(torch.float32).max))[..., None]
    q = f32(b * r)
    return (torch.sign(q) * pick(e2m1, q.abs()) * sf[..., None] * s[..., None]).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        out, x_out = [], []
        for i in range(c["segments"]):
            at = slice(s["off"][i], s["off"][i + 1])
            r = s["x"][at].double()
            if c["y"]:
                y = s["y"][at].double()
                if c["post"]:
                    y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / c["width"] + s["eps"]) * s["y_weight"][i].double()
                r = r * c["x_scale"] + y * s["gate"][i].double()
            x_out.append(r)
            mean = r.sum(-1, keepdim=True) / c["width"] if c["layer"] else 0.0
            z = (r - mean) / torch.sqrt((r - mean).pow(2).sum(-1, keepdim=True) / c["width"] + s["eps"])
            if c["weight"]:
                z = z * s["weight"][i].double()
            if c["mod"]:
                z = z + z * s["scale"][i].double() + s["shift"][i].double()
            out.append(z)
        got = dict(out=torch.cat(out))
        if c["y"]:
            got["x_out"] = torch.cat(x_out)
        if c["amax"]:
            got["amax"] = None                                  # of rounded values: it has none in 64 bits
        return got
    if c["op"] == "rows":
        y = torch.empty(c["rows"], c["out"], dtype=torch.float64, device="cuda")
        tiles = s["w_sf"].view(-1, c["width"] // 64, 32, 4, 4)
        for n in range(0, c["out"], 4096):
            at = torch.arange(n, min(n + 4096, c["out"]), device="cuda")
            sf = tiles[at // 128, :, at % 32, at % 128 // 32].flatten(1)
            y[:, at] = s["x"].double() @ _held(s["w_codes"][at], sf, s["w_gscale"].double()).T
        y += s["bias"].double()
        if c["swiglu"]:
            g, u = y.unflatten(-1, (-1, 2, 128)).unbind(-2)
            return (g * torch.sigmoid(g) * u).flatten(-2)
        return s["resid"].double() + s["gate"].double() * y if c["gated"] else y
    hk, d, page = c["hk"], c["d"], c["page"]
    if c["op"] == "store":
        got = []
        for name in ("k", "v"):
            new = _nearest(s[name], s[name + "_gscale"][:, None])
            for i, (n, t) in enumerate(zip(s["rows"], s["total"])):
                mine = new[int(s["row_off"][i]):int(s["row_off"][i]) + n]
                if c["whole"]:
                    ids = s["table"][i, :(t + page - 1) // page].long()
                    held = _held(s[name + "_codes"][ids].flatten(0, 1)[:t - n],
                                 s[name + "_sf"].view(torch.uint8)[ids].flatten(0, 1)[:t - n],
                                 s[name + "_gscale"].double()[:, None])
                    mine = torch.cat([held, mine])
                got.append(mine)
        half = len(got) // 2
        return torch.cat(got[:half]), torch.cat(got[half:])
    out = torch.zeros(c["rows"], s["hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["rows"], s["hq"], dtype=torch.float64, device="cuda")
    at = _offsets(s["rows"])
    for i, (n, t) in enumerate(zip(s["rows"], s["total"])):
        ids = s["table"][i, :(t + page - 1) // page].long()
        k, v = (_held(s[x + "_codes"][ids].flatten(0, 1)[:t], s[x + "_sf"].view(torch.uint8)[ids].flatten(0, 1)[:t],
                      s[x + "_gscale"].double()[:, None]) for x in ("k", "v"))
        for h in range(s["hq"]):
            kv = h * hk // s["hq"]
            z = s["q"][at[i]:at[i] + n, h].double() @ k[:, kv].T * s["scale"]
            if c["causal"]:
                late = torch.arange(t, device="cuda") > torch.arange(t - n, t, device="cuda")[:, None]
                z[late] = -math.inf
            m = torch.logsumexp(z, -1)
            out[at[i]:at[i] + n, h] = torch.exp(z - m[:, None]) @ v[:, kv]
            lse[at[i]:at[i] + n, h] = m
    return out if s["lse"] is None else (out, lse)
