"""The attention side of a block, as cases to time and compare: the per-head norm with rotation of Q and K, the
attention to an encoder's states, and the attention of a batch that shares a context.

``run`` computes a case either with elementary torch operations in fp32 (``own`` false) or with the package's calls
(``own`` true) on what ``prepare`` made.  Head shapes and row counts come from the repository's workloads (24 heads of
128, 8192 to 32768 rows, a video + audio split of 30720 + 1024) or are generic.

Cases are dicts: ``op`` ("norm_rope", "cross", "shared") and sizes.  Ragged lengths follow from the case's ``split``
number alone, so ``work`` knows them without a GPU.
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------------------- sizes of a case

def _lengths(total, n, split, empty=False):
    """``n`` segment lengths that add up to ``total``: equal ones for split 0 (the first ones one longer where they
    have to be), else ragged; ``empty`` empties the second one."""
    if n == 1:
        return [total]
    if split == 0:
        return [total // n + (i < total % n) for i in range(n)]
    r = random.Random(split)
    w = [r.uniform(0.3, 1.7) for _ in range(n)]
    if empty:
        w[1] = 0.0
    out = [int(total * x / sum(w)) for x in w]
    out[0] += total - sum(out)
    return out


def _offsets(lengths):
    return [0] + [int(v) for v in np.cumsum(lengths)]


def _q_lengths(c):
    return _lengths(c["rows"], c["segments"], c["split"])


def _kv_lengths(c):
    return _lengths(c["keys"], c["segments"], c["split"] and c["split"] + 1, c.get("empty", False))


def _valid(lengths, part):
    """How many keys of each segment its mask keeps: the first ``part`` of them (a prompt padded at its end)."""
    return [min(n, int(math.ceil(n * part))) for n in lengths]


# ---------------------------------------------------------------------------------------------------- listed and drawn

def listed():
    return [
        # one token of a stream that is generated step by step: nothing but latency
        dict(name="norm_rope_one_token", op="norm_rope", rows=1, hq=24, hk=24, d=128, rot=128, pairs=False, segments=1,
             split=0, weights=True),
        # Q and K of the qkv workload's output (8192 rows of 3 x 24 x 128), read as strided views
        dict(name="norm_rope_qkv", op="norm_rope", rows=8192, hq=24, hk=24, d=128, rot=128, pairs=False, segments=1,
             split=0, weights=True),
        # the packed video + audio rows of the attn_out workload, with each modality's own weights
        dict(name="norm_rope_video_audio", op="norm_rope", rows=31744, hq=24, hk=24, d=128, rot=128, pairs=False,
             segments=2, split=4, weights=True),
        # shared key heads of 80, adjacent pairs, a part of each head rotated, an odd number of rows
        dict(name="norm_rope_gqa_odd", op="norm_rope", rows=4099, hq=20, hk=5, d=80, rot=48, pairs=True, segments=3,
             split=7, weights=True),
        # the video rows attend to a prompt's encoder states
        dict(name="cross_video_text", op="cross", rows=30720, keys=512, hq=24, hk=24, d=128, segments=1, split=0,
             valid=1.0, lse=False),
        # prompts of several samples, ragged and padded, one of them without any state
        dict(name="cross_ragged_masked", op="cross", rows=9001, keys=1801, hq=24, hk=8, d=96, segments=6, split=11,
             valid=0.7, empty=True, lse=True),
        # the audio rows attend to the video states: few query rows, a long key axis
        dict(name="cross_audio_video", op="cross", rows=1024, keys=30720, hq=24, hk=24, d=128, segments=1, split=0,
             valid=1.0, lse=False),
        # one token against a long encoder sequence with shared key heads
        dict(name="cross_one_token", op="cross", rows=1, keys=32768, hq=32, hk=8, d=128, segments=1, split=0,
             valid=1.0, lse=False),
        # a small call: one token per sample against short prompts
        dict(name="cross_small", op="cross", rows=4, keys=308, hq=24, hk=24, d=64, segments=4, split=0, valid=1.0,
             lse=True),
        # two samples of one prompt: each attends to the shared prompt and keyframe states and to its own rows
        dict(name="shared_block", op="shared", rows=16384, keys=16384, ctx=1024, hq=24, hk=24, d=128, segments=2,
             split=0, valid=1.0, ctx_valid=1.0, lse=False),
        # ragged samples, shared key heads of 64, a padded context of odd length
        dict(name="shared_ragged", op="shared", rows=4500, keys=4700, ctx=333, hq=16, hk=4, d=64, segments=6, split=21,
             valid=1.0, ctx_valid=0.8, lse=True),
        # one token for each of 48 samples over a long shared prefix and short suffixes of their own
        dict(name="shared_tokens", op="shared", rows=48, keys=9000, ctx=16384, hq=32, hk=8, d=128, segments=48,
             split=33, valid=1.0, ctx_valid=1.0, lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "cross", "shared"])
    d = rng.choice([64, 128, 128, rng.randrange(8, 129, 8)])
    hk = rng.choice([1, 2, 4, 5, 8, 24])
    hq = hk * rng.choice([1, 1, 2, 3, 4, 7] if hk <= 4 else [1, 1, 2, 4] if hk <= 8 else [1])
    split = rng.choice([0, rng.randrange(1, 1000)])
    if op == "norm_rope":
        d = rng.choice([d, 16 * rng.randrange(1, 17)])
        return dict(op=op, rows=_log(rng, 1, 31744 * 128 // max(128, d) * 24 // max(24, hq)), hq=hq, hk=hk, d=d,
                    rot=16 * rng.randrange(0, d // 16 + 1), pairs=rng.random() < 0.5, segments=rng.choice([1, 1, 2, 8]),
                    split=split, weights=rng.random() < 0.8)
    segments = rng.choice([1, 1, 2, 3, 8, 40])
    lse = rng.random() < 0.5
    valid = rng.choice([1.0, 1.0, 0.6])
    # rows x keys x heads is bounded by a quarter of the largest listed case's
    room = 16384 * 9216 * 24 // 4 // hq
    rows = _log(rng, 1, 30720)
    if op == "cross":
        keys = _log(rng, 1, max(1, min(32768, room // rows)))
        return dict(op=op, rows=rows, keys=keys, hq=hq, hk=hk, d=d, segments=segments, split=split, valid=valid,
                    empty=segments > 1 and split > 0 and rng.random() < 0.3, lse=lse)
    keys = _log(rng, 1, max(1, min(16384, room // rows)))
    ctx = _log(rng, 1, max(1, min(16384, room // rows)))
    return dict(op=op, rows=rows, keys=keys, ctx=ctx, hq=hq, hk=hk, d=d, segments=segments, split=split, valid=valid,
                ctx_valid=rng.choice([1.0, 0.5]), lse=lse)


# ---------------------------------------------------------------------------------------------------- inputs

def _heads(g, rows, h, d, spread=1.0):
    """bf16 [rows, h, d], normal, each channel with a gain of its own."""
    gain = torch.exp(spread * 0.25 * torch.randn(h, d, generator=g, device="cuda"))
    return (torch.randn(rows, h, d, generator=g, device="cuda") * gain).to(torch.bfloat16)


def _mask(lengths, part):
    """bool keys of all segments (True: attended to), None where every key is."""
    if part >= 1.0:
        return None
    keep = [np.arange(n) < v for n, v in zip(lengths, _valid(lengths, part))]
    return torch.from_numpy(np.concatenate(keep) if keep else np.zeros(0, bool)).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, d, hq, hk = case, case["d"], case["hq"], case["hk"]
    s = dict(case=c, d=d, hq=hq, hk=hk)
    if c["op"] == "norm_rope":
        # the projection's output [rows, (hq + 2 hk) * d]; Q and K are strided views of it
        rows, n = c["rows"], c["segments"]
        qkv = _heads(g, rows, hq + 2 * hk, d, 2.0)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["off"] = _offsets(_q_lengths(c))
        w = lambda: (1 + 0.2 * torch.randn(n, d, generator=g, device="cuda")) if c["weights"] else None  # noqa: E731
        s["qw"], s["kw"] = w(), w()
        if c["rot"]:
            # angles of positions along three axes, as a table for each row
            half = c["rot"] // 2
            pos = torch.randint(0, 256, (rows, 3), generator=g, device="cuda").float()
            axis = torch.arange(half, device="cuda") % 3
            freq = 10000.0 ** (-torch.arange(half, device="cuda").float() / half)
            ang = pos[:, axis] * freq
            s["cos"], s["sin"] = torch.cos(ang).contiguous(), torch.sin(ang).contiguous()
        else:
            s["cos"] = s["sin"] = None
        s["eps"] = 1e-6
        s["q_out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(rows, hk, d, dtype=torch.bfloat16, device="cuda")
        # which weight row each token takes, for the plain form
        s["seg"] = torch.repeat_interleave(torch.arange(n, device="cuda"),
                                           torch.tensor(_q_lengths(c), device="cuda"), output_size=rows)
        return s
    ql, kl = _q_lengths(c), _kv_lengths(c)
    s["q_off"], s["kv_off"] = _offsets(ql), _offsets(kl)
    s["mask"] = _mask(kl, c["valid"])
    s["scale"] = 1.0 / math.sqrt(d)
    if c["op"] == "cross":
        s["q"] = _heads(g, c["rows"], hq, d)
        kv = _heads(g, c["keys"], 2 * hk, d)                  # one projection of the states, K and V side by side
        s["k"], s["v"] = kv[:, :hk], kv[:, hk:]
    else:
        s["q"] = _heads(g, c["rows"], hq, d)
        s["k"] = _heads(g, c["keys"], hk, d)
        s["v"] = _heads(g, c["keys"], hk, d)
        kv = _heads(g, c["ctx"], 2 * hk, d)
        s["k_ctx"], s["v_ctx"] = kv[:, :hk], kv[:, hk:]
        s["ctx_mask"] = _mask([c["ctx"]], c["ctx_valid"])
    s["out"] = torch.empty(c["rows"], hq, d, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(c["rows"], hq, dtype=torch.float32, device="cuda") if c["lse"] else None
    # the plain form's padded batch: where each segment's rows go, and which places hold a key
    place = lambda n: (torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"),  # noqa: E731
                                               output_size=sum(n)),
                       torch.from_numpy(np.concatenate([np.arange(x) for x in n])).cuda())
    s["q_at"], s["k_at"] = place(ql), place(kl)
    s["q_most"], s["k_most"] = max(ql), max(1, max(kl))
    if own:
        import audio_dit_gb300 as A
        s["ws"] = A.alloc_attn_workspace(c["rows"], c["keys"], hq, hk, d, q_off=s["q_off"], kv_off=s["kv_off"],
                                         ctx=c.get("ctx", 0))
    return s


# ---------------------------------------------------------------------------------------------------- the plain forms

def _norm_rotate(x, w, s):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    if w is not None:
        y = y * w[s["seg"]][:, None, :]
    if s["cos"] is not None:
        half = s["cos"].shape[1]
        cos, sin = s["cos"][:, None, :], s["sin"][:, None, :]
        r = y[..., :2 * half]
        if s["case"]["pairs"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        y = torch.cat([r, y[..., 2 * half:]], -1)
    return y.to(torch.bfloat16)


def _padded(x, at, n, most):
    y = x.new_zeros((n, most, *x.shape[1:]))
    y[at] = x
    return y


def _attend(s):
    c, hk = s["case"], s["hk"]
    n, group = c["segments"], s["hq"] // s["hk"]
    q = _padded(s["q"].float() * s["scale"], s["q_at"], n, s["q_most"]).unflatten(2, (hk, group))
    k = _padded(s["k"].float(), s["k_at"], n, s["k_most"])
    v = _padded(s["v"].float(), s["k_at"], n, s["k_most"])
    there = torch.ones(c["keys"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    keep = _padded(there, s["k_at"], n, s["k_most"])
    score = torch.einsum("bqhgd,bkhd->bhgqk", q, k).masked_fill(~keep[:, None, None, None, :], -math.inf)
    if c["op"] == "shared":
        more = torch.einsum("bqhgd,khd->bhgqk", q, s["k_ctx"].float())
        if s["ctx_mask"] is not None:
            more = more.masked_fill(~s["ctx_mask"], -math.inf)
        score = torch.cat([more, score], -1)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)   # rows without a key
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    if c["op"] == "shared":
        m = s["k_ctx"].shape[0]
        y = torch.einsum("bhgqk,khd->bhgqd", p[..., :m], s["v_ctx"].float())
        y = y + torch.einsum("bhgqk,bkhd->bhgqd", p[..., m:], v)
    else:
        y = torch.einsum("bhgqk,bkhd->bhgqd", p, v)
    y = torch.where(total > 0, y / total, torch.zeros_like(y))
    out = y.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["q_at"]].to(torch.bfloat16)
    if s["lse"] is None:
        return out
    lse = (top + torch.log(total)).squeeze(-1)
    return out, lse.permute(0, 3, 1, 2).flatten(2, 3)[s["q_at"]]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        if op == "norm_rope":
            return _norm_rotate(s["q"], s["qw"], s), _norm_rotate(s["k"], s["kw"], s)
        return _attend(s)
    import audio_dit_gb300 as A
    if op == "norm_rope":
        A.h3fp4_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], q_weight=s["qw"], k_weight=s["kw"], cos=s["cos"],
                             sin=s["sin"], interleaved=s["case"]["pairs"], seg_off=s["off"], eps=s["eps"])
        return s["q_out"], s["k_out"]
    if op == "cross":
        A.h3fp4_cross_attn(s["q"], s["k"], s["v"], s["out"], s["ws"], q_off=s["q_off"], kv_off=s["kv_off"],
                           key_mask=s["mask"], scale=s["scale"], lse=s["lse"])
    else:
        A.h3fp4_shared_attn(s["q"], s["k"], s["v"], s["k_ctx"], s["v_ctx"], s["out"], s["ws"], q_off=s["q_off"],
                            kv_off=s["kv_off"], key_mask=s["mask"], ctx_mask=s["ctx_mask"], scale=s["scale"],
                            lse=s["lse"])
    return s["out"] if s["lse"] is None else (s["out"], s["lse"])


# ---------------------------------------------------------------------------------------------------- work and truth

def work(case):
    c, d, hq, hk = case, case["d"], case["hq"], case["hk"]
    if c["op"] == "norm_rope":
        values = c["rows"] * (hq + hk) * d
        table = c["rows"] * c["rot"] * 4                       # cos and sin, fp32, rot / 2 each
        return {"bytes": 4 * values + table + (8 * c["segments"] * d if c["weights"] else 0), "flops": 7 * values}
    ql, kl = _q_lengths(c), _kv_lengths(c)
    kept = _valid(kl, c["valid"])
    pairs = sum(a * b for a, b in zip(ql, kept))
    keys = sum(b for a, b in zip(ql, kept) if a)
    mask = c["keys"] if c["valid"] < 1 else 0
    if c["op"] == "shared":
        ctx = _valid([c["ctx"]], c["ctx_valid"])[0]
        pairs += c["rows"] * ctx
        keys += ctx
        mask += c["ctx"] if c["ctx_valid"] < 1 else 0
    return {"bytes": 4 * c["rows"] * hq * d + 4 * keys * hk * d + mask + (4 * c["rows"] * hq if c["lse"] else 0),
            "flops": 4 * pairs * hq * d}


def exact(case, seed):
    s = prepare(case, seed)
    c, d = s["case"], s["d"]
    if c["op"] == "norm_rope":
        off = s["off"]
        done = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            y = x.double()
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / d + s["eps"])
            if w is not None:
                for i in range(c["segments"]):
                    y[off[i]:off[i + 1]] *= w[i].double()
            if s["cos"] is not None:
                half = s["cos"].shape[1]
                turn = torch.complex(s["cos"].double(), s["sin"].double())[:, None, :]
                i = torch.arange(half, device="cuda")
                first, second = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + half)
                z = torch.complex(y[..., first], y[..., second]) * turn
                y[..., first], y[..., second] = z.real, z.imag
            done.append(y)
        return tuple(done)
    out = torch.zeros(c["rows"], s["hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["rows"], s["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    group = s["hq"] // s["hk"]
    for i in range(c["segments"]):
        q0, q1, k0, k1 = s["q_off"][i], s["q_off"][i + 1], s["kv_off"][i], s["kv_off"][i + 1]
        if q0 == q1:
            continue
        keep = torch.arange(k0, k1, device="cuda")
        if s["mask"] is not None:
            keep = keep[s["mask"][k0:k1]]
        key, val = s["k"][keep], s["v"][keep]
        if c["op"] == "shared":
            some = torch.arange(c["ctx"], device="cuda") if s["ctx_mask"] is None else s["ctx_mask"].nonzero()[:, 0]
            key, val = torch.cat([s["k_ctx"][some], key]), torch.cat([s["v_ctx"][some], val])
        if not len(key):
            continue
        for h in range(s["hq"]):
            z = s["q"][q0:q1, h].double() @ key[:, h // group].double().T * s["scale"]
            n = torch.logsumexp(z, -1)
            out[q0:q1, h] = torch.exp(z - n[:, None]) @ val[:, h // group].double()
            lse[q0:q1, h] = n
    return out if s["lse"] is None else (out, lse)
