"""Checks of the attention that one key lost or counted twice among tens of thousands fails, and inputs for them.

Counting: with queries of zero every kept key has the weight 1 exactly, so the log-sum-exp is the logarithm of how many
there are, and a column of V that is 1 at some keys gives their share.  Columns are 1 at every ``period``-th key, so that
no column counts more than some 100: one key more or less changes the share by 1 / 100, twice the 2^-8 of its rounding
to bf16 and more.

Norms: over V of a normal distribution a row's error is that of two roundings to bf16 (the weights' and the output's), each
uniform within 2^-8 / m of the value for a mantissa m between 1 and 2: 2^-8 / sqrt(3) times the root of the mean of
1 / m^2 (0.74 for mantissas whose logarithm is uniform) is 0.0016, both together 0.0023.  Over D >= 64 columns
their sum of squares is within some 50 % of its mean, and so is the output's own."""
import math

import numpy as np
import torch

ROW_ERROR = 0.0023 * 1.5 / 0.75     # one row of one head
ALL_ERROR = 0.0023 * 1.1            # a whole call


def period(keys, D):
    """Distance of the keys that a column counts: a multiple of D with some 100 of them at most."""
    return D * max(1, math.ceil(keys / (100 * D)))


def marked(first, n, heads, D, every, shift):
    """V of keys first..., 1 in column c at keys whose number is c + shift modulo ``every``."""
    at = (torch.arange(first, first + n) - shift) % every
    v = (at[:, None] == torch.arange(D)[None, :]).to(torch.bfloat16)
    return v[:, None, :].expand(n, heads, D).contiguous()


def counts(q_off, kv_off, ctx, D, every, shift, key_mask=None, ctx_mask=None):
    """(share of each column [segments, D], number of keys [segments]) in whole numbers' arithmetic."""
    most = ctx + max(b - a for a, b in zip(kv_off, kv_off[1:]))
    share, total = np.zeros((len(q_off) - 1, D)), np.zeros(len(q_off) - 1, np.int64)
    for i, (a, b) in enumerate(zip(kv_off, kv_off[1:])):
        on = np.zeros(most, bool)
        on[:ctx] = True if ctx_mask is None else np.asarray(ctx_mask)
        on[ctx:ctx + b - a] = True if key_mask is None else np.asarray(key_mask)[a:b]
        at = (np.nonzero(on)[0] - shift) % every
        total[i] = len(at)
        share[i] = np.bincount(at, minlength=every)[:D]
    return share, total


def counted(out, lse, q_off, share, total):
    """What is wrong with a counting call's outputs, or None.

    A share is rounded to bf16 once (2^-8 of it, and 2^-20 for the reciprocal); the logarithm is within 2 units of
    fp32 and rounded twice more."""
    for i, (a, b) in enumerate(zip(q_off, q_off[1:])):
        if a == b:
            continue
        o, l = out[a:b].double(), lse[a:b].double()
        if total[i] == 0:
            if bool((o != 0).any()) or not bool(torch.isneginf(l).all()):
                return f"segment {i} has no key"
            continue
        want = torch.from_numpy(share[i] / total[i])
        if not bool(((o - want).abs() <= want * (2.0 ** -8 + 2.0 ** -20)).all()):
            return f"segment {i}: shares off by up to {float(((o - want).abs() / want.clamp_min(1e-30)).max())}"
        log = math.log(total[i])
        if not bool(((l - log).abs() <= 2.0 ** -21 * log + 2.0 ** -22).all()):
            return f"segment {i}: log-sum-exp off by {float((l - log).abs().max())} of {log}"
    return None


def far_off(out, ref):
    """What is wrong with outputs over V of a normal distribution, or None (rows without a key: zeros)."""
    out, ref = out.double(), ref.double()
    some = (ref != 0).any(-1)
    if bool((out[~some] != 0).any()):
        return "a row without a key"
    off, size = (out - ref).norm(dim=-1)[some], ref.norm(dim=-1)[some]
    if not bool((off <= ROW_ERROR * size).all()):
        return f"a row is off by {float((off / size).max())}"
    if not float(off.norm()) <= ALL_ERROR * float(size.norm()):
        return f"off by {float(off.norm() / size.norm())}"
    return None
