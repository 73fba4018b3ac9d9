"""A paged 4-bit cache and its sequences for the GPU tests."""
import numpy as np
import torch


class Paged:
    """Sequences of lengths `total` in pages handed out in random order, their table padded with -1."""

    def __init__(self, rng, total, heads, D, page, spare=2, wide=1):
        import audio_dit_gb300 as A
        self.total, self.heads, self.D, self.page = list(total), heads, D, page
        need = [(n + page - 1) // page for n in total]
        self.n_pages = sum(need) + spare
        ids = rng.permutation(self.n_pages)
        self.table = np.full((len(total), max(need + [1]) + wide), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.cache = A.alloc_kv_cache(self.n_pages, heads, D, page)
        # what no token was written to may hold anything: NaN block scales, all codes set
        self.cache.fill_(0xFF)
        self.k_gscale, self.v_gscale = (torch.from_numpy(rng.uniform(0.001, 0.01, heads).astype(np.float32))
                                        for _ in range(2))

    def args(self, rows=None, total=None):
        """Positional arguments of a call whose last `rows` of each sequence are its own (None: one each)."""
        t = torch.from_numpy(self.table).cuda()
        n = torch.tensor(self.total if total is None else total, dtype=torch.int32).cuda()
        off = None if rows is None else torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32).cuda()
        return t, n, off

    def scales(self):
        return dict(k_gscale=self.k_gscale.cuda(), v_gscale=self.v_gscale.cuda())

    def fill(self, rng):
        """Random keys and values of all sequences into the cache: lists of bf16 [len, heads, D]."""
        import audio_dit_gb300 as A
        gain = torch.from_numpy(np.exp(0.4 * rng.standard_normal((self.heads, self.D))).astype(np.float32))
        kv = [(torch.from_numpy(rng.standard_normal((sum(self.total), self.heads, self.D), dtype=np.float32)) * gain)
              .to(torch.bfloat16) for _ in range(2)]
        if sum(self.total):
            A.h3fp4_cache_append(kv[0].cuda(), kv[1].cuda(), self.cache, *self.args(self.total), **self.scales())
        return [list(t.split(self.total)) for t in kv]
