"""Builders of paged batches for the tests of the operators of a step of many tokens."""
import numpy as np
import torch

from oracle import prompt
from packed_ternary_weight_b200 import tern


class Batch:
    """Sequences with the given new tokens and lengths, on shuffled pages of a cache filled with `fill` bytes."""

    def __init__(self, new, length, kvh, d, page, seed=0, fill=0xFF, spare=3, tail=0, pages=None):
        g = np.random.default_rng(seed)
        self.new, self.len = np.asarray(new), np.asarray(length)
        self.kvh, self.d, self.page = kvh, d, page
        need = -(-np.maximum(self.len, 0) // page)
        total = int(need.sum()) + spare
        ids = g.permutation(total)
        self.table = np.full((len(self.new), max(1, int(need.max(initial=0)))), -7, np.int32)  # unused entries name no page
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.tokens = int(self.start[-1])
        self.rows = self.tokens + tail
        self.raw = np.full(total * kvh * prompt.block_bytes(page, d), fill, np.uint8)
        self.g = g

    def oracle_cache(self, raw=None):
        return prompt.Cache(self.raw if raw is None else raw, self.kvh, self.d, self.page)

    def fill_values(self, spread=1.0):
        """Quantised normal keys and values at every position of every sequence (slots outside stay as filled)."""
        c = self.oracle_cache()
        for s in range(len(self.len)):
            for j in range(int(self.len[s])):
                for h in range(self.kvh):
                    for w in range(2):
                        x = (self.g.standard_normal(self.d) * spread + 0.2).astype(np.float32)
                        q, sc, m = prompt.quantize4(x[None])
                        c.put(int(self.table[s, j // self.page]), j % self.page, h, w, q[0], sc[0], m[0])

    def device(self, max_new=None, max_len=None):
        self.pages = torch.from_numpy(self.raw.copy()).cuda()
        cache = tern.KV4Cache(self.pages, self.kvh, self.d, self.page)
        dev = [torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda() for a in (self.start, self.len, self.table)]
        b = tern.KV4Batch(*dev, self.rows, int(self.new.max(initial=0)) if max_new is None else max_new,
                          int(self.len.max(initial=0)) if max_len is None else max_len)
        return cache, b

    def positions(self):
        """Sequence and position of every row."""
        return [(s, int(self.len[s]) - int(self.new[s]) + i) for s in range(len(self.new)) for i in range(int(self.new[s]))]


def bf16_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().bfloat16()


def workspace(cache, heads, seqs, max_new, max_len):
    n = cache.attention_workspace_size(seqs, max_new, max_len, heads)
    return torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
