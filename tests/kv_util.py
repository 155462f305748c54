"""A ragged batch over a paged 8-bit cache, held on the host beside the device
tensors, for the cache and attention tests."""
from __future__ import annotations

import numpy as np
import torch

import nested_bit_weight_int8_b200 as mq
from gpu_util import DEV

GARBAGE = 0xA7  # what unused bytes hold


class Batch:
    """seqs: list of (new rows, tokens with them). The held tokens' codes and
    scales are drawn; pages are scattered over the cache; table entries behind
    a sequence's last page are -1, bytes behind its last token garbage."""

    def __init__(self, seqs, heads, dim, page, seed=0, tail_rows=0, extra_pages=2, max_new=None, max_len=None,
                 fill="held"):
        rng = np.random.default_rng(seed)
        self.seqs, self.heads, self.dim, self.page = seqs, heads, dim, page
        self.starts = np.cumsum([0] + [n for n, _ in seqs])
        self.rows = int(self.starts[-1]) + tail_rows
        held = [-(-max(c, 0) // page) for _, c in seqs]
        n_pages = sum(held) + extra_pages
        order = rng.permutation(n_pages)[:sum(held)]
        self.table = np.full((len(seqs), max(max(held), 1)), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(held):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.codes = [np.full((n_pages, heads, page, dim), GARBAGE, dtype=np.uint8) for _ in range(2)]
        self.scales = [rng.uniform(0.004, 0.03, (n_pages, heads)).astype(np.float32) for _ in range(2)]
        for s, (n, c) in enumerate(seqs):
            have = c if fill == "all" else max(c - n, 0)
            for w in range(2):
                for j in range(-(-have // page)):
                    m = min(page, have - j * page)
                    x = np.clip(np.rint(rng.normal(0, 40, (heads, m, dim))), -127, 127)
                    self.codes[w][self.table[s, j], :, :m] = (x + 128).astype(np.uint8)
        self.k, self.v = (torch.from_numpy(c).to(DEV) for c in self.codes)
        self.ks, self.vs = (torch.from_numpy(c).to(DEV) for c in self.scales)
        self.cache = mq.KVCache(self.k, self.v, self.ks, self.vs)
        self.row_start = torch.tensor(self.starts, dtype=torch.int32, device=DEV)
        self.kv_len = torch.tensor([c for _, c in seqs], dtype=torch.int32, device=DEV)
        self.pages = torch.from_numpy(self.table).to(DEV)
        self.max_new = max(n for n, _ in seqs) if max_new is None else max_new
        self.max_len = max(c for _, c in seqs) if max_len is None else max_len
        self.batch = mq.KVBatch(self.row_start, self.kv_len, self.pages, self.rows, self.max_new, self.max_len)

    def host(self, which):
        """(codes, scales) of K (0) or V (1) now on the device."""
        t, c = ((self.k, self.ks), (self.v, self.vs))[which]
        return t.cpu().numpy(), c.cpu().numpy()

    def tokens(self, which, s, h, count, codes=None, scales=None):
        """Codes (count, dim) and page scales of one sequence and head."""
        codes = self.codes[which] if codes is None else codes
        scales = self.scales[which] if scales is None else scales
        pages = self.table[s, :-(-count // self.page)]
        c = codes[pages, h].reshape(-1, self.dim)[:count].astype(np.int64) - 128
        return c, scales[pages, h].copy()

    def places(self, s):
        n, c = self.seqs[s]
        return np.arange(c - n, c)


def bf16(x: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)
