"""The cache's write at the smallest scales and its read-back where more rows are asked for than a
sequence holds."""
import numpy as np
import pytest
import torch

import nested_bit_weight_int8_b200 as mq
from gpu_util import DEV
from kv_util import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held", [0, 3])
def test_codes_stay_in_range_on_pages_of_subnormal_values(held):
    # a page for each largest value k 2^-149, k = 1 .. 20000: the scale, k / 127 steps of 2^-149,
    # rounds by up to half of itself, so a quotient may pass 127 by far
    pages, page, dim = 20000, 16, 16
    n = page - held
    rng = np.random.default_rng(held)
    k = np.arange(1, pages + 1)
    x = (rng.uniform(-1, 1, (pages, n, dim)) * k[:, None, None]).round()
    x[:, -1, 3], x[:, 0, 5] = k, -k
    x = np.ldexp(x, -149).astype(np.float32)
    # pages that hold tokens are sequences of their own, the others one long sequence
    seqs = [(n, page)] * pages if held else [(page * pages, page * pages)]
    batches = [range(i, min(i + 10000, pages)) for i in range(0, pages, 10000)] if held else [range(pages)]
    for part in batches:
        b = Batch([seqs[i] for i in part] if held else seqs, 1, dim, page, seed=1)
        mine = b.table.reshape(-1)[:len(part)]
        old = np.ldexp(rng.integers(0, 3, len(b.scales[0])), -149).astype(np.float32)[:, None]
        for w, t in enumerate((b.ks, b.vs)):
            b.scales[w][:] = old
            t.copy_(torch.from_numpy(b.scales[w]))
        rows = torch.from_numpy(x[part.start:part.stop].reshape(-1, dim)).to(DEV)
        mq.kv_append(b.cache, b.batch, rows, rows, mq.MQ_F32, dim, dim)
        mq.device_status()
        new = x[part.start:part.stop]
        scale = np.abs(new).max((1, 2)) / np.float32(127)
        was = old[mine, 0]
        if held:
            scale = np.maximum(scale, was)
        with np.errstate(divide="ignore", invalid="ignore"):
            want = np.clip(np.rint(new / scale[:, None, None]), -127, 127)
            want[scale == 0] = 0
        for which in range(2):
            before = b.codes[which][mine, 0, :held].astype(np.float32) - 128
            with np.errstate(divide="ignore", invalid="ignore"):
                grown = np.rint(before * was[:, None, None] / scale[:, None, None])
            before = np.where((scale > was)[:, None, None], grown, before)
            codes, scales = b.host(which)
            assert np.array_equal(scales[mine, 0], scale)
            assert np.array_equal(codes[mine, 0, held:].astype(int) - 128, want.astype(int))
            assert np.array_equal(codes[mine, 0, :held].astype(int) - 128, before.astype(int))
