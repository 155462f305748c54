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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_back_of_more_rows_than_the_batch_has_tokens(dtype):
    # rows at or behind kv_len are left as they were, however many of them are asked for
    heads, dim, page = 2, 64, 32
    seqs, counts, first = [(1, 64), (1, 33), (1, 0)], [100, 64, 70], [0, 20, 0]
    b = Batch(seqs, heads, dim, page, seed=3, fill="all")
    assert max(counts) > b.max_len
    ends = np.cumsum([0] + counts)
    k, v = (torch.full((int(ends[-1]), heads * dim), 5.0, device=DEV, dtype=dtype) for _ in range(2))
    mq.kv_read(b.cache, b.batch, torch.tensor(first, dtype=torch.int32, device=DEV),
               torch.tensor(ends, dtype=torch.int32, device=DEV), int(ends[-1]), max(counts), k, v,
               mq.MQ_F32 if dtype == torch.float32 else mq.MQ_BF16, heads * dim)
    mq.device_status()
    for which, got in ((0, k), (1, v)):
        want = np.full((int(ends[-1]), heads, dim), 5.0, dtype=np.float32)
        for s, (_, c) in enumerate(seqs):
            for h in range(heads if c else 0):
                codes, scales = b.tokens(which, s, h, c)
                x = codes.astype(np.float32) * np.repeat(scales, page)[:c, None]
                want[ends[s]:ends[s] + c - first[s], h] = x[first[s]:]
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype).view(got.shape))


def test_read_back_of_more_rows_than_max_out_is_reported():
    b = Batch([(1, 64)], 1, 64, 32, seed=3, fill="all")
    k, v = (torch.full((100, 64), 5.0, device=DEV) for _ in range(2))
    zero, ends = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0], [0, 50]))
    mq.kv_read(b.cache, b.batch, zero, ends, 100, 49, k, v, mq.MQ_F32, 64)
    with pytest.raises(mq.MQError) as e:
        mq.device_status()
    assert e.value.status == mq.MQ_ERR_BOUNDS and torch.all(k == 5.0) and torch.all(v == 5.0)


@pytest.mark.parametrize("rows", [1, 200])
def test_idle_sequences_need_no_pages(rows):
    # a page table of no columns: nothing is written, every row attends to nothing
    heads, dim = 2, 64
    b = Batch([(1, 20)], heads, dim, 16, seed=4)
    i32 = dict(dtype=torch.int32, device=DEV)
    batch = mq.KVBatch(torch.tensor([0, rows, rows + 1], **i32), torch.zeros(2, **i32), torch.empty(2, 0, **i32), rows + 1, rows, 0)
    x = torch.randn(rows + 1, heads * dim, device=DEV)
    mq.kv_append(b.cache, batch, x, x, mq.MQ_F32, heads * dim, heads * dim)
    q = x.to(torch.bfloat16)
    out, lse = torch.full_like(q, 9.0), torch.full((rows + 1, heads), 9.0, device=DEV)
    scratch = torch.empty(mq.kv_attention_scratch_bytes(b.cache, batch, heads), dtype=torch.uint8, device=DEV)
    mq.kv_attention(b.cache, batch, q, heads * dim, heads, 0.1, out, heads * dim, scratch, lse=lse)
    mq.device_status()
    assert torch.all(out == 0) and torch.all(lse == -torch.inf)
    for which in range(2):
        codes, scales = b.host(which)
        assert np.array_equal(codes, b.codes[which]) and np.array_equal(scales, b.scales[which])


def test_calls_on_empty_tensors_do_nothing():
    b = Batch([(1, 20)], 2, 64, 16, seed=4)
    i32 = dict(dtype=torch.int32, device=DEV)
    batch = mq.KVBatch(torch.zeros(2, **i32), torch.zeros(1, **i32), b.pages, 0, 0, 20)
    x, q = torch.empty(0, 128, device=DEV), torch.empty(0, 128, device=DEV, dtype=torch.bfloat16)
    mq.kv_append(b.cache, batch, x, x, mq.MQ_F32, 128, 128, q=x, q_stride=128, n_q_heads=2, q_out=q)
    scratch = torch.empty(mq.kv_attention_scratch_bytes(b.cache, batch, 2), dtype=torch.uint8, device=DEV)
    mq.kv_attention(b.cache, batch, q, 128, 2, 0.1, q, 128, scratch)
    mq.rope(x, mq.MQ_F32, 0, 2, 64, 128, torch.empty(0, **i32), mq.RopeTable(1e4, 64, device=DEV), x, mq.MQ_F32, 128)
    mq.device_status()
    for which in range(2):
        codes, scales = b.host(which)
        assert np.array_equal(codes, b.codes[which]) and np.array_equal(scales, b.scales[which])


def test_calls_back_to_back_read_what_the_call_before_wrote():
    # each kernel may start beside the one before it: queries, codes and scales that change with every
    # call, the neighbours' scales in the same lines among them, bit for bit as with a wait between the calls
    heads, group, dim, page, seqs = 8, 4, 64, 16, 24
    hq, pitch = heads * group, (heads * group + 2 * heads) * dim
    i32 = dict(dtype=torch.int32, device=DEV)
    rows = 3 * seqs
    starts = torch.arange(0, rows + 1, 3, **i32)
    tables = torch.randperm(seqs * 8, generator=torch.Generator().manual_seed(0)).view(seqs, 8).to(**i32)
    table = mq.RopeTable(10000.0, dim, device=DEV)
    positions, back = (torch.full((rows,), p, **i32) for p in (3, -3))

    def run(wait):
        gen = torch.Generator(device=DEV).manual_seed(1)
        pool = [torch.full((seqs * 8, heads, page, dim), 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
        cache = mq.KVCache(*pool, *(torch.zeros(seqs * 8, heads, device=DEV) for _ in range(2)))
        kv_len = torch.zeros(seqs, **i32)
        batch = mq.KVBatch(starts, kv_len, tables, rows, 3, 128)
        scratch = torch.empty(mq.kv_attention_scratch_bytes(cache, batch, hq), dtype=torch.uint8, device=DEV)
        x = [torch.randn(rows, pitch, device=DEV, generator=gen) * (1 + step) for step in range(40)]  # scales grow each time
        y, q, out = torch.empty(rows, pitch, device=DEV), torch.empty(rows, hq * dim, device=DEV, dtype=torch.bfloat16), []
        first, ends = torch.zeros(seqs, **i32), torch.arange(0, seqs * 4 + 1, 4, **i32)
        for step in range(40):
            kv_len += 3
            got = [torch.empty(rows, hq * dim, device=DEV, dtype=torch.bfloat16), *(torch.zeros(seqs * 4, heads * dim, device=DEV) for _ in range(2))]  # the first read asks for one token too many
            for call in (lambda: mq.rope(x[step], mq.MQ_F32, rows, pitch // dim, dim, pitch, positions, table, y, mq.MQ_F32, pitch),
                         lambda: mq.rope(y, mq.MQ_F32, rows, pitch // dim, dim, pitch, back, table, y, mq.MQ_F32, pitch),
                         lambda: mq.kv_append(cache, batch, y[:, hq * dim:], y[:, (hq + heads) * dim:], mq.MQ_F32, pitch, pitch,
                                              rope=table, q=y, q_stride=pitch, n_q_heads=hq, q_out=q),
                         lambda: mq.kv_attention(cache, batch, q, hq * dim, hq, dim ** -0.5, got[0], hq * dim, scratch),
                         lambda: mq.kv_read(cache, batch, first, ends, seqs * 4, 4, got[1], got[2], mq.MQ_F32, heads * dim)):
                call()
                if wait:
                    torch.cuda.synchronize()
            out.append(got)
        mq.device_status()
        return out

    for a, b in zip(run(True), run(False)):
        for u, v in zip(a, b):
            assert torch.equal(u, v)
