"""The quantising cache write (mq_kv_append) and the read-back (mq_kv_read):
bytes and scales exactly where nothing is rotated, within half a step of the
float64 rotation where keys are; everything else of the cache untouched."""
import numpy as np
import pytest
import torch

import nested_bit_weight_int8_b200 as mq
from gpu_util import DEV
from kv_util import GARBAGE, Batch
from oracle import kv_cache as okv
from oracle import rope as orope

pytestmark = pytest.mark.gpu
KIND = {torch.float32: mq.MQ_F32, torch.bfloat16: mq.MQ_BF16}
LENGTHS = [  # (new rows, tokens with them): fresh, in a page, over pages, full pages, idle
    [(1, 1)], [(1, 17), (1, 16), (1, 0), (1, 400), (1, 129)], [(33, 33), (5, 40), (0, 20), (130, 131), (1, 64)],
    [(16, 32), (64, 64), (200, 260)],
]


def rows_of(b, heads, dtype, seed, gap=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(b.rows, heads * b.dim + gap, device=DEV, generator=g)
    x *= torch.rand(b.rows, 1, device=DEV, generator=g) * 4  # tokens of unlike sizes: scales grow
    return x.to(dtype)


def expect(b, which, x):
    """(codes, scales) after the write of x (rows, heads, dim) float32, from the start's."""
    codes, scales = b.codes[which].copy(), b.scales[which].copy()
    for s, (n, c) in enumerate(b.seqs):
        n = n if c else 0
        for h in range(b.heads):
            if n == 0:
                continue
            old, _ = b.tokens(which, s, h, c - n)
            pages = b.table[s, :-(-c // b.page)]
            co, sc = np.zeros((c, b.dim), dtype=np.int64), scales[pages, h].copy()
            co[:c - n] = old
            okv.write(co, sc, x[b.starts[s]:b.starts[s] + n, h], c - n, b.page)
            for j, p in enumerate(pages):
                m = min(b.page, c - j * b.page)
                if (j + 1) * b.page > c - n:
                    codes[p, h, :m] = (co[j * b.page:j * b.page + m] + 128).astype(np.uint8)
                    scales[p, h] = sc[j]
    return codes, scales


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("heads,dim,page", [(1, 16, 16), (2, 128, 64), (3, 96, 32), (1, 256, 128), (2, 80, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_bytes(lengths, heads, dim, page, dtype):
    b = Batch(lengths, heads, dim, page, seed=3, tail_rows=2)
    k, v = rows_of(b, heads, dtype, 1, gap=8), rows_of(b, heads, dtype, 2)
    for _ in range(2):  # the second write of the same tokens changes nothing
        mq.kv_append(b.cache, b.batch, k, v, KIND[dtype], heads * dim + 8, heads * dim)
        mq.device_status()
        for which, x in ((0, k[:, :heads * dim]), (1, v)):
            codes, scales = b.host(which)
            want, want_s = expect(b, which, x.float().cpu().numpy().reshape(b.rows, heads, dim))
            assert np.array_equal(scales, want_s)
            assert np.array_equal(codes, want)  # garbage behind the tokens and in other pages included


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("lengths", LENGTHS[1:])
@pytest.mark.parametrize("heads,group,dim,rot,page", [(2, 4, 128, 128, 64), (1, 7, 96, 48, 32), (2, 2, 256, 256, 16), (1, 1, 64, 8, 128)])
def test_append_rotated(layout, lengths, heads, group, dim, rot, page):
    b = Batch(lengths, heads, dim, page, seed=5, tail_rows=3)
    hq = heads * group
    qkv = rows_of(b, hq + 2 * heads, torch.float32, 9)
    pitch = qkv.shape[1]
    table = mq.RopeTable(10000.0, rot, layout, "yarn", (4.0, 32.0, 1.0, 4096.0), DEV)
    w, f = orope.frequencies(10000.0, rot, "yarn", (4.0, 32.0, 1.0, 4096.0))
    for positions in (None, torch.randint(0, 9999, (b.rows,), dtype=torch.int32, device=DEV)):
        b = Batch(lengths, heads, dim, page, seed=5, tail_rows=3)
        q_out = torch.full((b.rows, hq, dim), 3.0, device=DEV, dtype=torch.bfloat16)
        mq.kv_append(b.cache, b.batch, qkv[:, hq * dim:], qkv[:, (hq + heads) * dim:], mq.MQ_F32, pitch, pitch, rope=table,
                     positions=positions, q=qkv, q_stride=pitch, n_q_heads=hq, q_out=q_out)
        mq.device_status()
        x = qkv.cpu().numpy().reshape(b.rows, hq + 2 * heads, dim).astype(np.float64)
        real = b.starts[-1]
        at = np.concatenate([b.places(s) for s in range(len(b.seqs))]) if positions is None else positions[:real].cpu().numpy()
        turned = orope.rotate(x[:real], at, w, f, layout)
        tol = orope.f32_error(x[:real], rot, f, layout)
        q = q_out.float().cpu().numpy()
        assert np.all(np.abs(q[:real] - turned[:, :hq]) <= tol[:, :hq] + 2.0 ** -8 * (np.abs(turned[:, :hq]) + tol[:, :hq]) + 1e-30)
        assert np.all(q[real:] == 3.0)  # rows behind the last sequence
        codes, scales = b.host(1)
        want, want_s = expect(b, 1, x[:, hq + heads:].astype(np.float32))
        assert np.array_equal(codes, want) and np.array_equal(scales, want_s)
        # keys: the scale to rounding, each code the nearest to its value, up to the rotation's error
        codes, scales = b.host(0)
        for s, (n, c) in enumerate(b.seqs):
            for h in range(heads if c else 0):
                r0 = b.starts[s]
                y, e = turned[r0:r0 + n, hq + h], tol[r0:r0 + n, hq + h]
                got, got_s = b.tokens(0, s, h, c, codes, scales)
                for j in range((c - n) // page, -(-c // page)):
                    lo, hi = max(c - n, j * page), min(c, (j + 1) * page)
                    if lo >= hi:
                        continue
                    new, err = y[lo - (c - n):hi - (c - n)], e[lo - (c - n):hi - (c - n)]
                    m = np.abs(new).max() / 127
                    grown = max(m, b.scales[0][b.table[s, j], h]) if lo > j * page else m
                    assert abs(got_s[j] - grown) <= grown * 2.0 ** -23 + err.max() / 127
                    step = float(got_s[j])
                    assert np.all(np.abs(got[lo:hi] * step - new) <= step * 0.5 + err + 130 * step * 2.0 ** -23)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,dim,page", [(2, 128, 64), (1, 16, 16), (3, 80, 32), (1, 256, 128)])
def test_read_back(dtype, heads, dim, page):
    seqs = [(1, 300), (1, 1), (1, 0), (1, 128), (1, 77)]
    b = Batch(seqs, heads, dim, page, seed=7, fill="all")
    first = [37, 0, 0, 100, 60]
    counts = [200, 1, 2, 28, 40]  # the last asks for more tokens than there are, the third for an idle sequence's
    starts = np.cumsum([0] + counts)
    n = int(starts[-1])
    pad = 16
    outs = [torch.full((n, heads * dim + pad), 5.0, device=DEV, dtype=dtype) for _ in range(2)]
    mq.kv_read(b.cache, b.batch, torch.tensor(first, dtype=torch.int32, device=DEV),
               torch.tensor(starts, dtype=torch.int32, device=DEV), n, max(counts), *outs, KIND[dtype], heads * dim + pad)
    mq.device_status()
    for which in range(2):
        want = np.full((n, heads * dim + pad), 5.0, dtype=np.float32)
        for s, (_, c) in enumerate(seqs):
            m = min(counts[s], c - first[s])
            for h in range(heads if m > 0 else 0):
                co, sc = b.tokens(which, s, h, c)
                val = (co.astype(np.float32) * np.repeat(sc, page)[:c, None])[first[s]:first[s] + m]
                want[starts[s]:starts[s] + m, h * dim:(h + 1) * dim] = val
        want = torch.from_numpy(want).to(dtype)
        assert torch.equal(outs[which].cpu(), want)


def test_growing_token_by_token_keeps_half_a_step_each_time():
    # 40 calls of one token: the page's scale grows several times; each growth
    # moves a held value by at most half a new step
    heads, dim, page = 1, 32, 16
    b = Batch([(1, 1)], heads, dim, page, seed=1, extra_pages=6)
    b.pages = torch.tensor([[5, 1, 3]], dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(0)
    x = (rng.normal(size=(40, dim)) * np.linspace(0.5, 3, 40)[:, None]).astype(np.float32)
    dev = torch.from_numpy(x).to(DEV)
    kv_len = torch.zeros(1, dtype=torch.int32, device=DEV)
    batch = mq.KVBatch(b.row_start, kv_len, b.pages, 1, 1, 48)
    grown = np.zeros(40)
    last = {}
    for i in range(40):
        kv_len.fill_(i + 1)
        mq.kv_append(b.cache, batch, dev[i:], dev[i:], mq.MQ_F32, dim, dim)
        scale = float(b.vs[[5, 1, 3][i // page], 0])
        if scale > last.get(i // page, 0.0):
            grown[i // page * page:i + 1] += scale / 2  # this growth's rounding, the new token's included
        else:
            grown[i] += scale / 2
        last[i // page] = scale
    k = torch.empty(40, dim, device=DEV)
    v = torch.empty(40, dim, device=DEV)
    zero, ends = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0], [0, 40]))
    mq.kv_read(b.cache, batch, zero, ends, 40, 40, k, v, mq.MQ_F32, dim)
    mq.device_status()
    assert torch.equal(k, v)
    assert np.all(np.abs(v.cpu().numpy() - x) <= grown[:, None] * (1 + 2.0 ** -20))


def test_zero_tokens_zero_scale():
    b = Batch([(2, 2), (1, 20)], 2, 64, 16, seed=2)
    z = torch.zeros(3, 128, device=DEV)
    mq.kv_append(b.cache, b.batch, z, z, mq.MQ_F32, 128, 128)
    mq.device_status()
    codes, scales = b.host(0)
    p = b.table[0, 0]
    assert np.all(scales[p] == 0) and np.all(codes[p, :, :2] == 128) and np.all(codes[p, :, 2:] == GARBAGE)
    p = b.table[1, 1]  # a page that held tokens keeps its scale
    assert np.array_equal(scales[p], b.scales[0][p]) and np.all(codes[p, :, 3] == 128)


def test_a_captured_step_replays_with_the_lengths_of_then():
    heads, dim, page = 2, 64, 16
    b = Batch([(1, 1), (1, 1)], heads, dim, page, seed=4, extra_pages=10)
    b.pages = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32, device=DEV)
    kv_len = torch.ones(2, dtype=torch.int32, device=DEV)
    batch = mq.KVBatch(b.row_start, kv_len, b.pages, 2, 1, 48)
    x = torch.randn(2, heads * dim, device=DEV)
    mq.kv_append(b.cache, batch, x, x, mq.MQ_F32, heads * dim, heads * dim)
    b2 = [t.clone() for t in (b.k, b.v, b.ks, b.vs)]
    eager = mq.KVCache(*b2)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        mq.kv_append(b.cache, batch, x, x, mq.MQ_F32, heads * dim, heads * dim, stream=torch.cuda.current_stream())
    for i in range(2, 30):
        x.normal_()
        kv_len.fill_(i)
        graph.replay()
        mq.kv_append(eager, batch, x, x, mq.MQ_F32, heads * dim, heads * dim)
    torch.cuda.synchronize()
    mq.device_status()
    for a, c in zip((b.k, b.v, b.ks, b.vs), b2):
        assert torch.equal(a, c)


def test_batches_that_do_not_keep_their_bounds_are_reported_and_touch_nothing():
    heads, dim, page = 1, 64, 16
    x = torch.randn(8, dim, device=DEV)
    for spoil in ("page", "negative page", "rows", "length", "start"):
        b = Batch([(2, 20), (1, 3)], heads, dim, page, seed=6, max_new=2, max_len=20)
        if spoil == "page":
            b.pages[0, 1] = b.k.shape[0]
        elif spoil == "negative page":
            b.pages[0, 1] = -5
        elif spoil == "rows":
            b.row_start[1:] = torch.tensor([4, 5], dtype=torch.int32, device=DEV)
        elif spoil == "length":
            b.kv_len[0] = 21
        else:
            b.row_start[0] = -1
        mq.kv_append(b.cache, b.batch, x, x, mq.MQ_F32, dim, dim)
        with pytest.raises(mq.MQError) as e:
            mq.device_status()
        assert e.value.status == mq.MQ_ERR_BOUNDS
        codes, _ = b.host(0)
        p = b.table[0, :2]
        assert np.array_equal(codes[p], b.codes[0][p]), spoil
        mq.device_status()  # read and cleared


@pytest.mark.parametrize("low,high", [(-38, -30), (-44, -37), (-31, -29), (-3, 3), (20, 36)])
def test_codes_of_tiny_and_huge_values(low, high):
    # every quotient as correctly rounded, from subnormal scales to the largest
    b = Batch([(33, 70), (5, 5), (1, 16)], 2, 64, 16, seed=5)
    rng = np.random.default_rng(low + 100)
    with np.errstate(all="ignore"):
        x = (rng.standard_normal((b.rows, 2, 64)) * 10.0 ** rng.uniform(low, high, (b.rows, 2, 1))).astype(np.float32)
    x[3] = 0
    b.scales[0][:] = b.scales[1][:] = np.float32(10.0 ** low)
    b.ks.copy_(torch.from_numpy(b.scales[0]))
    b.vs.copy_(torch.from_numpy(b.scales[1]))
    rows = torch.from_numpy(x).to(DEV).view(b.rows, -1)
    mq.kv_append(b.cache, b.batch, rows, rows, mq.MQ_F32, 128, 128)
    mq.device_status()
    for which in range(2):
        codes, scales = expect(b, which, x)
        got_c, got_s = b.host(which)
        assert np.array_equal(got_s, scales) and np.array_equal(got_c, codes)


def test_more_sequences_than_one_round_finds():
    # the queries' search for their sequence beyond 32 sequences, and empty ones among them
    lengths = [(int(n), int(n) + int(c)) for n, c in np.random.default_rng(1).integers(0, 4, (150, 2))]
    b = Batch(lengths, 1, 64, 16, seed=6, tail_rows=3)
    table = mq.RopeTable(10000.0, 64, device=DEV)
    qkv = torch.randn(b.rows, 4 * 64, device=DEV)
    q = torch.full((b.rows, 2 * 64), 9.0, device=DEV, dtype=torch.bfloat16)
    mq.kv_append(b.cache, b.batch, qkv[:, 128:], qkv[:, 192:], mq.MQ_F32, 256, 256, rope=table, q=qkv, q_stride=256, n_q_heads=2,
                 q_out=q)
    mq.device_status()
    places = np.concatenate([b.places(s) for s in range(len(lengths))])
    w, f = orope.frequencies(10000.0, 64)
    x = qkv.cpu().numpy().astype(np.float64)[:len(places), :128].reshape(-1, 2, 64)
    want, tol = orope.rotate(x, places, w, f, "half"), orope.f32_error(x, 64, f, "half")
    got = q.float().cpu().numpy()
    assert np.all(np.abs(got[:len(places)].reshape(-1, 2, 64) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 1e-30)
    assert np.all(got[len(places):] == 9.0)


def test_pages_behind_the_first_four_gigabytes():
    # the same calls on a cache whose pages lie behind 2^32 bytes: the same bits
    seqs = [(3, 300), (200, 400), (1, 1000), (1, 0)]
    small = Batch(seqs, 8, 128, 128, seed=31)
    pages = 34000  # of 131072 bytes
    far = pages - small.k.shape[0] - 1
    assert far * 131072 > 1 << 32
    big = [torch.zeros(pages, 8, 128, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros(pages, 8, device=DEV) for _ in range(2)]
    for t, u in ((big[0], small.k), (big[1], small.v), (scales[0], small.ks), (scales[1], small.vs)):
        t[far:far + len(u)] = u
    table = torch.where(small.pages >= 0, small.pages + far, small.pages).contiguous()
    caches = [(small.cache, small.batch), (mq.KVCache(*big, *scales),
              mq.KVBatch(small.row_start, small.kv_len, table, small.rows, small.max_new, small.max_len))]
    qkv = torch.randn(small.rows, 48 * 128, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    rope, results = mq.RopeTable(10000.0, 128, device=DEV), []
    first = torch.zeros(4, dtype=torch.int32, device=DEV)
    ends = torch.tensor(np.cumsum([0] + [c for _, c in seqs]), dtype=torch.int32, device=DEV)
    n_out = int(ends[-1])
    for cache, batch in caches:
        q, out = (torch.empty(small.rows, 32 * 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        mq.kv_append(cache, batch, qkv[:, 32 * 128:], qkv[:, 40 * 128:], mq.MQ_F32, 48 * 128, 48 * 128, rope=rope, q=qkv,
                     q_stride=48 * 128, n_q_heads=32, q_out=q)
        scratch = torch.empty(mq.kv_attention_scratch_bytes(cache, batch, 32), dtype=torch.uint8, device=DEV)
        mq.kv_attention(cache, batch, q, 32 * 128, 32, 128 ** -0.5, out, 32 * 128, scratch)
        k, v = (torch.empty(n_out, 8 * 128, device=DEV) for _ in range(2))
        mq.kv_read(cache, batch, first, ends, n_out, 1000, k, v, mq.MQ_F32, 8 * 128)
        mq.device_status()
        results.append((q, out, k, v))
    for x, y in zip(*results):
        assert torch.equal(x, y)
    assert torch.equal(big[0][far:far + len(small.k)], small.k) and torch.equal(big[1][far:far + len(small.v)], small.v)
    assert not torch.any(scales[0][:far]) and not torch.any(scales[0][far + len(small.k):])
