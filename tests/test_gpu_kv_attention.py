"""Attention over the 8-bit cache (mq_kv_attention) against the float64 softmax:
ragged batches from one token to prompts, grouped heads, windows, caps, padded
rows, long caches, odd head sizes, pages that end inside a tile."""
import math

import numpy as np
import pytest
import torch

import nested_bit_weight_int8_b200 as mq
from gpu_util import DEV
from kv_util import Batch
from oracle import kv_cache as okv

pytestmark = pytest.mark.gpu


def attend(b, hq, q, softcap=0.0, window=0, scale=None, lse=True, stream=None, scratch=None, gap=0):
    dim = b.dim
    out = torch.full((b.rows, hq * dim + gap), 9.0, device=DEV, dtype=torch.bfloat16)
    log = torch.full((b.rows, hq), 9.0, device=DEV) if lse else None
    if scratch is None:
        scratch = torch.full((mq.kv_attention_scratch_bytes(b.cache, b.batch, hq),), 0xFF, dtype=torch.uint8, device=DEV)
    mq.kv_attention(b.cache, b.batch, q, q.stride(0), hq, dim ** -0.5 if scale is None else scale, out, hq * dim + gap, scratch,
                    lse=log, softcap=softcap, window=window, stream=stream)
    return out, log


def queries(b, hq, seed=0, size=1.0, gap=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(b.rows, hq * b.dim + gap, device=DEV, generator=g) * size).to(torch.bfloat16)


def check(b, hq, q, out, log, softcap=0.0, window=0, scale=None, gap=0, rows=None):
    dim, group = b.dim, hq // b.heads
    scale = dim ** -0.5 if scale is None else scale
    q64 = q.float().cpu().numpy().astype(np.float64)[:, :hq * dim].reshape(b.rows, hq, dim)
    got = out.float().cpu().numpy()
    lse = None if log is None else log.cpu().numpy().astype(np.float64)
    worst = 0.0
    for s, (n, c) in enumerate(b.seqs):
        r0 = b.starts[s]
        pick = np.arange(n) if rows is None else np.array([r for r in rows if r < n], dtype=int)
        for h in range(b.heads):
            (kc, ks), (vc, vs) = (b.tokens(w, s, h, c) for w in range(2))
            k, v = okv.values(kc, ks, b.page), okv.values(vc, vs, b.page)
            of_token = np.repeat(vs.astype(np.float64), b.page)[:c]
            for a in range(h * group, (h + 1) * group):
                x = q64[r0:r0 + n, a][pick]
                o, l, mass, gross = okv.attend(x, k, v, of_token, b.places(s)[pick], scale, softcap, window)
                delta = okv.score_error(x, ks.max(initial=0.0), scale, softcap)
                tol = okv.out_error(o, mass, gross, vs.max(initial=0.0), delta, c)
                err = np.abs(got[r0:r0 + n, a * dim:(a + 1) * dim][pick] - o)
                assert np.all(err <= tol), (s, a, (err / np.maximum(tol, 1e-30)).max())
                worst = max(worst, (err / np.maximum(tol, 1e-30)).max(initial=0.0))
                if lse is not None:
                    g = lse[r0:r0 + n, a][pick]
                    assert np.array_equal(np.isinf(g), np.isinf(l)) and np.all(g[np.isinf(l)] < 0)
                    f = np.isfinite(l)
                    assert np.all(np.abs(g[f] - l[f]) <= okv.lse_error(l, delta, c)[f])
    tail = int(b.starts[-1])
    assert np.all(got[tail:] == 9.0) and (gap == 0 or np.all(got[:, hq * dim:] == 9.0))
    return worst


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,group,dim", [(1, 1, 64), (2, 4, 128), (1, 8, 128), (2, 2, 256), (1, 7, 96), (3, 1, 16),
                                             (1, 16, 80), (1, 20, 128), (1, 17, 256), (2, 3, 192)])
def test_single_tokens(page, heads, group, dim):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 300, 777]
    b = Batch([(1, c) for c in lens], heads, dim, page, seed=dim + page, tail_rows=2, fill="all")
    q = queries(b, heads * group)
    out, log = attend(b, heads * group, q)
    mq.device_status()
    check(b, heads * group, q, out, log)


@pytest.mark.parametrize("window,softcap", [(0, 0.0), (1, 0.0), (5, 0.0), (37, 20.0), (64, 0.0), (200, 50.0), (100000, 0.0)])
@pytest.mark.parametrize("heads,group,dim,page", [(2, 4, 128, 64), (1, 2, 256, 16), (2, 1, 64, 32)])
def test_drafted_tokens_windows_and_caps(window, softcap, heads, group, dim, page):
    seqs = [(5, 5), (3, 40), (8, 130), (1, 0), (4, 2), (0, 50), (2, 257), (7, 64)]  # (4, 2): two padded rows
    b = Batch(seqs, heads, dim, page, seed=window, fill="all")
    q = queries(b, heads * group, size=2.0)
    out, log = attend(b, heads * group, q, softcap, window)
    mq.device_status()
    check(b, heads * group, q, out, log, softcap, window)


@pytest.mark.parametrize("heads,group,dim,page,window,softcap", [
    (1, 4, 128, 64, 0, 0.0), (2, 1, 64, 16, 50, 0.0), (1, 2, 256, 32, 0, 30.0), (1, 7, 96, 128, 0, 0.0), (2, 8, 128, 32, 333, 0.0),
    (1, 1, 192, 64, 0, 0.0), (1, 2, 32, 16, 17, 0.0)])
def test_prompts_beside_single_tokens(heads, group, dim, page, window, softcap):
    seqs = [(300, 300), (1, 500), (129, 700), (1, 0), (65, 65), (2, 3), (0, 10), (257, 400)]
    b = Batch(seqs, heads, dim, page, seed=11, tail_rows=1, fill="all")
    q = queries(b, heads * group)
    out, log = attend(b, heads * group, q, softcap, window)
    mq.device_status()
    check(b, heads * group, q, out, log, softcap, window)


@pytest.mark.parametrize("heads,group,dim,page", [(1, 3, 80, 16), (2, 1, 16, 32), (1, 2, 144, 64), (1, 1, 240, 16), (1, 40, 128, 32),
                                                  (1, 40, 256, 64), (2, 5, 48, 128)])
def test_prompts_of_odd_heads_and_wide_groups(heads, group, dim, page):
    seqs = [(150, 210), (1, 90), (3, 3), (33, 500), (1, 0)]
    b = Batch(seqs, heads, dim, page, seed=21, tail_rows=3, fill="all")
    q = queries(b, heads * group)
    out, log = attend(b, heads * group, q)
    mq.device_status()
    check(b, heads * group, q, out, log)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompts_with_padded_rows_and_rows_that_see_nothing(dim):
    # more rows than tokens: the first rows stand before the sequence and see nothing
    seqs = [(300, 0), (257, 100), (129, 129), (200, 1), (1, 0), (2, 900), (260, 0)]
    b = Batch(seqs, 2, dim, 32, seed=22, tail_rows=1, fill="all")
    for window in (0, 7):
        q = queries(b, 4)
        out, log = attend(b, 4, q, window=window)
        mq.device_status()
        check(b, 4, q, out, log, window=window)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompts_whose_scores_rise_and_scales_differ(dim):
    # each page's keys score higher than all before, V's scales jump over many
    # orders: the running maximum and the largest scale rise again and again
    b = Batch([(270, 900), (130, 513)], 1, dim, 16, seed=23, fill="all")
    rng = np.random.default_rng(23)
    for s in range(2):
        for j, page in enumerate(b.table[s]):
            if page >= 0:
                b.scales[0][page] = 0.002 * 1.12 ** j
                b.scales[1][page] = 10.0 ** rng.uniform(-20, 3)
    b.ks.copy_(torch.from_numpy(b.scales[0]))
    b.vs.copy_(torch.from_numpy(b.scales[1]))
    for size in (0.0, 0.3, 3.0):
        q = queries(b, 2, seed=int(size * 10), size=size)
        out, log = attend(b, 2, q)
        mq.device_status()
        check(b, 2, q, out, log)
    b.scales[0][:] = b.scales[1][:] = 0
    b.ks.zero_()
    b.vs.zero_()
    out, log = attend(b, 2, q)
    check(b, 2, q, out, log)


@pytest.mark.parametrize("seqs", [[(3, 200), (1, 17)], [(200, 300), (1, 17)]])
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_scales_of_either_sign(seqs, scale):
    b = Batch(seqs, 1, 128, 32, seed=24, fill="all")
    q = queries(b, 4)
    for cap in (0.0, 5.0):
        out, log = attend(b, 4, q, softcap=cap, scale=scale)
        mq.device_status()
        check(b, 4, q, out, log, softcap=cap, scale=scale)


@pytest.mark.parametrize("cap", [0.01, 64.0, 100.0, 5000.0, 1e6, 2.0 ** 60])
def test_narrow_and_wide_caps(cap):
    b = Batch([(200, 300), (3, 200), (1, 17)], 1, 128, 32, seed=28, fill="all")
    for size in (0.01, 2.0):
        q = queries(b, 2, size=size)
        out, log = attend(b, 2, q, softcap=cap)
        mq.device_status()
        check(b, 2, q, out, log, softcap=cap)


@pytest.mark.parametrize("dim", [64, 256])
def test_nan_and_infinite_queries_stay_in_their_rows_of_a_prompt(dim):
    b = Batch([(300, 350), (1, 9)], 1, dim, 16, seed=25, fill="all")
    q = queries(b, 1)
    bad = torch.zeros(b.rows, dtype=torch.bool, device=DEV)
    for row, value in ((5, "nan"), (131, "inf"), (299, "-inf")):
        q[row, row % dim] = float(value)
        bad[row] = True
    out, log = attend(b, 1, q)
    mq.device_status()
    # (not bit by bit: rows of a warp raise their maxima together)
    check(b, 1, q, out, log, rows=[r for r in range(300) if not bad[r]])
    assert torch.all(~torch.isfinite(out[bad])) and torch.all(~torch.isfinite(log[bad]))


def test_two_prompt_calls_at_once_and_a_graph_that_sees_new_lengths():
    for dim in (64, 128, 256):
        b = Batch([(260, 700), (1, 90), (140, 300)], 2, dim, 64, seed=26, fill="all")
        q = queries(b, 8)
        want = {}
        for c in (700, 650, 100):
            b.kv_len[0] = c
            want[c] = [t.clone() for t in attend(b, 8, q)]
        b.kv_len[0] = 700
        size = mq.kv_attention_scratch_bytes(b.cache, b.batch, 8)
        scr = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
        streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
        torch.cuda.synchronize()
        for _ in range(5):
            for s, m in zip(streams, scr):
                with torch.cuda.stream(s):
                    got.append(attend(b, 8, q, stream=s, scratch=m))
        torch.cuda.synchronize()
        for o, l in got:
            assert torch.equal(o, want[700][0]) and torch.equal(l, want[700][1])
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            out, log = attend(b, 8, q, stream=torch.cuda.current_stream(), scratch=scr[0])
        for c in (650, 100, 700):
            b.kv_len[0] = c
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[c][0]) and torch.equal(log, want[c][1])
        mq.device_status()


def test_a_long_cache_and_many_sequences():
    b = Batch([(1, 70001)], 2, 128, 128, seed=1, fill="all")
    q = queries(b, 8)
    out, log = attend(b, 8, q)
    check(b, 8, q, out, log)
    rng = np.random.default_rng(0)
    b = Batch([(1, int(c)) for c in rng.integers(0, 90, 700)], 1, 64, 16, seed=2, fill="all")
    q = queries(b, 2)
    out, log = attend(b, 2, q)
    mq.device_status()
    check(b, 2, q, out, log)


def test_peaked_flat_and_tiny_probabilities():
    # one far outweighing key, then keys of equal score whose weights sum the
    # values of a long cache, then values of very unlike scales
    b = Batch([(1, 900)], 1, 128, 16, seed=3, fill="all")
    for size in (0.0, 1e-3, 1.0, 40.0):
        q = queries(b, 4, seed=5, size=size)
        out, log = attend(b, 4, q)
        check(b, 4, q, out, log)
    b.scales[1][:] = 10.0 ** np.random.default_rng(4).uniform(-20, 3, b.scales[1].shape).astype(np.float32)
    b.vs.copy_(torch.from_numpy(b.scales[1]))
    q = queries(b, 4)
    out, log = attend(b, 4, q)
    check(b, 4, q, out, log)
    b.scales[1][:] = 0
    b.vs.zero_()
    out, log = attend(b, 4, q)
    check(b, 4, q, out, log)
    assert torch.all(out[:, :4 * 128] == 0)


def test_queries_of_unlike_sizes():
    b = Batch([(3, 200)], 1, 128, 32, seed=3, fill="all")
    q = queries(b, 4)
    q[0] *= 1e30
    q[1] *= 1e-30
    q[2, :64] *= 1e-6
    out, log = attend(b, 4, q, scale=1e-29)
    check(b, 4, q, out, log, scale=1e-29)


def test_what_lies_behind_the_tokens_has_no_part():
    # garbage scales and bytes in pages that the table does not name, garbage
    # behind kv_len in the last page: the same outputs, bit for bit
    for seqs in ([(1, 100), (2, 37)], [(200, 231)]):
        b = Batch(seqs, 2, 64, 32, seed=8, fill="all")
        q = queries(b, 4)
        out, log = attend(b, 4, q)
        used = {int(p) for p in b.table.ravel() if p >= 0}
        spare = [p for p in range(b.k.shape[0]) if p not in used]
        b.ks[spare], b.vs[spare] = float("nan"), float("inf")
        for s, (_, c) in enumerate(seqs):
            b.k[b.table[s, c // 32], :, c % 32:] = 255
            b.v[b.table[s, c // 32], :, c % 32:] = 0
        again, log2 = attend(b, 4, q)
        mq.device_status()
        assert torch.equal(out, again) and torch.equal(log, log2)


def test_nan_and_infinite_queries_stay_in_their_rows():
    b = Batch([(3, 50), (1, 9)], 1, 64, 16, seed=8, fill="all")
    q = queries(b, 2)
    out, log = attend(b, 2, q)
    q[1, 5] = float("nan")
    q[2, 64 + 7] = float("inf")
    again, log2 = attend(b, 2, q)
    mq.device_status()
    same = torch.tensor([[True, True], [False, True], [True, False], [True, True]], device=DEV)
    o, a = out.view(4, 2, 64), again.view(4, 2, 64)
    assert torch.equal(o[same], a[same]) and torch.equal(log[same], log2[same])
    assert torch.all(~torch.isfinite(a[~same])) and torch.all(~torch.isfinite(log2[~same]))


def test_the_same_call_gives_the_same_bits_and_strides_do_not_matter():
    b = Batch([(1, 5000), (4, 333), (1, 64)], 2, 128, 64, seed=9, fill="all")
    q = queries(b, 8, gap=24)
    outs = [attend(b, 8, q, gap=8, lse=i != 1) for i in range(3)]
    mq.device_status()
    check(b, 8, q, *outs[0], gap=8)
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and (l is None or torch.equal(l, outs[0][1]))


@pytest.mark.parametrize("heads,group,dim,page,seqs", [
    (1, 1, 64, 16, None), (2, 4, 128, 64, None), (1, 1, 192, 64, None), (1, 2, 256, 32, None),
    (4, 8, 256, 64, [(9, 500 + 37 * i) for i in range(16)]), (4, 8, 128, 64, [(17, 300 + 91 * i) for i in range(16)])])
def test_prompts_give_the_same_bits_every_time(heads, group, dim, page, seqs):
    seqs = seqs or [(300, 300), (1, 500), (129, 700), (65, 65), (257, 900)]
    b = Batch(seqs, heads, dim, page, seed=11, fill="all")
    q = queries(b, heads * group)
    out, log = attend(b, heads * group, q)
    check(b, heads * group, q, out, log)
    for _ in range(60):
        again, log2 = attend(b, heads * group, q)
        assert torch.equal(out, again) and torch.equal(log, log2)
    mq.device_status()


def test_two_streams_and_a_graph_that_sees_new_lengths():
    b = Batch([(1, 700), (1, 90)], 2, 128, 64, seed=10, fill="all")
    q = queries(b, 8)
    want = {}
    for c in (700, 650, 3):
        b.kv_len[0] = c
        want[c] = [t.clone() for t in attend(b, 8, q)]
    torch.cuda.synchronize()
    # two calls at once, each with its own scratch
    b.kv_len[0] = 700
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    size = mq.kv_attention_scratch_bytes(b.cache, b.batch, 8)
    scr = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, m in ((s1, scr[0]), (s2, scr[1])):
        with torch.cuda.stream(s):
            got.append(attend(b, 8, q, stream=s, scratch=m))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[700][0]) and torch.equal(l, want[700][1])
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        out, log = attend(b, 8, q, stream=torch.cuda.current_stream(), scratch=scr[0])
    for c in (650, 3, 700):
        b.kv_len[0] = c
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[c][0]) and torch.equal(log, want[c][1])
    mq.device_status()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_waits_that_give_up_are_reported_and_the_next_call_is_whole(dim):
    b = Batch([(200, 300), (1, 500), (3, 40)], 2, dim, 32, seed=27, fill="all")
    q = queries(b, 4)
    want = attend(b, 4, q)
    mq.device_status()
    mq.debug_set_wait_limit_ns(0)  # every wait gives up at once
    try:
        attend(b, 4, q)
        with pytest.raises(mq.MQError) as e:
            mq.device_status()
        assert e.value.status == mq.MQ_ERR_TIMEOUT
    finally:
        mq.debug_set_wait_limit_ns(2_000_000_000)
    out, log = attend(b, 4, q)
    mq.device_status()
    assert torch.equal(out, want[0]) and torch.equal(log, want[1])


@pytest.mark.parametrize("n", [1, 3, 200])
def test_pages_before_the_window_may_be_gone(n):
    b = Batch([(n, 700), (min(n, 5), 40)], 2, 64, 16, seed=14, fill="all")
    q = queries(b, 4)
    window = 100
    out, log = attend(b, 4, q, window=window)
    check(b, 4, q, out, log, window=window)
    gone = (700 - n - window + 1) // 16
    b.pages[0, :gone] = -1
    again, log2 = attend(b, 4, q, window=window)
    mq.device_status()
    assert torch.equal(out, again) and torch.equal(log, log2)


@pytest.mark.parametrize("n", [1, 200])
def test_bad_pages_and_bounds_are_reported(n):
    for spoil in ("page", "length", "rows"):
        b = Batch([(1, 40), (n, 33)], 1, 64, 16, seed=12, max_len=40, fill="all")
        q = queries(b, 2)
        out, _ = attend(b, 2, q)
        mq.device_status()
        if spoil == "page":
            b.pages[1, 1] = 1 << 30
        elif spoil == "length":
            b.kv_len[1] = 41
        else:
            b.row_start[2] = n + 2
        again, _ = attend(b, 2, q)
        with pytest.raises(mq.MQError) as e:
            mq.device_status()
        assert e.value.status == mq.MQ_ERR_BOUNDS
        assert torch.equal(out[0], again[0])  # the other sequence


def test_write_then_attend_then_read_as_a_decode_loop():
    # eight steps of two sequences: the attention of each step against the
    # float64 softmax over what the cache stands for at that step
    heads, group, dim, page = 2, 2, 64, 16
    hq = heads * group
    b = Batch([(1, 30), (1, 13)], heads, dim, page, seed=13, extra_pages=6)
    free = [p for p in range(b.k.shape[0]) if p not in set(b.table.ravel())]
    b.table = np.concatenate([b.table, np.array([[free[0]], [free[1]]], dtype=np.int32)], 1)
    b.table[1, 1] = free[2]
    b.pages = torch.from_numpy(b.table).to(DEV)
    table = mq.RopeTable(10000.0, dim, device=DEV)
    scratch = None
    for step in range(8):
        b.seqs = [(1, 30 + step), (1, 13 + step)]
        kv_len = torch.tensor([c for _, c in b.seqs], dtype=torch.int32, device=DEV)
        b.batch = mq.KVBatch(b.row_start, kv_len, b.pages, 2, 1, 48)
        qkv = torch.randn(2, (hq + 2 * heads) * dim, device=DEV)
        q = torch.empty(2, hq * dim, device=DEV, dtype=torch.bfloat16)
        pitch = qkv.shape[1]
        mq.kv_append(b.cache, b.batch, qkv[:, hq * dim:], qkv[:, (hq + heads) * dim:], mq.MQ_F32, pitch, pitch, rope=table,
                     q=qkv, q_stride=pitch, n_q_heads=hq, q_out=q)
        out, log = attend(b, hq, q, scratch=scratch)
        mq.device_status()
        (b.codes[0], b.scales[0]), (b.codes[1], b.scales[1]) = b.host(0), b.host(1)
        check(b, hq, q, out, log)
    assert math.isfinite(float(out.float().abs().sum()))
