"""Argument checks of the rotary positions, the cache and its attention: every
refusal happens on the host, before a launch (no GPU needed)."""
import ctypes
import math
import subprocess
import sys

import numpy as np
import pytest
import torch

import nested_bit_weight_int8_b200 as mq
from oracle import rope as orope

F = 1 << 20  # an aligned non-null address; never dereferenced by rejected calls
BAD, NOT_SERVED = mq.MQ_ERR_INVALID_ARG, mq.MQ_ERR_UNSUPPORTED


def cache(**kw):
    d = dict(k=F, v=F, k_scale=F, v_scale=F, n_pages=8, page_tokens=64, n_kv_heads=2, head_dim=128)
    return mq.KVCacheDesc(**{**d, **kw})


def batch(**kw):
    d = dict(row_start=F, kv_len=F, page_table=F, n_seqs=2, max_pages=4, n_rows=2, max_new=1, max_len=256)
    return mq.KVBatchDesc(**{**d, **kw})


def rope(**kw):
    return mq.RopePositions(**{**dict(turns=F, rot_dim=128, layout=0, factor=1.0), **kw})


def call(fn, base, **kw):
    return fn(*{**base, **kw}.values())


ROPE = dict(x=F, xt=0, rows=4, heads=2, dim=128, xs=256, pos=F, rope=rope(), y=F, yt=0, ys=256, stream=None)
APPEND = dict(c=cache(), b=batch(), k=F, v=F, dtype=0, ks=256, vs=256, rope=rope(), pos=None, q=F, qs=1024, hq=8, qo=F, stream=None)
READ = dict(c=cache(), b=batch(), first=F, out=F, n=4, m=2, k=F, v=F, dtype=0, stride=256, stream=None)
ATTEND = dict(c=cache(), b=batch(), q=F, qs=1024, hq=8, scale=0.1, cap=0.0, window=0, out=F, os=1024, lse=None, scr=F,
              size=1 << 40, stream=None)
CACHES = [(dict(k=None), BAD), (dict(v=F + 8), BAD), (dict(k_scale=F + 2), BAD), (dict(page_tokens=24), BAD),
          (dict(page_tokens=8), BAD), (dict(page_tokens=256), BAD), (dict(head_dim=24), BAD), (dict(head_dim=272), BAD),
          (dict(head_dim=0), BAD), (dict(n_pages=0), BAD), (dict(n_kv_heads=0), BAD), (dict(n_kv_heads=1025), NOT_SERVED)]
BATCHES = [(dict(n_seqs=-1), BAD), (dict(row_start=None), BAD), (dict(kv_len=F + 1), BAD), (dict(page_table=None), BAD),
           (dict(max_len=257), BAD), (dict(n_rows=-1), BAD), (dict(max_new=-1), BAD), (dict(n_seqs=65536), NOT_SERVED)]


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(xt=2), BAD), (dict(rows=-1), BAD), (dict(heads=0), BAD), (dict(dim=127), BAD),
    (dict(dim=514, xs=2000, ys=2000), NOT_SERVED), (dict(xs=255), BAD), (dict(ys=255), BAD), (dict(pos=None), BAD),
    (dict(pos=F + 2), BAD), (dict(rope=None), BAD), (dict(rope=rope(turns=None)), BAD), (dict(rope=rope(rot_dim=130)), BAD),
    (dict(rope=rope(rot_dim=7)), BAD), (dict(rope=rope(layout=2)), BAD), (dict(rope=rope(factor=math.inf)), BAD),
    (dict(x=F + 2), BAD), (dict(yt=1), BAD), (dict(ys=512), BAD)])  # the last two: in place with another type, stride
def test_rope_refuses(kw, want):
    assert call(mq._rope, ROPE, **kw) == want, kw
    assert "mq_rope" in mq.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), BAD), (dict(v=F + 8), BAD), (dict(dtype=3), BAD), (dict(ks=255), BAD), (dict(vs=258), BAD),
    (dict(rope=rope(rot_dim=20)), NOT_SERVED), (dict(rope=rope(rot_dim=256)), BAD), (dict(rope=None, pos=F), BAD),
    (dict(pos=F + 2), BAD), (dict(qo=None), BAD), (dict(q=None), BAD), (dict(hq=0), BAD), (dict(qs=1000), BAD),
    (dict(c=None), BAD), (dict(b=None), BAD)])
def test_append_refuses(kw, want):
    assert call(mq._kv_append, APPEND, **kw) == want, kw
    assert "mq_kv_append" in mq.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(first=None), BAD), (dict(out=F + 1), BAD), (dict(n=-1), BAD), (dict(m=-1), BAD), (dict(k=F + 8), BAD),
    (dict(v=None), BAD), (dict(stride=252), BAD), (dict(dtype=1, stride=260), BAD), (dict(dtype=2), BAD)])
def test_read_refuses(kw, want):
    assert call(mq._kv_read, READ, **kw) == want, kw
    assert "mq_kv_read" in mq.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), BAD), (dict(q=F + 8), BAD), (dict(qs=1020), BAD), (dict(qs=1000), BAD), (dict(hq=7), BAD), (dict(hq=0), BAD),
    (dict(hq=1), BAD), (dict(scale=math.nan), BAD), (dict(cap=-1.0), BAD), (dict(cap=math.inf), BAD), (dict(cap=2.0 ** -61), BAD),
    (dict(cap=2.0 ** 61), BAD), (dict(cap=math.nan), BAD), (dict(window=-1), BAD),
    (dict(out=None), BAD), (dict(os=1023), BAD), (dict(lse=F + 2), BAD), (dict(scr=None), BAD), (dict(scr=F + 128), BAD),
    (dict(size=64), BAD), (dict(hq=32768, qs=1 << 23, os=1 << 23), NOT_SERVED)])
def test_attention_refuses(kw, want):
    assert call(mq._kv_attention, ATTEND, **kw) == want, kw
    assert "mq_kv_attention" in mq.last_error()


@pytest.mark.parametrize("fn,base", [(mq._kv_append, APPEND), (mq._kv_read, READ), (mq._kv_attention, ATTEND)])
def test_every_cache_call_checks_the_cache_and_the_batch(fn, base):
    for kw, want in CACHES:
        assert call(fn, base, c=cache(**kw)) == want, kw
    for kw, want in BATCHES:
        assert call(fn, base, b=batch(**kw)) == want, kw


def test_nothing_to_do_is_no_error():
    for kw in (dict(n_seqs=0, row_start=None, kv_len=None, page_table=None), dict(n_rows=0), dict(max_new=0)):
        assert call(mq._kv_append, APPEND, b=batch(**kw)) == mq.MQ_OK
        assert call(mq._kv_attention, ATTEND, b=batch(**kw)) == mq.MQ_OK
    assert call(mq._kv_read, READ, n=0) == call(mq._kv_read, READ, m=0) == mq.MQ_OK
    assert call(mq._rope, ROPE, rows=0) == mq.MQ_OK


def test_scratch_bytes():
    small, c = mq._kv_scratch(cache(), batch(), 8), cache()
    assert small > 0 and small % 256 == 0
    assert mq._kv_scratch(c, batch(max_new=4), 8) > small
    assert mq._kv_scratch(c, batch(), 7) == 0 and "multiple" in mq.last_error()
    assert mq._kv_scratch(cache(head_dim=24), batch(), 8) == 0
    assert mq._kv_scratch(c, batch(n_seqs=0), 8) > 0


@pytest.mark.parametrize("args,what", [
    ((0.5, 128, 0, None), "theta"), ((math.inf, 128, 0, None), "theta"), ((1e4, 127, 0, None), "rot_dim"),
    ((1e4, 0, 0, None), "rot_dim"), ((1e4, 128, 4, None), "scaling"), ((1e4, 128, 1, None), "params"),
    ((1e4, 128, 1, (0.0,)), "positive"), ((1e4, 128, 2, (8.0, 4.0, 4.0, 8192.0)), "band"),
    ((1e4, 128, 3, (16.0, 32.0, math.nan, 4096.0)), "finite")])
def test_rope_table_refuses(args, what):
    theta, rot, scaling, params = args
    turns, factor = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    p = (ctypes.c_double * 4)(*(params or ())) if params else None
    assert mq._rope_table(theta, rot, scaling, p, ctypes.cast(turns, ctypes.c_void_p), ctypes.byref(factor)) == BAD
    assert what in mq.last_error()


@pytest.mark.parametrize("scaling,params", [("plain", ()), ("linear", (4.0,)), ("linear", (0.25,)), ("bands", (8.0, 1.0, 4.0, 8192.0)),
                                            ("yarn", (16.0, 32.0, 1.0, 4096.0)), ("yarn", (0.5, 32.0, 1.0, 4096.0))])
@pytest.mark.parametrize("theta,rot", [(10000.0, 128), (500000.0, 64), (1e6, 256), (10000.0, 2)])
def test_rope_table_values(scaling, params, theta, rot):
    t = mq.RopeTable(theta, rot, scaling=scaling, params=params)
    w, f = orope.frequencies(theta, rot, scaling, params)
    got = t.turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    want = np.mod(w, 2 * math.pi)
    # the oracle's powers are within a few 2^-53 of theirs, relatively
    assert np.all(np.abs(got - want) <= 64 * 2.0 ** -53 * (w + 2.0 ** -10))
    assert abs(t.factor - f) <= 2.0 ** -23 * f


def test_the_python_descriptors_refuse_other_layouts():
    codes, scales = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2)
    mq.KVCache(codes, codes, scales, scales)
    for bad in ((codes[:, :1], codes, scales, scales), (codes, codes.transpose(0, 1), scales, scales),
                (codes, codes.float(), scales, scales), (codes, codes, scales.double(), scales), (codes, codes, scales, scales[:2])):
        with pytest.raises(ValueError):
            mq.KVCache(*bad)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    mq.KVBatch(i(3), i(2), i(2, 4), 2, 1, 8)
    for bad in ((i(2), i(2), i(2, 4)), (i(3).long(), i(2), i(2, 4)), (i(3), i(2), i(3, 4)), (i(3), i(2), i(2, 8)[:, ::2]),
                (i(3), i(2).float(), i(2, 4))):
        with pytest.raises(ValueError):
            mq.KVBatch(*bad, 2, 1, 8)
    with pytest.raises(ValueError):
        mq.RopeTable(1e4, 64, scaling="yarn", params=(2.0,))


def chain_layer():
    layer = mq.ChainLayer()
    layer.r = 4
    for i in range(5):
        layer.packed[i] = layer.alpha[i] = layer.zero[i] = F
    return layer


CHAIN = dict(layers=(mq.ChainLayer * 1)(chain_layer()), caches=cache(), n=1, b=batch(), rope=rope(), cap=0.0, window=0, D=512, Dkv=256,
             F=1024, h=F, scr=F, size=1 << 40, flags=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(layers=None), BAD), (dict(caches=None), BAD), (dict(b=None), BAD), (dict(n=0), BAD), (dict(h=None), BAD), (dict(h=F + 2), BAD),
    (dict(scr=F + 128), BAD), (dict(size=64), BAD), (dict(flags=2), BAD), (dict(D=500), BAD), (dict(Dkv=128), BAD),
    (dict(Dkv=200), BAD), (dict(b=batch(n_rows=0)), BAD), (dict(b=batch(n_rows=33)), BAD), (dict(b=batch(n_seqs=0)), BAD),
    (dict(b=batch(max_new=0)), BAD), (dict(b=batch(max_len=257)), BAD), (dict(caches=cache(head_dim=24)), BAD),
    (dict(caches=cache(n_kv_heads=1)), BAD), (dict(caches=cache(k=None)), BAD), (dict(rope=rope(rot_dim=20)), NOT_SERVED),
    (dict(cap=-1.0), BAD), (dict(window=-1), BAD)])
def test_chain_decode_refuses(kw, want):
    assert call(mq._chain_decode, CHAIN, **kw) == want, kw
    assert "mq_chain_decode" in mq.last_error()


def test_chain_decode_scratch_bytes():
    small = mq._chain_decode_bytes(cache(), batch(), 512, 256, 1024)
    assert small > mq.chain_scratch_bytes(2, 512, 256, 1024) and small % 256 == 0
    assert mq._chain_decode_bytes(cache(), batch(n_rows=33), 512, 256, 1024) == 0
    assert mq._chain_decode_bytes(cache(), batch(), 500, 256, 1024) == 0
    assert mq._chain_decode_bytes(None, batch(), 512, 256, 1024) == 0
    plan = mq.ChainPlan([], 1, 512, 256, 1024, 128)
    with pytest.raises(ValueError):
        plan.decode_scratch_bytes(None)
    with pytest.raises(ValueError):
        mq.ChainPlan([], 1, 512, 256, 1024, 128, caches=[None])


def test_a_rope_table_on_the_host_is_refused_by_every_call():
    # without a device the table is for inspection: no kernel gets a host address
    table, t = mq.RopeTable(10000.0, 128), torch.zeros(16)
    assert not table.turns.is_cuda
    codes, scales = torch.zeros(4, 2, 16, 128, dtype=torch.uint8), torch.zeros(4, 2)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    c, b = mq.KVCache(codes, codes, scales, scales), mq.KVBatch(i(3), i(2), i(2, 4), 2, 1, 8)
    plan = mq.ChainPlan([], 1, 512, 256, 1024, 128, caches=[])
    for fn in (lambda: mq.rope(t, mq.MQ_F32, 1, 1, 16, 16, i(1), table, t, mq.MQ_F32, 16),
               lambda: mq.kv_append(c, b, t, t, mq.MQ_F32, 256, 256, rope=table),
               lambda: plan.decode(b, t, t, rope=table)):
        with pytest.raises(ValueError, match="host"):
            fn()


def test_the_python_descriptors_refuse_other_types_of_the_same_size():
    codes, scales = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2)
    signed, ints = codes.to(torch.int8), torch.zeros(4, 2, dtype=torch.int32)
    for bad in ((signed, codes, scales, scales), (codes, signed, scales, scales), (codes, codes.bool(), scales, scales),
                (codes, codes, ints, scales), (codes, codes, scales, ints)):
        with pytest.raises(ValueError):
            mq.KVCache(*bad)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for bad in ((i(3).to(torch.uint32), i(2), i(2, 4)), (i(3), i(2).to(torch.uint32), i(2, 4)), (i(3), i(2), i(2, 4).view(torch.uint32))):
        with pytest.raises(ValueError):
            mq.KVBatch(*bad, 2, 1, 8)


def test_calls_without_rows_take_empty_tensors():
    # an empty tensor's address is null; sizes and types are looked at all the same
    for kw in (dict(n_seqs=0, row_start=None, kv_len=None, page_table=None, n_rows=0), dict(n_rows=0)):
        b = batch(**kw)
        assert call(mq._kv_append, APPEND, b=b, k=None, v=None, q=None, qo=None) == mq.MQ_OK
        assert call(mq._kv_attention, ATTEND, b=b, q=None, out=None) == mq.MQ_OK
        assert call(mq._kv_append, APPEND, b=b, k=None, v=None, q=None, qo=None, ks=255) == BAD
        assert call(mq._kv_attention, ATTEND, b=b, q=None, out=None, os=1000) == BAD
    assert call(mq._rope, ROPE, rows=0, x=None, y=None, pos=None) == mq.MQ_OK
    assert call(mq._rope, ROPE, rows=0, x=None, y=None, pos=None, xs=255) == BAD
    # sequences that hold nothing need no pages
    idle = batch(max_pages=0, max_len=0, page_table=None, n_rows=0)
    assert call(mq._kv_append, APPEND, b=idle) == mq.MQ_OK
    assert call(mq._kv_attention, ATTEND, b=batch(max_pages=0, max_len=0, page_table=None), scr=None) == BAD
    assert "scratch" in mq.last_error()


def test_a_chain_that_finds_no_host_memory_reports_it():
    # the launch arguments of so many layers take some 20 MB; the process may have 4 MB more
    script = f"""
import ctypes, os, resource, sys
sys.path[:0] = {sys.path[:4]!r}
import nested_bit_weight_int8_b200 as mq
from test_kv_refusals import CHAIN, cache, chain_layer
n = 1 << 16
layers, caches = (mq.ChainLayer * n)(*[chain_layer()] * n), (mq.KVCacheDesc * n)(*[cache()] * n)
args = list({{**CHAIN, "layers": layers, "caches": caches, "n": n}}.values())
now = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (now + (4 << 20), resource.RLIM_INFINITY))
status = mq._chain_decode(*args)
os.write(1, b"%d " % status + mq._last_error())
os._exit(0)
"""
    got = subprocess.run([sys.executable, "-c", script], capture_output=True, timeout=300)
    assert got.returncode == 0, got.stderr[-500:]
    assert got.stdout.decode() == f"{mq.MQ_ERR_CUDA} no host memory"
