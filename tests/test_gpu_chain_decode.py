"""The chained stack over its layers' caches (mq_chain_decode): rotary positions,
the quantising write and the attention run together as a decode loop does, each
step of the last layer checked on the GPU's own inputs (as test_gpu_chain does),
the attention against the float64 softmax over what the cache then holds."""
import numpy as np
import pytest
import torch

import nested_bit_weight_int8_b200 as mq
import oracle.chain as och
import synth
from gpu_util import DEV, check_linear
from kv_util import Batch
from oracle import kv_cache as okv
from oracle import rope as orope
from test_gpu_chain import _read_views, build_chain

pytestmark = pytest.mark.gpu

D, DKV, F, HD, PAGE = 512, 128, 1024, 64, 16
HQ, HKV = D // HD, DKV // HD


def caches_of(layers, seqs, seed):
    """A cache per layer with the held tokens of seqs; the page tables are the same."""
    out = [Batch(seqs, HKV, HD, PAGE, seed=seed) for _ in range(layers)]
    for b, l in zip(out, range(layers)):
        b.k.random_(1, 256) if l else None
    return out


def check_attention(b, seqs, starts, v, q, softcap, window):
    a = v["a"].reshape(-1, HQ, HD)
    for s, (n, c) in enumerate(seqs):
        r0, places = starts[s], np.arange(c - n, c)
        for h in range(HKV):
            (kc, ks), (vc, vs) = ((b.tokens(w, s, h, c, *b.host(w))) for w in range(2))
            k, val = okv.values(kc, ks, PAGE), okv.values(vc, vs, PAGE)
            of_token = np.repeat(vs.astype(np.float64), PAGE)[:c]
            for x in range(h * HQ // HKV, (h + 1) * HQ // HKV):
                rows = q[r0:r0 + n, x]
                o, _, mass, gross = okv.attend(rows, k, val, of_token, places, HD ** -0.5, softcap, window)
                delta = okv.score_error(rows, ks.max(initial=0.0), HD ** -0.5, softcap)
                tol = okv.out_error(o, mass, gross, vs.max(initial=0.0), delta, c)
                assert np.all(np.abs(a[r0:r0 + n, x] - o) <= tol), (s, x)


def check_step(v, ref, h_out, b, seqs, starts, q, w, softcap, window, label):
    real = int(starts[-1])
    check_linear(v["qkv"], v["xn"], ref["qkv"], f"{label}: qkv")
    places = np.concatenate([np.arange(c - n, c) for n, c in seqs])
    x = v["qkv"][:real, :D].reshape(real, HQ, HD)
    want, tol = orope.rotate(x, places, w, 1.0, "half"), orope.f32_error(x, HD, 1.0, "half")
    assert np.all(np.abs(q[:real] - och.to_bf16(want)) <= och.bf16_flip(want, tol))
    check_attention(b, seqs, starts, v, q, softcap, window)
    assert np.all(v["a"][real:] == 0)
    check_linear(v["o"], v["a"], ref["o"], f"{label}: o")
    pre = och.silu(v["g"]) * v["u"]
    assert np.all(np.abs(v["act"] - och.to_bf16(pre)) <= och.bf16_flip(pre, och.swiglu_f32_error(v["g"], v["u"])))
    check_linear(v["down"], v["act"], ref["down"], f"{label}: down")
    assert np.array_equal(h_out, (v["h1"].astype(np.float32) + v["down"].astype(np.float32)).astype(np.float64))


def queries_of(scratch, M):
    at = mq.chain_scratch_bytes(M, D, DKV, F)
    raw = scratch[at:at + 2 * M * D].cpu().numpy().view(np.uint16).reshape(M, HQ, HD)
    return synth.f32_from_bf16_bits(raw).astype(np.float64)


@pytest.mark.parametrize("new,softcap,window", [(1, 0.0, 0), (3, 30.0, 9)])
def test_a_decode_loop_step_by_step(new, softcap, window):
    layers, steps = 3, 5
    ref, dev, _keep = build_chain(layers, [8, 4, 2], D, DKV, F, 500)
    lens = [0, 17, 30, 0]  # tokens held before; the last sequence stays idle (a padded row)
    room = [(new, c + new * steps) for c in lens[:3]] + [(1, 0)]
    own = [Batch(room, HKV, HD, PAGE, seed=40 + l, tail_rows=2, fill="held") for l in range(layers)]
    first = own[0]
    for b in own[1:]:  # one page table for all layers, as a serving engine keeps it
        b.table, b.pages = first.table, first.pages
    M = 3 * new + 1 + 2
    plan = mq.ChainPlan(dev, M, D, DKV, F, HD, caches=[b.cache for b in own])
    rope, (w, _) = mq.RopeTable(10000.0, HD, device=DEV), orope.frequencies(10000.0, HD)
    kv_len = torch.zeros(4, dtype=torch.int32, device=DEV)
    batch = mq.KVBatch(first.row_start, kv_len, first.pages, M, new, max(c for _, c in room))
    scratch = torch.full((plan.decode_scratch_bytes(batch),), 0xFF, dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(3)
    for step in range(steps):
        seqs = [(new, c + new * (step + 1)) for c in lens[:3]] + [(1, 0)]
        kv_len.copy_(torch.tensor([c for _, c in seqs], dtype=torch.int32))
        h = torch.from_numpy(rng.standard_normal((M, D)).astype(np.float32)).to(DEV)
        plan.decode(batch, h, scratch, rope=rope, softcap=softcap, window=window)
        mq.device_status()
        starts = np.cumsum([0] + [n for n, _ in seqs])
        check_step(_read_views(scratch, M, D, DKV, F), ref[-1], h.cpu().numpy().astype(np.float64), own[-1], seqs, starts,
                   queries_of(scratch, M), w, softcap, window, f"step {step}")


def test_a_captured_step_reads_the_lengths_of_its_replay():
    layers, M = 2, 3
    _, dev, _keep = build_chain(layers, [4, 3], D, DKV, F, 600)
    room = [(1, 20), (1, 33), (1, 5)]

    def engine():
        own = [Batch(room, HKV, HD, PAGE, seed=50 + l) for l in range(layers)]
        for b in own[1:]:
            b.table, b.pages = own[0].table, own[0].pages
        kv_len = torch.zeros(3, dtype=torch.int32, device=DEV)
        batch = mq.KVBatch(own[0].row_start, kv_len, own[0].pages, M, 1, 33)
        plan = mq.ChainPlan(dev, M, D, DKV, F, HD, caches=[b.cache for b in own])
        scratch = torch.empty(plan.decode_scratch_bytes(batch), dtype=torch.uint8, device=DEV)
        return own, kv_len, batch, plan, scratch

    rope = mq.RopeTable(10000.0, HD, device=DEV)
    rng = np.random.default_rng(4)
    xs = [torch.from_numpy(rng.standard_normal((M, D)).astype(np.float32)).to(DEV) for _ in range(5)]
    results = []
    for graph in (False, True):
        own, kv_len, batch, plan, scratch = engine()
        s, h, outs = torch.cuda.Stream(), torch.empty(M, D, device=DEV), []
        for step, x in enumerate(xs):
            with torch.cuda.stream(s):
                kv_len.copy_(torch.tensor([15 + step, 28 + step, step], dtype=torch.int32))
                h.copy_(x)
                plan.decode(batch, h, scratch, rope=rope, graph=graph, stream=s)
            s.synchronize()
            mq.device_status(s)
            outs.append(h.clone())
        results.append((outs, [b.k.clone() for b in own], [b.ks.clone() for b in own], own))
    (a, ka, sa, _), (b, kb, sb, _) = results
    # the linears' sums differ in their order from call to call: codes may flip at a border
    for x, y in zip(a, b):
        assert torch.allclose(x, y, rtol=0, atol=2e-2 * float(x.square().mean().sqrt()))
    for x, y in zip(ka, kb):
        assert float((x.int() - y.int()).abs().float().mean()) < 0.05
    mq.release_workspace()
