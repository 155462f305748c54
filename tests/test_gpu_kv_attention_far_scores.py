"""Attention over the 8-bit cache where scores are far from zero or far apart:
rows of very large scores, and keys that far outweigh those before them."""
import numpy as np
import pytest
import torch

import nested_bit_weight_int8_b200 as mq
from gpu_util import DEV
from kv_util import Batch
from oracle import kv_cache as okv
from test_gpu_kv_attention import attend

pytestmark = pytest.mark.gpu


def equal_keys(seqs, heads, dim, page, seed):
    """A batch whose keys are all ones times 2^-6, and values of pages of unlike scales."""
    b = Batch(seqs, heads, dim, page, seed=seed, fill="all")
    rng = np.random.default_rng(seed)
    b.codes[0][:] = 129
    b.scales[0][:] = 2.0 ** -6
    b.scales[1][:] = 10.0 ** rng.uniform(-4, 0, b.scales[1].shape)
    for t, c in ((b.k, b.codes[0]), (b.ks, b.scales[0]), (b.vs, b.scales[1])):
        t.copy_(torch.from_numpy(c))
    return b


def queries_of_size(b, hq, seed, power):
    """Each row and head one number, (1 + j / 128) 2^e of either sign, in all its values: sums of
    it are exact. scale q . k of `equal_keys` is then of the order of 2^power at scale 1."""
    rng = np.random.default_rng(seed)
    e = power + 6 - int(np.log2(b.dim))
    x = (1 + rng.integers(0, 128, (b.rows, hq)) / 128) * rng.choice([-1.0, 1.0], (b.rows, hq)) * 2.0 ** e
    return torch.from_numpy(np.repeat(x, b.dim, 1)).to(torch.bfloat16).to(DEV)


def check_equal_scores(b, hq, q, out, log, window, softcap):
    """A row's scores are the same number for every key, so its weights are equal whatever its size:
    scores add no error but the roundings of a weight's exponent below 2^12 (2^-24 of the score each,
    base 2, that of the score and that of the maximum with the scale's logarithm; above 2^12 the
    maximum is taken off exactly); for the cap and the products before it 8 u of the lse."""
    q64 = q.double().cpu().numpy().reshape(b.rows, hq, b.dim)
    got, lse = out.float().cpu().numpy(), log.double().cpu().numpy()
    u = 2.0 ** -24
    for s, (n, c) in enumerate(b.seqs):
        r0 = b.starts[s]
        for a in range(hq):
            h = a // (hq // b.heads)
            (kc, ks), (vc, vs) = (b.tokens(w, s, h, c) for w in range(2))
            k, v = okv.values(kc, ks, b.page), okv.values(vc, vs, b.page)
            x = q64[r0:r0 + n, a]
            o, l, mass, gross = okv.attend(x, k, v, np.repeat(vs.astype(np.float64), b.page)[:c], b.places(s), 1.0, softcap, window)
            size = np.where(np.isfinite(l), np.abs(l), 0.0)
            delta = 2 * u * np.minimum(size, 4096.0)
            err = np.abs(got[r0:r0 + n, a * b.dim:(a + 1) * b.dim] - o)
            tol = okv.out_error(o, mass, gross, vs.max(initial=0.0), delta, c)
            assert np.all(err <= tol), (s, a, np.nanmax(err / tol))
            f = np.isfinite(l)
            assert np.all(np.abs(lse[r0:r0 + n, a][f] - l[f]) <= okv.lse_error(l, delta + 8 * u * size, c)[f]), (s, a)
            assert np.all(lse[r0:r0 + n, a][~f] == -np.inf)


POWERS = [6, 11, 12, 13, 16, 20, 24, 25, 26, 27, 28, 30, 60, 100]


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("dim,group,window,softcap", [(64, 2, 0, 0.0), (128, 2, 0, 0.0), (128, 1, 50, 0.0), (256, 2, 0, 0.0),
                                                      (128, 2, 0, 2.0 ** 60)])
def test_prompts_of_very_large_scores(power, dim, group, window, softcap):
    # rows over cached tokens (whole tiles that nothing masks) and rows that see few tokens
    b = equal_keys([(200, 460), (140, 140), (130, 700)], 1, dim, 32, seed=power)
    q = queries_of_size(b, group, power, power)
    out, log = attend(b, group, q, softcap=softcap, window=window, scale=1.0)
    mq.device_status()
    check_equal_scores(b, group, q, out, log, window, softcap)


def one_far_key(dim, n, held, seed, places, low):
    """Sequences of n rows upon `held` tokens; sequence i's key at places[i] is 127 in every value, all
    others are `low`."""
    b = Batch([(n, held + n)] * len(places), 1, dim, 32, seed=seed, fill="all")
    b.codes[0][:] = 128 + low
    for i, p in enumerate(places):
        b.codes[0][b.table[i, p // 32], 0, p % 32] = 255
    b.scales[0][:] = 1.0
    for t, c in ((b.k, b.codes[0]), (b.ks, b.scales[0])):
        t.copy_(torch.from_numpy(c))
    return b


def check_far_key(b, q, out, log, scale, softcap, small=False):
    """The others' scores are one number, and what stands next to the far key weighs 2^-90 at most: scores
    add no error to the outputs (8 u of the far one where the gap is small), 8 u of themselves and of the cap
    to the lse. All sequences at once."""
    (n, c), seqs, u = b.seqs[0], len(b.seqs), 2.0 ** -24
    pages = b.pages[:, :-(-c // b.page)].long()
    k, v = (((t[pages, 0].reshape(seqs, -1, b.dim)[:, :c].double() - 128) * s) for t, s in (
        (b.k, b.ks[pages, 0].double().repeat_interleave(b.page, 1)[:, :c, None]),
        (b.v, b.vs[pages, 0].double().repeat_interleave(b.page, 1)[:, :c, None])))
    score = q.double().view(seqs, n, b.dim) @ k.transpose(1, 2) * scale
    if softcap:
        score = softcap * torch.tanh(score / softcap)
    score = score.masked_fill(torch.ones(n, c, dtype=torch.bool, device=DEV).triu(c - n + 1), -torch.inf)
    p, l = score.softmax(-1), score.logsumexp(-1).flatten().cpu().numpy()
    o, mass = ((p @ x).view(-1, b.dim).cpu().numpy() for x in (v, v.abs()))
    gross = (p @ b.vs[pages, 0].double().repeat_interleave(b.page, 1)[:, :c, None]).flatten().cpu().numpy() * 383
    err = np.abs(out.float().cpu().numpy() - o)
    tol = okv.out_error(o, mass, gross, float(b.vs.max()), 8 * u * np.abs(l) * small, c)
    assert np.all(err <= tol), [(r // n, r % n) for r in np.unique(np.argwhere(~(err <= tol))[:, 0])[:8]]
    assert np.all(np.abs(log.double().cpu().numpy()[:, 0] - l) <= okv.lse_error(l, 8 * u * (np.abs(l) + softcap), c))


# gaps in base 2
@pytest.mark.parametrize("gap,softcap", [(g, 0.0) for g in (90, 118, 120, 125, 130, 140, 200, 254, 400, 600)] +
                         [(g, 200.0) for g in (90, 120, 125, 130, 200)] + [(140, 50.0)])
@pytest.mark.parametrize("dim,n", [(64, 100), (64, 150), (128, 100), (128, 150), (256, 100)])
def test_prompts_with_one_far_outweighing_key(dim, n, gap, softcap):
    held = 260
    # each place of 64 in turn: behind the first 32 tokens, in a later tile, among the masked
    for seed, start in enumerate((32, 160, held)):
        b = one_far_key(dim, n, held, seed, [start + i for i in range(64)], -127 if softcap == 50.0 else 0)
        size = gap * np.log(2) if softcap != 50.0 else gap * np.log(2) / 2  # of the far key's score; -size of the others then
        scale = (softcap * np.arctanh(size / softcap) if softcap else size) / (127 * dim)
        for rows in ("all", "one"):
            q = torch.zeros(b.rows, dim, device=DEV, dtype=torch.bfloat16)
            if rows == "all":
                q[:] = 1
            else:  # the last row of each sequence, alone in its warp: no other's sum tells of the step
                q[torch.from_numpy(b.starts[1:] - 1).to(DEV)] = 1
            out, log = attend(b, 1, q, softcap=softcap, scale=float(np.float32(scale)))
            mq.device_status()
            check_far_key(b, q, out, log, float(np.float32(scale)), softcap)


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("dim,group,window,softcap", [(64, 2, 0, 0.0), (128, 4, 0, 0.0), (128, 1, 50, 0.0), (256, 2, 0, 0.0),
                                                      (128, 2, 0, 2.0 ** 60)])
def test_few_rows_of_very_large_scores(power, dim, group, window, softcap):
    b = equal_keys([(1, 700), (3, 3), (1, 1), (5, 460), (1, 0), (2, 33)], 1, dim, 32, seed=power)
    q = queries_of_size(b, group, power, power)
    out, log = attend(b, group, q, softcap=softcap, window=window, scale=1.0)
    mq.device_status()
    check_equal_scores(b, group, q, out, log, window, softcap)


@pytest.mark.parametrize("gap,softcap", [(5, 0.0), (7, 0.0), (40, 0.0), (125, 0.0), (600, 0.0), (125, 200.0), (140, 50.0)])
@pytest.mark.parametrize("dim,n", [(64, 4), (128, 2), (256, 5)])
def test_few_rows_with_one_far_outweighing_key(dim, n, gap, softcap):
    held = 260
    for seed, start in enumerate((0, 160, held - 60)):
        b = one_far_key(dim, n, held, seed, [start + i for i in range(64)], -127 if softcap == 50.0 else 0)
        size = gap * np.log(2) / (2 if softcap == 50.0 else 1)
        scale = float(np.float32((softcap * np.arctanh(size / softcap) if softcap else size) / (127 * dim)))
        q = torch.ones(b.rows, dim, device=DEV, dtype=torch.bfloat16)
        out, log = attend(b, 1, q, softcap=softcap, scale=scale)
        mq.device_status()
        check_far_key(b, q, out, log, scale, softcap, small=gap < 90)


@pytest.mark.parametrize("seqs", [[(3, 200), (1, 17)], [(90, 500), (200, 300)]])
@pytest.mark.parametrize("dim,window", [(64, 0), (128, 50), (256, 0)])
def test_a_query_that_is_no_number_gives_no_number(seqs, dim, window):
    # outputs and lse alike, in its row and head alone; -infinity is for rows that see nothing
    b = Batch(seqs, 1, dim, 32, seed=29, fill="all")
    q = torch.randn(b.rows, 2 * dim, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(torch.bfloat16)
    bad = torch.zeros(b.rows, 2, dtype=torch.bool, device=DEV)
    for row in (0, int(b.starts[1]) - 1, int(b.starts[2]) - 1):
        q[row, dim + row % dim] = float("nan")
        bad[row, 1] = True
    out, log = attend(b, 2, q, window=window)
    mq.device_status()
    assert torch.equal(torch.isnan(log), bad)
    assert torch.equal(torch.isnan(out).view(b.rows, 2, dim), bad[:, :, None].expand(-1, -1, dim))


@pytest.mark.parametrize("further", [10, 12, 13, 16, 20])
@pytest.mark.parametrize("dim,n", [(64, 100), (64, 150), (128, 100), (128, 150), (256, 100)])
def test_prompts_keep_a_weight_when_a_larger_one_follows_in_its_tile(dim, n, further):
    # scores (base 2) 0, then 13 (a page whose V scale is 2^-7 of the largest, so that it stays within the
    # running maximum's slack), then `further` more in the same tile: the second's weight, 2^-further, counts,
    # as the third's values are small or zero
    held, seqs = 260, 8
    for second, third in ((34, 100), (262, 300), (130, 215)):
        b = Batch([(n, held + n)] * seqs, 1, dim, 16, seed=7, fill="all")
        rng = np.random.default_rng(further)
        b.codes[0][:] = b.codes[1][:] = 128
        b.scales[0][:] = b.scales[1][:] = 1.0
        for pages in b.table:
            at, far = (pages[second // 16], 0, second % 16), (pages[third // 16], 0, third % 16)
            b.codes[0][at], b.codes[0][far] = 128 + 13, 128 + 13 + further
            b.codes[1][at], b.codes[1][far] = 255, 128 + rng.integers(-9, 10, dim) * rng.integers(0, 2, dim)
            b.scales[1][at[0]], b.scales[1][far[0]] = 2.0 ** -7, 2.0 ** -14
        for t, c in ((b.k, b.codes[0]), (b.v, b.codes[1]), (b.ks, b.scales[0]), (b.vs, b.scales[1])):
            t.copy_(torch.from_numpy(c))
        q, scale = torch.ones(b.rows, dim, device=DEV, dtype=torch.bfloat16), float(np.float32(np.log(2) / dim))
        out, log = attend(b, 1, q, scale=scale)
        mq.device_status()
        check_far_key(b, q, out, log, scale, 0.0, small=True)
