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
