"""Measured cases of the serving operators around the 8-bit key/value cache: rotary
positions, the cache's quantising write and its read-back, and attention over it.

`run` computes a pass in plain torch (`own` false) or through the framework's entry points
(`own` true). The cache holds one unsigned byte per value, offset 128, in pages of `page`
tokens; each page has one fp32 scale per key/value head for K and one for V:
value = scale * (byte - 128). A sequence's tokens are found through its row of page numbers.
"""
import math
import random

import torch

own = False

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # four decode rows' query and key heads of the 7B-shaped stack: pure latency
        dict(name="rope_decode", op="rope", rows=4, heads=40, dim=128, rot=128, layout="half", scaling="plain",
             theta=10000.0, furthest=4096, dtype="bf16"),
        # a long prompt's rows at far positions, the long-context ramp, wide heads, as the products leave them
        dict(name="rope_far", op="rope", rows=8192, heads=24, dim=256, rot=256, layout="half", scaling="yarn",
             theta=1000000.0, furthest=1000000, dtype="f32"),
        # part of the head, interleaved pairs, wavelength bands, an odd number of rows
        dict(name="rope_part", op="rope", rows=1023, heads=12, dim=96, rot=32, layout="interleaved", scaling="bands",
             theta=500000.0, furthest=131072, dtype="bf16"),
        # a decode batch's step: one token for each sequence written, the open pages read back
        dict(name="cache_decode", op="cache", seqs=32, new=1, ctx=4096, ragged=True, mix=False, idle=2, heads=32, kv_heads=8,
             dim=128, page=64, rot=128, layout="half", scaling="plain", theta=10000.0, dtype="f32", read="open"),
        # prompts of several sequences written behind what they hold already, then read whole
        dict(name="cache_prompt", op="cache", seqs=4, new=2000, ctx=2500, ragged=True, mix=False, idle=0, heads=16,
             kv_heads=8, dim=256, page=32, rot=256, layout="half", scaling="plain", theta=10000.0, dtype="f32", read="all"),
        # one user's next token: few keys, few heads
        dict(name="attend_one", op="attend", seqs=1, new=1, ctx=777, ragged=False, mix=False, idle=0, heads=32, kv_heads=8,
             dim=128, page=64, window=0, softcap=0.0),
        # a serving batch of ragged lengths, three of its rows padding
        dict(name="attend_batch", op="attend", seqs=64, new=1, ctx=8192, ragged=True, mix=False, idle=3, heads=32,
             kv_heads=8, dim=128, page=64, window=0, softcap=0.0),
        # one sequence with a very long cache: the long axis has to be split
        dict(name="attend_long", op="attend", seqs=1, new=1, ctx=131072, ragged=False, mix=False, idle=0, heads=32,
             kv_heads=8, dim=128, page=128, window=0, softcap=0.0),
        # five drafted tokens for each sequence, wide heads, a sliding window and capped scores
        dict(name="attend_drafts", op="attend", seqs=16, new=5, ctx=6000, ragged=True, mix=False, idle=0, heads=16,
             kv_heads=8, dim=256, page=16, window=4096, softcap=50.0),
        # prompts in chunks of 2048 tokens upon as many cached ones: bound by arithmetic
        dict(name="attend_prompt", op="attend", seqs=2, new=2048, ctx=4096, ragged=False, mix=False, idle=0, heads=32,
             kv_heads=8, dim=128, page=64, window=0, softcap=0.0),
        # one prompt's chunk next to decode rows of other sequences
        dict(name="attend_mixed", op="attend", seqs=9, new=500, ctx=5000, ragged=True, mix=True, idle=0, heads=16,
             kv_heads=8, dim=128, page=64, window=0, softcap=0.0),
        # sequences on their way out of the cache: each writes its last token and is read back whole
        dict(name="cache_out", op="cache", seqs=7, new=1, ctx=16000, ragged=True, mix=False, idle=0, heads=32, kv_heads=8,
             dim=128, page=128, rot=64, layout="interleaved", scaling="linear", theta=10000.0, dtype="bf16", read="all"),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))

    op = rng.choice(["rope", "cache", "attend", "attend"])
    dim = rng.choice([64, 96, 128, 128, 256])
    rotary = dict(rot=rng.choice([dim, dim // 2]), layout=rng.choice(["half", "interleaved"]),
                  scaling=rng.choice(["plain", "linear", "bands", "yarn"]), theta=rng.choice([10000.0, 500000.0]),
                  dtype=rng.choice(["f32", "bf16"]))
    if op == "rope":
        heads = rng.randint(1, 40)
        return dict(op=op, rows=spread(1, 8192 * 24 * 256 // (heads * dim)), heads=heads, dim=dim,
                    furthest=spread(128, 1000000), **rotary)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 7, 8])
    shape = dict(heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]))
    if op == "cache":
        seqs = spread(1, 48)
        new = rng.choice([1, spread(1, max(1, 8000 // seqs))])
        ctx = new + spread(1, max(1, 16000 // seqs))
        return dict(op=op, seqs=seqs, new=new, ctx=ctx, ragged=True, mix=False, idle=rng.choice([0, 1]) if seqs > 1 else 0,
                    read=rng.choice(["open", "all"]), **shape, **rotary)
    masks = dict(window=rng.choice([0, 0, spread(1, 4096)]), softcap=rng.choice([0.0, 0.0, 30.0]))
    seqs, mix = spread(1, 64), False
    if rng.random() < 0.6:
        new = rng.choice([1, 1, rng.randint(2, 8)])
        ctx = new + spread(1, min(65536, 400000 // seqs))
    else:
        seqs, new = min(seqs, 8), spread(9, 2048)
        ctx = new + spread(1, 2048)
        while 4 * seqs * new * ctx * heads * dim > 2e11:
            seqs, new, ctx = (seqs - 1, new, ctx) if seqs > 1 else (1, new // 2, ctx - new // 2)
        mix = seqs > 1 and rng.random() < 0.5
    return dict(op=op, seqs=seqs, new=new, ctx=ctx, ragged=rng.random() < 0.8, mix=mix,
                idle=rng.choice([0, 1]) if seqs > 1 else 0, **shape, **masks)


def _lengths(case):
    """(new rows, cached tokens with the new ones) of each sequence: the same for every seed."""
    rng = random.Random(case["seqs"] * 1000003 + case["new"] * 1009 + case["ctx"])
    n, live = case["seqs"], case["seqs"] - case["idle"]
    if case["ragged"]:
        new = [case["new"]] + [1 if case["mix"] else rng.randint(1, case["new"]) for _ in range(live - 1)]
        kv = [case["ctx"]] + [max(a, rng.randint(max(1, case["ctx"] // 4), case["ctx"])) for a in new[1:]]
    else:
        new, kv = [case["new"]] * live, [case["ctx"]] * live
    return new + [1] * (n - live), kv + [0] * (n - live)  # an idle sequence: a padded row with no tokens


def _visible(case):
    """Pairs of query row and visible key, and keys that some row of its sequence sees."""
    new, kv = _lengths(case)
    window = case["window"] or case["ctx"] + 1
    ends = [range(c - a + 1, c + 1) for a, c in zip(new, kv) if c]
    pairs = sum(min(e, window) for r in ends for e in r)
    keys = sum(r[-1] - max(0, r[0] - window) for r in ends)
    return pairs, keys


def _read_ranges(case):
    """(first token, end) that the read-back covers: from the start of the page the new rows begin in, or all."""
    new, kv = _lengths(case)
    return [(((c - a) // case["page"] * case["page"] if case["read"] == "open" else 0), c) if c else (0, 0)
            for a, c in zip(new, kv)]


def work(case):
    item = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "rope":
        n = case["rows"] * case["heads"] * case["dim"]
        return {"bytes": 2 * item * n + 4 * case["rows"], "flops": 3 * case["rows"] * case["heads"] * case["rot"]}
    new, kv = _lengths(case)
    rows, h, g, d = sum(new), case["heads"], case["kv_heads"], case["dim"]
    written = sum(a for a, c in zip(new, kv) if c)
    total = {"bytes": 4 * (2 * len(new) + sum(-(-c // case["page"]) for c in kv)), "flops": 0}
    if case["op"] == "cache":
        tokens = sum(e - f for f, e in _read_ranges(case))
        total["bytes"] += item * rows * (h + 2 * g) * d + 2 * written * g * d + 2 * rows * h * d + tokens * 2 * g * d * 3
        total["flops"] += 3 * rows * (h + g) * case["rot"] + 4 * written * g * d + tokens * 2 * g * d
    else:
        pairs, keys = _visible(case)
        total["bytes"] += keys * 2 * g * d + 4 * rows * h + 4 * rows * h * d
        total["flops"] += 4 * pairs * h * d
    return total


# ------------------------------------------------------------------ inputs
def _scaling(case):
    """The arguments of a position scaling for long contexts."""
    return {"plain": (), "linear": (4.0,), "bands": (8.0, 1.0, 4.0, 8192.0), "yarn": (16.0, 32.0, 1.0, 4096.0)}[case["scaling"]]


def _frequencies(case, dev):
    """Angle per position of each rotated pair in 64 bits, and the factor on the rotated values."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev)
    f = case["theta"] ** (-2.0 * i / case["rot"])
    a = _scaling(case)
    if case["scaling"] == "linear":
        return f / a[0], 1.0
    if case["scaling"] == "bands":  # long wavelengths are stretched, short ones kept, a blend between
        blend = ((a[3] * f / (2 * math.pi) - a[1]) / (a[2] - a[1])).clamp(0, 1)
        return f / a[0] * (1 - blend) + f * blend, 1.0
    if case["scaling"] == "yarn":  # a ramp over the pairs between two numbers of turns
        low, high = (case["rot"] * math.log(a[3] / (b * 2 * math.pi)) / (2 * math.log(case["theta"])) for b in a[1:3])
        low, high = max(math.floor(low), 0), min(math.ceil(high), case["rot"] - 1)
        keep = 1 - ((i - low) / (high - low if high > low else 0.001)).clamp(0, 1)
        return f / a[0] * (1 - keep) + f * keep, 0.1 * math.log(a[0]) + 1.0
    return f, 1.0


def _mq():
    import nested_bit_weight_int8_b200 as mq
    return mq


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed) & 0x7FFFFFFF)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(case=case)
    if "rot" in case:
        s["inv"], s["factor"] = _frequencies(case, dev)
        if own:
            s["table"] = _mq().RopeTable(case["theta"], case["rot"], layout=case["layout"], scaling=case["scaling"],
                                         params=_scaling(case), device=dev)
    if case["op"] == "rope":
        t, h, d = case["rows"], case["heads"], case["dim"]
        s["x"] = normal(t, h, d).to(_DTYPES[case["dtype"]])
        s["positions"] = torch.randint(0, case["furthest"], (t,), generator=gen, device=dev, dtype=torch.int32)
        s["y"] = torch.empty_like(s["x"])
        return s
    new, kv = _lengths(case)
    h, g, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    rows, held = sum(new), [-(-c // page) for c in kv]
    n_pages = sum(held) + 3  # the last page and two others are no sequence's
    order = torch.randperm(n_pages - 1, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(kv), max(held)), -1, dtype=torch.int32, device=dev)
    at = torch.arange(max(held), device=dev)[None, :] < torch.tensor(held, device=dev)[:, None]
    table[at] = order[: sum(held)]

    def cached(outliers):  # what earlier steps left: a few channels larger than the others
        wide = 1 + 3 * (torch.rand(g, 1, d, generator=gen, device=dev) < 0.05) * outliers
        codes = torch.empty(n_pages, g, page, d, dtype=torch.uint8, device=dev)
        scales = torch.empty(n_pages, g, device=dev)
        for lo in range(0, n_pages, 2048):
            x = normal(min(2048, n_pages - lo), g, page, d) * wide
            scales[lo:lo + 2048] = x.abs().amax((2, 3)) / 127
            codes[lo:lo + 2048] = (torch.round(x / scales[lo:lo + 2048, :, None, None]) + 128).to(torch.uint8)
        return codes, scales, wide

    s["k"], s["k_scale"], k_wide = cached(1.0)
    s["v"], s["v_scale"], _ = cached(0.0)
    s["row_start"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=dev)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["table_of_pages"] = table
    s["rows"], s["max_new"], s["max_len"] = rows, max(new), max(kv)
    if own:
        s["cache"] = _mq().KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = _mq().KVBatch(s["row_start"], s["kv_len"], table, n_rows=rows, max_new=max(new), max_len=max(kv))
    if case["op"] == "cache":
        qkv = normal(rows, h + 2 * g, d)
        qkv[:, h:h + g] *= k_wide[:, 0]
        s["qkv"] = qkv.view(rows, -1).to(_DTYPES[case["dtype"]])
        s["q_out"] = torch.empty(rows, h, d, dtype=torch.bfloat16, device=dev)
        ranges = _read_ranges(case)
        ends = [sum(e - f for f, e in ranges[:i]) for i in range(len(ranges) + 1)]
        s["first"] = torch.tensor([f for f, _ in ranges], dtype=torch.int32, device=dev)
        s["out_start"] = torch.tensor(ends, dtype=torch.int32, device=dev)
        s["n_out"], s["max_out"] = ends[-1], max(e - f for f, e in ranges)
        s["k_out"] = torch.empty(s["n_out"], g, d, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    s["q"] = normal(rows, h, d).to(torch.bfloat16)
    s["out"] = torch.empty(rows, h, d, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.empty(rows, h, device=dev)
    if own:
        size = _mq().kv_attention_scratch_bytes(s["cache"], s["batch"], h)
        s["scratch"] = torch.empty(size, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "rope":
        return _rotate(s, s["x"].float(), s["positions"]).to(s["x"].dtype)
    if case["op"] == "cache":
        q = _write(s)
        return [q, *_read(s)]
    return list(_attend(s, s["q"]))


def _run_own(s, case):
    mq = _mq()
    h, g, d = case["heads"], case.get("kv_heads"), case["dim"]
    if case["op"] == "rope":
        kind = mq.MQ_F32 if case["dtype"] == "f32" else mq.MQ_BF16
        mq.rope(s["x"], kind, case["rows"], h, d, h * d, s["positions"], s["table"], s["y"], kind, h * d)
        return s["y"]
    if case["op"] == "cache":
        kind, qkv, pitch = mq.MQ_F32 if case["dtype"] == "f32" else mq.MQ_BF16, s["qkv"], (h + 2 * g) * d
        mq.kv_append(s["cache"], s["batch"], qkv[:, h * d:], qkv[:, (h + g) * d:], kind, pitch, pitch, rope=s["table"],
                     q=qkv, q_stride=pitch, n_q_heads=h, q_out=s["q_out"])
        mq.kv_read(s["cache"], s["batch"], s["first"], s["out_start"], s["n_out"], s["max_out"], s["k_out"], s["v_out"],
                   mq.MQ_BF16, g * d)
        return [s["q_out"], s["k_out"], s["v_out"]]
    mq.kv_attention(s["cache"], s["batch"], s["q"], h * d, h, d ** -0.5, s["out"], h * d, s["scratch"], lse=s["lse"],
                    softcap=case["softcap"], window=case["window"])
    return [s["out"], s["lse"]]


def _rotate(s, x, positions):
    """Rotary positions of x (rows, heads, dim), in 32 bits; the angles in 64."""
    rot, half = s["case"]["rot"], s["case"]["rot"] // 2
    angle = positions.double()[:, None] * s["inv"]
    c, n = (torch.cos(angle) * s["factor"]).float()[:, None], (torch.sin(angle) * s["factor"]).float()[:, None]
    if s["case"]["layout"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        return torch.cat([a * c - b * n, b * c + a * n, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2), x[..., rot:]], -1)


def _row_places(s):
    """Of each row its sequence and its token's place in it, and each sequence's number of rows."""
    row = torch.arange(s["rows"], device=s["kv_len"].device)
    start = s["row_start"].long()
    seq = torch.searchsorted(start[1:], row, right=True)
    new = start[1:] - start[:-1]
    return seq, s["kv_len"].long()[seq] - new[seq] + row - start[seq], new


def _write(s):
    """The rows' keys (rotated) and values quantised into the cache; returns the rotated queries."""
    case = s["case"]
    h, g, page = case["heads"], case["kv_heads"], case["page"]
    x = s["qkv"].float().view(s["rows"], h + 2 * g, case["dim"])
    seq, place, new = _row_places(s)
    turned = _rotate(s, x[:, :h + g], place)
    table, kv = s["table_of_pages"].long(), s["kv_len"].long()
    spare = s["k"].shape[0] - 1  # stands in for the pages that a padded row does not have
    start = (kv - new).clamp(min=0)
    # the pages that new tokens fall in, each sequence's last repeated up to the same number
    most = (s["max_new"] + page - 2) // page + 1
    nth = (start // page)[:, None] + torch.arange(most, device=kv.device)
    nth = torch.minimum(nth, ((kv - 1).clamp(min=0) // page)[:, None])
    pages = torch.where((kv == 0)[:, None], spare, table.gather(1, nth))
    held = (start[:, None] - nth * page).clamp(0, page)  # tokens that the page holds already
    row_page = torch.where(place >= 0, table[seq, place.clamp(min=0) // page], spare)
    slot = place.clamp(min=0) % page
    _quantise(s["k"], s["k_scale"], turned[:, h:], pages, held, row_page, slot, spare)
    _quantise(s["v"], s["v_scale"], x[:, h + g:], pages, held, row_page, slot, spare)
    return turned[:, :h].to(torch.bfloat16)


def _quantise(codes, scales, x, pages, held, row_page, slot, spare):
    """Writes x (rows, heads, dim): a page's scale only grows, and what it holds is rounded to the new one."""
    page, real = codes.shape[2], (pages != spare)[..., None]
    largest = torch.zeros_like(scales).index_reduce_(0, row_page, x.abs().amax(2), "amax")
    old = torch.where((held > 0)[..., None], scales[pages], 0.0)  # a page that is empty has no scale yet
    scale = torch.where(real, torch.maximum(old, largest[pages] / 127), scales[pages])
    kept = codes[pages].float() - 128
    again = torch.round(kept * old[..., None, None] / torch.where(scale > 0, scale, 1.0)[..., None, None])
    grown = (real & (scale > old))[..., None, None]
    inside = (torch.arange(page, device=x.device) < held[..., None])[:, :, None, :, None]
    codes[pages] = (torch.where(grown & inside, again, kept) + 128).to(torch.uint8)
    scales[pages] = scale
    of_row = scales[row_page]
    fresh = torch.round(x / torch.where(of_row > 0, of_row, 1.0)[..., None]).clamp(-127, 127) + 128
    codes[row_page, :, slot] = torch.where((row_page != spare)[:, None, None], fresh.to(torch.uint8), codes[row_page, :, slot])


def _read(s):
    case, out = s["case"], torch.arange(s["n_out"], device=s["k"].device)
    start = s["out_start"].long()
    seq = torch.searchsorted(start[1:], out, right=True)
    token = s["first"].long()[seq] + out - start[seq]
    page, slot = s["table_of_pages"].long()[seq, token // case["page"]], token % case["page"]
    return [((c[page, :, slot].float() - 128) * t[page][..., None]).to(torch.bfloat16)
            for c, t in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))]


def _attend(s, q):
    """Softmax attention of each row over its sequence's visible tokens, and the log of the sum of exponentials."""
    case = s["case"]
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    seq, place, new = _row_places(s)
    table, kv = s["table_of_pages"].long().clamp(min=0), s["kv_len"].long()
    keys, values = (((c[table].float() - 128) * t[table][..., None, None]).transpose(1, 2).flatten(2, 3)
                    for c, t in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
    b, most, length = len(new), s["max_new"], keys.shape[2]
    nth = torch.arange(most, device=q.device)
    rows = (s["row_start"].long()[:-1, None] + nth).clamp(max=s["rows"] - 1)
    x = q.float()[rows].view(b, most, g, h // g, d).permute(0, 2, 3, 1, 4).reshape(b, g, -1, d)
    score = x @ keys.transpose(2, 3) * d ** -0.5
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    at, token = (kv - new)[:, None, None] + nth[:, None], torch.arange(length, device=q.device)
    seen = token <= at
    if case["window"]:
        seen = seen & (token > at - case["window"])
    score = score.view(b, g, h // g, most, length).masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = p.view(b, g, -1, length) @ values / torch.where(total > 0, total, 1.0).view(b, g, -1, 1)
    lse = (top + torch.log(total)).view(b, h, most)
    out = out.view(b, h, most, d).permute(0, 2, 1, 3)
    inner = torch.arange(s["rows"], device=q.device) - s["row_start"].long()[seq]
    return out[seq, inner].to(torch.bfloat16), lse.permute(0, 2, 1)[seq, inner]


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(case, s["x"].double(), s["positions"].double())
    starts, lens, h, g = s["row_start"].tolist(), s["kv_len"].tolist(), case["heads"], case["kv_heads"]
    page, d, pages = case["page"], case["dim"], s["table_of_pages"]
    results, ranges = [], _read_ranges(case) if case["op"] == "cache" else None
    for b, n_kv in enumerate(lens):
        r0, r1 = starts[b], starts[b + 1]
        n = r1 - r0
        held = pages[b, : -(-n_kv // page)].long()
        store = [c[held].double().sub(128).mul(t[held].double()[:, :, None, None]).transpose(0, 1).reshape(g, -1, d)
                 for c, t in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))]
        if case["op"] == "cache":
            at = torch.arange(n_kv - n, n_kv, device=pages.device).double()
            x = s["qkv"][r0:r1].double().view(n, h + 2 * g, d)
            x = torch.cat([_exact_turn(case, x[:, :h + g], at), x[:, h + g:]], 1)
            old, (f, e) = n_kv - n, ranges[b]
            if n_kv:
                store = [_exact_write(v[:, :old], t[held], u.transpose(0, 1), old, page)
                         for v, t, u in zip(store, (s["k_scale"], s["v_scale"]), (x[:, h:h + g], x[:, h + g:]))]
            results.append([x[:, :h]] + [v[:, f:e].transpose(0, 1) for v in store])
            continue
        q = s["q"][r0:r1].double()
        q = q.view(n, g, h // g, d).permute(1, 2, 0, 3)
        at, token = torch.arange(n_kv - n, n_kv, device=q.device)[:, None], torch.arange(n_kv, device=q.device)
        seen = (token <= at) & (token > at - (case["window"] or 1 << 40))
        outs, logs = [], []
        for i in range(g):
            score = torch.matmul(q[i], store[0][i, :n_kv].T) / math.sqrt(d)
            if case["softcap"]:
                score = torch.tanh(score / case["softcap"]) * case["softcap"]
            score = torch.where(seen, score, -math.inf)
            logs.append(torch.logsumexp(score, -1) if n_kv else score.new_full((h // g, n), -math.inf))
            weight = torch.where(seen, torch.exp(score - logs[-1][..., None]), 0.0)
            outs.append(torch.matmul(weight, store[1][i, :n_kv]))
        results.append([torch.stack(outs).permute(2, 0, 1, 3).reshape(n, h, d), torch.stack(logs).permute(2, 0, 1).reshape(n, h)])
    return [torch.cat(v) for v in zip(*results)]


def _exact_turn(case, x, at):
    """The rotation as products of complex numbers."""
    rot = case["rot"]
    pair = torch.arange(rot // 2, device=x.device).double()
    f, a, factor = torch.exp(pair * (-2 * math.log(case["theta"]) / rot)), _scaling(case), 1.0
    if case["scaling"] == "linear":
        f = f / a[0]
    if case["scaling"] == "bands":
        turns = a[3] * f / (2 * math.pi)
        mix = (turns - a[1]) / (a[2] - a[1])
        f = torch.where(turns > a[2], f, torch.where(turns < a[1], f / a[0], (1 - mix) * f / a[0] + mix * f))
    if case["scaling"] == "yarn":
        def place(turns):
            return rot * math.log(a[3] / (turns * 2 * math.pi)) / (2 * math.log(case["theta"]))
        low, high = max(math.floor(place(a[1])), 0), min(math.ceil(place(a[2])), rot - 1)
        stretch = torch.clamp((pair - low) / (max(high - low, 0) or 0.001), 0, 1)
        f, factor = f * (1 - stretch) + f / a[0] * stretch, 1 + 0.1 * math.log(a[0])
    angle = at[:, None] * f
    z = torch.polar(torch.full_like(angle, factor), angle)[:, None]
    if case["layout"] == "half":
        w = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * z
        return torch.cat([w.real, w.imag, x[..., rot:]], -1)
    w = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z
    return torch.cat([torch.view_as_real(w).flatten(-2), x[..., rot:]], -1)


def _exact_write(old_values, scales, new_values, old, page):
    """The values that the cache stands for after new_values (heads, tokens, dim) went in behind `old` tokens."""
    values, end = torch.cat([old_values, new_values], 1), old + new_values.shape[1]
    for p in range(old // page, -(-end // page)):
        lo, hi = p * page, min(end, (p + 1) * page)
        first = max(lo, old)
        scale = values[:, first:hi].abs().amax((1, 2)) / 127
        if first > lo:
            before = scales[p].double()
            scale = torch.maximum(scale, before)
            codes = torch.round(values[:, lo:first] / before[:, None, None])
            codes = torch.where((scale > before)[:, None, None], torch.round(codes * (before / scale)[:, None, None]), codes)
            values[:, lo:first] = codes * scale[:, None, None]
        values[:, first:hi] = torch.round(values[:, first:hi] / scale[:, None, None]) * scale[:, None, None]
    return values
