"""Rotary positions (mq_rope) against the float64 rotation: every layout,
scaling and type, odd sizes, strides, far and negative positions, in place."""
import numpy as np
import pytest
import torch

import nested_bit_weight_int8_b200 as mq
from gpu_util import DEV
from oracle import rope as orope

pytestmark = pytest.mark.gpu
SCALINGS = {"plain": (), "linear": (4.0,), "bands": (8.0, 1.0, 4.0, 8192.0), "yarn": (16.0, 32.0, 1.0, 4096.0)}
KIND = {torch.float32: mq.MQ_F32, torch.bfloat16: mq.MQ_BF16}


def run(x, positions, table, y, heads, dim, xs=None, ys=None, rows=None, stream=None):
    mq.rope(x, KIND[x.dtype], x.shape[0] if rows is None else rows, heads, dim, xs or heads * dim, positions, table, y,
            KIND[y.dtype], ys or heads * dim, stream)


def check(x, y, positions, theta, rot, layout, scaling):
    """y against the rotation of x (rows, heads, dim); both on the device."""
    x64 = x.float().cpu().numpy().astype(np.float64)
    w, f = orope.frequencies(theta, rot, scaling, SCALINGS[scaling])
    want = orope.rotate(x64, positions.cpu().numpy(), w, f, layout)
    tol = orope.f32_error(x64, rot, f, layout)
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert np.all(np.abs(y.float().cpu().numpy() - want) <= tol + 1e-30)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("rows,heads,dim,rot", [(1, 1, 2, 2), (3, 5, 64, 64), (7, 40, 128, 128), (33, 12, 96, 32),
                                               (5, 3, 80, 20), (2, 3, 66, 34), (1, 24, 256, 256), (400, 2, 512, 512)])
def test_rope_layouts_and_scalings(layout, scaling, rows, heads, dim, rot):
    g = torch.Generator(device=DEV).manual_seed(rows * dim)
    x = torch.randn(rows, heads, dim, device=DEV, generator=g)
    pos = torch.randint(0, 100000, (rows,), device=DEV, generator=g, dtype=torch.int32)
    table = mq.RopeTable(10000.0, rot, layout, scaling, SCALINGS[scaling], DEV)
    y = torch.full_like(x, float("nan"))
    run(x, pos, table, y, heads, dim)
    check(x, y, pos, 10000.0, rot, layout, scaling)


@pytest.mark.parametrize("ti", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("to", [torch.float32, torch.bfloat16])
def test_rope_types_strides_and_far_positions(ti, to):
    rows, heads, dim, rot = 9, 3, 128, 64
    for xs, ys, shift in [(500, 404, 0), (512, 384, 4), (513, 385, 1)]:  # aligned or not, gaps between rows
        buf = torch.randn(rows * xs + 8, device=DEV).to(ti)
        out = torch.full((rows * ys + 8,), 7.0, device=DEV, dtype=to)
        x = torch.as_strided(buf, (rows, heads, dim), (xs, dim, 1), shift)
        y = torch.as_strided(out, (rows, heads, dim), (ys, dim, 1), shift)
        pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1000003, 77, 4095, 8], dtype=torch.int32, device=DEV)
        table = mq.RopeTable(500000.0, rot, "interleaved", device=DEV)
        run(x, pos, table, y, heads, dim, xs, ys)
        # 2^31 radians in float64 are off by 2^-22: the oracle's angles by extended precision
        w = np.longdouble(500000.0) ** (-2 * np.arange(rot // 2, dtype=np.longdouble) / rot)
        t = np.fmod(pos.cpu().numpy().astype(np.longdouble)[:, None] * w, 2 * np.arccos(np.longdouble(-1))).astype(np.float64)
        x64 = x.float().cpu().numpy().astype(np.float64)
        a, b, c, s = x64[..., 0:rot:2], x64[..., 1:rot:2], np.cos(t)[:, None], np.sin(t)[:, None]
        want = x64.copy()
        want[..., 0:rot:2], want[..., 1:rot:2] = a * c - b * s, b * c + a * s
        tol = orope.f32_error(x64, rot, 1.0, "interleaved") * 1.5  # + 2^-64 turns a position: 2^31 2^-64 2 pi < 2^-30
        if to == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        assert np.all(np.abs(y.float().cpu().numpy() - want) <= tol + 1e-30)
        untouched = torch.ones_like(out, dtype=torch.bool)
        torch.as_strided(untouched, (rows, heads, dim), (ys, dim, 1), shift)[:] = False
        assert torch.all(out[untouched] == 7.0)


def test_rope_in_place_back_and_as_a_gradient():
    rows, heads, dim = 6, 4, 64
    x = torch.randn(rows, heads, dim, device=DEV)
    pos = torch.arange(100, 106, dtype=torch.int32, device=DEV)
    table = mq.RopeTable(10000.0, dim, "half", device=DEV)
    y = torch.empty_like(x)
    run(x, pos, table, y, heads, dim)
    z = x.clone()
    run(z, pos, table, z, heads, dim)
    assert torch.equal(z, y)
    run(z, -pos, table, z, heads, dim)  # the rotation back
    assert torch.all((z - x).abs() <= 16 * 2.0 ** -24 * x.abs().amax() * 2)
    # <dy, R x> = <R^T dy, x>: the gradient is the rotation at the negative position
    dy = torch.randn_like(x)
    dx = torch.empty_like(x)
    run(dy, -pos, table, dx, heads, dim)
    lhs, rhs = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    n = x.numel()
    assert abs(lhs - rhs) <= 2 * 14 * 2.0 ** -24 * dy.double().norm() * x.double().norm() * 2 and n


def test_rope_no_rows_many_rows_a_graph_and_a_stream():
    table = mq.RopeTable(10000.0, 32, "half", device=DEV)
    x = torch.randn(70001, 1, 32, device=DEV).to(torch.bfloat16)
    pos = torch.arange(70001, dtype=torch.int32, device=DEV)
    y = torch.zeros_like(x)
    run(x, pos, table, y, 1, 32, rows=0)
    assert torch.all(y == 0)
    run(x, pos, table, y, 1, 32)
    check(x, y, pos, 10000.0, 32, "half", "plain")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    z = torch.zeros_like(x)
    with torch.cuda.graph(graph, stream=side):
        run(x, pos, table, z, 1, 32, stream=torch.cuda.current_stream())
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, y * 2)
