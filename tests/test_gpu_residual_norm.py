"""gdnb_residual_norm against its formula in 64 bits.

Bounds, with e = 2^-24.  A sum of C squares in fp32 is off by (log2 C + 16) e of itself at most (eight or sixteen in a row a
thread, then a tree over threads and warps), its root by half of that, division and root by 2 e.  u is a product of four or five
factors (5 e), x' adds one rounding (e of the larger term), h three more.  Each output adds half a step of its type."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.attn_layers_helpers import E32, HALF_STEP0, HALF_ULP, TYPES, guarded, intact

pytestmark = pytest.mark.gpu


def check(rows, c, x="f32", y="bf16", h="bf16", post=True, pre=True, gate="none", scale=1.0, eps=1e-6, pad=8, before=8, seed=0, size=1.0,
          with_x=True, with_h=True, with_y=True, in_place=False):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=gen)                                         # noqa: E731
    xs = torch.empty(before + rows * (c + pad), dtype=TYPES[x], device="cuda")[before:].view(rows, c + pad)
    xs.copy_(rand(rows, c + pad) * 2 * size)
    ys = (rand(rows, c + pad) * size).to(TYPES[y]).cuda()
    g = None if gate == "none" else (rand(rows if gate == "rows" else 1, c + pad) * 0.5).to(TYPES[y]).cuda()
    pw, qw = (1 + 0.1 * rand(c)).cuda() if post else None, (1 + 0.1 * rand(c)).cuda() if pre else None
    x64, y64 = xs[:, :c].double(), ys[:, :c].double()
    g64 = 1.0 if g is None else g[:, :c].double()
    tree = (np.log2(max(c, 2)) + 16) * E32
    if with_y:
        u = y64
        if post:
            u = u / ((y64 * y64).mean(-1, keepdim=True) + eps).sqrt() * pw.double()
        u = scale * g64 * u
        want_x = x64 + u
        tol_x = (tree + 6 * E32) * u.abs() + 2 * E32 * (x64.abs() + u.abs())
    else:
        want_x, tol_x = x64, torch.zeros_like(x64)
    root = ((want_x * want_x).mean(-1, keepdim=True) + eps).sqrt()
    want_h = want_x / root * (qw.double() if pre else 1.0)
    rel = tree + 6 * E32 + (tol_x.square().mean(-1, keepdim=True).sqrt() / root)
    tol_h = want_h.abs() * rel + tol_x / root * 1.2 * (1 + 0.6 * pre)
    whole_x, xo = guarded(rows, c, c + pad, x, before=before)
    whole_h, ho = guarded(rows, c, c + pad, h, before=before)
    if in_place:
        xo, ho = xs, ys
    gdn.gdnb_residual_norm(xs, ys if with_y else None, xo if with_x else None, ho if with_h else None, gate=g if with_y else None,
                           post=pw if with_y else None, pre=qw, rows=rows, c=c, scale=scale, eps=eps, x_stride=c + pad, y_stride=c + pad,
                           gate_stride=c + pad if gate == "rows" else 0, x_out_stride=c + pad, h_stride=c + pad)
    torch.cuda.synchronize()
    for on, out, want, tol, t in ((with_x, xo, want_x, tol_x, x), (with_h, ho, want_h, tol_h, h)):
        if not on:
            assert in_place or (out == 77).all()
            continue
        off = (out[:, :c].double() - want).abs() - (tol + HALF_ULP[t] * 1.001 * want.abs() + HALF_STEP0[t])
        assert (off <= 0).all(), (float(off.max()), torch.nonzero(off > 0)[:5])
    if not in_place:
        assert intact(whole_x, xo[:, :c]) and intact(whole_h, ho[:, :c])


@pytest.mark.parametrize("c", [1, 7, 8, 31, 96, 256, 264, 1000, 1024, 2881, 4096, 5120, 8192, 8200, 12000, 16383, 16384])
@pytest.mark.parametrize("rows", [1, 3, 700])
def test_widths(cuda_lib, c, rows):
    check(rows, c, gate="rows", scale=0.5, seed=c)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("y", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c", [640, 641])
def test_types(cuda_lib, x, y, h, c):
    check(650, c, x, y, h, gate="one", scale=0.22, seed=1)


@pytest.mark.parametrize("c", [512, 5120, 9000])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gate", ["none", "one", "rows"])
@pytest.mark.parametrize("outs", [(True, True), (True, False), (False, True)])
def test_parts(cuda_lib, c, post, pre, gate, outs):
    check(40, c, post=post, pre=pre, gate=gate, scale=-1.5, with_x=outs[0], with_h=outs[1], seed=2)


@pytest.mark.parametrize("c,rows", [(512, 3000), (4096, 2000), (16384, 400)])
def test_rows_one_after_the_other(cuda_lib, c, rows):
    """More rows than blocks: sums of neighbouring rows do not mix, with one sum and with two."""
    check(rows, c, "bf16", "bf16", "bf16", gate="rows")
    check(rows, c, "bf16", "bf16", "bf16", with_h=False)
    check(rows, c, "f32", "f32", "f32", post=False)


@pytest.mark.parametrize("c", [512, 4096, 2881])
def test_no_block_before(cuda_lib, c):
    check(300, c, with_y=False, with_x=False)
    check(300, c, "bf16", with_y=False)


@pytest.mark.parametrize("c,rows", [(4096, 1500), (2881, 20), (12000, 500)])
def test_in_place(cuda_lib, c, rows):
    check(rows, c, "bf16", "bf16", "bf16", gate="rows", in_place=True)
    check(rows, c, "f32", "f32", "f32", gate="one", in_place=True)


@pytest.mark.parametrize("pad,before", [(0, 0), (1, 1), (8, 3), (4, 8)])
def test_alignment(cuda_lib, pad, before):
    check(30, 1024, "bf16", "bf16", "f32", gate="rows", pad=pad, before=before)


@pytest.mark.parametrize("c", [63, 65, 71, 1023, 1030, 4095, 8191, 16369, 16370, 16371])
@pytest.mark.parametrize("rows", [9, 1300])
@pytest.mark.parametrize("gate", ["rows", "one"])
def test_rows_that_begin_anywhere(cuda_lib, c, rows, gate):
    """Odd widths side by side: every phase of eight elements, first and last groups of a row in part; one row a block and many."""
    check(rows, c, "bf16", "bf16", "bf16", gate=gate, pad=0, seed=c)
    check(rows, c, "f32", "f16", "f32", gate=gate, pad=2, post=gate == "one", pre=gate == "rows", seed=c)


@pytest.mark.parametrize("before", [0, 1, 3, 7])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_first_row_anywhere(cuda_lib, before, x):
    check(300, 2881, x, h=x, with_y=False, pad=0, before=before)
    check(2000, 777, x, h=x, with_y=False, with_x=False, pad=1, before=before)
    check(1500, 999, x, x, x, in_place=True, pad=0, before=before)


@pytest.mark.parametrize("c,rows", [(2881, 1500), (513, 3000), (12001, 400)])
def test_odd_widths_in_place(cuda_lib, c, rows):
    check(rows, c, "bf16", "bf16", "bf16", gate="rows", in_place=True, pad=0)
    check(rows, c, "f32", "f32", "f32", gate="one", in_place=True, pad=0)


def test_zeros_and_large_values(cuda_lib):
    check(5, 640, "f32", "f32", "f32", size=0.0, eps=1e-6)
    check(5, 640, "f32", "bf16", "f32", size=1e12, eps=0.0)
    check(5, 640, "bf16", "bf16", "bf16", size=1e-12, eps=1e-6)


def test_values_that_are_not_finite_stay_in_their_row(cuda_lib):
    x, y = torch.randn(6, 512, device="cuda"), torch.randn(6, 512, device="cuda")
    y[2, 100] = float("nan")
    x[4, 7] = float("inf")
    xo, h = torch.empty_like(x), torch.empty_like(x)
    w = torch.ones(512, device="cuda")
    gdn.gdnb_residual_norm(x, y, xo, h, post=w, pre=w, rows=6, c=512)
    bad = ~torch.isfinite(h).all(1)
    assert bad.tolist() == [False, False, True, False, True, False]


def test_streams_and_graph(cuda_lib):
    x, y, w = torch.randn(64, 1024, device="cuda"), torch.randn(64, 1024, device="cuda"), torch.ones(1024, device="cuda")
    xo, h = torch.empty_like(x), torch.empty_like(x)
    gdn.gdnb_residual_norm(x, y, xo, h, post=w, pre=w, rows=64, c=1024)
    torch.cuda.synchronize()
    want = h.clone()
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        gdn.gdnb_residual_norm(x, y, xo, h, post=w, pre=w, rows=64, c=1024)
    h.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want)
    y.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(h, want)
