"""gdna_qk_norm_rope against the formulas in 64 bits.

Bounds.  fp32: the mean of D squares carries at most D/32 + 6 roundings (a lane's
chain and the tree over lanes), rsqrt 2, the products with the weight and the scale
3, a rotation 3 of |a| + |b| <= sqrt(2) |y|max: under 32 half units in the last place
of the row's largest |y| for D <= 256.  Then the one rounding to the output's type."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.attn_layers_helpers import (Cache, E32, HALF_STEP0, HALF_ULP, TYPES, f64, guarded, intact, rotate64)

pytestmark = pytest.mark.gpu

FP32 = 32 * E32 * 1.5


def bound(want, kind, row_top):
    return FP32 * row_top + (HALF_ULP[kind] * np.abs(want) + HALF_STEP0[kind]) * 1.001 + 1e-30


def case(rows, nq, nkv, d, rot, inter=False, norm=True, dtype="f32", cache="bf16", layout="tokens", shift=0, gated=False,
         page=16, seed=0, k_out=False, scale=1.0, size=1.0, pad=3, stream=None, in_place=False, eps=1e-6):
    rng = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    n_pos = 300
    big = (torch.randn((rows, nq * 2 * d + pad), generator=rng) * size).to(t).cuda()
    hs = 2 * d if gated else d
    q = big[:, :nq * hs].unflatten(1, (nq, hs))[:, :, :d]
    k = (torch.randn((rows, nkv * d + pad), generator=rng) * size).to(t).cuda()
    v = (torch.randn((rows, nkv * d + 2 * pad), generator=rng) * size).to(t).cuda()
    qn, kn = (1 + 0.2 * torch.randn((2, d), generator=rng)).cuda() if norm else (None, None)
    angle = np.arange(n_pos)[:, None] * 10000.0 ** (-2 * np.arange(rot // 2) / max(rot, 1))[None]
    table = torch.tensor(np.concatenate([np.cos(angle), np.sin(angle)], 1), dtype=torch.float32).cuda()
    positions = torch.randint(0, n_pos, (rows,), generator=rng, dtype=torch.int32)
    store = Cache((rows + 20) // page + 1, page, nkv, d, cache, layout, shift)
    slots = torch.randperm(store.pages * page, generator=rng)[:rows]
    if rows > 2:
        slots[rows // 2] = -1
        slots[0] = store.pages * page          # one past the end: not stored
    before = store.buf.view(torch.uint8).clone()
    q_whole, q_out = guarded(rows, nq * d, nq * d + pad, dtype)
    q64 = f64(q)
    if in_place:
        q_out, q_stride_out = q, big.stride(0)
    else:
        q_stride_out = q_out.stride(0)
    k_whole, k_rot = guarded(rows, nkv * d, nkv * d + 2, dtype) if k_out else (None, None)
    kp, vp = store.addresses()
    cargs = store.args()
    torch.cuda.synchronize()
    gdn.gdna_qk_norm_rope(q, k, v, qn, kn, table, positions.cuda(), slots.cuda(), q_out, kp, vp, k_rot, rows=rows,
                          nq=nq, nkv=nkv, d=d, rot=rot, n_pos=n_pos, interleaved=inter, eps=eps, k_scale=scale,
                          v_scale=scale, q_stride=big.stride(0), q_head_stride=hs, k_stride=k.stride(0),
                          v_stride=v.stride(0), q_out_stride=q_stride_out, k_out_stride=nkv * d + 2, stream=stream,
                          **cargs)
    torch.cuda.synchronize()

    at = f64(table)[positions.numpy()]
    cos, sin = at[:, None, :rot // 2], at[:, None, rot // 2:]

    def head(x, w):
        if w is not None:
            x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * f64(w)
        return rotate64(x, cos, sin, rot, inter)

    want_q = head(q64, qn)
    want_k = head(f64(k[:, :nkv * d]).reshape(rows, nkv, d), kn)
    want_v = f64(v[:, :nkv * d]).reshape(rows, nkv, d)

    def near(got, want, kind, by=1.0):
        top = np.abs(want).max(-1, keepdims=True)
        want, top = want / by, top / by
        assert np.isfinite(got).all()
        miss = np.abs(got - want) - bound(want, kind, top)
        assert (miss <= 0).all(), (miss.max(), np.unravel_index(miss.argmax(), miss.shape))

    near(f64(q_out).reshape(rows, nq, d), want_q, dtype)
    if not in_place:
        assert intact(q_whole, q_out)
    if k_out:
        near(f64(k_rot).reshape(rows, nkv, d), want_k, dtype)
        assert intact(k_whole, k_rot)
    ok = (slots >= 0) & (slots < store.pages * page)
    page_at, token_at = (slots[ok] // page).cuda(), (slots[ok] % page).cuda()
    for which, want in (("k", want_k), ("v", want_v)):
        got = getattr(store, which)
        got = got.view(torch.uint8)[page_at, token_at].view(got.dtype) if cache == "e4m3" else got[page_at, token_at]
        near(f64(got), want[ok.numpy()], cache, scale)
    # nothing else of the cache was written
    mark = Cache(store.pages, page, nkv, d, cache, layout, shift)
    for which in ("k", "v"):
        m, s = getattr(mark, which), getattr(store, which)
        if cache == "e4m3":
            m, s = m.view(torch.uint8), s.view(torch.uint8)
        m[page_at, token_at] = s[page_at, token_at]
    assert torch.equal(mark.buf.view(torch.uint8), store.buf.view(torch.uint8))
    assert before.numel() == mark.buf.view(torch.uint8).numel()


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 32), (256, 64), (256, 256), (256, 0), (96, 96),
                                   (80, 40), (4, 2), (33, 32), (1, 0), (250, 250), (128, 24), (256, 8)])
@pytest.mark.parametrize("inter", [False, True])
def test_head_sizes(cuda_lib, d, rot, inter):
    case(7, 6, 2, d, rot, inter, seed=d + rot)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("d,rot,inter", [(128, 64, False), (64, 64, True), (256, 64, False), (72, 36, False)])
def test_types(cuda_lib, dtype, cache, d, rot, inter):
    case(19, 5, 1, d, rot, inter, dtype=dtype, cache=cache, scale=0.25 if cache == "e4m3" else 1.0, seed=3, pad=8)


@pytest.mark.parametrize("layout", ["tokens", "heads", "pair", "beside", "padded"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("page", [16, 5])
def test_cache_layouts(cuda_lib, layout, shift, page):
    case(23, 8, 4, 128, 128, layout=layout, shift=shift, page=page, dtype="bf16", seed=page, pad=8, k_out=True)


@pytest.mark.parametrize("rows", [1, 2, 3, 31, 400])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (24, 4), (20, 5), (3, 3)])
def test_rows_and_heads(cuda_lib, rows, nq, nkv):
    case(rows, nq, nkv, 64, 64, seed=rows, gated=rows % 2 == 1, pad=0, k_out=rows == 3)


@pytest.mark.parametrize("pad", [1, 4])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_strides_and_gated_rows(cuda_lib, pad, dtype):
    case(17, 6, 2, 128, 64, dtype=dtype, gated=True, pad=pad, seed=9)


def test_without_norm_and_in_place(cuda_lib):
    case(11, 6, 2, 128, 128, norm=False, seed=1, pad=0)
    case(11, 6, 2, 128, 128, seed=1, in_place=True)
    case(11, 6, 2, 100, 60, seed=1, in_place=True)


def test_small_and_large_values(cuda_lib):
    """Values near 1e-12 (eps decides) and 1e12 (squares past 1e24); and e4m3 that saturates."""
    case(9, 4, 2, 128, 64, size=1e-12, cache="bf16", seed=2)
    case(9, 4, 2, 128, 64, size=1e12, cache="bf16", seed=2)
    k = torch.full((1, 64), 1e4, device="cuda")
    out = torch.zeros((1, 64), device="cuda")
    c = Cache(1, 1, 1, 64, "e4m3")
    slot = torch.zeros(1, dtype=torch.int64, device="cuda")
    gdn.gdna_qk_norm_rope(out, k, -k, None, None, None, None, slot, out.clone(), *c.addresses(), rows=1, nq=1, nkv=1,
                          d=64, rot=0, n_pos=0, **c.args())
    assert (f64(c.k) == 448).all() and (f64(c.v) == -448).all()


def test_position_outside_the_table(cuda_lib):
    for d in (128, 100):
        q = torch.randn((4, d), device="cuda")
        out = torch.zeros_like(q)
        table = torch.ones((10, 64), device="cuda")
        pos = torch.tensor([0, -1, 10, 9], dtype=torch.int32, device="cuda")
        gdn.gdna_qk_norm_rope(q, None, None, None, None, table, pos, None, out, rows=4, nq=1, nkv=0, d=d, rot=64, n_pos=10)
        bad = torch.isnan(out)
        assert bad[1:3, :64].all() and not bad[1:3, 64:].any() and not bad[0].any() and not bad[3].any()


def test_keys_alone_and_cache_alone(cuda_lib):
    """Only keys to a plain array; K and V to the cache without queries; K cache without V."""
    k = torch.randn((6, 2, 128), device="cuda")
    table = torch.zeros((4, 128), device="cuda")
    table[:, :64] = 1.0                                            # no turn
    pos = torch.zeros(6, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(k)
    gdn.gdna_qk_norm_rope(None, k, None, None, None, table, pos, None, None, None, None, out, rows=6, nq=0, nkv=2, d=128,
                          rot=128, n_pos=4)
    assert torch.equal(out, k)
    c = Cache(2, 4, 2, 128, "f16")
    slot = torch.arange(6, device="cuda")
    gdn.gdna_qk_norm_rope(None, k, None, None, None, table, pos, slot, None, c.addresses()[0], None, rows=6, nq=0, nkv=2,
                          d=128, rot=128, n_pos=4, **c.args())
    assert torch.equal(c.k.flatten(0, 1)[:6], k.half()) and torch.isnan(c.v.float()).all()
    gdn.gdna_qk_norm_rope(None, k, k, None, None, table, pos, slot, None, *c.addresses(), rows=6, nq=0, nkv=2,
                          d=128, rot=128, n_pos=4, **c.args())
    assert torch.equal(c.v.flatten(0, 1)[:6], k.half())


def test_slots_past_32_bits(cuda_lib):
    """A cache whose last page begins past 2^31 elements."""
    page, nkv, d = 16, 1, 64
    pages = 2 ** 31 // (page * nkv * d) + 2
    k = torch.empty((pages, page, nkv, d), dtype=torch.uint8, device="cuda")
    k[0].zero_()
    k[-1].zero_()
    x = torch.randn((2, d), device="cuda")
    slots = torch.tensor([pages * page - 1, 0], device="cuda")
    kc = k.view(torch.float8_e4m3fn)
    gdn.gdna_qk_norm_rope(None, x, None, None, None, None, None, slots, None, kc, None, rows=2, nq=0, nkv=1, d=d, rot=0,
                          n_pos=0, pages=pages, page_size=page)
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(k[-1, -1, 0], want[0]) and torch.equal(k[0, 0, 0], want[1])
    assert not k[-1, :-1].any() and not k[0, 1:].any()


def test_another_stream(cuda_lib):
    case(31, 6, 2, 128, 64, seed=4, stream=torch.cuda.Stream())


def test_in_place_in_one_projection(cuda_lib):
    """q rotated where it lies in rows [q | k | v]; k and v read from the same rows."""
    rows, nq, nkv, d = 9, 4, 2, 64
    qkv = torch.randn((rows, (nq + 2 * nkv) * d), device="cuda")
    before = qkv.clone()
    table = torch.randn((10, d), device="cuda")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    c, plain = Cache(3, 4, nkv, d, "f16"), Cache(3, 4, nkv, d, "f16")
    slots = torch.arange(rows, device="cuda")
    w = qkv.stride(0)
    args = dict(rows=rows, nq=nq, nkv=nkv, d=d, rot=d, n_pos=10, q_stride=w, k_stride=w, v_stride=w)
    out = torch.empty((rows, nq * d), device="cuda")
    gdn.gdna_qk_norm_rope(before, before[:, nq * d:], before[:, (nq + nkv) * d:], None, None, table, pos, slots, out,
                          *plain.addresses(), **args, **plain.args())
    gdn.gdna_qk_norm_rope(qkv, qkv[:, nq * d:], qkv[:, (nq + nkv) * d:], None, None, table, pos, slots, qkv,
                          *c.addresses(), q_out_stride=w, **args, **c.args())
    assert torch.equal(qkv[:, :nq * d], out) and torch.equal(qkv[:, nq * d:], before[:, nq * d:])
    assert torch.equal(c.buf.view(torch.int16), plain.buf.view(torch.int16))
