"""gdna_attn_decode against softmax attention in 64 bits.

Bounds, with e = 2^-24 and S the largest sum |q_i k_i| * scale of a row.  A score is
a sum of D products in fp32 whose roundings are independent (8 standard deviations:
8 sqrt(D) e S), of queries in 16-bit parts that hold 20 bits or more (2^-20 S; fp32 queries over a bf16 cache with a
bf16 output and no log-sum-exp hold 16: no case here has that form with scores where it shows); both
its maximum and its own error enter a weight.  Weights enter the products in parts of
16 bits or more (2^-16, 2^-20 with an fp32 output), the sums over n keys add 8 sqrt(n) e,
the running maximum's rescales a few e more.  All of it scales max |v|; the output's
type adds half a unit in its last place."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.attn_layers_helpers import (Cache, E32, HALF_STEP0, HALF_ULP, NOWHERE, TYPES, attention64, f64, guarded, intact)

pytestmark = pytest.mark.gpu


def make(lens, nq, nkv, d, q_len=1, dtype="bf16", cache="bf16", layout="tokens", shift=0, page=16, seed=0, scale=None,
         k_scale=1.0, peaked=1.0, spare=2, pad=0):
    rng = torch.Generator().manual_seed(seed)
    batch = len(lens)
    held = [-(-max(n, 0) // page) for n in lens]
    pages, max_pages = sum(held) + spare, max(held) + 2
    store = Cache(pages, page, nkv, d, cache, layout, shift)
    ids = torch.randperm(pages, generator=rng).tolist()
    table = torch.full((batch, max_pages + 3), NOWHERE, dtype=torch.int32)
    keys, values = [], []
    for b, n in enumerate(lens):
        mine, ids = ids[:held[b]], ids[held[b]:]
        table[b, :held[b]] = torch.tensor(mine, dtype=torch.int32)
        j = torch.arange(max(n, 0))
        if n <= 0:
            keys.append(np.zeros((0, nkv, d)))
            values.append(np.zeros((0, nkv, d)))
            continue
        at = torch.tensor(mine)[j // page]
        keys.append(store.put("k", at, j % page, torch.randn((n, nkv, d), generator=rng) / k_scale) * k_scale)
        values.append(store.put("v", at, j % page, torch.randn((n, nkv, d), generator=rng) / k_scale) * k_scale)
    q = (torch.randn((batch * q_len, nq * d + pad), generator=rng) * peaked).to(TYPES[dtype]).cuda()
    return dict(lens=lens, nq=nq, nkv=nkv, d=d, q_len=q_len, store=store, table=table.cuda(), max_pages=max_pages, keys=keys,
                values=values, q=q, dtype=dtype, k_scale=k_scale, scale=d ** -0.5 if scale is None else scale, rng=rng)


def call(s, out, lse=None, gate=None, gate_strides=(None, None), stream=None, q=None, ws=None, out_stride=None):
    kp, vp = s["store"].addresses()
    need = gdn.gdna_attn_workspace(batch=len(s["lens"]), q_len=s["q_len"], nq=s["nq"], nkv=s["nkv"], d=s["d"])
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws       # NaN everywhere
    lens = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    gdn.gdna_attn_decode(s["q"] if q is None else q, kp, vp, s["table"], lens, out, ws, gate=gate, lse=lse,
                         batch=len(s["lens"]), q_len=s["q_len"], nq=s["nq"], nkv=s["nkv"], d=s["d"],
                         max_pages=s["max_pages"], table_stride=s["table"].stride(0), scale=s["scale"],
                         k_scale=s["k_scale"], v_scale=s["k_scale"], q_stride=s["q"].stride(0),
                         gate_stride=gate_strides[0], gate_head_stride=gate_strides[1],
                         out_stride=out.stride(0) if out_stride is None else out_stride, stream=stream,
                         **s["store"].args())
    torch.cuda.synchronize()


def check(s, out_type="bf16", gated=False, stream=None, with_lse=True, ws=None):
    rows, nq, d = len(s["lens"]) * s["q_len"], s["nq"], s["d"]
    whole, out = guarded(rows, nq * d, nq * d + 5, out_type)
    lse = torch.full((rows * nq + 4,), 77.0, device="cuda") if with_lse else None
    gate = gate64 = None
    if gated:
        big = torch.randn((rows, nq, 2 * d + 1), generator=s["rng"]).to(TYPES[s["dtype"]]).cuda()
        gate, gate64 = big[:, :, d:], f64(big[:, :, d:2 * d])
    call(s, out, lse, gate, (nq * (2 * d + 1), 2 * d + 1), stream, ws=ws)
    want, want_lse, size, vmax = attention64(f64(s["q"])[:, :nq * d].reshape(rows, nq, d), s["keys"], s["values"], s["lens"],
                                             s["q_len"], s["scale"], gate64)
    n = max(1, max(s["lens"]))
    score = (8 * np.sqrt(d) * E32 + 2.0 ** -20) * size
    part = 2.0 ** -20 if out_type == "f32" else 2.0 ** -16
    tol = vmax * (2 * score + part + (8 * np.sqrt(n) + 32) * E32) + HALF_ULP[out_type] * 1.001 * np.abs(want) + HALF_STEP0[out_type]
    got = f64(out).reshape(rows, nq, d)
    assert np.isfinite(got).all()
    miss = np.abs(got - want) - tol
    assert (miss <= 0).all(), (miss.max(), np.unravel_index(miss.argmax(), miss.shape))
    assert intact(whole, out)
    if with_lse:
        g = f64(lse)
        assert (g[rows * nq:] == 77.0).all()
        g = g[:rows * nq].reshape(rows, nq)
        empty = np.isinf(want_lse)
        assert (g[empty] == -np.inf).all()
        off = np.abs(g[~empty] - want_lse[~empty])
        lim = (score[..., 0] + (8 * np.sqrt(n) + 8) * E32 + 4 * E32 * np.abs(want_lse))[~empty]
        assert (off <= lim).all(), (off - lim).max()
    return got


SHORT = [1, 2, 15, 16, 17, 63, 64, 65, 130]


@pytest.mark.parametrize("d", [64, 128, 256, 96, 80, 33, 4, 1])
@pytest.mark.parametrize("nq,nkv", [(4, 1), (6, 2), (5, 5)])
def test_head_sizes(cuda_lib, d, nq, nkv):
    check(make(SHORT, nq, nkv, d, seed=d))


@pytest.mark.parametrize("cache", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256, 72])
def test_types(cuda_lib, cache, dtype, out, d):
    check(make([0, 5, 100, 257], 6, 2, d, dtype=dtype, cache=cache, seed=1, k_scale=0.125 if cache == "e4m3" else 1.0),
          out, gated=True)


@pytest.mark.parametrize("group", [1, 3, 6, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("q_len", [1, 2, 3, 8])
@pytest.mark.parametrize("d", [64, 256])
def test_groups_and_tokens(cuda_lib, group, q_len, d):
    check(make([1, 3, 40, 200], 2 * group, 2, d, q_len=q_len, seed=group))


@pytest.mark.parametrize("q_len", [1, 2, 5, 20])
@pytest.mark.parametrize("d", [128, 48])
def test_rows_without_a_key(cuda_lib, q_len, d):
    """Sequences with no key at all, fewer keys than tokens, negative lengths: zeros and -inf."""
    s = make([0, 1, q_len - 1, 0, q_len, -4, q_len + 40, 0], 6, 2, d, q_len=q_len, seed=q_len)
    got = check(s, "f32").reshape(8, q_len, -1)
    assert (got[0] == 0).all() and (got[5] == 0).all() and (got[7] == 0).all()
    check(make([0], 4, 2, d, q_len=q_len))
    check(make([0] * 700, 4, 2, d, q_len=1))


@pytest.mark.parametrize("layout", ["tokens", "heads", "pair", "beside", "padded"])
@pytest.mark.parametrize("page", [1, 5, 16, 24, 64])
@pytest.mark.parametrize("cache,shift", [("bf16", 0), ("bf16", 1), ("e4m3", 0), ("e4m3", 3)])
def test_cache_layouts(cuda_lib, layout, page, cache, shift):
    check(make([3, 77, 300], 8, 2, 128, cache=cache, layout=layout, page=page, shift=shift, seed=page))


@pytest.mark.parametrize("d,cache,lens,nq,nkv,q_len", [
    (256, "bf16", [20000], 24, 4, 1), (128, "f16", [9999, 1, 3000], 16, 2, 2), (64, "e4m3", [30001], 8, 8, 1),
    (128, "bf16", [5000, 4999, 777, 16], 32, 2, 4), (100, "bf16", [6000, 50], 4, 1, 1), (256, "e4m3", [12345], 6, 1, 3)])
def test_long_caches(cuda_lib, d, cache, lens, nq, nkv, q_len):
    """Items that lie in many blocks, and several items in one block."""
    s = make(lens, nq, nkv, d, q_len=q_len, cache=cache, page=16, seed=7, k_scale=0.125 if cache == "e4m3" else 1.0,
             peaked=1.5)
    a = check(s, "f32")
    b = check(s, "f32")
    assert np.array_equal(a, b)                         # the same bits every time


@pytest.mark.parametrize("d,nq,nkv,batch", [(128, 32, 8, 300), (64, 4, 4, 1100), (256, 6, 1, 700), (40, 4, 2, 500)])
def test_many_sequences(cuda_lib, d, nq, nkv, batch):
    rng = np.random.default_rng(d)
    lens = np.exp(rng.uniform(0, np.log(90), batch)).astype(int)
    lens[rng.random(batch) < 0.1] = 0
    check(make(lens.tolist(), nq, nkv, d, seed=batch), with_lse=False)


def test_peaked_and_flat_scores(cuda_lib):
    """One weight near 1 (scores of hundreds), equal scores, and all weight on the last or the first key."""
    check(make([500, 40], 6, 2, 128, peaked=60.0, dtype="f32", seed=1), "f32")
    s = make([500, 40], 6, 2, 128, peaked=0.0, dtype="f32", seed=1)
    check(s, "f32")
    check(make([300], 6, 2, 128, dtype="f32", seed=1, peaked=1e-6), "f32")


@pytest.mark.parametrize("dtype,cache", [("f32", "f16"), ("bf16", "f16"), ("bf16", "e4m3"), ("f32", "bf16")])
@pytest.mark.parametrize("size", [1e-7, 3e5])
def test_queries_outside_half_precision(cuda_lib, dtype, cache, size):
    """Queries far larger and smaller than fp16's range, at a scale that brings the scores back."""
    check(make([90, 33], 6, 2, 128, dtype=dtype, cache=cache, peaked=size, scale=128 ** -0.5 / size, seed=5,
               k_scale=0.125 if cache == "e4m3" else 1.0), "f32")


@pytest.mark.parametrize("d", [64, 128, 256, 40])
@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("group", [2, 11])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_what_a_row_does_not_see_does_not_reach_it(cuda_lib, d, cache, group, bad):
    """The newest token's key and value are not finite: only its own row may show it."""
    if cache == "e4m3" and bad == "inf":
        bad = "nan"                                     # the type has no infinity
    q_len = 3
    s = make([70, 3, 32, 5], 2 * group, 2, d, q_len=q_len, cache=cache, seed=8)
    rows = len(s["lens"]) * q_len
    out = torch.zeros((rows, 2 * group * d), device="cuda")
    clean = torch.zeros_like(out)
    call(s, clean)
    for b, n in enumerate(s["lens"]):
        page, token = int(s["table"][b, (n - 1) // 16]), (n - 1) % 16
        for which in ("k", "v"):
            dst = getattr(s["store"], which)
            if cache == "e4m3":
                dst.view(torch.uint8)[page, token] = 0x7F
            else:
                dst[page, token] = float(bad)
    call(s, out)
    out, clean = out.view(4, q_len, -1), clean.view(4, q_len, -1)
    assert torch.isfinite(out[:, :2]).all() and not torch.isfinite(out[:, 2]).any()
    # the same keys and weights; a path that adds them one by one may round the sums differently
    off = (out[:, :2] - clean[:, :2]).abs().max()
    assert off <= 1e-4, off


def test_page_numbers_outside_the_cache(cuda_lib):
    """They read as pages of zeros, and nothing outside the cache is touched."""
    for d in (128, 56):
        s = make([40], 4, 2, d, dtype="f32", seed=2)
        for wrong in (-1, s["store"].pages, 2 ** 31 - 1, -2 ** 31):
            s["table"][0, 1] = wrong
            k, v = s["keys"][0].copy(), s["values"][0].copy()
            k[16:32] = 0
            v[16:32] = 0
            check({**s, "keys": [k], "values": [v]}, "f32")


def test_length_past_the_table(cuda_lib):
    """kv_len above what the table row holds is cut to it."""
    s = make([64], 4, 2, 128, seed=2)
    s["max_pages"] = 4
    out = torch.zeros((1, 4 * 128), device="cuda")
    call(s, out)
    more = torch.zeros_like(out)
    call({**s, "lens": [2 ** 31 - 1]}, more)
    assert torch.equal(out, more)


def test_cache_past_32_bits(cuda_lib):
    """Pages past 2^31 elements of the cache."""
    page, d = 16, 64
    pages = 2 ** 31 // (page * d) + 3
    k = torch.empty((pages, page, 1, d), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    rng = torch.Generator().manual_seed(3)
    x = (torch.randn((2, 2, page, 1, d), generator=rng)).to(torch.float8_e4m3fn)
    for i, at in enumerate((pages - 1, 1)):
        k[at] = x[0, i].view(torch.uint8).cuda()
        v[at] = x[1, i].view(torch.uint8).cuda()
    q = torch.randn((1, 2 * d), generator=rng).cuda()
    out = torch.zeros((1, 2 * d), device="cuda")
    ws = torch.empty(gdn.gdna_attn_workspace(batch=1, q_len=1, nq=2, nkv=1, d=d), dtype=torch.uint8, device="cuda")
    gdn.gdna_attn_decode(q, k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn),
                         torch.tensor([[pages - 1, 1]], dtype=torch.int32, device="cuda"),
                         torch.tensor([30], dtype=torch.int32, device="cuda"), out, ws, batch=1, nq=2, nkv=1, d=d,
                         pages=pages, page_size=page, max_pages=2)
    kk, vv = (f64(y).reshape(32, 1, d)[:30] for y in x)
    want, _, size, vmax = attention64(f64(q).reshape(1, 2, d), [kk], [vv], [30], 1, d ** -0.5)
    assert (np.abs(f64(out).reshape(1, 2, d) - want) <= vmax * (2.0 ** -19 * (2 * size + 1))).all()


def test_one_workspace_for_many_shapes_and_another_stream(cuda_lib):
    """A workspace is scratch: calls of other shapes one after the other leave nothing that matters."""
    need = max(gdn.gdna_attn_workspace(batch=9, q_len=8, nq=40, nkv=1, d=256), 1)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    for lens, nq, nkv, d, q_len in (([4000], 8, 2, 128, 1), ([3, 9], 40, 1, 256, 8), ([2500, 1], 5, 1, 64, 1),
                                    ([900] * 9, 6, 2, 48, 2), ([4000], 8, 2, 128, 1)):
        check(make(lens, nq, nkv, d, q_len=q_len), ws=ws, stream=stream)


def test_inputs_on_any_boundary(cuda_lib):
    """q, gate and out need only their own alignment."""
    for d in (128, 64):
        s = make([50, 7], 6, 2, d, dtype="bf16", pad=1, seed=4)
        check(s, "f16", gated=True)


def test_empty_calls(cuda_lib):
    gdn.gdna_attn_decode(0, 0, 0, 0, 0, 0, 0, batch=0, nq=2, nkv=1, d=64, pages=1, page_size=1, max_pages=1, dtype=0,
                         cache_dtype=1, out_dtype=0, workspace_bytes=0)


@pytest.mark.parametrize("d,cache,page", [(128, "bf16", 16), (256, "f16", 64), (64, "e4m3", 32), (128, "f16", 24)])
def test_a_wait_that_gives_up(cuda_lib, d, cache, page):
    """With no polls every bounded wait gives up at once: rows come out NaN, the event is counted, nothing hangs, and
    the next call is whole again."""
    s = make([3000, 70, 1], 6, 2, d, q_len=2, cache=cache, page=page, seed=6, k_scale=0.125 if cache == "e4m3" else 1.0)
    out = torch.zeros((6, 6 * d), device="cuda")
    lse = torch.zeros((36,), device="cuda")
    before = gdn.gdn_device_wait_timeouts()
    try:
        gdn.gdn_set_wait_polls(0)
        call(s, out, lse)
    finally:
        gdn.gdn_set_wait_polls(gdn.GDN_DEFAULT_WAIT_POLLS)
    assert gdn.gdn_device_wait_timeouts() > before
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    before = gdn.gdn_device_wait_timeouts()
    check(s, "f32", gated=True)
    assert gdn.gdn_device_wait_timeouts() == before


@pytest.mark.parametrize("d,cache,page", [(128, "bf16", 16), (256, "f16", 64), (64, "e4m3", 32), (128, "f16", 24)])
def test_no_wait_gives_up_in_a_healthy_run(cuda_lib, d, cache, page):
    before = gdn.gdn_device_wait_timeouts()
    check(make([9000, 70, 0, 4000] * 8, 6, 2, d, cache=cache, page=page, seed=6, k_scale=0.125 if cache == "e4m3" else 1.0))
    assert gdn.gdn_device_wait_timeouts() == before


@pytest.mark.parametrize("page", [2, 4, 6, 8, 12, 40, 100, 128])
@pytest.mark.parametrize("d,cache", [(64, "f16"), (128, "bf16"), (256, "bf16"), (64, "e4m3"), (128, "e4m3"), (112, "f16")])
def test_page_sizes(cuda_lib, page, d, cache):
    """Blocks of 16 keys that lie in one page, in 2, 4 or 8 pieces of pages."""
    check(make([2000, 5, 0, 333], 6, 2, d, page=page, cache=cache, seed=page, k_scale=0.125 if cache == "e4m3" else 1.0))


@pytest.mark.parametrize("d", [8, 16, 32, 40, 48, 72, 104, 136, 160, 192, 200, 248])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [3, 12, 50])
def test_head_sizes_in_between(cuda_lib, d, cache, group):
    """Head sizes that run padded to 64, 128 or 256, whole and in parts."""
    s = make([700, 3, 64, 9], 2 * group, 2, d, q_len=2, cache=cache, layout="padded", seed=d, dtype="f32",
             k_scale=0.125 if cache == "e4m3" else 1.0)
    check(s, "f32" if group == 3 else "bf16", gated=True)


@pytest.mark.parametrize("page", [8, 16, 24])
@pytest.mark.parametrize("d,cache,nq,nkv,q_len,batch,longest", [
    (64, "e4m3", 8, 8, 1, 500, 128), (64, "f16", 72, 6, 1, 560, 64), (64, "bf16", 48, 8, 3, 420, 64),
    (48, "f16", 20, 20, 9, 200, 40), (64, "e4m3", 18, 6, 8, 560, 64), (128, "e4m3", 64, 8, 5, 420, 40),
    (256, "e4m3", 48, 4, 3, 420, 30)])
def test_many_short_items_a_block(cuda_lib, page, d, cache, nq, nkv, q_len, batch, longest):
    """Blocks that take ten items and more of one step each, in the shapes whose rings are deepest: every row's output and
    log-sum-exp is its own, and nothing lands in front of either array."""
    rng = np.random.default_rng(page * d + batch)
    lens = rng.integers(1, longest + 1, batch)
    lens[rng.random(batch) < 0.05] = 0
    s = make(lens.tolist(), nq, nkv, d, q_len=q_len, cache=cache, page=page, seed=page, k_scale=0.125 if cache == "e4m3" else 1.0)
    rows = batch * q_len
    check(s, "f32")
    before = 40 * nq                                    # room for the row of a sequence -1 and more
    whole, out = guarded(rows, nq * d, nq * d, "f32", before=before * d)
    lse = torch.full((before + rows * nq + before,), 77.0, device="cuda")
    call(s, out, lse[before:])
    assert intact(whole, out) and (lse[:before] == 77.0).all() and (lse[before + rows * nq:] == 77.0).all()


@pytest.mark.parametrize("cache", ["f16", "e4m3", "bf16"])
@pytest.mark.parametrize("d,group", [(128, 32), (64, 20), (64, 3), (128, 12), (256, 40)])
@pytest.mark.parametrize("ahead", [10.0, 14.0, 18.0])
@pytest.mark.parametrize("worth", [0.0, 0.01])
def test_small_weights_beside_a_large_one(cuda_lib, cache, d, group, ahead, worth):
    """A first key `ahead` nats above the others, with a value near zero: the output is what the small weights bring.
    The bound is relative to sum w |v| / l, which is as small, and beside it a weight's last place: 2^-40 of the row's largest
    (8 sqrt(n) of them, their roundings independent).  Enough items that most lie within one block."""
    nkv, n, batch = 4, 500, 80
    rng = torch.Generator().manual_seed(d + group)
    u = 0.1 * (1.0 - 2.0 * torch.randint(0, 2, (nkv, d), generator=rng))
    s = make([n] * batch, nkv * group, nkv, d, dtype="f32", cache=cache, seed=group, k_scale=0.125 if cache == "e4m3" else 1.0)
    q = u[None, :, None, :] + 0.005 * torch.randn((batch, nkv, group, d), generator=rng)
    s["q"] = q.reshape(batch, -1).cuda()
    first, at = s["table"][:, 0].cpu().long(), torch.zeros(batch, dtype=torch.long)
    k0 = (ahead / (s["scale"] * (u * u).sum(-1, keepdim=True)) * u).expand(batch, nkv, d)
    v0 = worth * torch.randn((batch, nkv, d), generator=rng)
    for which, mine, x in (("k", s["keys"], k0), ("v", s["values"], v0)):
        stored = s["store"].put(which, first, at, x / s["k_scale"]) * s["k_scale"]
        for b in range(batch):
            mine[b][0] = stored[b]
    out = torch.zeros((batch, nkv * group * d), device="cuda")
    lse = torch.zeros((batch * nkv * group,), device="cuda")
    call(s, out, lse)
    rows = s["q"].double().view(batch, nkv, group, d)
    k, v = (torch.tensor(np.stack(x), device="cuda") for x in (s["keys"], s["values"]))
    scores = torch.einsum("bhgd,bnhd->bhgn", rows, k) * s["scale"]
    w = torch.softmax(scores, -1)
    flat = lambda x: x.reshape(batch, nkv * group, -1).cpu().numpy()               # noqa: E731
    want, around = (flat(torch.einsum("bhgn,bnhd->bhgd", w, x)) for x in (v, v.abs()))
    size = flat(torch.einsum("bhgd,bnhd->bhgn", rows.abs(), k.abs()).amax(-1) * s["scale"])
    vmax = flat(v.abs().amax((1, 3))[:, :, None].expand(batch, nkv, group))
    want_lse = flat(torch.logsumexp(scores, -1))[..., 0]
    score = (8 * np.sqrt(d) * E32 + 2.0 ** -20) * size
    tol = around * (2 * score + 2.0 ** -20 + (8 * np.sqrt(n) + 32) * E32) + 8 * np.sqrt(n) * 2.0 ** -40 * vmax
    miss = np.abs(f64(out).reshape(want.shape) - want) - tol
    assert (miss <= 0).all(), (miss.max(), np.abs(want).max())
    lim = score[..., 0] + (8 * np.sqrt(n) + 8) * E32 + 4 * E32 * np.abs(want_lse)
    assert (np.abs(f64(lse).reshape(want_lse.shape) - want_lse) <= lim).all()


@pytest.mark.parametrize("cache", ["bf16", "f16"])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 3), (256, 12), (128, 40)])
@pytest.mark.parametrize("out_type", ["f32", "f16", "bf16"])
def test_bits_of_an_fp32_query(cuda_lib, cache, d, group, out_type):
    """Scores of hundreds that hang on the last bits of fp32 queries.  A query has two elements, x and y, the first key picks
    x, the second y: a score is one element times the scale, exact but for the query's parts (2^-23), the scale in units of
    log2, its product and the subtraction of the maximum: 8 roundings of 2^-24.  The log-sum-exp shows the error itself, with
    its own 4 roundings; a weight of two keys a quarter of it."""
    batch, nkv, scale = 3, 2, 512.0
    s = make([2, 1, 2], nkv * group, nkv, d, dtype="f32", cache=cache, seed=d)
    # x's rest after two bf16 parts is nearly half a unit of the second: 2^-17 (1 - 2^-5)
    x, y = 1.0 + 2.0 ** -8 - 2.0 ** -16 + 2.0 ** -17 - 2.0 ** -22, 1.0 + 2.0 ** -9
    q = torch.zeros((batch, nkv * group, d))
    q[..., 0], q[..., 1] = x, y
    rest = q[0, 0, 0] - q[0, 0, 0].bfloat16().float()
    assert abs(rest - rest.bfloat16().float()) > 2.0 ** -17.2
    s.update(scale=scale, q=q.view(batch, -1).cuda())
    for b, n in enumerate(s["lens"]):
        for j in range(n):
            key = torch.zeros((1, nkv, d))
            key[..., j] = 1.0
            value = torch.full((1, nkv, d), 1.0 - 2.0 * j)
            at = s["table"][b, :1].cpu().long(), torch.tensor([j])
            s["keys"][b][j] = s["store"].put("k", *at, key)[0]
            s["values"][b][j] = s["store"].put("v", *at, value)[0]
    out = torch.zeros((batch, nkv * group * d), dtype=TYPES[out_type], device="cuda")
    lse = torch.zeros((batch * nkv * group,), device="cuda")
    call(s, out, lse)
    want, want_lse, size, _ = attention64(q.double().numpy(), s["keys"], s["values"], s["lens"], 1, scale)
    off = np.abs(f64(lse).reshape(want_lse.shape) - want_lse)
    assert (off <= 12 * E32 * size[..., 0]).all(), (off / size[..., 0]).max()
    part = 2.0 ** -20 if out_type == "f32" else 2.0 ** -16
    tol = 2 * 0.25 * 2 * 8 * E32 * size + part + 32 * E32 + HALF_ULP[out_type] * 1.001 * np.abs(want) + HALF_STEP0[out_type]
    miss = np.abs(f64(out).reshape(want.shape) - want) - tol
    assert (miss <= 0).all(), miss.max()


class KernelNode(ctypes.Structure):
    """The driver's CUDA_KERNEL_NODE_PARAMS."""
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launched_blocks(s):
    """Threads of a block of each kernel that a call launches, from a capture that is not run."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    call(s, torch.zeros((len(s["lens"]) * s["q_len"], s["nq"] * s["d"]), device="cuda"))
    out = torch.zeros((len(s["lens"]) * s["q_len"], s["nq"] * s["d"]), device="cuda")
    ws = torch.empty(gdn.gdna_attn_workspace(batch=len(s["lens"]), q_len=s["q_len"], nq=s["nq"], nkv=s["nkv"], d=s["d"]),
                     dtype=torch.uint8, device="cuda")
    lens = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    kp, vp = s["store"].addresses()
    torch.cuda.synchronize()
    handle, graph, n = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t(8)
    assert cu.cuStreamBeginCapture_v2(handle, 2) == 0
    gdn.gdna_attn_decode(s["q"], kp, vp, s["table"], lens, out, ws, batch=len(s["lens"]), q_len=s["q_len"], nq=s["nq"],
                         nkv=s["nkv"], d=s["d"], max_pages=s["max_pages"], table_stride=s["table"].stride(0),
                         q_stride=s["q"].stride(0), stream=stream, **s["store"].args())
    assert cu.cuStreamEndCapture(handle, ctypes.byref(graph)) == 0
    nodes, threads = (ctypes.c_void_p * 8)(), []
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    for node in nodes[:n.value]:
        params = KernelNode()
        assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(params)) == 0
        threads.append(params.block[0])
    assert cu.cuGraphDestroy(graph) == 0
    return sorted(threads)


@pytest.mark.parametrize("cache,full,sizes", [("bf16", 64, (8, 16, 32, 40, 48, 56)), ("f16", 64, (24,)), ("e4m3", 64, (16, 32, 48)),
                                              ("e4m3", 128, (80, 96, 112))])
def test_how_heads_of_one_panel_are_copied(cuda_lib, cache, full, sizes):
    """A head that fills its panel comes by tensor copies, which one warp issues; one that ends within it 16 bytes at a time,
    by two."""
    assert launched_blocks(make([100, 7], 6, 2, full, cache=cache)) == [128, 160]            # the join, the kernel
    for d in sizes:
        assert launched_blocks(make([100, 7], 6, 2, d, cache=cache)) == [128, 192], d
