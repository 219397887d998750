"""gdnb_attn_prompt against causal softmax attention in 64 bits, sequence by sequence (bounds: prompt_helpers)."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.attn_layers_helpers import TYPES, f64, guarded, intact
from tests.prompt_helpers import call_prompt, check_prompt, gate_of, make_prompt, prompt64, rand, tolerance

pytestmark = pytest.mark.gpu

# lengths at which tiles, blocks of 128 keys and pages begin and end
FRESH = [1, 2, 127, 128, 129, 0, 300]
CACHED = [0, 126, 1, 128, 0, 57, 255]


@pytest.mark.parametrize("d", [64, 128, 256, 96, 80, 200, 33, 4, 1])
@pytest.mark.parametrize("nq,nkv", [(4, 1), (6, 2), (3, 3)])
def test_head_sizes(cuda_lib, d, nq, nkv):
    check_prompt(make_prompt(FRESH, CACHED, nq, nkv, d, seed=d))


@pytest.mark.parametrize("cache", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_types(cuda_lib, cache, dtype, out, d):
    check_prompt(make_prompt([150, 1, 37], [20, 300, 0], 6, 2, d, dtype=dtype, cache=cache, seed=1,
                             scale8=0.125 if cache == "e4m3" else 1.0), out, gated=8)


@pytest.mark.parametrize("page,cache", [(1, "bf16"), (3, "f16"), (4, "e4m3"), (5, "e4m3"), (8, "bf16"), (12, "e4m3"), (16, "f16"),
                                        (24, "bf16"), (64, "e4m3"), (100, "f16"), (128, "bf16"), (200, "e4m3"), (256, "f16")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages(cuda_lib, page, cache, d):
    check_prompt(make_prompt([200, 3, 131], [70, 130, 0], 4, 2, d, cache=cache, page=page, seed=page,
                             scale8=0.25 if cache == "e4m3" else 1.0))


@pytest.mark.parametrize("layout", ["tokens", "heads", "pair", "beside", "padded"])
@pytest.mark.parametrize("shift", [0, 8, 1])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_layouts(cuda_lib, layout, shift, cache):
    check_prompt(make_prompt([140, 5], [20, 300], 4, 2, 128, cache=cache, layout=layout, shift=shift, seed=3,
                             scale8=0.25 if cache == "e4m3" else 1.0))


@pytest.mark.parametrize("group", [1, 2, 5, 7, 8, 16, 40, 100, 128])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_groups(cuda_lib, group, d):
    check_prompt(make_prompt([40, 1, 3], [3, 200, 0], 2 * group, 2, d, seed=group))


@pytest.mark.parametrize("d", [64, 128, 256, 40])
@pytest.mark.parametrize("cache", ["f16", "bf16"])
def test_keys_in_rows(cuda_lib, d, cache):
    """No pages: keys lie in rows like the queries, rows of no sequence hold NaN."""
    fresh = [1, 128, 129, 0, 77, 300]
    check_prompt(make_prompt(fresh, [0] * 6, 6, 2, d, dtype=cache, cache=cache, dense=True, first=2, seed=d), cache, gated=3)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_keys_in_rows_given_lengths(cuda_lib, d):
    """Lengths beside dense rows: a sequence's last tokens see fewer keys, its first none."""
    s = make_prompt([100, 30], [0, 0], 4, 2, d, dense=True)
    lens = torch.tensor([60, 200], dtype=torch.int32, device="cuda")     # 60 keys of 100 rows; cut to the 30 rows
    whole, out = guarded(s["rows"], 4 * d, 4 * d + 8, "bf16", before=8)
    ws = torch.empty(gdn.gdnb_attn_prompt_workspace(rows=s["rows"], batch=2, nq=4, nkv=2, d=d), dtype=torch.uint8, device="cuda")
    k, v = s["kv"][:, 0], s["kv"][:, 1]
    gdn.gdnb_attn_prompt(s["q"], k, v, torch.tensor(s["starts"], dtype=torch.int32, device="cuda"), lens, out, ws, rows=s["rows"],
                         batch=2, nq=4, nkv=2, d=d, token_stride=s["kv"].stride(0), head_stride=s["kv"].stride(2),
                         out_stride=out.stride(0))
    s["lens"] = [60, 30]
    want, size, vmax = prompt64(s)
    got = out.double().view(s["rows"], 4, d)
    assert (got[:40] == 0).all()                                         # tokens 0 .. 39 see no key
    lo, hi = s["starts"][0], s["starts"][-1]
    assert (((got - want).abs() - tolerance(want, size, vmax, 60, d, "bf16", "bf16", "bf16"))[lo:hi] <= 0).all()
    assert intact(whole, out)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_without_a_key(cuda_lib, d):
    """Lengths below the tokens' number (pages that were not to be had): the first tokens see nothing and give 0."""
    s = make_prompt([50, 7, 130, 4], [0, 0, 0, 0], 4, 2, d, seed=5)
    lens = [20, 0, 130, -3]
    s["lens"] = [max(n, 0) for n in lens]
    s["keys"], s["values"] = [x[:n] for x, n in zip(s["keys"], s["lens"])], [x[:n] for x, n in zip(s["values"], s["lens"])]
    got, _, _ = check_prompt(s)
    assert (got[:30] == 0).all() and (got[50:57] == 0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("gated", [0, 8])
def test_few_rows_over_many_keys(cuda_lib, d, gated):
    """Tiles split over the keys and joined."""
    check_prompt(make_prompt([33, 1, 90], [9000, 20000, 5000], 6, 2, d, page=64, seed=d), gated=gated)


@pytest.mark.parametrize("seed", range(12))
def test_split_anywhere(cuda_lib, seed):
    """Lengths at which a tile's keys begin and end anywhere in a block's share of the work."""
    cached = [900 + (seed * 1213 + i * (389 + 17 * seed)) % 5000 for i in range(5)]
    check_prompt(make_prompt([1 + (5 * seed + i) % 70 for i in range(5)], cached, 2, 1, 64, page=64, seed=seed))


@pytest.mark.parametrize("d,cache", [(64, "bf16"), (128, "f16"), (128, "e4m3"), (256, "bf16"), (256, "f16")])
def test_many_tiles(cuda_lib, d, cache):
    """More tiles than two a block of the grid: every block takes one after the other."""
    check_prompt(make_prompt([900, 1, 1500, 64, 0, 700, 1100], [30, 500, 0, 1, 10, 0, 333], 24, 8, d, cache=cache, page=32, seed=d,
                             scale8=0.25 if cache == "e4m3" else 1.0), gated=8)


def test_many_short_sequences(cuda_lib):
    fresh = [(7 * i) % 13 for i in range(700)]
    cached = [(11 * i) % 90 for i in range(700)]
    check_prompt(make_prompt(fresh, cached, 8, 2, 64, page=16, seed=7))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("cache,dtype", [("bf16", "bf16"), ("f16", "f16"), ("f16", "f32")])
def test_peaked_scores(cuda_lib, d, cache, dtype):
    """Scores of tens: the running maximum grows from block to block, queries in two parts keep what shows."""
    check_prompt(make_prompt([200, 40], [500, 3000], 4, 2, d, dtype=dtype, cache=cache, peaked=12.0, seed=11),
                 "f16" if cache == "f16" else "bf16")


@pytest.mark.parametrize("cache", ["bf16", "f16"])
def test_a_key_far_ahead_with_no_value(cuda_lib, cache):
    """A first key 11 nats ahead of the others whose value is zero: what is left are weights of 2^-16 and less."""
    d, n = 128, 300
    s = make_prompt([n], [0], 2, 1, d, dtype=cache, cache=cache, page=64, seed=2)
    q0 = torch.zeros(d)
    q0[0] = 8.0
    q = (s["q"].float().view(-1, 2, d).cpu() * 0.2)
    q[:, :, 0] = 8.0
    s["q"] = q.reshape(-1, 2 * d).to(TYPES[cache]).cuda()
    store = s["pages"].store
    at, tok = s["pages"].where[0]
    key = torch.zeros((1, 1, d))
    key[0, 0, 0] = 11.0 / 8.0 * d ** 0.5
    s["keys"][0][0] = torch.tensor(store.put("k", at[:1], tok[:1], key))[0].cuda()
    s["values"][0][0] = torch.tensor(store.put("v", at[:1], tok[:1], torch.zeros((1, 1, d))))[0].cuda()
    got, want, _ = check_prompt(s, cache)
    rows = slice(20, n)                                                  # relative to what is left: weights to 2^-8 (2^-9: fp16 steps)
    off = (got[rows] - want[rows]).norm() / want[rows].norm()
    assert off < 2.0 ** -8


@pytest.mark.parametrize("d,page,dense", [(64, 16, False), (128, 16, False), (256, 64, False), (128, 5, False), (128, 0, True)])
@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
def test_values_that_are_not_finite(cuda_lib, d, page, dense, cache):
    """A value that is not finite shows in its column, in the rows that see it and in no other; so does a key in its rows."""
    if dense and cache == "e4m3":
        pytest.skip("dense rows are 16-bit")
    n, c, nkv, nq = 190, 70, 2, 4
    c = 0 if dense else c
    s = make_prompt([n, 40], [c, 0], nq, nkv, d, cache=cache, page=max(page, 1), dense=dense, seed=9,
                    scale8=0.25 if cache == "e4m3" else 1.0)
    bad = [(c + 100, 0, 3, float("nan")), (c + 101, 0, 3, float("inf")), (c + 150, 1, d - 1, float("nan")), (c + n - 1, 0, 0, float("nan"))]
    bad_keys = [(c + 170, 1, 5, float("nan"))]
    for which, marks in (("v", bad), ("k", bad_keys)):
        for j, h, col, x in marks:
            if dense:
                s["kv"][s["starts"][0] + j, 1 if which == "v" else 0, h, col] = x
            else:
                at, tok = s["pages"].where[0]
                store = getattr(s["pages"].store, which)
                if cache == "e4m3":
                    store.view(torch.uint8)[at[j], tok[j], h, col] = 0x7F
                else:
                    store[at[j], tok[j], h, col] = x
    got, _, _ = check_prompt(s, finite=False)
    clean = dict(s)
    want, size, vmax = prompt64(dict(clean, keys=[x.nan_to_num(0, 0, 0) for x in s["keys"]], values=[x.nan_to_num(0, 0, 0) for x in s["values"]]))
    tol = tolerance(want, size, vmax, n + c, d, s["dtype"], cache, "bf16")
    hit = torch.zeros_like(want, dtype=torch.bool)
    r0, g = s["starts"][0], nq // nkv
    for j, h, col, _ in bad:
        hit[r0 + j - c:r0 + n, h * g:(h + 1) * g, col] = True
    for j, h, _, _ in bad_keys:
        hit[r0 + j - c:r0 + n, h * g:(h + 1) * g] = True
    rows = slice(s["starts"][0], s["starts"][-1])
    assert (~torch.isfinite(got[rows]))[hit[rows]].all()
    fine = ~hit[rows]
    assert torch.isfinite(got[rows][fine]).all()
    # (a weight of a key whose value was taken out is as large as before: only the value counts as zero)
    sees_bad = torch.zeros_like(hit[..., :1])
    for j, h, _, _ in bad + bad_keys:
        sees_bad[r0 + j - c:r0 + n, h * g:(h + 1) * g] = True
    sure = fine & ~sees_bad.expand_as(hit)[rows]
    assert ((got - want).abs() <= tol)[rows][sure].all()


@pytest.mark.parametrize("starts", [[0, 50, 20, 70], [60, 40, 90, 90], [-5, 30, 1000, 80]])
def test_starts_that_are_wrong(cuda_lib, starts):
    """Starts out of range or going back: nothing outside the rows is written, and the call ends."""
    s = make_prompt([30, 30, 30], [5, 5, 5], 4, 2, 128, behind=0)
    s["starts"] = starts
    whole, out = guarded(s["rows"], 4 * 128, 4 * 128 + 8, "bf16", before=8)
    before = gdn.gdn_device_wait_timeouts()
    call_prompt(s, out)
    torch.cuda.synchronize()
    assert gdn.gdn_device_wait_timeouts() == before and intact(whole, out)


def test_pages_that_are_wrong(cuda_lib):
    """A page number outside the cache reads as a page of zeros."""
    s = make_prompt([60], [100], 4, 2, 128, page=16, seed=4)
    s["pages"].table[0, 2] = -7
    s["pages"].table[0, 5] = 1 << 29
    for x in (s["keys"][0], s["values"][0]):
        x[32:48] = 0
        x[80:96] = 0
    check_prompt(s)


def test_unaligned_rows(cuda_lib):
    """Queries, gates and outputs that start anywhere."""
    s = make_prompt([150, 20], [0, 40], 4, 2, 96, pad=3, seed=6)
    check_prompt(s, gated=1, pad=3)


def test_the_same_in_both_orders_and_again(cuda_lib):
    """Results do not depend on timing: split and whole tiles, twice, bit for bit; a workspace with anything in it."""
    for fresh, cached in (([33, 5], [9000, 700]), ([2000] * 8, [10] * 8)):
        s = make_prompt(fresh, cached, 8, 4, 128, page=64, seed=8)
        outs = []
        need = gdn.gdnb_attn_prompt_workspace(rows=s["rows"], batch=len(fresh), nq=8, nkv=4, d=128)
        for fill in (0, 255, 77):
            out = torch.zeros((s["rows"], 8 * 128), dtype=torch.bfloat16, device="cuda")
            call_prompt(s, out, ws=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
            outs.append(out)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_streams_and_graphs(cuda_lib):
    """Two calls on two streams with workspaces of their own, and a captured call replayed on new inputs."""
    a, b = make_prompt([200, 60], [1000, 5], 4, 2, 128, seed=1), make_prompt([90, 300], [0, 7000], 4, 2, 256, seed=2)
    outs = [torch.zeros((s["rows"], 4 * s["d"]), dtype=torch.bfloat16, device="cuda") for s in (a, b)]
    wss = [torch.empty(gdn.gdnb_attn_prompt_workspace(rows=s["rows"], batch=2, nq=4, nkv=2, d=s["d"]), dtype=torch.uint8, device="cuda") for s in (a, b)]
    plain = []
    for s, out, ws in zip((a, b), outs, wss):
        call_prompt(s, out, ws=ws)
        torch.cuda.synchronize()
        plain.append(out.clone())
        out.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, out, ws, st in zip((a, b), outs, wss, streams):
            with torch.cuda.stream(st):
                i32 = dict(dtype=torch.int32, device="cuda")
                pages = s["pages"]
                s.setdefault("start_t", torch.tensor(s["starts"], **i32))
                s.setdefault("lens_t", torch.tensor(s["lens"], **i32))
                k, v = pages.store.addresses()
                gdn.gdnb_attn_prompt(s["q"], k, v, s["start_t"], s["lens_t"], out, ws, rows=s["rows"], batch=2, nq=4, nkv=2, d=s["d"],
                                     table=pages.table, table_stride=pages.table.stride(0), max_pages=pages.max_pages,
                                     **pages.store.args())
    torch.cuda.synchronize()
    for s, out, want in zip((a, b), outs, plain):
        lo, hi = s["starts"][0], s["starts"][-1]
        assert torch.equal(out[lo:hi], want[lo:hi])
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    pages = a["pages"]
    k, v = pages.store.addresses()
    with torch.cuda.graph(graph, stream=st):
        gdn.gdnb_attn_prompt(a["q"], k, v, a["start_t"], a["lens_t"], outs[0], wss[0], rows=a["rows"], batch=2, nq=4, nkv=2, d=128,
                             table=pages.table, table_stride=pages.table.stride(0), max_pages=pages.max_pages, **pages.store.args())
    outs[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    lo, hi = a["starts"][0], a["starts"][-1]
    assert torch.equal(outs[0][lo:hi], plain[0][lo:hi])
    a["q"].mul_(0.5)
    a["lens_t"].copy_(torch.tensor([1100, 65], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    want, size, vmax = prompt64(dict(a, lens=[1100, 65], keys=[x[:n] for x, n in zip(a["keys"], [1100, 65])],
                                     values=[x[:n] for x, n in zip(a["values"], [1100, 65])]))
    got = outs[0].double().view(a["rows"], 4, 128)
    assert (((got - want).abs() - tolerance(want, size, vmax, 1200, 128, "bf16", "bf16", "bf16"))[lo:hi] <= 0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_waits_that_run_out(cuda_lib, d):
    """With no polls allowed every block gives up: the call ends, it is counted, and the next call is right."""
    s = make_prompt([200, 10], [300, 5000], 4, 2, d, seed=3)
    before = gdn.gdn_device_wait_timeouts()
    gdn.gdn_set_wait_polls(0)
    try:
        whole, out = guarded(s["rows"], 4 * d, 4 * d + 8, "bf16", before=8)
        call_prompt(s, out)
        torch.cuda.synchronize()
    finally:
        gdn.gdn_set_wait_polls(gdn.GDN_DEFAULT_WAIT_POLLS)
    assert gdn.gdn_device_wait_timeouts() > before and intact(whole, out)
    check_prompt(s)


@pytest.mark.parametrize("d,cache", [(64, "bf16"), (128, "f16"), (128, "e4m3"), (256, "bf16")])
def test_long_items(cuda_lib, d, cache):
    """Tiles split into runs of some 40 blocks, whose keys are not taken from the first on."""
    check_prompt(make_prompt([300, 2], [90000, 30011], 4, 4, d, cache=cache, page=24, seed=d, scale8=0.25 if cache == "e4m3" else 1.0), gated=8)


def test_a_long_cache(cuda_lib):
    """Places in the cache beyond 2^31 elements."""
    d, nkv, page, n = 128, 2, 256, 5000
    pages = (1 << 31) // (page * nkv * d) + 40
    kc = torch.zeros((pages, page, nkv, d), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    held = -(-n // page)
    gen = torch.Generator(device="cuda").manual_seed(1)
    kc[-held:] = torch.randn((held, page, nkv, d), device="cuda", generator=gen, dtype=torch.float16)
    vc[-held:] = torch.randn((held, page, nkv, d), device="cuda", generator=gen, dtype=torch.float16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(pages - held, pages, **i32)[None]
    T, nq = 90, 4
    q = torch.randn((T, nq * d), device="cuda", generator=gen, dtype=torch.float16)
    out = torch.empty_like(q)
    ws = torch.empty(gdn.gdnb_attn_prompt_workspace(rows=T, batch=1, nq=nq, nkv=nkv, d=d), dtype=torch.uint8, device="cuda")
    gdn.gdnb_attn_prompt(q, kc, vc, torch.tensor([0, T], **i32), torch.tensor([n], **i32), out, ws, rows=T, batch=1, nq=nq, nkv=nkv,
                         d=d, table=table, pages=pages, page_size=page, max_pages=held)
    from tests.prompt_helpers import attention_rows
    k64, v64 = (x[-held:].reshape(-1, nkv, d)[:n].double() for x in (kc, vc))
    want, size, vmax = attention_rows(q.double().view(T, nq, d), k64, v64, n - T + 1 + torch.arange(T), d ** -0.5)
    assert ((out.double().view(T, nq, d) - want).abs() <= tolerance(want, size, vmax, n, d, "f16", "f16", "f16")).all()


def test_empty_calls(cuda_lib):
    gdn.gdnb_attn_prompt(0, 0, 0, 0, 0, 0, 0, rows=0, batch=3, nq=4, nkv=2, d=64, dtype=gdn.GDNA_BF16, cache_dtype=gdn.GDNA_BF16,
                         out_dtype=gdn.GDNA_BF16, workspace_bytes=0, table=1 << 20)
    gdn.gdnb_attn_prompt(0, 0, 0, 0, 0, 0, 0, rows=5, batch=0, nq=4, nkv=2, d=64, dtype=gdn.GDNA_BF16, cache_dtype=gdn.GDNA_BF16,
                         out_dtype=gdn.GDNA_BF16, workspace_bytes=0, table=1 << 20)
