"""gdnb_attn_shared against softmax attention in 64 bits over each request's whole list of keys, prefix and own (bounds:
prompt_helpers; the own keys' part is held closer than the prefix's)."""
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.attn_layers_helpers import HALF_ULP, TYPES, guarded, intact
from tests.prompt_helpers import Pages, attention_rows, gate_of, rand, tolerance

pytestmark = pytest.mark.gpu


def make_shared(prefixes, groups, lens, nq, nkv, d, q_len=1, dtype="bf16", cache="bf16", page=16, layout="tokens", shift=0, seed=0,
                scale8=1.0, pad=0, peaked=1.0):
    """groups: requests of each group; lens: own tokens of each request.  One cache holds prefixes and own tokens."""
    gen = torch.Generator().manual_seed(seed)
    n = len(prefixes)
    pages = Pages(list(prefixes) + list(lens), nkv, d, cache, page, layout, shift, scale8, gen=gen)
    start = [0]
    for g in groups:
        start.append(start[-1] + g)
    rows = len(lens) * q_len
    return dict(pages=pages, prefixes=prefixes, start=start, lens=lens, nq=nq, nkv=nkv, d=d, q_len=q_len, rows=rows, dtype=dtype,
                cache=cache, scale8=scale8, gen=gen, scale=d ** -0.5, groups=n,
                q=(rand(gen, rows, nq * d + pad) * peaked).to(TYPES[dtype]).cuda())


def call_shared(s, out, gate=None, gate_strides=(None, None), ws=None, **kw):
    i32 = dict(dtype=torch.int32, device="cuda")
    heads = dict(nq=s["nq"], nkv=s["nkv"], d=s["d"])
    need = gdn.gdnb_attn_shared_workspace(batch=len(s["lens"]), groups=s["groups"], q_len=s["q_len"], **heads)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
    pages, n = s["pages"], s["groups"]
    k, v = pages.store.addresses()
    a = dict(group_start=torch.tensor(s["start"], **i32), groups=n, batch=len(s["lens"]), q_len=s["q_len"], scale=s["scale"],
             k_scale=s["scale8"], v_scale=s["scale8"], q_stride=s["q"].stride(0), out_stride=out.stride(0), gate=gate,
             gate_stride=gate_strides[0], gate_head_stride=gate_strides[1], shared_stride=pages.table.stride(0),
             table_stride=pages.table.stride(0), max_shared_pages=pages.max_pages, max_pages=pages.max_pages, **heads,
             **pages.store.args())
    a.update(kw)
    shared_len, lens = torch.tensor(s["prefixes"], **i32), torch.tensor(s["lens"], **i32)
    torch.cuda.synchronize()
    gdn.gdnb_attn_shared(s["q"], k, v, pages.table[:n], shared_len, pages.table[n:], lens, out, ws, **a)


def check_shared(s, out_type="bf16", gated=0, pad=8, **kw):
    rows, nq, d, T = s["rows"], s["nq"], s["d"], s["q_len"]
    whole, out = guarded(rows, nq * d, nq * d + pad, out_type, before=8)
    gate, gate64, strides = gate_of(s, gated)
    before = gdn.gdn_device_wait_timeouts()
    call_shared(s, out, gate, strides, **kw)
    torch.cuda.synchronize()
    assert gdn.gdn_device_wait_timeouts() == before
    q = s["q"][:, :nq * d].double().view(rows, nq, d)
    got = out.double().view(rows, nq, d)
    pages = s["pages"]
    done = torch.zeros(rows, dtype=torch.bool)
    for g, n in enumerate(s["prefixes"]):
        n = max(n, 0)
        for b in range(s["start"][g], s["start"][g + 1]):
            m, r = max(s["lens"][b], 0), slice(b * T, (b + 1) * T)
            done[r] = True
            own = [max(0, m - (T - 1 - t)) for t in range(T)]
            keys = torch.cat([pages.keys[g], pages.keys[s["groups"] + b]])
            values = torch.cat([pages.values[g], pages.values[s["groups"] + b]])
            want, size, vmax = attention_rows(q[r], keys, values, [n + x for x in own], s["scale"])
            tol = tolerance(want, size, vmax, n + m, d, s["dtype"], s["cache"], out_type)
            if gate64 is not None:
                want, tol = want * torch.sigmoid(gate64[r]), tol + HALF_ULP[out_type] * want.abs()
            assert torch.isfinite(got[r]).all(), (g, b)
            miss = (got[r] - want).abs() - tol
            assert (miss <= 0).all(), (g, b, float(miss.max()))
    assert (got[~done] == 77).all()
    assert intact(whole, out)
    return got


@pytest.mark.parametrize("d", [64, 128, 256, 96, 40, 33])
@pytest.mark.parametrize("nq,nkv", [(6, 2), (4, 4)])
def test_head_sizes(cuda_lib, d, nq, nkv):
    check_shared(make_shared([300, 129], [3, 4], [5, 0, 130, 1, 64, 17, 200], nq, nkv, d, seed=d), gated=8)


@pytest.mark.parametrize("cache", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("times", [1, 16])
def test_types(cuda_lib, cache, dtype, out, d, times):
    """Few requests, whose own keys go with the prefix, and many."""
    check_shared(make_shared([400], [5 * times], [5, 0, 33, 1, 64] * times, 6, 2, d, dtype=dtype, cache=cache, seed=1, scale8=0.125 if cache == "e4m3" else 1.0),
                 out, gated=1)


@pytest.mark.parametrize("q_len", [1, 2, 3, 5])
@pytest.mark.parametrize("d,group", [(128, 3), (256, 8), (64, 16), (256, 60)])
@pytest.mark.parametrize("times", [1, 8])
def test_several_tokens(cuda_lib, q_len, d, group, times):
    """Tokens of a request see fewer own keys the earlier they come; some see the prefix alone.  (60 heads on a key head: a
    request's tokens make more than one tile.)"""
    check_shared(make_shared([1000, 77, 128], [4 * times, times, 5 * times], [9, 0, 2, 1, 40, 128, 3, 0, 5, 200] * times, 2 * group, 2, d,
                             q_len=q_len, seed=q_len))


@pytest.mark.parametrize("seed", range(12))
def test_prefix_lengths(cuda_lib, seed):
    """Prefixes of lengths at which a tile's keys begin and end anywhere in a block's share of the work."""
    lens = [1 + (seed * 613 + i * (89 + 7 * seed)) % 2300 for i in range(7)]
    check_shared(make_shared(lens, [1] * 7, [i for i in range(7)], 4, 2, 64, page=64, seed=seed))


def test_a_long_prefix(cuda_lib):
    check_shared(make_shared([30011], [40], [(37 * i) % 400 for i in range(40)], 12, 4, 128, page=64, seed=2), gated=8)


def test_many_groups(cuda_lib):
    n = 50
    check_shared(make_shared([(97 * i) % 500 for i in range(n)], [i % 4 for i in range(n)], [(31 * i) % 90 for i in range(sum(i % 4 for i in range(n)))],
                             4, 2, 64, page=24, seed=3))


@pytest.mark.parametrize("page,cache", [(5, "bf16"), (8, "f16"), (24, "e4m3"), (128, "bf16")])
def test_pages(cuda_lib, page, cache):
    check_shared(make_shared([517], [6], [5, 0, 33, 1, 64, 300], 8, 2, 128, cache=cache, page=page, seed=page, scale8=0.25 if cache == "e4m3" else 1.0))


def test_no_prefix_and_nothing_at_all(cuda_lib):
    """A prefix of length 0 leaves a request's own keys; without those the row is 0."""
    s = make_shared([0, 40], [3, 2], [20, 0, 1, 0, 7], 4, 2, 128, seed=4)
    got = check_shared(s)
    assert (got[1] == 0).all()


def test_one_group_of_all(cuda_lib):
    s = make_shared([260], [4], [5, 0, 33, 200], 4, 2, 64, seed=5)
    check_shared(s, group_start=None, groups=1)


def test_requests_of_no_group(cuda_lib):
    s = make_shared([100, 50], [2, 2], [5, 6, 7, 8, 9, 10], 4, 2, 128, seed=6)
    s["start"] = [1, 3, 5]                                     # the first and the last request belong to none
    check_shared(s)


@pytest.mark.parametrize("start", [[0, 5, 2], [4, 2, 6], [-3, 2, 900]])
def test_groups_that_are_wrong(cuda_lib, start):
    s = make_shared([100, 50], [3, 3], [5, 6, 7, 8, 9, 10], 4, 2, 128, seed=6)
    s["start"] = start
    whole, out = guarded(s["rows"], 4 * 128, 4 * 128 + 8, "bf16", before=8)
    before = gdn.gdn_device_wait_timeouts()
    call_shared(s, out)
    torch.cuda.synchronize()
    assert gdn.gdn_device_wait_timeouts() == before and intact(whole, out)


def test_as_one_list_of_keys(cuda_lib):
    """The prefix's pages in front of each request's own, read by gdna_attn_decode: the same up to rounding."""
    page, d, nq, nkv = 16, 128, 8, 2
    s = make_shared([page * 20], [5], [3, 40, 17, 1, 100], nq, nkv, d, page=page, seed=7)
    out = torch.zeros((5, nq * d), dtype=torch.bfloat16, device="cuda")
    call_shared(s, out)
    pages = s["pages"]
    table = torch.cat([pages.table[:1, :20].expand(5, 20), pages.table[1:]], 1).contiguous()
    lens = torch.tensor([page * 20 + n for n in s["lens"]], dtype=torch.int32, device="cuda")
    want = torch.zeros((5, nq * d), device="cuda")
    k, v = pages.store.addresses()
    ws = torch.empty(gdn.gdna_attn_workspace(batch=5, q_len=1, nq=nq, nkv=nkv, d=d), dtype=torch.uint8, device="cuda")
    gdn.gdna_attn_decode(s["q"], k, v, table, lens, want, ws, batch=5, nq=nq, nkv=nkv, d=d, max_pages=20 + pages.max_pages,
                         table_stride=table.stride(0), **pages.store.args())
    # weights rounded to 2^-8, of values of unit variance, over hundreds of keys; the output to 2^-8
    assert (out.float() - want).norm() <= 2.0 ** -8 * want.norm()


def test_again_and_captured(cuda_lib):
    s = make_shared([3000, 500], [6, 6], [(13 * i) % 200 for i in range(12)], 8, 2, 128, page=32, seed=8)
    outs = [torch.zeros((s["rows"], 8 * 128), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    need = gdn.gdnb_attn_shared_workspace(batch=12, groups=2, q_len=1, nq=8, nkv=2, d=128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for out in outs[:2]:
        call_shared(s, out, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    i32 = dict(dtype=torch.int32, device="cuda")
    pages, (k, v) = s["pages"], s["pages"].store.addresses()
    start, plen, lens = (torch.tensor(x, **i32) for x in (s["start"], s["prefixes"], s["lens"]))
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        for _ in range(2):                                     # one call after the other, the same workspace
            gdn.gdnb_attn_shared(s["q"], k, v, pages.table[:2], plen, pages.table[2:], lens, outs[2], ws, group_start=start, groups=2,
                                 batch=12, nq=8, nkv=2, d=128, shared_stride=pages.table.stride(0), table_stride=pages.table.stride(0),
                                 max_shared_pages=pages.max_pages, max_pages=pages.max_pages, **pages.store.args())
    outs[2].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2])


def test_waits_that_run_out(cuda_lib):
    s = make_shared([700], [3], [5, 6, 7], 4, 2, 128, seed=9)
    before = gdn.gdn_device_wait_timeouts()
    gdn.gdn_set_wait_polls(0)
    try:
        whole, out = guarded(3, 4 * 128, 4 * 128 + 8, "bf16", before=8)
        call_shared(s, out)
        torch.cuda.synchronize()
    finally:
        gdn.gdn_set_wait_polls(gdn.GDN_DEFAULT_WAIT_POLLS)
    assert gdn.gdn_device_wait_timeouts() > before and intact(whole, out)
    check_shared(s)
