"""Prompt and shared-prefix attention where a call's sizes, starts or values lie at the edge of what the header allows, against
64-bit references (bounds: prompt_helpers)."""
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.attn_layers_helpers import E32, HALF_ULP, TYPES, guarded, intact
from tests.prompt_helpers import (Pages, attention_rows, call_prompt, check_prompt, make_prompt, prompt64, rand, starts_of,
                                  tolerance)
from tests.test_gpu_attn_shared import call_shared, check_shared, make_shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,keys,page,nq,nkv", [
    (1000, 512, 64, 6, 2), (1000, 384, 64, 6, 2), (1000, 256, 64, 6, 2), (900, 500, 16, 8, 8), (1100, 512, 16, 16, 4),
    (1024, 512, 128, 64, 8), (3000, 130, 16, 4, 2), (2000, 512, 32, 1, 1), (1500, 700, 100, 6, 2), (5000, 3000, 64, 3, 1)])
def test_more_tokens_than_the_table_has_keys(cuda_lib, d, tokens, keys, page, nq, nkv):
    """Lengths are cut to the table and tokens are not: the first see nothing and give 0, the others' keys may lie in several
    blocks' share of the work.  (Tables of 512 keys and fewer are never split where all tokens' keys are there.)"""
    s = make_prompt([tokens, 3], [keys - tokens, 9], nq, nkv, d, page=page, seed=tokens)
    got, _, _ = check_prompt(s, max_pages=-(-keys // page))
    assert (got[:tokens - keys] == 0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths_beyond_the_table(cuda_lib, d):
    """A length above the table's keys counts as the table's."""
    s = make_prompt([1300, 700], [512 - 1300, 512 - 700], 6, 2, d, page=64, seed=d)
    lens = torch.tensor([1300, 1 << 30], dtype=torch.int32, device="cuda")
    whole = torch.full((s["rows"], 6 * d), 77.0, dtype=torch.bfloat16, device="cuda")
    want = whole.clone()
    call_prompt(s, want, max_pages=8)
    pages = s["pages"]
    k, v = pages.store.addresses()
    ws = torch.empty(gdn.gdnb_attn_prompt_workspace(rows=s["rows"], batch=2, nq=6, nkv=2, d=d), dtype=torch.uint8, device="cuda")
    start = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
    gdn.gdnb_attn_prompt(s["q"], k, v, start, lens, whole, ws, rows=s["rows"], batch=2, nq=6, nkv=2, d=d, table=pages.table,
                         table_stride=pages.table.stride(0), max_pages=8, **pages.store.args())
    torch.cuda.synchronize()
    assert torch.equal(whole, want)


@pytest.mark.parametrize("d,cache,page", [(64, "bf16", 16), (128, "bf16", 24), (128, "e4m3", 16), (128, "f16", 5), (256, "bf16", 64),
                                          (256, "e4m3", 32)])
@pytest.mark.parametrize("polls", [1, 2, 4, 8, 16, 40, 100, 300])
def test_waits_that_run_out_on_the_way(cuda_lib, d, cache, page, polls):
    """Too few polls for some of the waits: blocks give up with copies and products in flight, and wait those out before they
    end.  What is right is not asked of this call but of the next."""
    s = make_prompt([200, 10, 700], [300, 5000, 0], 4, 2, d, cache=cache, page=page, seed=3, scale8=0.25 if cache == "e4m3" else 1.0)
    whole, out = guarded(s["rows"], 4 * d, 4 * d + 8, "bf16", before=8)
    gdn.gdn_set_wait_polls(polls)
    try:
        for _ in range(3):
            call_prompt(s, out)
            torch.cuda.synchronize()
    finally:
        gdn.gdn_set_wait_polls(gdn.GDN_DEFAULT_WAIT_POLLS)
    gdn.gdn_device_wait_timeouts()
    assert intact(whole, out)
    check_prompt(s)


@pytest.mark.parametrize("d,cache", [(64, "bf16"), (128, "bf16"), (128, "e4m3"), (256, "f16")])
def test_waits_as_long_as_an_item(cuda_lib, d, cache):
    """Few polls a wait, and items of a million keys: a warp that has nothing to do until the next item, or until the last keys
    of this one, has polls enough.  (First an item of one row a block, then one of both row tiles: the second tile's warps
    wait for the first item's end.)  The list of keys is four pages again and again."""
    page, times, short, long = 64, 4096, torch.cuda.get_device_properties(0).multi_processor_count, 200
    n, cycle, batch = 4 * page * times, 4 * page, 2 * short
    gen = torch.Generator().manual_seed(d)
    store = Pages([cycle], 1, d, cache, page, scale=0.25 if cache == "e4m3" else 1.0, gen=gen)
    at = store.where[0][0][::page].to(torch.int32)
    table = at.repeat(times).repeat(batch, 1).cuda()
    fresh = [1] * short + [long] * short
    starts = torch.tensor(starts_of(fresh), dtype=torch.int32, device="cuda")
    rows = sum(fresh)
    q = rand(gen, rows, d).to(TYPES["f16" if cache != "bf16" else "bf16"]).cuda()
    whole, out = guarded(rows, d, d + 8, "bf16", before=8)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    ws = torch.empty(gdn.gdnb_attn_prompt_workspace(rows=rows, batch=batch, nq=1, nkv=1, d=d), dtype=torch.uint8, device="cuda")
    k, v = store.store.addresses()
    scale8 = store.scale
    before = gdn.gdn_device_wait_timeouts()
    gdn.gdn_set_wait_polls(40)
    try:
        gdn.gdnb_attn_prompt(q, k, v, starts, lens, out, ws, rows=rows, batch=batch, nq=1, nkv=1, d=d, table=table, max_pages=4 * times,
                             k_scale=scale8, v_scale=scale8, out_stride=out.stride(0), **store.store.args())
        torch.cuda.synchronize()
    finally:
        gdn.gdn_set_wait_polls(gdn.GDN_DEFAULT_WAIT_POLLS)
    assert gdn.gdn_device_wait_timeouts() == before
    behind = torch.cat([torch.full((f,), f - 1) - torch.arange(f) for f in fresh]).cuda()      # keys at the end that a row does not see
    count = times - (torch.arange(cycle, device="cuda")[None] >= cycle - behind[:, None]).double()
    keys, values = store.keys[0][:, 0].double(), store.values[0][:, 0].double()
    s = q.double() @ keys.T * d ** -0.5
    want = torch.softmax(s + torch.log(count), -1) @ values
    size = (q.double().abs() @ keys.abs().T * d ** -0.5).amax(-1, keepdim=True)
    tol = tolerance(want, size, values.abs().amax(), n, d, "bf16", cache, "bf16")
    assert ((out.double() - want).abs() <= tol).all() and intact(whole, out)


def test_scratch_of_the_largest_step(cuda_lib):
    """Scratch allocated once, for the largest batch, serves steps of fewer requests and tokens, whichever way their own keys go."""
    nq, nkv, d, most = 16, 4, 128, 60
    ws = torch.full((gdn.gdnb_attn_shared_workspace(batch=most, groups=3, q_len=3, nq=nq, nkv=nkv, d=d),), 255, dtype=torch.uint8, device="cuda")
    for batch, q_len, prefixes in ((60, 3, [300, 70, 9]), (39, 1, [200]), (38, 3, [500, 40]), (38, 1, [100, 30, 7]), (5, 2, [1000]), (1, 1, [40])):
        n = len(prefixes)
        groups = [batch * (g + 1) // n - batch * g // n for g in range(n)]
        check_shared(make_shared(prefixes, groups, [(7 * b) % 45 for b in range(batch)], nq, nkv, d, q_len=q_len, seed=batch), ws=ws)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache", ["f16", "e4m3", "bf16"])
@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("n", [2, 4000])
def test_all_that_an_fp32_query_holds(cuda_lib, d, cache, out, n):
    """Two keys whose scores of a hundred and more differ by what lies beyond the first 11 (8) bits of half a query's elements, all
    the same way: rounded to those the two weights would be equal.  The bound is the one of two parts whatever the output."""
    h, c = d // 2, 28.0 if cache == "e4m3" else 40.0
    s = make_prompt([1], [n - 1], 2, 1, d, dtype="f32", cache=cache, page=64, seed=1)
    at, tok = s["pages"].where[0]
    key, value = torch.full((n, 1, d), -c), torch.zeros((n, 1, d))
    key[:2] = 0.0
    key[0, 0, :h], key[1, 0, h:] = c, c
    value[0], value[1] = 1.0, -1.0
    store = s["pages"].store
    s["keys"][0] = torch.tensor(store.put("k", at, tok, key), device="cuda")
    s["values"][0] = torch.tensor(store.put("v", at, tok, value), device="cuda")
    q = torch.ones((s["rows"], 2, d))
    q[:, :, :h] += 0.9 * (2.0 ** -8 if cache == "bf16" else 2.0 ** -11)
    s["q"] = q.reshape(-1, 2 * d).cuda()
    got, want, _ = check_prompt(s, out)
    got, want = got[s["starts"][0]], want[s["starts"][0]]
    size = 2 * c * h * d ** -0.5                                  # of the other keys, as large as it gets
    bound = (2 * ((2.0 ** -16 if cache == "bf16" else 2.0 ** -22) + 8 * d ** 0.5 * E32) * size + (8 * n ** 0.5 + 32) * E32
             + (2.0 ** -8 if cache == "bf16" else 2.0 ** -11 + n * 2.0 ** -32) + HALF_ULP[out] * want.abs())
    assert (want.abs() > 0.02).all() and ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache", ["f16", "bf16"])
@pytest.mark.parametrize("cached", [0, 5000])
def test_infinite_keys(cuda_lib, d, cache, cached):
    """An infinite key's score is +inf, and the row NaN, or -inf, and the key's weight 0; a row of no other key gives 0."""
    n, col = 40, 5
    s = make_prompt([n, 1, 1], [cached, 0, 0], 6, 1, d, dtype=cache, cache=cache, page=64, seed=d)
    bad = [(0, cached + 10, 1.0), (1, 0, 1.0), (2, 0, -1.0)]
    for b, j, sign in bad:
        at, tok = s["pages"].where[b]
        s["pages"].store.k[at[j], tok[j], 0, col] = sign * float("inf")
        s["keys"][b][j, 0, col] = 0.0
    want, size, vmax = prompt64(s)
    s["keys"][0][cached + 10, 0, col] = 1e30                      # a weight of 0 where the query's element is below 0
    without = prompt64(s)[0]
    got, _, _ = check_prompt(s, cache, finite=False)
    tol = tolerance(without, size, vmax, n + cached, d, cache, cache, cache)
    q5 = s["q"].view(-1, 6, d)[:, :, col].double()
    r0 = s["starts"][0]
    for r in range(n):
        up = (q5[r0 + r] > 0) & (r >= 10)
        assert torch.isnan(got[r0 + r][up]).all()
        assert ((got[r0 + r] - without[r0 + r]).abs() <= tol[r0 + r])[~up].all()
    for b, _, sign in bad[1:]:
        r = s["starts"][b]
        up = sign * q5[r] > 0
        assert torch.isnan(got[r][up]).all() and (got[r][~up] == 0).all()


@pytest.mark.parametrize("times", [1, 30])
@pytest.mark.parametrize("cache", ["f16", "bf16"])
def test_infinite_keys_of_a_prefix(cuda_lib, times, cache):
    nq, nkv, d, col = 4, 2, 128, 7
    s = make_shared([300], [5 * times], [5, 0, 33, 1, 64] * times, nq, nkv, d, dtype=cache, cache=cache, seed=3)
    pages = s["pages"]
    at, tok = pages.where[0]
    pages.store.k[at[200], tok[200], 1, col] = float("-inf")
    out = torch.zeros((s["rows"], nq * d), dtype=TYPES[cache], device="cuda")
    call_shared(s, out)
    torch.cuda.synchronize()
    got, q = out.double().view(-1, nq, d), s["q"].double().view(-1, nq, d)
    for r, m in enumerate(s["lens"]):
        keys, values = (torch.cat([x[0], x[1 + r]]) for x in (pages.keys, pages.values))
        keys[200, 1, col] = 0.0
        _, size, vmax = attention_rows(q[r:r + 1], keys, values, torch.tensor([300 + m]), s["scale"])
        keys[200, 1, col] = -1e30
        want = attention_rows(q[r:r + 1], keys, values, torch.tensor([300 + m]), s["scale"])[0]
        up = (q[r, :, col] < 0) & (torch.arange(nq, device="cuda") >= nq // nkv)
        tol = tolerance(want, size, vmax, 300 + m, d, cache, cache, cache)
        assert torch.isnan(got[r][up]).all() and ((got[r] - want[0]).abs() <= tol[0])[~up].all()


def owners(starts, rows):
    """For each row the sequences (or groups) it belongs to, and where those end: starts are cut to the rows, ends to their starts."""
    mine = [[] for _ in range(rows)]
    for b, (x, y) in enumerate(zip(starts, starts[1:])):
        lo = min(max(x, 0), rows)
        hi = min(max(y, lo), rows)
        for r in range(lo, hi):
            mine[r].append((b, hi))
    return mine


def random_starts(seed, n, rows):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-20, rows + 20, (n + 1,), generator=gen).tolist()


@pytest.mark.parametrize("starts", [[-5, 30, 80, 1000], [60, 40, 90, 90], [0, 50, 20, 70], [-5, 30, 1000, 80], [10, 10, 60, 61], [95, 99, 120, 130],
                                    1, 2, 3, 4])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cached", [5, 3000])
def test_starts_out_of_range(cuda_lib, starts, d, cached):
    """Starts are cut to the rows; rows of no sequence stay as they were; elements of rows of several hold one of their results."""
    nq = 4
    s = make_prompt([30, 30, 30], [cached, cached, cached], nq, 2, d, behind=0)
    rows = s["rows"]
    starts = random_starts(starts, 3, rows) if isinstance(starts, int) else starts
    whole, out = guarded(rows, nq * d, nq * d + 8, "bf16", before=8)
    before = gdn.gdn_device_wait_timeouts()
    call_prompt(dict(s, starts=starts), out)
    torch.cuda.synchronize()
    assert gdn.gdn_device_wait_timeouts() == before and intact(whole, out)
    got, q = out.double().view(rows, nq, d), s["q"].double().view(rows, nq, d)
    for r, mine in enumerate(owners(starts, rows)):
        fits = (got[r] == 77) if not mine else torch.zeros_like(got[r], dtype=torch.bool)
        for b, end in mine:
            n = s["lens"][b]
            want, size, vmax = attention_rows(q[r:r + 1], s["keys"][b], s["values"][b], torch.tensor([n - (end - 1 - r)]), s["scale"])
            fits |= (got[r] - want[0]).abs() <= tolerance(want, size, vmax, n, d, "bf16", "bf16", "bf16")[0]
        assert fits.all(), (r, mine)


@pytest.mark.parametrize("start", [[0, 5, 2], [4, 2, 6], [-3, 2, 900], [6, 9, 12], [1, 1, 4], [0, 5, 2, 6], [2, 6, -1, 3]])
@pytest.mark.parametrize("times", [1, 30])
def test_groups_out_of_range(cuda_lib, start, times):
    """As above; where groups overlap nothing may be written at all."""
    nq, nkv, d, n = 4, 2, 128, len(start) - 1
    s = make_shared([100, 50, 300][:n], [6 * times] + [0] * (n - 1), [5, 6, 7, 8, 9, 10] * times, nq, nkv, d, seed=6)
    start = [x if x < 0 or x == 900 else x * times for x in start]
    batch, pages = 6 * times, s["pages"]
    whole, out = guarded(s["rows"], nq * d, nq * d + 8, "bf16", before=8)
    before = gdn.gdn_device_wait_timeouts()
    call_shared(dict(s, start=start), out)
    torch.cuda.synchronize()
    assert gdn.gdn_device_wait_timeouts() == before and intact(whole, out)
    got, q = out.double().view(-1, nq, d), s["q"].double().view(-1, nq, d)
    mine = owners(start, batch)
    apart = max(len(x) for x in mine) <= 1
    for r in range(batch):
        fits = (got[r] == 77) if not mine[r] or not apart else torch.zeros_like(got[r], dtype=torch.bool)
        for g, _ in mine[r]:
            keys, values = (torch.cat([x[g], x[n + r]]) for x in (pages.keys, pages.values))
            m = keys.shape[0]
            want, size, vmax = attention_rows(q[r:r + 1], keys, values, torch.tensor([m]), s["scale"])
            fits |= (got[r] - want[0]).abs() <= tolerance(want, size, vmax, m, d, "bf16", "bf16", "bf16")[0]
        assert fits.all(), (r, mine[r])


@pytest.mark.parametrize("d,pad,dtype", [(256, 8, "bf16"), (256, 5, "f16"), (255, 5, "f32"), (200, 5, "bf16"), (128, 5, "bf16"), (64, 8, "f16")])
@pytest.mark.parametrize("keys", [[2, 2, 0], [300, 0, 0, 0, 0, 0, 0], [1, 0, 1, 1, 0, 0, 1, 0, 0, 0]])
@pytest.mark.parametrize("times", [1, 40, 110])
def test_sequences_without_a_key_among_others(cuda_lib, d, pad, dtype, keys, times):
    """Rows that see nothing, in the blocks that also have rows of few keys: their output does not count as the others'."""
    fresh = [2 if n else 1 for n in keys] * times
    cached = [n - f for n, f in zip(keys * times, fresh)]
    cache = "f16" if dtype == "f16" else "bf16"
    s = make_prompt(fresh, cached, 6, 2, d, dtype=dtype, cache=cache, page=16, seed=len(keys))
    check_prompt(s, cache, gated=1, pad=pad)


@pytest.mark.parametrize("d,nq", [(128, 32), (256, 16)])
def test_rows_beyond_2_31_elements(cuda_lib, d, nq):
    """Queries, gates, outputs and dense keys behind the 2^31st element."""
    nkv, each, batch = 2, 100, 5300
    rows = each * batch
    assert rows * nq * d > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    kv = torch.randn((rows, 2 * nkv * d), device="cuda", generator=gen, dtype=torch.bfloat16)
    q = torch.empty((rows, nq * d), device="cuda", dtype=torch.bfloat16)
    for i in range(0, rows, each * 100):
        q[i:i + each * 100] = torch.randn((min(each * 100, rows - i), nq * d), device="cuda", generator=gen, dtype=torch.bfloat16)
    out = torch.zeros_like(q)
    starts = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * each
    ws = torch.empty(gdn.gdnb_attn_prompt_workspace(rows=rows, batch=batch, nq=nq, nkv=nkv, d=d), dtype=torch.uint8, device="cuda")
    gdn.gdnb_attn_prompt(q, kv, kv[:, nkv * d:], starts, None, out, ws, rows=rows, batch=batch, nq=nq, nkv=nkv, d=d,
                         token_stride=2 * nkv * d, gate=q)
    torch.cuda.synchronize()
    for b in (0, 1, batch // 2, batch - 1):
        r = slice(b * each, (b + 1) * each)
        q64, k64, v64 = q[r].double().view(each, nq, d), kv[r, :nkv * d].double().view(each, nkv, d), kv[r, nkv * d:].double().view(each, nkv, d)
        want, size, vmax = attention_rows(q64, k64, v64, 1 + torch.arange(each), d ** -0.5)
        tol = tolerance(want, size, vmax, each, d, "bf16", "bf16", "bf16")
        want = want * torch.sigmoid(q64)
        assert ((out[r].double().view(each, nq, d) - want).abs() <= tol + HALF_ULP["bf16"] * want.abs()).all(), b


@pytest.mark.parametrize("c", [8192, 8191])
def test_norm_rows_beyond_2_31_elements(cuda_lib, c):
    rows = (1 << 31) // c + 500
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.zeros((rows, c), dtype=torch.bfloat16, device="cuda")
    x[-700:] = torch.randn((700, c), device="cuda", generator=gen)
    y = torch.zeros_like(x)
    y[-700:] = torch.randn((700, c), device="cuda", generator=gen)
    want = x[-700:].double() + 0.5 * y[-700:].double()
    gdn.gdnb_residual_norm(x, y, x, y, rows=rows, c=c, scale=0.5)
    torch.cuda.synchronize()
    assert ((x[-700:].double() - want).abs() <= (HALF_ULP["bf16"] + 4 * E32) * want.abs() + 4 * E32).all()
    normed = want / (want.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    assert ((y[-700:].double() - normed).abs() <= (HALF_ULP["bf16"] + 40 * E32) * normed.abs() + 4 * E32).all()
    assert (x[:1000] == 0).all() and (y[:1000] == 0).all()
