"""The attention layer's calls as a server uses them: page assignment, cache rows and attention after one another, over
several steps, on one stream and captured in a graph, with pages that fill up and begin in the middle of a step."""
import os
import sys

import numpy as np
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.attn_layers_helpers import attention64, f64, rotate64

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example(cuda_lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import hybrid_decode
    finally:
        sys.path.pop(0)
    assert hybrid_decode.main(lengths=(5, 200, 16, 1, 333), steps=6) < 4e-3


@pytest.mark.parametrize("d,page,kind", [(128, 16, torch.float16), (64, 24, torch.bfloat16), (96, 5, torch.float16)])
def test_steps_of_two_tokens(cuda_lib, d, page, kind):
    """Verify steps: two tokens of every request a step, keys and values written through their slots; every step's
    attention against the history kept on the host."""
    nq, nkv, batch, t_new, steps, max_pages, rot = 6, 2, 5, 2, 9, 40, d // 2 // 8 * 8
    gen = torch.Generator().manual_seed(d)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens = [torch.tensor([0, 3, page - 1, page, 2 * page + 7], **i32), torch.zeros(batch, **i32)]
    start = lens[0].tolist()
    pages = sum(-(-n // page) for n in start) + batch * (t_new * steps // page + 2)
    free = torch.randperm(pages, generator=gen).to(**i32)
    head = [torch.zeros(1, **i32), torch.zeros(1, **i32)]
    table = torch.full((batch, max_pages), -1, **i32)
    kc = torch.full((pages, page, nkv, d), float("nan"), dtype=kind, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    keys, values = [np.zeros((0, nkv, d))] * batch, [np.zeros((0, nkv, d))] * batch
    n_pos = 400
    cs = torch.empty((n_pos, rot))
    gdn.gdna_rope_table(cs, n_pos=n_pos, rot=rot, base=1e4)
    ws = torch.empty(gdn.gdna_attn_workspace(batch=batch, q_len=t_new, nq=nq, nkv=nkv, d=d), dtype=torch.uint8, device="cuda")
    zero, unserved = torch.zeros(batch, **i32), torch.zeros(1, **i32)

    def store(fresh, rows, turn, q, k, v):
        slots, pos = torch.empty(rows, dtype=torch.int64, device="cuda"), torch.empty(rows, **i32)
        gdn.gdna_page_assign(lens[turn], fresh, table, free, head[turn], lens[1 - turn], torch.empty(batch + 1, **i32), slots,
                             pos, head[1 - turn], unserved, batch=batch, rows=rows, page_size=page, max_pages=max_pages)
        out = torch.empty_like(q)
        gdn.gdna_qk_norm_rope(q, k, v, None, None, cs.cuda(), pos, slots, out, kc, vc, rows=rows, nq=nq, nkv=nkv, d=d, rot=rot,
                              n_pos=n_pos, pages=pages, page_size=page)
        at = f64(cs)[pos.cpu().numpy()]
        turned = lambda x: rotate64(f64(x), at[:, None, :rot // 2], at[:, None, rot // 2:], rot, False)   # noqa: E731
        return out, torch.tensor(turned(k)).to(kind).double().numpy(), f64(v.to(kind)), turned(q)

    def rand(*shape):
        return torch.randn(shape, generator=gen).cuda()

    first = torch.tensor(start, **i32)
    lens[0].copy_(zero)
    rows = int(first.sum())
    _, k64, v64, _ = store(first, rows, 0, rand(rows, nq, d), rand(rows, nkv, d), rand(rows, nkv, d))
    at = np.cumsum([0] + start)
    for b in range(batch):
        keys[b], values[b] = k64[at[b]:at[b + 1]], v64[at[b]:at[b + 1]]
    fresh = torch.full((batch,), t_new, **i32)
    for i in range(steps):
        turn = (i + 1) % 2
        rows = batch * t_new
        q, k64, v64, q64 = store(fresh, rows, turn, rand(rows, nq, d), rand(rows, nkv, d), rand(rows, nkv, d))
        for b in range(batch):
            keys[b] = np.concatenate([keys[b], k64[b * t_new:(b + 1) * t_new]])
            values[b] = np.concatenate([values[b], v64[b * t_new:(b + 1) * t_new]])
        out = torch.empty((rows, nq, d), device="cuda")
        gdn.gdna_attn_decode(q, kc, vc, table, lens[1 - turn], out, ws, batch=batch, q_len=t_new, nq=nq, nkv=nkv, d=d,
                             pages=pages, page_size=page, max_pages=max_pages)
        now = [n + t_new * (i + 1) for n in start]
        assert lens[1 - turn].tolist() == now and unserved.item() == 0
        want, _, _, vmax = attention64(q64, keys, values, now, t_new, d ** -0.5)
        # a stored key may round to the other neighbour where the fp32 rotation and the 64-bit one straddle a tie
        # (2^-8 of a value for bf16, rarely); the attention itself is far nearer
        assert (np.abs(f64(out) - want) <= 2.0 ** -9 * np.maximum(vmax, 1)).all()


@pytest.mark.parametrize("page,d", [(16, 128), (8, 64), (5, 128)])
def test_a_table_written_just_before_it_is_read(cuda_lib, page, d):
    """Page assignment and attention back to back, no wait between them, into a table whose entries the last turn left
    pointing elsewhere: every turn reads the pages that its own assignment wrote.  (Keys are zero and a page's values its
    number, so a row is the mean of its pages.)"""
    batch, nq, turns, held = 96, 4, 24, 2
    i32 = dict(dtype=torch.int32, device="cuda")
    pages = 1021
    kc = torch.zeros((pages, page, 1, d), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc) + torch.arange(pages, device="cuda", dtype=torch.float16)[:, None, None, None]
    free = [torch.randperm(pages, generator=torch.Generator().manual_seed(i)).to(**i32) for i in range(turns)]
    table = torch.zeros((batch, held), **i32)
    cached, fresh, head = torch.zeros(batch, **i32), torch.full((batch,), held * page, **i32), torch.zeros(1, **i32)
    kv_len, start, head_out, unserved = torch.zeros(batch, **i32), torch.zeros(batch + 1, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
    rows = batch * held * page
    slots, pos = torch.zeros(rows, dtype=torch.int64, device="cuda"), torch.zeros(rows, **i32)
    q = torch.randn((batch, nq * d), device="cuda")
    out = torch.zeros((turns, batch, nq * d), device="cuda")
    ws = torch.empty(gdn.gdna_attn_workspace(batch=batch, q_len=1, nq=nq, nkv=1, d=d), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for i in range(turns):
        gdn.gdna_page_assign(cached, fresh, table, free[i], head, kv_len, start, slots, pos, head_out, unserved, batch=batch,
                             rows=rows, page_size=page, max_pages=held)
        gdn.gdna_attn_decode(q, kc, vc, table, kv_len, out[i], ws, batch=batch, nq=nq, nkv=1, d=d, pages=pages,
                             page_size=page, max_pages=held)
    for i in range(turns):
        want = free[i][:batch * held].view(batch, held).double().mean(1)
        assert (out[i].double() - want[:, None]).abs().max() <= 2.0 ** -19 * pages
