"""The decoder block's operators as a server runs them: norm, cache rows, attention over prompts in one piece and in several,
and a decode step of requests that share the prompt's pages; on one stream, captured in a graph, against 64 bits."""
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.prompt_helpers import attention_rows, tolerance

pytestmark = pytest.mark.gpu

NQ, NKV, N_POS, PAGE, MAX_PAGES = 6, 2, 2048, 16, 64


class Server:
    """One cache, a free list, and the tensors that a step needs."""

    def __init__(self, d, kind, pages=400, seed=0):
        self.d, self.kind = d, kind
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.i32 = dict(dtype=torch.int32, device="cuda")
        self.pages = pages
        self.k = torch.full((pages, PAGE, NKV, d), float("nan"), dtype=kind, device="cuda")
        self.v = torch.full_like(self.k, float("nan"))
        self.free = torch.randperm(pages, device="cuda", generator=self.gen).to(torch.int32)
        self.head = torch.zeros(1, **self.i32)
        table = torch.empty((N_POS, d))
        gdn.gdna_rope_table(table, n_pos=N_POS, rot=d, base=1e4)
        self.cos_sin = table.cuda()
        self.norm = torch.rand(d, device="cuda", generator=self.gen) + 0.5

    def rand(self, *shape, dtype=torch.float32):
        return torch.randn(shape, device="cuda", generator=self.gen).to(dtype)

    def assign(self, cached, fresh, table, rows):
        """Pages for new tokens; returns kv_len, row_start, slots and positions."""
        b = len(cached)
        out = [torch.empty(n, **self.i32) for n in (b, b + 1, rows, 1, 1)]
        slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        gdn.gdna_page_assign(torch.tensor(cached, **self.i32), torch.tensor(fresh, **self.i32), table, self.free, self.head, out[0], out[1],
                             slots, out[2], out[3], out[4], batch=b, rows=rows, page_size=PAGE, max_pages=MAX_PAGES)
        self.head = out[3]
        assert out[4].item() == 0
        return out[0], out[1], slots, out[2]

    def store(self, q, k, v, positions, slots):
        rows, d = q.shape[0], self.d
        out = torch.empty_like(q)
        gdn.gdna_qk_norm_rope(q, k, v, self.norm, self.norm, self.cos_sin, positions, slots, out, self.k, self.v, rows=rows, nq=NQ, nkv=NKV,
                              d=d, rot=d, n_pos=N_POS, pages=self.pages, page_size=PAGE)
        return out

    def cached(self, row, n):
        """The first n keys and values of a table's row, in 64 bits."""
        used = row[: -(-n // PAGE)].long()
        return (x[used].flatten(0, 1)[:n].double() for x in (self.k, self.v))

    def prompt(self, q, row_start, kv_len, table, rows):
        ws = torch.empty(gdn.gdnb_attn_prompt_workspace(rows=rows, batch=len(kv_len), nq=NQ, nkv=NKV, d=self.d), dtype=torch.uint8, device="cuda")
        out = torch.zeros((rows, NQ * self.d), dtype=self.kind, device="cuda")
        gdn.gdnb_attn_prompt(q, self.k, self.v, row_start, kv_len, out, ws, rows=rows, batch=len(kv_len), nq=NQ, nkv=NKV, d=self.d, table=table,
                             pages=self.pages, page_size=PAGE, max_pages=MAX_PAGES)
        return out


def near(got, q, keys, values, seen, d, kind):
    name = "f16" if kind == torch.float16 else "bf16"
    want, size, vmax = attention_rows(q.double().view(-1, NQ, d), keys, values, seen, d ** -0.5)
    off = (got.double().view(-1, NQ, d) - want).abs() - tolerance(want, size, vmax, keys.shape[0], d, name, name, name)
    assert (off <= 0).all(), float(off.max())


@pytest.mark.parametrize("d,kind", [(64, torch.float16), (128, torch.bfloat16), (256, torch.bfloat16)])
def test_prompts_in_pieces(cuda_lib, d, kind):
    """Three prompts of different lengths taken in three uneven pieces: every piece's rows against the whole list of keys, and a
    decode step of gdna_attn_decode behind them."""
    s = Server(d, kind)
    total = [300, 37, 129]
    pieces = [[100, 37, 1], [63, 0, 128], [137, 0, 0]]
    table = torch.full((3, MAX_PAGES), -1, **s.i32)
    width = 2 * NQ * d
    hidden = s.rand(sum(total), width, dtype=kind)                       # the residual stream of all tokens, packed by sequence
    weight = torch.rand(width, device="cuda", generator=s.gen) + 0.5
    proj = s.rand(width, (NQ + 2 * NKV) * d, dtype=kind) * width ** -0.5
    begin = [0, 300, 337]
    cached = [0, 0, 0]
    for fresh in pieces:
        rows = sum(fresh)
        x = torch.cat([hidden[begin[b] + cached[b]:begin[b] + cached[b] + fresh[b]] for b in range(3)])
        normed, mixed_in = torch.empty_like(x), x.clone()
        gdn.gdnb_residual_norm(x, None, None, normed, pre=weight, rows=rows, c=width)
        want = x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
        assert (normed.double() - want).abs().max() <= 2.0 ** -7 * want.abs().max()
        qkv = normed @ proj
        q, k, v = (y.contiguous() for y in qkv.split([NQ * d, NKV * d, NKV * d], 1))
        kv_len, row_start, slots, positions = s.assign(cached, fresh, table, rows)
        q = s.store(q, k, v, positions, slots)
        out = s.prompt(q, row_start, kv_len, table, rows)
        at = 0
        for b, f in enumerate(fresh):
            n = cached[b] + f
            if f:
                keys, values = s.cached(table[b], n)
                near(out[at:at + f], q[at:at + f], keys, values, cached[b] + 1 + torch.arange(f), d, kind)
            at += f
            cached[b] = n
        y = torch.cat([out, out], 1)
        gdn.gdnb_residual_norm(mixed_in, y, mixed_in, normed, post=weight, pre=weight, rows=rows, c=width, scale=0.5)
        u = y.double() / (y.double().square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
        assert (mixed_in.double() - (x.double() + 0.5 * u)).abs().max() <= 2.0 ** -7 * (x.double() + 0.5 * u).abs().max()
    q, k, v = s.rand(3, NQ * d, dtype=kind), s.rand(3, NKV * d, dtype=kind), s.rand(3, NKV * d, dtype=kind)
    kv_len, row_start, slots, positions = s.assign(cached, [1, 1, 1], table, 3)
    q = s.store(q, k, v, positions, slots)
    one = s.prompt(q, row_start, kv_len, table, 3)                       # single tokens through the prompt's call as well
    ws = torch.empty(gdn.gdna_attn_workspace(batch=3, q_len=1, nq=NQ, nkv=NKV, d=d), dtype=torch.uint8, device="cuda")
    two = torch.empty_like(one)
    gdn.gdna_attn_decode(q, s.k, s.v, table, kv_len, two, ws, batch=3, nq=NQ, nkv=NKV, d=d, pages=s.pages, page_size=PAGE, max_pages=MAX_PAGES)
    for b in range(3):
        keys, values = s.cached(table[b], total[b] + 1)
        for out in (one, two):
            near(out[b:b + 1], q[b:b + 1], keys, values, [total[b] + 1], d, kind)


@pytest.mark.parametrize("d,kind", [(128, torch.bfloat16), (256, torch.bfloat16), (64, torch.float16)])
def test_answers_that_share_a_prompt(cuda_lib, d, kind):
    """A prompt is taken once; five requests answer it with pages of their own, three steps of a captured graph."""
    s = Server(d, kind, seed=1)
    n, batch, steps = 421, 5, 3
    shared = torch.full((1, MAX_PAGES), -1, **s.i32)
    q, k, v = s.rand(n, NQ * d, dtype=kind), s.rand(n, NKV * d, dtype=kind), s.rand(n, NKV * d, dtype=kind)
    kv_len, row_start, slots, positions = s.assign([0], [n], shared, n)
    q = s.store(q, k, v, positions, slots)
    out = s.prompt(q, row_start, kv_len, shared, n)
    k0, v0 = s.cached(shared[0], n)
    near(out, q, k0, v0, 1 + torch.arange(n), d, kind)

    table = torch.full((batch, MAX_PAGES), -1, **s.i32)
    lens = [torch.zeros(batch, **s.i32) for _ in range(2)]
    head = [s.head.clone(), torch.zeros(1, **s.i32)]
    one, rows = torch.ones(batch, **s.i32), batch
    start, positions, unserved = torch.empty(batch + 1, **s.i32), torch.empty(rows, **s.i32), torch.empty(1, **s.i32)
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    group = torch.tensor([0, batch], **s.i32)
    plen = torch.tensor([n], **s.i32)
    xs = [s.rand(rows, h * d, dtype=kind) for h in (NQ, NKV, NKV)]
    qs, out = torch.empty_like(xs[0]), torch.empty((rows, NQ * d), dtype=kind, device="cuda")
    ws = torch.empty(gdn.gdnb_attn_shared_workspace(batch=batch, groups=1, q_len=1, nq=NQ, nkv=NKV, d=d), dtype=torch.uint8, device="cuda")

    def step(turn):
        gdn.gdna_page_assign(lens[turn], one, table, s.free, head[turn], lens[1 - turn], start, slots, positions, head[1 - turn], unserved,
                             batch=batch, rows=rows, page_size=PAGE, max_pages=MAX_PAGES)
        positions.add_(n)                                                # own token j stands behind the prompt
        gdn.gdna_qk_norm_rope(*xs, s.norm, s.norm, s.cos_sin, positions, slots, qs, s.k, s.v, rows=rows, nq=NQ, nkv=NKV, d=d, rot=d, n_pos=N_POS,
                              pages=s.pages, page_size=PAGE)
        gdn.gdnb_attn_shared(qs, s.k, s.v, shared, plen, table, lens[1 - turn], out, ws, group_start=group, groups=1, batch=batch, nq=NQ,
                             nkv=NKV, d=d, pages=s.pages, page_size=PAGE, max_shared_pages=MAX_PAGES, max_pages=MAX_PAGES)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for turn in (0, 1):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step(turn)
            graphs.append(graph)
        for i in range(steps):
            for x in xs:
                x.copy_(s.rand(*x.shape, dtype=kind))
            graphs[i % 2].replay()
            stream.synchronize()
            assert unserved.item() == 0 and lens[(i + 1) % 2].tolist() == [i + 1] * batch
            for b in range(batch):
                k1, v1 = s.cached(table[b], i + 1)
                near(out[b:b + 1], qs[b:b + 1], torch.cat([k0, k1]), torch.cat([v0, v1]), [n + i + 1], d, kind)
