"""One decode step of a small hybrid model's two kinds of mixing layer, served from their caches.

A hybrid language model interleaves gated-delta-rule layers, whose cache is a fixed-size state, with softmax-attention
layers, whose cache grows by one key and value a token and lives in pages.  This walks a handful of requests of
different lengths through a few steps, one layer of each kind a step, with random weights:

    gdna_page_assign                       which cache slot each request's new token gets (once a step)
    gdn_decode_norm                        the gated-delta-rule layer: state update, readout, gated norm
    gdna_qk_norm_rope, gdna_attn_decode    the attention layer: head norms, rotation, cache rows; attention, output gate

The steps are captured in one CUDA graph and replayed: lengths, block table and free pages live on the GPU, so the host
does nothing between steps.  The attention layer's output is compared with a float64 recomputation at the end.

    python examples/hybrid_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_16_gb300 as gdn      # noqa: E402

# the gated-delta-rule layer: key heads, value heads, head size; the attention layer: query heads, key heads, head size
NK, NV, D = 4, 12, 128
NQ, NKV, HD, ROT = 8, 2, 256, 64
PAGE, MAX_PAGES, N_POS = 16, 64, 1024


class Requests:
    """Requests with their caches: a pool of pages, a block table, and the delta-rule states."""

    def __init__(self, lengths, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.batch = b = len(lengths)
        self.gen = gen
        rand = lambda *shape: torch.randn(shape, device="cuda", generator=gen)     # noqa: E731
        pages = sum(-(-n // PAGE) for n in lengths) + 2 * b
        order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
        self.pages = pages
        self.k_cache = torch.zeros((pages, PAGE, NKV, HD), dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.zeros_like(self.k_cache)
        self.table = torch.full((b, MAX_PAGES), -1, dtype=torch.int32, device="cuda")
        self.free_pages = order
        self.head = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.lens = [torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.unserved = torch.zeros(1, dtype=torch.int32, device="cuda")
        table = torch.empty((N_POS, ROT))
        gdn.gdna_rope_table(table, n_pos=N_POS, rot=ROT, base=1e6)
        self.cos_sin = table.cuda()
        self.qn, self.kn, self.gn = (1 + 0.1 * rand(n) for n in (HD, HD, D))
        self.state = 0.02 * rand(b, NV, D, D)
        self.workspace = torch.empty(gdn.gdna_attn_workspace(batch=b, q_len=1, nq=NQ, nkv=NKV, d=HD), dtype=torch.uint8,
                                     device="cuda")

    def assign(self, turn, fresh, rows):
        """Slots and positions of `rows` new token rows; lengths and the free list's head go from one buffer to the
        other."""
        slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        positions = torch.empty(rows, dtype=torch.int32, device="cuda")
        row_start = torch.empty(self.batch + 1, dtype=torch.int32, device="cuda")
        gdn.gdna_page_assign(self.lens[turn], fresh, self.table, self.free_pages, self.head[turn], self.lens[1 - turn],
                             row_start, slots, positions, self.head[1 - turn], self.unserved, batch=self.batch, rows=rows,
                             page_size=PAGE, max_pages=MAX_PAGES)
        return slots, positions

    def store(self, qkv, slots, positions):
        """Head norms, rotation and cache rows of a projection [rows, (q | gate) heads, k heads, v heads]; returns q."""
        rows, width = qkv.shape
        q = torch.empty((rows, NQ * HD), device="cuda")
        gdn.gdna_qk_norm_rope(qkv, qkv[:, 2 * NQ * HD:], qkv[:, (2 * NQ + NKV) * HD:], self.qn, self.kn, self.cos_sin,
                              positions, slots, q, self.k_cache, self.v_cache, rows=rows, nq=NQ, nkv=NKV, d=HD, rot=ROT,
                              n_pos=N_POS, pages=self.pages, page_size=PAGE, q_stride=width, q_head_stride=2 * HD,
                              k_stride=width, v_stride=width)
        return q

    def attend(self, turn, qkv, q):
        out = torch.empty((self.batch, NQ * HD), dtype=torch.bfloat16, device="cuda")
        gdn.gdna_attn_decode(q, self.k_cache, self.v_cache, self.table, self.lens[1 - turn], out, self.workspace,
                             gate=qkv[:, HD:], batch=self.batch, nq=NQ, nkv=NKV, d=HD, pages=self.pages, page_size=PAGE,
                             max_pages=MAX_PAGES, gate_stride=qkv.shape[1], gate_head_stride=2 * HD)
        return out

    def delta_rule(self, x):
        """The gated-delta-rule layer's step on random activations `x` (q, k, v, z side by side)."""
        q, k = (torch.nn.functional.normalize(y.view(-1, NK, D), dim=-1).flatten(1) for y in (x[:, :NK * D], x[:, NK * D:2 * NK * D]))
        v, z = x[:, 2 * NK * D:(2 * NK + NV) * D], x[:, (2 * NK + NV) * D:]
        alpha, beta = torch.full((2, self.batch, NV), 0.9, device="cuda")
        out = torch.empty((self.batch, NV * D), dtype=torch.bfloat16, device="cuda")
        gdn.gdn_decode_norm(self.state, q, k, v, alpha, beta, z, self.gn, out, batch=self.batch, nk=NK, nv=NV, d=D,
                            v_stride=x.stride(0), z_stride=x.stride(0))
        return out


def rand(r, *shape):
    return torch.randn(shape, device="cuda", generator=r.gen)


def prompts(r, lengths):
    """The prompts' keys and values into the cache (their attention and states are left out here)."""
    rows = sum(lengths)
    slots, positions = r.assign(0, torch.tensor(lengths, dtype=torch.int32, device="cuda"), rows)
    r.store(rand(r, rows, (2 * NQ + 2 * NKV) * HD), slots, positions)


def expected(r, lens, qkv, positions):
    """The attention layer's output in float64, from the cache's rows."""
    f = lambda x: x.double()                                                       # noqa: E731
    at = f(r.cos_sin)[positions.long()]
    cos, sin = at[:, None, :ROT // 2], at[:, None, ROT // 2:]
    heads = f(qkv[:, :2 * NQ * HD]).view(-1, NQ, 2 * HD)
    q, gate = heads[..., :HD], heads[..., HD:]
    q = q / (q.square().mean(-1, keepdim=True) + 1e-6).sqrt() * f(r.qn)
    a, b = q[..., :ROT // 2], q[..., ROT // 2:ROT]
    q = torch.cat([a * cos - b * sin, a * sin + b * cos, q[..., ROT:]], -1)
    out = torch.empty((r.batch, NQ, HD), dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens.tolist()):
        used = r.table[i, : -(-n // PAGE)].long()
        k, v = (f(c[used]).flatten(0, 1)[:n].repeat_interleave(NQ // NKV, 1) for c in (r.k_cache, r.v_cache))
        w = torch.softmax(torch.einsum("hd,nhd->hn", q[i], k) / HD ** 0.5, -1)
        out[i] = torch.einsum("hn,nhd->hd", w, v)
    return (out * torch.sigmoid(gate)).flatten(1)


def main(lengths=(5, 200, 16, 1, 333), steps=20):
    r = Requests(lengths)
    prompts(r, list(lengths))
    one = torch.ones(r.batch, dtype=torch.int32, device="cuda")
    qkv = torch.empty((r.batch, (2 * NQ + 2 * NKV) * HD), device="cuda")
    x = torch.empty((r.batch, (2 * NK + 2 * NV) * D), device="cuda")

    def step(turn):
        slots, positions = r.assign(turn, one, r.batch)
        mixed = r.delta_rule(x)
        q = r.store(qkv, slots, positions)
        return mixed, r.attend(turn, qkv, q), positions

    # the prompts left the lengths in buffer 1; a graph holds one step each way
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    lens, head, state = [b.clone() for b in r.lens], [b.clone() for b in r.head], r.state.clone()
    with torch.cuda.stream(stream):
        for turn in (1, 0):
            step(turn)                                                             # warm up outside the capture
        for kept, now in ((lens, r.lens), (head, r.head)):
            for a, b in zip(kept, now):
                b.copy_(a)
        r.state.copy_(state)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            first = step(1)
            second = step(0)
        for i in range(steps // 2):
            qkv.normal_(generator=r.gen)
            x.normal_(generator=r.gen)
            graph.replay()
        stream.synchronize()
    lens = r.lens[1]
    assert lens.tolist() == [n + steps // 2 * 2 for n in lengths] and r.unserved.item() == 0
    want = expected(r, lens, qkv, second[2])
    off = ((second[1].double() - want).norm() / want.norm()).item()
    print(f"{steps // 2 * 2} steps of {r.batch} requests, lengths now {lens.tolist()}: the attention layer is {off:.1e} off "
          f"float64 (bf16 output), the delta-rule layer's output has norm {second[0].float().norm().item():.1f}")
    assert off < 4e-3 and all(torch.isfinite(t.float()).all() for t in first[:2] + second[:2])
    return off


if __name__ == "__main__":
    main()
