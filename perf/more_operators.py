"""Cases of the decoder block's operators: residual norms, attention over whole prompts, attention over a shared prefix.

A hybrid model's decoder layers are chained by gdnb_residual_norm (the norm after one block, its gate and residual scale,
the norm before the next); its attention layers take prompts through gdnb_attn_prompt (packed sequences of different
lengths, over the paged cache or over rows that were never stored) and decode batches that begin alike through
gdnb_attn_shared (the common prefix read once for all requests).  A case names one of them ("op") and its sizes; listed()
has fixed cases, draw() any of the same ranges.  run() computes a case in plain torch operations, or, where `own` is true,
with this package's calls.
"""
import math

import torch

own = False

F32, F16, BF16, F8 = "f32", "f16", "bf16", "e4m3"
TYPES = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16, F8: torch.float8_e4m3fn}
SIZE = {F32: 4, F16: 2, BF16: 2, F8: 1}
SCALE8 = 0.0625           # scale of an e4m3 cache: values to 28
MOST_FLOPS = 1.6e12       # of a drawn case
MOST_SCORES = 3.0e9       # scores of one sequence that the plain form holds at once


# ------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # between two blocks of one decoding request: both norms, fp32 residual stream (latency)
        dict(name="norm_one", op="norm", rows=1, c=5120, x=F32, y=BF16, h=BF16, post=True, gate="none", scale=1.0),
        # 256 decoding requests, a gate for each token, odd width
        dict(name="norm_decode_odd", op="norm", rows=256, c=2881, x=F16, y=F16, h=F16, post=True, gate="rows", scale=0.5),
        # a prefill of 32768 tokens: bf16 throughout, one gate for all tokens, scaled residual
        dict(name="norm_prefill", op="norm", rows=32768, c=4096, x=BF16, y=BF16, h=BF16, post=True, gate="one", scale=0.22),

        # one short prompt: first token of an answer (latency); output gate beside each query head
        dict(name="prompt_one_short", op="prompt", batch=1, low=180, high=180, cached=0, ones=0, nq=24, nkv=4, d=256, page=16,
             dtype=BF16, cache=BF16, gate=True, dense=False),
        # eight prompts of 4096 tokens, head size 256
        dict(name="prompt_batch", op="prompt", batch=8, low=4096, high=4096, cached=0, ones=0, nq=24, nkv=4, d=256, page=64,
             dtype=BF16, cache=BF16, gate=True, dense=False),
        # a ragged batch of prompts that an admission step packs, some with history, beside decoding requests
        dict(name="prompt_packed", op="prompt", batch=40, low=17, high=6000, cached=900, ones=24, nq=48, nkv=8, d=128, page=16,
             dtype=F16, cache=F16, gate=False, dense=False),
        # the next 512 tokens of one long prompt that is taken in pieces: few rows, many keys
        dict(name="prompt_piece", op="prompt", batch=1, low=512, high=512, cached=60000, ones=0, nq=32, nkv=8, d=128, page=32,
             dtype=BF16, cache=BF16, gate=False, dense=False),
        # fp32 projections over an 8-bit cache, pages that no power of two divides far
        dict(name="prompt_e4m3", op="prompt", batch=6, low=700, high=3000, cached=500, ones=2, nq=16, nkv=2, d=128, page=24,
             dtype=F32, cache=F8, gate=True, dense=False),
        # sequences scored without a cache: head size 64, keys in the projections' own rows
        dict(name="prompt_dense", op="prompt", batch=64, low=33, high=1999, cached=0, ones=0, nq=20, nkv=5, d=64, page=0,
             dtype=BF16, cache=BF16, gate=False, dense=True),

        # four requests under one system prompt (latency)
        dict(name="shared_few", op="shared", groups=1, batch=4, q_len=1, prefix=3000, low=20, high=400, empty=0, nq=24, nkv=4,
             d=256, page=16, dtype=BF16, cache=BF16, gate=True),
        # 96 answers to one long document
        dict(name="shared_document", op="shared", groups=1, batch=96, q_len=1, prefix=65536, low=50, high=2500, empty=3, nq=48,
             nkv=8, d=128, page=64, dtype=BF16, cache=BF16, gate=False),
        # three documents with a batch of requests each, two tokens to verify, 8-bit cache
        dict(name="shared_verify_e4m3", op="shared", groups=3, batch=50, q_len=2, prefix=20011, low=1, high=900, empty=2, nq=32,
             nkv=4, d=128, page=32, dtype=BF16, cache=F8, gate=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "prompt", "prompt", "prompt", "shared", "shared"])
    if op == "norm":
        c = _log(rng, 96, 12000)
        if rng.random() < 0.7:
            c += -c % 64
        rows = min(_log(rng, 1, 40000), 130_000_000 // c)
        y = rng.choice([BF16, BF16, F16, F32])
        return dict(op=op, rows=rows, c=c, x=rng.choice([F32, y]), y=y, h=y, post=rng.random() < 0.7,
                    gate=rng.choice(["none", "rows", "one"]), scale=rng.choice([1.0, 1.0, 0.22, 0.5]))
    d = rng.choice([64, 128, 128, 256, 96])
    nkv = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    page = rng.choice([8, 16, 24, 32, 64, 100, 128])
    dtype, cache = rng.choice([(BF16, BF16), (BF16, BF16), (F16, F16), (F32, BF16), (BF16, F8), (F32, F8)])
    case = dict(op=op, nq=nkv * group, nkv=nkv, d=d, page=page, dtype=dtype, cache=cache, gate=rng.random() < 0.4)
    if op == "prompt":
        batch = _log(rng, 1, 64)
        high = _log(rng, 2, 8000)
        cached = rng.choice([0, 0, _log(rng, 1, 30000)])
        per_key = 4.0 * case["nq"] * d * high * batch          # the longest case would be all of the longest sequences
        while per_key * (high / 2 + cached) > MOST_FLOPS or case["nq"] * high * float(high + cached) > MOST_SCORES:
            high, cached = max(2, high * 3 // 4), cached * 3 // 4
            per_key = 4.0 * case["nq"] * d * high * batch
        case.update(batch=batch, low=_log(rng, 1, high), high=high, cached=cached, ones=rng.choice([0, 0, batch // 2]),
                    dense=cached == 0 and cache != F8 and rng.random() < 0.4)
        return case
    batch, q_len = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 4])
    prefix = _log(rng, 100, 65536)
    while 4.0 * case["nq"] * d * batch * q_len * prefix > MOST_FLOPS / 4 or case["nq"] * batch * q_len * float(prefix) > MOST_SCORES:
        prefix = prefix * 3 // 4
    high = _log(rng, 1, 3000)
    case.update(groups=min(batch, rng.choice([1, 1, 2, 5])), batch=batch, q_len=q_len, prefix=prefix, low=_log(rng, 1, high),
                high=high, empty=batch // 9 if rng.random() < 0.3 else 0)
    return case


def _spread(n, low, high):
    """n lengths spread evenly over the logarithm of [low, high], out of order."""
    return [int(round(low * (high / low) ** ((0.5 + b * 0.6180339887) % 1.0))) if high > low else high for b in range(n)]


def _prompt_lens(case):
    """New tokens and cached tokens of each sequence."""
    fresh = _spread(case["batch"], case["low"], case["high"])
    fresh[0] = case["high"]
    for i in range(min(case["ones"], case["batch"] - 1)):
        fresh[1 + i] = 1
    cached = [0] * case["batch"]
    if case["cached"]:
        cached = [int(case["cached"] * (1.0 if b == 0 else (b * 0.7548776662) % 1.0)) for b in range(case["batch"])]
    return fresh, cached


def _shared_lens(case):
    """Prefix lengths, first request of each group, and each request's own tokens."""
    groups, batch = case["groups"], case["batch"]
    prefix = [max(1, case["prefix"] * (groups - g) // groups) for g in range(groups)]
    start = [batch * g // groups for g in range(groups)] + [batch]
    lens = [max(n, case["q_len"]) for n in _spread(batch, case["low"], case["high"])]
    for i in range(case["empty"]):
        lens[(1 + 3 * i) % batch] = 0
    return prefix, start, lens


def _out(case):
    return F16 if case["dtype"] == F16 else BF16


def _rand(gen, shape, dtype, scale=1.0):
    """Normal values of a type, made in pieces where the tensor is large."""
    out = torch.empty(shape, dtype=TYPES[dtype], device="cuda")
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, device="cuda", generator=gen, dtype=torch.float32)
        flat[i:i + n].copy_(x.mul_(scale))
    return out


def _tables(held, host):
    """Block tables of sequences with so many pages each, pages in any order; and how many pages there are."""
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=host).to(torch.int32)
    table = torch.full((len(held), max(held) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case)
    if case["op"] == "norm":
        rows, c = case["rows"], case["c"]
        s.update(x_in=_rand(gen, (rows, c), case["x"], 2.0), y_in=_rand(gen, (rows, c), case["y"]),
                 post_w=1 + 0.1 * _rand(gen, (c,), F32) if case["post"] else None, pre_w=1 + 0.1 * _rand(gen, (c,), F32),
                 gate_in=None if case["gate"] == "none" else _rand(gen, (rows if case["gate"] == "rows" else 1, c), case["y"], 0.5),
                 x_out=torch.empty((rows, c), dtype=TYPES[case["x"]], device="cuda"),
                 h_out=torch.empty((rows, c), dtype=TYPES[case["h"]], device="cuda"))
        return s
    nq, nkv, d, page = case["nq"], case["nkv"], case["d"], case["page"]
    s["scale8"] = SCALE8 if case["cache"] == F8 else 1.0
    if case["op"] == "prompt":
        fresh, cached = _prompt_lens(case)
        rows, lens = sum(fresh), [f + c for f, c in zip(fresh, cached)]
        starts = [0]
        for f in fresh:
            starts.append(starts[-1] + f)
        if case["dense"]:
            kv = _rand(gen, (rows, 2, nkv, d), case["cache"])
            s.update(k=kv[:, 0], v=kv[:, 1], table=None, kv_len=None, pages=1, max_pages=1, page=rows)
        else:
            table, pages = _tables([-(-n // page) for n in lens], host)
            s.update(table=table.to("cuda"), pages=pages, max_pages=table.shape[1], kv_len=torch.tensor(lens, **i32),
                     k=_rand(gen, (pages, page, nkv, d), case["cache"], 1.0 / s["scale8"]),
                     v=_rand(gen, (pages, page, nkv, d), case["cache"], 1.0 / s["scale8"]))
        s.update(rows=rows, starts=starts, lens=lens, row_start=torch.tensor(starts, **i32))
    else:
        rows = case["batch"] * case["q_len"]
        prefix, start, lens = _shared_lens(case)
        table, pages = _tables([-(-n // page) for n in prefix + lens], host)
        shared, mine = table[:case["groups"]], table[case["groups"]:]
        s.update(rows=rows, starts=start, prefixes=prefix, lens=lens, pages=pages, max_pages=table.shape[1],
                 shared_table=shared.to("cuda"), table=mine.to("cuda"), shared_len=torch.tensor(prefix, **i32),
                 group_start=torch.tensor(start, **i32), kv_len=torch.tensor(lens, **i32),
                 k=_rand(gen, (pages, page, nkv, d), case["cache"], 1.0 / s["scale8"]),
                 v=_rand(gen, (pages, page, nkv, d), case["cache"], 1.0 / s["scale8"]))
    q = _rand(gen, (rows, nq, 2 * d if case["gate"] else d), case["dtype"])
    s.update(q=q[:, :, :d].contiguous().mul_(1.5), gate_in=q[:, :, d:] if case["gate"] else None,
             out_t=torch.empty((rows, nq, d), dtype=TYPES[_out(case)], device="cuda"))
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_norm(s):
    x, y = s["x_in"].float(), s["y_in"].float()
    if s["post_w"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * s["post_w"]
    if s["gate_in"] is not None:
        y = y * s["gate_in"].float()
    x = x + s["scale"] * y
    h = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["pre_w"]
    return dict(x=x.to(s["x_out"].dtype), h=h.to(s["h_out"].dtype))


def _tokens(cache, pages, n, scale8):
    """The n tokens of some pages in 32 bits, [heads, n, d]."""
    x = cache.view(torch.uint8)[pages].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else cache[pages]
    return (x.flatten(0, 1)[:n].float() * scale8).transpose(0, 1)


def _softmax_rows(q, k, v, seen):
    """q [H, G, T, D], k and v [H, L, D]; token t sees the first seen[t] keys."""
    H, G, T, D = q.shape
    score = torch.matmul(q.reshape(H, G * T, D), k.transpose(1, 2)).mul_(1.0 / math.sqrt(D)).view(H, G, T, -1)
    score.masked_fill_(torch.arange(k.shape[1], device=q.device)[None] >= seen[:, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(H, G * T, -1), v).view(H, G, T, D)
    return o / torch.where(total == 0, 1.0, total), top + torch.log(total)


def _plain_prompt(s):
    H, D, G = s["nkv"], s["d"], s["nq"] // s["nkv"]
    out = torch.empty((s["rows"], s["nq"], D), device="cuda")
    for b, n in enumerate(s["lens"]):
        r0, r1 = s["starts"][b], s["starts"][b + 1]
        T = r1 - r0
        if s["table"] is None:
            k, v = (s[x][r0:r1].float().transpose(0, 1) for x in ("k", "v"))
        else:
            used = s["table"][b, : -(-n // s["page"])].long()
            k, v = (_tokens(s[x], used, n, s["scale8"]) for x in ("k", "v"))
        q = s["q"][r0:r1].float().view(T, H, G, D).permute(1, 2, 0, 3)
        seen = n - T + 1 + torch.arange(T, device="cuda")
        out[r0:r1] = _softmax_rows(q, k, v, seen)[0].permute(2, 0, 1, 3).reshape(T, H * G, D)
    if s["gate_in"] is not None:
        out = out * torch.sigmoid(s["gate_in"].float())
    return dict(out=out.to(s["out_t"].dtype))


def _plain_shared(s):
    B, T, H, D, G = s["batch"], s["q_len"], s["nkv"], s["d"], s["nq"] // s["nkv"]
    q = s["q"].float().view(B, T, H, G, D)
    o = torch.empty((2, B, T, H, G, D), device="cuda")
    lse = torch.empty((2, B, T, H, G), device="cuda")
    for g, n in enumerate(s["prefixes"]):                               # the prefix, for all requests of a group at once
        b0, b1 = s["starts"][g], s["starts"][g + 1]
        used = s["shared_table"][g, : -(-n // s["page"])].long()
        k, v = (_tokens(s[x], used, n, s["scale8"]) for x in ("k", "v"))
        rows = q[b0:b1].permute(2, 3, 0, 1, 4).reshape(H, G, (b1 - b0) * T, D)
        part, log = _softmax_rows(rows, k, v, torch.full(((b1 - b0) * T,), n, device="cuda"))
        o[0, b0:b1] = part.view(H, G, b1 - b0, T, D).permute(2, 3, 0, 1, 4)
        lse[0, b0:b1] = log.view(H, G, b1 - b0, T).permute(2, 3, 0, 1)
    at = s["table"][:, : max(1, -(-max(s["lens"]) // s["page"]))].long().clamp(min=0)         # every request's own tokens
    raw = s["k"].dtype == torch.float8_e4m3fn

    def own_tokens(cache):
        x = cache.view(torch.uint8)[at].view(cache.dtype) if raw else cache[at]
        return (x.float() * s["scale8"]).flatten(1, 2).transpose(1, 2)

    score = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D), own_tokens(s["k"]).transpose(2, 3)) * (1.0 / math.sqrt(D))
    L = score.shape[-1]
    seen = s["kv_len"][:, None] - (T - 1 - torch.arange(T, device="cuda"))[None]
    shut = torch.arange(L, device="cuda")[None, None] >= seen[:, :, None]
    score = score.view(B, H, T, G, L).masked_fill(shut[:, None, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(-1, keepdim=True)
    part = torch.matmul(p.view(B, H, T * G, L), own_tokens(s["v"])).view(B, H, T, G, D)
    o[1] = (part / torch.where(total == 0, 1.0, total)).permute(0, 2, 1, 3, 4)
    lse[1] = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3)
    w = torch.exp(lse - lse.amax(0, keepdim=True))
    out = ((o * w[..., None]).sum(0) / w.sum(0)[..., None]).view(B * T, H * G, D)
    if s["gate_in"] is not None:
        out = out * torch.sigmoid(s["gate_in"].float())
    return dict(out=out.to(s["out_t"].dtype))


# ------------------------------------------------------------------------------------------------ this package

_space = {}                # the attention workspace, one for all calls of a program as for all layers of a model


def _workspace(need):
    if "ws" not in _space or _space["ws"].numel() < need:
        _space["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return _space["ws"]


def _own(s):
    import gated_deltanet_linear_16_gb300 as gdn
    if s["op"] == "norm":
        gdn.gdnb_residual_norm(s["x_in"], s["y_in"], s["x_out"], s["h_out"], gate=s["gate_in"], post=s["post_w"], pre=s["pre_w"],
                               rows=s["rows"], c=s["c"], scale=s["scale"], eps=1e-6,
                               gate_stride=s["c"] if s["gate"] == "rows" else 0)
        return dict(x=s["x_out"], h=s["h_out"])
    gate = dict(gate=s["gate_in"], gate_stride=2 * s["nq"] * s["d"], gate_head_stride=2 * s["d"]) if s["gate"] else {}
    heads = dict(nq=s["nq"], nkv=s["nkv"], d=s["d"])
    if s["op"] == "prompt":
        ws = _workspace(gdn.gdnb_attn_prompt_workspace(rows=s["rows"], batch=s["batch"], **heads))
        where = dict(token_stride=s["k"].stride(0)) if s["table"] is None else dict(
            table=s["table"], pages=s["pages"], page_size=s["page"], max_pages=s["max_pages"])
        gdn.gdnb_attn_prompt(s["q"], s["k"], s["v"], s["row_start"], s["kv_len"], s["out_t"], ws, rows=s["rows"],
                             batch=s["batch"], k_scale=s["scale8"], v_scale=s["scale8"], **heads, **where, **gate)
    else:
        ws = _workspace(gdn.gdnb_attn_shared_workspace(batch=s["batch"], groups=s["groups"], q_len=s["q_len"], **heads))
        gdn.gdnb_attn_shared(s["q"], s["k"], s["v"], s["shared_table"], s["shared_len"], s["table"], s["kv_len"], s["out_t"], ws,
                             group_start=s["group_start"], groups=s["groups"], batch=s["batch"], q_len=s["q_len"],
                             pages=s["pages"], page_size=s["page"], max_shared_pages=s["max_pages"], max_pages=s["max_pages"],
                             k_scale=s["scale8"], v_scale=s["scale8"], **heads, **gate)
    return dict(out=s["out_t"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "prompt": _plain_prompt, "shared": _plain_shared}[state["op"]](state)


# ------------------------------------------------------------------------------------------------ work, exact values

def work(case):
    if case["op"] == "norm":
        rows, c = case["rows"], case["c"]
        per = 2 * SIZE[case["x"]] + SIZE[case["y"]] * (2 if case["gate"] == "rows" else 1) + SIZE[case["h"]]
        return dict(bytes=rows * c * per + 4 * c * (2 if case["post"] else 1), flops=10 * rows * c)
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    if case["op"] == "prompt":
        fresh, cached = _prompt_lens(case)
        rows, keys = sum(fresh), sum(fresh) + sum(cached)
        pairs = sum(f * c + f * (f + 1) // 2 for f, c in zip(fresh, cached))
    else:
        prefix, start, lens = _shared_lens(case)
        T = case["q_len"]
        rows, keys = case["batch"] * T, sum(prefix) + sum(lens)
        pairs = sum(T * n * (start[g + 1] - start[g]) for g, n in enumerate(prefix))
        pairs += sum(max(0, n - (T - 1 - t)) for n in lens for t in range(T))
    per_row = nq * d * (SIZE[case["dtype"]] * (2 if case["gate"] else 1) + SIZE[_out(case)])
    return dict(bytes=2 * keys * nkv * d * SIZE[case["cache"]] + rows * per_row, flops=4 * pairs * nq * d)


def exact(case, seed):
    """What run() returns, in 64 bits: attention row block by row block over one list of keys for each sequence."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        y = s["y_in"].to(f64)
        if case["post"]:
            y = s["post_w"].to(f64) * y / (y.square().sum(-1, keepdim=True) / case["c"] + 1e-6).sqrt()
        if s["gate_in"] is not None:
            y *= s["gate_in"].to(f64)
        x = torch.add(s["x_in"].to(f64), y, alpha=case["scale"])
        return dict(x=x, h=s["pre_w"].to(f64) * x / (x.square().sum(-1, keepdim=True) / case["c"] + 1e-6).sqrt())
    if work(case)["flops"] > 2.5e12:
        return None
    H, D, G = case["nkv"], case["d"], case["nq"] // case["nkv"]
    out = torch.zeros((s["rows"], case["nq"], D), dtype=f64, device="cuda")

    def stored(cache, numbers, n):
        numbers = torch.tensor(numbers, device="cuda", dtype=torch.long)
        x = cache.view(torch.uint8)[numbers].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else cache[numbers]
        return x.reshape(-1, H, D)[:n].to(f64) * s["scale8"]

    def attend(row0, row1, keys, values, seen):
        """Rows [row0, row1), row r over the first seen(r) keys."""
        step = max(1, int(1.5e8 / max(1, keys.shape[0] * G)))
        for a in range(row0, row1, step):
            b = min(row1, a + step)
            limit = torch.tensor([seen(r) for r in range(a, b)], device="cuda")
            far = int(limit.max())
            if far <= 0:
                continue
            hidden = torch.arange(far, device="cuda")[None] >= limit[:, None]
            for h in range(H):
                score = s["q"][a:b, h * G:(h + 1) * G].to(f64).transpose(0, 1) @ keys[:far, h].T / math.sqrt(D)
                score.masked_fill_(hidden, -math.inf)
                out[a:b, h * G:(h + 1) * G] = (torch.softmax(score, -1).nan_to_num_(0.0) @ values[:far, h]).transpose(0, 1)

    if case["op"] == "prompt":
        for i, n in enumerate(s["lens"]):
            r0, r1 = s["starts"][i], s["starts"][i + 1]
            if s["table"] is None:
                k, v = s["k"][r0:r1].to(f64), s["v"][r0:r1].to(f64)
            else:
                numbers = s["table"][i].tolist()[: -(-n // s["page"])]
                k, v = stored(s["k"], numbers, n), stored(s["v"], numbers, n)
            attend(r0, r1, k, v, lambda r: n - (r1 - 1 - r))
    else:
        T = case["q_len"]
        for g, n in enumerate(s["prefixes"]):
            numbers = s["shared_table"][g].tolist()[: -(-n // s["page"])]
            k0, v0 = stored(s["k"], numbers, n), stored(s["v"], numbers, n)
            for i in range(s["starts"][g], s["starts"][g + 1]):
                m = s["lens"][i]
                mine = s["table"][i].tolist()[: -(-m // s["page"])]
                k, v = torch.cat([k0, stored(s["k"], mine, m)]), torch.cat([v0, stored(s["v"], mine, m)])
                attend(i * T, (i + 1) * T, k, v, lambda r: n + max(0, m - (T - 1 - (r - i * T))))
    if s["gate_in"] is not None:
        out *= torch.sigmoid(s["gate_in"].to(f64))
    return dict(out=out)
