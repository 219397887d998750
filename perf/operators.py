"""Cases of the attention-layer operators: cache pages, q/k norm + rotation + cache store, paged decode attention.

A hybrid model serves its gated-delta-rule layers with gdn_decode* and its softmax-attention layers with three
calls: gdna_page_assign (once a step: which cache page each new token goes to), gdna_qk_norm_rope (per layer: the
head norms, the rotary positions and the cache rows) and gdna_attn_decode (per layer: the new tokens' attention over
the paged cache).  A case names one of them ("op") and its sizes; listed() has fixed cases, draw() any of the same
ranges.  run() computes a case in plain torch operations, or, where `own` is true, with this package's calls.
"""
import math

import torch

own = False

F32, F16, BF16, F8 = "f32", "f16", "bf16", "e4m3"
TYPES = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16, F8: torch.float8_e4m3fn}
SIZE = {F32: 4, F16: 2, BF16: 2, F8: 1}
SCALE8 = 0.0625           # scale of an e4m3 cache: values to 28, where normalised keys and values stay
MOST_BYTES = 1.0e9        # largest drawn case


# ------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 256 running requests: one token each, a page taken by one request in sixteen
        dict(name="pages_decode", op="pages", batch=256, fresh=1, long_every=0, long=0, page=16, max_pages=1024),
        # a step that admits prompts: every eighth request brings up to 32768 tokens, the others decode
        dict(name="pages_prompts", op="pages", batch=200, fresh=1, long_every=8, long=32768, page=64, max_pages=1024),
        # one request, one token: fp32 projections with the output gate beside each query head, head size 256, a
        # quarter of it rotated (latency)
        dict(name="rope_one", op="rope", rows=1, nq=24, nkv=4, d=256, rot=64, inter=False, norm=True, gated=True,
             dtype=F32, cache=BF16, page=16, spare=512),
        # 256 decoding requests, head size 128 rotated whole, interleaved pairs
        dict(name="rope_decode", op="rope", rows=256, nq=48, nkv=8, d=128, rot=128, inter=True, norm=True, gated=False,
             dtype=BF16, cache=F16, page=16, spare=4096),
        # 32 requests with two tokens to verify, 8-bit cache
        dict(name="rope_verify_e4m3", op="rope", rows=64, nq=16, nkv=2, d=256, rot=64, inter=False, norm=True, gated=True,
             dtype=BF16, cache=F8, page=16, spare=2048),
        # a prefill of 8 prompts of 4096 tokens
        dict(name="rope_prefill", op="rope", rows=32768, nq=24, nkv=4, d=256, rot=64, inter=False, norm=True, gated=False,
             dtype=F32, cache=BF16, page=64, spare=0),
        # one request early in its answer (latency); gate fused
        dict(name="attn_one_short", op="attn", batch=1, q_len=1, nq=24, nkv=4, d=256, low=500, high=500, empty=0,
             page=16, dtype=F32, cache=BF16, out=BF16, gate=True),
        # one request at the end of a 262144-token context
        dict(name="attn_one_long", op="attn", batch=1, q_len=1, nq=24, nkv=4, d=256, low=262144, high=262144, empty=0,
             page=64, dtype=BF16, cache=BF16, out=BF16, gate=True),
        # 32 running requests of mixed lengths
        dict(name="attn_batch", op="attn", batch=32, q_len=1, nq=48, nkv=8, d=128, low=500, high=16000, empty=0,
             page=16, dtype=BF16, cache=BF16, out=BF16, gate=False),
        # the verify step that goes with the two-token state update: 2 tokens of 32 requests
        dict(name="attn_verify", op="attn", batch=32, q_len=2, nq=24, nkv=4, d=256, low=1000, high=6000, empty=0,
             page=16, dtype=F16, cache=F16, out=F16, gate=True),
        # 256 requests over an 8-bit cache
        dict(name="attn_many_e4m3", op="attn", batch=256, q_len=1, nq=32, nkv=4, d=128, low=200, high=8192, empty=0,
             page=32, dtype=BF16, cache=F8, out=BF16, gate=False),
        # odd everything: pages of 24, head size 64, three tokens, some requests without a key, fp32 results
        dict(name="attn_odd", op="attn", batch=37, q_len=3, nq=20, nkv=5, d=64, low=1, high=1999, empty=5,
             page=24, dtype=F32, cache=F16, out=F32, gate=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["pages", "rope", "rope", "attn", "attn", "attn"])
    page = rng.choice([8, 16, 24, 32, 64, 100])
    if op == "pages":
        batch = _log(rng, 1, 1024)
        long = rng.choice([0, _log(rng, 16, 32768)])
        every = rng.randint(2, 16) if long else 0
        if every:
            batch = min(batch, max(1, 2_000_000 * every // long))
        return dict(op=op, batch=batch, fresh=rng.choice([1, 1, 2, 5]), long_every=every, long=long, page=page,
                    max_pages=(65536 + page - 1) // page)
    d = rng.choice([64, 128, 128, 256, 256])
    nkv = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
    if nkv * group * d == 12 * 256:
        group += 1
    cache = rng.choice([BF16, BF16, F16, F8])
    if op == "rope":
        inter = rng.random() < 0.5
        rows = min(_log(rng, 1, 32768), int(MOST_BYTES / (10 * nkv * (group + 2) * d)))
        if cache == F8:
            rows = min(rows, 4_000_000 // (nkv * d) - 4 * page)
        return dict(op=op, rows=rows, nq=nkv * group, nkv=nkv, d=d, rot=rng.choice([d, d // 2, d // 4]), inter=inter,
                    norm=rng.random() < 0.8, gated=rng.random() < 0.4, dtype=rng.choice([F32, F16, BF16]), cache=cache,
                    page=page, spare=rng.choice([0, 2 * page]))
    batch = _log(rng, 1, 256)
    most = MOST_BYTES / (2 * nkv * d * SIZE[cache] * batch)
    high = max(4, min(262144 if batch < 4 else 16384, int(most)))
    high = _log(rng, min(high, 16), high)
    low = _log(rng, 1, high)
    dtype = rng.choice([F32, F16, BF16, BF16])
    return dict(op=op, batch=batch, q_len=rng.choice([1, 1, 1, 2, 3, 5, 8]), nq=nkv * group, nkv=nkv, d=d, low=low,
                high=high, empty=batch // 9 if rng.random() < 0.3 else 0, page=page, dtype=dtype, cache=cache,
                out=rng.choice([dtype, BF16]), gate=rng.random() < 0.5)


def _lens(case):
    """Cache lengths of an attention case: spread evenly over the logarithm of [low, high], out of order."""
    n, low, high = case["batch"], case["low"], case["high"]
    lens = [int(round(low * (high / low) ** ((0.5 + b * 0.6180339887) % 1.0))) if high > low else high for b in range(n)]
    lens[0] = high
    for i in range(case["empty"]):
        lens[(1 + 3 * i) % n if n > 1 else 0] = i % 2 * (case["q_len"] - 1)     # no key at all, or fewer than tokens
    return lens


def _fresh(case):
    """New tokens of each sequence of a pages case."""
    got = [case["fresh"]] * case["batch"]
    if case["long_every"]:
        for i, b in enumerate(range(0, case["batch"], case["long_every"])):
            got[b] = 1 + int(case["long"] * ((0.9 + i * 0.6180339887) % 1.0))
    return got


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    dev = "cuda"
    s = dict(case)
    i32 = dict(dtype=torch.int32, device=dev)
    if case["op"] == "pages":
        page, batch = case["page"], case["batch"]
        fresh = torch.tensor(_fresh(case))
        room = case["max_pages"] * page - fresh
        cached = (torch.rand(batch, generator=host) * room.clamp(max=4096)).long()
        have, want = (cached + page - 1) // page, (cached + fresh + page - 1) // page
        new = int((want - have).sum())
        ids = torch.randperm(int(want.sum()) + 64, generator=host)
        table = torch.full((batch, case["max_pages"]), -1, dtype=torch.int32)
        held = torch.arange(case["max_pages"])[None] < have[:, None]
        table[held] = ids[: int(have.sum())].to(torch.int32)
        rows = int(fresh.sum())
        s.update(cached=cached.to(**i32), fresh_n=fresh.to(**i32), table=table.to(dev), head=torch.tensor([32], **i32),
                 free=torch.cat([ids[-32:], ids[int(have.sum()):-32]]).to(**i32), rows=rows + -rows % 64,
                 kv_len=torch.empty(batch, **i32), row_start=torch.empty(batch + 1, **i32),
                 slots=torch.empty(rows + -rows % 64, dtype=torch.int64, device=dev),
                 positions=torch.empty(rows + -rows % 64, **i32), head_out=torch.empty(1, **i32),
                 unserved=torch.empty(1, **i32))
        assert new <= s["free"].numel() - 32
        return s
    nq, nkv, d, page = case["nq"], case["nkv"], case["d"], case["page"]
    s["scale8"] = SCALE8 if case["cache"] == F8 else 1.0
    if case["op"] == "rope":
        rows, rot, dt = case["rows"], case["rot"], case["dtype"]
        q = _rand(gen, (rows, nq, 2 * d if case["gated"] else d), dt)
        kv = _rand(gen, (rows, 2, nkv, d), dt)
        pages = (rows + case["spare"]) // page + 2
        n_pos = 8192
        angle = torch.arange(n_pos, device=dev, dtype=torch.float64)[:, None] * (
            1e6 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot))[None]
        s.update(q=q[:, :, :d], k=kv[:, 0], v=kv[:, 1], n_pos=n_pos, pages=pages, q_stride=q.stride(0),
                 q_head_stride=q.stride(1), kv_stride=kv.stride(0),
                 qn=1 + 0.1 * _rand(gen, (d,), F32) if case["norm"] else None,
                 kn=1 + 0.1 * _rand(gen, (d,), F32) if case["norm"] else None,
                 cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
                 positions=torch.randint(0, n_pos, (rows,), generator=host).to(**i32),
                 slots=torch.randperm(pages * page, generator=host)[:rows].to(dev),
                 q_out=torch.empty((rows, nq, d), dtype=TYPES[dt], device=dev),
                 k_cache=torch.zeros((pages, page, nkv, d), dtype=torch.uint8 if case["cache"] == F8 else TYPES[case["cache"]],
                                     device=dev).view(TYPES[case["cache"]]),
                 v_cache=torch.zeros((pages, page, nkv, d), dtype=torch.uint8 if case["cache"] == F8 else TYPES[case["cache"]],
                                     device=dev).view(TYPES[case["cache"]]))
        return s
    lens = torch.tensor(_lens(case))
    batch, q_len = case["batch"], case["q_len"]
    held = (lens + page - 1) // page
    pages, max_pages = int(held.sum()) + 3, int(held.max()) + 1
    table = torch.full((batch, max_pages), -1, dtype=torch.int32)
    table[torch.arange(max_pages)[None] < held[:, None]] = torch.randperm(pages, generator=host)[: int(held.sum())].to(torch.int32)
    q = _rand(gen, (batch * q_len, nq, 2 * d if case["gate"] else d), case["dtype"])
    s.update(q=q[:, :, :d].contiguous().mul_(1.5), gate_in=q[:, :, d:] if case["gate"] else None, lens=lens.to(**i32),
             table=table.to(dev), pages=pages, max_pages=max_pages,
             k_cache=_rand(gen, (pages, page, nkv, d), case["cache"], 1.0 / s["scale8"]),
             v_cache=_rand(gen, (pages, page, nkv, d), case["cache"], 1.0 / s["scale8"]),
             out_t=torch.empty((batch * q_len, nq, d), dtype=TYPES[case["out"]], device=dev),
             lse=torch.empty((batch * q_len, nq), dtype=torch.float32, device=dev))
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_pages(s):
    P, rows, batch, mp = s["page"], s["rows"], s["batch"], s["max_pages"]
    c, f = s["cached"].long(), s["fresh_n"].long()
    have, want = (c + P - 1) // P, (c + f + P - 1) // P
    fits = (f == 0) | (want <= mp)
    need = torch.where(fits, want - have, 0)
    ends, row_ends = need.cumsum(0), f.cumsum(0)
    head = s["head"].long()
    served = fits & ((need == 0) | (head + ends <= s["free"].numel())) & ((f == 0) | (row_ends <= rows))
    r = torch.arange(rows, device=c.device)
    seq = torch.searchsorted(row_ends, r, right=True)
    real = seq < batch
    seq = seq.clamp(max=batch - 1)
    pos = c[seq] + r - (row_ends - f)[seq]
    pg = pos // P
    given = s["free"][(head + (ends - need)[seq] + pg - have[seq]).clamp(0, s["free"].numel() - 1)].long()
    number = torch.where(pg < have[seq], s["table"][seq, pg.clamp(max=mp - 1)].long(), given)
    good = real & served[seq]
    flat = torch.cat([s["table"].reshape(-1), s["table"].new_zeros(1)])
    flat[torch.where(good, seq * mp + pg, batch * mp)] = number.to(torch.int32)
    start = torch.cat([row_ends.new_zeros(1), row_ends]).clamp(max=rows)
    return dict(table=flat[:-1].view(batch, mp), kv_len=torch.where(served, c + f, c).to(torch.int32),
                row_start=start.to(torch.int32), slots=torch.where(good, number * P + pos % P, -1),
                positions=torch.where(real, pos, 0).to(torch.int32),
                head=(head + torch.where(served & (need > 0), ends, 0).max()).to(torch.int32),
                unserved=(~served & (f > 0)).sum(0, keepdim=True).to(torch.int32))


def _rotate(x, cos, sin, rot, inter):
    turned, rest = x[..., :rot], x[..., rot:]
    if inter:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., : rot // 2], turned[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1)


def _store(cache, slots, x, scale):
    """Rows of x into the cache at their slots, rounded once to its type."""
    x = x / scale
    rows = cache.view(-1, *cache.shape[2:])
    if cache.dtype == torch.float8_e4m3fn:
        rows.view(torch.uint8)[slots] = x.clamp(-448.0, 448.0).to(cache.dtype).view(torch.uint8)
    else:
        rows[slots] = x.to(cache.dtype)


def _plain_rope(s):
    rot = s["rot"]
    at = s["cos_sin"][s["positions"].long()]
    cos, sin = at[:, None, : rot // 2], at[:, None, rot // 2:]

    def head(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        return _rotate(x, cos, sin, rot, s["inter"])

    q = head(s["q"], s["qn"]).to(s["q_out"].dtype)
    _store(s["k_cache"], s["slots"], head(s["k"], s["kn"]), s["scale8"])
    _store(s["v_cache"], s["slots"], s["v"].float(), s["scale8"])
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_attn(s):
    B, T, H, D, G = s["batch"], s["q_len"], s["nkv"], s["d"], s["nq"] // s["nkv"]
    at = s["table"].long().clamp(min=0)
    raw = s["k_cache"].dtype == torch.float8_e4m3fn

    def gather(cache):                                  # [B, H, L, D] in 32 bits
        x = cache.view(torch.uint8)[at].view(cache.dtype) if raw else cache[at]
        return (x.float() * s["scale8"]).flatten(1, 2).transpose(1, 2)

    q = s["q"].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    score = torch.matmul(q, gather(s["k_cache"]).transpose(2, 3)) * (1.0 / math.sqrt(D))
    L = score.shape[-1]
    seen = s["lens"][:, None] - (T - 1 - torch.arange(T, device=q.device))[None]            # keys of each token
    shut = torch.arange(L, device=q.device)[None, None] >= seen[:, :, None]                # [B, T, L]
    score = score.view(B, H, T, G, L).masked_fill(shut[:, None, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, T * G, L), gather(s["v_cache"])).view(B, H, T, G, D)
    o = o / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * T, H * G, D)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B * T, H * G)
    if s["gate_in"] is not None:
        o = o * torch.sigmoid(s["gate_in"].float())
    return dict(out=o.to(s["out_t"].dtype), lse=lse)


# ------------------------------------------------------------------------------------------------ this package

_space = {}                # the attention workspace, one for all calls of a program as for all layers of a model


def _workspace(gdn, s):
    need = gdn.gdna_attn_workspace(batch=s["batch"], q_len=s["q_len"], nq=s["nq"], nkv=s["nkv"], d=s["d"])
    if "ws" not in _space or _space["ws"].numel() < need:
        _space["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return _space["ws"]


def _own(s):
    import gated_deltanet_linear_16_gb300 as gdn
    if s["op"] == "pages":
        gdn.gdna_page_assign(s["cached"], s["fresh_n"], s["table"], s["free"], s["head"], s["kv_len"], s["row_start"],
                             s["slots"], s["positions"], s["head_out"], s["unserved"], batch=s["batch"], rows=s["rows"],
                             page_size=s["page"], max_pages=s["max_pages"])
        return dict(table=s["table"], kv_len=s["kv_len"], row_start=s["row_start"], slots=s["slots"],
                    positions=s["positions"], head=s["head_out"], unserved=s["unserved"])
    if s["op"] == "rope":
        gdn.gdna_qk_norm_rope(s["q"], s["k"], s["v"], s["qn"], s["kn"], s["cos_sin"], s["positions"], s["slots"],
                              s["q_out"], s["k_cache"], s["v_cache"], rows=s["rows"], nq=s["nq"], nkv=s["nkv"], d=s["d"],
                              rot=s["rot"], interleaved=s["inter"], n_pos=s["n_pos"], eps=1e-6, pages=s["pages"],
                              page_size=s["page"], k_scale=s["scale8"], v_scale=s["scale8"],
                              q_stride=s["q_stride"], q_head_stride=s["q_head_stride"], k_stride=s["kv_stride"],
                              v_stride=s["kv_stride"])
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    gdn.gdna_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out_t"], _workspace(gdn, s),
                         gate=s["gate_in"], lse=s["lse"], batch=s["batch"], q_len=s["q_len"], nq=s["nq"], nkv=s["nkv"],
                         d=s["d"], pages=s["pages"], page_size=s["page"], max_pages=s["max_pages"],
                         k_scale=s["scale8"], v_scale=s["scale8"], gate_stride=2 * s["nq"] * s["d"],
                         gate_head_stride=2 * s["d"])
    return dict(out=s["out_t"], lse=s["lse"])


def run(state):
    if own:
        return _own(state)
    return {"pages": _plain_pages, "rope": _plain_rope, "attn": _plain_attn}[state["op"]](state)


# ------------------------------------------------------------------------------------------------ work, exact values

def work(case):
    if case["op"] == "pages":
        rows, batch = sum(_fresh(case)), case["batch"]
        new = rows // case["page"]
        return dict(bytes=12 * (rows + -rows % 64) + 8 * new + 20 * batch, flops=0)
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    if case["op"] == "rope":
        rows, e, c = case["rows"], SIZE[case["dtype"]], SIZE[case["cache"]]
        per = 2 * nq * d * e + 2 * nkv * d * (e + c) + 12 + 4 * case["rot"]
        return dict(bytes=rows * per, flops=rows * (nq + nkv) * (4 * d + 3 * case["rot"]))
    T, lens = case["q_len"], _lens(case)
    rows = case["batch"] * T * nq
    keys = sum(lens)
    pairs = sum(max(0, n - (T - 1 - t)) for n in lens for t in range(T))
    e, c = SIZE[case["dtype"]], SIZE[case["cache"]]
    return dict(bytes=2 * keys * nkv * d * c + rows * d * (e * (2 if case["gate"] else 1) + SIZE[case["out"]]) + 4 * rows,
                flops=4 * pairs * nq * d)


def exact(case, seed):
    """What run() returns, in 64 bits: rotations as complex products, attention one sequence after the other."""
    if case["op"] == "pages":
        return None                                     # whole numbers only
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "rope":
        rot, half = s["rot"], s["rot"] // 2
        cs = s["cos_sin"].to(f64)[s["positions"].long()]
        turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]

        def head(x, w):
            x = x.to(f64)
            if w is not None:
                x = x / ((x ** 2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.to(f64)
            a = x[..., :rot].unflatten(-1, (half, 2) if s["inter"] else (2, half))
            z = torch.complex(*(a.unbind(-1) if s["inter"] else a.unbind(-2))) * turn
            x[..., :rot] = torch.stack([z.real, z.imag], -1 if s["inter"] else -2).flatten(-2)
            return x

        def stored(cache, x):
            full = torch.zeros(cache.shape, dtype=f64, device=cache.device)
            full.view(-1, *cache.shape[2:]).index_copy_(0, s["slots"], x / s["scale8"])
            return full

        return dict(q=head(s["q"].clone(), s["qn"]), k_cache=stored(s["k_cache"], head(s["k"].clone(), s["kn"])),
                    v_cache=stored(s["v_cache"], s["v"].to(f64)))
    T, H, D = case["q_len"], case["nkv"], case["d"]
    G, scale8 = case["nq"] // H, s["scale8"]
    out = torch.zeros((case["batch"] * T, H * G, D), dtype=f64, device="cuda")
    lse = torch.full((case["batch"] * T, H * G), float("-inf"), dtype=f64, device="cuda")
    table = s["table"].tolist()
    for b, n in enumerate(_lens(case)):
        used = table[b][: -(-n // case["page"])]
        if not used:
            continue
        used = torch.tensor(used, device="cuda")
        raw = [c.view(torch.uint8)[used].view(c.dtype) if c.dtype == torch.float8_e4m3fn else c[used]
               for c in (s["k_cache"], s["v_cache"])]
        k, v = (x.flatten(0, 1)[:n].to(f64) * scale8 for x in raw)
        for t in range(T):
            m = n - (T - 1 - t)
            if m <= 0:
                continue
            q = s["q"][b * T + t].to(f64).view(H, G, D)
            score = torch.einsum("hgd,nhd->hgn", q, k[:m]) / math.sqrt(D)
            total = score.logsumexp(-1)
            w = (score - total[..., None]).exp()
            out[b * T + t] = torch.einsum("hgn,nhd->hgd", w, v[:m]).reshape(H * G, D)
            lse[b * T + t] = total.reshape(-1)
    if s["gate_in"] is not None:
        out = out / (1.0 + (-s["gate_in"].to(f64)).exp())
    return dict(out=out, lse=lse)
