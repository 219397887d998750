"""64-bit references and calls for the tests of the prompt and shared-prefix attention.

Bounds, with e = 2^-24, S the largest sum |q_i k_i| * scale of a row and vmax the largest |v| it sees.  A score is a sum of D
exact products in fp32 (8 sqrt(D) e S, as independent roundings; tcgen05 adds 16 at a time and cuts instead of rounding,
D / 16 cuts of 2 e S at most, which is less), of queries that hold 16 bits (fp32 over a bf16 cache: 2^-16 S), 22 (fp32 over the
others: 2^-22 S; 11 with a bf16 output: 2^-11 S) or all of theirs; its own error and its maximum's enter a weight.  A weight enters its product rounded
once, to 2^-8 (bf16) or 2^-11 (fp16, or 2^-32 of the largest, which n keys make n 2^-32) of itself; the sum of weights is of unrounded ones,
so all of that scales vmax.  Sums over n keys add 8 sqrt(n) e, the exponentials and rescales 32 e more.  The output's type adds
half a unit in its last place, the gate a few e of the output."""
import numpy as np
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.attn_layers_helpers import E32, HALF_STEP0, HALF_ULP, NOWHERE, TYPES, Cache, f64, guarded, intact


def attention_rows(q, keys, values, seen, scale):
    """q [n, nq, d] and the sequence's keys and values [len, nkv, d], 64-bit torch tensors on the GPU; row r sees the first
    seen[r] keys.  Returns out, S and vmax [n, nq, .]."""
    n, nq, d = q.shape
    out = torch.zeros((n, nq, d), dtype=torch.float64, device=q.device)
    size, vmax = (torch.zeros((n, nq, 1), dtype=torch.float64, device=q.device) for _ in range(2))
    length = keys.shape[0]
    if length == 0:
        return out, size, vmax
    g = nq // keys.shape[1]
    hidden = torch.arange(length, device=q.device)[None] >= torch.as_tensor(seen, device=q.device)[:, None]
    for h in range(nq):
        k, v = keys[:, h // g], values[:, h // g]
        s = (q[:, h] @ k.T * scale).masked_fill(hidden, -torch.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(top == -torch.inf, 0.0, top)).masked_fill(hidden, 0.0)
        total = p.sum(-1, keepdim=True)
        out[:, h] = p @ v / torch.where(total == 0, 1.0, total)
        size[:, h, 0] = (q[:, h].abs() @ k.abs().T * scale).masked_fill(hidden, 0.0).amax(-1)
        vmax[:, h, 0] = v.abs().amax(-1)[None].expand(n, -1).masked_fill(hidden, 0.0).amax(-1)
    return out, size, vmax


def tolerance(want, size, vmax, n, d, dtype, cache, out_type):
    part_q = 0.0 if dtype != "f32" else 2.0 ** -16 if cache == "bf16" else 2.0 ** -11 if out_type == "bf16" else 2.0 ** -22
    score = (8 * np.sqrt(d) * E32 + part_q) * size
    part = 2.0 ** -8 if cache == "bf16" else 2.0 ** -11 + n * 2.0 ** -32
    return (vmax * (2 * score + part + (8 * np.sqrt(max(n, 1)) + 32) * E32) * 1.01 + HALF_ULP[out_type] * 1.001 * want.abs()
            + HALF_STEP0[out_type] + 8 * E32 * want.abs())


def rand(gen, *shape):
    return torch.randn(shape, generator=gen)


class Pages:
    """A paged cache with sequences of given lengths in pages of any order: NaN where no token lives."""

    def __init__(self, lens, nkv, d, kind, page, layout="tokens", shift=0, scale=1.0, spare=2, gen=None):
        self.gen = gen or torch.Generator().manual_seed(0)
        held = [-(-max(n, 0) // page) for n in lens]
        self.lens, self.scale = lens, scale
        self.pages, self.max_pages = sum(held) + spare, max(held + [0]) + 2
        self.store = Cache(self.pages, page, nkv, d, kind, layout, shift)
        ids = torch.randperm(self.pages, generator=self.gen).tolist()
        self.table = torch.full((len(lens), self.max_pages + 3), NOWHERE, dtype=torch.int32)
        self.keys, self.values, self.where = [], [], []
        for b, n in enumerate(lens):
            n = max(n, 0)
            mine, ids = ids[:held[b]], ids[held[b]:]
            self.table[b, :held[b]] = torch.tensor(mine, dtype=torch.int32)
            j = torch.arange(n)
            at = torch.tensor(mine, dtype=torch.long)[j // page] if n else torch.zeros(0, dtype=torch.long)
            self.where.append((at, j % page))
            for which, kept in (("k", self.keys), ("v", self.values)):
                x = self.store.put(which, at, j % page, rand(self.gen, n, nkv, d) / scale) if n else np.zeros((0, nkv, d))
                kept.append(torch.tensor(x * scale, device="cuda"))
        self.table = self.table.cuda()


def starts_of(fresh, first=0):
    return [first] + [first + int(x) for x in np.cumsum(fresh)]


def make_prompt(fresh, cached, nq, nkv, d, dtype="bf16", cache="bf16", page=16, layout="tokens", shift=0, seed=0, peaked=1.0,
                scale8=1.0, pad=0, first=0, behind=3, dense=False):
    """Sequences of fresh[b] new and cached[b] old tokens; `first` rows before the first sequence, `behind` after the last."""
    gen = torch.Generator().manual_seed(seed)
    lens = [f + c for f, c in zip(fresh, cached)]
    starts = starts_of(fresh, first)
    rows = starts[-1] + behind
    s = dict(fresh=fresh, lens=lens, starts=starts, rows=rows, nq=nq, nkv=nkv, d=d, dtype=dtype, cache=cache, scale8=scale8,
             gen=gen, scale=d ** -0.5, dense=dense)
    if dense:
        kv = torch.full((rows, 2, nkv, d + 8), float("nan"))
        for b in range(len(fresh)):
            kv[starts[b]:starts[b + 1], :, :, :d] = rand(gen, fresh[b], 2, nkv, d)
        s["kv"] = kv.to(TYPES[cache]).cuda()
        s["keys"] = [s["kv"][starts[b]:starts[b + 1], 0, :, :d].double() for b in range(len(fresh))]
        s["values"] = [s["kv"][starts[b]:starts[b + 1], 1, :, :d].double() for b in range(len(fresh))]
    else:
        s["pages"] = Pages(lens, nkv, d, cache, page, layout, shift, scale8, gen=gen)
        s["keys"], s["values"] = s["pages"].keys, s["pages"].values
    s["q"] = (rand(gen, rows, nq * d + pad) * peaked).to(TYPES[dtype]).cuda()
    return s


def call_prompt(s, out, gate=None, gate_strides=(None, None), ws=None, stream=None, **kw):
    need = gdn.gdnb_attn_prompt_workspace(rows=s["rows"], batch=len(s["fresh"]), nq=s["nq"], nkv=s["nkv"], d=s["d"])
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws          # NaN everywhere
    i32 = dict(dtype=torch.int32, device="cuda")
    start, lens = torch.tensor(s["starts"], **i32), torch.tensor(s["lens"], **i32)
    torch.cuda.synchronize()
    a = dict(rows=s["rows"], batch=len(s["fresh"]), nq=s["nq"], nkv=s["nkv"], d=s["d"], scale=s["scale"], k_scale=s["scale8"],
             v_scale=s["scale8"], q_stride=s["q"].stride(0), out_stride=out.stride(0), gate=gate, gate_stride=gate_strides[0],
             gate_head_stride=gate_strides[1], stream=stream)
    if s["dense"]:
        k, v, lens = s["kv"][:, 0], s["kv"][:, 1], None
        a.update(token_stride=s["kv"].stride(0), head_stride=s["kv"].stride(2))
    else:
        pages = s["pages"]
        k, v = pages.store.addresses()
        a.update(table=pages.table, table_stride=pages.table.stride(0), max_pages=pages.max_pages, **pages.store.args())
    a.update(kw)
    gdn.gdnb_attn_prompt(s["q"], k, v, start, lens, out, ws, **a)


def prompt64(s):
    """out, S and vmax of all rows in 64 bits (rows of no sequence: 0)."""
    q = s["q"][:, :s["nq"] * s["d"]].double().view(s["rows"], s["nq"], s["d"])
    parts = [torch.zeros((s["rows"], s["nq"], w), dtype=torch.float64, device="cuda") for w in (s["d"], 1, 1)]
    for b, n in enumerate(s["lens"]):
        r0, r1 = s["starts"][b], s["starts"][b + 1]
        if r1 > r0:
            got = attention_rows(q[r0:r1], s["keys"][b], s["values"][b], n - (r1 - r0) + 1 + torch.arange(r1 - r0), s["scale"])
            for x, y in zip(parts, got):
                x[r0:r1] = y
    return parts


def gate_of(s, gated):
    if not gated:
        return None, None, (None, None)
    big = rand(s["gen"], s["rows"], s["nq"], 2 * s["d"] + gated).to(TYPES[s["dtype"]]).cuda()
    return big[:, :, s["d"]:], big[:, :, s["d"]:2 * s["d"]].double(), (big.stride(0), big.stride(1))


def check_prompt(s, out_type="bf16", gated=0, pad=5, finite=True, **kw):
    rows, nq, d = s["rows"], s["nq"], s["d"]
    whole, out = guarded(rows, nq * d, nq * d + pad, out_type, before=8 if pad % 8 == 0 else 5)
    gate, gate64, strides = gate_of(s, gated)
    before = gdn.gdn_device_wait_timeouts()
    call_prompt(s, out, gate, strides, **kw)
    torch.cuda.synchronize()
    assert gdn.gdn_device_wait_timeouts() == before
    want, size, vmax = prompt64(s)
    tol = tolerance(want, size, vmax, max(s["lens"] + [1]), d, s["dtype"], s["cache"], out_type)
    if gate64 is not None:
        want, tol = want * torch.sigmoid(gate64), tol + HALF_ULP[out_type] * want.abs()
    got = out.double().view(rows, nq, d)
    lo, hi = s["starts"][0], s["starts"][-1]
    assert (got[:lo] == 77).all() and (got[hi:] == 77).all()
    miss = ((got - want).abs() - tol)[lo:hi]
    if finite:
        assert torch.isfinite(got[lo:hi]).all(), torch.nonzero(~torch.isfinite(got[lo:hi]))[:8]
        assert (miss <= 0).all(), (float(miss.max()), torch.nonzero(miss > 0)[:8], float((miss > 0).double().mean()))
    assert intact(whole, out)
    return got, want, tol
