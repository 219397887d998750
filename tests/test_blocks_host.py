"""Checks of the decoder-block entry points that need no GPU: what they refuse, empty calls, the workspaces' sizes, header
and exports, and the binding's checks of types."""
import os
import re
import subprocess

import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdnb.h")
OK, ARG, UNSUP, ALIGN, ALIAS = 0, 1, 2, 3, 4
G = 1 << 34
A = [G * (i + 1) for i in range(20)]        # fake, far apart addresses: never dereferenced by a rejected call
NAMES = ["gdnb_attn_prompt", "gdnb_attn_prompt_workspace", "gdnb_attn_shared", "gdnb_attn_shared_workspace", "gdnb_residual_norm"]


@pytest.fixture(scope="module")
def built():
    gdn.build()
    return gdn.load()


@pytest.fixture(scope="module")
def lib(built):
    if torch.cuda.is_available():
        pytest.skip("fake-pointer validation tests run only on hosts without a GPU")
    return built


def test_header_and_exports_agree(built):
    assert sorted(set(re.findall(r"GDN_API\s+[\w\s\*]*?\b(gdnb_\w+)\s*\(", open(HEADER).read()))) == NAMES
    out = subprocess.run(["nm", "-D", "--defined-only", gdn.library_path()], capture_output=True, text=True, check=True).stdout
    assert sorted({x.split()[-1] for x in out.splitlines() if x.split()[-1].startswith("gdnb_")}) == NAMES
    for name in NAMES:
        assert name in gdn.__all__ and hasattr(gdn, name)


def test_the_header_is_plain_c(built, tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "gdnb.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER), str(src)], check=True)


def norm(lib, **kw):
    a = dict(x=A[0], xd=0, y=A[1], yd=2, gate=A[2], post=A[3], pre=A[4], scale=1.0, eps=1e-6, xo=A[5], h=A[6], hd=2, rows=8, c=512,
             xs=512, ys=512, gs=512, xos=512, hs=512)
    a.update(kw)
    return lib.gdnb_residual_norm(*[a[k] for k in ("x", "xd", "y", "yd", "gate", "post", "pre", "scale", "eps", "xo", "h", "hd", "rows",
                                                   "c", "xs", "ys", "gs", "xos", "hs")], None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), ARG), (dict(c=0), ARG), (dict(c=-4), ARG), (dict(c=16385), UNSUP), (dict(xd=3), UNSUP), (dict(yd=3), UNSUP),
    (dict(hd=3), UNSUP), (dict(xd=9), UNSUP), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(x=None), ARG), (dict(xo=None, h=None), ARG), (dict(y=None), ARG), (dict(y=None, gate=None), ARG), (dict(gs=-1), ARG),
    (dict(xs=511), ARG), (dict(ys=511), ARG), (dict(gs=100), ARG), (dict(xos=5), ARG), (dict(hs=511), ARG),
    (dict(x=A[0] + 2), ALIGN), (dict(y=A[1] + 1), ALIGN), (dict(pre=A[4] + 2), ALIGN), (dict(h=A[6] + 1), ALIGN),
    (dict(xo=A[0], xos=520, xs=512), ALIAS), (dict(xo=A[0] + 16), ALIAS), (dict(h=A[0]), ALIAS), (dict(h=A[1], hd=0), ALIAS),
    (dict(h=A[2]), ALIAS), (dict(xo=A[1]), ALIAS), (dict(xo=A[3]), ALIAS), (dict(h=A[5]), ALIAS), (dict(h=A[1], hs=600), ALIAS),
    (dict(rows=1 << 62), ARG), (dict(rows=0), OK), (dict(rows=0, x=None), OK)])
def test_residual_norm_refuses(lib, kw, want):
    assert norm(lib, **kw) == want


def prompt(lib, **kw):
    a = dict(q=A[0], dtype=2, gate=A[1], k=A[2], v=A[3], cdt=2, ks=1.0, vs=1.0, table=A[4], tstride=8, start=A[5], kv=A[6], scale=0.1,
             out=A[7], odt=2, ws=A[8], wsb=1 << 33, rows=30, batch=3, nq=8, nkv=2, d=128, pages=10, page=16, max_pages=8, qs=1024, gs=1024,
             ghs=128, os=1024, ps=4096, ts=256, hs=128)
    a.update(kw)
    return lib.gdnb_attn_prompt(*[a[k] for k in ("q", "dtype", "gate", "k", "v", "cdt", "ks", "vs", "table", "tstride", "start", "kv", "scale",
                                                 "out", "odt", "ws", "wsb", "rows", "batch", "nq", "nkv", "d", "pages", "page", "max_pages",
                                                 "qs", "gs", "ghs", "os", "ps", "ts", "hs")], None)


COMMON = [
    (dict(batch=-1), ARG), (dict(nq=0), ARG), (dict(nkv=0), ARG), (dict(d=0), ARG), (dict(max_pages=0), ARG), (dict(nq=9), UNSUP),
    (dict(nq=258, qs=1 << 20, os=1 << 20, gs=1 << 20), UNSUP), (dict(d=257), UNSUP), (dict(dtype=3), UNSUP), (dict(odt=0), UNSUP),
    (dict(odt=3), UNSUP), (dict(cdt=0), UNSUP), (dict(cdt=4), UNSUP), (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(ks=-1.0), ARG), (dict(vs=float("inf")), ARG), (dict(ks=1e-30, scale=1e-30), ARG), (dict(q=None), ARG), (dict(k=None), ARG),
    (dict(v=None), ARG), (dict(kv=None), ARG), (dict(out=None), ARG), (dict(ws=None), ARG), (dict(wsb=100), ARG), (dict(ghs=127), ARG),
    (dict(qs=1000), ARG), (dict(os=1000), ARG), (dict(gs=500), ARG), (dict(tstride=7), ARG), (dict(pages=0), ARG), (dict(page=0), ARG),
    (dict(ps=100), ARG), (dict(ts=127), ARG), (dict(hs=127), ARG), (dict(pages=1 << 31), UNSUP), (dict(q=A[0] + 1), ALIGN),
    (dict(k=A[2] + 1), ALIGN), (dict(ws=A[8] + 8), ALIGN), (dict(table=A[4] + 2), ALIGN), (dict(out=A[0]), ALIAS), (dict(out=A[1] + 64), ALIAS),
    (dict(out=A[2]), ALIAS), (dict(ws=A[2]), ALIAS), (dict(ws=A[0]), ALIAS), (dict(out=A[8] + 256), ALIAS), (dict(batch=0), OK)]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(rows=-1), ARG), (dict(rows=1 << 31), UNSUP), (dict(batch=65537), UNSUP), (dict(start=None), ARG), (dict(start=A[5] + 1), ALIGN),
    (dict(out=A[5]), ALIAS), (dict(table=None, cdt=3), UNSUP), (dict(table=None, ts=255), ARG), (dict(table=None, hs=100), ARG),
    (dict(table=None, k=None), ARG), (dict(table=None, kv=None, ts=200), ARG), (dict(table=None, out=A[3]), ALIAS), (dict(rows=0), OK)])
def test_attn_prompt_refuses(lib, kw, want):
    assert prompt(lib, **kw) == want


def shared(lib, **kw):
    a = dict(q=A[0], dtype=2, gate=A[1], k=A[2], v=A[3], cdt=2, ks=1.0, vs=1.0, gstart=A[9], groups=2, stable=A[10], sstride=8, slen=A[11],
             table=A[4], tstride=8, kv=A[6], scale=0.1, out=A[7], odt=2, ws=A[8], wsb=1 << 33, batch=3, q_len=2, nq=8, nkv=2, d=128, pages=10,
             page=16, max_shared=8, max_pages=8, qs=1024, gs=1024, ghs=128, os=1024, ps=4096, ts=256, hs=128)
    a.update(kw)
    return lib.gdnb_attn_shared(*[a[k] for k in ("q", "dtype", "gate", "k", "v", "cdt", "ks", "vs", "gstart", "groups", "stable", "sstride", "slen",
                                                 "table", "tstride", "kv", "scale", "out", "odt", "ws", "wsb", "batch", "q_len", "nq", "nkv",
                                                 "d", "pages", "page", "max_shared", "max_pages", "qs", "gs", "ghs", "os", "ps", "ts", "hs")], None)


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(q_len=-1), ARG), (dict(groups=0), ARG), (dict(gstart=None), ARG), (dict(groups=65537, sstride=8), UNSUP), (dict(max_shared=0), ARG),
    (dict(stable=None), ARG), (dict(slen=None), ARG), (dict(sstride=7), ARG), (dict(batch=(1 << 20) + 1), UNSUP), (dict(q_len=1 << 22), UNSUP),
    (dict(table=None), ARG), (dict(out=A[10]), ALIAS), (dict(ws=A[11]), ALIAS), (dict(q_len=0), OK)])
def test_attn_shared_refuses(lib, kw, want):
    assert shared(lib, **kw) == want


def test_workspaces(built):
    p = lambda **kw: gdn.gdnb_attn_prompt_workspace(**dict(dict(rows=100, batch=3, nq=8, nkv=2, d=128), **kw))      # noqa: E731
    s = lambda **kw: gdn.gdnb_attn_shared_workspace(**dict(dict(batch=3, groups=1, q_len=1, nq=8, nkv=2, d=128), **kw))   # noqa: E731
    assert 0 < p() <= p(rows=10 ** 6, batch=60) < 1 << 28 and p(rows=10 ** 9, batch=65536) < 1 << 28
    assert p(nq=9) == p(d=257) == p(rows=1 << 31) == p(batch=65537) == p(nq=258) == p(rows=-1) == p(nkv=0) == 0
    assert 0 < s() <= s(batch=50, groups=4, q_len=2)
    assert s(nq=9) == s(d=0) == s(groups=0) == s(groups=65537) == s(batch=1 << 21) == s(q_len=-1) == 0


def test_the_binding_checks_types(built):
    f, b, i = torch.zeros(64), torch.zeros(64, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdnb_residual_norm(f, b, b, b, rows=1, c=64, stream=0)                     # x_out of another type than x
    with pytest.raises(ValueError):
        gdn.gdnb_residual_norm(f, b, f, b, pre=b, rows=1, c=64, stream=0)
    with pytest.raises(ValueError):
        gdn.gdnb_residual_norm(f, b, f, b, gate=f, rows=1, c=64, stream=0)
    heads = dict(nq=1, nkv=1, d=64, batch=1, stream=0)
    with pytest.raises(ValueError):
        gdn.gdnb_attn_prompt(b, b, f, i, i, b, b, rows=1, table=i, **heads)
    with pytest.raises(ValueError):
        gdn.gdnb_attn_prompt(b, b, b, i.long(), i, b, b, rows=1, table=i, **heads)
    with pytest.raises(ValueError):
        gdn.gdnb_attn_prompt(b, b, b, i, i, b, b, rows=1, table=i, gate=f, **heads)
    with pytest.raises(ValueError):
        gdn.gdnb_attn_shared(b, b, b, i, i.float(), i, i, b, b, pages=1, page_size=1, max_shared_pages=1, max_pages=1, **heads)
