"""Checks of the attention-layer entry points that need no GPU: what they refuse, the workspace's size, and the
host's table of cosines and sines against its definition in extended precision."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdna.h")
OK, ARG, UNSUP, ALIGN, ALIAS = 0, 1, 2, 3, 4
G = 1 << 32
A = [G * (i + 1) for i in range(20)]        # fake, far apart addresses: never dereferenced by a rejected call


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
    want = sorted(set(re.findall(r"GDN_API\s+[\w\s\*]*?\b(gdna_\w+)\s*\(", open(HEADER).read())))
    assert want == ["gdna_attn_decode", "gdna_attn_workspace", "gdna_page_assign", "gdna_qk_norm_rope", "gdna_rope_table"]
    out = subprocess.run(["nm", "-D", "--defined-only", gdn.library_path()], capture_output=True, text=True,
                         check=True).stdout
    assert sorted({x.split()[-1] for x in out.splitlines() if x.split()[-1].startswith("gdna_")}) == want
    for name in want:
        assert name in gdn.__all__ and hasattr(gdn, name)


def test_the_headers_are_plain_c(built, tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "gdna.h"\nint main(void) { return (int)sizeof(gdna_dtype) - (int)sizeof(int); }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER), str(src)], check=True)


def pages(lib, **kw):
    a = dict(cached=A[0], fresh=A[1], table=A[2], stride=8, free=A[3], n_free=100, head=A[4], kv=A[5], start=A[6],
             slots=A[7], pos=A[8], head_out=A[9], unserved=A[10], batch=4, rows=16, page=16, max_pages=8)
    a.update(kw)
    return lib.gdna_page_assign(a["cached"], a["fresh"], a["table"], a["stride"], a["free"], a["n_free"], a["head"],
                                a["kv"], a["start"], a["slots"], a["pos"], a["head_out"], a["unserved"], a["batch"],
                                a["rows"], a["page"], a["max_pages"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), ARG), (dict(rows=-1), ARG), (dict(page=0), ARG), (dict(max_pages=0), ARG), (dict(n_free=-1), ARG),
    (dict(batch=(1 << 20) + 1), UNSUP), (dict(rows=1 << 31), UNSUP), (dict(n_free=1 << 31), UNSUP),
    (dict(cached=None), ARG), (dict(fresh=None), ARG), (dict(table=None), ARG), (dict(free=None), ARG),
    (dict(head=None), ARG), (dict(kv=None), ARG), (dict(start=None), ARG), (dict(slots=None), ARG), (dict(pos=None), ARG),
    (dict(head_out=None), ARG), (dict(unserved=None), ARG), (dict(stride=7), ARG),
    (dict(table=A[2] + 2), ALIGN), (dict(slots=A[7] + 4), ALIGN),
    (dict(kv=A[0]), ALIAS), (dict(head_out=A[4]), ALIAS), (dict(start=A[5] + 12), ALIAS), (dict(slots=A[2] + 64), ALIAS),
    (dict(unserved=A[3] + 396), ALIAS), (dict(batch=0), OK), (dict(batch=0, cached=None), OK)])
def test_page_assign_refuses(lib, kw, want):
    assert pages(lib, **kw) == want


def rope(lib, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], dtype=0, qn=A[3], kn=A[4], eps=1e-6, cs=A[5], n_pos=100, rot=64, inter=0, pos=A[6],
             slots=A[7], qo=A[8], ko=A[9], kc=A[10], vc=A[11], cdt=2, ks=1.0, vs=1.0, rows=8, nq=4, nkv=2, d=128,
             pages=10, page=16, qs=512, qhs=128, kst=256, vst=256, qos=512, kos=256, ps=4096, ts=256, hs=128)
    a.update(kw)
    return lib.gdna_qk_norm_rope(a["q"], a["k"], a["v"], a["dtype"], a["qn"], a["kn"], a["eps"], a["cs"], a["n_pos"],
                                 a["rot"], a["inter"], a["pos"], a["slots"], a["qo"], a["ko"], a["kc"], a["vc"], a["cdt"],
                                 a["ks"], a["vs"], a["rows"], a["nq"], a["nkv"], a["d"], a["pages"], a["page"], a["qs"],
                                 a["qhs"], a["kst"], a["vst"], a["qos"], a["kos"], a["ps"], a["ts"], a["hs"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), ARG), (dict(nq=-1), ARG), (dict(nkv=-1), ARG), (dict(nq=0, nkv=0), ARG), (dict(d=0), ARG),
    (dict(d=257), UNSUP), (dict(dtype=3), UNSUP), (dict(dtype=9), UNSUP), (dict(cdt=0), UNSUP), (dict(cdt=7), UNSUP),
    (dict(rot=63), ARG), (dict(rot=130), ARG), (dict(rot=-2), ARG), (dict(n_pos=0), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(ks=0.0), ARG), (dict(vs=float("inf")), ARG), (dict(ks=-1.0), ARG), (dict(vs=float("nan")), ARG),
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(vc=None), ARG), (dict(cs=None), ARG),
    (dict(pos=None), ARG), (dict(slots=None), ARG), (dict(qo=None), ARG), (dict(kc=None, vc=None, v=None, ko=None), ARG),
    (dict(nkv=0, k=None, v=None, vc=None), ARG),                    # a cache and no keys
    (dict(qs=511), ARG), (dict(qhs=127), ARG), (dict(kst=255), ARG), (dict(vst=1), ARG), (dict(qos=511), ARG),
    (dict(kos=255), ARG), (dict(pages=0), ARG), (dict(page=0), ARG), (dict(pages=1 << 31), UNSUP),
    (dict(ps=4095), ARG), (dict(ts=255), ARG), (dict(hs=127), ARG), (dict(ts=-256), ARG), (dict(ts=128, hs=128), ARG),
    (dict(q=A[0] + 2), ALIGN), (dict(kc=A[10] + 1), ALIGN), (dict(slots=A[7] + 4), ALIGN), (dict(cs=A[5] + 1), ALIGN),
    (dict(qo=A[0] + 16), ALIAS), (dict(qo=A[1]), ALIAS), (dict(ko=A[1]), ALIAS), (dict(kc=A[2]), ALIAS),
    (dict(vc=A[10]), ALIAS), (dict(vc=A[10] + 64), ALIAS), (dict(qo=A[0], qhs=256, qs=1024), ALIAS),
    (dict(qo=A[3]), ALIAS), (dict(ko=A[10]), ALIAS), (dict(qo=A[7]), ALIAS),
    (dict(rows=0), OK), (dict(rows=0, q=None, k=None, v=None, vc=None), OK)])
def test_qk_norm_rope_refuses(lib, kw, want):
    assert rope(lib, **kw) == want


def attn(lib, **kw):
    a = dict(q=A[0], dtype=2, gate=A[1], k=A[2], v=A[3], cdt=2, ks=1.0, vs=1.0, table=A[4], tstride=8, kv=A[5], scale=0.1,
             out=A[6], odt=2, lse=A[7], ws=A[8], wsb=1 << 30, batch=3, q_len=2, nq=8, nkv=2, d=128, pages=10, page=16,
             max_pages=8, qs=1024, gs=1024, ghs=128, os=1024, ps=4096, ts=256, hs=128)
    a.update(kw)
    return lib.gdna_attn_decode(a["q"], a["dtype"], a["gate"], a["k"], a["v"], a["cdt"], a["ks"], a["vs"], a["table"],
                                a["tstride"], a["kv"], a["scale"], a["out"], a["odt"], a["lse"], a["ws"], a["wsb"],
                                a["batch"], a["q_len"], a["nq"], a["nkv"], a["d"], a["pages"], a["page"], a["max_pages"],
                                a["qs"], a["gs"], a["ghs"], a["os"], a["ps"], a["ts"], a["hs"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), ARG), (dict(q_len=-1), ARG), (dict(nq=0), ARG), (dict(nkv=0), ARG), (dict(d=0), ARG),
    (dict(max_pages=0), ARG), (dict(nq=9), UNSUP), (dict(d=257), UNSUP), (dict(dtype=3), UNSUP), (dict(odt=3), UNSUP),
    (dict(cdt=0), UNSUP), (dict(cdt=4), UNSUP), (dict(batch=(1 << 20) + 1), UNSUP), (dict(q_len=1 << 22), UNSUP),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(ks=0.0), ARG), (dict(vs=float("nan")), ARG), (dict(ks=1e-30, scale=1e-30), ARG),
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(table=None), ARG), (dict(kv=None), ARG),
    (dict(out=None), ARG), (dict(ws=None), ARG), (dict(wsb=1000), ARG),
    (dict(tstride=7), ARG), (dict(qs=1023), ARG), (dict(gs=1023), ARG), (dict(ghs=127), ARG), (dict(os=1023), ARG),
    (dict(pages=0), ARG), (dict(page=0), ARG), (dict(ps=4095), ARG), (dict(ts=255), ARG), (dict(hs=100), ARG),
    (dict(q=A[0] + 1), ALIGN), (dict(out=A[6] + 1), ALIGN), (dict(ws=A[8] + 8), ALIGN), (dict(lse=A[7] + 2), ALIGN),
    (dict(k=A[2] + 1), ALIGN), (dict(kv=A[5] + 2), ALIGN),
    (dict(out=A[0]), ALIAS), (dict(out=A[2] + 4096), ALIAS), (dict(lse=A[6] + 16), ALIAS), (dict(ws=A[4]), ALIAS),
    (dict(out=A[1] + 128), ALIAS), (dict(lse=A[5]), ALIAS),
    (dict(batch=0), OK), (dict(q_len=0), OK), (dict(batch=0, q=None, ws=None), OK)])
def test_attn_decode_refuses(lib, kw, want):
    assert attn(lib, **kw) == want


def test_layouts_that_are_not_refused_reach_the_launch(lib):
    """Heads first, K and V interleaved by page or by head: sound strides pass the checks (the launch then fails
    without a GPU)."""
    for kw in (dict(ps=4096, ts=128, hs=2048), dict(v=A[2] + 2 * 4096, ps=8192), dict(v=A[2] + 2 * 128, ps=8192, ts=512, hs=256),
               dict(v=A[2])):
        assert attn(lib, **kw) == 5, kw
    assert rope(lib, vc=A[10] + 2 * 4096, ps=8192) == 5 and rope(lib, qo=A[0]) == 5


def test_rows_side_by_side_are_no_alias(lib):
    """q in place in the rows of one projection [q | k | v]; columns that reach into each other are refused."""
    packed = dict(qs=1024, kst=1024, vst=1024, qos=1024, qo=A[0], k=A[0] + 512 * 4, v=A[0] + 768 * 4)
    assert rope(lib, **packed) == 5
    assert rope(lib, **{**packed, "k": A[0] + 511 * 4}) == ALIAS
    assert rope(lib, **{**packed, "v": A[0] + 769 * 4}) == ALIAS
    assert rope(lib, **{**packed, "kst": 1028}) == ALIAS
    assert attn(lib, out=A[0] + 2 * 1024, qs=2048, os=2048) == 5 and attn(lib, out=A[0] + 2 * 1023, qs=2048, os=2048) == ALIAS


def test_more_work_than_64_bits_count_is_refused(lib):
    assert attn(lib, batch=1 << 20, q_len=1, nq=1 << 24, nkv=1 << 24, d=1, page=(1 << 31) - 1, max_pages=(1 << 31) - 1,
                pages=1, hs=1, ts=1 << 24, ps=1 << 56, qs=1 << 24, gs=1 << 24, ghs=1, os=1 << 24, tstride=1 << 31) == UNSUP


def test_workspace_grows_with_rows_and_d(built):
    size = lambda **kw: gdn.gdna_attn_workspace(**{**dict(batch=3, q_len=1, nq=8, nkv=2, d=128), **kw})   # noqa: E731
    assert size() > 0 and size() == size(batch=1000) and size(nq=9) == 0 and size(d=257) == 0 and size(d=0) == 0
    seen = [size(q_len=t) for t in (1, 2, 3, 5, 9, 17, 100)]
    assert seen == sorted(seen) and size(d=256) > size(d=64)


def table_of(**kw):
    a = {**dict(n_pos=5, rot=64, base=1e4), **kw}
    t = torch.full((a["n_pos"], a["rot"]), 7.0)
    gdn.gdna_rope_table(t, **a)
    return t.double().numpy()


def want_table(n, freq, amplitude=1.0):
    angle = np.asarray(n, np.longdouble)[:, None] * np.asarray(freq, np.longdouble)[None]
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float64) * amplitude


def freqs(rot, base):
    return np.array([np.longdouble(base) ** (np.longdouble(-2 * i) / rot) for i in range(rot // 2)])


@pytest.mark.parametrize("rot,base", [(64, 1e4), (128, 1e6), (2, 1e4), (256, 5e5)])
def test_rope_table(built, rot, base):
    """Half a unit in the last place of fp32 (|entry| <= 1: 2^-25), and the 64-bit angle's error, n * 2^-52."""
    got = table_of(n_pos=4000, rot=rot, base=base)
    assert np.abs(got - want_table(range(4000), freqs(rot, base))).max() <= 2.0 ** -25 + 4000 * 2.0 ** -50


def test_rope_table_far_positions(built):
    n = 262144
    got = table_of(n_pos=n, rot=8, base=1e4)
    assert np.abs(got[-5:] - want_table(range(n - 5, n), freqs(8, 1e4))).max() <= 2.0 ** -25 + n * 2.0 ** -50


def test_rope_scaling(built):
    f = freqs(64, 1e4)
    close = lambda kw, freq, amp=1.0: np.abs(table_of(n_pos=900, **kw) - want_table(range(900), freq, amp)).max() <= amp * 2e-7  # noqa: E731
    assert close(dict(kind=gdn.GDNA_ROPE_LINEAR, factor=4.0), f / 4)
    assert close(dict(kind=gdn.GDNA_ROPE_LINEAR, factor=1.0), f)
    ntk = freqs(64, 1e4 * 8 ** (64 / 62))
    assert close(dict(kind=gdn.GDNA_ROPE_NTK, factor=8.0), ntk)
    assert ntk[0] == f[0] and abs(ntk[-1] * 8 / f[-1] - 1) < 1e-12       # the fastest kept, the slowest divided
    # by parts: where a pair turns 32 times or more in 4096 positions it is kept, at one turn or less divided
    low = math.floor(64 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(1e4)))
    high = math.ceil(64 * math.log(4096 / (2 * math.pi)) / (2 * math.log(1e4)))
    ramp = np.clip((np.arange(32) - low) / (high - low), 0, 1)
    yarn = f * (1 - ramp) + f / 16 * ramp
    assert yarn[0] == f[0] and yarn[-1] == f[-1] / 16 and ((yarn <= f) & (yarn >= f / 16)).all()
    amp = 0.1 * math.log(16) + 1
    assert close(dict(kind=gdn.GDNA_ROPE_YARN, factor=16.0, original_len=4096.0, amplitude=amp), yarn, amp)


@pytest.mark.parametrize("kw,want", [
    (dict(n_pos=-1), ARG), (dict(rot=0), ARG), (dict(rot=3), ARG), (dict(base=0.0), ARG), (dict(base=float("inf")), ARG),
    (dict(amplitude=0.0), ARG), (dict(amplitude=float("nan")), ARG), (dict(kind=9), UNSUP),
    (dict(kind=1, factor=0.5), ARG), (dict(kind=2, factor=float("nan")), ARG), (dict(kind=2, factor=2.0, rot=2), ARG),
    (dict(kind=3, factor=2.0), ARG), (dict(kind=3, factor=2.0, original_len=100.0, beta_fast=1.0), ARG),
    (dict(kind=3, factor=2.0, original_len=100.0, beta_slow=0.0), ARG), (dict(table=None), ARG), (dict(n_pos=0), OK)])
def test_rope_table_refuses(built, kw, want):
    buf = (ctypes.c_float * 400)()
    a = dict(table=ctypes.addressof(buf), n_pos=4, rot=64, base=1e4, kind=0, factor=1.0, original_len=0.0, beta_fast=32.0,
             beta_slow=1.0, amplitude=1.0)
    a.update(kw)
    assert built.gdna_rope_table(a["table"], a["n_pos"], a["rot"], a["base"], a["kind"], a["factor"], a["original_len"],
                                 a["beta_fast"], a["beta_slow"], a["amplitude"]) == want
    if want != OK:
        assert not any(buf)


def test_binding_refuses_other_types(built):
    with pytest.raises(ValueError):
        gdn.gdna_attn_decode(torch.zeros(4, dtype=torch.int32), 0, 0, 0, 0, 0, 0, batch=1, nq=1, nkv=1, d=4, pages=1,
                             page_size=1, max_pages=1)
    with pytest.raises(ValueError):
        gdn.gdna_attn_decode(1 << 20, 0, 0, 0, 0, 0, 0, batch=1, nq=1, nkv=1, d=4, pages=1, page_size=1, max_pages=1)


def test_the_queue_of_parts_holds_every_part_in_use():
    """The tensor-core attention kernel's producer runs ahead of the consumers: a replay of the two, with one step a part
    (the furthest it gets), finds no part told into the slot of one that is still being added up."""
    source = open(os.path.join(os.path.dirname(HEADER), "..", "gated_deltanet_linear_16_gb300", "csrc", "gdna_attn_tc.cuh")).read()
    most = int(re.search(r"constexpr int kMaxStages = (\d+);", source)[1])
    slots = eval(re.search(r"constexpr int kQueue = ([^;]+);", source)[1], {"kMaxStages": most})
    for stages in range(2, most + 1):
        for in_use in range(100):                       # its step is released, its rows are being added up
            step = 0
            while True:
                told = step + 1                         # before the wait for the step's stage
                assert told <= in_use or told % slots != in_use % slots, (stages, in_use, told)
                if step - stages > in_use:              # that stage is not released yet
                    break
                step += 1


@pytest.mark.parametrize("stride", [1 << 60, 1 << 62, (1 << 63) - 1, (1 << 63) // 3 + 1])
def test_head_strides_whose_products_pass_64_bits_are_refused(lib, stride):
    """The last head's offset, and an array's bytes, are counted without wrapping."""
    for rows in (1, 2):
        assert rope(lib, qhs=stride, qs=stride, rows=rows) == ARG
        assert attn(lib, ghs=stride, gs=stride, batch=rows, q_len=1) == ARG
    assert rope(lib, qhs=stride, nq=1, qs=128) == 5                       # one head: the stride is not used
    assert attn(lib, ghs=stride, gs=128, nq=1, nkv=1) == 5


def test_more_heads_than_the_general_kernel_counts_are_refused(lib):
    """2^20 heads of 2^14 rows are 2^34, of 2^17 rows 2^37: more blocks of eight than a grid has."""
    far = [(1 << 45) * (i + 1) for i in range(5)]
    big = dict(q=far[0], k=None, v=None, qo=far[1], ko=None, kc=None, vc=None, cs=far[2], pos=far[3], slots=far[4], qn=None,
               kn=None, d=1, rot=0, nq=1 << 20, nkv=0, qs=1 << 20, qhs=1, qos=1 << 20)
    for rows in (1 << 14, 1 << 15, 1 << 17):
        assert rope(lib, **big, rows=rows) == UNSUP
    assert rope(lib, **big, rows=(1 << 14) - 1) == 5
    vec = {**big, "d": 64, "qhs": 64, "qs": 1 << 26, "qos": 1 << 26}      # the vector kernel: blocks of rows
    assert rope(lib, **vec, rows=1 << 14) == 5


I32, I64, F16, BF16, F32, F64 = torch.int32, torch.int64, torch.float16, torch.bfloat16, torch.float32, torch.float64


def binding_refuses(call, types, name, wrong):
    """A call whose operands have these types, but for one: the binding says which, and the library is not asked."""
    host = {n: torch.zeros(64, dtype=wrong if n == name else t) for n, t in types.items()}
    with pytest.raises(ValueError, match=rf"^{name} is {wrong}"):
        call(host)


@pytest.mark.parametrize("name,wrong", [(n, I64) for n in ("cached", "fresh", "table", "free_pages", "free_head", "kv_len",
                                                           "row_start", "positions", "free_head_out", "unserved")] + [("slots", I32)])
def test_page_assign_checks_types(built, name, wrong):
    types = {n: I32 for n in ("cached", "fresh", "table", "free_pages", "free_head", "kv_len", "row_start", "slots", "positions",
                              "free_head_out", "unserved")}
    types["slots"] = I64
    binding_refuses(lambda x: gdn.gdna_page_assign(**x, batch=2, rows=4, page_size=4, max_pages=4, stream=0), types, name, wrong)


@pytest.mark.parametrize("name,wrong", [("k", BF16), ("v", F16), ("q_out", BF16), ("k_out", F16), ("qn", BF16), ("kn", F64),
                                        ("cos_sin", F64), ("positions", I64), ("slots", I32), ("v_cache", BF16)])
def test_qk_norm_rope_checks_types(built, name, wrong):
    types = dict(q=F32, k=F32, v=F32, qn=F32, kn=F32, cos_sin=F32, positions=I32, slots=I64, q_out=F32, k_out=F32, k_cache=F16,
                 v_cache=F16)
    binding_refuses(lambda x: gdn.gdna_qk_norm_rope(**x, rows=1, nq=2, nkv=1, d=8, rot=4, n_pos=8, pages=2, page_size=4, stream=0),
                    types, name, wrong)


@pytest.mark.parametrize("name,wrong", [("gate", F32), ("v_cache", BF16), ("table", I64), ("kv_len", I64), ("lse", BF16)])
def test_attn_decode_checks_types(built, name, wrong):
    types = dict(q=BF16, k_cache=F16, v_cache=F16, table=I32, kv_len=I32, out=BF16, workspace=torch.uint8, gate=BF16, lse=F32)
    binding_refuses(lambda x: gdn.gdna_attn_decode(**x, batch=1, nq=2, nkv=1, d=8, pages=2, page_size=4, max_pages=2, stream=0),
                    types, name, wrong)


def test_rope_table_checks_types(built):
    with pytest.raises(ValueError, match="^table is torch.float64"):
        gdn.gdna_rope_table(torch.zeros((4, 8), dtype=F64), n_pos=4, rot=8, base=1e4)


def test_given_types_and_raw_addresses_are_taken_at_their_word(lib):
    """With `dtype` and `cache_dtype` the operands are what the caller says, as for raw addresses; the call then reaches the
    launch, which fails without a GPU."""
    raw = torch.zeros(1 << 22, dtype=torch.uint8)
    at = lambda i: raw[i << 18:(i + 1) << 18]                                      # noqa: E731
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdna_attn_decode(at(0), at(1), at(2), at(3).view(I32), raw.data_ptr() + (4 << 18), at(5), at(6).data_ptr(), gate=at(13),
                             batch=1, nq=2, nkv=1, d=8, pages=2, page_size=4, max_pages=2, stream=0, dtype=2, cache_dtype=3,
                             out_dtype=0, workspace_bytes=1 << 40)
    assert e.value.status == 5
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdna_qk_norm_rope(at(0), at(1), at(2), None, None, None, None, at(3).view(I64), at(4), at(5), at(6), rows=1, nq=2, nkv=1,
                              d=8, rot=0, n_pos=0, pages=2, page_size=4, stream=0, dtype=1, cache_dtype=3)
    assert e.value.status == 5


@pytest.mark.parametrize("kw", [dict(batch=(1 << 20) + 1), dict(q_len=1 << 22), dict(nq=1 << 25), dict(batch=1 << 20, q_len=1 << 12)])
def test_the_workspace_of_a_shape_that_is_refused_is_zero(lib, kw):
    """gdna_attn_workspace says 0 for what gdna_attn_decode refuses."""
    shape = {**dict(batch=3, q_len=2, nq=8, nkv=2, d=128), **kw}
    rows = shape["nq"] * 128
    assert attn(lib, **shape, qs=rows, gs=rows, os=rows) == UNSUP
    assert gdn.gdna_attn_workspace(**shape) == 0
