"""Prompt and shared-prefix attention where a call's sizes, starts or values lie at the edge of what the header allows, against
64-bit references (bounds: prompt_helpers)."""
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.attn_layers_helpers import guarded, intact
from tests.prompt_helpers import call_prompt, check_prompt, make_prompt

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
