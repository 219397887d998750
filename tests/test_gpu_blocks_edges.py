"""Prompt and shared-prefix attention where a call's sizes, starts or values lie at the edge of what the header allows, against
64-bit references (bounds: prompt_helpers)."""
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn
from tests.prompt_helpers import check_prompt, make_prompt

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
    from tests.prompt_helpers import call_prompt
    call_prompt(s, want, max_pages=8)
    pages = s["pages"]
    k, v = pages.store.addresses()
    ws = torch.empty(gdn.gdnb_attn_prompt_workspace(rows=s["rows"], batch=2, nq=6, nkv=2, d=d), dtype=torch.uint8, device="cuda")
    start = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
    gdn.gdnb_attn_prompt(s["q"], k, v, start, lens, whole, ws, rows=s["rows"], batch=2, nq=6, nkv=2, d=d, table=pages.table,
                         table_stride=pages.table.stride(0), max_pages=8, **pages.store.args())
    torch.cuda.synchronize()
    assert torch.equal(whole, want)
