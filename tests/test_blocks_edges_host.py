"""Checks of the decoder-block entry points at the edges, without a GPU: the workspaces' sizes as calls shrink."""
import pytest

import gated_deltanet_linear_16_gb300 as gdn
from tests.test_blocks_host import A, ARG, shared


@pytest.fixture(scope="module")
def built():
    gdn.build()
    return gdn.load()


@pytest.mark.parametrize("nq,nkv,d", [(48, 8, 128), (8, 1, 128), (24, 4, 256), (32, 32, 64), (16, 16, 256), (128, 1, 256), (128, 1, 64),
                                      (200, 200, 128), (6, 2, 33)])
def test_a_shared_step_s_scratch_serves_all_smaller_steps(built, nq, nkv, d):
    """Own keys go with the prefix up to some number of their tiles, and need a partial result for each; behind it they do not."""
    def need(batch, groups=1, q_len=1):
        return gdn.gdnb_attn_shared_workspace(batch=batch, groups=groups, q_len=q_len, nq=nq, nkv=nkv, d=d)
    batches = list(range(0, 170)) + [200, 256, 300, 511, 1000, 5000]
    for q_len in (1, 2, 3, 5):
        sizes = [need(b, 1, q_len) for b in batches]
        assert sizes == sorted(sizes) and sizes[0] > 0
    for batch in (1, 2, 7, 20, 38, 39, 153, 400):
        sizes = [need(batch, 1, q) for q in list(range(0, 40)) + [60, 100, 128, 129, 255, 256, 257, 300, 511, 520, 1024, 3000]]
        assert sizes == sorted(sizes)
        sizes = [need(batch, g, 2) for g in (1, 2, 3, 5, 8, 20, 50, 400, 65536)]
        assert sizes == sorted(sizes)


@pytest.mark.parametrize("nq,nkv,d", [(48, 8, 128), (8, 1, 64), (24, 4, 256)])
def test_a_prompt_call_s_scratch_serves_all_smaller_calls(built, nq, nkv, d):
    sizes = [gdn.gdnb_attn_prompt_workspace(rows=r, batch=7, nq=nq, nkv=nkv, d=d) for r in list(range(0, 700)) + [1000, 5000, 10 ** 6]]
    assert sizes == sorted(sizes)
    sizes = [gdn.gdnb_attn_prompt_workspace(rows=900, batch=b, nq=nq, nkv=nkv, d=d) for b in list(range(0, 400)) + [1000, 65536]]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("batch", [3, 20, 200])
def test_a_shared_step_asks_for_the_scratch_that_it_names(built, batch):
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake-pointer validation tests run only on hosts without a GPU")
    need = gdn.gdnb_attn_shared_workspace(batch=batch, groups=2, q_len=2, nq=8, nkv=2, d=128)
    call = dict(batch=batch, pages=1000, ws=A[15])
    assert shared(built, wsb=need - 1, **call) == ARG and shared(built, wsb=need, **call) != ARG
