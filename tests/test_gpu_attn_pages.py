"""gdna_page_assign against a plain Python walk over the sequences: whole numbers, equal everywhere."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_16_gb300 as gdn

pytestmark = pytest.mark.gpu


def walk(cached, fresh, table, free, head, rows, page, max_pages):
    """The definition, one sequence after the other."""
    table = table.copy()
    kv_len, start = [], []
    slots, positions = np.full(rows, -1, np.int64), np.zeros(rows, np.int64)
    row, used, unserved = 0, 0, 0
    for b, (c, f) in enumerate(zip(np.maximum(cached, 0).tolist(), np.maximum(fresh, 0).tolist())):
        have, want = -(-c // page), -(-(c + f) // page)
        fits = f == 0 or (want <= max_pages and c + f < 2 ** 31)
        need = want - have if fits else 0
        served = fits and (need == 0 or head + used + need <= len(free)) and (f == 0 or row + f <= rows)
        start.append(min(row, rows))
        kv_len.append(c + f if served else c)
        if served:
            for i in range(need):
                table[b, have + i] = free[head + used + i]
        elif f > 0:
            unserved += 1
        for i in range(min(f, max(0, rows - row))):
            pos = c + i
            positions[row + i] = min(pos, 2 ** 31 - 1)
            if served and table[b, pos // page] >= 0:
                slots[row + i] = int(table[b, pos // page]) * page + pos % page
        row += f
        # from the first that finds too few pages on, sequences that need one are not served
        used += need if served else (len(free) + 1 if need and head + used + need > len(free) else need)
    return dict(table=table, kv_len=kv_len, row_start=start + [min(row, rows)], slots=slots, positions=positions,
                unserved=unserved)


def run(cached, fresh, table, free, head, rows, page, max_pages, stride=None, stream=None):
    batch, stride = len(cached), stride or max_pages
    i32 = dict(dtype=torch.int32, device="cuda")
    wide = torch.full((batch, stride), -7, **i32)
    wide[:, :max_pages] = torch.tensor(table, **i32)
    out = dict(kv_len=torch.full((batch + 2,), -9, **i32), row_start=torch.full((batch + 3,), -9, **i32),
               slots=torch.full((rows + 3,), -9, dtype=torch.int64, device="cuda"),
               positions=torch.full((rows + 3,), -9, **i32), head=torch.full((3,), -9, **i32),
               unserved=torch.full((3,), -9, **i32))
    args = [torch.tensor(np.asarray(x, np.int32), device="cuda") for x in (cached, fresh, free, [head])]
    torch.cuda.synchronize()
    gdn.gdna_page_assign(args[0], args[1], wide, args[2], args[3], out["kv_len"], out["row_start"], out["slots"],
                         out["positions"], out["head"], out["unserved"], batch=batch, rows=rows, page_size=page,
                         max_pages=max_pages, table_stride=stride, stream=stream)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in out.items()}
    for k, n in (("kv_len", batch), ("row_start", batch + 1), ("slots", rows), ("positions", rows), ("head", 1),
                 ("unserved", 1)):
        assert (got[k][n:] == -9).all(), k
        got[k] = got[k][:n]
    wide = wide.cpu().numpy()
    assert (wide[:, max_pages:] == -7).all()
    got["table"] = wide[:, :max_pages]
    return got


def compare(got, want, head):
    for k in ("kv_len", "row_start", "slots", "positions", "table"):
        assert np.array_equal(got[k], want[k]), k
    assert got["unserved"][0] == want["unserved"]


def setup(rng, batch, page, max_pages, low, high, spare=0, few=0):
    """Random lengths: cached within the table, fresh in [low, high]; a free list that just suffices."""
    fresh = rng.integers(low, high + 1, batch)
    cached = (rng.random(batch) * np.maximum(0, max_pages * page - fresh)).astype(np.int64)
    cached[rng.random(batch) < 0.2] = 0
    have, want = -(-cached // page), -(-(cached + fresh) // page)
    ids = rng.permutation(int(want.sum()) + spare + 40)
    table = np.full((batch, max_pages), -1, np.int64)
    at = 0
    for b in range(batch):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = ids[at:]
    return cached, fresh, table, free, 3, int((want - have).sum())


@pytest.mark.parametrize("batch,page,max_pages,low,high", [
    (1, 16, 8, 1, 1), (1, 1, 40, 1, 7), (3, 16, 64, 0, 0), (7, 24, 50, 0, 300), (256, 16, 64, 1, 1),
    (257, 16, 64, 0, 2), (1000, 8, 16, 0, 3), (5, 64, 200, 900, 5000), (64, 100, 30, 0, 2500), (3000, 3, 20, 0, 9)])
@pytest.mark.parametrize("pad", [0, 1, 777])
def test_equal_to_the_walk(cuda_lib, batch, page, max_pages, low, high, pad):
    rng = np.random.default_rng(batch * 7 + page + pad)
    cached, fresh, table, free, head, need = setup(rng, batch, page, max_pages, low, high)
    rows = int(fresh.sum()) + pad
    got = run(cached, fresh, table, free, head, rows, page, max_pages, stride=max_pages + 5)
    want = walk(cached, fresh, table, free, head, rows, page, max_pages)
    compare(got, want, head)
    assert got["head"][0] == head + need and got["unserved"][0] == 0


@pytest.mark.parametrize("lack", [1, 5, 10 ** 6])
def test_pages_run_out(cuda_lib, lack):
    rng = np.random.default_rng(lack)
    page, max_pages = 16, 40
    cached, fresh, table, free, head, need = setup(rng, 300, page, max_pages, 0, 40)
    free = free[:max(head, head + need - lack)]
    rows = int(fresh.sum())
    got = run(cached, fresh, table, free, head, rows, page, max_pages)
    want = walk(cached, fresh, table, free, head, rows, page, max_pages)
    compare(got, want, head)
    assert got["unserved"][0] > 0 and head <= got["head"][0] <= len(free)
    # a page is given to one sequence only, and every one before the new head was given
    new = got["table"][got["table"] != table]
    assert len(set(new.tolist())) == len(new) == got["head"][0] - head


def test_rows_run_out(cuda_lib):
    rng = np.random.default_rng(5)
    cached, fresh, table, free, head, _ = setup(rng, 200, 16, 40, 0, 20)
    rows = int(fresh.sum()) * 2 // 3
    got = run(cached, fresh, table, free, head, rows, 16, 40)
    compare(got, walk(cached, fresh, table, free, head, rows, 16, 40), head)
    assert got["unserved"][0] > 0
    got = run(cached, fresh, table, free, head, 0, 16, 40)
    compare(got, walk(cached, fresh, table, free, head, 0, 16, 40), head)


def test_a_row_of_the_table_is_too_short(cuda_lib):
    rng = np.random.default_rng(6)
    cached, fresh, table, free, head, _ = setup(rng, 60, 16, 10, 0, 30, spare=600)
    fresh[5], fresh[17], fresh[40] = 161, 10 ** 6, 4000
    cached[40] = 10 ** 9                                # not a length the table could hold at all
    rows = int(fresh.sum())
    got = run(cached, fresh, table, free, head, rows, 16, 10)
    compare(got, walk(cached, fresh, table, free, head, rows, 16, 10), head)
    assert got["unserved"][0] == 3


def test_invalid_device_values(cuda_lib):
    """Negative lengths count as 0; a negative page gives slot -1; a head outside the list serves nobody new."""
    table = np.array([[4, -1, -1], [5, 6, -1], [-3, -1, -1]])
    cached, fresh = np.array([-5, 30, 8]), np.array([3, -2, 4])
    got = run(cached, fresh, table, np.array([9, 8]), 0, 7, 16, 3)
    compare(got, walk(cached, fresh, table, np.array([9, 8]), 0, 7, 16, 3), 0)
    assert got["kv_len"].tolist() == [3, 30, 12] and got["slots"].tolist() == [144, 145, 146, -1, -1, -1, -1]
    for head in (-1, 2, 1000):
        got = run(cached, fresh, table, np.array([9, 8]), head, 7, 16, 3)
        assert got["unserved"][0] == 1 and got["head"][0] == head and (got["table"] == table).all()


def test_slots_past_32_bits(cuda_lib):
    page = 64
    table = np.array([[2 ** 31 - 1, -1], [2 ** 30, -1]])
    free = np.array([2 ** 31 - 2, 2 ** 29])
    got = run(np.array([60, 3]), np.array([6, 2]), table, free, 0, 9, page, 2)
    want = walk(np.array([60, 3]), np.array([6, 2]), table, free, 0, 9, page, 2)
    compare(got, want, 0)
    assert got["slots"].max() > 2 ** 36


def test_empty_calls_and_another_stream(cuda_lib):
    one = torch.zeros(4, dtype=torch.int32, device="cuda")
    gdn.gdna_page_assign(one, one, one, one, one, one, one, one, one, one, one, batch=0, rows=0, page_size=1, max_pages=1)
    rng = np.random.default_rng(1)
    cached, fresh, table, free, head, _ = setup(rng, 30, 16, 40, 0, 9)
    rows = int(fresh.sum())
    got = run(cached, fresh, table, free, head, rows, 16, 40, stream=torch.cuda.Stream())
    compare(got, walk(cached, fresh, table, free, head, rows, 16, 40), head)


@pytest.mark.parametrize("rows", [0, 5])
def test_a_batch_of_zero_writes_nothing(cuda_lib, rows):
    """An empty call, as the header says: the head stays where the caller has it, and no slot, start or count changes."""
    outs = [torch.full((8,), -9, dtype=torch.int64 if i == 2 else torch.int32, device="cuda") for i in range(6)]
    ins = [torch.full((8,), 3, dtype=torch.int32, device="cuda") for _ in range(5)]
    kv_len, start, slots, positions, head_out, unserved = outs
    cached, fresh, table, free, head = ins
    gdn.gdna_page_assign(cached, fresh, table, free, head, kv_len, start, slots, positions, head_out, unserved, batch=0,
                         rows=rows, page_size=16, max_pages=1)
    torch.cuda.synchronize()
    assert all((x == -9).all() for x in outs) and all((x == 3).all() for x in ins)


def test_a_batch_without_new_tokens_or_rows(cuda_lib):
    """rows 0 with a batch is a call: lengths, starts, head and count are written."""
    got = run(np.array([5, 0, 40]), np.array([0, 0, 0]), np.array([[4, -1, -1], [-1, -1, -1], [5, 6, 7]]), np.array([9, 8]), 1, 0, 16, 3)
    assert got["kv_len"].tolist() == [5, 0, 40] and got["row_start"].tolist() == [0, 0, 0, 0]
    assert got["head"][0] == 1 and got["unserved"][0] == 0
