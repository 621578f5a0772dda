"""dsa_slot_map against the rule in Python."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from top_sparse_attention_chunked_gb300 import build_lib, dsa
    build_lib.build()
    dsa.load_library()
    return dsa


def rule(q, t, tokens, table=None, bs=0, blocks=0, cap=0):
    slots, pos, rows, first = [], [], [], [0]
    for b, (n, total) in enumerate(zip(q, t)):
        for i in range(max(0, n)):
            if len(slots) == tokens:
                break
            p, s = total - n + i, -1
            if table is None:
                s = b * cap + p if 0 <= p < cap else -1
            elif 0 <= p < len(table[b]) * bs and 0 <= table[b][p // bs] < blocks:
                s = table[b][p // bs] * bs + p % bs
            slots.append(s)
            pos.append(max(p, 0))
            rows.append(b)
        first.append(min(tokens, first[-1] + max(0, n)))
    k = tokens - len(slots)
    return slots + [-1] * k, pos + [0] * k, rows + [-1] * k, first


def run(D, q, t, tokens, table=None, bs=0, blocks=0, cap=0):
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.full((tokens,), 99, **i32) for _ in range(3)] + [torch.full((len(q) + 1,), 99, **i32)]
    pages = None if table is None else D.make_pages(torch.tensor(table, **i32), bs, blocks)
    D.dsa_slot_map(torch.tensor(q, **i32), torch.tensor(t, **i32), out[0], pages=pages, capacity=cap, positions=out[1],
                   rows=out[2], first=out[3])
    want = rule(q, t, tokens, table, bs, blocks, cap)
    for name, x, w in zip(("slots", "positions", "rows", "first"), out, want):
        assert x.tolist() == w, name
    only = torch.full((tokens,), 99, **i32)
    D.dsa_slot_map(torch.tensor(q, **i32), torch.tensor(t, **i32), only, pages=pages, capacity=cap)
    assert only.tolist() == want[0]


def batch(seed, rows, most_new, most, bs):
    r = random.Random(seed)
    q = [r.choice([0, 1, 1, r.randint(0, most_new)]) for _ in range(rows)]
    t = [x + r.randint(0, most - x) for x in q]
    per_seq = -(-most // bs)
    need = [-(-x // bs) for x in t]
    order = list(range(sum(need) + 3))
    r.shuffle(order)
    table, k = [], 0
    for n in need:
        table.append(order[k:k + n] + [-1] * (per_seq - n))
        k += n
    return q, t, table, len(order)


@pytest.mark.parametrize("rows", [1, 2, 31, 255, 256, 257, 1000, 4095, 4096])
@pytest.mark.parametrize("bs", [128, 1024])
def test_paged(D, rows, bs):
    q, t, table, blocks = batch(rows, rows, 300 if rows < 300 else 6, 3000, bs)
    for spare in (0, 1, 700):
        run(D, q, t, sum(q) + spare, table, bs, blocks)
    run(D, q, t, max(0, sum(q) - 3), table, bs, blocks)           # a step that does not hold them all
    run(D, q, t, sum(q) // 2, table, bs, blocks)


@pytest.mark.parametrize("rows,cap", [(1, 1), (3, 700), (200, 64)])
def test_dense(D, rows, cap):
    r = random.Random(rows)
    q = [r.randint(0, cap) for _ in range(rows)]
    run(D, q, [x + r.randint(0, cap - x) for x in q], sum(q) + 5, cap=cap)


def test_one_long_request_and_empty_ones(D):
    run(D, [0] * 20 + [5000] + [0] * 20, [3] * 20 + [5000] + [7] * 20, 5000, cap=5000)
    run(D, [0, 0, 0], [0, 5, 9], 4, cap=10)
    run(D, [0, 0, 0], [0, 5, 9], 0, cap=10)


def test_lengths_and_entries_out_of_range(D):
    """What the device holds may be anything: no slot, and no access outside the table."""
    big = 2 ** 31 - 1
    run(D, [3, -5, 2, 4], [1, 9, 300, 2], 12, cap=256)            # positions below 0, lengths below 0, behind the cache
    run(D, [2, 2, 2], [200, 400, 600], 6, [[5, -1], [0, 1 << 30], [1, 2]], 256, 5)
    i32 = dict(dtype=torch.int32, device="cuda")
    slots, pos = torch.full((4,), 9, **i32), torch.full((4,), 9, **i32)
    D.dsa_slot_map(torch.tensor([2, big, big], **i32), torch.tensor([2, big, 5], **i32), slots, capacity=100, positions=pos)
    assert slots.tolist() == [0, 1, 100, 101] and pos.tolist() == [0, 1, 0, 1]
    D.dsa_slot_map(torch.tensor([-big, 3, big], **i32), torch.tensor([big, -big, big], **i32), slots, capacity=100, positions=pos)
    assert slots.tolist() == [-1, -1, -1, 200] and pos.tolist() == [0, 0, 0, 0]


def test_captured_with_lengths_that_change(D):
    i32 = dict(dtype=torch.int32, device="cuda")
    q, t, table, blocks = batch(7, 40, 20, 1000, 128)
    q2, t2, _, _ = batch(8, 40, 20, 1000, 128)
    dq, dt, slots = torch.tensor(q, **i32), torch.tensor(t, **i32), torch.zeros(500, **i32)
    pages = D.make_pages(torch.tensor(table, **i32), 128, blocks)
    D.dsa_slot_map(dq, dt, slots, pages=pages)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.dsa_slot_map(dq, dt, slots, pages=pages)
    dq.copy_(torch.tensor(q2, **i32))
    dt.copy_(torch.tensor(t2, **i32))
    g.replay()
    assert slots.tolist() == rule(q2, t2, 500, table, 128, blocks)[0]
