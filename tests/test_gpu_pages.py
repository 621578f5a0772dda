"""dsa_pages_update / dsa_pages_compact against the rules in plain Python:
every table entry, every count, every byte of every pool."""
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


def update(table, refs, bs, parent, keep, new, first=None):
    """The new (table, refs, copies [(src, dst)]) or the reason why not."""
    rows, W, nb = len(table), len(table[0]), len(refs)
    first = first or [0] * rows
    for r in range(rows):
        if not (-1 <= parent[r] < rows and 0 <= keep[r] <= new[r] <= W * bs and 0 <= first[r] <= keep[r]):
            return "bad"
        if parent[r] < 0 and keep[r]:
            return "bad"
    if any(x >= nb for row in table for x in row):
        return "bad"
    after, out = list(refs), []
    for row in table:
        for x in row:
            if x >= 0:
                after[x] -= 1
    for r in range(rows):
        kept = -(-keep[r] // bs)
        row = [table[parent[r]][j] if j >= first[r] // bs else -1 for j in range(kept)]
        row = [x if x >= 0 else -1 for x in row]
        out.append(row)
        for x in row:
            if x >= 0:
                after[x] += 1
    writers = {}
    for r in range(rows):
        if keep[r] % bs and new[r] > keep[r]:
            if out[r][-1] < 0:
                return "bad"
            writers.setdefault(out[r][-1], []).append(r)
    free = [x for x in range(nb) if after[x] == 0]
    copies, at = [], 0
    plan = []
    for r in range(rows):
        copy = False
        if keep[r] % bs and new[r] > keep[r]:
            x = out[r][-1]
            copy = not (after[x] == len(writers[x]) and writers[x][0] == r)
        plan.append(copy)
        at += (-(-new[r] // bs) - len(out[r])) + copy
    if at > len(free):
        return "full"
    counts, at = list(after), 0
    for r in range(rows):
        if plan[r]:
            src = out[r].pop()
            counts[src] -= 1
            copies.append((src, free[at]))
        while len(out[r]) < -(-new[r] // bs):
            out[r].append(free[at])
            counts[free[at]] += 1
            at += 1
        out[r] += [-1] * (W - len(out[r]))
    return out, counts, copies


def compact(table, refs):
    live = [x for x in range(len(refs)) if refs[x] > 0]
    n = len(live)
    holes = [x for x in range(n) if refs[x] <= 0]
    movers = [x for x in live if x >= n]
    remap = [x if refs[x] > 0 else -1 for x in range(len(refs))]
    for a, b in zip(movers, holes):
        remap[a] = b
    counts = [0] * len(refs)
    for x in live:
        counts[remap[x]] = refs[x]
    return [[remap[x] if x >= 0 else x for x in row] for row in table], counts, remap, list(zip(movers, holes))


class State:
    def __init__(self, D, table, refs, bs, shapes=((64, torch.bfloat16), (2 * 128, torch.bfloat16), (2, torch.float32)),
                 layers=2, seed=0):
        self.D, self.bs, self.nb = D, bs, len(refs)
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda")
        self.refs = torch.tensor(refs, dtype=torch.int32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pools = [torch.randn(self.nb * bs, n, device="cuda", generator=g).to(dt)
                      for _ in range(layers) for n, dt in shapes]
        self.st = D.make_page_state(self.table, self.refs, bs)
        self.arr = D.make_page_pools(self.pools, self.nb)
        self.ws = D.alloc_pages_workspace(self.st)
        self.ws.fill_(0xCD)

    def moved(self, copies):
        want = [p.clone().view(self.nb, -1) for p in self.pools]
        for w, p in zip(want, self.pools):
            for s, d in copies:
                w[d] = p.view(self.nb, -1)[s]
        return want

    def same_pools(self, want):
        return all(torch.equal(p.view(self.nb, -1), w) for p, w in zip(self.pools, want))


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_update(D, table, refs, bs, parent, keep, new, first=None, in_place=True, **kw):
    s = State(D, table, refs, bs, **kw)
    want = update(table, refs, bs, parent, keep, new, first)
    ok = not isinstance(want, str)
    pools = s.moved(want[2] if ok else [])
    counts = torch.full((2,), -9, dtype=torch.int32, device="cuda")
    t_out = None if in_place else torch.full_like(s.table, -9)
    r_out = None if in_place else torch.full_like(s.refs, -9)
    D.dsa_pages_update(s.st, dev(parent), dev(keep), dev(new), s.arr, s.ws, t_out, r_out,
                       first_key=None if first is None else dev(first), counts=counts)
    torch.cuda.synchronize()
    t, r = (s.table, s.refs) if in_place else (t_out, r_out)
    if ok:
        assert D.dsa_read_device_status(s.ws) == 0
        assert t.tolist() == want[0]
        assert r.tolist() == want[1]
        assert counts.tolist() == [len(want[2]), sum(x == 0 for x in want[1])]
    else:
        with pytest.raises(D.DsaError) as e:
            D.dsa_read_device_status(s.ws)
        assert e.value.status == (D.DSA_ERR_INVALID_ARG if want == "bad" else D.DSA_ERR_WORKSPACE)
        assert t.tolist() == table and r.tolist() == refs
        assert counts.tolist() == [-1, sum(x == 0 for x in refs)]
    if not in_place:
        assert s.table.tolist() == table and s.refs.tolist() == refs
    assert s.same_pools(pools), "pool contents"
    return want


def counts_of(table, nb, pins=()):
    refs = [0] * nb
    for row in table:
        for x in row:
            if x >= 0:
                refs[x] += 1
    for x in pins:
        refs[x] += 1
    return refs


def test_fork_reorder_grow_by_hand(D):
    bs = 128
    # two requests of two rows: rows 0, 1 share block 5 and write into 1 and 2; rows 2, 3 share everything
    table = [[5, 1, -1], [5, 2, -1], [7, 0, -1], [7, 0, -1]]
    refs = counts_of(table, 10)
    for in_place in (True, False):
        out, counts, copies = check_update(D, table, refs, bs, [1, 1, 2, 3], [200, 200, 130, 130], [201, 201, 131, 257],
                                           in_place=in_place)
        # row 0 and 1 continue row 1: row 0 keeps block 2, row 1 copies it into the lowest free block (1 is
        # free now); row 2 keeps block 0, row 3 copies it and takes another for its third
        assert out == [[5, 2, -1], [5, 1, -1], [7, 0, -1], [7, 3, 4]]
        assert copies == [(2, 1), (0, 3)]


def test_holders_that_do_not_write_keep_a_block_shared(D):
    bs = 128
    table = [[4, 2], [4, 2], [4, -1]]
    refs = counts_of(table, 6)
    check_update(D, table, refs, bs, [0, 1, 2], [130, 256, 100], [131, 256, 101])   # row 1 holds 2 full, rows 0, 1 hold 4 full
    check_update(D, table, refs, bs, [0, 1, 2], [130, 130, 128], [130, 131, 128])   # row 0 does not write
    refs = counts_of(table, 6, pins=[2])                                           # held outside the table
    check_update(D, table, refs, bs, [0, -1, 2], [130, 0, 128], [131, 0, 129])


def test_end_truncate_empty_and_holes(D):
    bs = 128
    table = [[0, 1, 2], [3, -1, 4], [-1, -1, -1]]
    refs = counts_of(table, 5)
    check_update(D, table, refs, bs, [-1, -1, -1], [0, 0, 0], [0, 0, 0])
    check_update(D, table, refs, bs, [-1, 1, 0], [0, 384, 256], [200, 384, 384])
    check_update(D, table, refs, bs, [0, 1, 2], [100, 300, 0], [100, 300, 0])
    check_update(D, table, refs, bs, [0, 1, 1], [300, 300, 128], [301, 301, 129], first=[256, 290, 128])
    check_update(D, table, refs, bs, [0, 1, 2], [300, 300, 0], [300, 300, 0], first=[127, 128, 0])


@pytest.mark.parametrize("what", ["parent", "parent_low", "keep", "shrink", "long", "orphan", "entry", "first", "hole"])
@pytest.mark.parametrize("in_place", [True, False])
def test_out_of_range_changes_nothing(D, what, in_place):
    bs = 128
    table = [[0, 1, -1], [2, 3, 4]]
    refs = counts_of(table, 8)
    a = dict(parent=[0, 1], keep=[200, 300], new=[201, 301], first=[0, 0])
    if what == "parent":
        a["parent"][1] = 2
    elif what == "parent_low":
        a["parent"][1] = -2
    elif what == "keep":
        a["keep"][0] = -1
    elif what == "shrink":
        a["new"][0] = 199
    elif what == "long":
        a["new"][1] = 3 * bs + 1
    elif what == "orphan":
        a["parent"][0] = -1
    elif what == "entry":
        table[1][1] = 8
    elif what == "first":
        a["first"][1] = 301
    elif what == "hole":
        table[0][1] = -1
        refs = counts_of(table, 8)
    assert check_update(D, table, refs, bs, a["parent"], a["keep"], a["new"], a["first"], in_place=in_place) == "bad"


@pytest.mark.parametrize("in_place", [True, False])
def test_too_few_blocks_changes_nothing(D, in_place):
    table = [[0, 1, -1, -1], [0, 2, -1, -1]]
    refs = counts_of(table, 5)
    assert check_update(D, table, refs, 128, [0, 0], [200, 200], [512, 384], in_place=in_place) == "full"
    assert not isinstance(check_update(D, table, refs, 128, [0, 0], [200, 200], [384, 384], in_place=in_place), str)


def random_state(rng, rows, W, nb, bs):
    """Rows that share prefixes, lengths, counts with some pins."""
    free = list(range(nb))
    rng.shuffle(free)
    table, lens = [], []
    for r in range(rows):
        n = rng.randint(0, W)
        row = []
        if table and rng.random() < 0.6:
            p = rng.choice(table)
            row = [x for x in p if x >= 0][:rng.randint(0, n)]
        while len(row) < n and free:
            row.append(free.pop())
        lens.append(max(0, len(row) * bs - rng.choice([0, 0, 1, bs // 2, bs - 1])) if row else 0)
        table.append(row + [-1] * (W - len(row)))
    pins = [x for x in range(nb) if rng.random() < 0.05]
    return table, lens, counts_of(table, nb, pins)


@pytest.mark.parametrize("rows,W,nb,bs", [(1, 1, 1, 128), (5, 3, 20, 128), (33, 7, 200, 128), (64, 40, 3000, 128),
                                          (300, 9, 2000, 256), (1500, 3, 5001, 128)])
def test_random_updates(D, rows, W, nb, bs):
    rng = random.Random(rows * 7 + W)
    small = dict(shapes=((4, torch.bfloat16), (1, torch.float32)), layers=1) if nb > 1000 else {}
    seen = set()
    for i in range(6):
        table, lens, refs = random_state(rng, rows, W, nb, bs)
        parent = [rng.choice([-1, r, rng.randrange(rows)]) for r in range(rows)]
        keep = [0 if p < 0 else (lens[p] if rng.random() < 0.7 else rng.randint(0, lens[p])) for p in parent]
        new = [min(W * bs, k + rng.choice([0, 0, 1, 5, bs, 2 * bs + 3])) for k in keep]
        got = check_update(D, table, refs, bs, parent, keep, new, in_place=bool(i & 1), **small)
        seen.add(got if isinstance(got, str) else "ok")
    assert "ok" in seen


@pytest.mark.parametrize("rows,W,nb,bs", [(1, 1, 1, 128), (5, 3, 20, 128), (33, 7, 200, 128), (64, 40, 3000, 128)])
def test_compact(D, rows, W, nb, bs):
    rng = random.Random(nb)
    small = dict(shapes=((4, torch.bfloat16), (1, torch.float32)), layers=1) if nb > 1000 else {}
    for i in range(5):
        table, lens, refs = random_state(rng, rows, W, nb, bs)
        if i == 4:
            table, refs = [[-1] * W for _ in range(rows)], [0] * nb
        s = State(D, table, refs, bs, **small)
        want, counts, remap, moves = compact(table, refs)
        pools = s.moved(moves)
        t_out, r_out = (None, None) if i & 1 else (torch.full_like(s.table, -9), torch.full_like(s.refs, -9))
        rm = torch.full_like(s.refs, -9)
        cnt = torch.full((2,), -9, dtype=torch.int32, device="cuda")
        D.dsa_pages_compact(s.st, s.arr, s.ws, t_out, r_out, remap=rm if i < 3 else None, counts=cnt)
        torch.cuda.synchronize()
        assert D.dsa_read_device_status(s.ws) == 0
        assert (s.table if i & 1 else t_out).tolist() == want
        assert (s.refs if i & 1 else r_out).tolist() == counts
        if i < 3:
            assert rm.tolist() == remap
        assert cnt.tolist() == [len(moves), sum(x <= 0 for x in refs)]
        assert s.same_pools(pools)


def test_compact_refuses_entries_without_a_count(D):
    for bad in (3, 7):
        for in_place in (True, False):
            table, refs = [[0, bad], [6, -1]], [1, 0, 0, 0, 0, 0, 1]
            s = State(D, table, refs, 128)
            pools = s.moved([])
            t_out, r_out = (None, None) if in_place else (torch.full_like(s.table, -9), torch.full_like(s.refs, -9))
            D.dsa_pages_compact(s.st, s.arr, s.ws, t_out, r_out)
            with pytest.raises(D.DsaError):
                D.dsa_read_device_status(s.ws)
            assert (s.table if in_place else t_out).tolist() == table
            assert (s.refs if in_place else r_out).tolist() == refs
            assert s.same_pools(pools)


def test_captured_update_replays_on_new_parents(D):
    bs = 128
    table = [[0, 1, -1, -1], [0, 2, -1, -1], [0, 3, -1, -1]]
    refs = counts_of(table, 12)
    s = State(D, table, refs, bs)
    parent, keep, new = dev([0, 1, 2]), dev([200] * 3), dev([201] * 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.dsa_pages_update(s.st, parent, keep, new, s.arr, s.ws)
    host, n = table, 200
    for step, ps in enumerate([[2, 2, 0], [1, 0, 0], [0, 1, 2], [1, 1, 1]]):
        parent.copy_(dev(ps))
        keep.fill_(n)
        new.fill_(n + 40)
        want = update(host, s.refs.tolist(), bs, ps, [n] * 3, [n + 40] * 3)
        pools = s.moved(want[2])
        graph.replay()
        torch.cuda.synchronize()
        assert s.table.tolist() == want[0] and s.refs.tolist() == want[1] and s.same_pools(pools)
        host, n = want[0], n + 40


def test_many_pools_and_large_blocks(D):
    """256 pools, and a block of several copy pieces whose last is a short one."""
    table = [[3, -1], [3, -1], [0, 2]]
    refs = counts_of(table, 6)
    check_update(D, table, refs, 128, [0, 0, 2], [100, 100, 200], [101, 101, 200],
                 shapes=((1, torch.float32), (3, torch.float32)), layers=128)
    check_update(D, table, refs, 256, [0, 0, 2], [100, 100, 300], [101, 101, 301],
                 shapes=((1000, torch.float32), (4, torch.float32)), layers=1)


def test_no_pools_and_binding_refusals(D):
    table = [[0, -1], [0, -1]]
    s = State(D, table, counts_of(table, 4), 128)
    D.dsa_pages_update(s.st, dev([0, 1]), dev([100, 100]), dev([101, 101]), None, s.ws)
    assert s.table.tolist() == [[0, -1], [1, -1]]
    with pytest.raises(ValueError):
        D.dsa_pages_update(s.st, dev([0]), dev([100, 100]), dev([101, 101]), None, s.ws)
    with pytest.raises(ValueError):
        D.make_page_pools([torch.zeros(7, device="cuda")], 4)
    with pytest.raises(D.DsaError):   # overlapping, not the same
        big = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
        st = D.make_page_state(big[:2], s.refs, 128)
        D.dsa_pages_update(st, dev([0, 1]), dev([0, 0]), dev([0, 0]), None, s.ws, table_out=big[1:])
