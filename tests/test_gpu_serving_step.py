"""Beam search on a paged cache, the calls together as a server makes them:
prompt, fork, then append, full attention, selection and page update every
step, with compaction in between. Each step is held against the same search in
64 bits, from the tokens alone."""
import math

import numpy as np
import pytest
import torch

from dsa_inputs import DTYPES, quantize_int8

pytestmark = pytest.mark.gpu

HQ, HKV, BLOCK, VOCAB, PAD = 8, 2, 128, 1501, 3
BATCH, BEAMS, STEPS, ENDED = 2, 3, 70, 40            # a token below ENDED ends its beam
ROWS = BATCH * BEAMS
PROMPT = (200, 131)


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from top_sparse_attention_chunked_gb300 import build_lib, dsa
    build_lib.build()
    dsa.load_library()
    return dsa


class Tables:
    """A model without layers: a token's query, key and value, and the output's projection."""

    def __init__(self, kv):
        g = torch.Generator().manual_seed(5)
        self.q, self.k, self.v = ((torch.randn(VOCAB, h, 128, generator=g) * s).half()
                                  for h, s in ((HQ, 1.5), (HKV, 1.0), (HKV, 1.0)))
        self.w = torch.randn(HQ * 128, VOCAB, generator=g) * 0.2
        k, v = self.k.double(), self.v.double()
        if kv == "int8":
            (kc, ks), (vc, vs) = (quantize_int8(x.float()) for x in (self.k, self.v))
            k, v = kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None]
        self.kd, self.vd, self.qd, self.wd = k.numpy(), v.numpy(), self.q.double().numpy(), self.w.double().numpy()
        # roundings of the weights in the second product: FP16, or a BF16 pair
        self.step = 2.0 ** -16 if kv == "int8" else 2.0 ** -11

    def logits(self, hist):
        """(logits of what follows the tokens `hist`, their bound, attention output, sum of |weight * value|)"""
        t = np.asarray(hist)
        out, mag = np.zeros((HQ, 128)), np.zeros((HQ, 128))
        for h in range(HQ):
            k, v, q = self.kd[t, h // (HQ // HKV)], self.vd[t, h // (HQ // HKV)], self.qd[t[-1], h]
            z = k @ q / math.sqrt(128)
            # fp32 products and sums of 128 terms; the exponent in units of log2 e
            err = (np.abs(k) @ np.abs(q)) / math.sqrt(128) * 130 * 2.0 ** -24 + np.abs(z).max() * 2.0 ** -20
            p = np.exp(z - z.max())
            p /= p.sum()
            out[h], mag[h] = p @ v, (p @ np.abs(v)) * (1.01 * self.step + 2.5 * err.max() + 2.0 ** -19) + \
                np.abs(v).sum(0) * 2.0 ** -32        # (FP16's smallest step, per key)
        x, e = out.reshape(-1), mag.reshape(-1)
        # the projection: fp32 products and sums of 1,024 terms
        bound = e @ np.abs(self.wd) + np.abs(x) @ np.abs(self.wd) * 1026 * 2.0 ** -24
        return x @ self.wd, bound, out, mag


def log_softmax(x):
    return x - (x.max() + math.log(np.exp(x - x.max()).sum()))


@pytest.mark.parametrize("kv", ["fp16", "int8"])
def test_beam_search_on_pages(D, kv):
    m = Tables(kv)
    dev = "cuda"
    nb, width = 24, 3
    cap = width * BLOCK
    int8 = kv == "int8"
    pools = [torch.zeros(nb * BLOCK, HKV, 128, dtype=DTYPES[kv], device=dev) for _ in range(2)]
    scales = [torch.zeros(nb * BLOCK, HKV, device=dev) if int8 else None for _ in range(2)]
    kI = torch.zeros(nb * BLOCK, 64, dtype=torch.bfloat16, device=dev)
    table = torch.full((ROWS, width), -1, dtype=torch.int32, device=dev)
    refs = torch.zeros(nb, dtype=torch.int32, device=dev)
    state = D.make_page_state(table, refs, BLOCK)
    move = D.make_page_pools(pools + [s for s in scales if s is not None] + [kI], nb)
    pages = D.make_pages(table, BLOCK, nb)
    pws = D.alloc_pages_workspace(state)
    wq, wk, wv, ww = m.q.to(dev), m.k.to(dev), m.v.to(dev), m.w.to(dev)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def ok(ws):
        assert D.dsa_read_device_status(ws) == 0

    def append(total, tokens):
        """The tokens [B, S] of the table's first B rows, whose lengths with them are `total`."""
        b, s = tokens.shape
        p = D.make_problem(b, s, total, 16, HQ, HKV, cache_capacity=cap, q_dtype="fp16", kv_dtype=kv)
        D.dsa_cache_append(p, torch.zeros(b, s, 64, dtype=torch.bfloat16, device=dev), wk[tokens], wv[tokens], kI, *pools,
                           *scales, pages=pages)

    def attend(q_len, total, tokens):
        p = D.make_full_attn_problem(q_len, total, HQ, HKV, cap, q_dtype="fp16", kv_dtype=kv, out_dtype="fp32")
        ws = D.alloc_full_attn_workspace(p)
        out = torch.empty(len(tokens), HQ, 128, device=dev)
        D.dsa_full_attn(p, wq[tokens], *pools, *scales, out, ws, pages=pages)
        ok(ws)
        return out

    # prompts: rows 0 and 1 are given their blocks, written and read
    g = torch.Generator().manual_seed(9)
    prompts = [torch.randint(ENDED, VOCAB, (n,), generator=g).tolist() for n in PROMPT]
    grow = list(PROMPT) + [0] * (ROWS - BATCH)
    D.dsa_pages_update(state, i32([-1] * ROWS), i32([0] * ROWS), i32(grow), move, pws)
    ok(pws)
    for b in range(BATCH):
        one = D.make_pages(table[b:b + 1], BLOCK, nb)
        p = D.make_problem(1, PROMPT[b], PROMPT[b], 16, HQ, HKV, cache_capacity=cap, q_dtype="fp16", kv_dtype=kv)
        t = torch.tensor(prompts[b], device=dev)
        D.dsa_cache_append(p, torch.zeros(1, PROMPT[b], 64, dtype=torch.bfloat16, device=dev), wk[t][None], wv[t][None], kI,
                           *pools, *scales, pages=one)
    both = torch.tensor(prompts[0] + prompts[1], device=dev)
    out = attend(list(PROMPT) + [0] * (ROWS - BATCH), grow, both)
    last = out[torch.tensor(np.cumsum(PROMPT) - 1, device=dev)]
    logits = (last.reshape(BATCH, -1) @ ww).repeat_interleave(BEAMS, 0).contiguous()
    # every beam starts from its prompt's row; the first counts, the others have score -infinity
    keep = [PROMPT[r // BEAMS] for r in range(ROWS)]
    D.dsa_pages_update(state, i32([r // BEAMS for r in range(ROWS)]), i32(keep), i32(keep), move, pws)
    ok(pws)
    assert torch.equal(refs[table[0, :2].long()], i32([BEAMS] * 2))     # shared, not copied
    scores = torch.full((ROWS,), -math.inf, device=dev)
    scores[::BEAMS] = 0.0
    hist = [list(prompts[r // BEAMS]) for r in range(ROWS)]
    total64 = [0.0 if r % BEAMS == 0 else -math.inf for r in range(ROWS)]
    slack = [0.0] * ROWS                                               # what the totals may be off by
    ended = [False] * ROWS

    bp = D.make_beam_problem(BATCH, BEAMS, VOCAB, BEAMS, "fp32", pad_token=PAD)
    bws = D.alloc_beam_workspace(bp)
    tokens = torch.empty(BATCH, BEAMS, dtype=torch.int32, device=dev)
    parents = torch.empty_like(tokens)
    copied = torch.empty(2, dtype=torch.int32, device=dev)
    moves = forks = 0
    for step in range(STEPS):
        # the same step in 64 bits, for every beam
        cand, cand_err = [], []
        for r in range(ROWS):
            lg, err, _, _ = m.logits(hist[r])
            if ended[r]:
                c, e = np.full(VOCAB, -np.inf), np.full(VOCAB, slack[r])
                c[PAD] = total64[r]
            else:
                c, e = total64[r] + log_softmax(lg), slack[r] + err + err.max() + 2.0 ** -18
            cand.append(c)
            cand_err.append(e)
        D.dsa_beam_select(bp, logits, scores, scores.view(BATCH, BEAMS), tokens, parents, bws,
                          finished=torch.tensor(ended, device=dev))
        ok(bws)
        tk, pr, sc = tokens.flatten().tolist(), parents.flatten().tolist(), scores.tolist()
        new_total, new_slack = [], []
        for b in range(BATCH):
            rows = range(b * BEAMS, (b + 1) * BEAMS)
            picked = [(pr[r], tk[r]) for r in rows]
            assert len(set(picked)) == BEAMS and all(p in rows for p, _ in picked)
            every = np.concatenate([cand[r] for r in rows])
            best = np.sort(every)[::-1][BEAMS - 1]
            worst_err = max(e.max() for e in (cand_err[r] for r in rows))
            for r, (p, t) in zip(rows, picked):
                assert abs(sc[r] - cand[p][t]) <= cand_err[p][t] + abs(cand[p][t]) * 2.0 ** -23
                assert cand[p][t] >= best - 2 * worst_err          # among the best, as far as it can be told
                new_total.append(cand[p][t])
                new_slack.append(cand_err[p][t] + abs(cand[p][t]) * 2.0 ** -23)
            assert sc[rows[0]:rows[-1] + 1] == sorted(sc[rows[0]:rows[-1] + 1], reverse=True)
        # (the 64-bit search follows the choices, so that near ties do not part the two)
        ended = [ended[pr[r]] or tk[r] < ENDED for r in range(ROWS)]
        hist = [hist[pr[r]] + [tk[r]] for r in range(ROWS)]
        total64, slack = new_total, new_slack
        length = [len(h) for h in hist]
        D.dsa_pages_update(state, parents.flatten(), i32([n - 1 for n in length]), i32(length), move, pws, counts=copied)
        ok(pws)
        forks += int(copied[0])
        if step % 16 == 7:
            D.dsa_pages_compact(state, move, pws, counts=copied)
            ok(pws)
            moves += int(copied[0])
        held = table[table >= 0].long()
        assert torch.equal(torch.bincount(held, minlength=nb).int(), refs)
        now = tokens.flatten().long()
        append(length, now[:, None])
        out = attend([1] * ROWS, length, now)
        logits = out.reshape(ROWS, -1) @ ww
    assert forks > BATCH * (BEAMS - 1)
    # what the sparse step reads on the same pages, with every key selected
    sp = D.make_problem(ROWS, 1, length, cap, HQ, HKV, cache_capacity=cap, q_dtype="fp16", kv_dtype=kv, out_dtype="fp32")
    sws = D.alloc_workspace(sp, D.DSA_OP_DECODE)
    sparse = torch.empty(ROWS, 1, HQ, 128, device=dev)
    D.dsa_sparse_attn_decode(sp, wq[now][:, None], torch.zeros(ROWS, 1, 16, 64, dtype=torch.bfloat16, device=dev),
                             torch.zeros(ROWS, 1, 16, device=dev), kI, *pools, *scales,
                             torch.empty(ROWS, 1, cap, dtype=torch.int32, device=dev), sparse, sws, pages=pages)
    for r in range(ROWS):
        _, _, o, tol = m.logits(hist[r])
        assert (np.abs(out[r].double().cpu().numpy() - o) <= tol + 1e-30).all()
        # (its weights have 16 bits of whatever type: half a step of BF16, twice)
        diff = np.abs(sparse[r, 0].double().cpu().numpy() - o)
        assert (diff <= tol + 2.0 ** -7 * np.abs(m.vd[np.asarray(hist[r])]).max()).all()


def calls(D, seed, kv="bf16"):
    """One of each call with its own tensors: [(call, outputs)], nothing run yet."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    res = []
    nb, table = 40, torch.randperm(40, device="cuda", generator=g)[:24].int().view(4, 6).contiguous()
    k, v = ((rnd(nb * 128, 2, 128).to(DTYPES[kv]) if kv != "int8" else
             torch.randint(-127, 128, (nb * 128, 2, 128), device="cuda", generator=g, dtype=torch.int8)) for _ in range(2))
    ks, vs = (rnd(nb * 128, 2).abs() * 0.02 if kv == "int8" else None for _ in range(2))
    p = D.make_full_attn_problem([1, 40, 0, 3], [700, 768, 5, 300], 8, 2, 768, window=500, kv_dtype=kv)
    q, out, ws = rnd(44, 8, 128).bfloat16(), rnd(44, 8, 128).bfloat16(), D.alloc_full_attn_workspace(p)
    lse, pages = rnd(44, 8), D.make_pages(table, 128, nb)
    res.append((lambda: D.dsa_full_attn(p, q, k, v, ks, vs, out, ws, lse=lse, pages=pages), [out, lse]))

    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    refs[table.flatten().long()] = 1
    state = D.make_page_state(table, refs, 128)
    pool = rnd(nb, 128, 8)
    pws, arr = D.alloc_pages_workspace(state), D.make_page_pools([pool], nb)
    t2, r2 = torch.empty_like(table), torch.empty_like(refs)
    par, keep, new = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 0, 3, 3], [700, 650, 20, 768], [701, 768, 21, 768]))
    # (not in place: the state stays, so a repeated call has the same to do; what is copied goes to free blocks)
    res.append((lambda: D.dsa_pages_update(state, par, keep, new, arr, pws, table_out=t2, refs_out=r2), [t2, r2, pool]))
    t3, r3, remap, cws = torch.empty_like(table), torch.empty_like(refs), torch.empty_like(refs), D.alloc_pages_workspace(state)
    res.append((lambda: D.dsa_pages_compact(state, None, cws, table_out=t3, refs_out=r3, remap=remap), [t3, r3, remap]))

    bp = D.make_beam_problem(2, 4, 30011, 8)
    x, s = rnd(8, 30011).bfloat16(), rnd(8)
    o = [torch.empty(2, 8, device="cuda")] + [torch.empty(2, 8, dtype=torch.int32, device="cuda") for _ in range(2)]
    bws = D.alloc_beam_workspace(bp)
    res.append((lambda: D.dsa_beam_select(bp, x, s, *o, bws), o))
    return res


def results(cs):
    torch.cuda.synchronize()
    return [[o.clone() for o in outs] for _, outs in cs]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for p, q in zip(a, b) for x, y in zip(p, q))


def first_call_is_captured(kv):
    """Run in a process of its own: nothing of the library has run before the capture."""
    from top_sparse_attention_chunked_gb300 import build_lib, dsa
    build_lib.build()
    torch.zeros(1, device="cuda")
    cs = calls(dsa, 3, kv)
    torch.cuda.synchronize()
    graphs = []
    for call, _ in cs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for _ in range(3):
        for gr in graphs:
            gr.replay()
        got = results(cs)
    for call, _ in cs:
        call()
    assert same(got, results(cs))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_first_call_inside_a_capture(D, kv):
    import subprocess
    import sys
    subprocess.run([sys.executable, "-c", f"import sys; sys.path[:0] = {sys.path!r}\n"
                    f"import test_gpu_serving_step as t; t.first_call_is_captured({kv!r})"], check=True, timeout=600)


@pytest.mark.parametrize("kv", ["bf16", "fp16", "int8"])
def test_two_streams_at_once(D, kv):
    """Two sets of the calls with their own workspaces, eager and replayed, on two streams at a time."""
    sets = [calls(D, 3, kv), calls(D, 4, kv)]
    for cs in sets:
        for call, _ in cs:
            call()
    want = [results(cs) for cs in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    for cs, s in zip(sets, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            for call, _ in cs:
                call()
    for replay in (False, True):
        for cs in sets:
            for _, outs in cs:
                for o in outs[:2]:        # (not the pool)
                    o.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for cs, s, gr in zip(sets, streams, graphs):
                with torch.cuda.stream(s):
                    if replay:
                        gr.replay()
                    else:
                        for call, _ in cs:
                            call()
        assert [same(results(cs), w) for cs, w in zip(sets, want)] == [True, True]
