"""dsa_sample against the definition in 64 bits: the same token, and its log
probability to fp32 rounding.

Weights are right to 2^-31 of themselves, so a draw (or a cut) that falls within that
much of a border between two tokens may go either way; the references check that
theirs does not."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NEAR = 2.0 ** -29        # of the sum: nearer to a border than this a case says nothing


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from top_sparse_attention_chunked_gb300 import build_lib, dsa
    build_lib.build()
    dsa.load_library()
    return dsa


def reference(x, u, heat, k, p, low):
    """(token, log probability, distance from the nearest border, of the sum) of one row in 64 bits."""
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1, -np.inf, 1.0
    if not heat > 0 or top == np.inf:
        return int(x.argmax()), 0.0, 1.0
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        w = np.exp((x - top) / heat) if np.isfinite(heat) else np.where(x > -np.inf, 1.0, 0.0)
    order = np.argsort(-x, kind="stable")
    ranked = w[order]
    n, near = len(x), 1.0
    if k > 0:
        n = min(n, k)
    if p < 1:
        c = np.cumsum(ranked[:n])
        need = p * c[-1]
        cut = min(int(np.searchsorted(c, need, side="left")) + 1, n)
        border = [b for b in (cut - 2, cut - 1) if 0 <= b < n - 1]
        exact = float(need).is_integer() and (ranked == ranked[0])[:n].all()      # whole numbers on both sides
        if border and not exact:
            near = min(abs(c[b] - need) for b in border) / c[-1]
        n = cut
    if low > 0:
        n = min(n, max(1, int((ranked >= min(low, 1.0)).sum())))
    kept = np.zeros(len(x))
    kept[order[:n]] = w[order[:n]]
    c = np.cumsum(kept)
    t = min(max(u, 0.0), 1 - 2.0 ** -24) * c[-1]
    tok = int(np.searchsorted(c, t, side="right"))
    if u > 0:      # (0 is the first token that is kept)
        near = min(near, abs(c[tok] - t) / c[-1], abs(c[tok] - kept[tok] - t) / c[-1] if c[tok] > kept[tok] else 1.0)
    return tok, math.log(kept[tok] / c[-1]), near


def run(D, logits, u, heat=None, k=None, p=None, low=None, least=0.9):
    """logits: CPU tensor [rows, vocab], any strides. The share of rows that are away from a border is `least` or more."""
    n, v = logits.shape
    name = {t: s for s, t in DT.items()}[logits.dtype]
    dev = logits.cuda() if logits.is_contiguous() else torch.empty_strided(
        (logits.untyped_storage().nbytes() // logits.element_size(),), (1,), dtype=logits.dtype, device="cuda")
    if not logits.is_contiguous():
        flat = torch.empty(0, dtype=logits.dtype).set_(logits.untyped_storage())
        dev = flat.cuda().as_strided(logits.shape, logits.stride(), logits.storage_offset())
    plan = D.make_sample_problem(n, v, name, row_stride=logits.stride(0) if n > 1 else 0)
    f = lambda t, dt: None if t is None else torch.as_tensor(t, dtype=dt).expand(n).contiguous().cuda()
    args = dict(temperature=f(heat, torch.float32), top_k=f(k, torch.int32), top_p=f(p, torch.float32), min_p=f(low, torch.float32))
    tok, lp = torch.full((n,), -9, dtype=torch.int32, device="cuda"), torch.full((n,), 9.0, device="cuda")
    uu = f(u, torch.float32)
    D.dsa_sample(plan, dev, uu, tok, logprobs=lp, **args)
    only = torch.full_like(tok, -9)
    D.dsa_sample(plan, dev, uu, only, **args)
    assert torch.equal(tok, only)
    get = lambda t, d: d if t is None else t.tolist()
    rows = zip(logits.double().numpy(), uu.tolist(), get(args["temperature"], [1.0] * n), get(args["top_k"], [0] * n),
               get(args["top_p"], [1.0] * n), get(args["min_p"], [0.0] * n))
    sure = 0
    for i, row in enumerate(rows):
        want, wlp, near = reference(*row)
        if near < NEAR:
            continue
        sure += 1
        assert int(tok[i]) == want, (i, int(tok[i]), want, near, row[1:])
        got = float(lp[i])
        # w / sum to 2^-30, a few roundings of the logarithm and of (x - max) / T
        assert got == wlp or abs(got - wlp) <= 2.0 ** -29 + abs(wlp) * 2.0 ** -21, (i, got, wlp)
    # (a row of 40,000 tokens is near one with a probability of 2 x 40,000 x 2^-29 = 1.5e-4: one of a call's may be)
    assert sure >= least * n - 1, f"{sure} of {n} rows say something"


def logits_of(rows, vocab, dtype="fp32", std=2.0, seed=0, peaks=20):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * std
    for r in range(rows):
        at = torch.randperm(vocab, generator=g)[:peaks]
        x[r, at] += 3 + 7 * torch.rand(len(at), generator=g)
    return x.to(DT[dtype])


def uniform(n, seed=0):
    return torch.rand(n, generator=torch.Generator().manual_seed(1000 + seed))


SETTINGS = [dict(), dict(heat=0.7), dict(heat=0.0), dict(k=1), dict(k=40), dict(k=3000), dict(p=0.9), dict(p=0.3, heat=1.7), dict(p=0.999),
            dict(low=0.05), dict(k=50, p=0.95, low=0.02, heat=0.8), dict(k=5000, p=0.99, heat=2.5), dict(low=1.0), dict(p=0.0)]


@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 64, 257, 1000, 4096, 5003, 32000, 50257])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_sizes(D, vocab, dtype):
    for i, s in enumerate(SETTINGS):
        run(D, logits_of(5, vocab, dtype, seed=vocab + i, peaks=min(vocab, 20)), uniform(5, i), **s)


@pytest.mark.parametrize("rows,vocab,dtype", [(1, 131072, "bf16"), (3, 262144, "fp32"), (40, 131075, "bf16"), (160, 20000, "fp32"), (2, 524288, "fp32"),
                                              (2, 524287, "bf16"), (9, 262144, "fp16"), (80, 100000, "bf16")])
def test_long_rows_and_many(D, rows, vocab, dtype):
    """From one block a row to clusters of sixteen."""
    x = logits_of(rows, vocab, dtype, seed=rows)
    for i, s in enumerate(SETTINGS if rows < 20 else SETTINGS[::3]):
        run(D, x, uniform(rows, i), **s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("std,heat", [(0.01, 1.0), (1.0, 3.0), (0.3, 0.1), (20.0, 1.0), (1e-3, 1e-3), (300.0, 10.0), (1.0, 1e30), (5.0, 1e-6), (1e4, 1.0), (1e30, 1e29)])
def test_flat_and_steep_rows(D, dtype, std, heat):
    """Wide nuclei, many ties, logits far from 0 and temperatures of every size."""
    x = logits_of(8, 40000, dtype, std=std, seed=2, peaks=0)
    if std == 1.0:
        x = (x.float() + 900).to(DT[dtype])
    for i, s in enumerate((dict(), dict(p=0.9), dict(k=30000), dict(k=700, p=0.5), dict(k=20000, p=0.7, low=1e-3), dict(p=0.2))):
        run(D, x, uniform(8, i), heat=heat, **s)


@pytest.mark.parametrize("rows,vocab,dtype,std", [(48, 131072, "bf16", 1.6), (48, 131072, "fp32", 1.3), (24, 262144, "fp16", 2.5), (60, 65536, "bf16", 0.8)])
def test_cuts_among_many_tokens_of_like_weight(D, rows, vocab, dtype, std):
    """Nuclei that end where a 32nd of a factor of two holds some 500 to 2,000 tokens, at every place within one."""
    x = logits_of(rows, vocab, dtype, std=std, seed=vocab + rows, peaks=5)
    for i, (a, b) in enumerate(((0.2, 0.95), (0.6, 0.7))):
        p = a + (b - a) * uniform(rows, 40 + i)
        run(D, x, uniform(rows, i), p=p)
        run(D, x, uniform(rows, 9 + i), p=p, k=torch.where(torch.arange(rows) % 2 == 0, vocab, vocab // 3), low=1e-4)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab,offset,step,heat", [(60000, 500.0, 2.0, 0.7), (233039, 0.0, 1.5, 1.0), (30000, -300.0, 4.0, 1.3), (90000, 8.0, 0.25, 0.2)])
def test_cuts_next_to_the_border_of_a_heavy_value(D, dtype, vocab, offset, step, heat):
    """A few values that thousands of tokens share, far apart, and cuts a little above and below where one's tokens end."""
    g = torch.Generator().manual_seed(vocab)
    x = ((torch.randn(vocab, generator=g) * 1.2).round() * step + offset).to(DT[dtype])
    x[:: 10] = torch.finfo(DT[dtype]).min
    v, n = x.double().unique(return_counts=True)
    w = ((v - v[-1]) / heat).exp() * n
    ends = (w.flip(0).cumsum(0) / w.sum())[1:5]
    p = torch.tensor([float(e) + d for e in ends for d in (1e-3, 1e-4, 1.5e-5, 2e-6, 3e-7, -3e-7, -2e-6, -1.5e-5, -1e-4, -1e-3)]).clamp(max=0.99999)
    x = x.expand(len(p), vocab).contiguous()
    run(D, x, uniform(len(p), 3), heat=heat, p=p, least=0.3)
    run(D, x, uniform(len(p), 4), heat=heat, p=p, k=vocab - 5, least=0.3)


def test_rows_of_equal_logits(D):
    """Ties go to the lower index, in top-k, in top-p and with the cut inside a tie."""
    for vocab in (10, 1000, 70000, 300000):
        x = torch.zeros(6, vocab)
        for s in (dict(), dict(k=7), dict(k=vocab // 2 + 1), dict(p=0.5), dict(p=0.25, k=vocab // 3 + 1), dict(low=1.0), dict(p=1e-9)):
            run(D, x, torch.tensor([0.0, 0.1, 0.5, 0.51, 0.999, 0.9999999]), **s, least=0.3)
        x[:, ::3] = 1.0
        x[:, 1::7] = -1.5
        for s in (dict(k=vocab // 5 + 1), dict(p=0.5), dict(p=0.8), dict(k=vocab // 2, p=0.9)):
            run(D, x, torch.tensor([0.01, 0.1, 0.5, 0.51, 0.999, 0.99]), **s, least=0.3)


def test_masks_infinities_and_nan(D):
    x = logits_of(9, 6000, "fp32", seed=4)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 1:] = -math.inf                      # one token left
    x[3, :5990] = -math.inf
    x[4, 17], x[4, 90] = math.inf, math.inf   # the lowest of them
    x[5, ::2] = math.nan
    x[6] = torch.finfo(torch.float32).min     # a mask of the type's lowest value, on every token
    x[7, 100:] = torch.finfo(torch.float32).min
    x[8, :] = -math.inf
    x[8, 5999] = -3e38
    for i, s in enumerate(SETTINGS):
        run(D, x, uniform(9, i), **s)
    for dt in ("bf16", "fp16"):
        y = x[[0, 1, 2, 3, 5]].to(DT[dt])
        for i, s in enumerate(SETTINGS):
            run(D, y, uniform(5, i), **s)
        z = torch.full((2, 3000), torch.finfo(DT[dt]).min).to(DT[dt])
        z[1, 7:9] = 1.0
        run(D, z, uniform(2), k=40, p=0.9)


def test_settings_of_every_row_and_odd_values(D):
    n = 24
    x = logits_of(n, 9001, "bf16", seed=6)
    heat = torch.tensor([1.0, 0.5, 0.0, -1.0, math.nan, 2.0, 1e-20, 1e20, math.inf, 0.9, 1.0, 1.0] * 2)
    k = torch.tensor([0, -5, 3, 3, 3, 9001, 9002, 2 ** 31 - 1, 9000, 40, 1, 2] * 2)
    p = torch.tensor([1.0, 2.0, 0.5, 0.5, 0.5, math.nan, 0.9, 0.9, 1.0, 0.4, 0.9, -1.0] * 2)
    low = torch.tensor([0.0, -1.0, 0.1, 0.1, 0.1, 0.2, 0.0, 0.0, math.nan, 0.5, 3.0, 0.0] * 2)
    u = uniform(n)
    u[:3] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0])
    p_ref = torch.where(p.isnan(), 1.0, p)
    low_ref = torch.where(low.isnan(), 0.0, low)
    run(D, x, u, heat, k, p_ref, low_ref)
    # NaN of top_p and min_p: off
    f = [t.cuda() for t in (heat, k.int(), p, low, p_ref, low_ref, u)]
    plan = D.make_sample_problem(n, 9001, "bf16")
    a, b = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    D.dsa_sample(plan, x.cuda(), f[6], a, temperature=f[0], top_k=f[1], top_p=f[2], min_p=f[3])
    D.dsa_sample(plan, x.cuda(), f[6], b, temperature=f[0], top_k=f[1], top_p=f[4], min_p=f[5])
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab,stride,off", [(5001, 5003, 1), (5000, 5008, 8), (131, 140, 3), (40001, 40001, 5)])
def test_strides_and_offsets(D, dtype, vocab, stride, off):
    """Rows at any alignment; what lies around them is NaN."""
    flat = torch.full((6 * stride + off + 9,), math.nan).to(DT[dtype])
    x = flat.as_strided((6, vocab), (stride, 1), off)
    x.copy_(logits_of(6, vocab, dtype, seed=off))
    for i, s in enumerate(SETTINGS):
        run(D, x, uniform(6, i), **s)


def test_draws_follow_the_probabilities(D):
    """A grid of random numbers gives every token its share."""
    x = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5]).expand(20000, 5).contiguous()
    u = (torch.arange(20000) + 0.5) / 20000
    plan = D.make_sample_problem(20000, 5, "fp32")
    tok = torch.empty(20000, dtype=torch.int32, device="cuda")
    D.dsa_sample(plan, x.cuda(), u.cuda(), tok)
    share = torch.bincount(tok.cpu().long(), minlength=5).double() / 20000
    assert (share - torch.softmax(x[0].double(), 0)).abs().max() <= 1.01 / 20000


def test_captured_and_on_another_stream(D):
    x, u = logits_of(12, 32000, "bf16", seed=8).cuda(), uniform(12).cuda()
    f = dict(temperature=torch.full((12,), 0.8, device="cuda"), top_k=torch.full((12,), 50, dtype=torch.int32, device="cuda"),
             top_p=torch.full((12,), 0.9, device="cuda"))
    plan = D.make_sample_problem(12, 32000, "bf16")
    a, la = torch.zeros(12, dtype=torch.int32, device="cuda"), torch.zeros(12, device="cuda")
    D.dsa_sample(plan, x, u, a, logprobs=la, **f)
    assert D.dsa_last_launches() == ["sample_kernel"]
    want, wl = a.clone(), la.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.dsa_sample(plan, x, u, a, logprobs=la, **f)
    a.zero_(), la.zero_()
    g.replay()
    assert torch.equal(a, want) and torch.equal(la, wl)
    st, b = torch.cuda.Stream(), torch.zeros_like(a)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(20):
            D.dsa_sample(plan, x, u, b, **f)
    for _ in range(20):
        D.dsa_sample(plan, x, u, a, **f)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
