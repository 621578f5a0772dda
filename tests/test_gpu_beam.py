"""dsa_beam_select against the definition in 64 bits: the same tokens and
parents, in the same order, and scores within fp32 rounding."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from top_sparse_attention_chunked_gb300 import build_lib, dsa
    build_lib.build()
    dsa.load_library()
    return dsa


def reference(logits, scores, batch, beams, select, finished=None, pad=0):
    """logits [batch * beams, V], scores [batch * beams] in fp64 (numpy)."""
    V = logits.shape[1]
    out = np.full((batch, select), -np.inf), np.full((batch, select), -1), np.full((batch, select), -1)
    for b in range(batch):
        vals, places = [], []
        for i in range(beams):
            r = b * beams + i
            x = logits[r]
            if finished is not None and finished[r]:
                t = np.full(V, -np.inf)
                t[pad] = scores[r]
            else:
                m = x.max()
                with np.errstate(all="ignore"):
                    lse = m + math.log(np.exp(x - m).sum()) if np.isfinite(m) else np.nan
                    t = x + (scores[r] - lse)
            keep = np.nonzero(t > -np.inf)[0]
            keep = keep[np.argsort(-t[keep], kind="stable")][:select]
            vals.append(t[keep])
            places.append(i * V + keep)
        v, p = np.concatenate(vals), np.concatenate(places)
        order = np.lexsort((p, -v))[:select]
        n = len(order)
        out[0][b, :n], out[1][b, :n], out[2][b, :n] = v[order], p[order] % V, b * beams + p[order] // V
    return out


def run(D, logits, scores, batch, beams, select, finished=None, pad=0, exact=True):
    """logits: a CUDA tensor [batch * beams, V], rows any stride apart."""
    V = logits.shape[1]
    name = {v: k for k, v in DT.items()}[logits.dtype]
    p = D.make_beam_problem(batch, beams, V, select, name, pad_token=pad, row_stride=logits.stride(0) if logits.shape[0] > 1 else 0)
    ws = D.alloc_beam_workspace(p)
    ws.fill_(0xEE)
    outs = (torch.full((batch, select), 7.0, device="cuda"), torch.full((batch, select), 7, dtype=torch.int32, device="cuda"),
            torch.full((batch, select), 7, dtype=torch.int32, device="cuda"))
    D.dsa_beam_select(p, logits, scores, *outs, ws, finished=finished)
    torch.cuda.synchronize()
    assert D.dsa_read_device_status(ws) == 0
    ref = reference(logits.double().cpu().numpy(), scores.double().cpu().numpy(), batch, beams, select,
                    None if finished is None else finished.cpu().numpy(), pad)
    got = [o.cpu().numpy() for o in outs]
    np.testing.assert_array_equal(got[1], ref[1])
    np.testing.assert_array_equal(got[2], ref[2])
    fin = np.isfinite(ref[0])
    assert (got[0][~fin] == -np.inf).all()
    # one rounding to fp32, and sums of exponentials good to 2^-20
    assert (np.abs(got[0][fin] - ref[0][fin]) <= np.abs(ref[0][fin]) * 2.0 ** -24 + 2.0 ** -20).all()
    return outs


def rand(n, V, dtype, seed, std=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.randn(n, V, device="cuda", generator=g) * std).to(DT[dtype]),
            -4 * torch.rand(n, device="cuda", generator=g))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("batch,beams,V,select", [(1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 7, 4), (1, 4, 100, 8), (3, 5, 1001, 10),
                                                  (1, 1, 4096, 64), (2, 64, 513, 64), (7, 2, 50001, 4), (1, 64, 9000, 64),
                                                  (1, 4, 131072, 8), (5, 1, 70001, 1), (40, 8, 3001, 16)])
def test_sizes(D, dtype, batch, beams, V, select):
    x, s = rand(batch * beams, V, dtype, V + beams)
    run(D, x, s, batch, beams, select)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ties_go_to_the_lower_place(D, dtype):
    for V in (300, 20000):
        x = torch.zeros(6, V, dtype=DT[dtype], device="cuda")
        run(D, x, torch.zeros(6, device="cuda"), 2, 3, 40)           # all equal, all beams alike
        g = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randint(0, 3, (6, V), device="cuda", generator=g).to(DT[dtype])
        x[3:] = x[:3]
        s = torch.tensor([0.0, -1.0, 0.0, 0.0, -1.0, 0.0], device="cuda")
        x[2], x[5] = x[0], x[0]                                       # beam 2 is beam 0 again
        run(D, x, s, 2, 3, 64)


def test_ascending_and_descending_rows(D):
    V = 30000
    up = torch.arange(V, device="cuda", dtype=torch.float32) * 1e-3
    run(D, torch.stack([up, up.flip(0)]), torch.tensor([0.0, -0.5], device="cuda"), 1, 2, 64)


def test_masked_tokens_and_beams(D):
    V = 9001
    x, s = rand(8, V, "fp32", 3)
    x[0] = -math.inf                       # nothing allowed
    x[1, 5:] = -math.inf                   # five tokens allowed, the rest of the row (whole slices) masked
    x[2, :-3] = -math.inf
    x[3] = torch.finfo(torch.float32).min  # masked with the type's lowest value: all alike
    x[4, 17] = math.nan
    x[5, 8999] = math.inf
    s[6] = -math.inf
    s[7] = math.nan
    run(D, x, s, 1, 8, 16)
    run(D, x, s, 8, 1, 16)
    run(D, x, s, 2, 4, 64)


def test_first_step_has_one_live_beam(D):
    x, _ = rand(4, 32000, "bf16", 9)
    x[1:] = x[0]
    run(D, x, torch.tensor([0.0] + [-math.inf] * 3, device="cuda"), 1, 4, 8)


def test_finished_beams(D):
    for dtype in ("bf16", "fp32"):
        x, s = rand(12, 5003, dtype, 11)
        f = torch.tensor([0, 1, 0, 1, 1, 1, 0, 0, 0, 0, 0, 7], dtype=torch.uint8, device="cuda")
        s[3] = -math.inf
        x[1] = math.nan                    # a finished beam's logits are not looked at
        run(D, x, s, 3, 4, 8, finished=f, pad=2)
        run(D, x, s, 4, 3, 6, finished=f, pad=5002)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("off,stride", [(0, 5001), (1, 5003), (3, 5008), (7, 6000)])
def test_strides_and_alignment(D, dtype, off, stride):
    buf = torch.full((off + 6 * stride,), math.nan, dtype=DT[dtype], device="cuda")
    x = buf[off:off + 6 * stride].view(6, stride)[:, :4999]
    v, s = rand(6, 4999, dtype, off)
    x.copy_(v)
    run(D, x, s, 2, 3, 12)


def test_large_magnitudes(D):
    x, s = rand(4, 3001, "fp32", 4, std=1e4)
    run(D, x, s - 1e5, 1, 4, 8)
    x, s = rand(4, 3001, "fp32", 5, std=1e-4)
    run(D, x, s * 1e-3, 1, 4, 8)


def test_captured_and_repeated(D):
    x, s = rand(16, 40001, "bf16", 21)
    outs = run(D, x, s, 2, 8, 16)
    p = D.make_beam_problem(2, 8, 40001, 16, "bf16")
    ws = D.alloc_beam_workspace(p)
    got = tuple(torch.empty_like(o) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.dsa_beam_select(p, x, s, *got, ws)
    for _ in range(20):
        for o in got:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs))


def test_binding_refusals(D):
    x, s = rand(4, 100, "bf16", 1)
    p = D.make_beam_problem(1, 4, 100, 8)
    ws = D.alloc_beam_workspace(p)
    o = (torch.empty(1, 8, device="cuda"), torch.empty(1, 8, dtype=torch.int32, device="cuda"),
         torch.empty(1, 8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        D.dsa_beam_select(p, x.half(), s, *o, ws)
    with pytest.raises(ValueError):
        D.dsa_beam_select(p, x[:, ::2], s, *o, ws)
    with pytest.raises(ValueError):
        D.dsa_beam_select(p, x, s[:3], *o, ws)
    with pytest.raises(D.DsaError):
        D.dsa_beam_select(p, x, s, *o, ws[:256])


def test_scores_in_place(D):
    x, s = rand(24, 9001, "bf16", 31)
    want = run(D, x, s, 4, 6, 6)
    p = D.make_beam_problem(4, 6, 9001, 6)
    o = tuple(torch.empty_like(w) for w in want[1:])
    D.dsa_beam_select(p, x, s, s.view(4, 6), *o, D.alloc_beam_workspace(p))
    assert torch.equal(s.view(4, 6), want[0]) and torch.equal(o[0], want[1]) and torch.equal(o[1], want[2])
    with pytest.raises(D.DsaError):
        D.dsa_beam_select(p, x, s, want[0], s.view(torch.int32).view(4, 6), o[1], D.alloc_beam_workspace(p))
