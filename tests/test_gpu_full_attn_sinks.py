"""dsa_full_attn with a window beside which every sequence's first keys stay
visible, against the definition in 64 bits. Keys between the first ones and the
window hold NaN, and blocks of nothing else are unmapped."""
import math

import pytest
import torch

from tests.test_gpu_full_attn import D, HALF_STEP, check, make  # noqa: F401 (D is a fixture)

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "fp16"), ("fp16", "fp16"), ("bf16", "int8"), ("fp16", "int8")]


def unseen(c, b, window, sinks):
    """Keys [a, e) of sequence b that no query sees, between the first ones and the window."""
    n, t, f = c["q_len"][b], c["total_len"][b], c["first_key"][b]
    if n == 0:
        return 0, t
    a, e = min(t, f + sinks), max(f, t - n - window + 1)
    return (a, e) if a < e else (0, 0)


def poison(c, window, sinks):
    for b in range(len(c["q_len"])):
        a, e = unseen(c, b, window, sinks)
        for name in ("k", "v", "k_scale", "v_scale"):
            x = c["pools"][name] if c["block"] else c[name]
            if x is None:
                continue
            bad = 127 if x.dtype == torch.int8 else math.nan
            if not c["block"]:
                x[b, a:e] = bad
                continue
            for t in range(a, e):
                blk = int(c["table"][b, t // c["block"]])
                if blk >= 0:
                    x[blk * c["block"] + t % c["block"]] = bad
        if c["block"]:
            first = -(-a // c["block"])
            c["table"][b, first:max(first, e // c["block"])] = -1
    return c


def reference(c, window, sinks, softcap=0.0, slopes=None):
    """As the plain function of test_gpu_full_attn, vectorised, with the first keys visible."""
    scale = 1 / math.sqrt(128)
    grp, n_all = c["hq"] // c["hkv"], sum(c["q_len"])
    out, mag = (torch.zeros(n_all, c["hq"], 128, dtype=torch.float64, device="cuda") for _ in range(2))
    lse = torch.full((n_all, c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    dz = torch.zeros_like(lse)
    tiny = 2.0 ** -32 / HALF_STEP["fp16"] if c["kvdt"] == "fp16" else 0.0
    n0 = 0
    for b, (n, t, f) in enumerate(zip(c["q_len"], c["total_len"], c["first_key"])):
        if n == 0 or t == 0:
            n0 += n
            continue
        k, v = (c[x][b, :t].cuda().double() for x in ("k", "v"))
        if c["k_scale"] is not None:
            k, v = k * c["k_scale"][b, :t, :, None].cuda().double(), v * c["v_scale"][b, :t, :, None].cuda().double()
        pos = torch.arange(t - n, t, device="cuda")[:, None]
        key = torch.arange(t, device="cuda")[None]
        seen = (key <= pos) & (key >= f) & ((key < f + sinks) | (key > pos - window))
        none = ~seen.any(1)
        k, v = (torch.where(seen.any(0)[:, None, None], x, torch.zeros_like(x)) for x in (k, v))
        for h in range(c["hq"]):
            q = c["q"][n0:n0 + n, h].cuda().double()
            kk, vv = k[:, h // grp], v[:, h // grp]
            z = q @ kk.T * scale
            err = scale * (q.abs() @ kk.abs().T) * 130 * 2.0 ** -24 + z.abs() * 2.0 ** -21
            if softcap:
                z = softcap * torch.tanh(z / softcap)
                err = err + softcap * 2.0 ** -20
            if slopes is not None:
                d = float(slopes[h]) * (key - pos).double()
                z, err = z + d, err + d.abs() * 2.0 ** -22
            zs = z.masked_fill(~seen, 0.0)
            z = z.masked_fill(~seen, -math.inf)
            m = z.amax(1, keepdim=True).masked_fill(none[:, None], 0.0)
            err = (err + (zs.abs().amax(1, keepdim=True) + (zs - m).abs()) * 2.0 ** -22).masked_fill(~seen, 0.0)
            p = (z - m).exp()
            s = p.sum(1, keepdim=True)
            lse[n0:n0 + n, h] = (m + s.log()).view(-1)
            p = torch.where(s > 0, p / s, torch.zeros_like(p))
            out[n0:n0 + n, h], mag[n0:n0 + n, h] = p @ vv, (p + tiny * seen) @ vv.abs()
            dz[n0:n0 + n, h] = (p * err).sum(1) + err.masked_fill(p <= 1e-9, 0.0).amax(1)
        n0 += n
    return tuple(x.cpu().numpy() for x in (out, lse, mag, dz))


def run(D, c, window, sinks, softcap=0.0, slopes=None, out_dtype=None, first=False):  # noqa: F811
    out_dtype = out_dtype or c["qdt"]
    ref = reference(c, window, sinks, softcap, slopes)
    poison(c, window, sinks)
    p = D.make_full_attn_problem(c["q_len"], c["total_len"], c["hq"], c["hkv"], cache_capacity=c["cap"], window=window,
                                 softcap=softcap, first_key=c["first_key"], q_dtype=c["qdt"], kv_dtype=c["kvdt"],
                                 out_dtype=out_dtype)
    src = c["pools"] if c["block"] else c
    dev = [src[n].cuda() if src[n] is not None else None for n in ("k", "v", "k_scale", "v_scale")]
    q = c["q"].cuda()
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[out_dtype]
    out, lse = torch.full(q.shape, 77.0, dtype=dt, device="cuda"), torch.full(q.shape[:2], 77.0, device="cuda")
    pages = D.make_pages(c["table"].cuda(), c["block"], c["nb"]) if c["block"] else None
    ws = D.alloc_full_attn_workspace(p)
    ws.fill_(0xAB)
    D.dsa_full_attn(p, q, *dev, out, ws, slopes=None if slopes is None else slopes.cuda(), lse=lse, pages=pages, sinks=sinks)
    torch.cuda.synchronize()
    assert D.dsa_read_device_status(ws) == 0
    n = sum(c["q_len"])
    assert (out[n:] == 77).all() and (lse[n:] == 77).all(), "rows behind the last sequence changed"
    check(c, out, lse, ref, out_dtype)


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 4), (100, 4), (128, 128), (130, 127), (300, 129), (1, 600), (500, 2000)])
def test_single_tokens(D, q, kv, window, sinks):  # noqa: F811
    """One token on caches from a key to several tiles, the first keys within a tile, a whole one, or more."""
    run(D, make([1] * 7, [1, 2, 128, 129, 500, 1300, 2100], 12, 2, q, kv, block=128, seed=sinks), window, sinks)
    run(D, make([1, 1, 1], [5, 700, 1500], 24, 2, q, kv, seed=window), window, sinks)


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 1), (70, 5), (200, 128), (257, 300), (2000, 3)])
def test_chunks_beside_tokens(D, q, kv, window, sinks):  # noqa: F811
    run(D, make([300, 1, 0, 90, 17], [1500, 1400, 5, 91, 900], 8, 2, q, kv, block=128, seed=window), window, sinks)
    run(D, make([140, 3], [140, 1111], 6, 2, q, kv, seed=sinks), window, sinks, out_dtype="fp32")


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("kw", [dict(softcap=20.0), dict(slopes=True), dict(softcap=5.0, slopes=True)])
def test_caps_and_bias(D, q, kv, kw):  # noqa: F811
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = torch.tensor([2.0 ** (-4 - 0.25 * h) for h in range(12)])
    run(D, make([1, 150, 2], [900, 700, 3], 12, 2, q, kv, block=256, seed=3), 150, 7, **kw)


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("block", [None, 128])
def test_padded_prompts(D, q, kv, block):  # noqa: F811
    """The first keys are counted from first_key; queries below it see nothing."""
    for window, sinks in ((1, 1), (60, 40), (30, 128), (200, 2)):
        run(D, make([3, 100, 2, 300], [1700, 300, 5, 1000], 8, 2, q, kv, block, first_key=[390, 240, 5, 650], seed=sinks),
            window, sinks)


@pytest.mark.parametrize("q,kv", TYPES)
def test_several_tiles_and_segments_a_block(D, q, kv):  # noqa: F811
    """More tiles than thread blocks: runs begin and end among the first keys' tiles and the window's."""
    run(D, make([1] * 40, [9000 - 150 * i for i in range(40)], 8, 2, q, kv, block=128, seed=5), 1500, 300)
    run(D, make([700, 1, 400], [6000, 5000, 1200], 8, 4, q, kv, seed=6, first_key=[100, 0, 37]), 1100, 700)


@pytest.mark.parametrize("kv", ["fp16", "int8"])
def test_zero_first_keys_are_the_window_alone(D, kv):  # noqa: F811
    """sinks = 0, or a window that reaches them, give the other call's bits."""
    c = make([1, 200, 3], [600, 900, 1000], 8, 2, "bf16", kv, block=128, seed=8)
    q, table = c["q"].cuda(), c["table"].cuda()
    dev = [c["pools"][n].cuda() if c["pools"][n] is not None else None for n in ("k", "v", "k_scale", "v_scale")]
    for window, sinks, other in ((300, 0, 300), (1001, 50, 1001), (0, 9, 0)):
        res = []
        for w, s in ((window, sinks), (other, 0)):
            p = D.make_full_attn_problem(c["q_len"], c["total_len"], 8, 2, cache_capacity=c["cap"], window=w, kv_dtype=kv)
            out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
            lib = D.load_library()
            ws = D.alloc_full_attn_workspace(p)
            pages = D.make_pages(table, 128, c["nb"])
            if (w, s) == (window, sinks):   # the entry point itself, sinks = 0 too
                import ctypes
                D._check(lib.dsa_full_attn_sinks(ctypes.byref(p), s, ctypes.byref(pages), q.data_ptr(),
                                                 *[None if x is None else x.data_ptr() for x in dev], None, out.data_ptr(),
                                                 lse.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream))
            else:
                D.dsa_full_attn(p, q, *dev, out, ws, lse=lse, pages=pages)
            res.append((out, lse))
        assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_captured_and_replayed(D):  # noqa: F811
    c = make([1, 1], [3000, 2500], 8, 2, "bf16", "bf16", block=128, seed=9)
    p = D.make_full_attn_problem([1, 1], [3000, 2500], 8, 2, cache_capacity=c["cap"], window=500)
    q, pages = c["q"].cuda(), D.make_pages(c["table"].cuda(), 128, c["nb"])
    k, v = c["pools"]["k"].cuda(), c["pools"]["v"].cuda()
    out, ws = torch.zeros_like(q), D.alloc_full_attn_workspace(p)
    D.dsa_full_attn(p, q, k, v, None, None, out, ws, pages=pages, sinks=4)
    want, g = out.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.dsa_full_attn(p, q, k, v, None, None, out, ws, pages=pages, sinks=4)
    out.zero_()
    ws.fill_(0x55)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and D.dsa_read_device_status(ws) == 0
