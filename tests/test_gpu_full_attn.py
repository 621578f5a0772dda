"""dsa_full_attn against the definition in 64 bits: element by element within
a bound made of the roundings the call is documented to take."""
import math

import numpy as np
import pytest
import torch

from dsa_inputs import DTYPES, quantize_int8

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from top_sparse_attention_chunked_gb300 import build_lib, dsa
    build_lib.build()
    dsa.load_library()
    return dsa


def make(q_len, total_len, hq, hkv, q="bf16", kv="bf16", block=None, first_key=None, seed=0, spare=2,
         q_std=1.5, extra=3):
    """Inputs on the CPU; whatever no query sees is NaN (16-bit), 127 with NaN scales (INT8), or an
    unmapped block. block: the paged pool's block size (None: a dense cache)."""
    g = torch.Generator().manual_seed(seed)
    B, cap = len(q_len), max(max(total_len), 1)
    if block:
        cap = -(-cap // block) * block
    first_key = first_key or [0] * B
    c = dict(q_len=list(q_len), total_len=list(total_len), first_key=list(first_key), hq=hq, hkv=hkv, qdt=q,
             kvdt=kv, cap=cap, block=block)
    c["q"] = (torch.randn(sum(q_len) + extra, hq, 128, generator=g) * q_std).to(DTYPES[q])
    for n in ("k", "v"):
        x = torch.randn(B, cap, hkv, 128, generator=g)
        if kv == "int8":
            c[n], c[n + "_scale"] = quantize_int8(x)
        else:
            c[n], c[n + "_scale"] = x.to(DTYPES[kv]), None
    for b in range(B):
        for a, e in ((0, first_key[b]), (total_len[b], cap)):
            for n in ("k", "v"):
                if kv == "int8":
                    c[n][b, a:e] = 127
                    c[n + "_scale"][b, a:e] = math.nan
                else:
                    c[n][b, a:e] = math.nan
    if block:
        need = [-(-t // block) for t in total_len]
        nb = sum(need) + spare
        order = torch.randperm(nb, generator=g).tolist()
        table = torch.full((B, cap // block), -1, dtype=torch.int32)
        pools = {}
        for n in ("k", "v", "k_scale", "v_scale"):
            if c[n] is None:
                pools[n] = None
                continue
            pools[n] = torch.full((nb * block,) + tuple(c[n].shape[2:]), 127 if c[n].dtype == torch.int8 else math.nan,
                                  dtype=c[n].dtype)
        i = 0
        for b in range(B):
            for j in range(need[b]):
                x, i = order[i], i + 1
                if (j + 1) * block <= first_key[b]:
                    continue              # a block that was given back: -1
                table[b, j] = x
                for n, pool in pools.items():
                    if pool is not None:
                        pool[x * block:(x + 1) * block] = c[n][b, j * block:(j + 1) * block]
        c["pools"], c["table"], c["nb"] = pools, table, nb
    return c


def reference(c, window=0, softcap=0.0, slopes=None, scale=None):
    """(out, lse, bound of out, bound of lse) in 64 bits, [N, Hq, ...]."""
    scale = scale or 1 / math.sqrt(128)
    grp = c["hq"] // c["hkv"]
    n_all = sum(c["q_len"])
    out, mag = np.zeros((n_all, c["hq"], 128)), np.zeros((n_all, c["hq"], 128))
    lse, dz = np.full((n_all, c["hq"]), -np.inf), np.zeros((n_all, c["hq"]))
    # an FP16 weight below 2^-14 is rounded to a multiple of 2^-24, off by 2^-25 at most; the weight at the
    # maximum is taken as 2^7 or more and their sum is no less, so a key's share of the output is off by up
    # to 2^-32 |v| beside the relative half step that `check` counts
    tiny = 2.0 ** -32 / HALF_STEP["fp16"] if c["kvdt"] == "fp16" else 0.0
    n0 = 0
    for b, (n, t) in enumerate(zip(c["q_len"], c["total_len"])):
        k, v = (c[x][b, :t].double().numpy() for x in ("k", "v"))
        if c["k_scale"] is not None:
            k = k * c["k_scale"][b, :t].double().numpy()[..., None]
            v = v * c["v_scale"][b, :t].double().numpy()[..., None]
        for i in range(n):
            pos = t - n + i
            lo = max(c["first_key"][b], pos - window + 1 if window else 0)
            if lo > pos:
                continue
            for h in range(c["hq"]):
                q = c["q"][n0 + i, h].double().numpy()
                kk, vv = k[lo:pos + 1, h // grp], v[lo:pos + 1, h // grp]
                z = kk @ q * scale
                # fp32 products and sums of 128 terms, a few roundings of the result
                err = scale * (np.abs(kk) @ np.abs(q)) * 130 * 2.0 ** -24 + np.abs(z) * 2.0 ** -21
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                    err = err + softcap * 2.0 ** -20      # tanh to 2^-20 of its range
                if slopes is not None:
                    d = float(slopes[h]) * (np.arange(lo, pos + 1) - pos)
                    z = z + d
                    err = err + np.abs(d) * 2.0 ** -22
                m = z.max()
                # the exponent is formed in units of log2 e from logits of this size
                err = err + (np.abs(z).max() + np.abs(z - m)) * 2.0 ** -22
                p = np.exp(z - m)
                lse[n0 + i, h] = m + math.log(p.sum())
                p /= p.sum()
                out[n0 + i, h], mag[n0 + i, h] = p @ vv, (p + tiny) @ np.abs(vv)
                dz[n0 + i, h] = (p * err).sum() + err[p > 1e-9].max()
        n0 += n
    return out, lse, mag, dz


def check(c, got, lse, ref, out_dtype):
    """The weights enter the second product in 16 bits: half a step of the type it is taken in, FP16 for an
    FP16 cache, a BF16 pair for an FP16 query on an INT8 cache, BF16 otherwise; the statistics are off by their logits' error, 2^-21 for the exponential."""
    out, lse_ref, mag, dz = ref
    u_p = HALF_STEP["fp16"] if c["kvdt"] == "fp16" else HALF_STEP["bf16"]
    if c["kvdt"] == "int8" and c["qdt"] == "fp16":
        u_p = HALF_STEP["bf16"] ** 2                # a BF16 pair
    tol = HALF_STEP[out_dtype] * np.abs(out) + mag * (1.01 * u_p + 2.5 * dz[..., None] + 2.0 ** -19) + 1e-30
    if out_dtype == "fp16":
        tol = tol + 2.0 ** -25                      # its smallest step
    g = got.double().cpu().numpy()[:out.shape[0]]
    bad = ~(np.abs(g - out) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside; first {np.argwhere(bad)[0]}: "
                           f"{g[tuple(np.argwhere(bad)[0])]} for {out[tuple(np.argwhere(bad)[0])]}")
    gl = lse.double().cpu().numpy()[:out.shape[0]]
    none = np.isinf(lse_ref)
    assert (gl[none] == -np.inf).all() and (g[none] == 0).all(), "a query that sees no key"
    err = np.abs(gl - np.where(none, 0, lse_ref))[~none]
    assert (err <= (dz + 2.0 ** -19 + np.abs(np.where(none, 0, lse_ref)) * 2.0 ** -21)[~none]).all(), "lse"


def call(D, c, window=0, softcap=0.0, slopes=None, out_dtype=None, scale=0.0, ws=None):
    out_dtype = out_dtype or c["qdt"]
    p = D.make_full_attn_problem(c["q_len"], c["total_len"], c["hq"], c["hkv"], cache_capacity=c["cap"],
                                 window=window, softcap=softcap, first_key=c["first_key"], q_dtype=c["qdt"],
                                 kv_dtype=c["kvdt"], out_dtype=out_dtype, softmax_scale=scale)
    src = c["pools"] if c["block"] else c
    dev = {n: (src[n].cuda() if src[n] is not None else None) for n in ("k", "v", "k_scale", "v_scale")}
    q = c["q"].cuda()
    out = torch.full(q.shape, 77.0, dtype=DTYPES[out_dtype], device="cuda")
    lse = torch.full(q.shape[:2], 77.0, device="cuda")
    pages = D.make_pages(c["table"].cuda(), c["block"], c["nb"]) if c["block"] else None
    ws = ws if ws is not None else D.alloc_full_attn_workspace(p)
    ws.fill_(0xAB)
    D.dsa_full_attn(p, q, dev["k"], dev["v"], dev["k_scale"], dev["v_scale"], out, ws,
                    slopes=None if slopes is None else slopes.cuda(), lse=lse, pages=pages)
    torch.cuda.synchronize()
    assert D.dsa_read_device_status(ws) == 0
    n = sum(c["q_len"])
    assert (out[n:] == 77).all() and (lse[n:] == 77).all(), "rows behind the last sequence changed"
    return out, lse, dict(p=p, q=q, dev=dev, pages=pages)


def run(D, c, **kw):
    out, lse, _ = call(D, c, **kw)
    ref_kw = {k: v for k, v in kw.items() if k in ("window", "softcap", "slopes", "scale")}
    check(c, out, lse, reference(c, **ref_kw), kw.get("out_dtype") or c["qdt"])


@pytest.mark.parametrize("total", [1, 2, 15, 127, 128, 129, 255, 257, 1000, 4097])
@pytest.mark.parametrize("block", [None, 128, 256])
def test_single_token_lengths(D, total, block):
    run(D, make([1], [total], 8, 2, block=block, seed=total))


@pytest.mark.parametrize("q,kv", [("bf16", "bf16"), ("bf16", "fp16"), ("fp16", "fp16"), ("bf16", "int8"),
                                  ("fp16", "int8")])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (24, 2), (7, 7), (40, 2), (130, 1)])
def test_types_and_heads(D, q, kv, hq, hkv):
    run(D, make([1, 0, 5, 2], [300, 17, 261, 2], hq, hkv, q, kv, block=128, seed=hq + hkv))
    run(D, make([3, 1], [140, 1], hq, hkv, q, kv, seed=hq))


@pytest.mark.parametrize("q_len,total", [([64], [64]), ([200], [200]), ([129], [1000]), ([33, 1, 0, 90], [33, 700, 5, 391]),
                                         ([300, 17], [301, 1040])])
@pytest.mark.parametrize("kv", ["bf16", "fp16", "int8"])
def test_chunks(D, q_len, total, kv):
    run(D, make(q_len, total, 6, 2, "bf16", kv, block=128, seed=sum(q_len)))
    run(D, make(q_len, total, 4, 4, "bf16", kv, seed=sum(total)))


@pytest.mark.parametrize("out_dtype", ["bf16", "fp16", "fp32"])
def test_output_types(D, out_dtype):
    run(D, make([4, 150], [260, 150], 8, 2, "bf16", "fp16", block=256), out_dtype=out_dtype)


@pytest.mark.parametrize("q_len,total", [([1], [700]), ([90, 3], [300, 1111])])
@pytest.mark.parametrize("kw", [dict(), dict(window=150, softcap=5.0)])
def test_fp16_query_on_int8_keeps_fp16_precision(D, q_len, total, kw):
    c = make(q_len, total, 12, 2, "fp16", "int8", block=128, seed=17)
    run(D, c, out_dtype="fp32", **kw)
    run(D, c, **kw)


@pytest.mark.parametrize("kv", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("q_len,total", [([1], [600]), ([140], [700]), ([3, 260], [900, 260])])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=130), dict(softcap=2.0), dict(softcap=50.0),
                                dict(slopes=True), dict(window=257, softcap=20.0, slopes=True), dict(scale=0.5)])
def test_window_cap_bias(D, kv, q_len, total, kw):
    c = make(q_len, total, 12, 2, "bf16", kv, block=128, seed=5)
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = torch.tensor([2.0 ** (-0.5 * h) for h in range(12)])
    run(D, c, **kw)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("block", [None, 128])
def test_first_key_and_rows_that_see_nothing(D, kv, block):
    # the second sequence's first 40 queries see no key, the third sequence's none at all; blocks below
    # the first key are unmapped
    c = make([3, 100, 2], [700, 300, 5], 8, 2, "bf16", kv, block, first_key=[390, 240, 5])
    run(D, c)
    run(D, c, window=70)


@pytest.mark.parametrize("q,kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp16"), ("fp16", "int8")])
@pytest.mark.parametrize("kw", [dict(softcap=200.0), dict(softcap=30.0), dict(softcap=12.0), dict(softcap=7.0), dict(softcap=1e4),
                                dict(softcap=0.01), dict(softcap=40.0, scale=0.6), dict(softcap=0.05, scale=1e-4)])
def test_caps_from_narrow_to_wide(D, q, kv, kw):
    """Arguments of the cap in each range that it is formed in, and scales far below it."""
    run(D, make([1, 150], [600, 300], 8, 2, q, kv, block=128, seed=12), out_dtype="fp32", **kw)


@pytest.mark.parametrize("kv", ["fp16", "int8"])
@pytest.mark.parametrize("q_len,total,first", [([2, 1], [5, 130], [5, 0]), ([2], [5], [5]), ([1, 3, 1], [7, 9, 300], [7, 9, 300]),
                                               ([2, 1, 2], [5, 9000, 4], [5, 0, 4])])
def test_leading_sequences_that_see_nothing(D, kv, q_len, total, first):
    run(D, make(q_len, total, 8, 2, "bf16", kv, 128, first_key=first))


def test_nothing_to_do(D):
    c = make([0, 0], [5, 0], 8, 2)
    out, lse, _ = call(D, c)
    p = D.make_full_attn_problem([0], [0], 8, 2, cache_capacity=1)
    assert D.dsa_full_attn_workspace_size(p) > 0


def test_large_and_small_queries(D):
    """A BF16 query far outside FP16's range on an FP16 cache, and one far below it."""
    c = make([2, 3], [400, 131], 8, 2, "bf16", "fp16", block=128)
    c["q"] = (c["q"].float() * 2.0 ** 17).to(torch.bfloat16)
    run(D, c, scale=2.0 ** -20)
    c["q"] = (c["q"].float() * 2.0 ** -50).to(torch.bfloat16)
    run(D, c, scale=2.0 ** 28)


def test_large_scales_int8(D):
    c = make([2, 3], [400, 131], 8, 2, "bf16", "int8", block=128)
    for n, f in (("k_scale", 2.0 ** 10), ("v_scale", 2.0 ** 60)):
        c[n] *= f
        c["pools"][n] *= f
    run(D, c, scale=2.0 ** -14, out_dtype="fp32")


def test_peaked_softmax_rescales(D):
    """Logits that grow along the cache by far more than a 16-bit weight can hold."""
    c = make([1, 140], [1500, 1400], 8, 2, "fp16", "fp16", seed=3, q_std=1.0)
    ramp = torch.linspace(0, 60, c["cap"])[None, :, None, None]
    c["k"] = (torch.sign(c["k"].float()) * 0.02 + ramp * 0.05).to(torch.float16)
    for b, t in enumerate(c["total_len"]):
        c["k"][b, t:] = math.nan
    c["q"] = c["q"].abs()
    run(D, c)


@pytest.mark.parametrize("q_len,total", [([1], [700]), ([4, 150], [300, 411])])
@pytest.mark.parametrize("kv", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("scale", [0.0, 1e-6, 1e-38])
def test_zero_queries(D, q_len, total, kv, scale):
    """Rows of zeros, and of BF16's smallest numbers, beside ordinary ones: even weights, under masks too."""
    c = make(q_len, total, 8, 2, "bf16", kv, block=128, seed=3)
    c["q"][:, ::2] = 0
    c["q"][:, 1] = 2.0 ** -133
    run(D, c, scale=scale, window=300)


@pytest.mark.parametrize("q", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,n", [(1, 1, 1), (8, 8, 1), (15, 1, 1), (16, 2, 2), (16, 1, 1), (17, 1, 1), (32, 2, 1), (34, 2, 1)])
def test_few_rows_int8(D, q, hq, hkv, n):
    """Up to 16 rows and just above, many sequences: whole items and parts in every block."""
    g = torch.Generator().manual_seed(hq)
    total = [n] + (torch.randint(n, 2600, (22,), generator=g)).tolist() + [2600]
    run(D, make([n] * 24, total, hq, hkv, q, "int8", block=256, seed=hq))
    run(D, make([n] * 24, total, hq, hkv, q, "int8", seed=n), window=300, softcap=9.0,
        slopes=torch.tensor([2.0 ** (-0.3 * h) for h in range(hq)]))


@pytest.mark.parametrize("n", [1, 3, 40])
def test_peaked_softmax_rescales_int8(D, n):
    c = make([n], [1500], 8, 2, "bf16", "int8", seed=3, q_std=1.0)
    c["k"] = torch.where(c["k"] == 127, c["k"], c["k"].abs().clamp(1, 90))
    c["k_scale"] = torch.linspace(1e-4, 3e-2, c["cap"])[None, :, None].repeat(1, 1, 2).contiguous()
    c["v_scale"] = (c["v_scale"] * torch.exp2(torch.linspace(-9, 9, c["cap"]))[None, :, None]).contiguous()
    c["q"] = c["q"].abs()
    run(D, c, out_dtype="fp32")


def test_dense_equals_paged(D):
    for kv in ("fp16", "int8"):
        c = make([5, 200], [900, 333], 24, 2, "bf16", kv, block=256, seed=9)
        paged = call(D, c)
        dense = call(D, dict(c, block=None))
        assert torch.equal(paged[0], dense[0]) and torch.equal(paged[1], dense[1])


def test_repeats_are_bit_identical(D):
    c = make([8, 1, 300], [9000, 4000, 2000], 24, 2, "bf16", "fp16", block=256, seed=4)
    out, lse, st = call(D, c)
    ws = D.alloc_full_attn_workspace(st["p"])
    for _ in range(20):
        o, s = torch.empty_like(out), torch.empty_like(lse)
        D.dsa_full_attn(st["p"], st["q"], st["dev"]["k"], st["dev"]["v"], None, None, o, ws, lse=s, pages=st["pages"])
        n = sum(c["q_len"])
        assert torch.equal(o[:n], out[:n]) and torch.equal(s[:n], lse[:n])


def test_captured_and_replayed_on_new_values(D):
    c = make([4, 130], [5000, 700], 24, 2, "bf16", "bf16", block=256, seed=8)
    out, lse, st = call(D, c)
    ws = D.alloc_full_attn_workspace(st["p"])
    o = torch.empty_like(out)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        D.dsa_full_attn(st["p"], st["q"], st["dev"]["k"], st["dev"]["v"], None, None, o, ws, pages=st["pages"])
    q0 = st["q"].clone()
    for scale in (1.0, 0.25):
        st["q"].copy_(q0 * scale)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(out)
        D.dsa_full_attn(st["p"], st["q"], st["dev"]["k"], st["dev"]["v"], None, None, want, D.alloc_full_attn_workspace(st["p"]),
                        pages=st["pages"])
        n = sum(c["q_len"])
        torch.cuda.synchronize()
        assert torch.equal(o[:n], want[:n])


def test_two_streams_with_their_own_workspaces(D):
    cs = [make([2, 60], [3000, 500], 24, 2, "bf16", "fp16", block=256, seed=s) for s in (1, 2)]
    want = [call(D, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    wss = [D.alloc_full_attn_workspace(w[2]["p"]) for w in want]
    outs = [torch.empty_like(w[0]) for w in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for w, s, ws, o in zip(want, streams, wss, outs):
            st = w[2]
            D.dsa_full_attn(st["p"], st["q"], st["dev"]["k"], st["dev"]["v"], None, None, o, ws, pages=st["pages"], stream=s)
    torch.cuda.synchronize()
    for c, w, o in zip(cs, want, outs):
        n = sum(c["q_len"])
        assert torch.equal(o[:n], w[0][:n])


def test_bad_block_entry_is_reported_not_followed(D):
    from top_sparse_attention_chunked_gb300.dsa import DSA_ERR_INVALID_ARG, DsaError
    c = make([1], [300], 8, 2, block=128)
    c["table"][0, 1] = c["nb"] + 5
    c["pools"]["k"].fill_(0.5)
    c["pools"]["v"].fill_(0.5)
    p = D.make_full_attn_problem([1], [300], 8, 2, cache_capacity=c["cap"])
    ws = D.alloc_full_attn_workspace(p)
    out = torch.empty(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    D.dsa_full_attn(p, c["q"].cuda(), c["pools"]["k"].cuda(), c["pools"]["v"].cuda(), None, None, out, ws,
                    pages=D.make_pages(c["table"].cuda(), 128, c["nb"]))
    with pytest.raises(DsaError) as e:
        D.dsa_read_device_status(ws)
    assert e.value.status == DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("kv,heads", [("fp16", 8), ("int8", 8)])
def test_rows_beyond_32_bit_offsets(D, kv, heads):
    """A pool of over 2^31 elements whose last blocks hold the sequence."""
    bs, nb = 256, 8400 + 3                            # 8,403 * 256 * 8 * 128 = 2.2e9 elements
    c = make([2], [600], 16, heads, "bf16", kv, block=bs, seed=6, spare=0)
    table = torch.tensor([[nb - 1, nb - 3, nb - 2]], dtype=torch.int32)
    dev = {}
    for n in ("k", "v", "k_scale", "v_scale"):
        if c[n] is None:
            dev[n] = None
            continue
        dev[n] = torch.zeros((nb * bs,) + tuple(c[n].shape[2:]), dtype=c[n].dtype, device="cuda")
        for j in range(3):
            x = int(table[0, j])
            dev[n][x * bs:(x + 1) * bs] = c[n][0, j * bs:(j + 1) * bs].cuda()
    p = D.make_full_attn_problem([2], [600], 16, heads, cache_capacity=c["cap"], q_dtype="bf16", kv_dtype=kv)
    ws = D.alloc_full_attn_workspace(p)
    q = c["q"].cuda()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    D.dsa_full_attn(p, q, dev["k"], dev["v"], dev["k_scale"], dev["v_scale"], out, ws, lse=lse,
                    pages=D.make_pages(table.cuda(), bs, nb))
    torch.cuda.synchronize()
    check(c, out, lse, reference(c), "bf16")


def test_binding_refusals(D):
    c = make([2], [300], 8, 2)
    p = D.make_full_attn_problem([2], [300], 8, 2)
    ws = D.alloc_full_attn_workspace(p)
    q, k, v = c["q"].cuda(), c["k"].cuda(), c["v"].cuda()
    out = torch.empty_like(q)
    with pytest.raises(ValueError):
        D.dsa_full_attn(p, q[:1], k, v, None, None, out, ws)
    with pytest.raises(ValueError):
        D.dsa_full_attn(p, q, k.half(), v, None, None, out, ws)
    with pytest.raises(ValueError):
        D.dsa_full_attn(p, c["q"], k, v, None, None, out, ws)
    with pytest.raises(D.DsaError):
        D.dsa_full_attn(p, q, k, v, None, None, out, ws[:64])
