"""dsa_rope_axes_append against the formula in 64 bits.

fp32 throughout: the sum of 128 squares (16 a lane, then 3 additions), half of whose
roundings reach the vector, the reciprocal root and two products stay within 2^-20 of
it; a rotated element is off by three roundings of |x cos| + |x' sin| more."""
import numpy as np
import pytest
import torch

from dsa_inputs import quantize_int8

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from top_sparse_attention_chunked_gb300 import build_lib, dsa
    build_lib.build()
    dsa.load_library()
    return dsa


def axis_of(sections, in_turn):
    if not in_turn:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def make(tokens, hq, hkv, sections, q="bf16", seed=0, norm=True, max_pos=5000, angles="fp32", std=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    c = dict(tokens=tokens, hq=hq, hkv=hkv, sections=list(sections), half=sum(sections), qdt=q, max_pos=max_pos, angles=angles)
    width = (hq + 2 * hkv) * 128 + pad
    c["qkv"] = (torch.randn(tokens, width, generator=g) * std).to(DT[q])
    c["split"] = [hq * 128, hkv * 128, hkv * 128]
    # positions beyond the caches are clamped
    c["pos"] = torch.randint(-3, max_pos + 3, (len(sections), tokens), generator=g, dtype=torch.int32)
    ang = torch.arange(max_pos).double()[:, None] * 1e4 ** (-torch.arange(c["half"]).double() / c["half"])
    dt = torch.float32 if angles == "fp32" else torch.bfloat16
    c["cos"], c["sin"] = ang.cos().to(dt), ang.sin().to(dt)
    c["gq"] = 1 + 0.3 * torch.randn(128, generator=g) if norm else None
    c["gk"] = 1 + 0.3 * torch.randn(128, generator=g) if norm else None
    c["rows"] = tokens + 9
    c["slots"] = torch.randperm(c["rows"], generator=g)[:tokens].to(torch.int32)
    c["slots"][1::5] = -1
    c["slots"][3::7] = c["rows"] + 3
    return c


def reference(c, in_turn, eps):
    n, h = c["tokens"], c["half"]
    ax = axis_of(c["sections"], in_turn)
    p = c["pos"].long().clamp(0, c["max_pos"] - 1)[ax].T.numpy()                      # [N, r / 2]
    cos, sin = (c[x].double().numpy()[p, np.arange(h)][:, None] for x in ("cos", "sin"))
    res = []
    parts = c["qkv"][:, :sum(c["split"])].split(c["split"], 1)
    for x, gamma in ((parts[0], c["gq"]), (parts[1], c["gk"])):
        x = x.double().numpy().reshape(n, -1, 128)
        e = 0.0
        if gamma is not None:
            with np.errstate(all="ignore"):
                x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma.double().numpy()
            e = 2.0 ** -20
        a, b = x[..., :h], x[..., h:2 * h]
        y = np.concatenate([a * cos - b * sin, b * cos + a * sin, x[..., 2 * h:]], -1)
        m = np.concatenate([np.abs(a * cos) + np.abs(b * sin), np.abs(b * cos) + np.abs(a * sin), np.abs(x[..., 2 * h:])], -1)
        res.append((y, m * (e + 3 * 2.0 ** -24)))
    return res


def call(D, c, kv, in_turn, eps, in_place=False, q=None):
    """(q_out, K, V, K scales, V scales); the caches start as 77."""
    dev = {n: None if c[n] is None else c[n].cuda() for n in ("cos", "sin", "gq", "gk", "pos", "slots")}
    qkv = c["qkv"].cuda()
    q, k, v = qkv[:, :sum(c["split"])].split(c["split"], 1)
    p = D.make_rope_axes_problem(c["tokens"], c["hq"], c["hkv"], c["rows"], c["sections"], c["max_pos"], in_turn, eps, c["qdt"], kv,
                                 c["angles"])
    out = q if in_place else torch.full((c["tokens"], c["hq"], 128), 9.0, device="cuda").to(DT[c["qdt"]])
    shape = (c["rows"], c["hkv"], 128)
    K, V = (torch.full(shape, 77, device="cuda").to(DT[kv]) for _ in range(2))
    ks, vs = (torch.full(shape[:2], 77.0, device="cuda") if kv == "int8" and c["hkv"] else None for _ in range(2))
    D.dsa_rope_axes_append(p, q if c["hq"] else None, k if c["hkv"] else None, v if c["hkv"] else None, dev["gq"], dev["gk"], dev["cos"],
                           dev["sin"], dev["pos"], dev["slots"] if c["hkv"] else None, out if c["hq"] else None,
                           K if c["hkv"] else None, V if c["hkv"] else None, ks, vs)
    if not in_place:
        assert torch.equal(qkv.cpu(), c["qkv"]), "inputs changed"
    return out.reshape(c["tokens"], c["hq"], 128), K, V, ks, vs, qkv


def run(D, c, kv="bf16", in_turn=False, eps=1e-6):
    out, K, V, ks, vs, _ = call(D, c, kv, in_turn, eps)
    (q, eq), (k, ek) = reference(c, in_turn, eps)
    half = HALF[c["qdt"]]
    sub = 2.0 ** -25 if c["qdt"] == "fp16" else 1e-39
    if c["hq"]:
        assert (np.abs(out.double().cpu().numpy() - q) <= half * (np.abs(q) + eq) + eq + sub).all(), "q"
    if not c["hkv"]:
        return
    slots = c["slots"].long()
    live = (slots >= 0) & (slots < c["rows"])
    at = slots[live]
    rest = torch.ones(c["rows"], dtype=torch.bool)
    rest[at] = False
    K, V = K.cpu(), V.cpu()
    assert (K[rest].float() == 77).all() and (V[rest].float() == 77).all(), "rows that no token has"
    v = c["qkv"][:, :sum(c["split"])].split(c["split"], 1)[2].reshape(c["tokens"], c["hkv"], 128)[live]
    # the rotated keys in q's type, from a cache of it: what the other caches convert
    k16 = (K if kv == c["qdt"] else call(D, c, c["qdt"], in_turn, eps)[1].cpu())[at]
    ref, err = k[live.numpy()], ek[live.numpy()]
    assert (np.abs(k16.double().numpy() - ref) <= half * (np.abs(ref) + err) + err + sub).all(), "k"
    if kv == "int8":
        for x, cache, scale in ((k16, K, ks), (v, V, vs)):
            codes, s = quantize_int8(x.float())
            assert torch.equal(cache[at], codes) and torch.equal(scale.cpu()[at], s)
            assert (scale.cpu()[rest] == 77).all()
    else:
        assert torch.equal(K[at], k16.to(DT[kv])) and torch.equal(V[at], v.to(DT[kv]))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (24, 2), (7, 7), (5, 0), (0, 3), (32, 8), (12, 1), (33, 11)])
@pytest.mark.parametrize("q,kv", [("bf16", "bf16"), ("bf16", "fp16"), ("fp16", "fp16"), ("bf16", "int8"), ("fp16", "int8")])
@pytest.mark.parametrize("tokens", [1, 2, 33])
def test_heads_and_types(D, hq, hkv, q, kv, tokens):
    run(D, make(tokens, hq, hkv, (16, 24, 24), q, seed=hq), kv)


@pytest.mark.parametrize("sections", [(64,), (1,), (3,), (32, 32), (8, 12, 12), (24, 20, 20), (16, 16, 16), (1, 2, 60), (0, 33, 0, 5), (16, 8, 8, 8),
                                      (4, 4), (63,)])
@pytest.mark.parametrize("in_turn", [False, True])
@pytest.mark.parametrize("angles", ["fp32", "bf16"])
def test_sections(D, sections, in_turn, angles):
    for norm in (True, False):
        c = make(50, 6, 2, sections, seed=sum(sections), norm=norm, angles=angles)
        for kv in ("fp16", "int8"):
            run(D, c, kv, in_turn)


@pytest.mark.parametrize("tokens", [1, 7, 8, 300, 3000, 9000])
def test_tokens(D, tokens):
    run(D, make(tokens, 9, 3, (24, 20, 20), seed=tokens), "bf16", True)
    run(D, make(tokens, 2, 1, (5, 6), seed=tokens, pad=8), "bf16", False)


@pytest.mark.parametrize("std,eps", [(1e30, 0.0), (1e-30, 0.0), (1e-30, 1e-6), (2e36, 1e-6), (1e-38, 0.0), (1.0, 1e20)])
def test_large_and_small_vectors(D, std, eps):
    for sections in ((16, 24, 24), (7, 4)):
        run(D, make(20, 4, 2, sections, seed=4, std=std), "bf16", eps=eps)


def test_one_position_for_all_axes(D):
    """Text: positions [N] give what [axes, N] with equal rows gives, and one axis alone."""
    c = make(70, 6, 2, (20, 20, 24), seed=6)
    c["pos"][:] = c["pos"][:1]
    a = call(D, c, "bf16", True, 1e-6)
    full = c["pos"]
    c["pos"] = full[0].contiguous()
    b = call(D, c, "bf16", True, 1e-6)
    c["pos"], c["sections"] = full[:1].contiguous(), [64]
    d = call(D, c, "bf16", False, 1e-6)
    for x, y, z in zip(a[:3], b[:3], d[:3]):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_in_place_in_the_projection(D):
    for sections in ((16, 24, 24), (9,)):
        c = make(100, 8, 2, sections, seed=8, pad=16)
        a, b = call(D, c, "bf16", False, 1e-6), call(D, c, "bf16", False, 1e-6, in_place=True)
        for x, y in zip(a[:3], b[:3]):
            assert torch.equal(x, y)
        assert torch.equal(b[5].cpu()[:, 1024:], c["qkv"][:, 1024:]), "keys, values and what is behind them stay"


def test_text_positions_agree_with_the_fused_prologue(D):
    """One axis, tokens of one length: dsa_rope_append's results to a rounding."""
    B, S, T, hq, hkv = 2, 3, 40, 4, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
    q, qI, k, kI, v = r(B, S, hq, 128), r(B, S, 16, 64), r(B, S, hkv, 128), r(B, S, 64), r(B, S, hkv, 128)
    gam = [1 + 0.2 * torch.randn(n, device="cuda", generator=g) for n in (128, 128, 64, 64)]
    ang = torch.arange(64, device="cuda")[:, None] * 1e4 ** (-torch.arange(64, device="cuda") / 64)
    cos, sin = ang.cos().contiguous(), ang.sin().contiguous()
    K, V = (torch.zeros(B, T, hkv, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    KI = torch.zeros(B, T, 64, device="cuda", dtype=torch.bfloat16)
    K2, V2 = torch.zeros_like(K), torch.zeros_like(V)
    q2 = torch.empty(B * S, hq, 128, device="cuda", dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    slots, pos = torch.empty(B * S, **i32), torch.empty(B * S, **i32)
    D.dsa_slot_map(torch.tensor([S] * B, **i32), torch.tensor([20, 33], **i32), slots, capacity=T, positions=pos)
    p2 = D.make_rope_axes_problem(B * S, hq, hkv, B * T, [64], 64)
    D.dsa_rope_axes_append(p2, q.view(B * S, hq, 128), k.view(B * S, hkv, 128), v.view(B * S, hkv, 128), gam[0], gam[1], cos, sin, pos,
                           slots, q2, K2.view(B * T, hkv, 128), V2.view(B * T, hkv, 128))
    p = D.make_problem(batch=B, q_len=S, total_len=[20, 33], top_k=8, num_q_heads=hq, num_kv_heads=hkv, cache_capacity=T)
    D.dsa_rope_append(p, q, qI, k, kI, v, KI, K, V, None, None, *gam, cos=cos, sin=sin, cos_index=cos[:, ::2].contiguous(),
                      sin_index=sin[:, ::2].contiguous())
    assert torch.equal(V, V2)
    for a, b in ((q.view_as(q2), q2), (K, K2)):
        a, b = a.double(), b.double()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -18).all()        # a step of BF16
        assert (a != b).double().mean() < 0.01


@pytest.mark.parametrize("q", ["bf16", "fp16"])
def test_codes_are_the_appends(D, q):
    """Values and unturned keys as codes: dsa_cache_append's, bit for bit, at scales of every size."""
    B, S, hkv = 1, 20000, 3
    dt = torch.bfloat16 if q == "bf16" else torch.float16
    g = torch.Generator(device="cuda").manual_seed(17)
    k, v = (torch.randn(B, S, hkv, 128, device="cuda", generator=g) for _ in range(2))
    low, high = (-130, 100) if q == "bf16" else (-20, 10)
    v *= torch.exp2(torch.randint(low, high, (B, S, hkv, 1), device="cuda", generator=g).float())
    k[:, ::5] = torch.randint(-200, 200, (B, S // 5, hkv, 128), device="cuda", generator=g).float() / 2     # many ties
    v[:, 7] = 0
    k, v = k.to(dt), v.to(dt)
    new = lambda *s, t: torch.full(s, 9, device="cuda", dtype=t)
    K, V, K2, V2 = (new(B, S, hkv, 128, t=torch.int8) for _ in range(4))
    ks, vs, ks2, vs2 = (new(B, S, hkv, t=torch.float32) for _ in range(4))
    p = D.make_problem(batch=B, q_len=S, total_len=[S], top_k=8, num_q_heads=hkv, num_kv_heads=hkv, cache_capacity=S, q_dtype=q, kv_dtype="int8")
    D.dsa_cache_append(p, new(B, S, 64, t=torch.bfloat16), k, v, new(B, S, 64, t=torch.bfloat16), K, V, ks, vs)
    p2 = D.make_rope_axes_problem(S, 0, hkv, S, [64], 4, q_dtype=q, kv_dtype="int8")
    i32 = dict(dtype=torch.int32, device="cuda")
    D.dsa_rope_axes_append(p2, None, k.view(S, hkv, 128), v.view(S, hkv, 128), None, None, torch.ones(4, 64, device="cuda"),
                           torch.zeros(4, 64, device="cuda"), torch.zeros(S, **i32), torch.arange(S, **i32), None, K2.view(S, hkv, 128),
                           V2.view(S, hkv, 128), ks2.view(S, hkv), vs2.view(S, hkv))
    assert torch.equal(vs, vs2) and torch.equal(ks, ks2)
    assert torch.equal(V, V2) and torch.equal(K, K2)


def test_captured_and_replayed_on_new_inputs(D):
    c, c2 = make(64, 8, 2, (16, 24, 24), seed=1), make(64, 8, 2, (16, 24, 24), seed=2)
    want = call(D, c2, "fp16", False, 1e-6)
    dev = {n: c[n].cuda() for n in ("cos", "sin", "gq", "gk", "pos", "slots", "qkv")}
    q, k, v = dev["qkv"].split(c["split"], 1)
    p = D.make_rope_axes_problem(64, 8, 2, c["rows"], c["sections"], c["max_pos"], kv_dtype="fp16")
    out = torch.zeros(64, 8, 128, device="cuda", dtype=torch.bfloat16)
    K, V = (torch.full((c["rows"], 2, 128), 77, device="cuda").half() for _ in range(2))
    args = (p, q, k, v, dev["gq"], dev["gk"], dev["cos"], dev["sin"], dev["pos"], dev["slots"], out, K, V)
    D.dsa_rope_axes_append(*args)
    assert D.dsa_last_launches() == ["rope_axes_append_kernel"]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.dsa_rope_axes_append(*args)
    for n in ("gq", "gk", "pos", "slots", "qkv"):
        dev[n].copy_(c2[n])
    K.fill_(77), V.fill_(77)
    g.replay()
    for x, y in zip((out, K, V), want):
        assert torch.equal(x, y)
