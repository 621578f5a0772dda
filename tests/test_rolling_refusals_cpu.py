"""Host-side refusals of the calls for packed steps with rolling caches: bad
arguments and overlaps are refused before CUDA is touched."""
import ctypes

import pytest

from tests.test_serving_calls_cpu import D, full  # noqa: F401 (D is a fixture)


def fine(D):  # noqa: F811
    """What a valid call gives without a GPU; with one, valid calls on these addresses are not made."""
    import torch
    return None if torch.cuda.is_available() else D.DSA_ERR_NO_DEVICE


def expect(D, got, want):  # noqa: F811
    assert got == want, D.load_library().dsa_last_error_string().decode()


def call_sinks(D, p, sinks=4, pages=None, **kw):  # noqa: F811
    v = dict(q=0x1000000, k=0x2000000, v=0x3000000, ks=None, vs=None, slopes=None, out=0x4000000, lse=None, ws=0x10000, n=1 << 40)
    v.update(kw)
    return D.load_library().dsa_full_attn_sinks(ctypes.byref(p), sinks, None if pages is None else ctypes.byref(pages),
                                                *[v[n] for n in ("q", "k", "v", "ks", "vs", "slopes", "out", "lse", "ws", "n")], None)


def test_sinks(D):  # noqa: F811
    p = full(D, window=50)
    assert call_sinks(D, p, -1) == D.DSA_ERR_INVALID_ARG
    assert "sinks" in D.load_library().dsa_last_error_string().decode()
    assert call_sinks(D, p, q=0) == D.DSA_ERR_INVALID_ARG
    assert call_sinks(D, p, out=0x4000008) == D.DSA_ERR_MISALIGNED
    assert call_sinks(D, p, ws=None) == D.DSA_ERR_WORKSPACE
    assert call_sinks(D, full(D, window=-1)) == D.DSA_ERR_INVALID_ARG
    assert call_sinks(D, p, pages=D.DsaKvPages(64, 10, 8, 0x7000)) == D.DSA_ERR_UNSUPPORTED
    if fine(D):
        for sinks in (0, 1, 300, 2 ** 31 - 1):
            assert call_sinks(D, p, sinks) == D.DSA_ERR_NO_DEVICE
            # the other call's workspace is enough, whatever the number
            assert call_sinks(D, p, sinks, n=D.dsa_full_attn_workspace_size(p)) == D.DSA_ERR_NO_DEVICE


@pytest.mark.parametrize("window", [0, 1, 200, 5000])
def test_workspace_holds_any_number_of_first_keys(D, window):  # noqa: F811
    if not fine(D):
        pytest.skip("makes valid calls on addresses that are none")
    for q_len, total in (([1], [1]), ([1], [9000]), ([1] * 40, [300 * i + 1 for i in range(40)]), ([700, 3], [6000, 100])):
        p = full(D, q_len=q_len, total_len=total, cache_capacity=12032, window=window)
        for sinks in (0, 1, 128, 700, 20000):
            assert call_sinks(D, p, sinks, n=D.dsa_full_attn_workspace_size(p)) == D.DSA_ERR_NO_DEVICE


def call_slots(D, rows=4, tokens=100, pages=None, cap=64, **kw):  # noqa: F811
    v = dict(q=0x1000, t=0x2000, slots=0x3000, pos=0x4000, row=0x5000, first=0x6000)
    v.update(kw)
    return D.load_library().dsa_slot_map(rows, tokens, None if pages is None else ctypes.byref(pages), cap,
                                         *[v[n] for n in ("q", "t", "slots", "pos", "row", "first")], None)


def test_slot_map(D):  # noqa: F811
    bad = D.DSA_ERR_INVALID_ARG
    for kw in (dict(rows=0), dict(rows=4097), dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(cap=0), dict(rows=4096, cap=1 << 20), dict(q=None),
               dict(t=None), dict(slots=None), dict(pos=0x3000), dict(row=0x3000 + 396), dict(first=0x5000 + 396), dict(slots=0x1004), dict(first=0x2000 - 16),
               dict(pages=(128, 10, 0, 0x7000)), dict(pages=(1 << 20, 10, 1 << 20, 0x7000)), dict(pages=(128, 10, 4, None)),
               dict(pages=(128, 10, 4, 0x3000 - 60)), dict(pages=(0, 10, 4, 0x7000))):
        if "pages" in kw:
            kw["pages"] = D.DsaKvPages(*kw["pages"])
        assert call_slots(D, **kw) == bad, kw
    assert call_slots(D, pages=D.DsaKvPages(96, 10, 4, 0x7000)) == D.DSA_ERR_UNSUPPORTED
    assert call_slots(D, q=0x1002) == D.DSA_ERR_MISALIGNED
    assert call_slots(D, tokens=0, slots=None, pos=None, row=None, first=None) == D.DSA_OK
    if fine(D):
        for kw in (dict(), dict(pos=None, row=None, first=None), dict(pages=D.DsaKvPages(128, 10, 4, 0x7000), cap=0), dict(tokens=0)):
            expect(D, call_slots(D, **kw), D.DSA_ERR_NO_DEVICE)


def axes_problem(D, **kw):  # noqa: F811
    a = dict(tokens=10, num_q_heads=4, num_kv_heads=2, cache_rows=100, sections=[16, 24, 24], max_pos=50)
    fields = {k: kw.pop(k) for k in list(kw) if k.endswith("_stride") or k in ("axes", "sections_raw")}
    a.update(kw)
    p = D.make_rope_axes_problem(**a)
    for k, v in fields.items():
        if k == "sections_raw":
            for i, x in enumerate(v):
                p.sections[i] = x
        else:
            setattr(p, k, v)
    return p


def call_axes(D, p, **kw):  # noqa: F811
    v = dict(q=0x100000, k=0x200000, v=0x300000, gq=0x400000, gk=0x410000, cos=0x420000, sin=0x430000, pos=0x440000, slots=0x450000,
             out=0x500000, kc=0x600000, vc=0x700000, ks=None, vs=None)
    v.update(kw)
    return D.load_library().dsa_rope_axes_append(ctypes.byref(p), *[v[n] for n in ("q", "k", "v", "gq", "gk", "cos", "sin", "pos", "slots", "out",
                                                                                   "kc", "vc", "ks", "vs")], None)


def test_rope_axes(D):  # noqa: F811
    bad, unbuilt = D.DSA_ERR_INVALID_ARG, D.DSA_ERR_UNSUPPORTED
    for kw, want in ((dict(tokens=-1), bad), (dict(head_dim=64), unbuilt), (dict(num_q_heads=0, num_kv_heads=0), bad), (dict(num_q_heads=-1), bad),
                     (dict(axes=0), bad), (dict(axes=5), bad), (dict(sections=[0, 0]), bad), (dict(sections=[64, 1]), bad),
                     (dict(sections=[-1, 3]), bad), (dict(max_pos=0), bad), (dict(cos_dtype="fp16"), unbuilt), (dict(eps=-1.0), bad),
                     (dict(eps=float("inf")), bad), (dict(eps=float("nan")), bad), (dict(q_dtype="fp32"), unbuilt), (dict(kv_dtype="e4m3"), unbuilt),
                     (dict(q_dtype="fp16", kv_dtype="bf16"), unbuilt), (dict(cache_rows=0), bad), (dict(cache_rows=-5), bad),
                     (dict(cache_rows=1 << 31), bad), (dict(q_stride=508), bad), (dict(q_stride=516), bad), (dict(k_stride=128), bad),
                     (dict(out_stride=-512), bad), (dict(pos_stride=-1), bad)):
        expect(D, call_axes(D, axes_problem(D, **kw)), want)
    p, p8 = axes_problem(D), axes_problem(D, kv_dtype="int8")
    for name in ("q", "k", "v", "cos", "sin", "pos", "slots", "out", "kc", "vc"):
        assert call_axes(D, p, **{name: None}) == bad, name
    assert call_axes(D, p, ks=0x800000, vs=0x810000) == bad and call_axes(D, p8) == bad and call_axes(D, p8, ks=0x800000) == bad
    assert call_axes(D, p, q=0x100008) == D.DSA_ERR_MISALIGNED and call_axes(D, p, slots=0x450002) == D.DSA_ERR_MISALIGNED
    # what is written overlaps nothing: 10 x 4 x 256 bytes of q_out, 100 x 2 x 256 of a cache
    for kw in (dict(out=0x200000), dict(out=0x100010), dict(out=0x450000 - 16), dict(kc=0x100000), dict(vc=0x600000 + 51184), dict(kc=0x440000 - 51184),
               dict(vc=0x500000 - 51184), dict(kc=0x420000), dict(out=0x400000)):
        assert call_axes(D, p, **kw) == bad, kw
    assert call_axes(D, p8, ks=0x800000, vs=0x800000 + 796) == bad
    assert call_axes(D, axes_problem(D, tokens=0), q=None, k=None, v=None, pos=None, slots=None, out=None) == D.DSA_OK
    if fine(D):
        wide = axes_problem(D, q_stride=1024, k_stride=1024, v_stride=1024, out_stride=1024)
        for q, kw in ((p, {}), (p, dict(gq=None, gk=None)), (p8, dict(ks=0x800000, vs=0x810000)), (p, dict(out=0x100000)),
                      (wide, dict(k=0x100000 + 1024, v=0x100000 + 1536, out=0x100000)),       # columns of one projection, in place
                      (axes_problem(D, num_kv_heads=0, cache_rows=0), dict(k=None, v=None, slots=None, kc=None, vc=None)),
                      (axes_problem(D, num_q_heads=0), dict(q=None, out=None)), (axes_problem(D, cos_dtype="bf16", sections=[1, 0, 2, 3]), {})):
            expect(D, call_axes(D, q, **kw), D.DSA_ERR_NO_DEVICE)
    # in place in rows whose keys would be overwritten
    assert call_axes(D, axes_problem(D, q_stride=1024, k_stride=1024, v_stride=1024, out_stride=1024), k=0x100000 + 512, out=0x100000) == bad


def call_norm(D, p, **kw):  # noqa: F811
    v = dict(x=0x100000, r=0x200000, g=0x300000, h=0x400000, y=0x500000, s=None)
    v.update(kw)
    return D.load_library().dsa_add_rmsnorm(ctypes.byref(p), *[v[n] for n in "xrghys"], None)


def test_add_rmsnorm(D):  # noqa: F811
    bad, unbuilt = D.DSA_ERR_INVALID_ARG, D.DSA_ERR_UNSUPPORTED
    make = D.make_norm_problem
    for args, kw, want in (((-1, 64), {}, bad), ((4, 0), {}, unbuilt), ((4, 32769), {}, unbuilt), ((4, 64, "int8"), {}, unbuilt),
                           ((4, 64, "bf16", "fp32"), {}, unbuilt), ((4, 64), dict(scale_group=128), unbuilt),
                           ((4, 64, "bf16", "e4m3"), dict(scale_group=64), unbuilt), ((4, 64), dict(eps=-1e-6), bad), ((4, 64), dict(eps=float("nan")), bad)):
        expect(D, call_norm(D, make(*args, **kw)), want)
    p, p8 = make(4, 64), make(4, 64, "bf16", "e4m3")
    for name in "xgy":
        assert call_norm(D, p, **{name: None}) == bad
    assert call_norm(D, p, r=None) == bad                       # a sum without a residual
    assert call_norm(D, p, s=0x600000) == bad and call_norm(D, p8) == bad
    assert call_norm(D, p, x=0x100001) == D.DSA_ERR_MISALIGNED and call_norm(D, p, g=0x300002) == D.DSA_ERR_MISALIGNED
    short = make(4, 64)
    short.y_stride = 63
    assert call_norm(D, short) == bad
    for kw in (dict(h=0x100010), dict(y=0x200000 - 16), dict(y=0x400000), dict(h=0x300000), dict(y=0x300000 + 128)):
        assert call_norm(D, p, **kw) == bad, kw
    assert call_norm(D, p8, s=0x600000, y=0x100000) == bad      # codes are of another size than x
    other = make(4, 64)
    other.h_stride = 128
    assert call_norm(D, other, h=0x100000) == bad               # the same place, but not the same rows
    assert call_norm(D, make(0, 64), x=None, r=None, g=None, h=None, y=None) == D.DSA_OK
    if fine(D):
        for q, kw in ((p, {}), (p, dict(h=None)), (p, dict(r=None, h=None)), (p, dict(h=0x200000, y=0x100000)), (p, dict(h=0x100000)),
                      (p8, dict(s=0x600000)), (make(4, 33, "fp32", "int8", scale_group=128), dict(s=0x600000)), (make(4, 64), dict(x=0x100002))):
            expect(D, call_norm(D, q, **kw), D.DSA_ERR_NO_DEVICE)


def call_sample(D, problem, **kw):  # noqa: F811
    v = dict(logits=0x1000000, u=0x2000, heat=0x3000, k=0x4000, p=0x5000, low=0x6000, tok=0x7000, lp=0x8000)
    v.update(kw)
    return D.load_library().dsa_sample(ctypes.byref(problem), *[v[n] for n in ("logits", "u", "heat", "k", "p", "low", "tok", "lp")], None)


def test_sample(D):  # noqa: F811
    bad, make = D.DSA_ERR_INVALID_ARG, D.make_sample_problem
    for args, want in (((0, 10), bad), ((65536, 10), bad), ((4, 0), bad), ((4, (1 << 19) + 1), D.DSA_ERR_UNSUPPORTED), ((4, 10, "int8"), D.DSA_ERR_UNSUPPORTED),
                       ((4, 10, "bf16", 9), bad), ((4, 10, "bf16", -10), bad)):
        expect(D, call_sample(D, make(*args)), want)
    p = make(4, 1000, "fp32")
    for name in ("logits", "u", "tok"):
        assert call_sample(D, p, **{name: None}) == bad
    assert call_sample(D, p, logits=0x1000002) == D.DSA_ERR_MISALIGNED and call_sample(D, p, k=0x4001) == D.DSA_ERR_MISALIGNED
    for kw in (dict(tok=0x2000), dict(lp=0x5008), dict(tok=0x1000000 + 15996), dict(lp=0x7004), dict(tok=0x4000 - 4)):
        assert call_sample(D, p, **kw) == bad, kw
    if fine(D):
        for q, kw in ((p, {}), (p, dict(heat=None, k=None, p=None, low=None, lp=None)), (make(4, 1000, "bf16", 1003), dict(logits=0x1000002)),
                      (make(1, 1 << 19, "fp32"), {})):
            expect(D, call_sample(D, q, **kw), D.DSA_ERR_NO_DEVICE)


def test_problem_structs_match_the_header(D):  # noqa: F811
    assert ctypes.sizeof(D.DsaAxesProblem) == 7 * 8 + 4 * (4 + D.DSA_MAX_AXES + 6)
    assert D.DsaAxesProblem.sections.offset == 7 * 8 + 16
    assert ctypes.sizeof(D.DsaNormProblem) == 5 * 8 + 5 * 4 + 4 and ctypes.sizeof(D.DsaSampleProblem) == 24
