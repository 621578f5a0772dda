"""dsa_add_rmsnorm against the formula in 64 bits, element by element.

The sum of squares is taken in fp32, 32 terms a thread at most and then over at most
1,024 threads: some 45 roundings, half of which reach y; the reciprocal root, the
products and the mean add a few. E = |y| 2^-19 covers 32 of them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
E = 2.0 ** -19


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from top_sparse_attention_chunked_gb300 import build_lib, dsa
    build_lib.build()
    dsa.load_library()
    return dsa


def inputs(rows, hidden, x, seed=0, mul=1.0):
    g = torch.Generator().manual_seed(seed)
    a = (torch.randn(rows, hidden, generator=g) * mul).to(DT[x])
    b = (torch.randn(rows, hidden, generator=g) * 3 * mul).to(DT[x])
    return a, b, 1 + 0.3 * torch.randn(hidden, generator=g)


def check(h, gamma, y, scale, out, group, eps):
    """h: what is normalised, as stored."""
    h64 = h.double().numpy()
    with np.errstate(invalid="ignore"):
        ref = h64 * gamma.double().numpy() / np.sqrt((h64 ** 2).mean(1, keepdims=True) + eps)
    # sums that overflow their type are infinite, as the addition says: NaN there, 0 beside them
    over = np.isinf(h64)
    if out in HALF:
        got = y.double().cpu().numpy()
        assert np.isnan(got[over]).all()
        got, ref = got[~over], ref[~over]
        tol = HALF[out] * np.abs(ref) * (1 + E) + np.abs(ref) * E + (2.0 ** -25 if out == "fp16" else 1e-39)
        assert (np.abs(got - ref) <= tol).all()
        return
    finite = ~over.any(1)                         # (rows of codes are unspecified then)
    y, scale, ref = y[torch.from_numpy(finite).to(y.device)], scale[torch.from_numpy(finite).to(y.device)], ref[finite]
    top = 448.0 if out == "e4m3" else 127.0
    width = group or h.shape[1]
    got, s = y.double().cpu().numpy(), scale.double().cpu().numpy()
    for g in range(s.shape[1]):
        part = ref[:, g * width:(g + 1) * width]
        want = np.abs(part).max(1) / top
        assert (np.abs(s[:, g] - want) <= want * 2 * E + 2.0 ** -149).all()
        live = want > 0
        assert (s[~live, g] == 0).all() and (got[~live, g * width:(g + 1) * width] == 0).all()
        q = part[live] / want[live, None]
        err = np.abs(got[live, g * width:(g + 1) * width] - q)
        # half a step (e4m3's smallest step is 2^-9), and what the quotient is off by
        step = np.maximum(np.abs(q) * 2.0 ** -4, 2.0 ** -10) if out == "e4m3" else 0.5
        assert (err <= step + np.abs(q) * 4 * E).all()


def run(D, rows, hidden, x, out, group=0, add=True, eps=1e-6, seed=0, mul=1.0, data=None):
    a, b, gamma = data or inputs(rows, hidden, x, seed, mul)
    p = D.make_norm_problem(rows, hidden, x, out, eps=eps, scale_group=group)
    y = torch.full((rows, hidden), 3, device="cuda").to(DT[out])
    h = torch.full((rows, hidden), 5.0, device="cuda").to(DT[x]) if add else None
    groups = -(-hidden // group) if group else 1
    scale = torch.full((rows, groups), 7.0, device="cuda") if out in ("e4m3", "int8") else None
    D.dsa_add_rmsnorm(p, a.cuda(), b.cuda() if add else None, gamma.cuda(), h, y, scale)
    want = (a.float() + b.float()).to(DT[x]) if add else a
    if add:
        assert torch.equal(h.cpu(), want)
    check(want, gamma, y, scale, out, group, eps)
    return h, y, scale


@pytest.mark.parametrize("hidden", [1, 2, 7, 8, 33, 64, 127, 128, 129, 256, 264, 1000, 1025, 2056, 4097, 5120, 8192, 12345, 16392, 32768])
@pytest.mark.parametrize("out,group", [("bf16", 0), ("e4m3", 0), ("e4m3", 128), ("int8", 128)])
def test_sizes(D, hidden, out, group):
    run(D, 3, hidden, "bf16", out, group, seed=hidden)


@pytest.mark.parametrize("rows", [1, 2, 9, 151, 700])
@pytest.mark.parametrize("hidden", [96, 515, 2048, 6000])
def test_rows(D, rows, hidden):
    run(D, rows, hidden, "bf16", "bf16", seed=rows)
    run(D, rows, hidden, "fp16", "e4m3", 128, seed=rows)


@pytest.mark.parametrize("x", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("out,group", [("bf16", 0), ("fp16", 0), ("e4m3", 0), ("e4m3", 128), ("int8", 0), ("int8", 128)])
@pytest.mark.parametrize("add", [True, False])
def test_types(D, x, out, group, add):
    for hidden in (384, 1001, 7168):
        run(D, 40, hidden, x, out, group, add, seed=hidden)
    run(D, 400, 1000, x, out, group, add, eps=0.0)


@pytest.mark.parametrize("x,mul,eps", [("bf16", 1e36, 0.0), ("fp32", 1e37, 1e-6), ("fp32", 1e-30, 0.0), ("bf16", 1e-36, 0.0), ("fp32", 1e-44, 0.0),
                                       ("bf16", 1e-22, 1e-6), ("fp32", 1e-18, 1e-30), ("bf16", 1e18, 1e30), ("fp16", 1e-6, 1e-12),
                                       ("fp16", 8000.0, 1e-6)])
def test_large_and_small_values(D, x, mul, eps):
    """Squares that leave fp32, beside an eps that does or does not count."""
    for hidden in (136, 1003, 4096):
        for out, group in (("bf16", 0), ("e4m3", 128), ("int8", 0)):
            run(D, 5, hidden, x, out, group, eps=eps, mul=mul, seed=3)


def test_rows_of_zeros_and_single_values(D):
    a, b, gamma = inputs(6, 640, "bf16", 1)
    a[1], b[1] = 0, 0
    a[2], b[2] = -1.5, 1.5                       # the sum is zero
    a[3], b[3] = 0, 0
    a[3, 600] = 2.0                              # only the last group has a value
    gamma[128:256] = 0
    for out, group in (("bf16", 0), ("e4m3", 0), ("e4m3", 128), ("int8", 128), ("int8", 0)):
        run(D, 6, 640, "bf16", out, group, data=(a, b, gamma))


@pytest.mark.parametrize("hidden", [1024, 1000, 333])
def test_strides_and_offsets(D, hidden):
    """Rows that are columns of wider buffers, at any element's alignment."""
    rows, g = 20, torch.Generator(device="cuda").manual_seed(5)
    for off, pad in ((0, 8), (0, 3), (1, 7), (8, 8), (3, 0)):
        wide = [torch.randn(rows, hidden + off + pad, device="cuda", generator=g).to(torch.bfloat16) for _ in range(4)]
        x, r, h, y = (w[:, off:off + hidden] for w in wide)
        keep = [w.clone() for w in wide]
        gamma = 1 + torch.rand(hidden, device="cuda", generator=g)
        p = D.make_norm_problem(rows, hidden, "bf16", "bf16")
        D.dsa_add_rmsnorm(p, x, r, gamma, h, y)
        want = (x.float() + r.float()).to(torch.bfloat16)
        assert torch.equal(h, want)
        check(want.cpu(), gamma.cpu(), y, None, "bf16", 0, 1e-6)
        for w, k in zip(wide, keep):              # nothing beside the rows changed
            assert torch.equal(w[:, :off], k[:, :off]) and torch.equal(w[:, off + hidden:], k[:, off + hidden:])
        q, s = torch.zeros(rows, hidden + off + pad, device="cuda").to(DT["e4m3"]), torch.zeros(rows, -(-hidden // 128), device="cuda")
        D.dsa_add_rmsnorm(D.make_norm_problem(rows, hidden, "bf16", "e4m3", scale_group=128), x, r, gamma, None,
                          q[:, off:off + hidden], s)
        check(want.cpu(), gamma.cpu(), q[:, off:off + hidden].contiguous(), s, "e4m3", 128, 1e-6)


def test_in_place(D):
    a, b, gamma = (t.cuda() for t in inputs(50, 2048, "bf16", 9))
    p = D.make_norm_problem(50, 2048)
    h, y = torch.empty_like(a), torch.empty_like(a)
    D.dsa_add_rmsnorm(p, a, b, gamma, h, y)
    x1, r1 = a.clone(), b.clone()
    D.dsa_add_rmsnorm(p, x1, r1, gamma, r1, x1)   # the usual layer: the residual is updated, x becomes y
    assert torch.equal(r1, h) and torch.equal(x1, y)
    x2 = a.clone()
    D.dsa_add_rmsnorm(p, x2, b, gamma, x2, y2 := torch.empty_like(a))
    assert torch.equal(x2, h) and torch.equal(y2, y)
    x3 = a.clone()
    D.dsa_add_rmsnorm(p, x3, b, gamma, None, x3)
    assert torch.equal(x3, y)


def test_captured_on_another_stream(D):
    a, b, gamma = (t.cuda() for t in inputs(64, 4096, "bf16", 2))
    p = D.make_norm_problem(64, 4096, "bf16", "e4m3", scale_group=128)
    h, y, s = torch.empty_like(a), torch.empty(64, 4096, device="cuda", dtype=DT["e4m3"]), torch.empty(64, 32, device="cuda")
    D.dsa_add_rmsnorm(p, a, b, gamma, h, y, s)
    want = h.clone(), y.view(torch.uint8).clone(), s.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.dsa_add_rmsnorm(p, a, b, gamma, h, y, s)
    for t in (h, y.view(torch.uint8), s):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t, w) for t, w in zip((h, y.view(torch.uint8), s), want))
    st = torch.cuda.Stream()
    h.zero_()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        D.dsa_add_rmsnorm(p, a, b, gamma, h, y, s)
    st.synchronize()
    assert torch.equal(h, want[0])
    D.dsa_add_rmsnorm(D.make_norm_problem(0, 64), torch.empty(0, 64, device="cuda", dtype=DT["bf16"]), None,
                      torch.ones(64, device="cuda"), None, torch.empty(0, 64, device="cuda", dtype=DT["bf16"]))
    assert D.dsa_last_launches() == []
