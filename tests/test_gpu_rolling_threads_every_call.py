"""Several host threads that call at once, each on a stream of its own: every single call's results are those
of a call alone. (The results are kept on the device and compared at the end, so that nothing waits between
the calls.)"""
import threading

import pytest
import torch

from tests.test_gpu_sample import D  # noqa: F401 (D is a fixture)

pytestmark = pytest.mark.gpu

CALLS = 60


def at_once(work):
    """work[i]() makes a call and gives its results: CALLS times on a thread and a stream each."""
    alone = []
    for f in work:
        alone.append([t.clone() for t in f()])
    torch.cuda.synchronize()
    errors, wrong, gate = [], [None] * len(work), threading.Barrier(len(work))

    def run(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                gate.wait(30)
                kept = []
                for _ in range(CALLS):
                    kept.append([t.clone() for t in work[i]()])
                st.synchronize()
                wrong[i] = [n for n, got in enumerate(kept) if not all(torch.equal(a, b) for a, b in zip(alone[i], got))]
        except Exception as e:                         # (a thread's own would be lost)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    assert wrong == [[]] * len(work), f"calls that differ: {wrong}"


def sampler(D, rows, vocab, dtype, k=None):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (2 * torch.randn(rows, vocab, device="cuda", generator=g)).to(dtype)
    u, p = torch.rand(rows, device="cuda", generator=g), torch.full((rows,), 0.9, device="cuda")
    kk = None if k is None else torch.full((rows,), k, dtype=torch.int32, device="cuda")
    plan = D.make_sample_problem(rows, vocab, "bf16" if dtype is torch.bfloat16 else "fp32")
    tok, lp = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, device="cuda")

    def f():
        D.dsa_sample(plan, x, u, tok, top_k=kk, top_p=p, logprobs=lp)
        return tok, lp
    return f


def norm(D, plan, pitch):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(pitch)
    x, r, h = (torch.randn(64, pitch, device="cuda", generator=g).to(torch.bfloat16)[:, :1000] for _ in range(3))
    y, s = torch.zeros(64, 1000, device="cuda").to(torch.float8_e4m3fn), torch.zeros(64, 8, device="cuda")
    gamma = torch.ones(1000, device="cuda")

    def f():
        D.dsa_add_rmsnorm(plan, x, r, gamma, h, y, s)
        return h, y.view(torch.uint8), s
    return f


def rope(D, plan, pitch):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(pitch)
    n, hq, hkv = 300, 8, 2
    qkv = torch.randn(n, pitch, device="cuda", generator=g).to(torch.bfloat16)
    q, k, v = qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:1536]
    cos, sin = torch.rand(500, 64, device="cuda", generator=g), torch.rand(500, 64, device="cuda", generator=g)
    pos = torch.randint(0, 500, (2, n), device="cuda", generator=g, dtype=torch.int32)
    slots = torch.randperm(n, device="cuda", generator=g).to(torch.int32)
    out = torch.zeros(n, hq, 128, device="cuda", dtype=torch.bfloat16)
    K, V = (torch.zeros(n, hkv, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))

    def f():
        D.dsa_rope_axes_append(plan, q, k, v, None, None, cos, sin, pos, slots, out, K, V)
        return out, K, V
    return f


def test_sampling_from_vocabularies_of_every_size(D):  # noqa: F811
    bf = torch.bfloat16
    at_once([sampler(D, 3, 500, bf), sampler(D, 9, 80000, bf), sampler(D, 40, 5000, bf, k=50), sampler(D, 2, 300000, bf),
             sampler(D, 5, 40000, torch.float32, k=700), sampler(D, 1, 524288, torch.float32)])


def test_problems_that_threads_share(D):  # noqa: F811
    """One problem for rows of several strides."""
    plan = D.make_norm_problem(64, 1000, "bf16", "e4m3", scale_group=128)
    axes = D.make_rope_axes_problem(300, 8, 2, 300, [40, 24], 500)
    at_once([norm(D, plan, 1000), norm(D, plan, 1008), norm(D, plan, 4001), rope(D, axes, 1536), rope(D, axes, 1544), rope(D, axes, 2048)])


def test_unlike_calls_side_by_side(D):  # noqa: F811
    plan = D.make_norm_problem(64, 1000, "bf16", "e4m3", scale_group=128)
    axes = D.make_rope_axes_problem(300, 8, 2, 300, [40, 24], 500)
    i32 = dict(dtype=torch.int32, device="cuda")
    q_len, total = torch.randint(0, 9, (200,), **i32), torch.randint(9, 500, (200,), **i32)

    def slots(n):
        out, pos, row = (torch.zeros(n, **i32) for _ in range(3))

        def f():
            D.dsa_slot_map(q_len, total, out, capacity=600, positions=pos, rows=row)
            return out, pos, row
        return f

    at_once([norm(D, plan, 1016), rope(D, axes, 1536), slots(2000), slots(300), sampler(D, 20, 60000, torch.bfloat16, k=9)])
