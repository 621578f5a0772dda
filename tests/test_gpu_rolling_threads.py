"""Two host threads that call at once, each on a stream of its own: what one asks for
does not reach the other's launch."""
import threading

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


def at_once(work):
    """Runs work[i](check) 40 times on a thread and a stream each; check: results stay the first's."""
    errors, gate = [], threading.Barrier(len(work))

    def run(f):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                want = [t.clone() for t in f()]
                st.synchronize()
                gate.wait(30)
                for _ in range(40):
                    got = [t.clone() for t in f()]
                st.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        except Exception as e:                         # (a thread's own would be lost)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in work]
    torch.cuda.synchronize()
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors


def test_sampling_from_vocabularies_of_every_size(D):
    def sampler(rows, vocab, dtype):
        g = torch.Generator(device="cuda").manual_seed(vocab)
        x = (2 * torch.randn(rows, vocab, device="cuda", generator=g)).to(dtype)
        u, p = torch.rand(rows, device="cuda", generator=g), torch.full((rows,), 0.9, device="cuda")
        plan = D.make_sample_problem(rows, vocab, "bf16" if dtype is torch.bfloat16 else "fp32")
        tok, lp = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, device="cuda")

        def f():
            D.dsa_sample(plan, x, u, tok, top_p=p, logprobs=lp)
            assert D.dsa_last_launches() == ["sample_kernel"]
            return tok, lp
        return f

    bf = torch.bfloat16
    at_once([sampler(3, 500, bf), sampler(9, 80000, bf), sampler(40, 5000, bf), sampler(2, 300000, bf), sampler(5, 40000, torch.float32)])


def test_norms_of_one_problem_with_rows_apart_and_together(D):
    plan = D.make_norm_problem(64, 1000, "bf16", "e4m3", scale_group=128)     # shared by the threads

    def norm(pitch):
        g = torch.Generator(device="cuda").manual_seed(pitch)
        x, r, h = (torch.randn(64, pitch, device="cuda", generator=g).to(torch.bfloat16)[:, :1000] for _ in range(3))
        y, s, gamma = torch.zeros(64, 1000, device="cuda").to(torch.float8_e4m3fn), torch.zeros(64, 8, device="cuda"), torch.ones(1000, device="cuda")

        def f():
            D.dsa_add_rmsnorm(plan, x, r, gamma, h, y, s)
            return h, y.view(torch.uint8), s
        return f

    at_once([norm(1000), norm(1008), norm(1500), norm(4001)])
