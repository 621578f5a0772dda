"""How the binding takes strides from the tensors of a call: rows that are all the same
are refused, and a problem that several calls share stays as it was."""
import pytest
import torch

from top_sparse_attention_chunked_gb300 import dsa as D


class Recorder:
    """Stands for the library: keeps the problem that a call was given."""

    def __getattr__(self, name):
        def call(p, *args):
            self.problem = type(p._obj).from_buffer_copy(p._obj)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    """Calls on CPU tensors that end at the library."""
    r = Recorder()
    monkeypatch.setattr(D, "load_library", lambda *a: r)
    monkeypatch.setattr(D, "_current_device", lambda: -1)
    monkeypatch.setattr(D, "_stream_here", lambda *a: None)
    return r


def norm_args(**kw):
    t = dict(x=torch.zeros(4, 64), residual=torch.zeros(4, 64), gamma=torch.ones(64), h=torch.zeros(4, 64), y=torch.zeros(4, 64).bfloat16())
    t.update(kw)
    return t.values()


def test_norm_strides(lib):
    p = D.make_norm_problem(4, 64, "fp32", "bf16")
    D.dsa_add_rmsnorm(p, *norm_args(x=torch.zeros(4, 80)[:, :64], h=torch.zeros(8, 64)[::2]))
    c = lib.problem
    assert (c.x_stride, c.residual_stride, c.h_stride, c.y_stride) == (80, 64, 128, 64)
    assert (p.x_stride, p.residual_stride, p.h_stride, p.y_stride) == (0, 0, 0, 0), "the caller's problem stays"
    for name in ("x", "residual", "h", "y"):
        t = torch.zeros(1, 64, dtype=torch.bfloat16 if name == "y" else torch.float32)
        with pytest.raises(ValueError, match=name):
            D.dsa_add_rmsnorm(p, *norm_args(**{name: t.expand(4, 64)}))
    with pytest.raises(ValueError, match="x's rows"):
        D.dsa_add_rmsnorm(p, *norm_args(x=torch.zeros(64, 4).t()))
    one = D.make_norm_problem(1, 64, "fp32", "bf16")
    D.dsa_add_rmsnorm(one, *(None if t is None else t[:1] if t.dim() == 2 else t for t in norm_args(x=torch.zeros(1, 64).expand(4, 64))))
    assert lib.problem.x_stride == 0


def axes_args(n=3, **kw):
    bf = dict(dtype=torch.bfloat16)
    t = dict(q=torch.zeros(n, 512, **bf), k=torch.zeros(n, 256, **bf), v=torch.zeros(n, 2, 128, **bf), gq=None, gk=None, cos=torch.ones(9, 64),
             sin=torch.zeros(9, 64), pos=torch.zeros(2, n, dtype=torch.int32), slots=torch.zeros(n, dtype=torch.int32),
             out=torch.zeros(n, 4, 128, **bf), K=torch.zeros(50, 2, 128, **bf), V=torch.zeros(50, 2, 128, **bf))
    t.update(kw)
    return t.values()


def test_axes_strides(lib):
    p = D.make_rope_axes_problem(3, 4, 2, 50, [40, 24], 9)
    wide = torch.zeros(3, 1024, dtype=torch.bfloat16)
    D.dsa_rope_axes_append(p, *axes_args(q=wide[:, :512], k=wide[:, 512:768], v=wide[:, 768:].view(3, 2, 128)))
    c = lib.problem
    assert (c.q_stride, c.k_stride, c.v_stride, c.out_stride, c.pos_stride) == (1024, 1024, 1024, 512, 3)
    assert (p.q_stride, p.k_stride, p.v_stride, p.out_stride, p.pos_stride) == (0, 0, 0, 0, 0), "the caller's problem stays"
    for name, width in (("q", 512), ("k", 256), ("v", 256), ("out", 512)):
        with pytest.raises(ValueError, match="q_out" if name == "out" else name):
            D.dsa_rope_axes_append(p, *axes_args(**{name: torch.zeros(1, width, dtype=torch.bfloat16).expand(3, width)}))
    for name, width in (("q", 512), ("k", 256)):
        with pytest.raises(ValueError, match="contiguous"):
            D.dsa_rope_axes_append(p, *axes_args(**{name: torch.zeros(width, 3, dtype=torch.bfloat16).t()}))


def test_sample_strides(lib):
    p, f = D.make_sample_problem(4, 100, "fp32"), torch.zeros(4)
    tok = torch.zeros(4, dtype=torch.int32)
    D.dsa_sample(p, torch.zeros(4, 100), f, tok)
    D.dsa_sample(D.make_sample_problem(4, 100, "fp32", 120), torch.zeros(4, 120)[:, :100], f, tok)
    for x in (torch.zeros(1, 100).expand(4, 100), torch.zeros(4, 120)[:, :100], torch.zeros(100, 4).t()):
        with pytest.raises(ValueError, match="logits"):
            D.dsa_sample(p, x, f, tok)
