"""How the binding takes the axes' stride from a call's positions: a slice of a longer buffer is one."""
import pytest
import torch

from tests.test_rolling_binding_cpu import axes_args, lib  # noqa: F401 (lib is a fixture)
from top_sparse_attention_chunked_gb300 import dsa as D


def test_positions_of_a_longer_buffer(lib):  # noqa: F811
    p = D.make_rope_axes_problem(3, 4, 2, 50, [40, 24], 9)
    long = torch.zeros(2, 100, dtype=torch.int32)
    for pos, stride in ((long[:, :3], 100), (long[:, 50:53], 100), (long[:1, :3].expand(2, 3), 0), (long[0, :3], 0),
                        (torch.zeros(4, 3, dtype=torch.int32)[::2], 6), (torch.zeros(2, 3, dtype=torch.int32), 3)):
        D.dsa_rope_axes_append(p, *axes_args(pos=pos))
        assert lib.problem.pos_stride == stride
    one = D.make_rope_axes_problem(3, 4, 2, 50, [64], 9)
    D.dsa_rope_axes_append(one, *axes_args(pos=long[:1, :3]))
    assert lib.problem.pos_stride == 0
    single = D.make_rope_axes_problem(1, 4, 2, 50, [40, 24], 9)
    D.dsa_rope_axes_append(single, *axes_args(n=1, pos=torch.zeros(1, 2, dtype=torch.int32).t()))
    assert lib.problem.pos_stride == 1


def test_positions_that_are_refused(lib):  # noqa: F811
    p = D.make_rope_axes_problem(3, 4, 2, 50, [40, 24], 9)
    for pos in (torch.zeros(3, 2, dtype=torch.int32).t(), torch.zeros(6, dtype=torch.int32)[::2], torch.zeros(2, 4, dtype=torch.int32),
                torch.zeros(3, 3, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3)[:, :3], torch.zeros((), dtype=torch.int32),
                torch.zeros(1, 2, 3, dtype=torch.int32)):
        with pytest.raises(ValueError, match="positions"):
            D.dsa_rope_axes_append(p, *axes_args(pos=pos))


def test_the_package_offers_the_serving_calls():
    import top_sparse_attention_chunked_gb300 as pkg
    for name in ("dsa_full_attn", "dsa_slot_map", "dsa_rope_axes_append", "dsa_add_rmsnorm", "dsa_sample", "dsa_beam_select", "dsa_pages_update"):
        assert getattr(pkg, name) is getattr(D, name)
