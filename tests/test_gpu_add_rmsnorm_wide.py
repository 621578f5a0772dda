"""dsa_add_rmsnorm on the widest rows, of vectors and of single elements, against the formula in 64 bits."""
import pytest

from tests.test_gpu_add_rmsnorm import D, run  # noqa: F401 (D is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden", [16384, 16385, 16392, 20001, 24576, 32765, 32767, 32768])
@pytest.mark.parametrize("x", ["bf16", "fp16", "fp32"])
def test_wide_rows(D, hidden, x):  # noqa: F811
    for out, group in (("bf16", 0), ("fp16", 0), ("e4m3", 128), ("int8", 0)):
        for add in (True, False):
            run(D, 3, hidden, x, out, group, add, seed=hidden)
    run(D, 400, hidden, x, "bf16", seed=1)
    run(D, 2, hidden, x, "e4m3", 128, eps=0.0, mul=1e3 if x == "fp16" else 1e18, seed=2)
