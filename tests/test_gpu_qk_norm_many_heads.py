"""The norm of queries and keys with their rotation with more heads than a grid has blocks in y."""
import pytest

from test_gpu_qk_norm_rotary import _case, _check_all, la  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_heads_than_a_grid_is_high(la, dtype, per_head):   # noqa: F811
    _check_all(la, _case(3, 40000, 30000, 8, (4,), dtype, per_head, seed=11), False)
