"""The gradient norm where its sums could lose something: beyond fp32's range
in a tensor of more than 2^32 elements."""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mr():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()
    import collective_reduction_math_gb300 as m
    m.load()
    return m


def test_most_of_the_largest(mr):
    """2^33 elements of bf16's largest value: the norm, 2^16.5 times that, reads
    +inf, and the factor still comes from the norm itself."""
    import torch
    n, x, most = 1 << 33, 255 * 2.0 ** 120, 2.0 ** 60
    t = torch.full((n,), x, dtype=torch.bfloat16, device="cuda")
    norm = torch.zeros(1, device="cuda")
    mr.mr_clip_grad_norm([t], [t], most, norm=norm)
    assert float(norm) == float("inf")
    # most / 2^16.5, rounded to bf16: 1.41421 * 2^43 lies 0.0038 of itself from the nearest
    # point between two bf16 values, which the factor's few U do not reach
    want = torch.tensor(most / 2 ** 16.5, dtype=torch.float64).bfloat16()
    wrong = sum(int((part != want.cuda()).sum()) for part in t.split(1 << 30))
    assert wrong == 0
