"""The example that runs the token-score operators with the collectives."""
import pytest

pytestmark = pytest.mark.gpu


def test_post_training_example_learns():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()
    from collective_reduction_math_gb300 import example_post_training as ex
    import collective_reduction_math_gb300 as mr
    before = mr.mr_launch_count()
    losses = ex.run(steps=12, T=128, V=2001, H=32, K=16, log=lambda s: None)
    assert mr.mr_launch_count() - before == 12 * (2 * 4 + 1)
    assert all(a == a and a < 1e4 for a in losses)
    assert losses[-1] < 0.8 * losses[0], losses
