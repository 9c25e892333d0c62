"""Columns that nothing concerns keep their bits, whatever lists name them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("penalty", ["frequency", "presence"])
@pytest.mark.parametrize("W", [1, 3])
def test_prompts_do_not_concern_what_is_said(mr, dtype, penalty, W):
    """A prompt's columns under a penalty on what was said alone: NaN of any payload
    among the scores come back bit by bit, in place and into another buffer."""
    import torch
    rng = np.random.default_rng(5)
    T, V, L, P = 7, 1003, 60, 40
    kind = np.int16 if dtype == "bf16" else np.int32
    nan = {"bf16": [0x7F81, -0x3F, 0x7FA5], "fp32": [0x7F800001, -0x3F0001, 0x7FA55AA5]}[dtype]
    bits = torch.randn(T, V, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    bits = bits.view(torch.int16 if dtype == "bf16" else torch.int32).numpy().copy()
    history = rng.integers(0, V, (T, L))
    said = np.zeros((T, V), dtype=bool)
    for t in range(T):
        bits[t, rng.permutation(V)[:300]] = rng.choice(np.array(nan, dtype=kind), 300)
        bits[t, history[t, :5]] = np.array(nan, dtype=kind)[[0, 1, 2, 0, 1]]
        said[t, history[t, P:]] = True
    x = torch.from_numpy(bits).view(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    cuts = [r * V // W for r in range(W + 1)]
    cols = lambda t: [t[:, lo:hi] for lo, hi in zip(cuts, cuts[1:])]  # noqa: E731
    lists = {"history": torch.from_numpy(history).cuda(), "n_prompt": torch.full((T,), P, device="cuda"), penalty: torch.full((T,), 0.5, device="cuda")}
    out, place = torch.empty_like(x), x.clone()
    mr.mr_adjust_logits(cols(x), cols(out), **lists)
    mr.mr_adjust_logits(cols(place), cols(place), **lists)
    for got in (out, place):
        kept = got.view(torch.int16 if dtype == "bf16" else torch.int32).cpu().numpy() == bits
        assert kept[~said].all()
        assert not kept[said & ~np.isnan(x.float().cpu().numpy())].any()        # the others are lower
