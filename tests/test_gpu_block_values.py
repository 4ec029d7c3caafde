"""The operators around the layer on the GPU, where values go wrong: gradients that are not finite
in the optimizer's states."""
import pytest
import torch

from expert_token_routing_amd import occ
from test_gpu_block import F32, adam_desc, adam_inputs, moments

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    occ.lib()


# ---------------------------------------------------------------------- AdamW

def adam_case(n, bits, zero, seed):
    """A tensor with states and gradients, or all zeros but p."""
    t = adam_inputs([n], bits, F32, seed=seed)[0]
    if zero:
        for key in t:
            if key != "p":
                t[key].zero_()
    return t


@pytest.mark.parametrize("zero", [False, True], ids=["full", "zeros"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("n,at", [(1, 0), (3, 2), (256, 255), (600, 300), (1000, 999), (5000, 1024),
                                  (5000, 0)])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_gradient_that_is_not_finite_stays_in_the_states(bits, n, at, bad, zero):
    """One such gradient: its element's p, m and v are not finite, in 8 bits its whole block's m
    and v; everything else is what a finite one leaves there."""
    t = adam_case(n, bits, zero, seed=n)
    clean = {key: v.clone() for key, v in t.items()}
    opt = adam_desc(bits, F32)
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, [clean]))
    t["g"][at] = bad
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, [t]))
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[at] = True
    assert not t["p"][at].isfinite() and torch.equal(t["p"][~hit], clean["p"][~hit])
    if bits == 8:
        hit[at // 256 * 256:at // 256 * 256 + 256] = True
    for got, want in zip(moments(t), moments(clean)):
        assert not got[hit].isfinite().any()
        assert torch.equal(got[~hit], want[~hit])
    # and stays there: the next step makes p so wherever the states are
    t["g"].fill_(1e-3)
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, [t]))
    assert not t["p"][hit].isfinite().any() and t["p"][~hit].isfinite().all()
    for got in moments(t):
        assert not got[hit].isfinite().any() and got[~hit].isfinite().all()
