"""The operators around the layer on the GPU, where values go wrong: gradients that are not finite
in the optimizer's states, and rows near the smallest normal number."""
import pytest
import torch

from expert_token_routing_amd import occ
from test_gpu_block import (BF16, F32, FORMS, SCALE, adam_desc, adam_inputs, check_norm, check_norm_back,
                            moments, norm_inputs, run_norm, run_norm_back)

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


# ---------------------------------------------------------------------- norms

TINY_FORMS = ["first", "first_alone", "prenorm", "prenorm_channel", "prenorm_token", "last"]


@pytest.mark.parametrize("form", TINY_FORMS)
@pytest.mark.parametrize("dtype,T,d", [(F32, 37, 16), (F32, 21, 1040), (BF16, 37, 64), (BF16, 300, 2048)])
def test_norm_backward_of_rows_near_the_smallest_normal_number(dtype, T, d, form):
    """Rows whose mean square is of the size of the smallest eps (2^-126), where 1 / rms is 2^63:
    its square and its cube leave fp32, the gradients do not.  The squares round to steps of 2^-149
    there, 2^-24 of eps together: no more than any other rounding of the statistic."""
    t, grads, _ = norm_inputs(dtype, T, d, form, seed=d)
    size = 2.0 ** -63 * 2.0 ** torch.linspace(-4, 4, T, device="cuda")[:, None]
    t["x"] = (t["x"].float() * size).to(dtype)
    if t["y"] is not None:
        t["y"] = (t["y"].float() * size).to(dtype)
    # gradients along the rows, so that the projection onto the row is as large as it can be
    for key in ("dr", "dh"):
        if grads[key] is not None:
            along = t["x"] if t["y"] is None or FORMS[form][3] else t["y"]
            grads[key] = (1000 * torch.sign(along.float()) * grads[key].float().abs()).to(dtype)
    opt = occ.NormDesc(eps=2.0 ** -126, scale=SCALE, gate=FORMS[form][2])
    r, h = run_norm(t, opt, dtype)
    check_norm(t, opt, r, h)
    kept = r if r is not None else t["x"]
    out = run_norm_back(t, grads, kept, opt, dtype)
    assert all(v.isfinite().all() for v in out.values() if v is not None)
    check_norm_back(t, grads, kept, opt, out)
