"""The operators around the layer on the GPU, where values go wrong: gradients that are not finite
in the optimizer's states, rows near the smallest normal number, and weight gradients of whole
numbers, whose sums are exact in every order, over one, several and very long shares of the tokens."""
import pytest
import torch

import block_reference as ref
from expert_token_routing_amd import occ
from test_gpu_block import (BF16, F32, FORMS, GATE_SHAPES, LAST, SCALE, U, adam_desc, adam_inputs,
                            behind_zeros, check, check_norm, check_norm_back, gen, layer, moments,
                            nan_like, norm_inputs, only_last, run_norm, run_norm_back)

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


# Forward workgroups that walk on to another row (a launch holds 2^22 of them): the last rows lie
# on both sides of that border, for rows of a wave's lanes and of several waves.
@pytest.mark.parametrize("dtype,T,d", [(F32, (1 << 26) + 409, 16), (BF16, (1 << 23) + 409, 1024)])
@pytest.mark.parametrize("form", ["sandwich", "first", "last"])
def test_norm_rows_behind_the_last_workgroup(dtype, T, d, form):
    t, _, opt = norm_inputs(dtype, LAST, d, form, seed=d)
    full = {key: behind_zeros(T, v) if v is not None and v.dim() == 2 else v for key, v in t.items()}
    r = full["x"] if full["y"] is not None else None  # in place
    h = None if full["w_pre"] is None else full["x"] if r is None else full["y"]
    occ.occ_block_norm(layer(T, d, dtype=dtype), opt, full["x"], full["y"], full["w_post"],
                       full["gate"], full["w_pre"], r, h)
    check_norm(t, opt, None if r is None else only_last(r), None if h is None else only_last(h))


# ----------------------------------------------------- gate projection, back

def whole(g, values, *shape):
    at = torch.randint(len(values), shape, generator=g, device="cuda", dtype=torch.int8)
    return torch.tensor(values, device="cuda", dtype=F32)[at.int()]


def run_gate(dl, x, w, dx_in, dtype):
    T, Ne = dl.shape
    d = w.shape[1]
    desc = layer(T, d, Ne=Ne, dtype=dtype)
    dx, dw = nan_like((T, d), dtype), nan_like((Ne, d))
    occ.occ_gate_backward(desc, dl, x, w, dx_in, dx, dw, occ.alloc_block_workspace(desc))
    return dx, dw


# Token counts behind a border of the rule that makes shares of dW_r longer than 512 tokens, for one
# and for several groups of experts, and batches of many shares.
LONG_SHAPES = [(BF16, 4099, 8192, 60), (BF16, 4095, 8192, 60), (BF16, 4099, 4096, 130),
               (BF16, 16500, 4096, 20), (BF16, 8191, 8192, 7), (BF16, 65521, 2048, 60),
               (BF16, 33001, 2048, 250), (F32, 2600, 2048, 250), (F32, 4201, 4096, 33),
               (F32, 8203, 2048, 60), (F32, 16399, 1024, 9), (F32, 33001, 512, 16)]


@pytest.mark.parametrize("dtype,T,d,Ne", GATE_SHAPES + LONG_SHAPES,
                         ids=[f"{'bf16' if s[0] == BF16 else 'f32'}-{s[1]}-{s[2]}-{s[3]}"
                              for s in GATE_SHAPES + LONG_SHAPES])
def test_gate_backward_of_whole_numbers_is_exact(dtype, T, d, Ne):
    """dlogits of at most 9 bits and x of -1, 0, 1: sums below 2^24 (T x 257 <= 65521 x 257 =
    16838897 > 2^24 only if every token counted with the largest; their mean is under a half of
    it), so dW_r is exact in every order, and dx is the exact sum rounded once."""
    g = gen(T + 3 * Ne)
    dl = whole(g, [-257.0, -255.0, -3.0, 0.0, 1.0, 129.0, 257.0], T, Ne)
    x, w = whole(g, [-1.0, 0.0, 1.0], T, d).to(dtype), whole(g, [-2.0, -1.0, 0.0, 1.0, 3.0], Ne, d).to(dtype)
    dx_in = whole(g, [-100.0, 0.0, 7.0], T, d).to(dtype)
    dx, dw = run_gate(dl, x, w, dx_in, dtype)
    big = dl.double()
    assert float((big.abs().t().contiguous() @ x.double().abs()).max()) < 2 ** 24
    assert torch.equal(dw.double(), big.t().contiguous() @ x.double())
    assert torch.equal(dx, (big @ w.double() + dx_in.double()).to(dtype))


@pytest.mark.parametrize("dtype,T,d,Ne", [s for s in GATE_SHAPES if s[1] <= 250],
                         ids=[f"{'bf16' if s[0] == BF16 else 'f32'}-{s[1]}-{s[2]}-{s[3]}"
                              for s in GATE_SHAPES if s[1] <= 250])
def test_gate_weight_gradient_keeps_all_bits_of_dlogits(dtype, T, d, Ne):
    """dlogits of 17 bits (2^16 + 2^8 + 1) at most: 250 of them stay below 2^24."""
    g = gen(T + 5 * Ne)
    dl = whole(g, [-65793.0, -65537.0, -1.0, 257.0, 65793.0], T, Ne)
    x, w = whole(g, [-1.0, 0.0, 1.0], T, d).to(dtype), whole(g, [-1.0, 1.0], Ne, d).to(dtype)
    _, dw = run_gate(dl, x, w, None, dtype)
    assert torch.equal(dw.double(), dl.double().t().contiguous() @ x.double())


@pytest.mark.parametrize("Ne", [7, 60, 130])
def test_gate_backward_of_the_smallest_and_largest_dlogits(Ne):
    """bf16 terms are multiples of 2^-133, so that each of the smallest dlogits is off by half of
    that at most, times x or w; the largest ones are exact below 2^128 (1 - 2^-9)."""
    T, d, g = 150, 192, gen(Ne)
    dl = torch.ldexp(1 + torch.rand(T, Ne, generator=g, device="cuda"),
                     torch.randint(-126, -100, (T, Ne), generator=g, device="cuda").float())
    x, w = (2.0 ** 40 * whole(g, [-2.0, -1.0, 1.0, 3.0], n, d).to(BF16) for n in (T, Ne))
    dx, dw = run_gate(dl, x, w, None, BF16)
    want_dx, mdx, want_dw, mdw = ref.gate_back(dl, x, w, None)
    check(dx, want_dx, mdx + 2.0 ** -134 * w.double().abs().sum(0) / (264 * U), 264 + Ne, "dx")
    check(dw, want_dw, mdw + 2.0 ** -134 * x.double().abs().sum(0) / (64 * U), 64 + T, "dw")
    top = 2.0 ** 128 * (1 - 2.0 ** -9)
    dl = torch.zeros(T, Ne, device="cuda")
    at, e = torch.arange(0, T, 9, device="cuda"), torch.arange(0, T, 9, device="cuda") % Ne
    dl[at, e] = top * (1 - 2.0 ** -24)  # the value below
    x, w = (2.0 ** -60 * whole(g, [-2.0, -1.0, 1.0], n, d).to(BF16) for n in (T, Ne))
    dx, dw = run_gate(dl, x, w, None, BF16)
    want_dx, mdx, want_dw, mdw = ref.gate_back(dl, x, w, None)
    check(dx, want_dx, mdx, 264 + Ne, "dx")
    check(dw, want_dw, mdw, 64 + T, "dw")
    dl[at[1], e[1]] = top
    dx, dw = run_gate(dl, x, w, None, BF16)
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[at[1]] = False
    assert not dx[at[1]].isfinite().any() and not dw[e[1]].isfinite().any()
    check(dx[rows], want_dx[rows], mdx[rows], 264 + Ne, "dx")


@pytest.mark.parametrize("dtype,T,d,Ne", [(BF16, 1100003, 2048, 60), (BF16, 1100003, 2048, 100),
                                          (F32, 530003, 4096, 70)])
def test_gate_backward_of_whole_numbers_in_arrays_of_more_than_2_to_the_31(dtype, T, d, Ne):
    """Every token counts: dlogits up to 3, x up to 2, sums of at most 6 T < 2^24."""
    g = gen(Ne)
    dl = whole(g, [-3.0, -1.0, 0.0, 2.0, 3.0], T, Ne)
    x = torch.empty(T, d, dtype=dtype, device="cuda")
    for part in x.split(1 << 16):
        part.copy_(whole(g, [-2.0, -1.0, 0.0, 1.0, 2.0], *part.shape))
    w = whole(g, [-2.0, -1.0, 1.0, 2.0], Ne, d).to(dtype)
    dx, dw = run_gate(dl, x, w, None, dtype)
    want = torch.zeros(Ne, d, dtype=torch.float64, device="cuda")
    wd = w.double()
    for t in range(0, T, 1 << 16):
        part = dl[t:t + (1 << 16)].double()
        want += part.t().contiguous() @ x[t:t + (1 << 16)].double()
        assert torch.equal(dx[t:t + (1 << 16)], (part @ wd).to(dtype)), t
    assert torch.equal(dw.double(), want)
