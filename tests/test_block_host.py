"""The operators around the layer on the host (no GPU): the 64-bit reference's gradients against
differences, the workspace size, and every refusal of the C ABI and of the binding before any work
is queued."""
import ctypes
import os

import numpy as np
import pytest
import torch

import block_reference as ref
from expert_token_routing_amd import occ, synth, workloads as W

INV, UNS, WS = occ.OCC_ERR_INVALID_ARG, occ.OCC_ERR_UNSUPPORTED, occ.OCC_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(occ.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return occ.lib()


def fake(n=1):
    """A non-null, 256-byte aligned address that no call may reach."""
    return ctypes.c_void_p(0x1000 * n)


NULL = ctypes.c_void_p(0)
BIG = 1 << 50


# ------------------------------------------- the reference against differences

def central(f, v, direction, h=1e-6):
    return (f(v + h * direction) - f(v - h * direction)) / (2 * h)


def assert_directional(f, v, grad, gen):
    """<grad, u> against a central difference.  The difference's own error is h^2 f''' / 6 plus
    2^-53 |f| / h, here under 1e-8 of the values' size; 1e-6 leaves room for |f'''|."""
    u = torch.randn(v.shape, generator=gen, dtype=torch.float64)
    want, got = central(f, v, u), (grad * u).sum()
    size = (grad.abs() * u.abs()).sum()
    assert abs(want - got) <= 1e-6 * size + 1e-9, (want, got)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("post", [True, False])
def test_reference_norm_gradients_against_differences(kind, post):
    gen = torch.Generator().manual_seed(1 + kind)
    T, d, eps, scale = 5, 12, 1e-3, 0.6
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    v = dict(x=rnd(T, d), y=rnd(T, d), w_post=rnd(d) if post else None,
             gate=None if kind == 0 else rnd(d) if kind == 1 else rnd(T), w_pre=rnd(d))
    dr, dh = rnd(T, d), rnd(T, d)

    def goal(**over):
        r, h, _ = ref.block_norm(**{**v, **over}, kind=kind, eps=eps, scale=scale)
        return (r * dr).sum() + (h * dh).sum()

    r, _, _ = ref.block_norm(**v, kind=kind, eps=eps, scale=scale)
    g, _ = ref.block_norm_back(dr, dh, r, v["y"], v["w_post"], v["gate"], v["w_pre"], kind, eps,
                               scale)
    for name, grad in (("x", "dx"), ("y", "dy"), ("w_post", "dw_post"), ("gate", "dgate"),
                       ("w_pre", "dw_pre")):
        if v[name] is not None:
            assert_directional(lambda a: goal(**{name: a}), v[name], g[grad], gen)


@pytest.mark.parametrize("masked", [False, True])
def test_reference_balance_gradient_against_differences(masked):
    gen = torch.Generator().manual_seed(7)
    T, Ne, k, coef, up = 9, 6, 2, (0.3, 0.2, 0.1), 1.7
    logits = torch.randn(T, Ne, generator=gen, dtype=torch.float64)
    ids = torch.topk(logits, k).indices.int()
    valid = torch.rand(T, generator=gen) < 0.6 if masked else None
    group = torch.tensor([0, 1, 2, 0, 1, 2])
    kept = ref.balance(logits, ids, valid, group, k, coef)[3]
    grad, _ = ref.balance_back(logits, kept, coef, up, None)
    f = lambda l: up * ref.balance(l, ids, valid, group, k, coef)[0][0]
    assert_directional(f, logits, grad, gen)


def test_reference_balance_is_one_coefficient_when_even():
    # every expert equally likely and equally loaded: f = 1, F = 1, P = 1 / Ne
    Ne, k, T = 6, 2, 6
    ids = torch.tensor([[t % Ne, (t + 1) % Ne] for t in range(T)], dtype=torch.int32)
    loss, probs, counts, _ = ref.balance(torch.zeros(T, Ne), ids, None,
                                         torch.tensor([0, 0, 1, 1, 2, 2]), k, (0.5, 0.25, 0.0))
    assert torch.allclose(loss, torch.tensor([0.75, 0.5, 0.25, 0.0], dtype=torch.float64))
    assert counts.tolist() == [2] * 6 + [6] and torch.allclose(probs, torch.full((6,), 1 / 6).double())


def test_reference_gate_gradients_against_differences():
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    x, w, dl = rnd(7, 5), rnd(3, 5), rnd(7, 3)
    dx, _, dw, _ = ref.gate_back(dl, x, w, None)
    assert_directional(lambda a: ((a @ w.t()) * dl).sum(), x, dx, gen)
    assert_directional(lambda a: ((x @ a.t()) * dl).sum(), w, dw, gen)


def test_reference_adamw_against_torch():
    gen = torch.Generator().manual_seed(5)
    a = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, grad_scale=1.0)
    p = torch.randn(50, generator=gen, dtype=torch.float64)
    q = torch.nn.Parameter(p.clone())
    opt = torch.optim.AdamW([q], lr=a["lr"], betas=(0.9, 0.95), eps=a["eps"], weight_decay=0.1)
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    for step in range(1, 6):
        g = torch.randn(50, generator=gen, dtype=torch.float64)
        q.grad = g.clone()
        opt.step()
        p, m, v, _ = ref.adamw(p, g, m, v, dict(a, step=step))
        assert torch.allclose(p, q.detach(), rtol=1e-12, atol=1e-14)


def test_reference_quantisation_round_trips_within_half_a_step():
    gen = torch.Generator().manual_seed(6)
    v = torch.randn(1000, generator=gen, dtype=torch.float64) * torch.exp(
        3 * torch.randn(1000, generator=gen, dtype=torch.float64))
    code, unit = ref.quantise(v, False)
    err = (ref.dequantise(code, unit) - v).abs()
    step = unit.double().repeat_interleave(256)[:1000]
    assert (err <= 2.0 ** -4 * v.abs() * (1 + 1e-6) + 2.0 ** -10 * step).all()
    code, unit = ref.quantise(torch.zeros(300, dtype=torch.float64), True)
    assert not code.float().any() and not unit.any()


# ------------------------------------------------------------------- refusals

def test_block_workspace_size(L):
    n = ctypes.c_size_t(0)
    for wl in W.ALL:
        desc = occ.desc_of(wl)
        assert L.occ_block_workspace_size(ctypes.byref(desc), ctypes.byref(n)) == occ.OCC_OK
        assert 0 < n.value < 256 << 20 and n.value % 256 == 0
        assert n.value == occ.occ_block_workspace_size(desc)
    assert L.occ_block_workspace_size(ctypes.byref(desc), None) == INV
    bad = occ.desc_of(W.OLMOE, T=0)
    assert L.occ_block_workspace_size(ctypes.byref(bad), ctypes.byref(n)) == INV
    assert L.occ_block_workspace_size(None, ctypes.byref(n)) == INV


def norm_status(L, desc=None, opt=None, **over):
    a = dict(x=fake(1), y=fake(2), w_post=fake(3), gate=NULL, w_pre=fake(4), r=fake(5), h=fake(6))
    a.update(over)
    desc = desc or occ.desc_of(W.OLMOE)
    opt = opt or occ.NormDesc(eps=1e-6, scale=1.0, gate=0)
    return L.occ_block_norm(ctypes.byref(desc), ctypes.byref(opt), *a.values(), NULL)


@pytest.mark.parametrize("over", [
    dict(x=NULL), dict(r=NULL), dict(h=NULL), dict(w_pre=NULL),
    dict(y=NULL), dict(y=NULL, r=NULL), dict(y=NULL, w_post=NULL),
    dict(y=NULL, r=NULL, w_post=NULL, w_pre=NULL, h=NULL),  # nothing to do
    dict(gate=fake(7)),                                     # a gate of kind none
    dict(x=ctypes.c_void_p(0x1008)), dict(h=ctypes.c_void_p(0x1002)),
    dict(w_pre=ctypes.c_void_p(0x1008)),
])
def test_norm_refuses_pointers(L, over):
    assert norm_status(L, **over) == INV


@pytest.mark.parametrize("over", [dict(r=fake(6)), dict(r=fake(3)), dict(h=fake(3)),
                                  dict(h=fake(4))])
def test_norm_refuses_an_output_in_another_array(L, over):
    assert norm_status(L, **over) == INV


@pytest.mark.parametrize("kind", [1, 2])
def test_norm_refuses_a_missing_gate(L, kind):
    assert norm_status(L, opt=occ.NormDesc(eps=1e-6, scale=1.0, gate=kind)) == INV
    at = ctypes.c_void_p(0x1008 if kind == 1 else 0x1002)
    assert norm_status(L, opt=occ.NormDesc(eps=1e-6, scale=1.0, gate=kind), gate=at) == INV


@pytest.mark.parametrize("bad", [dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")),
                                 dict(eps=float("inf")), dict(scale=float("nan")),
                                 dict(scale=float("inf")), dict(gate=3), dict(gate=-1)])
def test_norm_refuses_options(L, bad):
    opt = occ.NormDesc(**{**dict(eps=1e-6, scale=1.0, gate=0), **bad})
    assert norm_status(L, opt=opt) == INV
    assert norm_back_status(L, opt=opt) == INV


@pytest.mark.parametrize("eps", [1e-45, 1.1e-38])
def test_norm_refuses_an_eps_below_the_normal_numbers(L, eps):
    opt = occ.NormDesc(eps=eps, scale=1.0, gate=0)
    assert norm_status(L, opt=opt) == INV and norm_back_status(L, opt=opt) == INV


def test_norm_refuses_shapes(L):
    assert norm_status(L, desc=occ.desc_of(W.OLMOE, T=0)) == INV
    assert norm_status(L, desc=occ.desc_of(W.OLMOE, d=2000)) == UNS
    assert norm_status(L, desc=occ.desc_of(W.OLMOE, d=16384)) == UNS


def norm_back_status(L, desc=None, opt=None, **over):
    a = dict(dr=fake(1), dh=fake(2), r=fake(3), y=fake(4), w_post=fake(5), gate=NULL,
             w_pre=fake(6), dx=fake(7), dy=fake(8), dw_post=fake(9), dgate=NULL, dw_pre=fake(10),
             ws=fake(11), ws_bytes=BIG)
    a.update(over)
    desc = desc or occ.desc_of(W.OLMOE)
    opt = opt or occ.NormDesc(eps=1e-6, scale=1.0, gate=0)
    return L.occ_block_norm_backward(ctypes.byref(desc), ctypes.byref(opt), *a.values(), NULL)


@pytest.mark.parametrize("over,code", [
    (dict(dx=NULL), INV), (dict(dr=NULL, dh=NULL), INV), (dict(dh=NULL), INV),
    (dict(w_pre=NULL), INV), (dict(dw_pre=NULL), INV), (dict(dw_post=NULL), INV),
    (dict(w_post=NULL), INV), (dict(r=NULL), INV), (dict(y=NULL), INV), (dict(dy=NULL), INV),
    (dict(gate=fake(12)), INV), (dict(dgate=fake(12)), INV),
    (dict(dr=ctypes.c_void_p(0x1008)), INV), (dict(dy=ctypes.c_void_p(0x1008)), INV),
    (dict(dw_pre=ctypes.c_void_p(0x1002)), INV),
    (dict(ws=NULL), WS), (dict(ws=ctypes.c_void_p(0x1010)), WS), (dict(ws_bytes=64), WS),
])
def test_norm_backward_refuses_pointers(L, over, code):
    assert norm_back_status(L, **over) == code


@pytest.mark.parametrize("over", [
    dict(dx=fake(8)), dict(dx=fake(6)), dict(dy=fake(5)), dict(dw_post=fake(5)),
    dict(dw_pre=fake(5)), dict(dw_post=fake(10)), dict(dw_pre=fake(7)), dict(dw_pre=fake(2)),
    dict(dgate=fake(12)), dict(dgate=fake(9)),
])
def test_norm_backward_refuses_an_output_in_another_array(L, over):
    opt = occ.NormDesc(eps=1e-6, scale=1.0, gate=1)
    assert norm_back_status(L, opt=opt, **{**dict(gate=fake(12), dgate=fake(13)), **over}) == INV


def test_norm_backward_refuses_a_gate_without_its_gradient(L):
    opt = occ.NormDesc(eps=1e-6, scale=1.0, gate=2)
    assert norm_back_status(L, opt=opt, gate=fake(12)) == INV
    assert norm_back_status(L, opt=opt, dgate=fake(12)) == INV


def placement(wl=W.OLMOE):
    return np.ascontiguousarray(synth.contiguous_placement(wl))


def host(a):
    return ctypes.c_void_p(a.ctypes.data)


GOOD = placement()


def balance_status(L, opt=None, desc=None, **over):
    a = dict(logits=fake(1), ids=fake(2), valid=NULL, placement=host(GOOD), counts=fake(3),
             probs=fake(4), loss=fake(5), ws=fake(6), ws_bytes=BIG)
    a.update(over)
    desc = desc or occ.desc_of(W.OLMOE)
    opt = opt or occ.BalanceDesc(balance=1e-2, group=1e-3, z=1e-3)
    return L.occ_balance_loss(ctypes.byref(desc), ctypes.byref(opt), *a.values(), NULL)


def balance_back_status(L, opt=None, dloss=1.0, **over):
    a = dict(logits=fake(1), valid=NULL, placement=host(GOOD), counts=fake(2))
    b = dict(dlogits_in=fake(3), dlogits=fake(4))
    a.update({k: v for k, v in over.items() if k in a})
    b.update({k: v for k, v in over.items() if k in b})
    desc = occ.desc_of(W.OLMOE)
    opt = opt or occ.BalanceDesc(balance=1e-2, group=1e-3, z=1e-3)
    return L.occ_balance_backward(ctypes.byref(desc), ctypes.byref(opt), *a.values(), dloss,
                                  *b.values(), NULL)


@pytest.mark.parametrize("name", ["logits", "ids", "counts", "probs", "loss", "placement"])
def test_balance_refuses_missing_and_misaligned_arrays(L, name):
    assert balance_status(L, **{name: NULL}) == INV
    if name != "placement":
        assert balance_status(L, **{name: ctypes.c_void_p(0x1002)}) == INV


@pytest.mark.parametrize("name", ["logits", "counts", "dlogits", "placement"])
def test_balance_backward_refuses_missing_and_misaligned_arrays(L, name):
    assert balance_back_status(L, **{name: NULL}) == INV
    if name != "placement":
        assert balance_back_status(L, **{name: ctypes.c_void_p(0x1002)}) == INV


def test_balance_refuses_coefficients_placements_and_workspaces(L):
    for bad in (float("nan"), float("inf")):
        for f in ("balance", "group", "z"):
            opt = occ.BalanceDesc(**{**dict(balance=1.0, group=1.0, z=1.0), f: bad})
            assert balance_status(L, opt=opt) == INV
            assert balance_back_status(L, opt=opt) == INV
        assert balance_back_status(L, dloss=bad) == INV
    dup = GOOD.copy()
    dup[0, 0] = dup[0, 1]
    assert balance_status(L, placement=host(dup)) == INV
    assert balance_back_status(L, placement=host(dup)) == INV
    assert balance_status(L, ws=NULL) == WS
    assert balance_status(L, ws=ctypes.c_void_p(0x1010)) == WS
    assert balance_status(L, ws_bytes=16) == WS


@pytest.mark.parametrize("over", [dict(counts=fake(4)), dict(counts=fake(2)), dict(probs=fake(1)),
                                  dict(loss=fake(3)), dict(loss=fake(4)), dict(valid=fake(5))])
def test_balance_refuses_an_output_in_another_array(L, over):
    assert balance_status(L, **over) == INV


@pytest.mark.parametrize("over", [dict(dlogits=fake(2)), dict(valid=fake(4))])
def test_balance_backward_refuses_an_output_in_another_array(L, over):
    assert balance_back_status(L, **over) == INV


def gate_status(L, **over):
    a = dict(dlogits=fake(1), x=fake(2), w_router=fake(3), dx_in=fake(4), dx=fake(5),
             dw=fake(6), ws=fake(7), ws_bytes=BIG)
    a.update(over)
    desc = occ.desc_of(W.OLMOE)
    return L.occ_gate_backward(ctypes.byref(desc), *a.values(), NULL)


@pytest.mark.parametrize("over,code", [
    (dict(dlogits=NULL), INV), (dict(dx=NULL, dw=NULL), INV), (dict(dx=NULL, dx_in=NULL, dw=NULL), INV),
    (dict(dx=NULL), INV),        # dx_in without dx
    (dict(w_router=NULL), INV), (dict(x=NULL), INV),
    (dict(x=ctypes.c_void_p(0x1008)), INV), (dict(dw=ctypes.c_void_p(0x1004)), INV),
    (dict(dlogits=ctypes.c_void_p(0x1002)), INV),
    (dict(dx=fake(1)), INV), (dict(dx=fake(3)), INV), (dict(dx=fake(6)), INV),
    *[(dict(dw=fake(n)), INV) for n in (1, 2, 3, 4)],
    (dict(ws=NULL), WS), (dict(ws_bytes=16), WS), (dict(ws=ctypes.c_void_p(0x1010)), WS),
])
def test_gate_backward_refuses(L, over, code):
    assert gate_status(L, **over) == code


ADAM = dict(state=0, grad_dtype=0, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1,
            grad_scale=1.0, step=1)


def adam_status(L, tensor=None, opt=None, count=1, dynamic=NULL):
    row = occ.AdamwTensor(n=8, p=0x1000, g=0x2000, m=0x3000, v=0x4000, p_out=0x1000, m_out=0x3000,
                          v_out=0x4000)
    for name, value in (tensor or {}).items():
        setattr(row, name, value)
    desc = occ.AdamwDesc(**{**ADAM, **(opt or {})})
    return L.occ_adamw_step(ctypes.byref(desc), ctypes.byref(row), count, dynamic, NULL)


def test_adamw_structures_have_the_header_sizes():
    assert ctypes.sizeof(occ.AdamwDesc) == 64 and ctypes.sizeof(occ.AdamwTensor) == 104


def test_adamw_with_nothing_to_do_queues_nothing(L):
    assert adam_status(L, count=0) == occ.OCC_OK
    assert adam_status(L, tensor=dict(n=0, p=0, g=0)) == occ.OCC_OK


@pytest.mark.parametrize("tensor,code", [
    *[({name: 0}, INV) for name in ("p", "g", "m", "v", "p_out", "m_out", "v_out")],
    *[({name: 0x5002}, INV) for name in ("p", "g", "m", "v", "p_out", "m_out", "v_out")],
    *[({name: 0x5000}, INV) for name in ("m_scale", "v_scale", "m_scale_out", "v_scale_out")],
    (dict(p_bf16=0x5001), INV), (dict(n=-1), INV), (dict(n=(1 << 33) + 1), UNS),
])
def test_adamw_refuses_tensors(L, tensor, code):
    assert adam_status(L, tensor=tensor) == code


def test_adamw_refuses_missing_units_in_8_bits(L):
    scales = dict(m_scale=0x5000, v_scale=0x6000, m_scale_out=0x5000, v_scale_out=0x6000)
    for name in scales:
        assert adam_status(L, tensor={**scales, name: 0}, opt=dict(state=1)) == INV
        assert adam_status(L, tensor={**scales, name: 0x5002}, opt=dict(state=1)) == INV


@pytest.mark.parametrize("opt", [
    dict(state=2), dict(state=-1), dict(grad_dtype=2), dict(lr=-1e-3), dict(lr=float("nan")),
    dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0),
    dict(eps=-1.0), dict(eps=float("inf")), dict(weight_decay=-0.1),
    dict(grad_scale=float("inf")), dict(grad_scale=float("nan")), dict(step=0), dict(step=-3),
])
def test_adamw_refuses_options(L, opt):
    assert adam_status(L, opt=opt) == INV


def test_adamw_refuses_counts_and_dynamic(L):
    assert adam_status(L, count=-1) == INV
    assert adam_status(L, dynamic=ctypes.c_void_p(0x1002)) == INV
    desc = occ.AdamwDesc(**ADAM)
    assert L.occ_adamw_step(ctypes.byref(desc), None, 1, NULL, NULL) == INV
    assert L.occ_adamw_step(None, None, 0, NULL, NULL) == INV


@pytest.mark.parametrize("eps,code", [(1.1e-38, INV), (1e-45, INV), (1.2e-38, occ.OCC_OK)])
def test_adamw_takes_an_eps_that_is_a_normal_number(L, eps, code):
    assert adam_status(L, opt=dict(eps=eps), count=0) == code


@pytest.mark.parametrize("second", [dict(), dict(m=0x7000, m_out=0x7000, v=0x8000, v_out=0x8000),
                                    dict(p=0x6000, p_out=0x6000, v=0x8000, v_out=0x8000),
                                    dict(p=0x6000, p_out=0x6000, m=0x4000, m_out=0x4000)])
def test_adamw_refuses_an_array_written_twice(L, second):
    one = dict(n=8, p=0x1000, g=0x2000, m=0x3000, v=0x4000, p_out=0x1000, m_out=0x3000,
               v_out=0x4000)
    rows = (occ.AdamwTensor * 2)(occ.AdamwTensor(**one), occ.AdamwTensor(**{**one, **second}))
    desc = occ.AdamwDesc(**ADAM)
    assert L.occ_adamw_step(ctypes.byref(desc), rows, 2, NULL, NULL) == INV
    assert adam_status(L, tensor=dict(v_out=0x3000)) == INV


def test_binding_refuses_host_tensors_and_tables_that_do_not_fit(L):
    desc = occ.desc_of(W.TINY_F32)
    x = torch.zeros(W.TINY_F32.T, W.TINY_F32.d)
    opt = occ.NormDesc(eps=1e-6, scale=1.0, gate=0)
    with pytest.raises(ValueError, match="device tensor"):
        occ.occ_block_norm(desc, opt, x, None, None, None, x[0], None, x)
    with pytest.raises(ValueError, match="device tensor"):
        occ.occ_gate_backward(desc, torch.zeros(256, 8), x, x[:8], None, x, None, None)
    adam = occ.AdamwDesc(**ADAM)
    with pytest.raises(ValueError, match="device tensor"):
        occ.AdamwTensors(adam, [dict(p=x, g=x, m=x, v=x)])
    with pytest.raises(ValueError, match="unknown entries"):
        occ.AdamwTensors(adam, [dict(p=x, g=x, m=x, v=x, master=x)])
    with pytest.raises(ValueError, match="differ from the table"):
        occ.occ_adamw_step(occ.AdamwDesc(**{**ADAM, "state": 1}), occ.AdamwTensors(adam, []))
    with pytest.raises(ValueError, match="torch.bool"):
        occ.occ_balance_backward(desc, occ.BalanceDesc(), None, x, None, None, 1.0, None, None)
