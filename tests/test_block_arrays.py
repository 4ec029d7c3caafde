"""Refusals of the operators around the layer on the host (no GPU): arrays that a call writes, its
workspace among them, and that start like another array of the call, and optimizer values beyond
fp32."""
import ctypes

import pytest

from expert_token_routing_amd import occ
from test_block_host import (ADAM, INV, L, NULL, adam_status, balance_status, fake, gate_status,  # noqa: F401
                             norm_back_status)

# A tensor of its own arrays, and one of 8-bit states; written in place unless told otherwise.
ROW = dict(n=8, p=0x1000, g=0x2000, m=0x3000, v=0x4000, p_out=0x1000, m_out=0x3000, v_out=0x4000)
UNITS = dict(m_scale=0x5000, v_scale=0x6000, m_scale_out=0x5000, v_scale_out=0x6000)


def other(row):
    """The same tensor somewhere else."""
    return {key: v if key == "n" else v + 0x100000 for key, v in row.items()}


def adam_rows(L, rows, dynamic=NULL, **opt):
    table = (occ.AdamwTensor * len(rows))(*[occ.AdamwTensor(**r) for r in rows])
    desc = occ.AdamwDesc(**{**ADAM, **opt})
    return L.occ_adamw_step(ctypes.byref(desc), table, len(rows), dynamic, NULL)


@pytest.mark.parametrize("over", [
    dict(p_bf16=0x1000), dict(p_bf16=0x2000), dict(p_bf16=0x3000), dict(p_bf16=0x4000),
    dict(p_out=0x2000), dict(m_out=0x2000), dict(v_out=0x2000),      # over the gradient
    dict(p_out=0x3000, m_out=0x7000), dict(m_out=0x4000, v_out=0x7000),
    dict(v_out=0x1000, p_out=0x7000),                                 # over another one's old value
], ids=str)
def test_adamw_refuses_an_output_in_another_array(L, over):
    assert adam_rows(L, [{**ROW, **over}]) == INV
    assert adam_rows(L, [other(ROW), {**ROW, **over}]) == INV


@pytest.mark.parametrize("over", [
    dict(m_scale_out=0x6000, v_scale_out=0x6000), dict(m_scale_out=0x1000), dict(v_scale_out=0x3000),
    dict(m_scale_out=0x6000, v_scale_out=0x7000), dict(v_scale_out=0x2000), dict(p_bf16=0x5000),
    dict(p_bf16=0x6000), dict(p_out=0x5000), dict(m_out=0x6000),
], ids=str)
def test_adamw_refuses_units_in_another_array(L, over):
    row = {**ROW, **UNITS}
    assert adam_rows(L, [{**row, **over}], state=1) == INV
    assert adam_rows(L, [{**row, **over}, other(row)], state=1) == INV


@pytest.mark.parametrize("name", ["p", "g", "m", "v", "m_scale", "v_scale"])
@pytest.mark.parametrize("out", ["p_out", "m_out", "v_out", "m_scale_out", "v_scale_out", "p_bf16"])
def test_adamw_refuses_an_output_in_an_array_of_another_tensor(L, out, name):
    row = {**ROW, **UNITS}
    second = {**other(row), out: row[name]}
    assert adam_rows(L, [row, second], state=1) == INV
    assert adam_rows(L, [second, row], state=1) == INV
    # out of place: no output of the first tensor stands in the way
    away = {**row, **{key: v + 0x200000 for key, v in row.items() if key.endswith("_out")}}
    assert adam_rows(L, [away, second], state=1) == INV


@pytest.mark.parametrize("out", ["m_scale_out", "v_scale_out", "p_bf16"])
def test_adamw_refuses_units_and_copies_written_by_two_tensors(L, out):
    row = {**ROW, **UNITS, "p_bf16": 0x7000}
    assert adam_rows(L, [row, {**other(row), out: row[out]}], state=1) == INV


def test_adamw_refuses_an_output_in_the_dynamic_values(L):
    assert adam_rows(L, [{**ROW, "p_bf16": 0x7000}], dynamic=ctypes.c_void_p(0x7000)) == INV
    assert adam_rows(L, [ROW], dynamic=ctypes.c_void_p(0x1000)) == INV


@pytest.mark.parametrize("name", ["dr", "dh", "r", "y", "w_post", "w_pre", "gate", "dx", "dy",
                                  "dw_post", "dw_pre", "dgate"])
def test_norm_backward_refuses_a_workspace_in_another_array(L, name):
    opt = occ.NormDesc(eps=1e-6, scale=1.0, gate=1)
    arrays = dict(gate=fake(12), dgate=fake(13))
    assert norm_back_status(L, opt=opt, **{**arrays, name: fake(11)}) == INV


@pytest.mark.parametrize("name", ["logits", "ids", "valid", "counts", "probs", "loss"])
def test_balance_refuses_a_workspace_in_another_array(L, name):
    assert balance_status(L, **{name: fake(6)}) == INV


@pytest.mark.parametrize("name", ["dlogits", "x", "w_router", "dx_in", "dx", "dw"])
def test_gate_backward_refuses_a_workspace_in_another_array(L, name):
    assert gate_status(L, **{name: fake(7)}) == INV


@pytest.mark.parametrize("opt", [dict(lr=1e39), dict(eps=1e39), dict(weight_decay=1e300),
                                 dict(grad_scale=1e39), dict(grad_scale=-1e39)], ids=str)
def test_adamw_refuses_values_beyond_fp32(L, opt):
    assert adam_status(L, opt=opt, count=0) == INV


@pytest.mark.parametrize("opt", [dict(lr=3e38), dict(eps=3e38), dict(weight_decay=3e38),
                                 dict(grad_scale=-3e38), dict(lr=0.0), dict(lr=1e-60)], ids=str)
def test_adamw_takes_the_values_that_fp32_holds(L, opt):
    assert adam_status(L, opt=opt, count=0) == occ.OCC_OK
