"""The operators around the layer on the GPU against plain 64-bit implementations
(block_reference.py): the norms between two blocks, the router's losses, the gate projection's
backward and the AdamW step, at the sizes, masks, alignments and values where they can go wrong;
then in place, on side streams, captured and replayed, and together in one training step.

Tolerances are bounds by arithmetic, per element: half a step of the output's type, plus n u times
the sum of the magnitudes that the value is made of (u = 2^-24, n at least the number of fp32
roundings on its longest path), the magnitudes taken from the 64-bit reference."""
import ctypes

import numpy as np
import pytest
import torch

import block_reference as ref
from block_reference import U, half_step
from expert_token_routing_amd import occ, synth, workloads as W

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    occ.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def nan_like(shape, dtype=F32):
    """Outputs start as NaN, so that a value that is not written shows."""
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def layer(T, d=64, Ne=1, k=1, Nd=1, dtype=F32):
    return occ.LayerDesc(T=T, d=d, Ne=Ne, k=k, Nd=Nd, F=64, n_shared=0, F_shared=0, prune_rule=0,
                         prune_groups=0, dtype=occ.OCC_BF16 if dtype == BF16 else occ.OCC_F32,
                         flags=0)


def check(got, want, mag, n, what):
    """|got - want| within half a step of got's type and n u of the magnitudes."""
    bound = half_step(got.dtype) * want.abs() * (1 + 2.0 ** -8) + n * U * mag + 2.0 ** -126
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((off / bound).nan_to_num(1e9).max()))


# ---------------------------------------------------------------------- norms

EPS, SCALE = 1e-6, 0.7

# (y, norm behind, gate kind, norm in front, dr)
FORMS = {
    "sandwich": (True, True, 0, True, True),
    "channel": (True, True, 1, True, True),
    "token": (True, True, 2, True, True),
    "prenorm": (True, False, 0, True, True),
    "prenorm_token": (True, False, 2, True, False),
    "prenorm_channel": (True, False, 1, False, True),
    "last": (True, True, 0, False, True),
    "first": (False, False, 0, True, True),
    "first_alone": (False, False, 0, True, False),
}

# rows of one wave (1, 2 and 4 chunks a lane, full and partly empty) and of a workgroup (2 and 4),
# fewer rows than waves, more rows than the forward's and the backward's workgroups walk at once
NORM_SHAPES = [(BF16, 1, 64), (BF16, 3, 192), (BF16, 7, 512), (BF16, 130, 1024), (BF16, 33, 1088),
               (BF16, 1001, 2048), (BF16, 5, 2112), (BF16, 600, 4096), (BF16, 3, 4160),
               (BF16, 70, 8192), (BF16, 9000, 64), (F32, 1, 16), (F32, 37, 80), (F32, 11, 272),
               (F32, 300, 1024), (F32, 65, 1040), (F32, 6, 4096), (F32, 2100, 48), (BF16, 5000, 256), (F32, 70000, 16)]


def norm_inputs(dtype, T, d, form, seed):
    y, post, kind, pre, dr = FORMS[form]
    g = gen(seed)
    t = dict(x=(2 * randn(g, T, d)).to(dtype), y=randn(g, T, d).to(dtype) if y else None,
             w_post=(1 + 0.2 * randn(g, d)).to(dtype) if post else None,
             gate=(None if kind == 0 else (0.5 + 0.3 * randn(g, d)).to(dtype) if kind == 1
                   else torch.sigmoid(randn(g, T))),
             w_pre=(1 + 0.2 * randn(g, d)).to(dtype) if pre else None)
    grads = dict(dr=randn(g, T, d).to(dtype) if dr else None,
                 dh=randn(g, T, d).to(dtype) if pre else None)
    return t, grads, occ.NormDesc(eps=EPS, scale=SCALE, gate=kind)


def run_norm(t, opt, dtype, stream=None):
    T, d = t["x"].shape
    r = nan_like((T, d), dtype) if t["y"] is not None else None
    h = nan_like((T, d), dtype) if t["w_pre"] is not None else None
    occ.occ_block_norm(layer(T, d, dtype=dtype), opt, t["x"], t["y"], t["w_post"], t["gate"],
                       t["w_pre"], r, h, stream=stream)
    return r, h


def run_norm_back(t, grads, r, opt, dtype, ws=None, stream=None):
    T, d = t["x"].shape
    desc = layer(T, d, dtype=dtype)
    out = dict(dx=nan_like((T, d), dtype), dy=nan_like((T, d), dtype) if t["y"] is not None else None,
               dw_post=nan_like((d,)) if t["w_post"] is not None else None,
               dgate=nan_like(t["gate"].shape) if t["gate"] is not None else None,
               dw_pre=nan_like((d,)) if t["w_pre"] is not None else None)
    ws = occ.alloc_block_workspace(desc) if ws is None else ws
    occ.occ_block_norm_backward(desc, opt, grads["dr"], grads["dh"], r, t["y"], t["w_post"],
                                t["gate"], t["w_pre"], out["dx"], out["dy"], out["dw_post"],
                                out["dgate"], out["dw_pre"], ws, stream=stream)
    return out


def check_norm(t, opt, r, h):
    want_r, want_h, mag = ref.block_norm(**t, kind=opt.gate, eps=opt.eps, scale=opt.scale)
    # r: one row statistic (a sum of d squares in at most 64 + 10 steps, halved by the root), five
    # products and one addition
    if r is not None:
        check(r, want_r, mag, 64, "r")
    if h is not None:
        # the same error of r, its statistic and two products, through the norm
        rstd = 1 / torch.sqrt((want_r * want_r).mean(1, keepdim=True) + opt.eps)
        check(h, want_h, rstd * t["w_pre"].double().abs() * mag, 160, "h")


def check_norm_back(t, grads, r, opt, out):
    want, mag = ref.block_norm_back(grads["dr"], grads["dh"], r, t["y"], t["w_post"], t["gate"],
                                    t["w_pre"], opt.gate, opt.eps, opt.scale)
    for name, n in (("dx", 256), ("dy", 640), ("dw_pre", 256), ("dw_post", 512), ("dgate", 512)):
        assert (out[name] is None) == (name not in want), name
        if out[name] is not None:
            check(out[name], want[name], mag[name], n, name)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype,T,d", NORM_SHAPES,
                         ids=[f"{'bf16' if t == BF16 else 'f32'}-{T}-{d}" for t, T, d in NORM_SHAPES])
def test_norm_forward_and_backward(dtype, T, d, form):
    t, grads, opt = norm_inputs(dtype, T, d, form, seed=T + d)
    r, h = run_norm(t, opt, dtype)
    check_norm(t, opt, r, h)
    kept = r if r is not None else t["x"]
    out = run_norm_back(t, grads, kept, opt, dtype)
    check_norm_back(t, grads, kept, opt, out)


def test_norm_backward_without_y_when_nothing_reads_it():
    """Neither norm nor gate behind the block: dy = scale dr', with y or without."""
    t, grads, opt = norm_inputs(BF16, 50, 320, "prenorm", seed=9)
    r, _ = run_norm(t, opt, BF16)
    want = run_norm_back(t, grads, r, opt, BF16)
    dx, dy, dw = nan_like((50, 320), BF16), nan_like((50, 320), BF16), nan_like((320,))
    desc = layer(50, 320, dtype=BF16)
    occ.occ_block_norm_backward(desc, opt, grads["dr"], grads["dh"], r, None, None, None,
                                t["w_pre"], dx, dy, None, None, dw,
                                occ.alloc_block_workspace(desc))
    assert torch.equal(dx, want["dx"]) and torch.equal(dy, want["dy"])
    assert torch.equal(dw, want["dw_pre"])


def test_norm_rows_of_zeros_and_of_extreme_size():
    t, grads, opt = norm_inputs(BF16, 12, 256, "channel", seed=1)
    t["x"][0], t["y"][0] = 0, 0          # nothing in the row: h = 0, gradients finite
    t["y"][1] = 0                         # nothing from the block
    t["x"][2], t["y"][2] = t["x"][2] * 1e10, t["y"][2] * 1e10
    t["x"][3], t["y"][3] = t["x"][3] * 1e-10, t["y"][3] * 1e-10  # far below eps
    r, h = run_norm(t, opt, BF16)
    check_norm(t, opt, r, h)
    assert not h[0].any()
    out = run_norm_back(t, grads, r, opt, BF16)
    check_norm_back(t, grads, r, opt, out)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 256), (BF16, 2048), (BF16, 8192), (F32, 48),
                                     (F32, 4096)])
@pytest.mark.parametrize("form", list(FORMS))
def test_norm_backward_of_few_rows(form, dtype, d):
    """From one row to more than a single workgroup takes: 1, 2, 4, 8, ... rows and one more."""
    for T in (1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257):
        t, grads, opt = norm_inputs(dtype, T, d, form, seed=T)
        r, h = run_norm(t, opt, dtype)
        check_norm(t, opt, r, h)
        kept = r if r is not None else t["x"]
        check_norm_back(t, grads, kept, opt, run_norm_back(t, grads, kept, opt, dtype))


def test_norm_with_the_smallest_eps():
    t, _, _ = norm_inputs(F32, 5, 1040, "channel", seed=2)
    t["x"][1:3] = 0
    t["y"][2:4] = 0
    t["x"][4] *= 1e-18
    opt = occ.NormDesc(eps=2.0 ** -126, scale=SCALE, gate=1)
    r, h = run_norm(t, opt, F32)
    want_r, want_h, mag = ref.block_norm(**t, kind=1, eps=opt.eps, scale=SCALE)
    check(r, want_r, mag, 64, "r")
    assert (h[2] == 0).all() and h.isfinite().all()


def test_norm_keeps_what_is_not_finite_in_its_row():
    t, grads, opt = norm_inputs(BF16, 40, 2048, "token", seed=2)
    clean_r, clean_h = run_norm(t, opt, BF16)
    clean = run_norm_back(t, grads, clean_r, opt, BF16)
    t["y"][7, 100], t["x"][9, 5] = float("nan"), float("inf")
    r, h = run_norm(t, opt, BF16)
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[7] = rows[9] = False
    assert torch.equal(r[rows], clean_r[rows]) and torch.equal(h[rows], clean_h[rows])
    assert h[7].isnan().all() and h[9].isnan().any()
    out = run_norm_back(t, grads, r, opt, BF16)
    for name in ("dx", "dy", "dgate"):
        assert torch.equal(out[name][rows], clean[name][rows]), name


def test_norm_in_place_and_repeated_bitwise():
    for dtype, T, d in ((BF16, 517, 2048), (F32, 77, 4096)):
        t, grads, opt = norm_inputs(dtype, T, d, "channel", seed=3)
        r, h = run_norm(t, opt, dtype)
        out = run_norm_back(t, grads, r, opt, dtype)
        again = run_norm_back(t, grads, r, opt, dtype)
        assert all(torch.equal(out[key], again[key]) for key in out)
        x, y = t["x"].clone(), t["y"].clone()
        desc = layer(T, d, dtype=dtype)
        occ.occ_block_norm(desc, opt, x, y, t["w_post"], t["gate"], t["w_pre"], x, y)
        assert torch.equal(x, r) and torch.equal(y, h)
        dr, dh = grads["dr"].clone(), grads["dh"].clone()
        w = [nan_like((d,)) for _ in range(3)]
        occ.occ_block_norm_backward(desc, opt, dr, dh, r, t["y"], t["w_post"], t["gate"],
                                    t["w_pre"], dr, dh, *w, occ.alloc_block_workspace(desc))
        assert torch.equal(dr, out["dx"]) and torch.equal(dh, out["dy"])


@pytest.mark.parametrize("dtype,T,d", [(BF16, 3001, 128), (BF16, 1100, 2048), (F32, 900, 4096)])
@pytest.mark.parametrize("form", ["token", "channel"])
def test_norm_outputs_over_any_input_of_the_same_rows(form, dtype, T, d):
    t, grads, opt = norm_inputs(dtype, T, d, form, seed=5)
    r, h = run_norm(t, opt, dtype)
    want = run_norm_back(t, grads, r, opt, dtype)
    desc, ws = layer(T, d, dtype=dtype), occ.alloc_block_workspace(layer(T, d, dtype=dtype))
    for r_at, h_at in (("y", "x"), ("x", None), (None, "x"), ("y", None), (None, "y")):
        rows = {"x": t["x"].clone(), "y": t["y"].clone()}
        r2, h2 = rows.get(r_at, nan_like((T, d), dtype)), rows.get(h_at, nan_like((T, d), dtype))
        occ.occ_block_norm(desc, opt, rows["x"], rows["y"], t["w_post"], t["gate"], t["w_pre"], r2, h2)
        assert torch.equal(r2, r) and torch.equal(h2, h), (r_at, h_at)
    for dx_at, dy_at in (("dh", "dr"), ("r", "y"), ("y", "r"), ("r", "dh")):
        rows = {"dr": grads["dr"].clone(), "dh": grads["dh"].clone(), "r": r.clone(), "y": t["y"].clone()}
        gate = t["gate"].clone()
        dgate = gate if form == "token" else nan_like((d,))
        dw = [nan_like((d,)) for _ in range(2)]
        occ.occ_block_norm_backward(desc, opt, rows["dr"], rows["dh"], rows["r"], rows["y"],
                                    t["w_post"], gate, t["w_pre"], rows[dx_at], rows[dy_at], dw[0],
                                    dgate, dw[1], ws)
        got = dict(dx=rows[dx_at], dy=rows[dy_at], dw_post=dw[0], dgate=dgate, dw_pre=dw[1])
        assert all(torch.equal(got[key], want[key]) for key in got), (dx_at, dy_at)


# -------------------------------------------------------------- router losses

COEF = (0.3, 0.2, 0.05)

BALANCE_SHAPES = [(1, 1, 1, 1), (2, 2, 1, 1), (31, 8, 2, 2), (33, 15, 3, 5), (500, 16, 4, 4),
                  (129, 17, 2, 1), (64, 32, 8, 8), (100, 33, 1, 3), (5000, 60, 4, 4),
                  (512, 64, 8, 8), (77, 65, 5, 5), (300, 128, 8, 64), (41, 129, 6, 3),
                  (90, 200, 32, 10), (1000, 256, 8, 8), (20000, 64, 8, 4)]


def balance_inputs(T, Ne, k, Nd, mask, seed):
    g = gen(seed)
    logits = 2 * randn(g, T, Ne)
    ids = torch.topk(logits, k, dim=1).indices.int()
    valid = None
    if mask != "none":
        valid = torch.rand(T, generator=g, device="cuda") < 0.7
        if mask == "empty":
            valid[:] = False
        if mask == "one":
            valid[:] = False
            valid[T // 2] = True
        # what padding rows hold must not matter
        logits[~valid] = torch.tensor([float("nan"), float("inf"), -float("inf")],
                                      device="cuda").repeat(Ne)[:Ne]
        ids[~valid] = -7
    place = torch.randperm(Ne, generator=torch.Generator().manual_seed(seed)).int()
    place = place.view(Nd, Ne // Nd).numpy()
    group = torch.empty(Ne, dtype=torch.long)
    for q in range(Nd):
        group[torch.from_numpy(place[q]).long()] = q
    return logits, ids, valid, place, group.cuda()


def run_balance(T, Ne, k, Nd, logits, ids, valid, place, dlogits_in, up=0.5, coef=COEF, ws=None):
    desc = layer(T, Ne=Ne, k=k, Nd=Nd)
    opt = occ.BalanceDesc(balance=coef[0], group=coef[1], z=coef[2])
    counts = torch.full((Ne + 1,), -1, dtype=torch.int32, device="cuda")
    probs, loss, dlogits = nan_like((Ne,)), nan_like((4,)), nan_like((T, Ne))
    ws = occ.alloc_block_workspace(desc) if ws is None else ws
    occ.occ_balance_loss(desc, opt, logits, ids, valid, place, counts, probs, loss, ws)
    occ.occ_balance_backward(desc, opt, logits, valid, place, counts, up, dlogits_in, dlogits)
    return counts, probs, loss, dlogits


def check_balance(logits, ids, valid, group, k, dlogits_in, got, up=0.5, coef=COEF):
    counts, probs, loss, dlogits = got
    want_loss, want_p, want_c, kept = ref.balance(logits, ids, valid, group, k, coef)
    assert torch.equal(counts.long(), want_c)
    rows = slice(None) if valid is None else valid
    spread = 0.0
    if kept is not None:
        seen = logits[rows]
        seen = seen[seen.isfinite()]
        spread = float(seen.max() - seen.min()) if seen.numel() else 0.0
    # p: u times the exponents' size, a sum of up to 256 values (4 + 6 steps) and a division;
    # P: sums of p over a lane's tokens (at most 64 at these sizes), teams, waves
    n = 2 * spread + 32
    check(probs, want_p, want_p, n + 96, "probs")
    check(loss, want_loss.to(loss.device), want_loss.abs().to(loss.device), 2 * n + 128, "loss")
    want, mag = ref.balance_back(logits, kept, coef, up, dlogits_in)
    check(dlogits, want, mag, 2 * n + 32, "dlogits")


@pytest.mark.parametrize("mask", ["none", "some", "empty", "one"])
@pytest.mark.parametrize("T,Ne,k,Nd", BALANCE_SHAPES)
def test_balance_loss_and_gradient(T, Ne, k, Nd, mask):
    logits, ids, valid, place, group = balance_inputs(T, Ne, k, Nd, mask, seed=T + Ne)
    dlogits_in = randn(gen(9), T, Ne) * 1e-3 if T % 2 else None
    got = run_balance(T, Ne, k, Nd, logits, ids, valid, place, dlogits_in)
    check_balance(logits, ids, valid, group, k, dlogits_in, got)
    if valid is not None and mask == "empty":
        assert not got[2].any() and not got[1].any() and not got[0].any()
        assert torch.equal(got[3], torch.zeros_like(got[3]) if dlogits_in is None else dlogits_in)


def test_balance_with_masked_experts_lowest_values_and_empty_rows():
    T, Ne, k, Nd = 200, 60, 4, 4
    logits, ids, _, place, group = balance_inputs(T, Ne, k, Nd, "none", seed=4)
    logits[::3, :20] = -float("inf")              # experts masked out of some rows
    logits[1::5, 40:] = torch.finfo(F32).min      # a mask of the type's lowest value
    logits[7] = -float("inf")                     # a row with no expert left
    logits[8] = torch.finfo(F32).min              # all equal, however low
    coef = (0.3, 0.2, 0.0)  # the square of the lowest value's log-sum-exp is infinite
    got = run_balance(T, Ne, k, Nd, logits, ids, None, place, None, coef=coef)
    assert torch.isfinite(got[3]).all() and torch.isfinite(got[2][:3]).all()
    assert not got[3][7].any() and not got[3][::3][1:, :20].any()
    want_loss, want_p, want_c, kept = ref.balance(logits, ids, None, group, k, coef)
    assert torch.equal(got[0].long(), want_c)
    check(got[1], want_p, want_p, 160, "probs")
    want, mag = ref.balance_back(logits, kept, coef, 0.5, None)
    check(got[3], want, mag, 160, "dlogits")


def test_balance_ignores_ids_out_of_range_and_counts_repeats():
    T, Ne, k, Nd = 50, 8, 3, 2
    logits, ids, _, place, group = balance_inputs(T, Ne, k, Nd, "none", seed=5)
    ids[3], ids[4, 0], ids[5, 1] = 2, -1, Ne
    ids[6, 2] = 2 ** 31 - 1
    got = run_balance(T, Ne, k, Nd, logits, ids, None, place, None)
    check_balance(logits, ids, None, group, k, None, got)
    assert int(got[0][:Ne].sum()) == T * k - 3


@pytest.mark.parametrize("T,Ne", [(513, 64), (700, 100), (300, 252), (9, 36)])
@pytest.mark.parametrize("offset", [0, 1])
def test_balance_with_and_without_whole_vectors(offset, T, Ne):
    """Every fourth expert count with logits and dlogits on and off a vector's border."""
    logits, ids, valid, place, group = balance_inputs(T, Ne, 4, 1, "some", seed=Ne)
    into, out = (torch.empty(T * Ne + offset, device="cuda")[offset:].view(T, Ne) for _ in range(2))
    into.copy_(randn(gen(2), T, Ne))
    own = torch.empty(T * Ne + offset, device="cuda")[offset:].view(T, Ne).copy_(logits)
    got = run_balance(T, Ne, 4, 1, own, ids, valid, place, into)
    check_balance(logits, ids, valid, group, 4, into, got)
    desc, opt = layer(T, Ne=Ne, k=4), occ.BalanceDesc(balance=COEF[0], group=COEF[1], z=COEF[2])
    occ.occ_balance_backward(desc, opt, own, valid, place, got[0], 0.5, into, out)
    check_balance(logits, ids, valid, group, 4, into, (*got[:3], out))


def test_balance_in_place_uint8_mask_and_no_placement():
    T, Ne, k = 300, 60, 4
    logits, ids, valid, place, group = balance_inputs(T, Ne, k, 1, "some", seed=6)
    coef = (0.3, 0.0, 0.05)
    into = randn(gen(1), T, Ne)
    want = run_balance(T, Ne, k, 1, logits, ids, valid, place, into, coef=coef)
    desc, opt = layer(T, Ne=Ne, k=k), occ.BalanceDesc(balance=coef[0], group=0.0, z=coef[2])
    occ.occ_balance_backward(desc, opt, logits, valid.to(torch.uint8), None, want[0], 0.5, into, into)
    assert torch.equal(into, want[3])
    # over the logits themselves
    own = logits.clone()
    alone = nan_like((T, Ne))
    occ.occ_balance_backward(desc, opt, logits, valid, None, want[0], 0.5, None, alone)
    occ.occ_balance_backward(desc, opt, own, valid, None, want[0], 0.5, None, own)
    assert torch.equal(own, alone)


# ----------------------------------------------------- gate projection, back

GATE_SHAPES = [(BF16, T, d, Ne) for T, d, Ne in
               [(1, 64, 1), (15, 128, 7), (16, 192, 8), (17, 256, 16), (33, 320, 17),
                (127, 2048, 33), (128, 64, 60), (129, 2112, 64), (300, 512, 65), (1000, 256, 100),
                (257, 128, 128), (90, 576, 130), (513, 2048, 256), (3000, 128, 60),
                (40000, 64, 30), (8200, 1024, 70), (5000, 1984, 67), (40, 8192, 200),
                (128, 320, 66), (3000, 8192, 20), (1100, 2048, 90), (64, 2048, 250), (63, 128, 129),
                (1000, 2048, 65), (129, 8192, 96), (130, 128, 250)]] + \
              [(F32, T, d, Ne) for T, d, Ne in
               [(1, 16, 1), (5, 48, 3), (63, 80, 8), (64, 128, 17), (65, 272, 60), (300, 64, 64),
                (1000, 144, 65), (130, 1024, 129), (77, 336, 256), (20000, 32, 8), (700, 4096, 31), (64, 16, 16), (9, 64, 250),
                (31, 2048, 70), (33, 80, 100), (500, 2048, 250), (600, 4096, 66), (1100, 2048, 9),
                (1040, 2048, 40)]]


def gate_inputs(dtype, T, d, Ne, seed):
    g = gen(seed)
    return (randn(g, T, Ne) * torch.exp(randn(g, T, Ne)), randn(g, T, d).to(dtype),
            (0.3 * randn(g, Ne, d)).to(dtype), randn(g, T, d).to(dtype))


def check_gate(dl, x, w, dx_in, dx, dw, T, Ne, dtype):
    want_dx, mdx, want_dw, mdw = ref.gate_back(dl, x, w, dx_in)
    if dx is not None:
        # fp32 sums of Ne products; with bf16 tensors dlogits keep 16 bits: 2^-16 = 2^8 u
        check(dx, want_dx, mdx, Ne + 8 + (256 if dtype == BF16 else 0), "dx")
    if dw is not None:
        # sums of T products of exact terms, in three parts with bf16 tensors
        check(dw, want_dw, mdw, T + 64, "dw")


@pytest.mark.parametrize("dtype,T,d,Ne", GATE_SHAPES,
                         ids=[f"{'bf16' if s[0] == BF16 else 'f32'}-{s[1]}-{s[2]}-{s[3]}"
                              for s in GATE_SHAPES])
def test_gate_backward(dtype, T, d, Ne):
    dl, x, w, dx_in = gate_inputs(dtype, T, d, Ne, seed=T + Ne)
    desc = layer(T, d, Ne=Ne, dtype=dtype)
    ws = occ.alloc_block_workspace(desc)
    dx, dw = nan_like((T, d), dtype), nan_like((Ne, d))
    occ.occ_gate_backward(desc, dl, x, w, dx_in, dx, dw, ws)
    check_gate(dl, x, w, dx_in, dx, dw, T, Ne, dtype)
    # each product alone gives the same bits; without dx_in, the product itself
    dx2, dw2, bare = nan_like((T, d), dtype), nan_like((Ne, d)), nan_like((T, d), dtype)
    occ.occ_gate_backward(desc, dl, None, w, dx_in, dx2, None, None)
    occ.occ_gate_backward(desc, dl, x, None, None, None, dw2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    occ.occ_gate_backward(desc, dl, None, w, None, bare, None, None)
    check_gate(dl, x, w, None, bare, None, T, Ne, dtype)
    # in place, over dx_in and over x
    occ.occ_gate_backward(desc, dl, x, w, dx_in, dx_in, dw2, ws)
    assert torch.equal(dx_in, dx) and torch.equal(dw2, dw)
    occ.occ_gate_backward(desc, dl, x, w, None, x, dw2, ws)
    assert torch.equal(x, bare) and torch.equal(dw2, dw)


def test_gate_backward_unaligned_dlogits():
    T, d, Ne = 100, 256, 64
    dl, x, w, dx_in = gate_inputs(BF16, T, d, Ne, seed=3)
    desc = layer(T, d, Ne=Ne, dtype=BF16)
    ws = occ.alloc_block_workspace(desc)
    off = torch.empty(T * Ne + 1, device="cuda")[1:].view(T, Ne)
    off.copy_(dl)
    assert off.data_ptr() % 16 == 4 and off.is_contiguous()
    out = []
    for a in (dl, off):
        dx, dw = nan_like((T, d), BF16), nan_like((Ne, d))
        occ.occ_gate_backward(desc, a, x, w, dx_in, dx, dw, ws)
        out.append((dx, dw))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_gate_backward_of_empty_rows_is_dx_in():
    T, d, Ne = 70, 192, 20
    dl, x, w, dx_in = gate_inputs(BF16, T, d, Ne, seed=4)
    dl[10:50] = 0
    desc = layer(T, d, Ne=Ne, dtype=BF16)
    dx, dw = nan_like((T, d), BF16), nan_like((Ne, d))
    occ.occ_gate_backward(desc, dl, x, w, dx_in, dx, dw, occ.alloc_block_workspace(desc))
    assert torch.equal(dx[10:50], dx_in[10:50])
    check_gate(dl, x, w, dx_in, dx, dw, T, Ne, BF16)


# ---------------------------------------------------------------------- AdamW

ADAM = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=3, grad_scale=0.5)
SIZES = [1, 2, 3, 4, 5, 63, 255, 256, 257, 511, 1023, 1025, 4095, 4096, 4097, 10000, 70001]


def adam_inputs(sizes, bits, grad, seed, offset=0):
    g, tensors = gen(seed), []

    def place(v, dtype=F32):
        """v in a buffer of its own, `offset` elements behind an aligned start."""
        buf = torch.empty(v.numel() + offset, dtype=dtype, device="cuda")[offset:]
        buf.copy_(v.to(dtype))
        return buf

    for n in sizes:
        m, root = 1e-3 * randn(g, n), 1e-3 * torch.exp(randn(g, n))
        t = dict(p=place(randn(g, n)), g=place(2e-3 * randn(g, n), grad))
        if bits == 32:
            t.update(m=place(m), v=place(root * root))
        else:
            for key, value, keep in (("m", m, False), ("v", root, True)):
                code, unit = ref.quantise(value.double(), keep)
                t[key], t[key + "_scale"] = place(code, torch.float8_e4m3fn), unit
        tensors.append(t)
    return tensors


def adam_outputs(tensors, copy, in_place):
    out = []
    for t in tensors:
        o = {}
        if not in_place:
            o = {key + "_out": torch.empty_like(v) for key, v in t.items() if key != "g"}
        if copy:
            o["p_bf16"] = nan_like(t["p"].shape, BF16)
        out.append({**t, **o})
    return out


def adam_desc(bits, grad, **over):
    return occ.AdamwDesc(state=occ.OCC_ADAMW_8BIT if bits == 8 else occ.OCC_ADAMW_32BIT,
                         grad_dtype=occ.OCC_BF16 if grad == BF16 else occ.OCC_F32,
                         **{**ADAM, **over})


def moments(t, which=""):
    """A tensor's m and v in fp64."""
    m, v = t["m" + which], t["v" + which]
    if t.get("m_scale") is None:
        return m.double(), v.double()
    return (ref.dequantise(m, t["m_scale" + which]),
            ref.dequantise(v, t["v_scale" + which]) ** 2)


def check_adam(before, after, bits, a=ADAM):
    """after: dict of p, m, v (, scales, p_bf16) written by the step from `before`."""
    m0, v0 = moments(before)
    g = before["g"].double() * a["grad_scale"]
    p, m, v, step = ref.adamw(before["p"].double(), before["g"].double(), m0, v0, a)
    # the step: m's error of 4 u of its terms, v's of 6 u (halved by the root), the bias
    # corrections, root, addition, division and rate: 24 u of the step that m's terms would make
    m_mag = a["beta1"] * m0.abs() + (1 - a["beta1"]) * g.abs()
    c1, c2 = 1 - a["beta1"] ** a["step"], 1 - a["beta2"] ** a["step"]
    step_mag = a["lr"] / c1 * m_mag / (torch.sqrt(v / c2) + a["eps"])
    check(after["p"], p, p.abs() + 12 * step_mag, 2, "p")
    if after.get("p_bf16") is not None:
        assert torch.equal(after["p_bf16"], after["p"].to(BF16))
    if bits == 32:
        check(after["m"], m, m_mag, 4, "m")
        check(after["v"], v, v, 6, "v")
        return
    for key, want in (("m", m), ("v", torch.sqrt(v))):
        unit, code = after[key + "_scale"], after[key].float().double()
        top = ref.blocks(want).abs().max(1).values
        mag = ref.blocks(m_mag).max(1).values if key == "m" else top
        assert ((unit.double() - top / 448).abs() <= (mag * 8 * U) / 448 + 1e-40).all(), key
        each = unit.double().repeat_interleave(256)[:want.numel()]
        # half a step of e4m3 relative to the value, or of its smallest codes; a nonzero root is
        # raised to the smallest code at most
        slack = 8 * U * (m_mag if key == "m" else want)
        bound = 2.0 ** -4 * want.abs() * (1 + 1e-5) + 2.0 ** -10 * each + slack
        if key == "v":
            bound = torch.maximum(bound, 2.0 ** -9 * each + slack)
            assert ((code > 0) | (want == 0) | (each == 0)).all()
        assert ((code * each - want).abs() <= bound).all(), key


def after_of(t):
    return {key: t.get(key + "_out", t.get(key)) for key in
            ("p", "m", "v", "m_scale", "v_scale")} | {"p_bf16": t.get("p_bf16")}


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])
@pytest.mark.parametrize("offset", [0, 1], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("grad", [F32, BF16], ids=["gf32", "gbf16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_step(bits, grad, offset, in_place):
    tensors = adam_inputs(SIZES, bits, grad, seed=bits + offset, offset=offset)
    before = [{key: v.clone() for key, v in t.items()} for t in tensors]
    full = adam_outputs(tensors, copy=True, in_place=in_place)
    opt = adam_desc(bits, grad)
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, full))
    for b, t in zip(before, full):
        check_adam(b, after_of(t), bits)
        if not in_place:
            assert all(torch.equal(t[key].view(torch.uint8) if t[key].dtype.itemsize == 1 else t[key],
                                   b[key].view(torch.uint8) if b[key].dtype.itemsize == 1 else b[key])
                       for key in b)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_over_more_tensors_than_a_launch_holds_some_empty(bits):
    sizes = [0, 17] + [n % 700 + 1 for n in range(0, 70 * 311, 311)] + [0]
    tensors = adam_inputs(sizes, bits, F32, seed=8)
    before = [{key: v.clone() for key, v in t.items()} for t in tensors]
    full = adam_outputs(tensors, copy=False, in_place=True)
    opt = adam_desc(bits, F32)
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, full))
    for b, t in zip(before, full):
        if t["p"].numel():
            check_adam(b, after_of(t), bits)


def test_adamw_steps_from_gradients_whose_squares_are_subnormal():
    """v from 2^-106 down to 2^-134: products and sums round to steps of 2^-149 there, which two
    roundings move by 2^-149 together, and the root halves what that is of v."""
    n, g = 5000, gen(19)
    a = {**ADAM, "eps": 1e-30, "step": 1, "grad_scale": 1.0}
    size = torch.exp2(-51 - 13.5 * torch.rand(n, generator=g, device="cuda"))
    t = dict(p=1e-3 * randn(g, n), g=size * torch.sign(randn(g, n)),
             m=torch.zeros(n, device="cuda"), v=torch.zeros(n, device="cuda"))
    b = {key: v.clone() for key, v in t.items()}
    opt = adam_desc(32, F32, **{key: a[key] for key in ("eps", "step", "grad_scale")})
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, [t]))
    p, m, v, _ = ref.adamw(b["p"].double(), b["g"].double(), b["m"].double(), b["v"].double(), a)
    assert (v < 2.0 ** -104).all() and (v > 2.0 ** -136).all()
    assert ((t["v"].double() - v).abs() <= 6 * U * v + 2.0 ** -149).all()
    step = a["lr"]  # from zero moments each step is lr in size
    assert ((t["p"].double() - p).abs() <=
            2 * U * p.abs() + step * (24 * U + 2.0 ** -150 / v) * (1 + 1e-2)).all()


def test_adamw_first_steps_from_zero_states_follow_64_bits():
    """Five steps in fp32 from zero moments, against five in 64 bits: each step adds at most the
    bounds of one (2 u of p and 24 u of the step), so five add five times those."""
    n, g = 3001, gen(11)
    p0 = randn(g, n)
    t = dict(p=p0.clone(), g=torch.empty(n, device="cuda"), m=torch.zeros(n, device="cuda"),
             v=torch.zeros(n, device="cuda"))
    table = occ.AdamwTensors(adam_desc(32, F32), [t])
    p, m, v = p0.double(), torch.zeros(n, device="cuda").double(), torch.zeros(n, device="cuda").double()
    moved = torch.zeros_like(p)
    for step in range(1, 6):
        t["g"].copy_(randn(g, n))
        occ.occ_adamw_step(adam_desc(32, F32, step=step), table)
        p, m, v, s = ref.adamw(p, t["g"].double(), m, v, dict(ADAM, step=step))
        # m_mag / |m| can be large where gradients cancel; |m_hat| / root <= its value with every
        # gradient's magnitude, which is at most sqrt(1 / (1 - beta2)) here
        moved += ADAM["lr"] * (1 / (1 - ADAM["beta2"])) ** 0.5
    off = (t["p"].double() - p).abs()
    assert (off <= 5 * 2 * U * p0.abs().double() + 24 * U * moved + 5 * 2 * U * moved).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_zero_gradients_and_states(bits):
    t = adam_inputs([600], bits, F32, seed=12)[0]
    for key in t:
        if key != "p":
            t[key].zero_()
    p0 = t["p"].clone()
    opt = adam_desc(bits, F32)
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, [t]))
    want = p0.double() * (1 - ADAM["lr"] * ADAM["weight_decay"])
    check(t["p"], want, want.abs(), 2, "p")
    for key in set(t) - {"p", "g"}:
        assert not t[key].float().any(), key


def test_adamw_8bit_small_second_moments_keep_a_code():
    """One large gradient in a block: the others' roots fall below the smallest code and are held
    at it, so that the next step divides by them and not by eps."""
    n = 256
    t = dict(p=torch.zeros(n, device="cuda"), g=torch.full((n,), 1e-7, device="cuda"),
             m=torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda"),
             v=torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda"),
             m_scale=torch.zeros(1, device="cuda"), v_scale=torch.zeros(1, device="cuda"))
    t["g"][5] = 1.0
    opt = adam_desc(8, F32, grad_scale=1.0)
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, [t]))
    code = t["v"].float()
    assert code[5] == 448 and (code[:5] == 2.0 ** -9).all() and (code[6:] == 2.0 ** -9).all()
    assert not t["m"].float()[6:].any()


def test_adamw_keeps_what_is_not_finite_where_it_is():
    for bits in (32, 8):
        tensors = adam_inputs([1000, 300], bits, F32, seed=13)
        clean = [{key: v.clone() for key, v in t.items()} for t in tensors]
        opt = adam_desc(bits, F32)
        occ.occ_adamw_step(opt, occ.AdamwTensors(opt, clean))
        tensors[0]["g"][300], tensors[0]["g"][301] = float("nan"), float("inf")
        occ.occ_adamw_step(opt, occ.AdamwTensors(opt, tensors))
        assert not torch.isfinite(tensors[0]["p"][300]) and not torch.isfinite(tensors[0]["p"][301])
        keep = torch.ones(1000, dtype=torch.bool, device="cuda")
        keep[300:302] = False
        assert torch.equal(tensors[0]["p"][keep], clean[0]["p"][keep])
        if bits == 8:  # the whole block's states go with it
            keep[256:512] = False
        for key in ("m", "v"):
            assert torch.equal(tensors[0][key].float()[keep], clean[0][key].float()[keep])
        assert torch.equal(tensors[1]["p"], clean[1]["p"])


def test_adamw_dynamic_values_replace_the_descriptors():
    tensors = adam_inputs([5000], 32, F32, seed=14)
    before = {key: v.clone() for key, v in tensors[0].items()}
    a = dict(ADAM, lr=3e-3, step=250, grad_scale=2.0)
    dyn = torch.tensor([a["lr"], a["step"], a["grad_scale"]], device="cuda")
    opt = adam_desc(32, F32)  # other lr, step and scale
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, tensors), dynamic=dyn)
    # lr is fp32 here
    check_adam(before, after_of(tensors[0]), 32, dict(a, lr=float(np.float32(a["lr"]))))


@pytest.mark.parametrize("grad", [F32, BF16], ids=["gf32", "gbf16"])
@pytest.mark.parametrize("offset", [0, 1], ids=["aligned", "unaligned"])
def test_adamw_many_elements_in_fp32(offset, grad):
    """Around 2^27 elements in a launch: the last of two tensors is checked, and both their ends."""
    for first in ((1 << 27) - 3000, 1 << 27):
        big, small = (adam_inputs([n], 32, grad, seed=3, offset=offset)[0] for n in (2048, 1999))
        wide = {}
        for key, v in big.items():
            buf = torch.zeros(first + offset, dtype=v.dtype, device="cuda")[offset:]
            buf[:1000], buf[-1048:] = v[:1000], v[1000:]
            wide[key] = buf
        before = [{key: v.clone() for key, v in t.items()} for t in (big, small)]
        opt = adam_desc(32, grad)
        occ.occ_adamw_step(opt, occ.AdamwTensors(opt, [wide, small]))
        ends = {key: torch.cat([wide[key][:1000], wide[key][-1048:]]) for key in ("p", "m", "v")}
        check_adam(before[0], ends, 32)
        check_adam(before[1], small, 32)
        assert not wide["p"][1000:-1048].any() and not wide["v"][1000:-1048].any()


def test_adamw_largest_sizes_reach_the_last_element():
    """Offsets beyond 2^31 bytes: a tensor of 2^30 + 3 elements with 8-bit states."""
    n = (1 << 30) + 3
    t = dict(p=torch.zeros(n, device="cuda"), g=torch.zeros(n, dtype=BF16, device="cuda"),
             m=torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda"),
             v=torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda"),
             m_scale=torch.zeros(-(-n // 256), device="cuda"),
             v_scale=torch.zeros(-(-n // 256), device="cuda"))
    at = [0, 1 << 29, (1 << 30) - 1, n - 1]
    t["g"][at] = 1.0
    opt = adam_desc(8, BF16, grad_scale=1.0, step=1)
    occ.occ_adamw_step(opt, occ.AdamwTensors(opt, [t]))
    assert int((t["p"] != 0).sum()) == 4 and (t["p"][at] + ADAM["lr"]).abs().max() < 1e-5
    assert (t["m"][at].float() == 448).all()


# Arrays of more than 2^31 elements, zero but for their last rows: the sums over the tokens are
# those rows', and what lies in front of them stays zero.
LAST = 1000


def behind_zeros(T, v):
    out = torch.zeros(T, *v.shape[1:], dtype=v.dtype, device="cuda")
    out[-v.shape[0]:] = v
    return out


def only_last(full):
    """The last rows of an array whose other rows are zero (looked at in pieces)."""
    for part in full[:-LAST].split(1 << 17):
        assert not part.any()
    return full[-LAST:]


@pytest.mark.parametrize("dtype,T,d", [(BF16, 1100003, 2048), (BF16, 300001, 8192),
                                       (F32, 530003, 4096)])
def test_norm_rows_behind_two_to_the_31_elements(dtype, T, d):
    t, grads, opt = norm_inputs(dtype, LAST, d, "channel", seed=d)
    full = {key: behind_zeros(T, v) if v.dim() == 2 else v for key, v in t.items()}
    r, h = run_norm(full, opt, dtype)
    check_norm(t, opt, only_last(r), only_last(h))
    big = {key: behind_zeros(T, v) for key, v in grads.items()}
    out = run_norm_back(full, big, r, opt, dtype)
    small = {key: only_last(v) if v.dim() == 2 else v for key, v in out.items()}
    check_norm_back(t, grads, r[-LAST:], opt, small)


@pytest.mark.parametrize("dtype,T,d,Ne", [(BF16, 1100003, 2048, 60), (BF16, 1100003, 2048, 100),
                                          (F32, 530003, 4096, 70)])
def test_gate_backward_rows_behind_two_to_the_31_elements(dtype, T, d, Ne):
    dl, x, w, dx_in = gate_inputs(dtype, LAST, d, Ne, seed=Ne)
    desc = layer(T, d, Ne=Ne, dtype=dtype)
    dx, dw = nan_like((T, d), dtype), nan_like((Ne, d))
    occ.occ_gate_backward(desc, behind_zeros(T, dl), behind_zeros(T, x), w,
                          behind_zeros(T, dx_in), dx, dw, occ.alloc_block_workspace(desc))
    check_gate(dl, x, w, dx_in, only_last(dx), dw, LAST, Ne, dtype)


def test_balance_rows_behind_two_to_the_31_elements():
    T, Ne, k, Nd = (1 << 24) + 7, 129, 4, 3
    logits, ids, _, place, group = balance_inputs(LAST, Ne, k, Nd, "none", seed=3)
    valid = behind_zeros(T, torch.ones(LAST, dtype=torch.bool, device="cuda"))
    got = run_balance(T, Ne, k, Nd, behind_zeros(T, logits), behind_zeros(T, ids), valid,
                      place, None)
    check_balance(logits, ids, None, group, k, None, (*got[:3], only_last(got[3])))


# ------------------------------------------------- streams, graphs, together

def test_operators_on_a_side_stream():
    """Queued on a side stream behind a long fill of their inputs on that stream: they see it."""
    T, d, Ne = 400, 1024, 64
    s = torch.cuda.Stream()
    t, grads, opt = norm_inputs(BF16, T, d, "sandwich", seed=20)
    want_r, want_h = run_norm(t, opt, BF16)
    dl, x, w, dx_in = gate_inputs(BF16, T, d, Ne, seed=21)
    desc = layer(T, d, Ne=Ne, dtype=BF16)
    ws = occ.alloc_block_workspace(desc)
    want_dx, want_dw = nan_like((T, d), BF16), nan_like((Ne, d))
    occ.occ_gate_backward(desc, dl, x, w, dx_in, want_dx, want_dw, ws)
    late_x, late_dl = torch.zeros_like(t["x"]), torch.zeros_like(dl)
    big = torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    r, h = nan_like((T, d), BF16), nan_like((T, d), BF16)
    dx, dw = nan_like((T, d), BF16), nan_like((Ne, d))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            big.add_(1.0)
        late_x.copy_(t["x"])
        late_dl.copy_(dl)
    occ.occ_block_norm(layer(T, d, dtype=BF16), opt, late_x, t["y"], t["w_post"], None, t["w_pre"],
                       r, h, stream=s)
    occ.occ_gate_backward(desc, late_dl, x, w, dx_in, dx, dw, ws, stream=s)
    s.synchronize()
    assert torch.equal(r, want_r) and torch.equal(h, want_h)
    assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)


class Step:
    """One training step of a block: norm in front, gate, layer, the residual with its norm and
    gate, the router's losses, everything backward, and AdamW over the block's weights."""

    def __init__(self, seed=31, T=220, bits=32):
        wl = W.Workload("block_step", 40, T=T, d=256, Ne=8, k=2, Nd=4, F=256, n_shared=1,
                        F_shared=256, n_c=2, bonus=1.0)
        self.wl, inp = wl, synth.make_all(wl)
        self.place = inp["placement"]
        self.desc = occ.desc_of(wl, flags=occ.OCC_FLAG_TRAIN | occ.OCC_FLAG_DETERMINISTIC)
        g = gen(seed)
        T, d, Ne, F = wl.T, wl.d, wl.Ne, wl.F
        self.norm_in = occ.NormDesc(eps=1e-6, scale=1.0, gate=occ.OCC_GATE_NONE)
        self.norm_out = occ.NormDesc(eps=1e-6, scale=0.8, gate=occ.OCC_GATE_CHANNEL)
        self.loss_desc = occ.BalanceDesc(balance=2.0, group=1.0, z=0.1)
        w = {n: inp[n] for n in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")}
        w = {n: v.cuda() for n, v in w.items()}
        w["w_router"] = (randn(g, Ne, d) * 0.1).to(BF16)
        w["w_pre"] = (1 + 0.1 * randn(g, d)).to(BF16)
        w["w_post"] = (1 + 0.1 * randn(g, d)).to(BF16)
        w["gate"] = (0.7 + 0.1 * randn(g, d)).to(BF16)
        self.w = w
        self.x0, self.goal = randn(g, T, d).to(BF16), randn(g, T, d).to(BF16)
        self.valid = torch.rand(T, generator=g, device="cuda") < 0.9
        e = lambda *s, dtype=F32: nan_like(s, dtype)
        self.h, self.y, self.r = (e(T, d, dtype=BF16) for _ in range(3))
        self.logits, self.dlogits = e(T, Ne), e(T, Ne)
        self.counts = torch.zeros(Ne + 1, dtype=torch.int32, device="cuda")
        self.probs, self.loss = e(Ne), e(4)
        self.ws, self.ws2 = occ.alloc_workspace(self.desc), occ.alloc_block_workspace(self.desc)
        self.dr, self.dy, self.dh, self.dx = (e(T, d, dtype=BF16) for _ in range(4))
        self.grad = {n: e(*v.shape) for n, v in w.items()}
        self.adam = adam_desc(bits, F32, step=1, grad_scale=1.0)
        self.master, rows = {n: v.float() for n, v in w.items()}, []
        for n, v in w.items():
            units = -(-v.numel() // 256)
            kind = torch.float8_e4m3fn if bits == 8 else F32
            row = dict(p=self.master[n], g=self.grad[n], p_bf16=v,
                       m=torch.zeros(v.shape, device="cuda").to(kind),
                       v=torch.zeros(v.shape, device="cuda").to(kind))
            if bits == 8:
                row.update(m_scale=torch.zeros(units, device="cuda"),
                           v_scale=torch.zeros(units, device="cuda"))
            rows.append(row)
        self.table = occ.AdamwTensors(self.adam, rows)

    def forward_backward(self):
        w, g, D, wl = self.w, self.grad, self.desc, self.wl
        occ.occ_block_norm(D, self.norm_in, self.x0, None, None, None, w["w_pre"], None, self.h)
        occ.occ_gate(D, self.h, w["w_router"], self.logits)
        experts = [w[n] for n in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")]
        occ.occ_moe_forward(D, self.h, self.logits, self.place, *experts, self.y, self.ws)
        occ.occ_block_norm(D, self.norm_out, self.x0, self.y, w["w_post"], w["gate"], None,
                           self.r, None)
        view = occ.occ_forward_views(D, self.ws)
        self.ids = occ.ws_view(self.ws, view.ids, (wl.T, wl.k), torch.int32)
        occ.occ_balance_loss(D, self.loss_desc, self.logits, self.ids, self.valid, self.place,
                             self.counts, self.probs, self.loss, self.ws2)
        occ.occ_block_norm_backward(D, self.norm_out, self.goal, None, None, self.y, w["w_post"],
                                    w["gate"], None, self.dr, self.dy, g["w_post"], g["gate"],
                                    None, self.ws2)
        occ.occ_moe_backward(D, self.dy, self.h, self.logits, self.place, *experts, self.dh,
                             *[g[n] for n in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up",
                                              "ws_down")], None, self.dlogits, self.ws)
        occ.occ_balance_backward(D, self.loss_desc, self.logits, self.valid, self.place,
                                 self.counts, 1.0, self.dlogits, self.dlogits)
        occ.occ_gate_backward(D, self.dlogits, self.h, w["w_router"], self.dh, self.dh,
                              g["w_router"], self.ws2)
        occ.occ_block_norm_backward(D, self.norm_in, self.dr, self.dh, self.x0, None, None, None,
                                    w["w_pre"], self.dx, None, None, None, g["w_pre"], self.ws2)

    def optimise(self, dynamic=None):
        occ.occ_adamw_step(self.adam, self.table, dynamic=dynamic)

    def outputs(self):
        return {"dx": self.dx, "loss": self.loss, "counts": self.counts, "dlogits": self.dlogits,
                "r": self.r, **{"d" + n: v for n, v in self.grad.items()}}


def test_training_step_gradients_against_64_bits():
    """The step's gradients against differentiating the whole block in 64 bits, the routing held
    fixed.  Tolerances are the layer's own (2e-2 of the norm: its bf16 intermediates), which the
    rounding of h, y and dy between the operators (2^-8 each at most) stays under."""
    st = Step()
    st.forward_backward()
    torch.cuda.synchronize()
    wl, k = st.wl, st.wl.k
    v = {n: a.double().requires_grad_(True) for n, a in st.w.items()}
    x0 = st.x0.double().requires_grad_(True)
    unit = lambda a: a / torch.sqrt((a * a).mean(1, keepdim=True) + 1e-6)
    h = v["w_pre"] * unit(x0)
    logits = h @ v["w_router"].t()
    p = torch.softmax(logits, 1)
    ids = st.ids.long()
    y = torch.zeros_like(h)
    for e in range(wl.Ne):
        weight = (p[:, e] * (ids == e).any(1))[:, None]
        act = torch.nn.functional.silu(h @ v["w_gate"][e].t()) * (h @ v["w_up"][e].t())
        y = y + (weight * act) @ v["w_down"][e].t()
    act = torch.nn.functional.silu(h @ v["ws_gate"][0].t()) * (h @ v["ws_up"][0].t())
    y = y + act @ v["ws_down"][0].t()
    r = x0 + 0.8 * v["gate"] * v["w_post"] * unit(y)
    rows, n = st.valid, int(st.valid.sum())
    f = torch.bincount(ids[rows].flatten(), minlength=wl.Ne).double() * wl.Ne / (k * n)
    probs = p[rows].mean(0)
    group = torch.empty(wl.Ne, dtype=torch.long, device="cuda")
    for q in range(wl.Nd):
        group[torch.as_tensor(st.place[q], dtype=torch.long)] = q
    pool = torch.zeros(wl.Nd, dtype=torch.float64, device="cuda")
    loss = (2.0 * (f * probs).sum() +
            (pool.index_add(0, group, f) / (wl.Ne // wl.Nd) * pool.index_add(0, group, probs)).sum() +
            0.1 * torch.logsumexp(logits[rows], 1).square().mean())
    names = list(v)
    grads = torch.autograd.grad(loss + (r * st.goal.double()).sum(), [x0] + [v[n] for n in names])
    rel = lambda a, b: float((a.double() - b.detach()).norm() / b.detach().norm())
    assert abs(float(st.loss[0]) - float(loss.detach())) <= 2e-2 * abs(float(loss.detach()))
    assert rel(st.r, r) <= 2e-2
    for got, want, name in zip([st.dx] + [st.grad[n] for n in names], grads, ["x"] + names):
        assert rel(got, want) <= 2e-2, (name, rel(got, want))


@pytest.mark.parametrize("bits", [32, 8])
def test_training_step_updates_its_weights(bits):
    st = Step(bits=bits)
    st.forward_backward()
    before = [{key: a.clone() for key, a in row.items()} for row in st.table.tensors]
    st.optimise()
    for b, row in zip(before, st.table.tensors):
        flat = {key: a.flatten() for key, a in b.items()}
        after = {key: None if a is None else a.flatten() for key, a in after_of(row).items()}
        check_adam(flat, after, bits, dict(ADAM, step=1, grad_scale=1.0))
    st.forward_backward()  # the copies that the step wrote are the layer's weights now
    torch.cuda.synchronize()
    assert all(torch.isfinite(a.float()).all() for a in st.outputs().values())


def test_training_step_captured_and_replayed():
    """The whole step with its optimizer in one graph, replayed with eager work and other values
    in between: every replay equals the eager step bitwise (the layer's deterministic merge)."""
    eager, cap = Step(seed=33), Step(seed=33)
    dyn_e, dyn_c = (torch.tensor([1e-2, 1.0, 1.0], device="cuda") for _ in range(2))

    def whole(st, dyn):
        st.forward_backward()
        st.optimise(dynamic=dyn)

    whole(eager, dyn_e)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        whole(cap, dyn_c)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        whole(cap, dyn_c)
    for i in range(4):
        x = randn(gen(50 + i), *cap.x0.shape).to(BF16)
        for st, dyn in ((eager, dyn_e), (cap, dyn_c)):
            st.x0.copy_(x)
            dyn.copy_(torch.tensor([1e-2 / (i + 1), 2.0 + i, 1.0]))
        cap.ws2.fill_(0xff)  # scratch keeps nothing from call to call
        graph.replay()
        torch.cuda.synchronize()
        whole(eager, dyn_e)
        torch.cuda.synchronize()
        a, b = eager.outputs(), cap.outputs()
        for name in a:
            assert torch.equal(a[name], b[name]), (i, name)
        for n in eager.master:
            assert torch.equal(eager.master[n], cap.master[n]) and torch.equal(eager.w[n], cap.w[n])


def test_two_captured_graphs_share_a_workspace():
    """Two graphs over one scratch array, replayed in turn on one stream."""
    T, d, Ne = 300, 512, 60
    desc = layer(T, d, Ne=Ne, k=4, Nd=4, dtype=BF16)
    ws = occ.alloc_block_workspace(desc)
    t, grads, opt = norm_inputs(BF16, T, d, "channel", seed=60)
    r, _ = run_norm(t, opt, BF16)
    want = run_norm_back(t, grads, r, opt, BF16)
    dl, x, w, dx_in = gate_inputs(BF16, T, d, Ne, seed=61)
    dx, dw = nan_like((T, d), BF16), nan_like((Ne, d))
    occ.occ_gate_backward(desc, dl, x, w, dx_in, dx, dw, ws)
    want_dw = dw.clone()
    out = {key: nan_like(a.shape, a.dtype) for key, a in want.items()}

    def norm_back():
        occ.occ_block_norm_backward(desc, opt, grads["dr"], grads["dh"], r, t["y"], t["w_post"],
                                    t["gate"], t["w_pre"], out["dx"], out["dy"], out["dw_post"],
                                    out["dgate"], out["dw_pre"], ws)

    def gate_back():
        occ.occ_gate_backward(desc, dl, x, w, dx_in, dx, dw, ws)

    graphs = []
    for f in (norm_back, gate_back):
        f()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for _ in range(3):
        for a in (*out.values(), dw):
            a.fill_(float("nan"))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[key], want[key]) for key in want) and torch.equal(dw, want_dw)
        gate_back()
        torch.cuda.synchronize()


def test_binding_refuses_shapes_types_and_strides():
    T, d = 8, 64
    desc, opt = layer(T, d, dtype=BF16), occ.NormDesc(eps=1e-6, scale=1.0, gate=0)
    x, w = torch.zeros(T, d, dtype=BF16, device="cuda"), torch.ones(d, dtype=BF16, device="cuda")
    ok = lambda **o: occ.occ_block_norm(desc, opt, *{**dict(
        x=x, y=None, w_post=None, gate=None, w_pre=w, r=None, h=torch.empty_like(x)), **o}.values())
    ok()
    for bad in (dict(x=x.float()), dict(x=x[:4]), dict(w_pre=w.float()), dict(w_pre=w[:32]),
                dict(x=torch.zeros(d, T, dtype=BF16, device="cuda").t()), dict(h=x.cpu())):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(occ.OccError):
        ok(x=torch.zeros(T * d + 8, dtype=BF16, device="cuda")[1:T * d + 1].view(T, d))
    with pytest.raises(ValueError):
        occ.AdamwTensors(adam_desc(8, F32), [dict(p=x.float(), g=x.float(), m=x.float(),
                                                  v=x.float(), m_scale=w, v_scale=w)])
    short = adam_inputs([600], 8, F32, seed=1)[0]
    short["m_scale"] = short["m_scale"][:2]
    with pytest.raises(ValueError, match="m_scale"):
        occ.AdamwTensors(adam_desc(8, F32), [short])
