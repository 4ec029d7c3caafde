"""Routing by scores on the GPU against plain 64-bit implementations (score_reference.py): the
choice at ties, masks, groups and every expert count's edges, the weights, the gradient, the bias's
step, in place, on side streams, captured, and with the layer's forward and backward.

Tolerances are bounds by arithmetic.  ids and counts are equal.  Weights are formed in 64 bits and
rounded once: half a step of fp32.  The gradient is formed in fp32: n u of the magnitudes that it is
made of, n = 2 (largest distance of an exponent from its base) + 2 k + 24 for the exponentials'
arguments and values, the sums over k and the products."""
import numpy as np
import pytest
import torch

import score_reference as ref
from block_reference import U, half_step
from expert_token_routing_amd import occ

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    occ.lib()


def layer(T, Ne, k, Nd=1):
    return occ.LayerDesc(T=T, d=64, Ne=Ne, k=k, Nd=Nd, F=64, n_shared=0, F_shared=0, prune_rule=0,
                         prune_groups=0, dtype=occ.OCC_F32, flags=0)


def options(kind, top_groups=1, best=1, renorm=1, scale=1.0):
    return occ.ScoreDesc(score=kind, top_groups=top_groups, group_best=best, renormalise=renorm,
                         scale=scale)


def placement(Ne, Nd, seed=None):
    order = np.arange(Ne, dtype=np.int32)
    if seed is not None:
        order = np.random.default_rng(seed).permutation(Ne).astype(np.int32)
    return order.reshape(Nd, Ne // Nd)


def run_route(logits, bias, place, k, opt, Nd):
    T, Ne = logits.shape
    ids = torch.full((T, k), -7, dtype=I32, device="cuda")
    w = torch.full((T, k), NAN, device="cuda")
    occ.occ_route_scored(layer(T, Ne, k, Nd), opt, logits.cuda(),
                         None if bias is None else bias.cuda(), place, ids, w)
    return ids.cpu(), w.cpu()


def check_route(logits, bias, place, k, opt):
    got_ids, got_w = run_route(logits, bias, place, k, opt, place.shape[0])
    ids, w = ref.route(logits, bias, place, k, opt.score, opt.top_groups, opt.group_best,
                       opt.renormalise, opt.scale)
    assert torch.equal(got_ids, ids), (got_ids[(got_ids != ids).any(1)][:3],
                                       ids[(got_ids != ids).any(1)][:3])
    bound = half_step(F32) * w.abs() * (1 + 1e-6) + 2.0 ** -149
    off = (got_w.double() - w).abs()
    assert (off <= bound).all(), float((off / bound).max())
    return got_ids, got_w


# every lane layout's edges (16, 32, 64, 128, 256 experts), one expert, all of them chosen
SHAPES = [(1, 1, 1, 1), (5, 3, 3, 1), (33, 16, 4, 4), (17, 17, 5, 1), (70, 32, 8, 8), (9, 60, 4, 4),
          (130, 64, 8, 8), (64, 64, 32, 2), (31, 66, 7, 3), (20, 128, 8, 64), (7, 130, 12, 2),
          (25, 256, 8, 8), (6, 256, 32, 64), (11, 255, 1, 5)]


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("T,Ne,k,Nd", SHAPES)
def test_route(T, Ne, k, Nd, biased, kind):
    g = torch.Generator().manual_seed(Ne * 7 + k)
    logits = torch.randn(T, Ne, generator=g) * 2
    bias = torch.randn(Ne, generator=g) * 0.1 if biased else None
    n = Ne // Nd
    for top in sorted({-(-k // n), max(-(-k // n), Nd // 2), Nd}):
        for best in (1, 2):
            if best > n:
                continue
            check_route(logits, bias, placement(Ne, Nd, seed=Nd), k,
                        options(kind, top, best, renorm=best - 1, scale=2.5))


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("Ne,Nd", [(48, 4), (192, 8)])
def test_route_ties_go_to_the_lower_index_and_group(kind, Ne, Nd):
    """Logits of few values: experts and groups tie everywhere; equal bias or bias of few values."""
    g = torch.Generator().manual_seed(2)
    logits = torch.randint(-2, 3, (60, Ne), generator=g).float()
    logits[0] = 0.0
    logits[1, ::2] = -0.0  # -0 and +0 are one value
    logits[1, 1::2] = 0.0
    for bias in (None, torch.zeros(Ne), torch.randint(-1, 2, (Ne,), generator=g).float() * 0.5):
        for place in (placement(Ne, Nd), placement(Ne, Nd, seed=5)):
            for best in (1, 2):
                check_route(logits, bias, place, 6, options(kind, 2, best, scale=1.0))
                check_route(logits, bias, place, 6, options(kind, Nd, best, scale=1.0))


def test_route_near_ties_fall_as_in_64_bits():
    """Scores plus bias that 32 bits cannot tell apart: neighbours in fp32 whose order the bias
    turns by less than fp32's step at 1."""
    Ne, T = 64, 400
    g = torch.Generator().manual_seed(3)
    base = torch.randn(T, 1, generator=g) * 0.5 + 2
    logits = base + torch.arange(Ne)[None, torch.randperm(Ne, generator=g)] * 2.0 ** -22
    bias = 1 + torch.arange(Ne).float() * 2.0 ** -23
    for kind in (ref.SOFTMAX, ref.SIGMOID):
        check_route(logits, bias, placement(Ne, 8), 8, options(kind, 8))
        check_route(logits, bias, placement(Ne, 8), 8, options(kind, 3, 2))
        check_route(logits, -bias, placement(Ne, 8, seed=1), 8, options(kind, 3, 1))


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("Ne,Nd", [(40, 5), (160, 8)])
def test_route_masked_experts_and_empty_rows(kind, Ne, Nd):
    """-inf and NaN leave an expert out even where its bias would win; rows and groups without any
    expert; the type's lowest value is a number and does not."""
    g = torch.Generator().manual_seed(4)
    T = 50
    logits = torch.randn(T, Ne, generator=g)
    logits[torch.rand(T, Ne, generator=g) < 0.6] = -INF
    logits[torch.rand(T, Ne, generator=g) < 0.1] = NAN
    logits[0] = -INF
    logits[1] = NAN
    logits[2] = -INF
    logits[2, Ne - 1] = 0.5
    logits[3] = torch.finfo(F32).min
    logits[4] = torch.finfo(F32).min
    logits[4, 3] = 1.0
    logits[5, : Ne // Nd] = -INF
    bias = torch.randn(Ne, generator=g)
    for b in (None, bias):
        for place in (placement(Ne, Nd), placement(Ne, Nd, seed=8)):
            for top, best in ((Nd, 1), (2, 1), (2, 2)):
                for renorm in (0, 1):
                    check_route(logits, b, place, 7, options(kind, top, best, renorm, scale=0.5))


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("Ne,Nd,k,top", [(8, 2, 8, 2), (64, 8, 8, 1), (64, 8, 16, 2), (16, 1, 16, 1),
                                         (192, 8, 24, 1), (192, 8, 6, 3), (256, 8, 32, 1)])
def test_route_biases_that_are_not_finite(Ne, Nd, k, top, kind):
    """Infinite biases tie by index, also where the chosen are all that there are and nothing
    stands behind the last; -inf and NaN come last and score for no group."""
    g = torch.Generator().manual_seed(11)
    logits = torch.randn(20, Ne, generator=g)
    logits[3, ::2] = -INF
    place = placement(Ne, Nd, seed=12)
    bias = torch.full((Ne,), INF)
    check_route(logits, bias, place, k, options(kind, top))
    check_route(logits, -bias, place, k, options(kind, Nd))
    logits = torch.randn(20, Ne, generator=g)
    bias = torch.randn(Ne, generator=g) * 0.1
    for row in place:  # one of each in a group
        bias[int(row[0])], bias[int(row[1])], bias[int(row[2])] = INF, -INF, NAN
    # the reference sums a group's best two over every expert that is not left out: at least two
    # are finite or +inf, so that a -inf never enters
    seen = torch.where(bias == bias, bias, torch.full_like(bias, -INF))
    for best in (1, 2):
        got = run_route(logits, bias, place, k, options(kind, top, best), Nd)
        want = check_route(logits, seen, place, k, options(kind, top, best))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
def test_route_saturated_and_vanishing_scores(kind):
    """Without a bias the logits order experts whose scores are equal in 64 bits; scores down to
    e^-700 still share out their weights."""
    logits = torch.tensor([[50., 60., 55., 100., 40., 45.], [-700., -690., -695., -650., -640., -645.],
                           [-80., -100., -90., 0., 88., 89.], [1e30, 2e30, -1e30, 0., 3e30, 1.]])
    check_route(logits, None, placement(6, 2), 4, options(kind, 2, scale=1.0))
    ids, w = check_route(logits[:3], None, placement(6, 2), 3, options(kind, 1, 1, scale=1.0))
    assert torch.allclose(w.sum(1), torch.ones(3), atol=1e-6)


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("Ne,Nd,top", [(16, 4, 2), (48, 4, 4), (64, 8, 3), (120, 5, 5), (192, 8, 4)])
def test_route_of_a_token_does_not_depend_on_its_batch(Ne, Nd, top, biased, kind):
    """The same rows (of a normal, near ties, ties, masked, empty) in batches from one token to
    those in which a wave takes several: the reference's choice and the same bits in each."""
    g = torch.Generator().manual_seed(Ne)
    n, k = 60, 4
    rows = torch.randn(n, Ne, generator=g) * 2
    rows[20:35] = 2 + torch.arange(Ne)[torch.randperm(Ne, generator=g)] * 2.0 ** -22
    rows[35:45] = torch.randint(-1, 2, (10, Ne), generator=g).float()
    rows[45:55][torch.rand(10, Ne, generator=g) < 0.5] = -INF
    rows[55] = NAN
    bias = 1 + torch.arange(Ne).float() * 2.0 ** -23 if biased else None
    place, opt = placement(Ne, Nd, seed=1), options(kind, top, min(2, top), scale=1.5)
    ids, w = check_route(rows, bias, place, k, opt)
    for T in (1, 7, 2048, 2049, 8191, 8192, 8195):
        at = torch.arange(T) % n
        got_ids, got_w = run_route(rows[at], bias, place, k, opt, Nd)
        assert torch.equal(got_ids, ids[at]) and torch.equal(got_w, w[at]), T


def test_route_without_groups_needs_no_placement_and_repeats_bitwise():
    g = torch.Generator(device="cuda").manual_seed(5)
    T, Ne, k = 5000, 128, 8
    logits, bias = torch.randn(T, Ne, generator=g, device="cuda"), torch.zeros(Ne, device="cuda")
    desc, outs = layer(T, Ne, k, 4), []
    for place in (None, placement(Ne, 4), placement(Ne, 4, seed=1), None):
        ids, w = torch.empty(T, k, dtype=I32, device="cuda"), torch.empty(T, k, device="cuda")
        occ.occ_route_scored(desc, options(ref.SIGMOID, 4), logits, bias, place, ids, w)
        outs.append((ids, w))
    assert all(torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1]) for a, b in outs)
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(outs[0][0], order.int())


def test_route_softmax_is_the_layers_own_route_when_plain():
    """Softmax scores, no bias, no groups, not renormalised: occ_route's ids, and its weights
    within its own bound of 1e-6."""
    g = torch.Generator(device="cuda").manual_seed(6)
    T, Ne, k = 3000, 64, 8
    logits = torch.randn(T, Ne, generator=g, device="cuda") * 2
    desc, place = layer(T, Ne, k, 8), placement(Ne, 8)
    a, b = (torch.empty(T, k, dtype=I32, device="cuda") for _ in range(2))
    wa, wb = torch.empty(T, k, device="cuda"), torch.empty(T, k, device="cuda")
    occ.occ_route(desc, logits, place, a, wa)
    occ.occ_route_scored(desc, options(ref.SOFTMAX, 8, renorm=0), logits, None, place, b, wb)
    assert torch.equal(a, b) and ((wa - wb).abs() <= 1e-6 * wb + 2.0 ** -149).all()


# ----------------------------------------------- borders that 32 bits cannot tell

# experts, groups, kept groups, tokens: 16 lanes with 1, 2 and 4 experts each, a wave with 1, 2 and 4
BORDERS = [(3, 1, 1, 40), (4, 2, 2, 40), (16, 4, 2, 40), (32, 4, 4, 40), (32, 8, 3, 40),
           (64, 8, 8, 2100), (64, 8, 3, 2100), (64, 8, 8, 40), (64, 8, 3, 40), (128, 8, 8, 40),
           (128, 8, 3, 40), (256, 16, 16, 40), (256, 16, 4, 40), (256, 16, 4, 8200)]


def border_rows(Ne, seed):
    """Exact ties beside neighbours that 32 bits place level with them: saturated sigmoids, terms of
    a peaked softmax, neighbours of a few steps of fp32, logits rounded to bf16.  None above 28, where
    a sigmoid's own 64 bits still tell a step of bf16 apart (e^-28 / 8 is a hundred of their steps)."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for head in ([20., 20., 21.], [18., 18., 18.125], [0., -110., -110., -105.], [25., 24.75, 24.75, 25.]):
        for low in (-30., -120.):
            row = torch.full((Ne,), low)
            row[:min(len(head), Ne)] = torch.tensor(head[:Ne])
            rows += [row, row[torch.randperm(Ne, generator=g)], row.flip(0)]
    for _ in range(8):
        near = 2 + torch.randint(0, 8, (Ne,), generator=g) * 2.0 ** -22
        rows += [near, near - 3, torch.randint(128, 161, (Ne,), generator=g) / 8.0]
    for size in (1.0, 4.0, 8.0, 8.0):
        rows += list((torch.randn(8, Ne, generator=g) * size).to(BF16).float().clamp(max=28))
    return torch.stack(rows)


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("Ne,Nd,top,T", BORDERS)
def test_route_ties_at_the_border_hide_no_better_expert(Ne, Nd, top, T, kind):
    rows = border_rows(Ne, Ne + top)
    at = torch.arange(max(T, rows.shape[0])) % rows.shape[0]
    place = placement(Ne, Nd, seed=2)
    for bias in (torch.zeros(Ne), torch.full((Ne,), 0.5), (torch.arange(Ne) % 3) * 2.0 ** -23):
        for k in (1, 2, 3, 8):
            if k > top * (Ne // Nd):
                continue
            opt = options(kind, top, 1)
            ids, w = ref.route(rows, bias, place, k, kind, top, 1, 1, 1.0)
            got_ids, got_w = run_route(rows[at], bias, place, k, opt, Nd)
            wrong = (got_ids != ids[at]).any(1)
            assert not wrong.any(), (k, int(wrong.sum()), rows[at][wrong][0], got_ids[wrong][0],
                                     ids[at][wrong][0])
            assert ((got_w - w[at]).abs() <= half_step(F32) * w[at].abs() * (1 + 1e-6) + 2.0 ** -149).all()


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("Ne,Nd,top,T", [(16, 4, 2, 300), (16, 8, 3, 300), (32, 4, 1, 300),
                                         (64, 8, 4, 300), (64, 8, 4, 2100), (64, 32, 9, 300),
                                         (64, 32, 9, 2100), (128, 8, 4, 300), (128, 64, 20, 300),
                                         (256, 8, 3, 300), (256, 64, 20, 300)])
def test_route_groups_whose_best_two_cancel(Ne, Nd, top, T, kind):
    """One expert of a group with a bias of B or more, the others with as much less: the sum of the
    best two is near 0, its error is of B's size.  The groups lie some steps of B's fp32 apart."""
    g = torch.Generator().manual_seed(Nd + top)
    n, rows = Ne // Nd, 300
    place = placement(Ne, Nd, seed=6)
    for B in (1.0, 16.0, 64.0, 256.0, 1024.0, 65536.0):
        # one row of logits in every group, each shifted by some 2^-23 B to 2^-17 B either way: a
        # sum in fp32 may step up where its terms' rounded parts say down
        base = torch.randn(rows, 1, n, generator=g)
        size = B * 2.0 ** (torch.arange(rows) % 7 - 23)
        shift = (torch.rand(rows, Nd, n, generator=g).double() * 2 - 1) * size[:, None, None]
        logits, bias = torch.empty(rows, Ne), torch.empty(Ne)
        logits[:, place.flatten()] = (base.double() + shift).float().reshape(rows, Ne)
        # (of another size in each group: the chosen lie far apart, only the groups near)
        of_group = B * (1 + torch.arange(Nd) / Nd)[:, None] * torch.tensor([1.0] + [-1.0] * (n - 1))
        bias[place.flatten()] = of_group.flatten()
        k = top
        ids, w = ref.route(logits, bias, place, k, kind, top, 2, 1, 1.0)
        at = torch.arange(T) % rows
        got_ids, _ = run_route(logits[at], bias, place, k, options(kind, top, 2), Nd)
        # Groups whose logits came out equal tie but for the roundings of s + bias, which 64 bits do
        # not settle: scores within 2^-50 here and 2^-51 there, a sum rounded by 2^-53 (1 + 2 B), and
        # four such sums at a border: below 2^-46 (1 + 2 B) together
        c = (ref.scores(logits, kind) + bias.double())[:, place.flatten()].view(rows, Nd, n)
        ranked = c.topk(2, dim=2).values.sum(2).sort(1, descending=True).values
        told = ranked[:, top - 1] - ranked[:, top] > 2.0 ** -46 * (1 + 2 * B)
        assert told.sum() >= 240
        wrong = (got_ids != ids[at]).any(1) & told[at]
        assert not wrong.any(), (B, int(wrong.sum()))


# experts, groups, kept groups, k: the kept groups hold the chosen and no other, or one more, or lie
# on the lanes of a few (places a wave apart), in every lane layout
KEPT = [(8, 2, 1, 4), (16, 4, 4, 16), (32, 4, 2, 16), (64, 8, 1, 8), (64, 8, 1, 7), (64, 1, 1, 32),
        (128, 16, 2, 16), (128, 16, 2, 9), (128, 8, 1, 16), (256, 8, 1, 32), (256, 64, 4, 16),
        (256, 32, 4, 31), (192, 24, 4, 32)]


@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("Ne,Nd,top,k", KEPT)
def test_route_of_kept_groups_that_hold_little_more_than_the_chosen(Ne, Nd, top, k, kind):
    g = torch.Generator().manual_seed(Ne + k)
    rows = torch.randn(60, Ne, generator=g) * 2
    rows[20:40] = 2 + torch.randint(0, 6, (20, Ne), generator=g) * 2.0 ** -22
    rows[40:][torch.rand(20, Ne, generator=g) < 0.5] = -INF
    place = placement(Ne, Nd, seed=7)
    n = Ne // Nd
    # (the best of every group in places 64 apart, so that they are kept together)
    for shift in (0, 4.0):
        rows[:, place.flatten()[torch.arange(Ne) % 64 < n]] += shift
        for bias in (torch.randn(Ne, generator=g) * 0.1, 1 + torch.arange(Ne) * 2.0 ** -23, torch.zeros(Ne)):
            opt = options(kind, top, min(2, n), scale=1.5)
            ids, w = check_route(rows, bias, place, k, opt)
            at = torch.arange(2100) % 60
            got_ids, got_w = run_route(rows[at], bias, place, k, opt, Nd)
            assert torch.equal(got_ids, ids[at]) and torch.equal(got_w, w[at])


# ------------------------------------------------------------------- gradient

def run_back(logits, ids, dw, dlogits_in, opt, alias=None):
    T, Ne = logits.shape
    dev = [None if a is None else a.cuda() for a in (logits, ids, dw, dlogits_in)]
    out = {"in": dev[3], "logits": dev[0], None: torch.full((T, Ne), NAN, device="cuda")}[alias]
    occ.occ_route_scored_backward(layer(T, Ne, ids.shape[1]), opt, *dev, out)
    return out.cpu()


def spread(logits):
    v = logits.double()
    v = torch.where(ref.left_out(logits), torch.zeros_like(v), v)
    return float((v - v.amax(1, keepdim=True)).abs().max().clamp(max=200)) + float(
        v.clamp(max=0).abs().max().clamp(max=200))


def check_back(logits, ids, dw, dlogits_in, opt, got):
    grad, mag = ref.route_back(logits, ids, dw, opt.score, opt.renormalise, opt.scale)
    base = dlogits_in.double() if dlogits_in is not None else torch.zeros_like(grad)
    n = 2 * spread(logits) + 2 * ids.shape[1] + 24
    bound = n * U * mag + half_step(F32) * (grad + base).abs() * 1.01 + 2.0 ** -126
    off = (got.double() - grad - base).abs()
    assert (off <= bound).all(), (float((off / bound).max()), opt.score, opt.renormalise)


@pytest.mark.parametrize("renorm", [0, 1], ids=["scores", "renormalised"])
@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("T,Ne,k,Nd", SHAPES)
def test_route_backward(T, Ne, k, Nd, kind, renorm):
    g = torch.Generator().manual_seed(Ne + 31 * k)
    logits = torch.randn(T, Ne, generator=g) * 3
    ids = torch.stack([torch.randperm(Ne, generator=g)[:k] for _ in range(T)]).int()
    dw, dl = torch.randn(T, k, generator=g), torch.randn(T, Ne, generator=g)
    opt = options(kind, 1, 1, renorm, 1.75)
    for base in (None, dl):
        check_back(logits, ids, dw, base, opt, run_back(logits, ids, dw, base, opt))
    plain = run_back(logits, ids, dw, dl, opt)
    assert torch.equal(run_back(logits, ids, dw, dl, opt, alias="in"), plain)
    assert torch.equal(run_back(logits, ids, dw, dl, opt, alias="logits"), plain)


@pytest.mark.parametrize("renorm", [0, 1], ids=["scores", "renormalised"])
@pytest.mark.parametrize("kind", [ref.SOFTMAX, ref.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("Ne", [24, 200])
def test_route_backward_masked_experts_extremes_and_odd_ids(Ne, kind, renorm):
    """Left-out experts get 0 and their dw (here NaN) is not used; ids out of range count nothing
    and a repeated one twice; scores too small for fp32 still share out their gradient."""
    g = torch.Generator().manual_seed(9)
    T, k = 12, 6
    logits = torch.randn(T, Ne, generator=g)
    ids = torch.stack([torch.randperm(Ne, generator=g)[:k] for _ in range(T)]).int()
    dw = torch.randn(T, k, generator=g)
    logits[0] = -INF
    logits[1, ids[1, :3].long()] = -INF
    dw[1, :3] = NAN
    logits[2, ids[2, 1].long()] = NAN
    dw[2, 1] = NAN
    logits[3] -= 150  # sigmoid: e^-150 is 0 in fp32
    logits[4] += 60
    ids[5, 0], ids[5, 1] = -1, Ne
    dw[5, :2] = NAN
    logits[6] = torch.finfo(F32).min
    opt = options(kind, 1, 1, renorm, 1.0)
    check_back(logits, ids, dw, None, opt, run_back(logits, ids, dw, None, opt))
    ids[7, 2] = ids[7, 3]
    if renorm == 0:
        check_back(logits, ids, dw, None, opt, run_back(logits, ids, dw, None, opt))


# ----------------------------------------------------------------- bias's step

# one workgroup, the entries' border to several, many; every mask
@pytest.mark.parametrize("mask", ["none", "some", "empty", "one"])
@pytest.mark.parametrize("T,Ne,k", [(1, 1, 1), (3, 7, 2), (512, 64, 8), (8192, 60, 1),
                                    (8193, 60, 1), (2731, 256, 3), (70001, 250, 8)])
def test_bias_step(T, Ne, k, mask):
    g = torch.Generator().manual_seed(T + Ne)
    ids = torch.randint(0, Ne, (T, k), generator=g, dtype=I32)
    ids[torch.rand(T, k, generator=g) < 0.05] = -1
    ids[torch.rand(T, k, generator=g) < 0.05] = Ne
    valid = {"none": None, "some": torch.rand(T, generator=g) < 0.7,
             "empty": torch.zeros(T, dtype=torch.bool), "one": torch.arange(T) == T - 1}[mask]
    bias = torch.randn(Ne, generator=g)
    desc = layer(T, Ne, k)
    ws = occ.alloc_block_workspace(desc)
    ws.fill_(0xff)
    counts = torch.full((Ne + 1,), -7, dtype=I32, device="cuda")
    out = torch.full((Ne,), NAN, device="cuda")
    v = None if valid is None else valid.cuda()
    occ.occ_route_bias_step(desc, 1e-3, ids.cuda(), v, bias.cuda(), counts, out, ws)
    want_counts, want = ref.bias_step(ids, valid, bias, Ne, 1e-3)
    assert torch.equal(counts.cpu(), want_counts) and torch.equal(out.cpu(), want)
    place = bias.cuda()
    if v is not None:
        v = v.to(torch.uint8) * 3
    occ.occ_route_bias_step(desc, 1e-3, ids.cuda(), v, place, counts, place, ws)
    assert torch.equal(place.cpu(), want) and torch.equal(counts.cpu(), want_counts)


# -------------------------------------------------------------------- streams

def test_scored_on_a_side_stream_and_captured():
    """Forward, bias step and gradient on a side stream, then in one graph, replayed over new
    logits with eager work between: every replay equals the eager result bitwise."""
    T, Ne, k, Nd = 9000, 64, 8, 8
    g = torch.Generator(device="cuda").manual_seed(12)
    desc, opt, place = layer(T, Ne, k, Nd), options(ref.SIGMOID, 4, 2, 1, 2.5), placement(Ne, Nd)

    class Set:
        def __init__(self):
            self.logits = torch.zeros(T, Ne, device="cuda")
            self.bias, self.dw = torch.zeros(Ne, device="cuda"), torch.ones(T, k, device="cuda")
            self.new = torch.empty(Ne, device="cuda")
            self.ids = torch.empty(T, k, dtype=I32, device="cuda")
            self.w, self.dl = torch.empty(T, k, device="cuda"), torch.empty(T, Ne, device="cuda")
            self.counts = torch.empty(Ne + 1, dtype=I32, device="cuda")
            self.ws = occ.alloc_block_workspace(desc)

        def run(self, stream=None):
            occ.occ_route_scored(desc, opt, self.logits, self.bias, place, self.ids, self.w, stream)
            occ.occ_route_bias_step(desc, 1e-3, self.ids, None, self.bias, self.counts, self.new,
                                    self.ws, stream)
            occ.occ_route_scored_backward(desc, opt, self.logits, self.ids, self.dw, None, self.dl,
                                          stream)

        def outputs(self):
            return self.ids, self.w, self.counts, self.new, self.dl

    eager, cap = Set(), Set()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cap.run(stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap.run()
    for i in range(4):
        logits, dw = (torch.randn(*s, generator=g, device="cuda") for s in ((T, Ne), (T, k)))
        for st in (eager, cap):
            st.logits.copy_(logits)
            st.dw.copy_(dw)
            st.bias.fill_(0.01 * i)
        cap.ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        eager.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager.outputs(), cap.outputs())), i


def test_scored_rows_behind_two_to_the_31_elements():
    """The last rows of logits and dlogits that lie behind 2^31 elements."""
    T, Ne, k = 8_400_001, 256, 1
    g = torch.Generator(device="cuda").manual_seed(13)
    tail = 64
    logits = torch.zeros(T, Ne, device="cuda")
    logits[-tail:] = torch.randn(tail, Ne, generator=g, device="cuda")
    desc, opt = layer(T, Ne, k), options(ref.SIGMOID, 1, 1, 0, 1.0)
    ids, w = torch.empty(T, k, dtype=I32, device="cuda"), torch.empty(T, k, device="cuda")
    occ.occ_route_scored(desc, opt, logits, None, None, ids, w)
    want, ww = ref.route(logits[-tail:].cpu(), None, placement(Ne, 1), k, ref.SIGMOID, 1, 1, 0, 1.0)
    assert torch.equal(ids[-tail:].cpu(), want) and not ids[:-tail].any()
    assert ((w[-tail:].cpu() - ww).abs() <= half_step(F32) * ww * 1.01).all()
    dw = torch.ones(T, k, device="cuda")
    occ.occ_route_scored_backward(desc, opt, logits, ids, dw, None, logits)
    grad, _ = ref.route_back(torch.zeros(1, Ne), torch.zeros(1, 1, dtype=I32), torch.ones(1, 1),
                             ref.SIGMOID, 0, 1.0)
    assert torch.allclose(logits[5].cpu().double(), grad[0], atol=1e-6)
    assert torch.equal(logits[-tail - 1], logits[5]) and logits[-1].count_nonzero() == 1
