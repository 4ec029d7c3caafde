"""The layer with experts in 8 bits on the GPU against a plain 64-bit implementation
(score_reference.layer8): widths that end inside a line, few and many rows, uneven and empty experts,
shared experts, values that are zero, tiny or not finite, and the quantiser alone, bit for bit.

Tolerances are bounds by arithmetic, written in score_reference.py: half a step of bf16 for y and
for each term, the fp32 arithmetic in front of a code, and one code's weight where that arithmetic
cannot decide between two codes."""
import numpy as np
import pytest
import torch

import score_reference as ref
from expert_token_routing_amd import occ

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    occ.lib()


def layer(T, d, Ne, k, F, Nd=1, n_shared=0, F_shared=0, flags=0):
    return occ.LayerDesc(T=T, d=d, Ne=Ne, k=k, Nd=Nd, F=F, n_shared=n_shared, F_shared=F_shared,
                         prune_rule=0, prune_groups=0, dtype=occ.OCC_BF16, flags=flags)


def placement(Ne, Nd=1, seed=None):
    order = np.arange(Ne, dtype=np.int32)
    if seed is not None:
        order = np.random.default_rng(seed).permutation(Ne).astype(np.int32)
    return order.reshape(Nd, Ne // Nd)


# ------------------------------------------------------------------ quantiser

# a wave a row with 1, 2, 4 and 8 chunks a lane, a workgroup a row, ends inside each
QUANT = [(BF16, 1, 16), (BF16, 5, 64), (BF16, 3, 528), (BF16, 300, 1024), (BF16, 7, 2064),
         (BF16, 9, 4096), (BF16, 4, 4112), (BF16, 3, 20000), (F32, 1, 16), (F32, 6, 272),
         (F32, 65, 528), (F32, 11, 1040), (F32, 5, 2048), (F32, 5, 2064), (F32, 2, 9008)]


@pytest.mark.parametrize("dtype,rows,cols", QUANT, ids=lambda v: str(v).replace("torch.", ""))
def test_quantise_rows_bit_for_bit(dtype, rows, cols):
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(
        4 * torch.randn(rows, 1, generator=g))).to(dtype)
    q = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), -1.0, device="cuda")
    occ.occ_quantize_int8(x.cuda(), q, s)
    want_q, want_s = ref.quantise(x)
    assert torch.equal(q.cpu(), want_q) and torch.equal(s.cpu(), want_s)
    assert (want_q.abs().amax(1) == 127).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [64, 4800])
def test_quantise_rows_of_zeros_extremes_and_not_finite(dtype, cols):
    x = torch.randn(12, cols, generator=torch.Generator().manual_seed(1))
    x[0] = 0.0
    x[1] *= 2.0 ** -101 / x[1].abs().max()
    x[2] *= 2.0 ** -99 / x[2].abs().max()
    x[3] *= 1e38 / x[3].abs().max()
    x[4, cols - 1] = INF
    x[5, 0] = -INF
    x[6, cols // 2] = NAN
    x[7] = 1.0
    x[8] = -0.0
    x[9] = torch.finfo(dtype).max
    x[10] = torch.linspace(-127, 127, cols)  # halves between codes
    x[10, 0] = 127.0
    x = x.to(dtype)
    q, s = torch.empty(12, cols, dtype=torch.int8, device="cuda"), torch.empty(12, device="cuda")
    occ.occ_quantize_int8(x.cuda(), q, s)
    want_q, want_s = ref.quantise(x)
    assert torch.equal(q.cpu(), want_q)
    assert torch.equal(s.cpu().nan_to_num(-1.0), want_s.nan_to_num(-1.0))
    assert torch.isnan(s[4:7]).all() and not q[4:7].any() and s[0] == 0 and s[1] == 0 and s[2] > 0


def test_quantise_weights_of_many_rows():
    """Expert weights as they are laid out, over more rows than a launch has waves for."""
    w = torch.randn(3, 700_001, 16, generator=torch.Generator(device="cuda").manual_seed(2),
                    device="cuda")
    q, s = torch.empty_like(w, dtype=torch.int8), torch.empty(3, 700_001, device="cuda")
    occ.occ_quantize_int8(w, q, s)
    for part in (slice(0, 100), slice(-100, None)):
        want_q, want_s = ref.quantise(w[:, part].cpu())
        assert torch.equal(q[:, part].cpu(), want_q) and torch.equal(s[:, part].cpu(), want_s)
    assert ((q.float() * s[..., None] - w).abs() <= 0.5001 * s[..., None]).all()


# ---------------------------------------------------------------------- layer

def weights(g, N, F, d):
    def one(*shape):
        q = (torch.randn(*shape, generator=g) * 40).round().clamp(-127, 127).to(torch.int8)
        return q, (0.5 + torch.rand(*shape[:-1], generator=g)) * 1.5 / 40 / shape[-1] ** 0.5
    return [one(N, F, d), one(N, F, d), one(N, d, F)]


def on_gpu(group):
    if group is None:
        return None
    (gq, gs), (uq, us), (dq, ds) = [(q.cuda(), s.cuda()) for q, s in group]
    return occ.Int8Experts(gate=gq, up=uq, down=dq, gate_scale=gs, up_scale=us, down_scale=ds)


class Case:
    def __init__(self, T, d, Ne, k, F, Nd=1, n_shared=0, F_shared=0, seed=0, ids=None):
        g = torch.Generator().manual_seed(seed)
        self.desc = layer(T, d, Ne, k, F, Nd, n_shared, F_shared)
        self.x = torch.randn(T, d, generator=g).to(BF16)
        if ids is None:
            ids = torch.stack([torch.randperm(Ne, generator=g)[:k] for _ in range(T)])
        self.ids, self.w = ids.int(), torch.rand(T, k, generator=g) + 0.05
        self.experts = weights(g, Ne, F, d)
        self.shared = weights(g, n_shared, F_shared, d) if n_shared else None
        self.place = placement(Ne, Nd)

    def run(self, desc=None, place=None, stream=None):
        desc = desc or self.desc
        n = occ.occ_int8_workspace_size(desc)
        ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        y = torch.full((desc.T + 1, desc.d), NAN, dtype=BF16, device="cuda")
        occ.occ_moe_forward_int8(desc, self.x.cuda(), self.ids.cuda(), self.w.cuda(),
                                 self.place if place is None else place, on_gpu(self.experts),
                                 on_gpu(self.shared), y[:-1], ws[:n], stream)
        torch.cuda.synchronize()
        assert (ws[n:] == 0xA5).all() and torch.isnan(y[-1]).all()  # nothing behind the arrays
        return y[:-1].cpu()

    def check(self, y=None):
        y = self.run() if y is None else y
        want, bound = ref.layer8(self.x, self.ids, self.w, self.experts, self.shared)
        good = torch.isfinite(want)
        assert torch.equal(torch.isnan(y), ~good)
        off = (y.double() - want).abs()
        assert (off[good] <= bound[good] + 2.0 ** -126).all(), float((off / bound)[good].max())
        return y


# T, d, Ne, k, F, Nd, n_shared, F_shared: one token and one expert, lines that end half way (64
# more than a multiple of 128) in d, F and both, rows of one block and of many tiles of either
# height, hidden rows longer than a wave's registers, shared experts alone in size
LAYERS = [(1, 64, 1, 1, 64, 1, 0, 0), (1, 256, 8, 8, 128, 8, 0, 0), (1, 192, 16, 2, 320, 4, 1, 64),
          (2, 128, 4, 3, 192, 2, 0, 0), (3, 192, 8, 2, 320, 4, 2, 192), (5, 320, 6, 6, 64, 3, 0, 0),
          (17, 448, 5, 2, 192, 5, 0, 0), (64, 256, 64, 8, 128, 8, 0, 0), (130, 128, 2, 1, 128, 1, 1, 128),
          (300, 192, 8, 2, 192, 4, 1, 320), (700, 128, 4, 2, 256, 2, 0, 0),
          (401, 320, 3, 3, 448, 3, 2, 64), (1000, 64, 4, 4, 64, 2, 0, 0), (33, 64, 2, 1, 2112, 1, 0, 0),
          (450, 64, 2, 2, 2112, 2, 1, 2176), (9, 4160, 3, 1, 64, 3, 0, 0), (70, 8192, 2, 1, 64, 1, 0, 0),
          (650, 512, 60, 4, 192, 4, 1, 256), (257, 128, 256, 2, 64, 64, 0, 0),
          # few tokens: many slots, the widest rows, hidden rows longer than what a wave asks for
          # at once, shared experts alone long, widths that no workgroup's share divides
          (1, 64, 40, 32, 64, 2, 0, 0), (1, 8192, 3, 2, 64, 1, 1, 64), (4, 1088, 4, 2, 1088, 2, 0, 0),
          (2, 128, 3, 3, 4160, 1, 0, 0), (3, 2048, 2, 1, 64, 1, 2, 5632), (2, 1024, 8, 8, 1024, 8, 1, 2112),
          (1, 2112, 2, 1, 20480, 1, 0, 0), (1, 64, 2, 2, 40960, 1, 0, 0)]


@pytest.mark.parametrize("T,d,Ne,k,F,Nd,n_shared,F_shared", LAYERS)
def test_layer(T, d, Ne, k, F, Nd, n_shared, F_shared):
    case = Case(T, d, Ne, k, F, Nd, n_shared, F_shared, seed=T + d)
    y = case.check()
    # neither the placement nor the flags nor the run change a bit
    place = placement(Ne, Nd, seed=3)
    desc = layer(T, d, Ne, k, F, Nd, n_shared, F_shared, occ.OCC_FLAG_DETERMINISTIC)
    assert torch.equal(case.run(desc=desc, place=place), y)


# the shared experts' rows by the tokens, the routed ones' by their share: either tile for each
@pytest.mark.parametrize("T,d,Ne,k,F,Nd,n_shared,F_shared", [
    (1535, 128, 64, 2, 64, 4, 1, 320), (1536, 128, 64, 2, 64, 4, 1, 320), (2100, 192, 256, 8, 64, 8, 2, 192),
    (1535, 64, 4, 2, 128, 2, 1, 128), (1600, 64, 4, 2, 128, 2, 2, 64)])
def test_layer_of_many_tokens_with_shared_experts(T, d, Ne, k, F, Nd, n_shared, F_shared):
    case = Case(T, d, Ne, k, F, Nd, n_shared, F_shared, seed=T + Ne)
    y = case.check()
    # a part of the batch, on the other tiles: the same bits
    desc = layer(700, d, Ne, k, F, Nd, n_shared, F_shared)
    x, ids, w = (a[-700:].contiguous().cuda() for a in (case.x, case.ids, case.w))
    part = torch.empty(700, d, dtype=BF16, device="cuda")
    occ.occ_moe_forward_int8(desc, x, ids, w, case.place, on_gpu(case.experts), on_gpu(case.shared), part,
                             occ.alloc_int8_workspace(desc))
    assert torch.equal(part.cpu(), y[-700:])


@pytest.mark.parametrize("k,F,n_shared,F_shared", [(4, 1408, 1, 5632), (6, 1408, 2, 1408), (8, 1024, 0, 0)])
def test_layer_of_some_tokens_at_the_few_token_forms_end(k, F, n_shared, F_shared):
    """From three to nine tokens, where the choice of form changes: each token's bits as alone."""
    case = Case(9, 2048, 10, k, F, 2, n_shared, F_shared, seed=k + n_shared)
    whole = case.check()
    ex, sh = on_gpu(case.experts), on_gpu(case.shared)
    for T in range(1, 9):
        desc = layer(T, 2048, 10, k, F, 2, n_shared, F_shared)
        x, ids, w = (a[:T].contiguous().cuda() for a in (case.x, case.ids, case.w))
        n = occ.occ_int8_workspace_size(desc)
        ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        y = torch.empty(T, 2048, dtype=BF16, device="cuda")
        occ.occ_moe_forward_int8(desc, x, ids, w, case.place, ex, sh, y, ws[:n])
        assert torch.equal(y.cpu(), whole[:T]) and (ws[n:] == 0xA5).all(), T


@pytest.mark.parametrize("T,Ne,k", [(6, 32, 2), (900, 8, 1), (700, 64, 4)])
def test_layer_uneven_and_empty_experts(T, Ne, k):
    """Every token on the same experts, all others without rows; then half of the tokens."""
    ids = torch.arange(k).flip(0).expand(T, k) + Ne - k
    Case(T, 192, Ne, k, 128, seed=1, ids=ids).check()
    ids = ids.clone()
    ids[: T // 2] = torch.arange(k)
    Case(T, 192, Ne, k, 128, seed=2, ids=ids).check()


@pytest.mark.parametrize("T,Ne", [(4, 8), (300, 4)])
def test_layer_routing_of_any_values(T, Ne):
    """ids out of range and repeated become unused experts with weight 0; weights of zero and of
    either sign."""
    case = Case(T, 128, Ne, 3, 192, seed=4)
    case.ids[0] = torch.tensor([-1, Ne, 2 ** 30])
    case.ids[1] = 1
    case.ids[2, 1] = case.ids[2, 0]
    case.w[3] = torch.tensor([0.0, -1.5, 0.0])
    y = case.check()
    assert not y[0].any()


@pytest.mark.parametrize("T,Ne,k", [(1, 70, 20), (1, 256, 32), (40, 70, 20), (64, 256, 32)])
def test_layer_routing_of_many_slots_with_bad_ids(T, Ne, k):
    g = torch.Generator().manual_seed(k)
    ids = torch.randint(-3, Ne + 3, (T, k), generator=g)
    ids[0] = torch.arange(k) + Ne - k // 2  # the second half out of range
    Case(T, 64, Ne, k, 64, seed=11, ids=ids).check()


@pytest.mark.parametrize("d,F,F_shared", [(192, 320, 64), (2048, 1024, 1408)])
def test_layer_of_a_token_does_not_depend_on_its_batch(d, F, F_shared):
    """A token alone, with a few others and in batches of either tile height: the same bits."""
    case = Case(520, d, 8, 3, F, Nd=2, n_shared=1, F_shared=F_shared, seed=12)
    whole = case.run()
    ex, sh = on_gpu(case.experts), on_gpu(case.shared)
    for first, T in ((0, 1), (7, 1), (20, 3), (40, 10), (50, 11), (100, 100), (519, 1)):
        desc = layer(T, d, 8, 3, F, 2, 1, F_shared)
        x, ids, w = (a[first:first + T].contiguous().cuda() for a in (case.x, case.ids, case.w))
        y = torch.empty(T, d, dtype=BF16, device="cuda")
        occ.occ_moe_forward_int8(desc, x, ids, w, case.place, ex, sh, y, occ.alloc_int8_workspace(desc))
        assert torch.equal(y.cpu(), whole[first:first + T]), (first, T)


@pytest.mark.parametrize("T,Ne", [(7, 8), (300, 4)])
def test_layer_rows_of_zeros_tiny_and_not_finite(T, Ne):
    """What is not finite makes its own token's y NaN and no other's; a row of zeros gives zeros;
    rows too small for a scale are zeros."""
    case = Case(T, 192, Ne, 2, 192, seed=5, n_shared=1, F_shared=64)
    case.x[0] = 0.0
    case.x[1, 5] = NAN
    case.x[2, 191] = INF
    case.x[3] = case.x[3] * 2.0 ** -110
    case.w[4, 0] = NAN
    y = case.run()
    assert not y[0].any() and not y[3].any()
    assert torch.isnan(y[[1, 2, 4]]).all() and not torch.isnan(y[5:]).any()
    keep = torch.tensor([0, 3] + list(range(5, T)))
    case.w[4, 0] = 1.0
    case.x[1, 5], case.x[2, 191] = 0.0, 0.0
    want, bound = ref.layer8(case.x, case.ids, case.w, case.experts, case.shared)
    assert ((y.double() - want).abs() <= bound + 2.0 ** -126)[keep].all()


def test_layer_largest_codes_fill_the_sums():
    """Codes of 127 everywhere: the integer sums reach 127^2 K, exact."""
    case = Case(20, 8192, 2, 1, 2048, seed=6)
    case.x = torch.ones(20, 8192, dtype=BF16)
    for q, s in case.experts:
        q.fill_(127)
        s.fill_(1e-6)
    case.check()


def test_layer_channels_without_scale():
    case = Case(40, 128, 4, 2, 128, seed=7)
    for _, s in case.experts:
        s[1] = 0.0
        s[:, ::3] = 0.0
    y = case.check()
    assert not y[:, ::3].any()


def test_layer_on_streams_and_captured():
    """A side stream, then a graph replayed over new rows and routing with eager calls between;
    two graphs over one workspace, in turn."""
    T, d, Ne, k, F = 600, 256, 16, 4, 192
    case = Case(T, d, Ne, k, F, Nd=4, n_shared=1, F_shared=128, seed=8)
    few = Case(2, d, Ne, k, F, Nd=4, n_shared=1, F_shared=128, seed=8)
    ex, sh = on_gpu(case.experts), on_gpu(case.shared)
    ws = occ.alloc_int8_workspace(case.desc)
    ins = {c: [c.x.cuda(), c.ids.cuda(), c.w.cuda(), torch.empty(c.desc.T, d, dtype=BF16, device="cuda")]
           for c in (case, few)}

    def call(c, y=None, stream=None):
        x, ids, w, out = ins[c]
        occ.occ_moe_forward_int8(c.desc, x, ids, w, c.place, ex, sh, out if y is None else y, ws, stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(case, stream=side)
    side.synchronize()
    case.check(ins[case][3].cpu())
    graphs = {}
    for c in (case, few):
        call(c)
        torch.cuda.synchronize()
        graphs[c] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[c]):
            call(c)
    g = torch.Generator(device="cuda").manual_seed(9)
    for i in range(4):
        for c in (case, few):
            x, ids, w, out = ins[c]
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
            ids.copy_(torch.rand(c.desc.T, Ne, generator=g, device="cuda").argsort(1)[:, :k])
            out.fill_(NAN)
            graphs[c].replay()
        torch.cuda.synchronize()
        for c in (case, few):
            want = torch.empty_like(ins[c][3])
            call(c, want)
            torch.cuda.synchronize()
            assert torch.equal(ins[c][3], want), i


def test_layer_rows_behind_two_to_the_31_bytes():
    """Terms, hidden rows and codes behind 2^31 elements: equal tokens give equal rows."""
    T, d, Ne, k, F = 600_000, 1024, 4, 4, 1024
    case = Case(64, d, Ne, k, F, seed=10)
    desc = layer(T, d, Ne, k, F)
    rep = -(-T // 64)
    x, ids, w = (a.repeat(rep, 1)[:T].contiguous().cuda() for a in (case.x, case.ids, case.w))
    y, ws = torch.empty_like(x), occ.alloc_int8_workspace(desc)
    occ.occ_moe_forward_int8(desc, x, ids, w, case.place, on_gpu(case.experts), None, y, ws)
    first = y[:64].cpu()
    case.check(first)
    assert torch.equal(y[:T // 64 * 64].view(-1, 64, d), y[:64].expand(T // 64, -1, -1))


def test_binding_refuses_shapes_types_and_devices():
    case = Case(4, 128, 4, 2, 64)
    ex, ws = on_gpu(case.experts), occ.alloc_int8_workspace(case.desc)
    good = dict(x=case.x.cuda(), ids=case.ids.cuda(), w=case.w.cuda(), placement=case.place,
                experts=ex, shared=None, y=torch.empty(4, 128, dtype=BF16, device="cuda"), ws=ws)
    call = lambda **o: occ.occ_moe_forward_int8(case.desc, *{**good, **o}.values())
    call()
    other = on_gpu(weights(torch.Generator().manual_seed(1), 4, 128, 128))
    for bad in (dict(x=good["x"].float()), dict(x=good["x"][:2]), dict(ids=good["ids"].long()),
                dict(w=good["w"].double()), dict(y=good["y"].cpu()), dict(experts=other),
                dict(shared=ex)):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(experts=None), dict(ws=ws[:256]), dict(y=good["x"]), dict(placement=None)):
        with pytest.raises(occ.OccError):
            call(**bad)
    with pytest.raises(ValueError):
        occ.Int8Experts(gate=good["x"], up=None, down=None, gate_scale=None, up_scale=None,
                        down_scale=None)
