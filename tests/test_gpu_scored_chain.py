"""Routing by scores and experts in 8 bits together, as a program uses them: a training step (gate
projection, router by scores, the bias's step, the layer on that routing, everything backward)
against differentiating it in 64 bits, captured and replayed; and a serving step (weights quantised
once, gate projection, router, the layer in 8 bits) against its reference and the bf16 layer."""
import pytest
import torch

import score_reference as ref
from expert_token_routing_amd import occ, synth, workloads as W

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
WEIGHTS = ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    occ.lib()


def empty(*shape, dtype=F32):
    return torch.full(shape, float("nan"), device="cuda").to(dtype)


class Step:
    def __init__(self, kind, groups, renorm, T=300, seed=3):
        wl = W.Workload("scored_step", 41, T=T, d=256, Ne=16, k=4, Nd=4, F=256, n_shared=1,
                        F_shared=256, n_c=2, bonus=1.0)
        inp = synth.make_all(wl)
        self.wl, self.place = wl, inp["placement"]
        self.desc = occ.desc_of(wl, flags=occ.OCC_FLAG_TRAIN | occ.OCC_FLAG_DETERMINISTIC)
        self.opt = occ.ScoreDesc(score=kind, top_groups=groups, group_best=2, renormalise=renorm,
                                 scale=1.5)
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.w = {n: inp[n].cuda() for n in WEIGHTS}
        self.w["w_router"] = (randn(wl.Ne, wl.d) * 0.1).to(BF16)
        self.x, self.dy = randn(T, wl.d).to(BF16), randn(T, wl.d).to(BF16)
        self.bias = randn(wl.Ne) * 0.02
        T, Ne, k = wl.T, wl.Ne, wl.k
        self.logits, self.dlogits = empty(T, Ne), empty(T, Ne)
        self.ids, self.rw, self.dw = empty(T, k).to(I32), empty(T, k), empty(T, k)
        self.counts, self.new_bias = empty(Ne + 1).to(I32), empty(Ne)
        self.y, self.dx = empty(T, wl.d, dtype=BF16), empty(T, wl.d, dtype=BF16)
        self.grad = {n: empty(*v.shape) for n, v in self.w.items()}
        self.ws, self.ws2 = occ.alloc_workspace(self.desc), occ.alloc_block_workspace(self.desc)

    def run(self):
        D, w, g = self.desc, [self.w[n] for n in WEIGHTS], [self.grad[n] for n in WEIGHTS]
        occ.occ_gate(D, self.x, self.w["w_router"], self.logits)
        occ.occ_route_scored(D, self.opt, self.logits, self.bias, self.place, self.ids, self.rw)
        occ.occ_route_bias_step(D, 1e-3, self.ids, None, self.bias, self.counts, self.new_bias,
                                self.ws2)
        occ.occ_moe_forward_routed(D, self.x, self.ids, self.rw, self.place, *w, self.y, self.ws)
        occ.occ_moe_backward(D, self.dy, self.x, None, self.place, *w, self.dx, *g, self.dw, None,
                             self.ws)
        occ.occ_route_scored_backward(D, self.opt, self.logits, self.ids, self.dw, None,
                                      self.dlogits)
        occ.occ_gate_backward(D, self.dlogits, self.x, self.w["w_router"], self.dx, self.dx,
                              self.grad["w_router"], self.ws2)

    def outputs(self):
        return {"y": self.y, "dx": self.dx, "ids": self.ids, "rw": self.rw, "counts": self.counts,
                "bias": self.new_bias, "dlogits": self.dlogits, **self.grad}


def in_64_bits(st):
    """y and the gradients of <y, dy>, the choice held fixed."""
    wl, v = st.wl, {n: a.double().requires_grad_(True) for n, a in st.w.items()}
    x = st.x.double().requires_grad_(True)
    logits = x @ v["w_router"].t()
    s = torch.sigmoid(logits) if st.opt.score == ref.SIGMOID else torch.softmax(logits, 1)
    w = s.gather(1, st.ids.long())
    w = 1.5 * (w / w.sum(1, keepdim=True) if st.opt.renormalise else w)
    y = torch.zeros_like(x)
    for e in range(wl.Ne):
        weight = (w * (st.ids == e)).sum(1, keepdim=True)
        act = torch.nn.functional.silu(x @ v["w_gate"][e].t()) * (x @ v["w_up"][e].t())
        y = y + (weight * act) @ v["w_down"][e].t()
    act = torch.nn.functional.silu(x @ v["ws_gate"][0].t()) * (x @ v["ws_up"][0].t())
    y = y + act @ v["ws_down"][0].t()
    names = list(v)
    grads = torch.autograd.grad((y * st.dy.double()).sum(), [x] + [v[n] for n in names])
    return y.detach(), dict(zip(["x"] + names, grads))


@pytest.mark.parametrize("renorm", [0, 1], ids=["scores", "renormalised"])
@pytest.mark.parametrize("kind,groups", [(ref.SOFTMAX, 4), (ref.SIGMOID, 2)],
                         ids=["softmax", "sigmoid_groups"])
def test_training_step_gradients_against_64_bits(kind, groups, renorm):
    """The layer's own tolerance, 2e-2 of the norm (its bf16 intermediates); the routing's
    operators are fp32 and add nothing to it."""
    st = Step(kind, groups, renorm)
    st.run()
    torch.cuda.synchronize()
    ids, w = ref.route(st.logits.cpu(), st.bias.cpu(), st.place, st.wl.k, kind, groups, 2, renorm, 1.5)
    assert torch.equal(st.ids.cpu(), ids)
    assert torch.equal(st.counts.cpu(), ref.bias_step(ids, None, st.bias.cpu(), 16, 1e-3)[0])
    y, grads = in_64_bits(st)
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(st.y, y) <= 2e-2
    for name, want in grads.items():
        got = st.dx if name == "x" else st.grad[name]
        assert rel(got, want) <= 2e-2, (name, rel(got, want))


def test_training_step_captured_and_replayed():
    """The step in one graph, over new rows and gradients, with eager work between: the eager
    step's bits every time."""
    eager, cap = Step(ref.SIGMOID, 2, 1), Step(ref.SIGMOID, 2, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cap.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap.run()
    g = torch.Generator(device="cuda").manual_seed(9)
    for i in range(4):
        x, dy = (torch.randn(300, 256, generator=g, device="cuda").to(BF16) for _ in range(2))
        for st in (eager, cap):
            st.x.copy_(x)
            st.dy.copy_(dy)
            st.bias.mul_(-1)
        cap.ws2.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        eager.run()
        torch.cuda.synchronize()
        a, b = eager.outputs(), cap.outputs()
        assert all(torch.equal(a[n], b[n]) for n in a), [n for n in a if not torch.equal(a[n], b[n])]


def quantised(names, w):
    out = []
    for n in names:
        q = torch.empty_like(w[n], dtype=torch.int8)
        s = torch.empty(w[n].shape[:-1], device="cuda")
        occ.occ_quantize_int8(w[n], q, s)
        out.append((q, s))
    (gq, gs), (uq, us), (dq, ds) = out
    return out, occ.Int8Experts(gate=gq, up=uq, down=dq, gate_scale=gs, up_scale=us, down_scale=ds)


@pytest.mark.parametrize("T", [1, 3, 48, 700])
def test_serving_step(T):
    """Against the reference within its bound, and against the bf16 layer on the same routing: the
    codes of rows whose largest value is some 3 to 4 times their size are off by 0.29 of a step of
    1/127 of it, 0.7 to 0.9% each for x, the weights and twice that for h (a product of two, whose
    largest value stands out more): under 3% of y's norm together, taken twice."""
    st = Step(ref.SIGMOID, 2, 1, T=T)
    D = occ.desc_of(st.wl)
    plain, experts = quantised(WEIGHTS[:3], st.w)
    plain_sh, shared = quantised(WEIGHTS[3:], st.w)
    ws8, ws = occ.alloc_int8_workspace(D), occ.alloc_workspace(D)

    def serve(y):
        occ.occ_gate(D, st.x, st.w["w_router"], st.logits)
        occ.occ_route_scored(D, st.opt, st.logits, st.bias, st.place, st.ids, st.rw)
        occ.occ_moe_forward_int8(D, st.x, st.ids, st.rw, st.place, experts, shared, y, ws8)

    serve(st.y)
    y16 = torch.empty_like(st.y)
    occ.occ_moe_forward_routed(D, st.x, st.ids, st.rw, st.place, *[st.w[n] for n in WEIGHTS], y16, ws)
    torch.cuda.synchronize()
    host = lambda group: [(q.cpu(), s.cpu()) for q, s in group]
    want, bound = ref.layer8(st.x.cpu(), st.ids.cpu(), st.rw.cpu(), host(plain), host(plain_sh))
    assert ((st.y.cpu().double() - want).abs() <= bound + 2.0 ** -126).all()
    assert float((st.y.double() - y16.double()).norm() / y16.double().norm()) <= 6e-2
    graph, first = torch.cuda.CUDAGraph(), st.y.clone()
    with torch.cuda.graph(graph):
        serve(st.y)
    for i in range(3):
        st.y.fill_(float("nan"))
        ws8.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(st.y, first), i
        serve(y16)  # eager work between the replays
        torch.cuda.synchronize()


def test_two_layers_at_once():
    """Two calls on two streams with a workspace each, behind work that keeps both waiting."""
    a, b = Step(ref.SIGMOID, 2, 1, T=600), Step(ref.SOFTMAX, 4, 1, T=500, seed=4)
    calls, want = [], []
    for st in (a, b):
        D = occ.desc_of(st.wl)
        occ.occ_gate(D, st.x, st.w["w_router"], st.logits)
        occ.occ_route_scored(D, st.opt, st.logits, st.bias, st.place, st.ids, st.rw)
        experts, shared = quantised(WEIGHTS[:3], st.w)[1], quantised(WEIGHTS[3:], st.w)[1]
        args = (D, st.x, st.ids, st.rw, st.place, experts, shared, st.y, occ.alloc_int8_workspace(D))
        occ.occ_moe_forward_int8(*args)
        calls.append(args)
        want.append(st.y.clone())
    torch.cuda.synchronize()
    streams, busy = [torch.cuda.Stream(), torch.cuda.Stream()], torch.zeros(1 << 24, device="cuda")
    for _ in range(5):
        for st in (a, b):
            st.y.fill_(float("nan"))
        torch.cuda.synchronize()
        for s, args in zip(streams, calls):
            with torch.cuda.stream(s):
                busy.add_(0.0)
            for _ in range(3):
                occ.occ_moe_forward_int8(*args, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a.y, want[0]) and torch.equal(b.y, want[1])
