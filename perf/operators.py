"""Operator workloads of a training step around the MoE layer: the block's norms and residual, the
router's losses, the gate projection's backward and the optimizer step.

Every case runs one operator on inputs made from a seed.  With `own` false `run` computes it in
elementary torch operations, in 32 bits, rounded once to the outputs' types; with `own` true it
calls the library as a training or serving program does.  `exact` evaluates the definitions in 64
bits (gradients by differentiating the forward definition).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6          # the norms' epsilon
SCALE = 0.7         # residual scale of the block's output
COEF = (1e-2, 3e-3, 1e-3)  # balance, group balance and z-loss coefficients
UPSTREAM = 0.5      # gradient of the step's loss in the router loss
ADAM = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=100, grad_scale=0.5)
BLOCK = 256         # elements that share a scale in the 8-bit optimizer states
E4M3_MAX, E4M3_MIN = 448.0, 2.0 ** -9


# ---------------------------------------------------------------- cases ----

def listed():
    return [
        # one token of one request between two blocks: the sandwich norms and the residual in a
        # decode step of the OLMoE-shaped model, where only latency counts
        dict(name="norm_t1_bf16", op="norm", T=1, d=2048, dtype="bf16", y=True, post=True,
             gate="none", pre=True),
        # the same boundary over the long prefill batch of the Qwen-shaped layer, with a learned
        # gate per channel
        dict(name="norm_t65536_bf16", op="norm", T=65536, d=2048, dtype="bf16", y=True, post=True,
             gate="channel", pre=True),
        # its backward pass in a training step of the OLMoE-shaped layer
        dict(name="norm_back_t8192_bf16", op="norm_back", T=8192, d=2048, dtype="bf16", y=True,
             post=True, gate="channel", pre=True),
        # a full-precision backward pass with an odd token count, a gate per token and no norm
        # behind the block (a pre-norm model of odd width)
        dict(name="norm_back_t4099_f32", op="norm_back", T=4099, d=1408, dtype="f32", y=True,
             post=False, gate="token", pre=True),
        # router losses, counts and their gradient for the batch of a small training step
        dict(name="balance_t512_e64", op="balance", T=512, Ne=64, k=8, Nd=8, mask=False),
        # the same for the largest batch, with padding tokens at the end of its sequences
        dict(name="balance_t65536_e60", op="balance", T=65536, Ne=60, k=4, Nd=4, mask=True),
        # gate projection's backward: the full-precision tiny layer
        dict(name="gate_back_t256_f32", op="gate_back", T=256, d=128, Ne=8, dtype="f32", dx=True),
        # the OLMoE-shaped training step
        dict(name="gate_back_t8192_bf16", op="gate_back", T=8192, d=2048, Ne=64, dtype="bf16",
             dx=True),
        # the Qwen-shaped training step
        dict(name="gate_back_t65536_bf16", op="gate_back", T=65536, d=2048, Ne=60, dtype="bf16",
             dx=True),
        # optimizer step of one block's small tensors (router, norm weights, gate): launch-bound
        dict(name="adamw_block_f32", op="adamw", sizes="131072,2048,2048,2048,60,1", bits=32,
             grad="f32", copy=True),
        # optimizer step of one OLMoE-shaped layer's experts, states in 32 bits
        dict(name="adamw_experts_f32", op="adamw", sizes="134217728,134217728,134217728", bits=32,
             grad="f32", copy=True),
        # the Qwen-shaped shared expert with states in 8 bits, beside small tensors of odd length
        dict(name="adamw_shared_8bit", op="adamw",
             sizes="11534336,11534336,11534336,122880,2048,1001", bits=8, grad="f32", copy=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "balance", "gate_back", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    unit = 64 if dtype == "bf16" else 16
    if op in ("norm", "norm_back"):
        d = unit * _log_int(rng, 1 if dtype == "f32" else 2, (8192 if dtype == "bf16" else 4096) // unit)
        T = _log_int(rng, 1, min(65536, (65536 * 2048 if dtype == "bf16" else 65536 * 512) // d))
        y = rng.random() < 0.8
        return dict(op=op, T=T, d=d, dtype=dtype, y=y, post=y and rng.random() < 0.6,
                    gate=rng.choice(["none", "channel", "token"]) if y else "none",
                    pre=(not y) or rng.random() < 0.8)
    if op == "balance":
        Nd = rng.choice([1, 2, 3, 4, 8])
        Ne = Nd * rng.randint(2, 256 // Nd)
        return dict(op=op, T=_log_int(rng, 1, min(65536, 65536 * 60 // Ne)), Ne=Ne,
                    k=rng.randint(1, min(Ne, 8)), Nd=Nd, mask=rng.random() < 0.5)
    if op == "gate_back":
        d = unit * _log_int(rng, 2, 4096 // unit)
        Ne = rng.randint(2, 256)
        most = 65536 * 2048 * 60 // (4 if dtype == "f32" else 1)
        return dict(op=op, T=_log_int(rng, 1, min(65536, most // (d * max(Ne, 60)))), d=d, Ne=Ne,
                    dtype=dtype, dx=rng.random() < 0.8)
    sizes = [_log_int(rng, 1, 1 << 24) for _ in range(rng.randint(1, 10))]
    return dict(op=op, sizes=",".join(str(n) for n in sizes), bits=rng.choice([32, 8]),
                grad=rng.choice(["f32", "f32", "bf16"]), copy=rng.random() < 0.7)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        T, d = case["T"], case["d"]
        es = 2 if case["dtype"] == "bf16" else 4
        post, chan, pre = case["post"], case["gate"] == "channel", case["pre"]
        tok = 4 * T if case["gate"] == "token" else 0
        if op == "norm":  # x (, y) in, (r,) (h) out
            rows = 1 + 2 * case["y"] + pre
            return dict(bytes=rows * T * d * es + (post + chan + pre) * d * es + tok,
                        flops=(1 + 5 * case["y"] + 4 * post + 4 * pre) * T * d)
        # dr (, dh, r) (, y) in, dx (, dy) out; y only for its norm's and its gate's gradients
        rows = 2 + 2 * pre + case["y"] + (post or case["gate"] != "none")
        return dict(bytes=rows * T * d * es + (post + chan + pre) * d * (es + 4) + 2 * tok,
                    flops=(1 + 5 * case["y"] + 12 * post + 12 * pre + 3 * chan) * T * d)
    if op == "balance":
        T, Ne, k = case["T"], case["Ne"], case["k"]
        return dict(bytes=3 * 4 * T * Ne + 4 * T * k + T * case["mask"] + 8 * Ne,
                    flops=16 * T * Ne)
    if op == "gate_back":
        T, d, Ne = case["T"], case["d"], case["Ne"]
        es = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=(2 + case["dx"]) * T * d * es + 4 * T * Ne + Ne * d * (es + 4),
                    flops=4 * T * Ne * d)
    n = sum(int(s) for s in case["sizes"].split(","))
    state = 8 if case["bits"] == 32 else 2 + 8 / BLOCK
    per = 4 + (4 if case["grad"] == "f32" else 2) + state + 4 + state + 2 * case["copy"]
    return dict(bytes=per * n, flops=14 * n)


# --------------------------------------------------------------- inputs ----

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _placement(Ne, Nd):
    return torch.arange(Ne, dtype=torch.int32).view(Nd, Ne // Nd).numpy()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], dict(case=dict(case))
    if op in ("norm", "norm_back"):
        T, d, dt = case["T"], case["d"], DTYPES[case["dtype"]]
        # a residual stream a few units wide with some strong channels, a block's output of about
        # unit size, trained norm weights and gates
        chan = 1 + 4 * (torch.rand(d, generator=gen, device="cuda") < 0.02).float()
        s["x"] = (_randn(gen, T, d) * chan * 2).to(dt)
        s["y"] = (_randn(gen, T, d) * 0.8).to(dt) if case["y"] else None
        s["w_post"] = (1 + 0.2 * _randn(gen, d)).to(dt) if case["post"] else None
        s["w_pre"] = (1 + 0.2 * _randn(gen, d)).to(dt) if case["pre"] else None
        s["gate"] = None
        if case["gate"] == "channel":
            s["gate"] = (0.5 + 0.2 * _randn(gen, d)).to(dt)
        elif case["gate"] == "token":
            s["gate"] = torch.sigmoid(_randn(gen, T))
        if op == "norm":
            s["r_out"] = torch.empty_like(s["x"]) if case["y"] else None
            s["h_out"] = torch.empty_like(s["x"]) if case["pre"] else None
        else:
            s["dr"] = (_randn(gen, T, d) * 0.01).to(dt)
            s["dh"] = (_randn(gen, T, d) * 0.03).to(dt) if case["pre"] else None
            f32 = dict(dtype=torch.float32, device="cuda")
            s["dx"] = torch.empty_like(s["x"])
            s["dy"] = torch.empty_like(s["x"]) if case["y"] else None
            s["dw_post"] = torch.empty(d, **f32) if case["post"] else None
            s["dw_pre"] = torch.empty(d, **f32) if case["pre"] else None
            s["dgate"] = torch.empty(s["gate"].numel(), **f32) if s["gate"] is not None else None
        return s
    if op == "balance":
        T, Ne, k = case["T"], case["Ne"], case["k"]
        # a router in training: noise and a preference that loads some experts more than others
        s["logits"] = _randn(gen, T, Ne) + 0.7 * _randn(gen, Ne)
        s["ids"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
        s["valid"] = None
        if case["mask"]:
            s["valid"] = torch.rand(T, generator=gen, device="cuda") < 0.9
        s["dlogits"] = _randn(gen, T, Ne) * 1e-4 / max(1, T)
        s["placement"] = _placement(Ne, case["Nd"])
        f32 = dict(dtype=torch.float32, device="cuda")
        s["counts_out"] = torch.empty(Ne + 1, dtype=torch.int32, device="cuda")
        s["probs_out"], s["loss_out"] = torch.empty(Ne, **f32), torch.empty(4, **f32)
        s["dlogits_out"] = torch.empty(T, Ne, **f32)
        return s
    if op == "gate_back":
        T, d, Ne, dt = case["T"], case["d"], case["Ne"], DTYPES[case["dtype"]]
        s["x"] = _randn(gen, T, d).to(dt)
        s["w_router"] = (_randn(gen, Ne, d) * 0.05).to(dt)
        s["dlogits"] = _randn(gen, T, Ne) * torch.exp(_randn(gen, T, Ne)) * 1e-2
        s["dx_in"] = (_randn(gen, T, d) * 0.01).to(dt) if case["dx"] else None
        s["dx"] = torch.empty_like(s["x"])
        s["dw_router"] = torch.empty(Ne, d, dtype=torch.float32, device="cuda")
        return s
    s["tensors"] = []
    for n in (int(v) for v in case["sizes"].split(",")):
        t = dict(p=_randn(gen, n) * 0.02, g=_randn(gen, n) * 1e-3)
        m, r = _randn(gen, n) * 5e-4, torch.exp(0.5 * _randn(gen, n)) * 7e-4
        if case["grad"] == "bf16":
            t["g"] = t["g"].bfloat16()
        if case["bits"] == 32:
            t.update(m=m, v=r * r, m_scale=None, v_scale=None)
        else:
            t["m"], t["m_scale"] = _to_e4m3(m)
            t["v"], t["v_scale"] = _to_e4m3(r, keep_nonzero=True)
        t["out"] = {key: None if v is None else torch.empty_like(v) for key, v in t.items()
                    if key != "g"}
        t["out"]["copy"] = (torch.empty(n, dtype=torch.bfloat16, device="cuda") if case["copy"]
                            else None)
        s["tensors"].append(t)
    return s


# ---------------------------------------------------------- plain forms ----

def _unit_rows(v):
    """v / rms(v) by rows, and 1 / rms(v)."""
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * rstd, rstd


def _gate_of(s):
    gate = s["gate"].float()
    return gate[:, None] if s["case"]["gate"] == "token" else gate


def _plain_norm(s):
    dt, r = s["x"].dtype, s["x"].float()
    if s["y"] is not None:
        z = s["y"].float()
        if s["w_post"] is not None:
            z = _unit_rows(z)[0] * s["w_post"].float()
        if s["gate"] is not None:
            z = z * _gate_of(s)
        r = r + SCALE * z
    h = None if s["w_pre"] is None else (_unit_rows(r)[0] * s["w_pre"].float()).to(dt)
    return dict(r=None if s["y"] is None else r.to(dt), h=h)


def _unit_rows_back(dn, n, rstd):
    """The gradient at v of n = v / rms(v), from the gradient dn at n."""
    return rstd * (dn - n * (dn * n).mean(1, keepdim=True))


def _plain_norm_back(s):
    # x holds the forward's r here: the rows that its last norm read
    dt, out = s["x"].dtype, dict(dx=None, dy=None, dw_post=None, dw_pre=None, dgate=None)
    dr = s["dr"].float()
    if s["w_pre"] is not None:
        dh = s["dh"].float()
        n, rstd = _unit_rows(s["x"].float())
        out["dw_pre"] = (dh * n).sum(0)
        dr = dr + _unit_rows_back(dh * s["w_pre"].float(), n, rstd)
    out["dx"] = dr.to(dt)
    if s["y"] is None:
        return out
    y, dz = s["y"].float(), SCALE * dr
    if s["w_post"] is not None:
        n, rstd = _unit_rows(y)
        z = n * s["w_post"].float()
    else:
        z = y
    if s["gate"] is not None:
        out["dgate"] = (dz * z).sum(1 if s["case"]["gate"] == "token" else 0)
        dz = dz * _gate_of(s)
    if s["w_post"] is not None:
        out["dw_post"] = (dz * n).sum(0)
        dz = _unit_rows_back(dz * s["w_post"].float(), n, rstd)
    out["dy"] = dz.to(dt)
    return out


def _plain_balance(s):
    T, Ne, k, Nd = (s["case"][key] for key in ("T", "Ne", "k", "Nd"))
    logits, experts = s["logits"], torch.arange(Ne, device="cuda", dtype=torch.int32)
    chosen = s["ids"][:, :, None] == experts
    if s["valid"] is None:
        keep = torch.ones(T, 1, device="cuda")
    else:
        keep = s["valid"][:, None].float()
        chosen = chosen & s["valid"][:, None, None]
        logits = torch.where(s["valid"][:, None], logits, torch.zeros_like(logits))
    counts = chosen.sum((0, 1))
    n = keep.sum()
    top = logits.max(1, keepdim=True).values
    p = torch.exp(logits - top)
    total = p.sum(1, keepdim=True)
    p, lse = p / total, top + torch.log(total)
    div = torch.clamp(n, min=1.0)
    probs = (p * keep).sum(0) / div
    f = counts.float() * Ne / (k * div)
    f_grp = f.view(Nd, -1).mean(1)
    terms = torch.stack([COEF[0] * (f * probs).sum(),
                         COEF[1] * (f_grp * probs.view(Nd, -1).sum(1)).sum(),
                         COEF[2] * (lse * lse * keep).sum() / div])
    c = COEF[0] * (f - 1) + COEF[1] * (f_grp - 1).repeat_interleave(Ne // Nd)
    grad = p * (c - (c * p).sum(1, keepdim=True) + 2 * COEF[2] * lse)
    return dict(loss=torch.cat([terms.sum()[None], terms]), probs=probs,
                counts=torch.cat([counts, n.to(counts.dtype)[None]]).to(torch.int32),
                dlogits=s["dlogits"] + UPSTREAM / div * keep * grad)


def _plain_gate_back(s):
    dx = s["dlogits"] @ s["w_router"].float()
    if s["dx_in"] is not None:
        dx = dx + s["dx_in"].float()
    return dict(dx=dx.to(s["x"].dtype), dw_router=s["dlogits"].t() @ s["x"].float())


def _scaled_blocks(v):
    """v in rows of BLOCK values (zeros behind the last), and what one unit of each row stands for."""
    rows = torch.zeros(-(-v.numel() // BLOCK) * BLOCK, device=v.device)
    rows[:v.numel()] = v
    rows = rows.view(-1, BLOCK)
    top = rows.abs().max(1, keepdim=True).values
    return rows, top / E4M3_MAX


def _to_e4m3(v, keep_nonzero=False):
    rows, unit = _scaled_blocks(v)
    code = torch.where(unit > 0, rows / torch.where(unit > 0, unit, torch.ones_like(unit)),
                       torch.zeros_like(rows)).clamp(-E4M3_MAX, E4M3_MAX)
    if keep_nonzero:
        code = torch.where(rows > 0, code.clamp(min=E4M3_MIN), code)
    return code.view(-1)[:v.numel()].to(torch.float8_e4m3fn), unit[:, 0].contiguous()


def _from_e4m3(code, unit):
    return code.float() * unit.repeat_interleave(BLOCK)[:code.numel()]


def _plain_adamw(t):
    a = ADAM
    c1, c2 = 1 - a["beta1"] ** a["step"], 1 - a["beta2"] ** a["step"]
    g = t["g"].float() * a["grad_scale"]
    if t["m_scale"] is None:
        m, v = t["m"], t["v"]
    else:
        m, v = _from_e4m3(t["m"], t["m_scale"]), _from_e4m3(t["v"], t["v_scale"]).square()
    m = a["beta1"] * m + (1 - a["beta1"]) * g
    v = a["beta2"] * v + (1 - a["beta2"]) * g * g
    p = t["p"] * (1 - a["lr"] * a["weight_decay"])
    p = p - a["lr"] / c1 * m / (torch.sqrt(v) / math.sqrt(c2) + a["eps"])
    out = dict(p=p, m=m, v=v, m_scale=None, v_scale=None, copy=None)
    if t["m_scale"] is not None:
        out["m"], out["m_scale"] = _to_e4m3(m)
        out["v"], out["v_scale"] = _to_e4m3(torch.sqrt(v), keep_nonzero=True)
    if t["out"]["copy"] is not None:
        out["copy"] = p.bfloat16()
    return out


# ----------------------------------------------------- the library's calls ----

def _dtype_of(occ, name):
    return occ.OCC_BF16 if name == "bf16" else occ.OCC_F32


def _desc(occ, case):
    """The layer that the operator stands beside: sizes it does not use take any valid value."""
    return occ.LayerDesc(T=case["T"], d=case.get("d", 64), Ne=case.get("Ne", 1),
                         k=case.get("k", 1), Nd=case.get("Nd", 1), F=64, n_shared=0, F_shared=0,
                         prune_rule=0, prune_groups=0,
                         dtype=_dtype_of(occ, case.get("dtype", "f32")), flags=0)


def _handle(s, occ):
    """What a program keeps from call to call: descriptors, the workspace, the tensor table."""
    if "handle" not in s:
        case, h = s["case"], {}
        if case["op"] == "adamw":
            h["opt"] = occ.AdamwDesc(state=occ.OCC_ADAMW_8BIT if case["bits"] == 8
                                     else occ.OCC_ADAMW_32BIT,
                                     grad_dtype=_dtype_of(occ, case["grad"]), **ADAM)
            h["table"] = occ.AdamwTensors(h["opt"], [
                dict(p=t["p"], g=t["g"], m=t["m"], v=t["v"], m_scale=t["m_scale"],
                     v_scale=t["v_scale"], p_out=t["out"]["p"], m_out=t["out"]["m"],
                     v_out=t["out"]["v"], m_scale_out=t["out"]["m_scale"],
                     v_scale_out=t["out"]["v_scale"], p_bf16=t["out"]["copy"])
                for t in s["tensors"]])
        else:
            h["desc"] = _desc(occ, case)
            if case["op"] in ("norm", "norm_back"):
                kind = dict(none=occ.OCC_GATE_NONE, channel=occ.OCC_GATE_CHANNEL,
                            token=occ.OCC_GATE_TOKEN)[case["gate"]]
                h["opt"] = occ.NormDesc(eps=EPS, scale=SCALE, gate=kind)
            elif case["op"] == "balance":
                h["opt"] = occ.BalanceDesc(balance=COEF[0], group=COEF[1], z=COEF[2])
            if case["op"] != "norm":
                h["ws"] = occ.alloc_block_workspace(h["desc"])
        s["handle"] = h
    return s["handle"]


def _own_run(s):
    from expert_token_routing_amd import occ

    h, op = _handle(s, occ), s["case"]["op"]
    if op == "norm":
        occ.occ_block_norm(h["desc"], h["opt"], s["x"], s["y"], s["w_post"], s["gate"],
                           s["w_pre"], s["r_out"], s["h_out"])
        return dict(r=s["r_out"], h=s["h_out"])
    if op == "norm_back":
        occ.occ_block_norm_backward(h["desc"], h["opt"], s["dr"], s["dh"], s["x"], s["y"],
                                    s["w_post"], s["gate"], s["w_pre"], s["dx"], s["dy"],
                                    s["dw_post"], s["dgate"], s["dw_pre"], h["ws"])
        return {key: s[key] for key in ("dx", "dy", "dw_post", "dw_pre", "dgate")}
    if op == "balance":
        occ.occ_balance_loss(h["desc"], h["opt"], s["logits"], s["ids"], s["valid"],
                             s["placement"], s["counts_out"], s["probs_out"], s["loss_out"],
                             h["ws"])
        occ.occ_balance_backward(h["desc"], h["opt"], s["logits"], s["valid"], s["placement"],
                                 s["counts_out"], UPSTREAM, s["dlogits"], s["dlogits_out"])
        return dict(loss=s["loss_out"], probs=s["probs_out"], counts=s["counts_out"],
                    dlogits=s["dlogits_out"])
    if op == "gate_back":
        occ.occ_gate_backward(h["desc"], s["dlogits"], s["x"], s["w_router"], s["dx_in"],
                              s["dx"], s["dw_router"], h["ws"])
        return dict(dx=s["dx"], dw_router=s["dw_router"])
    occ.occ_adamw_step(h["opt"], h["table"])
    return [t["out"] for t in s["tensors"]]


def run(s):
    if own:
        return _own_run(s)
    op = s["case"]["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_back":
        return _plain_norm_back(s)
    if op == "balance":
        return _plain_balance(s)
    if op == "gate_back":
        return _plain_gate_back(s)
    return [_plain_adamw(t) for t in s["tensors"]]


# ---------------------------------------------------- definitions, 64 bits ----

def _rms64(v):
    return torch.sqrt(torch.square(v).sum(-1, keepdim=True) / v.shape[-1] + EPS)


def _block64(x, y, w_post, gate, w_pre, per_token):
    r = x
    if y is not None:
        out = y if w_post is None else w_post * y / _rms64(y)
        if gate is not None:
            out = gate.reshape(-1, 1) * out if per_token else gate * out
        r = x + SCALE * out
    return r, None if w_pre is None else w_pre * r / _rms64(r)


def _exact_norm(s):
    big = {key: None if s[key] is None else s[key].double()
           for key in ("x", "y", "w_post", "gate", "w_pre")}
    r, h = _block64(**big, per_token=s["case"]["gate"] == "token")
    return dict(r=r if s["y"] is not None else None, h=h)


def _exact_norm_back(s):
    """By differentiation; the residual input is what makes the forward's r equal s["x"]."""
    names = ("x", "y", "w_post", "gate", "w_pre")
    per_token = s["case"]["gate"] == "token"
    v = {key: None if s[key] is None else s[key].double() for key in names}
    if v["y"] is not None:
        v["x"] = v["x"] - (_block64(torch.zeros_like(v["x"]), v["y"], v["w_post"], v["gate"],
                                    None, per_token)[0])
    given = [key for key in names if v[key] is not None]
    for key in given:
        v[key].requires_grad_(True)
    r, h = _block64(**v, per_token=per_token)
    goal = (r * s["dr"].double()).sum()
    if h is not None:
        goal = goal + (h * s["dh"].double()).sum()
    grads = dict(zip(given, torch.autograd.grad(goal, [v[key] for key in given])))
    return dict(dx=grads["x"], dy=grads.get("y"), dw_post=grads.get("w_post"),
                dw_pre=grads.get("w_pre"), dgate=grads.get("gate"))


def _exact_balance(s):
    T, Ne, k, Nd = (s["case"][key] for key in ("T", "Ne", "k", "Nd"))
    rows = torch.arange(T, device="cuda") if s["valid"] is None else s["valid"].nonzero()[:, 0]
    n = rows.numel()
    counts = torch.bincount(s["ids"][rows].flatten().long(), minlength=Ne)
    if n == 0:
        zero = torch.zeros(4, dtype=torch.float64, device="cuda")
        return dict(loss=zero, probs=zero.new_zeros(Ne), counts=None,
                    dlogits=s["dlogits"].double())
    logits = s["logits"][rows].double().requires_grad_(True)
    probs = torch.softmax(logits, 1).mean(0)
    load = counts.double() / (n * k)  # share of the routed slots
    groups = torch.arange(Ne, device="cuda") // (Ne // Nd)
    pool = torch.zeros(Nd, dtype=torch.float64, device="cuda")
    terms = torch.stack([
        COEF[0] * Ne * torch.dot(load, probs),
        COEF[1] * Nd * torch.dot(pool.index_add(0, groups, load),
                                 pool.index_add(0, groups, probs)),
        COEF[2] * torch.logsumexp(logits, 1).square().mean()])
    total = terms.sum()
    grad = torch.autograd.grad(total, logits)[0]
    dlogits = s["dlogits"].double().index_add(0, rows, UPSTREAM * grad)
    return dict(loss=torch.cat([total[None], terms]).detach(), probs=probs.detach(), counts=None,
                dlogits=dlogits)


def _exact_gate_back(s):
    dl = s["dlogits"].double()
    dx = torch.matmul(dl, s["w_router"].double())
    if s["dx_in"] is not None:
        dx += s["dx_in"].double()
    return dict(dx=dx, dw_router=torch.matmul(dl.t().contiguous(), s["x"].double()))


def _exact_adamw(t):
    a, n = ADAM, t["p"].numel()
    eight = t["m_scale"] is not None
    block = torch.arange(n, device="cuda") // BLOCK if eight else None
    m, v = t["m"].double(), t["v"].double()
    if eight:
        m, v = m * t["m_scale"].double()[block], (v * t["v_scale"].double()[block]) ** 2
    g = a["grad_scale"] * t["g"].double()
    m = m + (1 - a["beta1"]) * (g - m)
    v = v + (1 - a["beta2"]) * (g * g - v)
    m_hat, v_hat = m / (1 - a["beta1"] ** a["step"]), v / (1 - a["beta2"] ** a["step"])
    p = t["p"].double()
    p = p - a["lr"] * (m_hat / (v_hat.sqrt() + a["eps"]) + a["weight_decay"] * p)
    out = dict(p=p, m=m, v=v, m_scale=None, v_scale=None,
               copy=p if t["out"]["copy"] is not None else None)
    if eight:
        for key, value in (("m", m), ("v", v.sqrt())):
            unit = torch.zeros(t[key + "_scale"].numel(), dtype=torch.float64, device="cuda")
            unit = unit.scatter_reduce(0, block, value.abs(), "amax") / E4M3_MAX
            out[key + "_scale"], out[key] = unit, value / unit[block]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        return [_exact_adamw(t) for t in s["tensors"]]
    return dict(norm=_exact_norm, norm_back=_exact_norm_back, balance=_exact_balance,
                gate_back=_exact_gate_back)[op](s)
