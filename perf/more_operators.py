"""Cases of the layers around the experts: what is measured, and their plain forms.

Between the embeddings' interaction and the click's probability stand dense
layers, norms on a residual stream, and the gate that sends samples ("tokens")
to experts.  Three operators do that and its training step:

  dense    z = x W^T + bias,  y = act(z) + residual, for x [T, K], W [N, K]; act is
           none, relu, silu, gelu (by erf) or sigmoid.  Training keeps z ("pre", in
           the inputs' type) and gives, with dz = dy * act'(pre),
               dx = dz W,  dW = dz^T x,  dbias = sum over t of dz.
           bf16, or fp32 to fp32's accuracy.
  norm     s = x + residual, in the inputs' type: the stream's new value;
           v = s / sqrt(mean(s^2) + eps) * gamma;  y = v, or its e4m3 codes with a
           scale per row and 128 columns, which the 8-bit products read:
               scale = max(amax, 2^-100) / 448,
               code  = e4m3(v * (448 / max(amax, 2^-100))).
           Training gives dx, the gradient of s (and so of x and of the residual),
           which the gradient ds that arrives on the stream is added to, and dgamma.
  balance  routing with a bias for balance: p = softmax or sigmoid of the scores
           (-inf: masked), key = p + bias, compared as real numbers, ties to the
           lower index; the groups of experts with the largest sums of their two
           best keys stay, of these the k largest keys are chosen; weights are p
           (not key) of the choices, divided by their sum where renormalised.  Then the stable order by expert, as in routing without
           balance.  Training gives the scores' gradient, the choices held fixed.

Training cases of `dense` take smooth activations: where z is next to zero, relu's
derivative is 0 or 1 by the last bit of a sum.  `own` selects between the plain
forms (torch operations, fp32; keys in 64 bits) and the library's calls.
"""
import math

import torch

own = False

TINY = 2.0 ** -100
EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
ACTS = ["none", "relu", "silu", "gelu", "sigmoid"]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request's sample through the first layer above the interaction (479 wide): latency only
        dict(name="dense_one", op="dense", tokens=1, kdim=479, n=512, dtype="f32", act="relu", bias=True, residual=False,
             train=False),
        # a small serving batch through a hidden layer: bound by the weights
        dict(name="dense_serve", op="dense", tokens=64, kdim=1024, n=2048, dtype="bf16", act="gelu", bias=True,
             residual=False, train=False),
        # a large scoring batch through a residual layer: bound by the tensor cores
        dict(name="dense_score", op="dense", tokens=65536, kdim=1024, n=1024, dtype="bf16", act="silu", bias=True,
             residual=True, train=False),
        # a training step of the first layer on the 479-wide interaction output, fp32: odd widths
        dict(name="dense_train_odd", op="dense", tokens=16384, kdim=479, n=512, dtype="f32", act="gelu", bias=True,
             residual=False, train=True),
        # a training step of a hidden layer, bf16
        dict(name="dense_train", op="dense", tokens=32768, kdim=1024, n=2048, dtype="bf16", act="silu", bias=True,
             residual=True, train=True),
        # one sample's hidden vector, into codes for the next 8-bit product: latency only
        dict(name="norm_one", op="norm", tokens=1, d=1024, dtype="bf16", residual=True, out="codes", train=False),
        # a serving batch of interaction outputs, 479 wide: rows off 16 bytes
        dict(name="norm_serve", op="norm", tokens=2048, d=479, dtype="f32", residual=False, out="values", train=False),
        # a large scoring batch on the residual stream, into codes
        dict(name="norm_score", op="norm", tokens=65536, d=2048, dtype="bf16", residual=True, out="codes", train=False),
        # a training step of the norm on the residual stream
        dict(name="norm_train", op="norm", tokens=65536, d=1024, dtype="bf16", residual=True, out="values", train=True),
        # one request's sample through a 64-expert gate with groups: latency only
        dict(name="balance_one", op="balance", tokens=1, experts=64, groups=8, group_k=4, k=6, dtype="f32",
             score="sigmoid", bias=True, renorm=True, masked=0.0, train=False),
        # a serving batch without groups, some scores masked and some samples padding
        dict(name="balance_batch", op="balance", tokens=2048, experts=26, groups=1, group_k=1, k=4, dtype="f32",
             score="softmax", bias=True, renorm=False, masked=0.05, train=False),
        # a training batch over 256 experts in 8 groups
        dict(name="balance_train", op="balance", tokens=65536, experts=256, groups=8, group_k=4, k=8, dtype="bf16",
             score="sigmoid", bias=True, renorm=True, masked=0.0, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dense", "dense", "norm", "balance"])
    dtype = rng.choice(["f32", "bf16"])
    train = rng.random() < 0.5
    if op == "dense":
        return dict(op=op, tokens=_log(rng, 1, 30_000), kdim=_log(rng, 16, 1500), n=_log(rng, 16, 1500), dtype=dtype,
                    act=rng.choice(["none", "silu", "gelu", "sigmoid"] if train else ACTS), bias=rng.random() < 0.7,
                    residual=rng.random() < 0.5, train=train)
    if op == "norm":
        return dict(op=op, tokens=_log(rng, 1, 60_000), d=_log(rng, 16, 2048), dtype=dtype,
                    residual=rng.random() < 0.6, out="values" if train else rng.choice(["values", "codes"]),
                    train=train)
    groups = rng.choice([1, 1, 2, 4, 8])
    experts = groups * _log(rng, 2, 256 // groups)
    group_k = rng.randint(1, groups)
    k = rng.randint(1, min(8, group_k * (experts // groups)))
    return dict(op=op, tokens=_log(rng, 1, 60_000), experts=experts, groups=groups, group_k=group_k, k=k, dtype=dtype,
                score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.7, renorm=rng.random() < 0.5,
                masked=rng.choice([0.0, 0.05, 0.3]), train=train)


def work(c):
    T, b = c["tokens"], BYTES[c["dtype"]]
    if c["op"] == "dense":
        K, N = c["kdim"], c["n"]
        n = T * K * b + N * K * b + T * N * b
        n += N * b if c["bias"] else 0
        n += T * N * b if c["residual"] else 0
        if c["train"]:  # pre out; dy in, dx and dw out
            n += T * N * b + T * N * b + T * K * b + N * K * b + (N * b if c["bias"] else 0)
        return {"bytes": n, "flops": (6 if c["train"] else 2) * T * N * K}
    if c["op"] == "norm":
        d = c["d"]
        n = T * d * b + d * 4
        if c["residual"]:
            n += 2 * T * d * b
        n += T * d * b if c["out"] == "values" else T * d + T * -(-d // 128) * 4
        if c["train"]:  # dy and ds in, dx and dgamma out
            n += 3 * T * d * b + d * 4
        return {"bytes": n, "flops": T * d * (14 if c["train"] else 5)}
    E, k = c["experts"], c["k"]
    n = T * E * b + T * k * 16 + (E + 1) * 4 + (E * 4 if c["bias"] else 0)
    if c["train"]:
        n += T * k * 4 + T * E * b
    return {"bytes": n, "flops": T * E * (8 if c["train"] else 5)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])


def _vectors(g, rows, d, dtype):
    """Activations: columns of different sizes, as interaction outputs have."""
    col = torch.exp(0.5 * torch.randn((1, d), generator=g, device="cuda"))
    return (torch.randn((rows, d), generator=g, device="cuda") * col).to(DT[dtype])


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 23)
    st = {"case": c}
    T, dt = c["tokens"], c["dtype"]
    if c["op"] == "dense":
        K, N = c["kdim"], c["n"]
        st["x"] = _vectors(g, T, K, dt)
        st["w"] = _normal(g, (N, K), dt, 1.0 / math.sqrt(K))
        st["bias"] = _normal(g, (N,), dt, 0.5) if c["bias"] else None
        st["residual"] = _normal(g, (T, N), dt) if c["residual"] else None
        if c["train"]:
            st["dy"] = _normal(g, (T, N), dt, 1e-3)
    elif c["op"] == "norm":
        st["x"] = _vectors(g, T, c["d"], dt)
        st["residual"] = _vectors(g, T, c["d"], dt) if c["residual"] else None
        st["gamma"] = 1.0 + 0.2 * torch.randn((c["d"],), generator=g, device="cuda")
        if c["train"]:
            st["dy"] = _normal(g, (T, c["d"]), dt, 1e-3)
            st["ds"] = _normal(g, (T, c["d"]), dt, 1e-3)
    else:
        E = c["experts"]
        s = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
        if c["masked"]:
            s[torch.rand((T, E), generator=g, device="cuda") < c["masked"]] = -math.inf
            s[torch.rand((T,), generator=g, device="cuda") < c["masked"] / 4] = -math.inf
        st["scores"] = s.to(DT[dt])
        st["bias"] = 0.05 * torch.randn((E,), generator=g, device="cuda") if c["bias"] else None
        if c["train"]:
            st["dweight"] = torch.randn((T, c["k"]), generator=g, device="cuda")
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "sigmoid":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 - s)
    return torch.ones_like(z)


def _dense_plain(st):
    c, dt = st["case"], DT[st["case"]["dtype"]]
    x, w = st["x"].float(), st["w"].float()
    z = x @ w.t()
    if st["bias"] is not None:
        z = z + st["bias"].float()
    y = _act(z, c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    if not c["train"]:
        return y.to(dt)
    pre = z.to(dt)
    dz = st["dy"].float() * _act_grad(pre.float(), c["act"])
    out = {"y": y.to(dt), "pre": pre, "dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt)}
    if st["bias"] is not None:
        out["dbias"] = dz.sum(0).to(dt)
    return out


def _codes_plain(v):
    """(codes, scales by block) of the rows of v, one scale per row and 128 columns."""
    T, d = v.shape
    p = torch.nn.functional.pad(v, (0, -d % 128)).view(T, -1, 128)
    top = torch.full((1,), 448.0, device=v.device)
    amax = p.abs().amax(2, keepdim=True).clamp(min=TINY)
    q = (p * torch.div(top, amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(T, -1), torch.div(amax, top)[:, :, 0].t().contiguous()


def _norm_plain(st):
    c, dt = st["case"], DT[st["case"]["dtype"]]
    s = st["x"]
    if st["residual"] is not None:
        s = (s.float() + st["residual"].float()).to(dt)
    f = s.float()
    rstd = 1 / torch.sqrt(f.square().mean(1, keepdim=True) + EPS)
    v = f * rstd * st["gamma"]
    out = {"s": s} if st["residual"] is not None else {}
    if c["out"] == "codes":
        out["codes"], out["scale"] = _codes_plain(v)
        return out
    out["y"] = v.to(dt)
    if c["train"]:
        dy = st["dy"].float()
        g = dy * st["gamma"]
        out["dx"] = (st["ds"].float() + rstd * (g - f * rstd.square() * (g * f).mean(1, keepdim=True))).to(dt)
        out["dgamma"] = (dy * f * rstd).sum(0)
    return out


def _balance_plain(st):
    c = st["case"]
    T, E, k, G = c["tokens"], c["experts"], c["k"], c["groups"]
    wide, dev = st["scores"].double(), st["scores"].device  # keys next to each other are told apart in 64 bits
    live = wide > -math.inf
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-wide))
    else:
        m = torch.where(live, wide, -1e300).amax(1, keepdim=True)
        e = torch.where(live, torch.exp(wide - m), 0.0)
        total = e.sum(1, keepdim=True)
        p = e / torch.where(total > 0, total, 1.0)
    key = torch.where(live, p + (st["bias"].double() if st["bias"] is not None else 0.0), -math.inf)
    if c["group_k"] < G:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values[:, :, :2]
        some = best[:, :, 0] > -math.inf
        total = torch.where(some, torch.where(best > -math.inf, best, 0.0).sum(2), -math.inf)
        pick = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :c["group_k"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=dev).scatter_(1, pick, True)
        key = torch.where(kept.repeat_interleave(E // G, 1), key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    top, choice = order.values[:, :k], order.indices[:, :k]
    has = top > -math.inf
    weight = torch.where(has, torch.gather(p, 1, choice), 0.0).float()
    if c["renorm"]:
        total = weight.sum(1, keepdim=True)
        weight = weight / torch.where(total > 0, total, 1.0)
    expert = torch.where(has, choice, -1)
    flat = torch.where(has, choice, E).reshape(-1)
    pos = torch.sort(flat, stable=True).indices
    rank = torch.empty_like(pos)
    rank[pos] = torch.arange(T * k, device=dev)
    slot = torch.where(has, rank.view(T, k), -1)
    offsets = torch.searchsorted(flat[pos], torch.arange(E + 1, device=dev))
    token = torch.where(torch.arange(T * k, device=dev) < offsets[E], pos // k, -1)
    i32 = torch.int32
    out = {"expert": expert.to(i32), "weight": weight, "slot": slot.to(i32), "token": token.to(i32),
           "offsets": offsets.to(i32)}
    if c["train"]:
        s = st["scores"].float()
        at = torch.where(has, choice, 0)
        g = torch.where(has, st["dweight"], 0.0)
        if c["renorm"]:
            d = weight * (g - (g * weight).sum(1, keepdim=True))
            if c["score"] == "sigmoid":
                d = d / (1 + torch.exp(torch.gather(s, 1, at)))
        elif c["score"] == "sigmoid":
            d = g * weight / (1 + torch.exp(torch.gather(s, 1, at)))
        else:
            full = torch.zeros_like(s).scatter_add_(1, at, g)
            q = p.float()
            out["dscores"] = (q * (full - (g * weight).sum(1, keepdim=True))).to(st["scores"].dtype)
            return out
        d = torch.where(has, d, 0.0)
        out["dscores"] = torch.zeros_like(s).scatter_add_(1, at, d).to(st["scores"].dtype)
    return out


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _buffers(st):
    """Output buffers and workspaces that a program keeps from call to call."""
    from sparse_embeddings_feature_gb300 import ctr
    c, b = st["case"], {}
    T = c["tokens"]
    if c["op"] == "dense":
        b["y"] = torch.empty((T, c["n"]), dtype=st["x"].dtype, device="cuda")
        b["pre"] = torch.empty_like(b["y"]) if c["train"] else None
        b["act"] = ctr.ACTIVATIONS[c["act"]]
        b["ws"] = ctr.workspace(ctr.ctr_dense_workspace_size(T, c["n"], c["kdim"], st["x"].dtype, c["train"]))
        if c["train"]:
            b["dx"], b["dw"] = torch.empty_like(st["x"]), torch.empty_like(st["w"])
            b["dbias"] = torch.empty_like(st["bias"]) if c["bias"] else None
    elif c["op"] == "norm":
        b["s"] = torch.empty_like(st["x"]) if c["residual"] else None
        b["y"] = torch.empty_like(st["x"]) if c["out"] == "values" else None
        b["q"] = b["scale"] = None
        if c["out"] == "codes":
            b["q"] = torch.empty((T, ctr.fp8_padded(c["d"])), dtype=torch.uint8, device="cuda")
            b["scale"] = torch.empty((ctr.fp8_blocks(c["d"]), T), device="cuda")
        b["ws"] = ctr.workspace(ctr.ctr_rms_norm_workspace_size(T, c["d"]))
        if c["train"]:
            b["dx"], b["dgamma"] = torch.empty_like(st["x"]), torch.empty_like(st["gamma"])
    else:
        E, k = c["experts"], c["k"]
        i32 = dict(dtype=torch.int32, device="cuda")
        b.update(expert=torch.empty((T, k), **i32), weight=torch.empty((T, k), device="cuda"),
                 slot=torch.empty((T, k), **i32), token=torch.empty((T * k,), **i32),
                 offsets=torch.empty((E + 1,), **i32), score=ctr.SCORES[c["score"]],
                 ws=ctr.workspace(ctr.ctr_expert_route_workspace_size(T, E, k)))
        if c["train"]:
            b["dscores"] = torch.empty_like(st["scores"])
    st["buffers"] = b
    return b


def _run_own(st):
    from sparse_embeddings_feature_gb300 import ctr
    c, b = st["case"], st.get("buffers") or _buffers(st)
    if c["op"] == "dense":
        ctr.ctr_dense(st["x"], st["w"], st["bias"], b["act"], st["residual"], b["y"], b["pre"], b["ws"])
        if not c["train"]:
            return b["y"]
        ctr.ctr_dense_bwd(st["dy"], st["x"], st["w"], b["pre"], b["act"], b["dx"], b["dw"], b["dbias"], b["ws"])
        out = {n: b[n] for n in ("y", "pre", "dx", "dw")}
        return {**out, "dbias": b["dbias"]} if c["bias"] else out
    if c["op"] == "norm":
        ctr.ctr_rms_norm(st["x"], st["residual"], st["gamma"], EPS, b["s"], b["y"], b["q"], b["scale"], b["ws"])
        out = {"s": b["s"]} if c["residual"] else {}
        if c["out"] == "codes":
            out["codes"], out["scale"] = b["q"].view(torch.float8_e4m3fn), b["scale"]
            return out
        out["y"] = b["y"]
        if c["train"]:
            ctr.ctr_rms_norm_bwd(st["dy"], st["ds"], b["s"] if c["residual"] else st["x"], st["gamma"], EPS, b["dx"],
                                 b["dgamma"], b["ws"])
            out.update(dx=b["dx"], dgamma=b["dgamma"])
        return out
    ctr.ctr_expert_route_balanced(st["scores"], c["k"], b["score"], st["bias"], c["groups"], c["group_k"], c["renorm"],
                                  1.0, b["expert"], b["weight"], b["slot"], b["token"], b["offsets"], b["ws"])
    out = {n: b[n] for n in ("expert", "weight", "slot", "token", "offsets")}
    if c["train"]:
        ctr.ctr_expert_route_balanced_bwd(st["dweight"], st["scores"], b["score"], c["renorm"], 1.0, b["expert"],
                                          b["dscores"], b["ws"])
        out["dscores"] = b["dscores"]
    return out


def run(st):
    if own:
        return _run_own(st)
    return {"dense": _dense_plain, "norm": _norm_plain, "balance": _balance_plain}[st["case"]["op"]](st)


# ---------------------------------------------------------------------------
# 64-bit values, written apart from the plain forms
# ---------------------------------------------------------------------------
def _e4m3(v):
    """The e4m3 value nearest to v (fp64; ties to even): 3 mantissa bits, steps of 2^-9 below 2^-6."""
    a = v.abs().clamp(max=448.0)
    ex = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(ex - 3)
    return torch.sign(v) * torch.round(a / step) * step


def _exact_dense(c, st):
    one = {"none": lambda z: (z, torch.ones_like(z)),
           "relu": lambda z: (z.clamp(min=0.0), (z > 0).double()),
           "sigmoid": lambda z: (torch.sigmoid(z), torch.sigmoid(z) * torch.sigmoid(-z)),
           "silu": lambda z: (z * torch.sigmoid(z), torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)),
           "gelu": lambda z: (z * torch.special.ndtr(z),
                              torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))}[c["act"]]
    x, w = st["x"].double(), st["w"].double()
    z = torch.einsum("tk,nk->tn", x, w)
    if st["bias"] is not None:
        z += st["bias"].double()[None, :]
    y = one(z)[0]
    if st["residual"] is not None:
        y = y + st["residual"].double()
    if not c["train"]:
        return y
    kept = z.to(DT[c["dtype"]]).double()
    dz = st["dy"].double() * one(kept)[1]
    out = {"y": y, "pre": z, "dx": torch.einsum("tn,nk->tk", dz, w), "dw": torch.einsum("tn,tk->nk", dz, x)}
    if st["bias"] is not None:
        out["dbias"] = torch.einsum("tn->n", dz)
    return out


def _exact_norm(c, st):
    x, gamma = st["x"].double(), st["gamma"].double()
    out = {}
    if st["residual"] is not None:
        x = (x + st["residual"].double()).to(DT[c["dtype"]]).double()
        out["s"] = x
    n = c["d"]
    r = torch.rsqrt(torch.einsum("td,td->t", x, x) / n + EPS)[:, None]
    unit = x * r
    v = unit * gamma
    if c["out"] == "codes":
        parts = [v[:, i:i + 128] for i in range(0, n, 128)]
        tops = [p.abs().max(1, keepdim=True).values.clamp(min=TINY) for p in parts]
        codes = torch.zeros((c["tokens"], len(parts) * 128), dtype=torch.float64, device=x.device)
        codes[:, :n] = torch.cat([_e4m3(p * (448.0 / t)) for p, t in zip(parts, tops)], 1)
        out["codes"], out["scale"] = codes, torch.cat(tops, 1).T / 448.0
        return out
    out["y"] = v
    if c["train"]:
        dy = st["dy"].double()
        du = dy * gamma
        # d(x r)/dx: r (I - unit unit^T / n)
        out["dx"] = st["ds"].double() + r * (du - unit * (torch.einsum("td,td->t", du, unit) / n)[:, None])
        out["dgamma"] = torch.einsum("td,td->d", dy, unit)
    return out


def _exact_balance(c, st):
    import numpy as np
    s = st["scores"].double().cpu().numpy()
    T, E, k, G = c["tokens"], c["experts"], c["k"], c["groups"]
    live = np.isfinite(s)
    if c["score"] == "sigmoid":
        z = np.exp(-np.abs(s))
        p = np.where(live, np.where(s >= 0, 1 / (1 + z), z / (1 + z)), 0.0)
    else:
        m = np.where(live.any(1), np.max(s, axis=1), 0.0)[:, None]
        z = np.where(live, np.exp(s - m), 0.0)
        p = z / np.maximum(z.sum(1, keepdims=True), 1e-300)
    key = p + (0.0 if st["bias"] is None else st["bias"].double().cpu().numpy()[None, :])
    key = np.where(live, key, -np.inf)
    rows = np.arange(T)[:, None]
    if c["group_k"] < G:
        members = key.reshape(T, G, -1)
        two = -np.partition(-members, 1, axis=2)[:, :, :2] if members.shape[2] > 2 else members
        worth = np.where(np.isfinite(two), two, 0.0).sum(2)
        worth = np.where(np.isfinite(two).any(2), worth, -np.inf)
        stays = np.zeros((T, G), dtype=bool)
        stays[rows, np.argsort(-worth, axis=1, kind="stable")[:, :c["group_k"]]] = True
        key = np.where(stays[:, np.arange(E) // (E // G)], key, -np.inf)
    choice = np.argsort(-key, axis=1, kind="stable")[:, :k]
    has = np.isfinite(key[rows, choice])
    picked = np.where(has, p[rows, choice], 0.0)
    total = picked.sum(1, keepdims=True)
    weight = picked / np.where(total > 0, total, 1.0) if c["renorm"] else picked
    flat = np.where(has, choice, E).ravel()
    order = np.argsort(flat, kind="stable")
    count = int(has.sum())
    slot = np.full(T * k, -1, dtype=np.int32)
    slot[order[:count]] = np.arange(count)
    token = np.full(T * k, -1, dtype=np.int32)
    token[:count] = order[:count] // k
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])]).astype(np.int32)
    out = {"expert": np.where(has, choice, -1).astype(np.int32), "weight": weight, "slot": slot.reshape(T, k),
           "token": token, "offsets": offsets}
    if c["train"]:
        g = np.where(has, st["dweight"].double().cpu().numpy(), 0.0)
        d = np.zeros((T, E))
        if c["score"] == "sigmoid":
            # d ln p / d score = 1 - p
            slope = 1 - p[rows, choice]
            inner = weight * (g - (weight * g).sum(1, keepdims=True)) if c["renorm"] else weight * g
            d[rows, choice] = np.where(has, inner * slope, 0.0)
        else:
            over = np.zeros((T, E))
            over[rows, choice] = np.where(has, weight, 0.0)
            base = over if c["renorm"] else p
            up = np.zeros((T, E))
            up[rows, choice] = g
            d = base * (up - (weight * g).sum(1, keepdims=True))
        out["dscores"] = d
    return out


def exact(c, seed):
    st = prepare(c, seed)
    return {"dense": _exact_dense, "norm": _exact_norm, "balance": _exact_balance}[c["op"]](c, st)
