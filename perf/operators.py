"""Cases of the expert layer's operators: what is measured, and their plain forms.

A mixture of experts on top of the interaction output sends every sample
("token") to its k best experts, multiplies the samples of each expert with
that expert's weight matrix, and adds the k results up under the router's
weights.  Four operators do that and its training step:

  route    scores [T, E] -> the k best experts of each token (ties to the lowest
           index; scores of -inf are masked), their softmax weights, and the
           stable order by expert: slot[t, j] is the sorted row of token t's
           j-th choice, token[r] the token of sorted row r, offsets[e] the
           first row of expert e.  Backward: the scores' gradient.
  rows     tokens copied into expert order, and results added back under the
           weights; backward: the gradient of every row, of every weight, and of
           the tokens.
  product  out[r] = W_g x[token[r]] for the rows r of each group g, in e4m3 with
           a scale for each block of 128: activations have one scale per row and
           128 columns, weights one per 128 x 128 block,
               scale = max(amax, 2^-100) / 448,
               code  = e4m3(x * (448 / max(amax, 2^-100))),
           in fp32 arithmetic; products and sums are of the values that the codes
           stand for.  Training also gives dx = dy W (dy quantised like x, the
           blocks of W transposed) and dW_g = dy_g^T x_g, where dy has one scale
           per column and 128 rows of the group, and x one per 128 x 128 block.
  clip     the global norm over many gradient tensors, and the gradients times
           min(1, max_norm / norm).

`own` selects between the plain forms (torch operations, fp32) and the
library's calls.
"""
import math

import torch

own = False

TINY = 2.0 ** -100
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request's sample through an 8-expert router: latency only
        dict(name="route_one", op="route", tokens=1, experts=8, k=2, dtype="f32", renorm=True, masked=0.0, train=False),
        # a serving batch of 2048, some scores masked and some samples padding
        dict(name="route_batch", op="route", tokens=2048, experts=26, k=4, dtype="f32", renorm=False, masked=0.05,
             train=False),
        # the training batch of 131072 samples, forward and backward
        dict(name="route_train", op="route", tokens=131072, experts=64, k=4, dtype="bf16", renorm=True, masked=0.02,
             train=True),
        # a small serving batch of interaction outputs (351 products + 128 dense), sorted and back
        dict(name="rows_serve", op="rows", tokens=64, d=479, experts=8, k=2, dtype="f32", train=False),
        # a training batch of hidden vectors, sorted and back, with every gradient
        dict(name="rows_train", op="rows", tokens=65536, d=1024, experts=32, k=2, dtype="bf16", train=True),
        # a single sample through one layer: latency, and a K that ends inside a block
        dict(name="product_one", op="product", tokens=1, k=1, experts=1, n=1024, kdim=479, dtype="bf16", out="bf16",
             train=False),
        # a small serving batch over 16 experts: a few rows each, bound by the weights
        dict(name="product_serve", op="product", tokens=64, k=2, experts=16, n=2048, kdim=1024, dtype="bf16",
             out="bf16", train=False),
        # one dense layer over a large scoring batch: bound by the tensor cores
        dict(name="product_dense", op="product", tokens=16384, k=1, experts=1, n=4096, kdim=4096, dtype="bf16",
             out="bf16", train=False),
        # a training step of 16 experts on the 479-wide interaction output: odd widths, ragged groups
        dict(name="product_train_odd", op="product", tokens=16384, k=2, experts=16, n=512, kdim=479, dtype="f32",
             out="f32", train=True),
        # a training step of 32 experts on hidden vectors
        dict(name="product_train", op="product", tokens=32768, k=2, experts=32, n=2048, kdim=1024, dtype="bf16",
             out="bf16", train=True),
        # the gradients of a small ranking net's layers: latency; the norm stays under the bound
        dict(name="clip_small", op="clip", tensors=12, numel=60_000, dtype="f32", max_norm=1.0),
        # the gradients of a large dense net, half of the tensors bf16: clipped
        dict(name="clip_large", op="clip", tensors=48, numel=500_000_000, dtype="mixed", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "rows", "product", "product", "clip"])
    dtype = rng.choice(["f32", "bf16"])
    train = rng.random() < 0.5
    if op == "route":
        experts = _log(rng, 2, 200)
        return dict(op=op, tokens=_log(rng, 1, 120_000), experts=min(experts, 64) if train else experts,
                    k=rng.randint(1, min(4, experts)), dtype=dtype, renorm=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.05, 0.3]), train=train)
    if op == "rows":
        tokens = _log(rng, 1, 40_000)
        return dict(op=op, tokens=tokens, d=_log(rng, 16, 1000), experts=_log(rng, 2, 64), k=rng.randint(1, 2),
                    dtype=dtype, train=train)
    if op == "product":
        experts = rng.choice([1, _log(rng, 2, 32)])
        return dict(op=op, tokens=_log(rng, 1, 16_000), k=1 if experts == 1 else 2, experts=experts,
                    n=_log(rng, 64, 2000), kdim=_log(rng, 64, 2000), dtype=dtype, out=rng.choice(["f32", "bf16"]),
                    train=train)
    return dict(op=op, tensors=_log(rng, 1, 60), numel=_log(rng, 10_000, 300_000_000),
                dtype=rng.choice(["f32", "bf16", "mixed"]), max_norm=rng.choice([0.1, 1.0]))


def work(c):
    if c["op"] == "route":
        T, E, k, b = c["tokens"], c["experts"], c["k"], BYTES[c["dtype"]]
        n = T * E * b + T * k * 16 + (E + 1) * 4
        if c["train"]:
            n += T * k * 4 + T * E * b
        return {"bytes": n, "flops": T * E * (6 if c["train"] else 3)}
    if c["op"] == "rows":
        T, d, k, b = c["tokens"], c["d"], c["k"], BYTES[c["dtype"]]
        # sorted copy: x in, k rows out; sum: k rows in, y out
        n = 2 * (T * d * b + T * k * d * b) + T * k * 12
        if c["train"]:  # dy and ys in, dys and dw out; dxs in, dx out
            n += T * d * b + 2 * T * k * d * b + T * k * d * b + T * d * b + T * k * 4
        return {"bytes": n, "flops": 2 * T * k * d * (4 if c["train"] else 1)}
    if c["op"] == "product":
        T, R, G, N, K = c["tokens"], c["tokens"] * c["k"], c["experts"], c["n"], c["kdim"]
        b, o = BYTES[c["dtype"]], BYTES[c["out"]]
        if not c["train"]:
            used = min(G, R)
            return {"bytes": T * K * b + used * N * K + R * N * o, "flops": 2 * R * N * K}
        return {"bytes": T * K * b + G * N * K * b + R * N * o + R * N * b + R * K * o + G * N * K * 4,
                "flops": 6 * R * N * K}
    n = sum(s * BYTES[dt] for s, dt in _clip_shapes(c))
    return {"bytes": 2 * n, "flops": 3 * c["numel"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])


def _vectors(g, rows, d, dtype):
    """Activations: columns of different sizes and a few large values, as interaction outputs have."""
    col = torch.exp(torch.randn((1, d), generator=g, device="cuda"))
    return (torch.randn((rows, d), generator=g, device="cuda") * col).to(DT[dtype])


def _scores(c, g):
    """Router scores: some experts are liked more; a share of the scores and of the samples is masked."""
    T, E = c["tokens"], c["experts"]
    s = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    if c.get("masked", 0.0):
        s[torch.rand((T, E), generator=g, device="cuda") < c["masked"]] = -math.inf
        s[torch.rand((T,), generator=g, device="cuda") < c["masked"] / 4] = -math.inf
    return s.to(DT[c["dtype"]])


def _routing(c, g):
    """A routing in hand: (expert, weight, slot, token, offsets), every token sent to its k experts."""
    s = _scores(dict(c, dtype="f32"), g)
    return _route_plain(s, c["k"], True)


def _clip_shapes(c):
    """The tensors' element counts and types: layers of falling size, every third a short vector."""
    n, total = c["tensors"], c["numel"]
    share = [1.0 / (i + 2) if i % 3 else 0.0005 for i in range(n)]
    unit = total / sum(share)
    kinds = ["f32", "bf16"] if c["dtype"] == "mixed" else [c["dtype"]]
    return [(max(1, int(share[i] * unit)), kinds[i % len(kinds)]) for i in range(n)]


def prepare(c, seed):
    g = _gen(seed)
    st = {"case": c}
    if c["op"] == "route":
        st["scores"] = _scores(c, g)
        if c["train"]:
            st["dweight"] = torch.randn((c["tokens"], c["k"]), generator=g, device="cuda")
    elif c["op"] == "rows":
        T, R, d = c["tokens"], c["tokens"] * c["k"], c["d"]
        _, st["weight"], st["slot"], st["token"], _ = _routing(c, g)
        st["x"] = _vectors(g, T, d, c["dtype"])
        st["ys"] = _normal(g, (R, d), c["dtype"])
        if c["train"]:
            st["dy"] = _normal(g, (T, d), c["dtype"])
            st["dxs"] = _normal(g, (R, d), c["dtype"])
    elif c["op"] == "product":
        T, R, G, N, K = c["tokens"], c["tokens"] * c["k"], c["experts"], c["n"], c["kdim"]
        if G > 1:
            _, _, _, st["token"], st["offsets"] = _routing(c, g)
        else:
            st["token"] = None
            st["offsets"] = torch.tensor([0, R], dtype=torch.int32, device="cuda")
        st["cap"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
        st["x"] = _vectors(g, T, K, c["dtype"])
        w = _normal(g, (G, N, K), c["dtype"], 1.0 / math.sqrt(K))
        if c["train"]:
            st["w"] = w
            st["dy"] = _normal(g, (R, N), c["dtype"], 1e-3)
        else:  # weights laid out once
            st["wq"], st["ws"] = _blocks_plain(w.float())
    else:
        st["grads"] = [_normal(g, (s,), dt, 1e-3) for s, dt in _clip_shapes(c)]
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _route_plain(s, k, renorm):
    T, E = s.shape
    s = s.float()
    order = torch.sort(s, dim=1, descending=True, stable=True)
    top, expert = order.values[:, :k], order.indices[:, :k]
    live = top > -math.inf
    m = torch.where(live[:, :1], top[:, :1], 0.0)
    e = torch.where(live, torch.exp(top - m), 0.0)
    total = e.sum(1, keepdim=True) if renorm else torch.exp(s - m).sum(1, keepdim=True)
    weight = torch.where(live, e / torch.where(total > 0, total, 1.0), 0.0)
    expert = torch.where(live, expert, -1)
    key = torch.where(live, expert, E).reshape(-1)
    pos = torch.sort(key, stable=True).indices
    rank = torch.empty_like(pos)
    rank[pos] = torch.arange(T * k, device=s.device)
    slot = torch.where(live, rank.view(T, k), -1)
    offsets = torch.searchsorted(key[pos], torch.arange(E + 1, device=s.device))
    token = torch.where(torch.arange(T * k, device=s.device) < offsets[E], pos // k, -1)
    i32 = torch.int32
    return expert.to(i32), weight, slot.to(i32), token.to(i32), offsets.to(i32)


def _route_grad_plain(dw, s, k, renorm):
    x = s.float()
    expert, weight = _route_plain(s, k, renorm)[:2]
    live = expert >= 0
    at = torch.where(live, expert, 0).long()
    gsel = torch.where(live, dw, 0.0)
    if renorm:
        d = weight * (gsel - (gsel * weight).sum(1, keepdim=True))
        return torch.zeros_like(x).scatter_add_(1, at, torch.where(live, d, 0.0)).to(s.dtype)
    m = x.max(1, keepdim=True).values
    e = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    total = e.sum(1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    full = torch.zeros_like(x).scatter_add_(1, at, gsel)
    return (p * (full - (gsel * weight).sum(1, keepdim=True))).to(s.dtype)


def _rounded(x, amax):
    """(values of the codes, scales) of x under the largest magnitudes amax (broadcast)."""
    top = torch.full((1,), 448.0, device=x.device)
    amax = amax.clamp(min=TINY)
    q = (x * torch.div(top, amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q, torch.div(amax, top)


def _pad128(x):
    r, c = -x.shape[-2] % 128, -x.shape[-1] % 128
    return torch.nn.functional.pad(x, (0, c, 0, r)) if r or c else x


def _rows_plain(x):
    """x [R, K] fp32 -> the values that its codes stand for, one scale per row and 128 columns."""
    R, K = x.shape
    p = torch.nn.functional.pad(x, (0, -K % 128)).view(R, -1, 128)
    q, s = _rounded(p, p.abs().amax(2, keepdim=True))
    return (q.float() * s).view(R, -1)[:, :K]


def _blocks_plain(w):
    """w [G, N, K] fp32 -> codes [G, N, K128] and scales [G, N/128, K/128], one per 128 x 128 block."""
    G, N, _ = w.shape
    p = _pad128(w)
    p = p.view(G, p.shape[1] // 128, 128, p.shape[2] // 128, 128)
    q, s = _rounded(p, p.abs().amax((2, 4), keepdim=True))
    q = q.reshape(G, p.shape[1] * 128, -1)[:, :N].contiguous()
    return q.view(torch.uint8), s[:, :, 0, :, 0].contiguous()


def _value_plain(q, s, K):
    """What block codes stand for, fp32 [G, N, K]."""
    N = q.shape[1]
    s = s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)
    return (q.view(torch.float8_e4m3fn).float() * s)[:, :, :K]


def _columns_plain(x, per_column):
    """x [G, C, D] fp32, groups' rows padded with zeros to C (a multiple of 128): the values of its
    codes with one scale per 128 rows and column, or per 128 rows and 128 columns."""
    G, C, D = x.shape
    p = torch.nn.functional.pad(x, (0, -D % 128)).view(G, C // 128, 128, -1, 128)
    q, s = _rounded(p, p.abs().amax(2 if per_column else (2, 4), keepdim=True))
    return (q.float() * s).view(G, C, -1)[:, :, :D]


def _placed(st, R):
    """(group, place in the group) of each sorted row."""
    r = torch.arange(R, device="cuda")
    off = st["offsets"].long()
    g = torch.searchsorted(off[1:], r, right=True)
    return g, r - off[g]


def _grouped_plain(x, w, g, at, cap):
    """x [R, K] times w[g] [N, K] by group: one batched product over groups padded to cap rows."""
    p = torch.zeros((w.shape[0], cap, x.shape[1]), device=x.device)
    p[g, at] = x
    return torch.bmm(p, w.transpose(1, 2))[g, at]


def _product_plain(st):
    c = st["case"]
    K, out = c["kdim"], DT[c["out"]]
    x = st["x"].float()
    x = x if st["token"] is None else x[st["token"].long()]
    g, at = _placed(st, x.shape[0])
    if not c["train"]:
        return _grouped_plain(_rows_plain(x), _value_plain(st["wq"], st["ws"], K), g, at, st["cap"]).to(out)
    dy = st["dy"].float()
    w = _value_plain(*_blocks_plain(st["w"].float()), K)
    y = _grouped_plain(_rows_plain(x), w, g, at, st["cap"])
    dx = _grouped_plain(_rows_plain(dy), w.transpose(1, 2), g, at, st["cap"])
    cap = (st["cap"] + 127) // 128 * 128
    xp = torch.zeros((w.shape[0], cap, K), device="cuda")
    xp[g, at] = x
    dp = torch.zeros((w.shape[0], cap, c["n"]), device="cuda")
    dp[g, at] = dy
    dw = torch.bmm(_columns_plain(dp, True).transpose(1, 2), _columns_plain(xp, False))
    return {"y": y.to(out), "dx": dx.to(out), "dw": dw}


def _rows_op_plain(st):
    c = st["case"]
    dt = DT[c["dtype"]]
    slot, token, weight = st["slot"].long(), st["token"].long(), st["weight"]
    ys = st["ys"].float()[slot]
    out = {"xs": st["x"][token], "y": (ys * weight[:, :, None]).sum(1).to(dt)}
    if c["train"]:
        dy = st["dy"].float()
        dys = torch.empty_like(st["ys"])
        dys[slot] = (dy[:, None, :] * weight[:, :, None]).to(dt)
        out["dys"] = dys
        out["dweight"] = (ys * dy[:, None, :]).sum(2)
        out["dx"] = st["dxs"].float()[slot].sum(1).to(dt)
    return out


def _clip_plain(st):
    grads, top = st["grads"], st["case"]["max_norm"]
    flat = torch.cat([x.float() for x in grads])
    norm = flat.square().sum().sqrt()
    flat = flat * torch.where(norm > top, top / norm, 1.0)
    parts = torch.split(flat, [x.numel() for x in grads])
    return {"norm": norm, "grads": [p.to(x.dtype) for p, x in zip(parts, grads)]}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def _f32(*shape):
    return torch.empty(shape, dtype=torch.float32, device="cuda")


def _u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def _buffers(st):
    """Output buffers and workspaces that a program keeps from call to call."""
    from sparse_embeddings_feature_gb300 import ctr
    c, b = st["case"], {}
    if c["op"] == "route":
        T, E, k = c["tokens"], c["experts"], c["k"]
        b.update(expert=_i32(T, k), weight=_f32(T, k), slot=_i32(T, k), token=_i32(T * k), offsets=_i32(E + 1),
                 ws=ctr.workspace(ctr.ctr_expert_route_workspace_size(T, E, k)))
        if c["train"]:
            b["dscores"] = torch.empty_like(st["scores"])
    elif c["op"] == "rows":
        b.update(xs=torch.empty_like(st["ys"]), y=torch.empty_like(st["x"]),
                 ws=ctr.workspace(ctr.ctr_expert_workspace_size()))
        if c["train"]:
            b.update(dys=torch.empty_like(st["ys"]), dweight=torch.empty_like(st["weight"]),
                     dx=torch.empty_like(st["x"]))
    elif c["op"] == "product":
        R, G, N, K = c["tokens"] * c["k"], c["experts"], c["n"], c["kdim"]
        Kp, Np, kb, nb = ctr.fp8_padded(K), ctr.fp8_padded(N), ctr.fp8_blocks(K), ctr.fp8_blocks(N)
        out = DT[c["out"]]
        b.update(xq=_u8(R, Kp), xs=_f32(kb, R), y=torch.empty((R, N), dtype=out, device="cuda"),
                 ws=ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(R, G, N, K)))
        if c["train"]:
            Rp = ctr.fp8_padded_rows(R, G)
            b.update(wq=_u8(G, N, Kp), wsc=_f32(G, nb, kb), wtq=_u8(G, K, Np), wts=_f32(G, kb, nb),
                     xcq=_u8(K, Rp), xcs=_f32(kb, Rp // 128), dq=_u8(R, Np), ds=_f32(nb, R), dcq=_u8(N, Rp),
                     dcs=_f32(Rp // 128, N), dx=torch.empty((R, K), dtype=out, device="cuda"), dw=_f32(G, N, K),
                     ws2=ctr.workspace(ctr.ctr_fp8_matmul_workspace_size(R, G, K, N)))
    else:
        outs = [torch.empty_like(x) for x in st["grads"]]
        b.update(outs=outs, list=ctr.grad_list(st["grads"], outs), norm=_f32(1),
                 ws=ctr.workspace(ctr.ctr_clip_grads_workspace_size()))
    st["buffers"] = b
    return b


def _run_own(st):
    from sparse_embeddings_feature_gb300 import ctr
    c, b = st["case"], st.get("buffers") or _buffers(st)
    if c["op"] == "route":
        ctr.ctr_expert_route(st["scores"], c["k"], c["renorm"], b["expert"], b["weight"], b["slot"], b["token"],
                             b["offsets"], b["ws"])
        out = {n: b[n] for n in ("expert", "weight", "slot", "token", "offsets")}
        if c["train"]:
            ctr.ctr_expert_route_bwd(st["dweight"], st["scores"], c["renorm"], b["expert"], b["dscores"], b["ws"])
            out["dscores"] = b["dscores"]
        return out
    if c["op"] == "rows":
        ctr.ctr_expert_dispatch(st["x"], st["slot"], st["token"], b["xs"], b["ws"])
        ctr.ctr_expert_combine(st["ys"], st["slot"], st["weight"], b["y"], b["ws"])
        out = {"xs": b["xs"], "y": b["y"]}
        if c["train"]:
            ctr.ctr_expert_combine_bwd(st["dy"], st["ys"], st["slot"], st["weight"], st["token"], b["dys"],
                                       b["dweight"], b["ws"])
            ctr.ctr_expert_combine(st["dxs"], st["slot"], None, b["dx"], b["ws"])
            out.update(dys=b["dys"], dweight=b["dweight"], dx=b["dx"])
        return out
    if c["op"] == "product":
        off = st["offsets"]
        if not c["train"]:
            ctr.ctr_fp8_quantize_rows(st["x"], b["xq"], b["xs"], b["ws"], row_index=st["token"])
            ctr.ctr_fp8_matmul(b["xq"], b["xs"], st["wq"], st["ws"], off, b["y"], b["ws"])
            return b["y"]
        ctr.ctr_fp8_quantize_rows_cols(st["x"], off, b["xq"], b["xs"], b["xcq"], b["xcs"], ctr.FP8_COLS_BY_BLOCK,
                                       b["ws"], row_index=st["token"])
        ctr.ctr_fp8_quantize_blocks(st["w"], b["wq"], b["wsc"], b["ws"], b["wtq"], b["wts"])
        ctr.ctr_fp8_matmul(b["xq"], b["xs"], b["wq"], b["wsc"], off, b["y"], b["ws"])
        ctr.ctr_fp8_quantize_rows_cols(st["dy"], off, b["dq"], b["ds"], b["dcq"], b["dcs"], ctr.FP8_COLS_BY_COLUMN,
                                       b["ws"])
        ctr.ctr_fp8_matmul(b["dq"], b["ds"], b["wtq"], b["wts"], off, b["dx"], b["ws2"])
        ctr.ctr_fp8_matmul_wgrad(b["dcq"], b["dcs"], b["xcq"], b["xcs"], off, b["dw"], b["ws"])
        return {"y": b["y"], "dx": b["dx"], "dw": b["dw"]}
    ctr.ctr_clip_grads(b["list"], c["max_norm"], b["norm"], b["ws"])
    return {"norm": b["norm"][0], "grads": b["outs"]}


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    if c["op"] == "route":
        names = ("expert", "weight", "slot", "token", "offsets")
        out = dict(zip(names, _route_plain(st["scores"], c["k"], c["renorm"])))
        if c["train"]:
            out["dscores"] = _route_grad_plain(st["dweight"], st["scores"], c["k"], c["renorm"])
        return out
    if c["op"] == "rows":
        return _rows_op_plain(st)
    if c["op"] == "product":
        return _product_plain(st)
    return _clip_plain(st)


# ---------------------------------------------------------------------------
# 64-bit values, written apart from the plain forms
# ---------------------------------------------------------------------------
def _e4m3(v):
    """The e4m3 value nearest to v (fp64; ties to even): 3 mantissa bits, steps of 2^-9 below 2^-6."""
    a = v.abs().clamp(max=448.0)
    ex = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(ex - 3)
    return torch.sign(v) * torch.round(a / step) * step


def _quantised(x, amax):
    """The values of x's codes (fp64): scale and product are fp32 numbers by definition."""
    amax = amax.float().clamp(min=TINY)
    inv = (torch.full_like(amax, 448.0) / amax)
    s = amax / torch.full_like(amax, 448.0)
    return _e4m3((x.float() * inv).double()) * s.double()


def _by_rows(x):
    parts = [x[:, c:c + 128] for c in range(0, x.shape[1], 128)]
    return torch.cat([_quantised(p, p.abs().max(1, keepdim=True).values) for p in parts], 1)


def _by_blocks(x):
    rows = [x[r:r + 128] for r in range(0, x.shape[0], 128)]
    parts = [[p[:, c:c + 128] for c in range(0, x.shape[1], 128)] for p in rows]
    return torch.cat([torch.cat([_quantised(p, p.abs().max()) for p in row], 1) for row in parts])


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "route":
        import numpy as np
        s = st["scores"].double().cpu().numpy()
        T, E, k = c["tokens"], c["experts"], c["k"]
        choice = np.argsort(-s, axis=1, kind="stable")[:, :k]
        top = np.take_along_axis(s, choice, 1)
        live = np.isfinite(top)
        some = live[:, :1]
        z = np.where(np.isfinite(s), np.exp(s - np.where(some, top[:, :1], 0.0)), 0.0)
        picked = np.zeros((T, E), dtype=bool)
        picked[np.arange(T)[:, None], choice] = live
        base = z * picked if c["renorm"] else z
        p = base / np.where(some, base.sum(1, keepdims=True), 1.0)
        weight = np.where(live, np.take_along_axis(p, choice, 1), 0.0)
        flat = np.where(live, choice, E).ravel()
        order = np.argsort(flat, kind="stable")
        count = int(live.sum())
        slot = np.full(T * k, -1, dtype=np.int32)
        slot[order[:count]] = np.arange(count)
        token = np.full(T * k, -1, dtype=np.int32)
        token[:count] = order[:count] // k
        offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])]).astype(np.int32)
        out = {"expert": np.where(live, choice, -1).astype(np.int32), "weight": weight, "slot": slot.reshape(T, k),
               "token": token, "offsets": offsets}
        if c["train"]:
            dw = st["dweight"].double().cpu().numpy()
            up = np.zeros((T, E))
            up[np.arange(T)[:, None], choice] = np.where(live, dw, 0.0)
            out["dscores"] = p * (up - (up * p).sum(1, keepdims=True))
        return out
    if c["op"] == "rows":
        token, slot, w = st["token"].long(), st["slot"].long(), st["weight"].double()
        ys = st["ys"].double()
        out = {"xs": st["x"].double()[token], "y": sum(ys[slot[:, j]] * w[:, j:j + 1] for j in range(c["k"]))}
        if c["train"]:
            dy = st["dy"].double()
            dys = torch.zeros_like(ys)
            for j in range(c["k"]):
                dys[slot[:, j]] = dy * w[:, j:j + 1]
            out["dys"] = dys
            out["dweight"] = torch.stack([torch.einsum("td,td->t", dy, ys[slot[:, j]]) for j in range(c["k"])], 1)
            out["dx"] = sum(st["dxs"].double()[slot[:, j]] for j in range(c["k"]))
        return out
    if c["op"] == "product":
        K, N, G = c["kdim"], c["n"], c["experts"]
        off = st["offsets"].tolist()
        x = st["x"] if st["token"] is None else st["x"][st["token"].long()]
        if not c["train"]:
            s = st["ws"].double()
            w = [st["wq"][g].view(torch.float8_e4m3fn).double() for g in range(G)]
            w = [(w[g] * s[g].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1))[:, :K] for g in range(G)]
            xq = _by_rows(x)
            return torch.cat([xq[off[g]:off[g + 1]] @ w[g].T for g in range(G)])
        w = [_by_blocks(st["w"][g]) for g in range(G)]
        xq, dq = _by_rows(x), _by_rows(st["dy"])
        y = torch.cat([xq[off[g]:off[g + 1]] @ w[g].T for g in range(G)])
        dx = torch.cat([dq[off[g]:off[g + 1]] @ w[g] for g in range(G)])
        dw = torch.zeros((G, N, K), dtype=torch.float64, device="cuda")
        for g in range(G):
            a, b = off[g], off[g + 1]
            if b > a:
                dw[g] = _by_rows(st["dy"][a:b].T) @ _by_blocks(x[a:b])
        return {"y": y, "dx": dx, "dw": dw}
    total = sum(float(x.double().square().sum()) for x in st["grads"])
    norm = math.sqrt(total)
    f = c["max_norm"] / norm if norm > c["max_norm"] else 1.0
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": [x.double() * f for x in st["grads"]]}
