"""Layers around the experts: device buffers and call sequences.

    ResidualBlock   y = act(norm(x) W1^T + b1) W2^T + b2 + x, with its backward pass
    NormProduct     s = x + residual, y = norm(s) W^T in 8 bits, for serving

Each owns its buffers for a fixed number of rows and runs as a sequence of libctr
calls on the current stream.  No arithmetic of the method happens here.

``python -m sparse_embeddings_feature_gb300.layers`` trains such layers behind the
CTR path (embeddings -> interaction -> dense layer -> residual block -> norm ->
balanced experts -> click probability) on synthetic clicks.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from . import ctr
from .experts import ExpertLayer


class ResidualBlock:
    """y = act(norm(x) W1^T + b1) W2^T + b2 + x for x [rows, width], with W1 [hidden, width] and W2 [width, hidden].

    Everything is fp32 or bf16 (`dtype`) but gamma, which is fp32.  Parameters are tensors of the caller's, given to
    every call as a dict with w1, b1, w2, b2 and gamma.  With `train`, forward keeps what backward needs but x and the
    parameters, which have to be as they were; backward(dy) returns (dx, gradients by the parameters' names) of the latest
    forward.  Results are the block's own buffers, which the next call writes."""

    def __init__(self, rows: int, width: int, hidden: int, dtype=torch.float32, act: str = "gelu", eps: float = 1e-6,
                 train: bool = False, device="cuda"):
        if dtype not in ctr.DTYPES:
            raise ValueError("dtype must be torch.float32 or torch.bfloat16")
        if act not in ctr.ACTIVATIONS:
            raise ValueError(f"act must be one of {', '.join(ctr.ACTIVATIONS)}")
        if min(rows, width, hidden) < 1 or width > ctr.MAX_NORM_WIDTH:
            raise ValueError(f"rows, width and hidden must be positive, width at most {ctr.MAX_NORM_WIDTH}")
        self.rows, self.width, self.hidden, self.dtype = rows, width, hidden, dtype
        self.act, self.eps, self.train = ctr.ACTIVATIONS[act], float(eps), bool(train)

        def buf(*shape, dt=dtype):
            return torch.empty(shape, dtype=dt, device=device)
        self.v, self.h, self.y = buf(rows, width), buf(rows, hidden), buf(rows, width)
        self.pre = buf(rows, hidden) if train else None
        if train:
            self.dh, self.dv, self.dx = buf(rows, hidden), buf(rows, width), buf(rows, width)
            self.grads: Dict[str, torch.Tensor] = {
                "w1": buf(hidden, width), "b1": buf(hidden), "w2": buf(width, hidden), "b2": buf(width),
                "gamma": buf(width, dt=torch.float32)}
        self.ws_norm = ctr.workspace(ctr.ctr_rms_norm_workspace_size(rows, width), device)
        self.ws_dense = ctr.workspace(max(ctr.ctr_dense_workspace_size(rows, hidden, width, dtype, train),
                                          ctr.ctr_dense_workspace_size(rows, width, hidden, dtype, train)), device)
        self.latest: Optional[Tuple[torch.Tensor, Dict[str, torch.Tensor]]] = None

    def forward(self, x: torch.Tensor, p: Dict[str, torch.Tensor]) -> torch.Tensor:
        """y [rows, width] of x [rows, width]."""
        self.latest = None   # until this forward is complete there is none
        ctr.ctr_rms_norm(x, None, p["gamma"], self.eps, None, self.v, None, None, self.ws_norm)
        ctr.ctr_dense(self.v, p["w1"], p["b1"], self.act, None, self.h, self.pre, self.ws_dense)
        ctr.ctr_dense(self.h, p["w2"], p["b2"], ctr.ACT_NONE, x, self.y, None, self.ws_dense)
        self.latest = (x, p)
        return self.y

    def backward(self, dy: torch.Tensor) -> Tuple[torch.Tensor, Dict[str, torch.Tensor]]:
        """(dx, the parameters' gradients) of the latest forward."""
        if not self.train or self.latest is None:
            raise RuntimeError("backward needs train=True and a forward")
        (x, p), g = self.latest, self.grads
        ctr.ctr_dense_bwd(dy, self.h, p["w2"], None, ctr.ACT_NONE, self.dh, g["w2"], g["b2"], self.ws_dense)
        ctr.ctr_dense_bwd(self.dh, self.v, p["w1"], self.pre, self.act, self.dv, g["w1"], g["b1"], self.ws_dense)
        ctr.ctr_rms_norm_bwd(self.dv, dy, x, p["gamma"], self.eps, self.dx, g["gamma"], self.ws_norm)
        return self.dx, g

    def check_status(self) -> dict:
        """Synchronise and read the workspaces' device errors (0: none)."""
        return {n: ctr.ctr_check_status(ws) for n, ws in (("norm", self.ws_norm), ("dense", self.ws_dense))}


class NormProduct:
    """s = x + residual and y = (norm(s) gamma) W^T for x [rows, width], the product in 8 bits, W [out_width, width]
    quantised when it is set, before the first forward: one layer of a serving stack.  The norm writes the codes that the
    product reads."""

    def __init__(self, rows: int, width: int, out_width: int, dtype=torch.bfloat16, eps: float = 1e-6, device="cuda"):
        if dtype not in ctr.DTYPES:
            raise ValueError("dtype must be torch.float32 or torch.bfloat16")
        if min(rows, width, out_width) < 1 or width > ctr.MAX_NORM_WIDTH:
            raise ValueError(f"rows, width and out_width must be positive, width at most {ctr.MAX_NORM_WIDTH}")
        kb, nb = ctr.fp8_blocks(width), ctr.fp8_blocks(out_width)
        self.rows, self.width, self.out_width, self.eps = rows, width, out_width, float(eps)

        def buf(*shape, dt=torch.float32):
            return torch.empty(shape, dtype=dt, device=device)
        self.s, self.y = buf(rows, width, dt=dtype), buf(rows, out_width, dt=dtype)
        self.q, self.scale = buf(rows, kb * 128, dt=torch.uint8), buf(kb, rows)
        self.wq, self.ws = buf(1, out_width, kb * 128, dt=torch.uint8), buf(1, nb, kb)
        self.room = ctr.workspace(max(ctr.ctr_rms_norm_workspace_size(rows, width),
                                      ctr.ctr_fp8_matmul_workspace_size(rows, 1, out_width, width)), device)
        self.has_weights = False

    def set_weights(self, w: torch.Tensor) -> None:
        if tuple(w.shape) != (self.out_width, self.width):
            raise ValueError(f"weights must be {(self.out_width, self.width)}")
        self.has_weights = False   # until the call is made
        ctr.ctr_fp8_quantize_blocks(w[None], self.wq, self.ws, self.room)
        self.has_weights = True

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor], gamma: Optional[torch.Tensor]):
        """(s, y), the layer's own buffers."""
        if not self.has_weights:
            raise RuntimeError("forward needs weights: set_weights")
        ctr.ctr_rms_norm(x, residual, gamma, self.eps, self.s, None, self.q, self.scale, self.room)
        ctr.ctr_fp8_matmul(self.q, self.scale, self.wq, self.ws, None, self.y, self.room)
        return self.s, self.y

    def check_status(self) -> int:
        return ctr.ctr_check_status(self.room)


def train_demo(steps: int = 60, batch: int = 2048, width: int = 128, hidden: int = 256, experts: int = 16, k: int = 2,
               lr: float = 0.05, max_norm: float = 1.0, seed: int = 0):
    """Embeddings -> interaction -> dense layer -> residual block -> norm -> balanced experts -> click probability on one
    synthetic batch; (losses, the experts' largest load over the mean one, by step).

    The clicks follow a random linear model of the interaction output.  Everything but the embedding rows, which follow the
    interaction's gradient, is plain SGD on clipped gradients; the balance bias goes down for experts with more than the
    mean load and up for the others."""
    from . import workload as W
    from .pipeline import CtrPath

    cfg = W.CONFIGS["full_step"].shrink(batch=batch, rows_per_table=tuple([5000] * 26))
    w = W.make_workload(cfg)
    path = CtrPath(cfg, w["ids"].size)
    path.upload(w)
    inputs = cfg.out_width
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def new(*shape):
        return torch.empty(shape, device="cuda")
    block = ResidualBlock(batch, width, hidden, train=True)
    layer = ExpertLayer(batch, width, hidden, experts, k, train=True, score="sigmoid", groups=4, group_k=2)
    stem = {"w": draw(width, inputs) / inputs ** 0.5, "b": torch.zeros(width, device="cuda")}
    params = {"w1": draw(hidden, width) / width ** 0.5, "b1": torch.zeros(hidden, device="cuda"),
              "w2": draw(width, hidden) / hidden ** 0.5, "b2": torch.zeros(width, device="cuda"),
              "gamma": torch.ones(width, device="cuda")}
    gamma, gate = torch.ones(width, device="cuda"), draw(experts, width) / width ** 0.5
    weights, head = draw(experts, hidden, width) / width ** 0.5, draw(1, hidden) / hidden ** 0.5
    bias = torch.zeros(experts, device="cuda")
    x0, pre, dx0, u, du, du2 = (new(batch, width) for _ in range(6))
    scores, logit, dh = new(batch, experts), new(batch, 1), new(batch, hidden)
    dstem = {n: torch.empty_like(t) for n, t in stem.items()}
    dgamma, dgate, dhead = torch.empty_like(gamma), torch.empty_like(gate), torch.empty_like(head)
    ws = ctr.workspace(max(ctr.ctr_dense_workspace_size(batch, n, kk, torch.float32, True)
                           for n, kk in ((width, inputs), (experts, width), (1, hidden))))
    ws_norm = ctr.workspace(ctr.ctr_rms_norm_workspace_size(batch, width))
    clicks, losses, skew = None, [], []
    for _ in range(steps):
        path.dedup()
        path.forward()
        path.interaction()
        if clicks is None:
            clicks = (path.out @ draw(inputs) / inputs ** 0.5 + 0.3 * draw(batch) > 0).float()
        layer.set_weights(weights)
        ctr.ctr_dense(path.out, stem["w"], stem["b"], ctr.ACT_SILU, None, x0, pre, ws)
        y = block.forward(x0, params)
        ctr.ctr_rms_norm(y, None, gamma, 1e-6, None, u, None, None, ws_norm)
        ctr.ctr_dense(u, gate, None, ctr.ACT_NONE, None, scores, None, ws)
        h = torch.relu(layer.forward(u, scores, bias))
        load = layer.loads().float()
        skew.append((load.max() / load.mean()).item())
        ctr.ctr_dense(h, head, None, ctr.ACT_NONE, None, logit, None, ws)
        losses.append(torch.nn.functional.binary_cross_entropy_with_logits(logit[:, 0], clicks).item())
        dlogit = ((torch.sigmoid(logit[:, 0]) - clicks) / batch)[:, None].contiguous()
        ctr.ctr_dense_bwd(dlogit, h, head, None, ctr.ACT_NONE, dh, dhead, None, ws)
        dh.mul_(h > 0)
        du_experts, dscores, dw = layer.backward(dh)
        ctr.ctr_dense_bwd(dscores, u, gate, None, ctr.ACT_NONE, du, dgate, None, ws)
        du.add_(du_experts)
        ctr.ctr_rms_norm_bwd(du, None, y, gamma, 1e-6, du2, dgamma, ws_norm)
        dx, grads = block.backward(du2)
        ctr.ctr_dense_bwd(dx, path.out, stem["w"], pre, ctr.ACT_SILU, path.dout, dstem["w"], dstem["b"], ws)
        step = [(weights, dw), (gate, dgate), (head, dhead), (gamma, dgamma), *((stem[n], dstem[n]) for n in stem),
                *((params[n], grads[n]) for n in params)]
        layer.clip(max_norm, [d for _, d in step[1:]])
        for t, d in step:
            t.sub_(d, alpha=20 * lr)
        bias.sub_(0.02 * torch.sign(load - load.mean()))
        path.interaction_bwd()
        path.bwd_update()
    bad = {n: v for n, v in {**layer.check_status(), **block.check_status(), **path.check_status(),
                             "dense layers": ctr.ctr_check_status(ws), "norm": ctr.ctr_check_status(ws_norm)}.items() if v}
    if bad:
        raise RuntimeError(f"device errors: {bad}")
    return losses, skew


if __name__ == "__main__":
    loss, skew = train_demo()
    for i in [*range(0, len(loss), 10), len(loss) - 1]:
        print(f"step {i:3d}  loss {loss[i]:.4f}  largest load {skew[i]:.2f} times the mean")
