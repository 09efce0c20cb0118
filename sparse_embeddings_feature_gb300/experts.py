"""An expert layer on the interaction output: device buffers and call sequence.

``ExpertLayer`` owns the buffers of a mixture of linear experts for a fixed batch
and runs it as a sequence of libctr calls on the current stream:

    forward    route -> row codes of the chosen experts' tokens -> products
               -> rows added back under the router's weights
    backward   rows' and weights' gradient -> codes -> input gradient, weight
               gradient -> tokens' gradient -> scores' gradient
    clip       the global norm over the layer's and any other gradients

Weights are quantised when they are set (`set_weights`), activations in every
call.  No arithmetic of the method happens here.

``python -m sparse_embeddings_feature_gb300.experts`` trains such a layer behind
the CTR path (embeddings -> interaction -> experts -> click probability) on
synthetic clicks: the layer's input gradient is the interaction's upstream
gradient, so the embedding rows learn too.
"""
from __future__ import annotations

from typing import Iterable, Optional, Union

import torch

from . import ctr


class ExpertLayer:
    """y[t] = sum over t's k experts e of weight(t, e) W_e x[t], with W [experts, out_width, width].

    x and y are fp32 or bf16 (`dtype`); rows of x may be strided.  With `train`, forward keeps what
    backward needs, a copy of the scores with it: backward(dy) returns (dx, dscores, dw) for the latest
    forward, whatever became of its arguments.  Results are the layer's own buffers, which the next call
    writes.  Its calls run on the current device, which has to be
    `device`.

    score ("softmax" or "sigmoid"), groups, group_k and factor, or a bias given to forward, make the routing a
    balanced one (ctr_expert_route_balanced): choices by score function + bias in the best groups, weights from
    the score function.  The bias is the program's: `loads` has what it goes by."""

    def __init__(self, tokens: int, width: int, out_width: int, experts: int, k: int, dtype=torch.float32,
                 renormalize: bool = True, train: bool = False, device="cuda", score: str = "softmax", groups: int = 1,
                 group_k: Optional[int] = None, factor: float = 1.0):
        if dtype not in ctr.DTYPES:
            raise ValueError("dtype must be torch.float32 or torch.bfloat16")
        if not 1 <= k <= min(experts, ctr.MAX_CHOICES) or experts > ctr.MAX_EXPERTS:
            raise ValueError(f"need 1 <= k <= min(experts, {ctr.MAX_CHOICES}) and experts <= {ctr.MAX_EXPERTS}")
        if min(tokens, width, out_width) < 1:
            raise ValueError("tokens, width and out_width must be positive")
        self.groups, self.group_k = groups, groups if group_k is None else group_k
        if score not in ctr.SCORES:
            raise ValueError(f"score must be one of {', '.join(ctr.SCORES)}")
        if not 1 <= groups <= ctr.MAX_GROUPS or experts % groups or not 1 <= self.group_k <= groups \
                or k > self.group_k * (experts // groups):
            raise ValueError(f"need groups <= {ctr.MAX_GROUPS} that divide experts, 1 <= group_k <= groups, and k experts in "
                             f"group_k groups")
        self.score, self.factor = ctr.SCORES[score], float(factor)
        self.balanced = score != "softmax" or self.group_k < groups or self.factor != 1.0
        self.tokens, self.width, self.out_width, self.experts, self.k = tokens, width, out_width, experts, k
        self.dtype, self.renormalize, self.train = dtype, bool(renormalize), bool(train)
        T, K, N, E, R = tokens, width, out_width, experts, tokens * k
        kb, nb = ctr.fp8_blocks(K), ctr.fp8_blocks(N)

        def buf(*shape, dt=torch.float32):
            return torch.empty(shape, dtype=dt, device=device)
        i32, u8 = torch.int32, torch.uint8
        # routing
        self.expert, self.slot, self.token = buf(T, k, dt=i32), buf(T, k, dt=i32), buf(R, dt=i32)
        self.offsets, self.weight = buf(E + 1, dt=i32), buf(T, k)
        # codes of the experts' rows and weights
        self.xq, self.xs = buf(R, kb * 128, dt=u8), buf(kb, R)
        self.wq, self.ws = buf(E, N, kb * 128, dt=u8), buf(E, nb, kb)
        self.ys, self.y = buf(R, N, dt=dtype), buf(T, N, dt=dtype)
        if train:
            P = ctr.fp8_padded_rows(R, E)
            self.wtq, self.wts = buf(E, K, nb * 128, dt=u8), buf(E, kb, nb)
            self.xcq, self.xcs = buf(K, P, dt=u8), buf(kb, P // 128)
            self.dys, self.dweight = buf(R, N, dt=dtype), buf(T, k)
            self.dq, self.ds = buf(R, nb * 128, dt=u8), buf(nb, R)
            self.dcq, self.dcs = buf(N, P, dt=u8), buf(P // 128, N)
            self.dxs, self.dx = buf(R, K, dt=dtype), buf(T, K, dt=dtype)
            self.dw = buf(E, N, K)
            self.kept = {}   # type of the scores -> their copy and their gradient; kept, as a captured graph uses them
        self.norm = buf(1)
        self.ws_route = ctr.workspace(ctr.ctr_expert_route_workspace_size(T, E, k), device)
        self.ws_rows = ctr.workspace(ctr.ctr_expert_workspace_size(), device)
        self.ws_mm = ctr.workspace(max(ctr.ctr_fp8_matmul_workspace_size(R, E, N, K),
                                       ctr.ctr_fp8_matmul_workspace_size(R, E, K, N)), device)
        self.ws_clip = ctr.workspace(ctr.ctr_clip_grads_workspace_size(), device)
        self.scores = None

    def set_weights(self, w: torch.Tensor) -> None:
        """Quantise the experts' weights [experts, out_width, width] (fp32 or bf16): once for serving, after
        every update in training.  The latest forward is then no longer there for backward, whose input
        gradient would be that of other weights."""
        if tuple(w.shape) != (self.experts, self.out_width, self.width):
            raise ValueError(f"weights must be {(self.experts, self.out_width, self.width)}")
        self.scores = None
        ctr.ctr_fp8_quantize_blocks(w, self.wq, self.ws, self.ws_mm, *((self.wtq, self.wts) if self.train else ()))

    def forward(self, x: torch.Tensor, scores: torch.Tensor, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y [tokens, out_width] of x [tokens, width] under the router's scores [tokens, experts] and, for balance, a
        bias [experts] (fp32) on the choices alone."""
        # the calls see the padded width of x and look its rows up through the map: its sizes are checked here
        if not isinstance(x, torch.Tensor) or x.shape != (self.tokens, self.width):
            raise ValueError(f"x must be {(self.tokens, self.width)}")
        self.scores = None   # until this forward is complete there is none
        self.by_balance = self.balanced or bias is not None
        maps = (self.expert, self.weight, self.slot, self.token, self.offsets, self.ws_route)
        if self.by_balance:
            ctr.ctr_expert_route_balanced(scores, self.k, self.score, bias, self.groups, self.group_k, self.renormalize,
                                          self.factor, *maps)
        else:
            ctr.ctr_expert_route(scores, self.k, self.renormalize, *maps)
        if self.train:
            if scores.dtype not in self.kept:
                self.kept[scores.dtype] = tuple(torch.empty(scores.shape, dtype=scores.dtype, device=scores.device)
                                                for _ in range(2))
            kept, self.dscores = self.kept[scores.dtype]
            kept.copy_(scores)
            ctr.ctr_fp8_quantize_rows_cols(x, self.offsets, self.xq, self.xs, self.xcq, self.xcs,
                                           ctr.FP8_COLS_BY_BLOCK, self.ws_mm, row_index=self.token)
        else:
            ctr.ctr_fp8_quantize_rows(x, self.xq, self.xs, self.ws_mm, row_index=self.token)
        ctr.ctr_fp8_matmul(self.xq, self.xs, self.wq, self.ws, self.offsets, self.ys, self.ws_mm)
        ctr.ctr_expert_combine(self.ys, self.slot, self.weight, self.y, self.ws_rows)
        if self.train:
            self.scores = kept
        return self.y

    def sorted_rows(self, x: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
        """x in the latest forward's row order (expert e has rows offsets[e] .. offsets[e+1]-1 of out
        [tokens*k, width]), for experts of another kind."""
        ctr.ctr_expert_dispatch(x, self.slot, self.token, out, self.ws_rows)
        return out

    def backward(self, dy: torch.Tensor, dx: Optional[torch.Tensor] = None):
        """(dx, dscores, dw) of the latest forward; dx goes to `dx` where one is given."""
        if not self.train or self.scores is None:
            raise RuntimeError("backward needs train=True and a forward since the weights were set")
        dx = self.dx if dx is None else dx
        ctr.ctr_expert_combine_bwd(dy, self.ys, self.slot, self.weight, self.token, self.dys, self.dweight, self.ws_rows)
        ctr.ctr_fp8_quantize_rows_cols(self.dys, self.offsets, self.dq, self.ds, self.dcq, self.dcs,
                                       ctr.FP8_COLS_BY_COLUMN, self.ws_mm)
        ctr.ctr_fp8_matmul(self.dq, self.ds, self.wtq, self.wts, self.offsets, self.dxs, self.ws_mm)
        ctr.ctr_fp8_matmul_wgrad(self.dcq, self.dcs, self.xcq, self.xcs, self.offsets, self.dw, self.ws_mm,
                                 rows=self.tokens * self.k)
        ctr.ctr_expert_combine(self.dxs, self.slot, None, dx, self.ws_rows)
        if self.by_balance:
            ctr.ctr_expert_route_balanced_bwd(self.dweight, self.scores, self.score, self.renormalize, self.factor,
                                              self.expert, self.dscores, self.ws_route)
        else:
            ctr.ctr_expert_route_bwd(self.dweight, self.scores, self.renormalize, self.expert, self.dscores, self.ws_route)
        return dx, self.dscores, self.dw

    def loads(self) -> torch.Tensor:
        """Rows of each expert [experts] (int32) in the latest forward, on the device: what a balance bias goes by."""
        return self.offsets[1:] - self.offsets[:-1]

    def grads(self, others: Iterable[torch.Tensor] = ()) -> ctr.GradList:
        """dw and `others` as a list for clip.  For tensors that stay where they are it is built once: it
        takes the host longer than the clipping of a small net's gradients takes the GPU."""
        if not self.train:
            raise RuntimeError("a layer has gradients with train=True")
        grads = [self.dw, *others]
        return ctr.grad_list(grads, grads)

    def clip(self, max_norm: float, others: Union[ctr.GradList, Iterable[torch.Tensor]] = ()) -> torch.Tensor:
        """Scale dw and `others` (tensors, or a list from `grads`) in place to a global norm of at most
        max_norm; the norm [1], on the device."""
        grads = others if isinstance(others, ctr.GradList) else self.grads(others)
        ctr.ctr_clip_grads(grads, max_norm, self.norm, self.ws_clip)
        return self.norm

    def check_status(self) -> dict:
        """Synchronise and read the workspaces' device errors (0: none)."""
        return {n: ctr.ctr_check_status(ws) for n, ws in
                (("route", self.ws_route), ("rows", self.ws_rows), ("products", self.ws_mm))}


def train_demo(steps: int = 60, batch: int = 2048, experts: int = 8, k: int = 2, hidden: int = 128, lr: float = 0.05,
               max_norm: float = 1.0, seed: int = 0):
    """Embeddings -> interaction -> experts -> click probability on one synthetic batch; the losses.

    The clicks follow a random linear model of the interaction output.  The gate, the experts and the
    head are plain SGD on clipped gradients; the embedding rows follow the interaction's gradient."""
    from . import workload as W
    from .pipeline import CtrPath

    cfg = W.CONFIGS["full_step"].shrink(batch=batch, rows_per_table=tuple([5000] * 26))
    w = W.make_workload(cfg)
    path = CtrPath(cfg, w["ids"].size)
    path.upload(w)
    width = cfg.out_width
    layer = ExpertLayer(batch, width, hidden, experts, k, train=True)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    weights, gate, head = draw(experts, hidden, width) / width ** 0.5, draw(width, experts) / width ** 0.5, \
        draw(hidden) / hidden ** 0.5
    clicks = None
    losses = []
    for _ in range(steps):
        path.dedup()
        path.forward()
        path.interaction()
        x = path.out
        if clicks is None:
            clicks = (x @ draw(width) / width ** 0.5 + 0.3 * draw(batch) > 0).float()
        layer.set_weights(weights)
        scores = x @ gate
        h = torch.relu(layer.forward(x, scores))
        logit = h @ head
        losses.append(torch.nn.functional.binary_cross_entropy_with_logits(logit, clicks).item())
        dlogit = (torch.sigmoid(logit) - clicks) / batch
        dhead = h.t() @ dlogit
        dh = dlogit[:, None] * head * (h > 0)
        dx, dscores, dw = layer.backward(dh, dx=path.dout)   # straight into the interaction's upstream gradient
        dgate = x.t() @ dscores
        dx.addmm_(dscores, gate.t())
        layer.clip(max_norm, [dgate, dhead])
        for p, d in ((weights, dw), (gate, dgate), (head, dhead)):
            p.sub_(d, alpha=20 * lr)
        path.interaction_bwd()
        path.bwd_update()
    bad = {n: v for n, v in {**layer.check_status(), **path.check_status()}.items() if v}
    if bad:
        raise RuntimeError(f"device errors: {bad}")
    return losses


if __name__ == "__main__":
    loss = train_demo()
    for i in range(0, len(loss), 10):
        print(f"step {i:3d}  loss {loss[i]:.4f}")
    print(f"step {len(loss) - 1:3d}  loss {loss[-1]:.4f}")
