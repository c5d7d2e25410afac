"""The expert operators in plain torch on the CPU, with the wrappers' arguments and
their habit of writing into the tensor they are given: for tests of what ExpertLayer
does around them."""
import torch


class Route:
    def __init__(self, tokens, topk, experts):
        self.tokens, self.topk, self.experts = tokens, topk, experts

    def sort(self, ids):
        flat = ids.reshape(-1).long()
        key = torch.where((flat < 0) | (flat >= self.experts),
                          torch.full_like(flat, self.experts), flat)
        self.order = torch.sort(key, stable=True).indices
        self.position = torch.empty_like(self.order)
        self.position[self.order] = torch.arange(flat.numel())
        counts = torch.bincount(key, minlength=self.experts + 1)
        self.offsets = counts.cumsum(0) - counts
        self.kept = (self.position < self.offsets[self.experts]).reshape(ids.shape)
        self.position = self.position.reshape(ids.shape)
        return self

    def gather(self, X):
        rows = X[self.order // self.topk].clone()
        rows[self.offsets[self.experts]:] = 0
        return rows

    def _sum(self, rows, weights, kept):
        rows = rows.reshape(self.tokens, self.topk, rows.shape[-1])
        if weights is not None:
            rows = rows * weights[:, :, None].to(rows.dtype)
        return torch.where(kept[:, :, None], rows, torch.zeros_like(rows)).sum(1)

    def combine(self, Ys, out=None, weights=None):
        return self._sum(Ys[self.position.reshape(-1)], weights, self.kept)

    def combine_slots(self, Ys, out=None, weights=None, ids=None):
        kept = torch.ones((self.tokens, self.topk), dtype=torch.bool) if ids is None else \
            (ids >= 0) & (ids < self.experts)
        return self._sum(Ys, weights, kept)

    def gather_grad(self, dXs):
        return self.combine(dXs)

    def combine_grad(self, dY, Ys, weights, out=None, dweights=None):
        pos = self.position
        zero = torch.zeros((), dtype=Ys.dtype)
        dw = torch.where(self.kept, (Ys[pos] * dY[:, None]).sum(-1), zero)
        grad = torch.where(self.kept[:, :, None],
                           dY[:, None] * weights[:, :, None].to(dY.dtype), zero)
        out = torch.empty_like(Ys) if out is None else out
        out[pos.reshape(-1)] = grad.reshape(-1, dY.shape[1])
        return out, dw


class Grouped:
    def __init__(self, rows, N, K, experts, op="forward", out="f16"):
        self.rows, self.N, self.K, self.experts, self.op = rows, N, K, experts, op

    def device_status(self):
        return 0

    def __call__(self, P, Q, offsets):
        E = self.experts
        shape = {"forward": (self.rows, self.N), "grad_input": (self.rows, self.K),
                 "grad_weight": (E, self.N, self.K)}[self.op]
        out = torch.zeros(shape, dtype=P.dtype)
        for e in range(E):
            s = slice(int(offsets[e]), int(offsets[e + 1]))
            if self.op == "forward":
                out[s] = P[s] @ Q[e].t()
            elif self.op == "grad_input":
                out[s] = P[s] @ Q[e]
            else:
                out[e] = P[s].t() @ Q[s]
        return out


class W4:
    def __init__(self, M, N, K, group=128, out="f16", experts=0, share=1):
        if M < 1:
            raise ValueError("M must be at least 1")
        self.M, self.N, self.K, self.group, self.experts, self.share = M, N, K, group, experts, share

    def device_status(self):
        return 0

    def __call__(self, X, packed, scales, zeros=None, ids=None):
        if tuple(scales.shape) != (self.experts, self.N, self.K // self.group):
            raise ValueError("scales must have shape %s" % (
                (self.experts, self.N, self.K // self.group),))
        q = torch.stack([packed & 15, packed >> 4], -1).reshape(scales.shape + (self.group,))
        z = 8.0 if zeros is None else zeros[..., None].to(X.dtype)
        w = ((q.to(X.dtype) - z) * scales[..., None].to(X.dtype)).flatten(-2)
        Y = torch.zeros((self.M, self.N), dtype=X.dtype)
        for m, e in enumerate(ids.reshape(-1).tolist()):
            if 0 <= e < self.experts:
                Y[m] = w[e] @ X[m // self.share]
        return Y


def install(monkeypatch):
    from tma_pipelined_tensor_fp16_gb300 import expert_layer
    monkeypatch.setattr(expert_layer, "ExpertRoute", Route)
    monkeypatch.setattr(expert_layer, "GroupedPlan", Grouped)
    monkeypatch.setattr(expert_layer, "W4Plan", W4)


def layer(experts=3, width=32, inner=64, topk=2, tokens=7, seed=0):
    """An ExpertLayer in 64 bits, X, ids and weights."""
    from tma_pipelined_tensor_fp16_gb300.expert_layer import ExpertLayer
    g = torch.Generator().manual_seed(seed)
    W1 = torch.randn((experts, inner, width), generator=g, dtype=torch.float64)
    W2 = torch.randn((experts, width, inner), generator=g, dtype=torch.float64)
    X = torch.randn((tokens, width), generator=g, dtype=torch.float64)
    top, ids = torch.randn((tokens, experts), generator=g).topk(topk, dim=1)
    return ExpertLayer(W1, W2, topk), X, ids.to(torch.int32), torch.softmax(top, 1)
