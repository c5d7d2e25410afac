"""A mixture-of-experts feed-forward on the library's operators, and a command
that runs it: a training step (forward, both gradients of every operator, an
update) and decoding with the experts' weights in 4 bits; then the same of a whole
block, which has a norm in front, an expert that every token passes in a block-scaled
format, and clipped gradients.

    python -m tma_pipelined_tensor_fp16_gb300.expert_layer [--tokens 8192]
        [--topk 4] [--experts 16] [--width 2048] [--inner 4096] [--steps 10]
        [--decode 4] [--shared 4096] [--format mxfp8] [--clip 1.0]

Y[t] = sum_j w[t, j] * W2[e] . relu(W1[e] . X[t]),  e = ids[t, j]: the slots are
sorted by expert, the tokens gathered, both products run grouped by expert, and
the experts' rows are summed back with their routing weights.  Prints the time
of a training step and of a decoding step, and how far the decoding step with
4-bit weights is from the same step with fp16 weights; then the times of a block's
training and decoding steps (--shared 0: without the block).
"""
import argparse
import functools

from .binding import GemmError
from .experts import ExpertRoute, GroupedPlan, W4Plan, w4_pack
from .layer import GradClip, rms_norm, rms_norm_grad
from .microscale import MXPlan, mx_quantize


class ExpertLayer:
    """W1 is experts x inner x width, W2 experts x width x inner (fp16).

    Calls may come on several streams and from several threads, and graphs that
    captured them may be replayed beside them: none of the plans that the layer keeps
    minds runs that overlap."""

    def __init__(self, W1, W2, topk):
        self.W1, self.W2, self.topk = W1, W2, topk
        self.experts, self.inner, self.width = W1.shape
        self._plans = {}
        self._packed = None

    def _plan(self, rows, N, K, op, out="f16"):
        key = (rows, N, K, op, out)
        if key not in self._plans:
            self._plans[key] = GroupedPlan(rows, N, K, self.experts, op=op, out=out)
        return self._plans[key]

    def plans(self):
        """The plans that the layer keeps."""
        return [plan for kept in self._plans.values()
                for plan in (kept if isinstance(kept, list) else [kept])]

    def device_status(self):
        """GEMM_OK, or the status of a plan with a wait that ran out inside a kernel, whose
        results are not whole; call after synchronising."""
        return next((s for s in [plan.device_status() for plan in self.plans()] if s != 0), 0)

    def forward(self, X, ids, weights):
        """Y (tokens x width) and what ``backward`` needs."""
        tokens = X.shape[0]
        rows = tokens * self.topk
        route = ExpertRoute(tokens, self.topk, self.experts).sort(ids)
        Xs = route.gather(X)
        H = self._plan(rows, self.inner, self.width, "forward")(Xs, self.W1, route.offsets)
        A = H.relu()
        Ys = self._plan(rows, self.width, self.inner, "forward")(A, self.W2, route.offsets)
        Y = route.combine(Ys, weights=weights)
        return Y, (route, Xs, H, A, Ys, weights)

    def backward(self, dY, saved, out=None):
        """Gradients (dX, dweights, dW1, dW2); the weights' in fp32, in the tensors
        `out` = (dW1, dW2) where it is given.  `saved` stays as it is, so the same forward
        can be differentiated again."""
        route, Xs, H, A, Ys, weights = saved
        rows, I, W = Xs.shape[0], self.inner, self.width
        to1, to2 = ((), ()) if out is None else (out[:1], out[1:])
        dYs, dweights = route.combine_grad(dY, Ys, weights)
        dW2 = self._plan(rows, W, I, "grad_weight", "f32")(dYs, A, route.offsets, *to2)
        dA = self._plan(rows, W, I, "grad_input")(dYs, self.W2, route.offsets)
        dH = dA.masked_fill_(H <= 0, 0.0)  # not a product: dA need not be finite there
        dW1 = self._plan(rows, I, W, "grad_weight", "f32")(dH, Xs, route.offsets, *to1)
        dXs = self._plan(rows, I, W, "grad_input")(dH, self.W1, route.offsets)
        return route.gather_grad(dXs), dweights, dW1, dW2

    def pack(self, group=128, zeros=True):
        """Lay the weights, as they are now, out in 4 bits for ``decode``."""
        self._packed = (group, w4_pack(self.W1, group, zeros), w4_pack(self.W2, group, zeros))

    def decode(self, X, ids, weights):
        """Y for a few tokens with the packed weights: no sort, every slot's row
        straight from its expert's codes."""
        if self._packed is None:
            raise RuntimeError("the weights have not been packed: call pack() first")
        tokens = X.shape[0]
        rows = tokens * self.topk
        if tokens == 0:  # a plan has a row at least
            return X.new_empty(X.shape)
        group, (p1, s1, z1), (p2, s2, z2) = self._packed
        key = ("w4", rows, group)
        if key not in self._plans:
            self._plans[key] = [
                W4Plan(rows, self.inner, self.width, group=group, experts=self.experts,
                       share=self.topk),
                W4Plan(rows, self.width, self.inner, group=group, experts=self.experts)]
        up, down = self._plans[key]
        A = up(X, p1, s1, zeros=z1, ids=ids).relu_()
        Ys = down(A, p2, s2, zeros=z2, ids=ids)
        return ExpertRoute(tokens, self.topk, self.experts).combine_slots(
            Ys, weights=weights, ids=ids)


def _plan_beside(first, M, N, K, out="f16"):
    return MXPlan(M, N, K, format=first.format, out=out, beside=first)


class SharedExpert:
    """Y = S2 . relu(S1 . X) for every token (S1 inner x width, S2 width x inner, fp16), its
    products on operands in a block-scaled format; gradients take the rounding as the
    identity.  ``quantize`` lays the weights out as they are now, for ``forward``: call it
    again once they have changed (``backward`` rounds them anew).

    A number of tokens that is new takes new plans on the host alone, beside one whose status
    record they share, and only the latest are kept; a graph that captured others replays
    without them."""

    def __init__(self, S1, S2, format="mxfp8"):
        self.S1, self.S2, self.format = S1, S2, format
        self.inner, self.width = S1.shape
        self._first = MXPlan(1, self.inner, self.width, format=format, device=S1.device)
        self._plan = functools.lru_cache(maxsize=64)(functools.partial(_plan_beside, self._first))
        self._weights = (None, None)
        self.quantize()

    def plans(self):
        """The plan whose status record is that of all."""
        return [self._first]

    def device_status(self):
        """GEMM_OK, or the status of a product with a wait that ran out; call after
        synchronising."""
        return self._first.device_status()

    def quantize(self):
        """The weights for ``forward``, always in the same memory."""
        self._weights = tuple(mx_quantize(S, self.format, out=q)
                              for S, q in zip((self.S1, self.S2), self._weights))

    def forward(self, Q):
        """Y (tokens x width) of quantised rows, and what ``backward`` needs."""
        T, I, W = Q.rows, self.inner, self.width
        if T == 0:  # a plan has a row at least
            return self.S1.new_empty((0, W)), self.S1.new_empty((0, I))
        A = self._plan(T, I, W)(Q, self._weights[0]).relu_()
        return self._plan(T, W, I)(mx_quantize(A, self.format), self._weights[1]), A

    def backward(self, dY, A, X, out=None):
        """(dX, dS1, dS2) for the rows X that forward had quantised; the weights' in fp32,
        in `out` = (dS1, dS2) where it is given."""
        T, I, W, f = A.shape[0], self.inner, self.width, self.format
        if T == 0:
            dS1, dS2 = out or (self.S1.float(), self.S2.float())
            return dY.new_empty((0, W)), dS1.zero_(), dS2.zero_()
        to1, to2 = ((), ()) if out is None else (out[:1], out[1:])
        dS2 = self._plan(W, I, T, "f32")(mx_quantize(dY, f, transpose=True),
                                         mx_quantize(A, f, transpose=True), *to2)
        dA = self._plan(T, I, W)(mx_quantize(dY, f), mx_quantize(self.S2, f, transpose=True))
        dH = dA.masked_fill_(A <= 0, 0.0)
        dS1 = self._plan(I, W, T, "f32")(mx_quantize(dH, f, transpose=True),
                                         mx_quantize(X, f, transpose=True), *to1)
        dX = self._plan(T, W, I)(mx_quantize(dH, f), mx_quantize(self.S1, f, transpose=True))
        return dX, dS1, dS2


class ExpertBlock:
    """A layer of a model: h = X + residual, z = norm(h) * norm_weight, and Y the sum of the
    experts' layer and of the shared expert on z.  The next block takes (Y, h).

    The weights' gradients (fp32) are the block's own tensors ``grads``, written anew by every
    ``backward``; ``clip`` scales them to a length."""

    def __init__(self, layer, shared, norm_weight, eps=1e-6):
        import torch
        self.layer, self.shared, self.norm_weight, self.eps = layer, shared, norm_weight, eps
        like = (layer.W1, layer.W2, shared.S1, shared.S2, norm_weight)
        self.grads = [torch.empty(t.shape, dtype=torch.float32, device=t.device) for t in like]
        self.clip = GradClip(self.grads)

    def device_status(self):
        return self.shared.device_status() or self.layer.device_status()

    def forward(self, X, residual, ids, weights):
        """(Y, H, saved)."""
        Z, H, Q = rms_norm(X, self.norm_weight, residual=residual, eps=self.eps,
                           format=self.shared.format)
        Y, routed = self.layer.forward(Z, ids, weights)
        S, A = self.shared.forward(Q)
        return Y.add_(S), H, (H, Z, A, routed)

    def backward(self, dY, dH, saved):
        """(dX, dweights) with dX the gradient of X and of the residual; dH is the gradient
        that reaches H by its other uses (None: none).  Writes ``grads``."""
        H, Z, A, routed = saved
        g1, g2, s1, s2, gn = self.grads
        dZ, dweights, _, _ = self.layer.backward(dY, routed, (g1, g2))
        dS, _, _ = self.shared.backward(dY, A, Z, (s1, s2))
        dX, _ = rms_norm_grad(dZ.add_(dS), H, self.norm_weight, dH=dH, eps=self.eps, dweight=gn)
        return dX, dweights

    def update(self, rate):
        """A plain gradient step of all weights."""
        w = (self.layer.W1, self.layer.W2, self.shared.S1, self.shared.S2, self.norm_weight)
        for t, g in zip(w, self.grads):
            t.sub_(g, alpha=rate)
        self.shared.quantize()

    def decode(self, X, residual, ids, weights):
        """(Y, H) for a few tokens, the experts' weights in 4 bits (``layer.pack``)."""
        Z, H, Q = rms_norm(X, self.norm_weight, residual=residual, eps=self.eps,
                           format=self.shared.format)
        Y = self.layer.decode(Z, ids, weights)
        return Y.add_(self.shared.forward(Q)[0]), H


def random_block(experts, width, inner, topk, shared, format="mxfp8", seed=0):
    import torch
    layer = random_layer(experts, width, inner, topk, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    S1 = torch.randn((shared, width), generator=g, device="cuda") * width ** -0.5
    S2 = torch.randn((width, shared), generator=g, device="cuda") * shared ** -0.5
    norm = 1.0 + 0.1 * torch.randn((width,), generator=g, device="cuda")
    return ExpertBlock(layer, SharedExpert(S1.half(), S2.half(), format), norm.half())


def random_layer(experts, width, inner, topk, seed=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    W1 = torch.randn((experts, inner, width), generator=g, device="cuda") * width ** -0.5
    W2 = torch.randn((experts, width, inner), generator=g, device="cuda") * inner ** -0.5
    return ExpertLayer(W1.half(), W2.half(), topk)


def random_batch(tokens, topk, experts, width, seed=1):
    """X, ids and routing weights that sum to one per token."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    X = torch.randn((tokens, width), generator=g, device="cuda").half()
    top, ids = torch.randn((tokens, experts), generator=g, device="cuda").topk(topk, dim=1)
    return X, ids.to(torch.int32).contiguous(), torch.softmax(top, dim=1).contiguous()


def _milliseconds(fn, steps):
    import torch
    for _ in range(3):
        fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(steps):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / steps


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 8192), ("topk", 4), ("experts", 16), ("width", 2048),
                        ("inner", 4096), ("steps", 10), ("decode", 4), ("shared", 4096)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--format", choices=("mxfp8", "mxfp4", "nvfp4"), default="mxfp8")
    ap.add_argument("--clip", type=float, default=1.0)
    a = ap.parse_args(argv)
    layer = random_layer(a.experts, a.width, a.inner, a.topk)
    X, ids, weights = random_batch(a.tokens, a.topk, a.experts, a.width)

    def train():
        Y, saved = layer.forward(X, ids, weights)
        dX, dweights, dW1, dW2 = layer.backward(Y, saved)  # loss = sum(Y^2) / 2
        layer.W1.sub_(dW1.mul_(1e-6))
        layer.W2.sub_(dW2.mul_(1e-6))

    ms = _milliseconds(train, a.steps)
    flops = 6.0 * 2.0 * a.tokens * a.topk * a.width * a.inner
    print("training step: %d tokens x %d of %d experts, %d -> %d -> %d: %.3f ms, %.0f TFLOP/s"
          % (a.tokens, a.topk, a.experts, a.width, a.inner, a.width, ms, flops / ms * 1e-9))

    layer.pack()
    x, i, w = random_batch(a.decode, a.topk, a.experts, a.width, seed=2)
    ms = _milliseconds(lambda: layer.decode(x, i, w), 10 * a.steps)
    exact, _ = layer.forward(x, i, w)
    coded = layer.decode(x, i, w)
    status = layer.device_status()
    if status != 0:
        raise GemmError(status, "a wait inside a kernel ran out")
    off = float((coded.float() - exact.float()).norm() / exact.float().norm())
    print("decoding step: %d tokens with 4-bit weights: %.1f us, %.3f of the fp16 layer's norm off"
          % (a.decode, ms * 1e3, off))
    if a.shared > 0:
        _run_block(a, X, ids, weights, x, i, w)


def _run_block(a, X, ids, weights, x, i, w):
    block = random_block(a.experts, a.width, a.inner, a.topk, a.shared, a.format)
    residual = X.flip(0)
    norms = []

    def train():
        Y, H, saved = block.forward(X, residual, ids, weights)
        block.backward(Y, H, saved)  # loss = (sum(Y^2) + sum(H^2)) / 2
        norms[:] = [block.clip(a.clip)]
        block.update(1e-3)

    ms = _milliseconds(train, a.steps)
    flops = 6.0 * 2.0 * a.tokens * a.width * (a.topk * a.inner + a.shared)
    status = block.device_status()
    if status != 0:
        raise GemmError(status, "a wait inside a kernel ran out")
    print("block's training step: norm, experts, shared expert of %d in %s, clipping to %g of %.3g"
          ": %.3f ms, %.0f TFLOP/s" % (a.shared, a.format, a.clip, float(norms[0]), ms,
                                     flops / ms * 1e-9))
    block.layer.pack()
    ms = _milliseconds(lambda: block.decode(x, x, i, w), 10 * a.steps)
    print("block's decoding step: %d tokens: %.1f us" % (a.decode, ms * 1e3))


if __name__ == "__main__":
    main()
