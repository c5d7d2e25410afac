"""A mixture-of-experts feed-forward on the library's operators, and a command
that runs it: a training step (forward, both gradients of every operator, an
update) and decoding with the experts' weights in 4 bits.

    python -m tma_pipelined_tensor_fp16_gb300.expert_layer [--tokens 8192]
        [--topk 4] [--experts 16] [--width 2048] [--inner 4096] [--steps 10]
        [--decode 4]

Y[t] = sum_j w[t, j] * W2[e] . relu(W1[e] . X[t]),  e = ids[t, j]: the slots are
sorted by expert, the tokens gathered, both products run grouped by expert, and
the experts' rows are summed back with their routing weights.  Prints the time
of a training step and of a decoding step, and how far the decoding step with
4-bit weights is from the same step with fp16 weights.
"""
import argparse

from .binding import GemmError
from .experts import ExpertRoute, GroupedPlan, W4Plan, w4_pack


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

    def backward(self, dY, saved):
        """Gradients (dX, dweights, dW1, dW2); the weights' in fp32.  `saved` stays as
        it is, so the same forward can be differentiated again."""
        route, Xs, H, A, Ys, weights = saved
        rows, I, W = Xs.shape[0], self.inner, self.width
        dYs, dweights = route.combine_grad(dY, Ys, weights)
        dW2 = self._plan(rows, W, I, "grad_weight", "f32")(dYs, A, route.offsets)
        dA = self._plan(rows, W, I, "grad_input")(dYs, self.W2, route.offsets)
        dH = dA.masked_fill_(H <= 0, 0.0)  # not a product: dA need not be finite there
        dW1 = self._plan(rows, I, W, "grad_weight", "f32")(dH, Xs, route.offsets)
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
                        ("inner", 4096), ("steps", 10), ("decode", 4)):
        ap.add_argument("--" + name, type=int, default=value)
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


if __name__ == "__main__":
    main()
