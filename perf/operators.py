"""Cases for measuring the expert-layer operators: tokens sorted by expert and
back (with routing weights and their gradient), the experts' grouped products
with their gradients, and matrix-vector products with 4-bit weights.

``listed()`` names the measured cases and ``draw(rng)`` makes more of the same
ranges; ``prepare`` makes a case's inputs, ``run`` makes one pass (``own``
selects the library's kernels or the plain form in elementary torch
operations), ``exact`` gives the same outputs in 64 bits and ``work`` the bytes
and operations that a pass cannot do without.
"""
import math

import torch

own = False

DEVICE = "cuda"

# The largest listed cases; drawn cases stay within them.
MAX_MOVED = 16384 * 8 * 2048      # elements of the sorted copy of the tokens
MAX_GROUPED_FLOPS = 2 * 16384 * 4096 * 4096
MAX_W4_WEIGHTS = 16384 * 16384
MAX_BYTES = 1.19e9


def listed():
    return [
        # Routing of one decoding step: a batch of 16 sequences, 8 experts per
        # token out of 64.  A few hundred KB: latency is what counts.
        dict(name="dispatch_decode", op="dispatch", tokens=16, topk=8, experts=64, width=4096,
             drop=0.0),
        # Routing of a training or prompt batch, with 3 % of the slots dropped
        # (capacity limits or padding tokens): the sorted copy is 0.5 GB.
        dict(name="dispatch_prompt", op="dispatch", tokens=16384, topk=8, experts=128,
             width=2048, drop=0.03),
        # Experts' outputs back to their tokens, 3 decoding tokens, odd counts.
        dict(name="combine_decode", op="combine", tokens=3, topk=6, experts=160, width=5120,
             drop=0.0, weighted=True, out="f16"),
        # Gradient of the weighted combination over a training batch: the
        # gradient of every expert row and of every routing weight.
        dict(name="combine_grad_train", op="combine_grad", tokens=16384, topk=4, experts=64,
             width=4096, drop=0.02),
        # Experts' product of a training batch: 16 experts of 4096 x 4096,
        # about a thousand rows each.
        dict(name="grouped_forward_train", op="grouped_forward", rows=16384, experts=16, N=4096,
             K=4096, out="f16", skew=0.5),
        # Few rows over many experts, some of them without any, odd sizes,
        # fp32 output: the experts' product of a short prompt.
        dict(name="grouped_forward_short", op="grouped_forward", rows=777, experts=40, N=1416,
             K=2056, out="f32", skew=1.5),
        # Gradient with respect to the rows (contraction over the outputs).
        dict(name="grouped_grad_input", op="grouped_grad_input", rows=8192, experts=32, N=2816,
             K=2048, out="f16", skew=0.5),
        # Gradient of the experts' weights (contraction over each expert's own
        # rows, whose number is odd and differs), fp32 for the optimiser.
        dict(name="grouped_grad_weight", op="grouped_grad_weight", rows=16384, experts=16,
             N=2048, K=4096, out="f32", skew=0.5),
        # One decoding token through a 4-bit 16384 x 16384 matrix (the skinny
        # workload's weights): 134 MB of codes, bound by memory.
        dict(name="w4_one_token", op="w4", M=1, N=16384, K=16384, group=128, zeros=False,
             out="f16"),
        # The skinny workload's 64 rows on a smaller matrix, groups of 32 with
        # zero points, fp32 output.
        dict(name="w4_batch", op="w4", M=64, N=8192, K=4096, group=32, zeros=True, out="f32"),
        # A prompt through 4-bit weights: the product, not the weights, counts.
        dict(name="w4_prompt", op="w4", M=2000, N=4096, K=4096, group=64, zeros=True, out="f16"),
        # Four decoding tokens through 8 of 64 experts each, 4-bit experts.
        dict(name="w4_experts_decode", op="w4_experts", tokens=4, topk=8, experts=64, N=2048,
             K=4096, group=128, zeros=False, out="f16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(value, m):
    return max(m, value // m * m)


def draw(rng):
    while True:
        case = _draw(rng)
        if work(case)["bytes"] <= MAX_BYTES and 3072 not in case.values():
            return case


def _draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "grouped_forward",
                     "grouped_grad_input", "grouped_grad_weight", "w4", "w4_experts"])
    if op in ("dispatch", "combine", "combine_grad"):
        experts = _log_int(rng, 2, 256)
        topk = rng.randint(1, min(8, experts))
        tokens = _log_int(rng, 1, 32768)
        width = _mult(_log_int(rng, 64, 8192), 8)
        tokens = max(1, min(tokens, MAX_MOVED // (topk * width)))
        case = dict(op=op, tokens=tokens, topk=topk, experts=experts, width=width,
                    drop=rng.choice([0.0, 0.03, 0.3]))
        if op == "combine":
            case.update(weighted=rng.random() < 0.7, out=rng.choice(["f16", "f32"]))
        return case
    if op.startswith("grouped"):
        N = _mult(_log_int(rng, 64, 4096), 8)
        K = _mult(_log_int(rng, 64, 4096), 8)
        rows = _log_int(rng, 1, 32768)
        rows = max(1, min(rows, MAX_GROUPED_FLOPS // (2 * N * K)))
        return dict(op=op, rows=rows, experts=_log_int(rng, 1, 96), N=N, K=K,
                    out=rng.choice(["f16", "f32"]), skew=rng.choice([0.0, 0.5, 1.5]))
    group = rng.choice([32, 64, 128])
    K = _mult(_log_int(rng, 256, 16384), group)
    N = _mult(_log_int(rng, 64, 16384), 8)
    if op == "w4":
        M = _log_int(rng, 1, 2048)
        out = "f16" if M > 64 else rng.choice(["f16", "f32"])
        if M > 64:  # keep the plain form's product within the largest case's
            N = min(N, 8192)
            K = min(K, 8192)
        return dict(op=op, M=M, N=N, K=K, group=group, zeros=rng.random() < 0.5, out=out)
    experts = _log_int(rng, 2, 64)
    while experts * N * K > MAX_W4_WEIGHTS * 4:
        N = _mult(N // 2, 8)
    return dict(op=op, tokens=_log_int(rng, 1, 16), topk=rng.randint(1, min(8, experts)),
                experts=experts, N=N, K=K, group=group, zeros=rng.random() < 0.5,
                out=rng.choice(["f16", "f32"]))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=torch.float16, scale=1.0):
    x = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)
    return (x * scale).to(dtype)


def _routing(case, g):
    """Expert ids (topk different ones per token, some experts more popular
    than others, dropped slots -1) and routing weights that sum to one over a
    token's slots."""
    T, k, E = case["tokens"], case["topk"], case["experts"]
    bias = torch.randn((1, E), generator=g, device=DEVICE) * 0.5
    logits = torch.randn((T, E), generator=g, device=DEVICE) + bias
    top, ids = logits.topk(k, dim=1)
    ids = ids.to(torch.int32)
    weights = torch.softmax(top, dim=1)
    if case.get("drop", 0.0) > 0.0:
        lost = torch.rand((T, k), generator=g, device=DEVICE) < case["drop"]
        ids = torch.where(lost, torch.full_like(ids, -1), ids)
    return ids.contiguous(), weights.contiguous()


def _sorted_positions(ids, experts):
    """Offsets, order and position of a stable sort by expert, dropped slots
    last, from comparisons and sums alone."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= experts), torch.full_like(flat, experts), flat)
    hit = (key[:, None] == torch.arange(experts + 1, device=flat.device)[None, :])
    upto = hit.to(torch.int32).cumsum(0, dtype=torch.int32)
    counts = upto[-1].long()
    ends = counts.cumsum(0)
    starts = ends - counts
    rank = upto.gather(1, key[:, None])[:, 0].long() - 1
    position = starts[key] + rank
    order = torch.empty_like(position)
    order[position] = torch.arange(flat.numel(), device=flat.device)
    return (starts.to(torch.int32), order.to(torch.int32),
            position.to(torch.int32).reshape(ids.shape))


def _expert_counts(case, g):
    """Rows per expert: a skewed share each, the remainder to the first."""
    E, R = case["experts"], case["rows"]
    w = torch.exp(torch.randn(E, generator=g, device=DEVICE).double() * case["skew"]).cpu()
    counts = torch.floor(w / w.sum() * R).long()
    counts[0] += R - int(counts.sum())
    return counts


def _dtype(out):
    return torch.float16 if out == "f16" else torch.float32


def _codes(g, E, N, K, group, zeros):
    """4-bit codes packed two to a byte (low half first), one fp16 scale per
    group of `group` weights and, with `zeros`, an integer zero point each."""
    packed = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEVICE, dtype=torch.uint8)
    scales = (torch.rand((E, N, K // group), generator=g, device=DEVICE) + 0.5)
    scales = (scales * (0.2 / math.sqrt(K))).to(torch.float16)
    z = None
    if zeros:
        z = torch.randint(5, 11, (E, N, K // group), generator=g, device=DEVICE,
                          dtype=torch.uint8)
    return packed, scales, z


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = dict(case=case)
    if own:
        import tma_pipelined_tensor_fp16_gb300 as tg
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, E, W = case["tokens"], case["topk"], case["experts"], case["width"]
        ids, weights = _routing(case, g)
        st.update(ids=ids, weights=weights)
        if op == "dispatch":
            st["X"] = _normal(g, (T, W))
        else:
            st["offsets"], st["order"], st["position"] = _sorted_positions(ids, E)
            st["Ys"] = _normal(g, (T * k, W))
        if op == "combine_grad":
            st["dY"] = _normal(g, (T, W))
        if own:
            route = tg.ExpertRoute(T, k, E)
            if op != "dispatch":
                route.load(st["offsets"], st["order"], st["position"])
            st["route"] = route
            if op == "dispatch":
                st["Xs"] = torch.empty((T * k, W), dtype=torch.float16, device=DEVICE)
            elif op == "combine":
                st["Y"] = torch.empty((T, W), dtype=_dtype(case["out"]), device=DEVICE)
            else:
                st["dYs"] = torch.empty((T * k, W), dtype=torch.float16, device=DEVICE)
                st["dweights"] = torch.empty((T, k), dtype=torch.float32, device=DEVICE)
        return st
    if op.startswith("grouped"):
        R, E, N, K = case["rows"], case["experts"], case["N"], case["K"]
        counts = _expert_counts(case, g)
        st["counts"] = counts.tolist()
        ends = counts.cumsum(0)
        st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long), ends]).to(
            device=DEVICE, dtype=torch.int32)
        if op != "grouped_grad_input":
            st["A"] = _normal(g, (R, K))
        if op != "grouped_forward":
            st["dC"] = _normal(g, (R, N))
        if op != "grouped_grad_weight":
            st["B"] = _normal(g, (E, N, K), scale=1.0 / math.sqrt(K))
        if own:
            kind = op[len("grouped_"):]
            st["plan"] = tg.GroupedPlan(R, N, K, E, op=kind, out=case["out"])
            shape = {"forward": (R, N), "grad_input": (R, K), "grad_weight": (E, N, K)}[kind]
            st["C"] = torch.empty(shape, dtype=_dtype(case["out"]), device=DEVICE)
        return st
    N, K, group = case["N"], case["K"], case["group"]
    if op == "w4":
        M, E = case["M"], 1
        st["X"] = _normal(g, (M, K))
    else:
        E = case["experts"]
        M = case["tokens"] * case["topk"]
        st["X"] = _normal(g, (case["tokens"], K))
        st["ids"], _ = _routing(case, g)
    packed, scales, zeros = _codes(g, E, N, K, group, case["zeros"])
    if op == "w4":
        packed, scales = packed[0], scales[0]
        zeros = zeros[0] if zeros is not None else None
    st.update(packed=packed, scales=scales, zeros=zeros)
    if own:
        if op == "w4":
            st["plan"] = tg.W4Plan(M, N, K, group=group, out=case["out"])
        else:
            st["plan"] = tg.W4Plan(M, N, K, group=group, out=case["out"], experts=E,
                                   share=case["topk"])
        st["Y"] = torch.empty((M, N), dtype=_dtype(case["out"]), device=DEVICE)
    return st


# -------------------------------------------------------------------- passes

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    case = st["case"]
    op = case["op"]
    if op == "dispatch":
        route = st["route"].sort(st["ids"])
        Xs = route.gather(st["X"], st["Xs"])
        return [route.offsets, route.order, route.position, Xs]
    if op == "combine":
        return [st["route"].combine(st["Ys"], st["Y"],
                                    weights=st["weights"] if case["weighted"] else None)]
    if op == "combine_grad":
        return list(st["route"].combine_grad(st["dY"], st["Ys"], st["weights"], st["dYs"],
                                             st["dweights"]))
    if op == "grouped_forward":
        return [st["plan"](st["A"], st["B"], st["offsets"], st["C"])]
    if op == "grouped_grad_input":
        return [st["plan"](st["dC"], st["B"], st["offsets"], st["C"])]
    if op == "grouped_grad_weight":
        return [st["plan"](st["dC"], st["A"], st["offsets"], st["C"])]
    if op == "w4":
        return [st["plan"](st["X"], st["packed"], st["scales"], st["Y"], zeros=st["zeros"])]
    return [st["plan"](st["X"], st["packed"], st["scales"], st["Y"], zeros=st["zeros"],
                       ids=st["ids"])]


def _segments(counts):
    r = 0
    for e, c in enumerate(counts):
        yield e, r, r + c
        r += c


def _weights_f32(packed, scales, zeros, group):
    lo = (packed & 15).float()
    hi = (packed >> 4).float()
    q = torch.stack([lo, hi], dim=-1).reshape(packed.shape[:-1] + (-1, group))
    z = 8.0 if zeros is None else zeros.float()[..., None]
    w = (q - z) * scales.float()[..., None]
    return w.reshape(packed.shape[:-1] + (-1,))


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "dispatch":
        offsets, order, position = _sorted_positions(st["ids"], case["experts"])
        Xs = st["X"][(order // case["topk"]).long()]
        inside = torch.arange(Xs.shape[0], device=Xs.device) < offsets[-1]
        Xs = torch.where(inside[:, None], Xs, torch.zeros_like(Xs))
        return [offsets, order, position, Xs]
    if op == "combine":
        T, k = case["tokens"], case["topk"]
        y = torch.zeros((T, case["width"]), device=DEVICE)
        total = st["offsets"][-1]
        for j in range(k):
            pos = st["position"][:, j]
            rows = st["Ys"][pos.long()].float()
            if case["weighted"]:
                rows = rows * st["weights"][:, j:j + 1]
            y += torch.where((pos < total)[:, None], rows, torch.zeros_like(rows))
        return [y.to(_dtype(case["out"]))]
    if op == "combine_grad":
        T, k = case["tokens"], case["topk"]
        total = st["offsets"][-1]
        dY = st["dY"].float()
        dYs = torch.empty_like(st["Ys"])
        dw = torch.empty((T, k), device=DEVICE)
        for j in range(k):
            pos = st["position"][:, j]
            kept = (pos < total)[:, None]
            rows = st["Ys"][pos.long()].float()
            dw[:, j] = torch.where(kept, rows * dY, torch.zeros_like(rows)).sum(1)
            grad = torch.where(kept, dY * st["weights"][:, j:j + 1], torch.zeros_like(dY))
            dYs[pos.long()] = grad.half()
        return [dYs, dw]
    if op.startswith("grouped"):
        R, E, N, K = case["rows"], case["experts"], case["N"], case["K"]
        dt = _dtype(case["out"])
        if op == "grouped_grad_weight":
            out = torch.zeros((E, N, K), dtype=dt, device=DEVICE)
            for e, r0, r1 in _segments(st["counts"]):
                out[e] = (st["dC"][r0:r1].float().t() @ st["A"][r0:r1].float()).to(dt)
            return [out]
        out = torch.zeros((R, N if op == "grouped_forward" else K), dtype=dt, device=DEVICE)
        for e, r0, r1 in _segments(st["counts"]):
            if r1 == r0:
                continue
            w = st["B"][e].float()
            if op == "grouped_forward":
                out[r0:r1] = (st["A"][r0:r1].float() @ w.t()).to(dt)
            else:
                out[r0:r1] = (st["dC"][r0:r1].float() @ w).to(dt)
        return [out]
    dt = _dtype(case["out"])
    if op == "w4":
        w = _weights_f32(st["packed"], st["scales"], st["zeros"], case["group"])
        return [(st["X"].float() @ w.t()).to(dt)]
    T, k, N = case["tokens"], case["topk"], case["N"]
    idx = st["ids"].reshape(-1).long()
    y = torch.empty((T * k, N), dtype=dt, device=DEVICE)
    x = st["X"].float()
    z = st["zeros"]
    for s in range(T * k):
        e = idx[s:s + 1]
        w = _weights_f32(st["packed"][e][0], st["scales"][e][0], None if z is None else z[e][0],
                         case["group"])
        y[s] = (w @ x[s // k]).to(dt)
    return [y]


# ---------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, E, W = case["tokens"], case["topk"], case["experts"], case["width"]
        S = T * k
        kept = S * (1.0 - case["drop"])
        if op == "dispatch":
            # ids, offsets, order, position; tokens read once, sorted rows written
            return dict(bytes=4 * S + 4 * (E + 1) + 8 * S + 2 * T * W + 2 * S * W, flops=S)
        if op == "combine":
            out = 2 if case["out"] == "f16" else 4
            return dict(bytes=2 * kept * W + 8 * S + out * T * W, flops=2 * kept * W)
        return dict(bytes=2 * T * W + 2 * kept * W + 2 * S * W + 12 * S, flops=3 * kept * W)
    if op.startswith("grouped"):
        R, E, N, K = case["rows"], case["experts"], case["N"], case["K"]
        out = 2 if case["out"] == "f16" else 4
        flops = 2 * R * N * K
        if op == "grouped_forward":
            return dict(bytes=2 * R * K + 2 * min(E, R) * N * K + out * R * N, flops=flops)
        if op == "grouped_grad_input":
            return dict(bytes=2 * R * N + 2 * min(E, R) * N * K + out * R * K, flops=flops)
        return dict(bytes=2 * R * (N + K) + out * E * N * K, flops=flops)
    N, K, group = case["N"], case["K"], case["group"]
    per_matrix = N * K / 2 + N * (K // group) * (3 if case["zeros"] else 2)
    out = 2 if case["out"] == "f16" else 4
    if op == "w4":
        M = case["M"]
        return dict(bytes=per_matrix + 2 * M * K + out * M * N, flops=2 * M * N * K)
    T, k, E = case["tokens"], case["topk"], case["experts"]
    S = T * k
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token takes
    return dict(bytes=used * per_matrix + 2 * T * K + out * S * N, flops=2 * S * N * K)


# ------------------------------------------------------------- 64-bit values

def _exact_dispatch(case, st):
    k, E = case["topk"], case["experts"]
    flat = st["ids"].reshape(-1).cpu().tolist()
    lists = [[] for _ in range(E + 1)]
    for slot, e in enumerate(flat):
        lists[e if 0 <= e < E else E].append(slot)
    order, starts = [], []
    for members in lists:
        starts.append(len(order))
        order.extend(members)
    position = [0] * len(flat)
    for p, slot in enumerate(order):
        position[slot] = p
    src = torch.tensor(order, device=DEVICE, dtype=torch.long)
    Xs = st["X"].double().index_select(0, torch.div(src, k, rounding_mode="floor"))
    Xs[starts[E]:] = 0.0
    return [torch.tensor(starts, dtype=torch.int32, device=DEVICE), src.to(torch.int32),
            torch.tensor(position, dtype=torch.int32, device=DEVICE).reshape(st["ids"].shape),
            Xs]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        return _exact_dispatch(case, st)
    if op in ("combine", "combine_grad"):
        T, k = case["tokens"], case["topk"]
        total = int(st["offsets"][-1])
        w = st["weights"].double()
        if op == "combine" and not case["weighted"]:
            w = torch.ones_like(w)
        kept = st["position"] < total
        w = w * kept
        step = max(1, (1 << 26) // (k * case["width"]))
        if op == "combine":
            y = torch.empty((T, case["width"]), dtype=torch.float64, device=DEVICE)
            for t0 in range(0, T, step):
                rows = st["Ys"][st["position"][t0:t0 + step].long()].double()
                y[t0:t0 + step] = torch.einsum("tk,tkw->tw", w[t0:t0 + step], rows)
            return [y]
        dYs = torch.zeros((T * k, case["width"]), dtype=torch.float64, device=DEVICE)
        dw = torch.zeros((T, k), dtype=torch.float64, device=DEVICE)
        for t0 in range(0, T, step):
            pos = st["position"][t0:t0 + step].long()
            dY = st["dY"][t0:t0 + step].double()
            dw[t0:t0 + step] = torch.einsum("tkw,tw->tk", st["Ys"][pos].double(), dY) \
                * kept[t0:t0 + step]
            dYs[pos.reshape(-1)] = torch.einsum("tk,tw->tkw", w[t0:t0 + step], dY).reshape(
                -1, case["width"])
        return [dYs, dw]
    if op.startswith("grouped"):
        ends = st["offsets"].cpu().tolist()
        parts = []
        for e in range(case["experts"]):
            s = slice(ends[e], ends[e + 1])
            if op == "grouped_grad_weight":
                parts.append(torch.einsum("rn,rk->nk", st["dC"][s].double(),
                                          st["A"][s].double()))
            elif op == "grouped_forward":
                parts.append(torch.einsum("rk,nk->rn", st["A"][s].double(), st["B"][e].double()))
            else:
                parts.append(torch.einsum("rn,nk->rk", st["dC"][s].double(), st["B"][e].double()))
        if op == "grouped_grad_weight":
            return [torch.stack(parts)]
        return [torch.cat(parts)]
    N, K, group = case["N"], case["K"], case["group"]
    shape = st["scales"].shape
    flat = st["packed"].reshape(-1, K // 2)
    scales = st["scales"].reshape(flat.shape[0], -1)
    zeros = st["zeros"].reshape(flat.shape[0], -1) if st["zeros"] is not None else None

    def product(row0, x):
        """Rows row0 .. row0 + N of the stacked weights times x, in 64 bits."""
        y = torch.empty((x.shape[0], N), dtype=torch.float64, device=DEVICE)
        for n0 in range(0, N, 1024):
            r = slice(row0 + n0, row0 + min(n0 + 1024, N))
            w = torch.empty((r.stop - r.start, K), dtype=torch.float64, device=DEVICE)
            w[:, 0::2] = torch.remainder(flat[r].to(torch.int32), 16).double()
            w[:, 1::2] = torch.div(flat[r].to(torch.int32), 16, rounding_mode="floor").double()
            s = scales[r].double().repeat_interleave(group, dim=1)
            z = 8.0 if zeros is None else zeros[r].double().repeat_interleave(group, dim=1)
            y[:, n0:n0 + w.shape[0]] = x @ ((w - z) * s).t()
        return y

    x = st["X"].double()
    if op == "w4":
        return [product(0, x)]
    assert shape[0] == case["experts"]
    k = case["topk"]
    idx = st["ids"].reshape(-1).cpu().tolist()
    y = torch.empty((len(idx), N), dtype=torch.float64, device=DEVICE)
    for e in sorted(set(idx)):
        rows = [s for s, v in enumerate(idx) if v == e]
        y[rows] = product(e * N, x[[s // k for s in rows]])
    return [y]
