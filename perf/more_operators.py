"""Measured cases of the cross entropy loss and of the product in 8-bit integers.

Four operators, each in a plain form (elementary torch operations in 32 bits) and,
where ``own`` is true, as the package's calls:

  loss      cross_entropy: from hidden states and the LM head's weight, the weighted loss
            with label smoothing and z loss, the log-sum-exp of every row and the weights' sum
  gradient  cross_entropy_backward: the gradients of the loss with respect to both
  linear    linear_int8: y = x . W^T for W held as 8-bit whole numbers with a scale per
            channel, x quantised per token within the call or given as such numbers
  quantize  quantize_int8 and dequantize_int8: a matrix to 8 bits, a scale per row, and back
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "int8": torch.int8}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1}
INV_TEMP = float(np.float32(1 / 0.7))


def listed():
    return [
        # A unit test's model, one short sequence: the loss's latency.
        dict(name="loss_tiny_64", op="loss", T=64, H=256, V=1024, weighted=False, reduction="mean",
             smoothing=0.0, z_loss=0.0, inv_temp=1.0),
        # A ragged evaluation batch on an odd vocabulary: a loss for every token, smoothed.
        dict(name="loss_ragged_300", op="loss", T=300, H=1032, V=32761, weighted=True,
             reduction="none", smoothing=0.1, z_loss=1e-4, inv_temp=INV_TEMP),
        # A fine-tuning batch (8 packed sequences of 512), prompts masked out by weights.
        dict(name="loss_train_4096", op="loss", T=4096, H=4096, V=151936, weighted=True,
             reduction="mean", smoothing=0.0, z_loss=1e-4, inv_temp=1.0),
        # The unit test's model again: the gradients' latency.
        dict(name="gradient_tiny_64", op="gradient", T=64, H=256, V=1024, weighted=False,
             reduction="mean", smoothing=0.0, z_loss=0.0, inv_temp=1.0),
        # A small ragged batch: odd vocabulary, smoothed, a gradient for every token's loss.
        dict(name="gradient_ragged_130", op="gradient", T=130, H=1032, V=50001, weighted=True,
             reduction="none", smoothing=0.1, z_loss=1e-4, inv_temp=INV_TEMP),
        # The fine-tuning batch's gradients.
        dict(name="gradient_train_4096", op="gradient", T=4096, H=4096, V=151936, weighted=True,
             reduction="mean", smoothing=0.0, z_loss=1e-4, inv_temp=1.0),
        # One new token through the LM head in 8 bits: fp32 logits.
        dict(name="linear_head_1", op="linear", T=1, N=151936, K=4096, x="bf16", out="fp32"),
        # A decode batch of 64 through it.
        dict(name="linear_head_64", op="linear", T=64, N=151936, K=4096, x="bf16", out="fp32"),
        # A small decode batch through an odd-sized projection whose tokens an earlier call
        # has quantised.
        dict(name="linear_proj_13_ragged", op="linear", T=13, N=5119, K=5152, x="int8", out="fp16"),
        # A prefill batch through a wide projection.
        dict(name="linear_prefill_4096", op="linear", T=4096, N=16384, K=4096, x="bf16", out="bf16"),
        # A new policy's LM head after a training step, quantised for the rollout engine.
        dict(name="quantize_head", op="quantize", N=151936, K=4096, dtype="bf16"),
        # A small odd projection.
        dict(name="quantize_proj_ragged", op="quantize", N=1009, K=2080, dtype="fp16"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm: odd, or eight times an odd
    one, where it is over 64."""
    n = min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))
    return n if n <= 64 else min(high, rng.choice([n | 1, 8 * (n // 8 | 1)]))


def draw(rng):
    op = rng.choice(["loss", "loss", "gradient", "gradient", "linear", "linear", "linear",
                     "quantize"])
    if op in ("loss", "gradient"):
        V = rng.choice([151936, 32768, _spread(rng, 500, 151936), _spread(rng, 500, 151936)])
        H = 8 * rng.choice([512, rng.randrange(8, 513), rng.randrange(8, 513)])
        return dict(op=op, T=_spread(rng, 1, 4096), H=H, V=V, weighted=rng.random() < 0.6,
                    reduction=rng.choice(["mean", "mean", "sum", "none"]),
                    smoothing=rng.choice([0.0, 0.0, 0.1]), z_loss=rng.choice([0.0, 1e-4]),
                    inv_temp=rng.choice([1.0, 1.0, INV_TEMP]))
    K = 16 * rng.choice([256, rng.randrange(16, 400), rng.randrange(16, 400)])
    if op == "quantize":
        N = min(_spread(rng, 500, 151936), 151936 * 4096 // K)
        return dict(op=op, N=N, K=K, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    x = rng.choice(["bf16", "bf16", "fp16", "int8"])
    out = rng.choice(["fp32", x if x != "int8" else "bf16"])
    T = _spread(rng, 1, 4096) if rng.random() < 0.5 else _spread(rng, 1, 64)
    most = min(151936, 151936 * 4096 // K) if T <= 64 else min(151936, 4096 * 16384 * 4096 // (T * K))
    return dict(op=op, T=T, N=_spread(rng, 500, max(500, most)), K=K, x=x, out=out)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if case["op"] in ("loss", "gradient"):
        return _prepare_loss(case, g)
    if case["op"] == "quantize":
        return dict(op="quantize", W=_normal(case["N"], case["K"], 0.02, DTYPES[case["dtype"]], g))
    return _prepare_linear(case, g)


def _normal(rows, cols, std, dtype, g):
    W = torch.empty(rows, cols, dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        W[r:r + n] = (torch.randn(n, cols, generator=g, device="cuda") * std).to(dtype)
    return W


def _prepare_loss(case, g):
    """RMS-normalised hidden states that lean towards their token's row of the weight, so that
    most targets are likely tokens, a few rows ignored and, with weights, prompts at 0."""
    T, H, V = case["T"], case["H"], case["V"]
    W = _normal(V, H, 1.28 / math.sqrt(H), torch.bfloat16, g)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    lean = torch.rand(T, 1, generator=g, device="cuda") * (16 / (1.28 * math.sqrt(H)))
    h = torch.randn(T, H, generator=g, device="cuda") + lean * (W[targets].float() * (math.sqrt(H) / 1.28))
    h = (h * torch.rsqrt(h.pow(2).mean(1, keepdim=True))).to(torch.bfloat16)
    pick = torch.rand(T, generator=g, device="cuda")
    targets = torch.where(pick > 0.97, torch.full_like(targets, -100), targets).to(torch.int32)
    weights = None
    if case["weighted"]:
        weights = torch.rand(T, generator=g, device="cuda") + 0.5
        weights = torch.where(torch.rand(T, generator=g, device="cuda") < 0.3, 0.0, weights)
    state = dict(op=case["op"], h=h, W=W, targets=targets, weights=weights,
                 reduction=case["reduction"], smoothing=case["smoothing"], z_loss=case["z_loss"],
                 inv_temp=case["inv_temp"])
    if case["op"] == "gradient":
        # what the forward call left: the log-sum-exp and the weights' sum
        lse = torch.full((T,), -math.inf, device="cuda")
        step = max(1, (1 << 28) // T)
        for v in range(0, V, step):
            z = h.float() @ W[v:v + step].float().t()
            lse = torch.logaddexp(lse, torch.logsumexp(z * case["inv_temp"], 1))
        counted = (targets >= 0).float()
        state["lse"] = lse
        state["total"] = (counted if weights is None else counted * weights).sum()
        if case["reduction"] == "none":
            state["grad"] = torch.randn(T, generator=g, device="cuda") / T
        else:
            state["grad"] = torch.rand((), generator=g, device="cuda") + 0.5
    return state


def _prepare_linear(case, g):
    """Tokens with a few large features, as a transformer's have; the weight as a checkpoint
    holds it: codes and a scale per channel."""
    T, N, K = case["T"], case["N"], case["K"]
    codes = torch.empty(N, K, dtype=torch.int8, device="cuda")
    scales = torch.empty(N, device="cuda")
    step = max(1, (1 << 26) // K)
    for r in range(0, N, step):
        n = min(step, N - r)
        w = torch.randn(n, K, generator=g, device="cuda") * 0.02
        scales[r:r + n] = w.abs().amax(1) / 127
        codes[r:r + n] = torch.round(w / scales[r:r + n, None]).to(torch.int8)
    x = torch.randn(T, K, generator=g, device="cuda")
    x = x * torch.where(torch.rand(K, generator=g, device="cuda") < 0.002, 8.0, 1.0)
    x = x * torch.rsqrt(x.pow(2).mean(1, keepdim=True))
    x_scales = None
    if case["x"] == "int8":
        x_scales = x.abs().amax(1) / 127
        x = torch.round(x / x_scales[:, None])
    return dict(op="linear", x=x.to(DTYPES[case["x"]]), x_scales=x_scales, codes=codes,
                scales=scales, out=DTYPES[case["out"]])


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"loss": _plain_loss, "gradient": _plain_gradient, "linear": _plain_linear,
            "quantize": _plain_quantize}[state["op"]](state)


def _run_own(s):
    import invariant_token_logprob_gb300 as rlk
    if s["op"] == "loss":
        return tuple(rlk.cross_entropy(s["h"], s["W"], s["targets"], weights=s["weights"],
                                       inv_temp=s["inv_temp"], label_smoothing=s["smoothing"],
                                       z_loss=s["z_loss"], reduction=s["reduction"]))
    if s["op"] == "gradient":
        return rlk.cross_entropy_backward(s["h"], s["W"], s["targets"], s["lse"], s["grad"],
                                          total=s["total"], weights=s["weights"],
                                          inv_temp=s["inv_temp"], label_smoothing=s["smoothing"],
                                          z_loss=s["z_loss"], reduction=s["reduction"])
    if s["op"] == "linear":
        return rlk.linear_int8(s["x"], s["codes"], s["scales"], x_scales=s["x_scales"],
                               out_dtype=s["out"])
    codes, scales = rlk.quantize_int8(s["W"])
    return rlk.dequantize_int8(codes, scales, out_dtype=s["W"].dtype), scales


def _counted(s):
    """Whether a row has a token (truth values), and its weight (0 where it has none)."""
    t = s["targets"]
    inside = (t >= 0) & (t < s["W"].shape[0])
    weight = inside.float() if s["weights"] is None else torch.where(inside, s["weights"], 0.0)
    return inside & (weight != 0), weight


def _plain_loss(s):
    V = s["W"].shape[0]
    z = (s["h"].float() @ s["W"].float().t()) * s["inv_temp"]
    m = z.amax(1, keepdim=True)
    lse = m[:, 0] + torch.log(torch.exp(z - m).sum(1))
    zt = z.gather(1, s["targets"].long().clamp(0, V - 1)[:, None])[:, 0]
    loss = lse - (1 - s["smoothing"]) * zt + s["z_loss"] * lse * lse
    if s["smoothing"]:
        loss = loss - (s["smoothing"] / V) * z.sum(1)
    counted, weight = _counted(s)
    loss = torch.where(counted, weight * loss, 0.0)
    total = weight.sum()
    if s["reduction"] == "none":
        return loss, lse, total
    loss = loss.sum()
    if s["reduction"] == "mean":
        loss = torch.where(total > 0, loss / total, 0.0)
    return loss, lse, total


def _plain_gradient(s):
    V = s["W"].shape[0]
    h, W = s["h"].float(), s["W"].float()
    counted, weight = _counted(s)
    a = torch.where(counted, s["grad"] * weight, 0.0)
    if s["reduction"] == "mean":
        a = a / s["total"]
    lse = s["lse"][:, None]
    p = torch.exp((h @ W.t()) * s["inv_temp"] - lse)
    dz = p * (1 + 2 * s["z_loss"] * lse) - s["smoothing"] / V
    t = s["targets"].long().clamp(0, V - 1)[:, None]
    dz = dz.scatter_add(1, t, torch.full_like(lse, s["smoothing"] - 1))
    dz = torch.where(counted[:, None], dz * (a * s["inv_temp"])[:, None], 0.0)
    return (dz @ W).to(s["h"].dtype), (dz.t() @ h).to(s["W"].dtype)


def _quantized(x):
    """Codes (as fp32 whole numbers) and scales of x's rows.  (By a tensor: torch multiplies by
    the reciprocal of a plain number.)"""
    scales = x.abs().amax(1) / torch.full((), 127.0, device=x.device)
    scales = torch.where(scales == 0, 1.0, scales)
    return torch.round(x / scales[:, None]).clamp(-127, 127), scales


def _plain_linear(s):
    x, x_scales = s["x"].float(), s["x_scales"]
    if x_scales is None:
        x, x_scales = _quantized(x)
    y = x @ s["codes"].float().t()
    return (y * x_scales[:, None] * s["scales"]).to(s["out"])


def _plain_quantize(s):
    q, scales = _quantized(s["W"].float())
    return (q * scales[:, None]).to(s["W"].dtype), scales


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"loss": _exact_loss, "gradient": _exact_gradient, "linear": _exact_linear,
            "quantize": _exact_quantize}[s["op"]](s)


def _weights64(s):
    """Weights in 64 bits, 0 for rows that have no token."""
    T, V = s["h"].shape[0], s["W"].shape[0]
    w = torch.ones(T, dtype=torch.float64, device="cuda") if s["weights"] is None else s["weights"].double()
    w = w.clone()
    w[s["targets"] < 0] = 0
    w[s["targets"] >= V] = 0
    return w


def _exact_loss(s):
    """loss_t = (1 - e) (-log p_target) + e mean_v (-log p_v) + l lse^2."""
    T, V = s["h"].shape[0], s["W"].shape[0]
    W = s["W"].double()
    lse = torch.empty(T, dtype=torch.float64, device="cuda")
    loss = torch.zeros_like(lse)
    step = max(1, (1 << 27) // V)
    for r in range(0, T, step):
        z = torch.mm(s["h"][r:r + step].double(), W.t()).mul_(s["inv_temp"])
        n = z.shape[0]
        l = torch.logsumexp(z, 1)
        lse[r:r + n] = l
        t = s["targets"][r:r + n].long()
        row = ((t >= 0) & (t < V)).nonzero()[:, 0]
        nll = l[row] - z[row, t[row]]
        every = l[row] - z.mean(1)[row]
        loss[r + row] = (1 - s["smoothing"]) * nll + s["smoothing"] * every + s["z_loss"] * l[row] ** 2
    w = _weights64(s)
    total = w.sum()
    if s["reduction"] == "none":
        return loss * w, lse, total
    value = torch.dot(loss, w)
    if s["reduction"] == "mean":
        value = value / total if float(total) > 0 else torch.zeros_like(value)
    return value, lse, total


def _exact_gradient(s):
    """The chain rule through (1 - e) nll + e mean nll + l lse^2, a block of the vocabulary
    after the other; lse and the weights' sum are inputs that the call is given."""
    (T, H), V = s["h"].shape, s["W"].shape[0]
    h = s["h"].double()
    a = _weights64(s) * s["grad"].double()
    if s["reduction"] == "mean" and float(s["total"]) > 0:
        a = a / s["total"].double()
    lse = s["lse"].double()
    gh = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    gW = torch.empty(V, H, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // T)
    for v in range(0, V, step):
        W = s["W"][v:v + step].double()
        d = torch.mm(h, W.t()).mul_(s["inv_temp"]).sub_(lse[:, None]).exp_()
        d.mul_((1 + 2 * s["z_loss"] * lse)[:, None]).sub_(s["smoothing"] / V)
        t = s["targets"].long() - v
        row = ((t >= 0) & (t < W.shape[0])).nonzero()[:, 0]
        d[row, t[row]] -= 1 - s["smoothing"]
        d.mul_((a * s["inv_temp"])[:, None])
        gh += torch.mm(d, W)
        gW[v:v + step] = torch.mm(d.t(), h)
    return gh, gW


def _codes64(x):
    """A row's scale is the fp32 quotient, its codes are rounded from fp32 quotients: a quotient
    of fp32 numbers taken in 64 bits and then rounded to 32 is the fp32 one."""
    scales = (x.double().abs().amax(1) / 127).float().double()
    scales[scales == 0] = 1
    return (x.double() / scales[:, None]).float().double().round().clamp(-127, 127), scales


def _exact_linear(s):
    if s["x_scales"] is None:
        x, x_scales = _codes64(s["x"])
    else:
        x, x_scales = s["x"].double(), s["x_scales"].double()
    N = s["codes"].shape[0]
    y = torch.empty(x.shape[0], N, dtype=torch.float64, device="cuda")
    for r in range(0, N, 16384):
        y[:, r:r + 16384] = torch.mm(x, s["codes"][r:r + 16384].double().t())
    return y.mul_(x_scales[:, None]).mul_(s["scales"].double())


def _exact_quantize(s):
    """The scales alone: the values stand on the rounded scales."""
    return None, s["W"].double().abs().amax(1) / 127


def work(case):
    """Bytes: each input read once, each output written once; operations: of the formulas (the
    gradient's are three products: the scores again, and one for each operand)."""
    if case["op"] in ("loss", "gradient"):
        T, H, V = case["T"], case["H"], case["V"]
        rows = T * (4 + (4 if case["weighted"] else 0) + 4 + (4 if case["reduction"] == "none" else 0))
        ends = 2 * H * (T + V)
        if case["op"] == "loss":
            return {"bytes": ends + rows, "flops": 2 * T * H * V}
        return {"bytes": 2 * ends + rows, "flops": 6 * T * H * V}
    N, K = case["N"], case["K"]
    if case["op"] == "linear":
        T = case["T"]
        x = T * K * SIZES[case["x"]] + (4 * T if case["x"] == "int8" else 0)
        return {"bytes": N * K + 4 * N + x + T * N * SIZES[case["out"]], "flops": 2 * T * N * K}
    return {"bytes": 4 * N * K + 4 * N, "flops": 4 * N * K}
