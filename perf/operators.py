"""Measured cases of the token log probability and 4-bit weight operators.

Four operators, each in a plain form (elementary torch operations in 32 bits) and,
where ``own`` is true, as the package's calls:

  logprobs  token_logprobs: from logits, the log probability of each row's token, the
            log-sum-exp, the entropy and the top alternatives with their ids
  backward  token_logprobs_backward: the gradient of those with respect to the logits
  linear    linear_w4: y = x . W^T for W held as 4-bit codes with group scales
  quantize  quantize_w4 and dequantize_w4: a weight to 4-bit codes and back
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
INV_TEMP = float(np.float32(1 / 0.7))


def listed():
    return [
        # One new token of one sequence: the head's fp32 logits, sampled at temperature
        # 0.7, and the 20 alternatives that a serving interface returns.
        dict(name="logprobs_decode_1", op="logprobs", T=1, V=151936, dtype="fp32", top_k=20,
             inv_temp=INV_TEMP, masked=False, pad=0),
        # A decode batch of 64 sequences under grammar masks: allowed-token bits, some
        # rows with few tokens left, one with none, NaN in forbidden places.
        dict(name="logprobs_decode_64_masked", op="logprobs", T=64, V=151936, dtype="bf16",
             top_k=5, inv_temp=1.0, masked=True, pad=0),
        # A ragged prefill scored by another engine: odd vocabulary, so rows start at every
        # alignment, and the most alternatives.
        dict(name="logprobs_prefill_odd", op="logprobs", T=300, V=32761, dtype="fp16", top_k=32,
             inv_temp=1.0, masked=False, pad=0),
        # Scoring for distillation: 1024 tokens with 20 alternatives each, fp32 logits in a
        # buffer with padded rows.
        dict(name="logprobs_distill_1024", op="logprobs", T=1024, V=151936, dtype="fp32",
             top_k=20, inv_temp=1.0, masked=False, pad=64),
        # A training batch (8 packed sequences of 512): log probability and entropy alone.
        dict(name="logprobs_train_4096", op="logprobs", T=4096, V=151936, dtype="bf16", top_k=0,
             inv_temp=1.0, masked=False, pad=0),
        # The same batch's gradient: policy loss and entropy bonus, bf16 logits.
        dict(name="backward_train_4096", op="backward", T=4096, V=151936, dtype="bf16", top_k=0,
             inv_temp=1.0, masked=False, pad=0),
        # A small distillation batch: gradients of all outputs, odd vocabulary, masked rows.
        dict(name="backward_distill_130_odd", op="backward", T=130, V=50001, dtype="fp32", top_k=8,
             inv_temp=INV_TEMP, masked=True, pad=0),
        # The 4-bit LM head for one new token.
        dict(name="linear_head_1", op="linear", T=1, N=151936, K=4096, group=128, zeros=False,
             dtype="bf16", out="fp32"),
        # A small decode batch through an odd-sized projection, fp16, zero points, a short
        # last group.
        dict(name="linear_proj_13_ragged", op="linear", T=13, N=5119, K=5152, group=64, zeros=True,
             dtype="fp16", out="fp16"),
        # The 4-bit LM head for a decode batch of 64, with zero points.
        dict(name="linear_head_64", op="linear", T=64, N=151936, K=4096, group=128, zeros=True,
             dtype="bf16", out="fp32"),
        # A new policy's LM head after a training step, quantised for the rollout engine.
        dict(name="quantize_head", op="quantize", N=151936, K=4096, group=128, zeros=False,
             dtype="bf16"),
        # A small odd projection with zero points and a short last group.
        dict(name="quantize_proj_ragged", op="quantize", N=1009, K=2080, group=64, zeros=True,
             dtype="fp16"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm: odd, or eight times an odd
    one (rows at every alignment, and rows at 16 bytes), where it is over 64."""
    n = min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))
    return n if n <= 64 else min(high, rng.choice([n | 1, 8 * (n // 8 | 1)]))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "backward", "linear", "linear", "quantize"])
    if op in ("logprobs", "backward"):
        V = rng.choice([151936, 32768, _spread(rng, 500, 250000), _spread(rng, 500, 250000)])
        top_k = rng.choice([0, 1, 5, 20, 32]) if op == "logprobs" else rng.choice([0, 0, 8, 32])
        masked = rng.random() < 0.3
        # the alternatives of every row are sorted in the plain form, and masks are unpacked
        most = 4096 * 151936 if not (top_k or masked) else 1024 * 151936
        T = min(_spread(rng, 1, 4096), most // V)
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        if dtype == "fp32":
            T = min(T, 2048 * 151936 // V)
        return dict(op=op, T=max(1, T), V=V, dtype=dtype, top_k=min(top_k, V),
                    inv_temp=rng.choice([1.0, INV_TEMP, 0.5]), masked=masked,
                    pad=rng.choice([0, 0, 8, 3]))
    N = rng.choice([151936, _spread(rng, 500, 151936), _spread(rng, 500, 151936)])
    K = 32 * (2 * rng.randrange(16, 80) + 1)
    if N * K > 151936 * 4096 or rng.random() < 0.2:
        K = 4096
    case = dict(op=op, N=N, K=K, group=rng.choice([32, 64, 128, 128]), zeros=rng.random() < 0.5,
                dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "linear":
        case["T"] = _spread(rng, 1, 64)
        case["out"] = rng.choice(["fp32", case["dtype"]])
    return case


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if case["op"] in ("logprobs", "backward"):
        return _prepare_logits(case, g)
    return _prepare_weight(case, g)


def _prepare_logits(case, g):
    """Logits with the spread of a language model's (a few tokens far above a broad rest),
    targets mostly among the likely tokens, a few rows ignored."""
    T, V, dt = case["T"], case["V"], DTYPES[case["dtype"]]
    buf = torch.empty(T, V + case["pad"], dtype=dt, device="cuda")
    logits = buf[:, :V]
    step = max(1, (1 << 26) // V)
    for r in range(0, T, step):
        n = min(step, T - r)
        logits[r:r + n] = (torch.randn(n, V, generator=g, device="cuda") * 2).to(dt)
    hot = torch.randint(0, V, (T, 8), generator=g, device="cuda")
    up = torch.rand(T, 8, generator=g, device="cuda") * 8 + 4
    logits.scatter_(1, hot, (logits.gather(1, hot).float() + up).to(dt))
    pick = torch.rand(T, generator=g, device="cuda")
    anywhere = torch.randint(0, V, (T,), generator=g, device="cuda")
    targets = torch.where(pick < 0.7, hot[:, 0], anywhere)
    targets = torch.where(pick > 0.97, torch.full_like(targets, -1), targets).to(torch.int32)
    state = dict(op=case["op"], logits=logits, targets=targets, inv_temp=case["inv_temp"],
                 top_k=case["top_k"], allowed=None)
    if case["masked"]:
        share = torch.rand(T, 1, generator=g, device="cuda") ** 3
        keep = torch.rand(T, V, generator=g, device="cuda") < share
        keep.scatter_(1, hot[:, :4], True)
        if T > 2:
            keep[T // 2] = False  # nothing is allowed in this row
        noise = torch.rand(T, V, generator=g, device="cuda") < 0.01
        logits.masked_fill_(noise & ~keep, float("nan"))
        words = (V + 31) // 32
        bits = torch.zeros(T, words * 32, dtype=torch.bool, device="cuda")
        bits[:, :V] = keep
        allowed = torch.zeros(T, words, dtype=torch.int32, device="cuda")
        for b in range(32):
            allowed |= bits[:, b::32].to(torch.int32) << b
        state["allowed"] = allowed
    if case["op"] == "backward":
        lse, ent = _statistics64(state)
        state["lse"], state["entropy"] = lse.float(), ent.float()
        state["grad_logp"] = torch.randn(T, generator=g, device="cuda") / T
        state["grad_entropy"] = torch.randn(T, generator=g, device="cuda") * (0.01 / T)
        state["top_ids"] = state["grad_top"] = state["grad_lse"] = None
        if case["top_k"]:
            x = _masked(state, 0, T)
            best, ids = torch.sort(x, dim=1, descending=True, stable=True)
            best, ids = best[:, :case["top_k"]], ids[:, :case["top_k"]]
            state["top_ids"] = torch.where(best > float("-inf"), ids, -1).to(torch.int32)
            state["grad_top"] = torch.randn(T, case["top_k"], generator=g, device="cuda") / T
            state["grad_lse"] = torch.randn(T, generator=g, device="cuda") * (0.01 / T)
    return state


def _prepare_weight(case, g):
    N, K, group, dt = case["N"], case["K"], case["group"], DTYPES[case["dtype"]]
    W = torch.empty(N, K, dtype=dt, device="cuda")
    step = max(1, (1 << 26) // K)
    for r in range(0, N, step):
        n = min(step, N - r)
        W[r:r + n] = (torch.randn(n, K, generator=g, device="cuda") * 0.02).to(dt)
    if case["op"] == "quantize":
        return dict(op="quantize", W=W, group=group, zeros=case["zeros"])
    # the weight as a checkpoint holds it: codes, scales and zero points; `codes` has one code
    # to a byte and `words` eight to a word (even k in the low half, odd k in the high half)
    G = (K + group - 1) // group
    codes = torch.empty(N, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(N, G, dtype=dt, device="cuda")
    zeros = torch.full((N, G), 8, dtype=torch.uint8, device="cuda") if case["zeros"] else None
    for r in range(0, N, step):
        n = min(step, N - r)
        w = torch.nn.functional.pad(W[r:r + n].float(), (0, G * group - K)).view(n, G, group)
        if case["zeros"]:
            low, high = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
            s = ((high - low) / 15).to(dt)
            z = torch.round(-low / s.float()).clamp(0, 15)
            q = (torch.round(w / s.float()[:, :, None]) + z[:, :, None]).clamp(0, 15)
            zeros[r:r + n] = z.to(torch.uint8)
        else:
            s = (w.abs().amax(2) / 7).to(dt)
            q = torch.round(w / s.float()[:, :, None]).clamp(-7, 7) + 8
        scales[r:r + n] = s
        codes[r:r + n] = q.view(n, G * group)[:, :K].to(torch.uint8)
    words = torch.zeros(N, K // 8, dtype=torch.int32, device="cuda")
    for j in range(8):
        words |= codes[:, j::8].to(torch.int32) << (4 * ((j & 1) * 4 + j // 2))
    x = torch.randn(case["T"], K, generator=g, device="cuda")
    x = (x * torch.rsqrt(x.pow(2).mean(1, keepdim=True))).to(dt)
    return dict(op="linear", x=x, codes=codes, words=words, scales=scales, zeros=zeros,
                group=group, out=DTYPES[case["out"]])


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"logprobs": _plain_logprobs, "backward": _plain_backward, "linear": _plain_linear,
            "quantize": _plain_quantize}[state["op"]](state)


def _run_own(s):
    import invariant_token_logprob_gb300 as rlk
    if s["op"] == "logprobs":
        return tuple(rlk.token_logprobs(s["logits"], s["targets"], top_k=s["top_k"],
                                        allowed=s["allowed"], inv_temp=s["inv_temp"]))
    if s["op"] == "backward":
        return rlk.token_logprobs_backward(
            s["logits"], s["targets"], s["lse"], s["entropy"], grad_logp=s["grad_logp"],
            grad_lse=s["grad_lse"], grad_entropy=s["grad_entropy"], top_ids=s["top_ids"],
            grad_top=s["grad_top"], allowed=s["allowed"], inv_temp=s["inv_temp"])
    if s["op"] == "linear":
        return rlk.linear_w4(s["x"], s["words"], s["scales"], zeros=s["zeros"], group=s["group"],
                             out_dtype=s["out"])
    words, scales, zeros = rlk.quantize_w4(s["W"], group=s["group"], asymmetric=s["zeros"])
    values = rlk.dequantize_w4(words, scales, zeros=zeros, group=s["group"])
    return (values, scales) if zeros is None else (values, scales, zeros)


def _masked(s, r, n):
    """Rows [r, r + n) of the logits in fp32, forbidden tokens at -inf."""
    x = s["logits"][r:r + n].float()
    if s["allowed"] is not None:
        shift = torch.arange(32, device=x.device, dtype=torch.int32)
        bits = (s["allowed"][r:r + n, :, None] >> shift) & 1
        x = torch.where(bits.reshape(n, -1)[:, :x.shape[1]] != 0, x, float("-inf"))
    return x


def _plain_logprobs(s):
    T, V = s["logits"].shape
    it, K = s["inv_temp"], s["top_k"]
    x = _masked(s, 0, T)
    z = x * it
    m = z.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    d = z - m
    e = torch.exp(d)
    total = e.sum(1)
    logs = torch.log(total)
    lse = m[:, 0] + logs
    u = torch.where(e > 0, e * d, 0.0).sum(1)
    entropy = torch.where(total > 0, logs - u / total, 0.0)
    t = s["targets"].long()
    inside = (t >= 0) & (t < V)
    zt = z.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]
    logp = torch.where(torch.isinf(zt), zt, zt - lse)
    logp = torch.where(inside, logp, 0.0)
    if K:
        best, ids = torch.sort(x, dim=1, descending=True, stable=True)
        best, ids = best[:, :K], ids[:, :K]
    else:
        best, ids = x[:, :0], t[:, None][:, :0]
    there = best > float("-inf")
    top_ids = torch.where(there, ids, -1).to(torch.int32)
    top_logp = torch.where(there, best * it - lse[:, None], float("-inf"))
    return logp, lse, entropy, top_ids, top_logp


def _plain_backward(s):
    T, V = s["logits"].shape
    it = s["inv_temp"]
    x = _masked(s, 0, T)
    lse = s["lse"][:, None]
    lp = x * it - torch.where(torch.isinf(lse), 0.0, lse)
    p = torch.exp(lp)
    t = s["targets"].long()
    inside = (t >= 0) & (t < V)
    g_logp = torch.where(inside, s["grad_logp"], 0.0)
    total = g_logp.clone()
    if s["grad_top"] is not None:
        there = s["top_ids"] >= 0
        g_top = torch.where(there, s["grad_top"], 0.0)
        total = total + g_top.sum(1)
    a = -total if s["grad_lse"] is None else s["grad_lse"] - total
    d = p * (a[:, None] - s["grad_entropy"][:, None] * (lp + s["entropy"][:, None]))
    d = d.scatter_add(1, t.clamp(0, V - 1)[:, None], g_logp[:, None])
    if s["grad_top"] is not None:
        d = d.scatter_add(1, s["top_ids"].long().clamp(min=0), g_top)
    d = torch.where(torch.isinf(x) | torch.isinf(lse), 0.0, d * it)
    return d.to(s["logits"].dtype)


def _plain_linear(s):
    K, group = s["codes"].shape[1], s["group"]
    scale = s["scales"].float().repeat_interleave(group, 1)[:, :K]
    if s["zeros"] is None:
        w = (s["codes"].float() - 8) * scale
    else:
        w = (s["codes"].float() - s["zeros"].float().repeat_interleave(group, 1)[:, :K]) * scale
    return (s["x"].float() @ w.t()).to(s["out"])


def _plain_quantize(s):
    W, group = s["W"], s["group"]
    N, K = W.shape
    G = (K + group - 1) // group
    w = torch.nn.functional.pad(W.float(), (0, G * group - K)).view(N, G, group)
    if s["zeros"]:
        low, high = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scales = ((high - low) / 15).to(W.dtype)
    else:
        scales = (w.abs().amax(2) / 7).to(W.dtype)
    scales = torch.where(scales == 0, torch.ones_like(scales), scales)
    f = scales.float()[:, :, None]
    if s["zeros"]:
        zeros = torch.round(-low[:, :, None] / f).clamp(0, 15)
        q = (torch.round(w / f) + zeros).clamp(0, 15) - zeros
    else:
        q = torch.round(w / f).clamp(-7, 7)
    values = (q * f).view(N, G * group)[:, :K].to(W.dtype)
    if s["zeros"]:
        return values, scales, zeros[:, :, 0].to(torch.uint8)
    return values, scales


# ---------------------------------------------------------------- 64 bits
def _rows64(s, r, n):
    x = s["logits"][r:r + n].double()
    if s["allowed"] is not None:
        v = torch.arange(x.shape[1], device=x.device)
        word = s["allowed"][r:r + n].long().index_select(1, v // 32)
        x[torch.bitwise_and(torch.bitwise_right_shift(word, v % 32), 1) == 0] = -math.inf
    return x


def _statistics64(s):
    """lse and entropy of every row in 64 bits (-inf and 0 for an empty row)."""
    T, V = s["logits"].shape
    lse = torch.empty(T, dtype=torch.float64, device="cuda")
    ent = torch.empty_like(lse)
    step = max(1, (1 << 26) // V)
    for r in range(0, T, step):
        n = min(step, T - r)
        z = _rows64(s, r, n).mul_(s["inv_temp"])
        lse[r:r + n] = torch.logsumexp(z, 1)
        lp = z.sub_(lse[r:r + n, None].clamp(min=-1e300))
        ent[r:r + n] = -torch.special.xlogy(torch.exp(lp), torch.exp(lp)).sum(1)
    return lse, ent


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "logprobs":
        return _exact_logprobs(s)
    if s["op"] == "backward":
        return _exact_backward(s)
    if s["op"] == "linear":
        return _exact_linear(s)
    return _exact_quantize(s)


def _exact_logprobs(s):
    T, V = s["logits"].shape
    K, it = s["top_k"], s["inv_temp"]
    lse, ent = _statistics64(s)
    logp = torch.zeros(T, dtype=torch.float64, device="cuda")
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    top = torch.empty(T, K, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // V)
    for r in range(0, T, step):
        n = min(step, T - r)
        x = _rows64(s, r, n)
        t = s["targets"][r:r + n].long()
        row = ((t >= 0) & (t < V)).nonzero()[:, 0]
        xt = x[row, t[row]]
        value = xt * it - lse[r:r + n][row]
        value[xt == -math.inf] = -math.inf
        logp[r + row] = value
        for k in range(K):  # the best left, lowest index first, taken out one after another
            best = x.amax(1)
            first = (x == best[:, None]).to(torch.uint8).argmax(1)
            none = best == -math.inf
            ids[r:r + n, k] = torch.where(none, -1, first).to(torch.int32)
            top[r:r + n, k] = torch.where(none, -math.inf, best * it - lse[r:r + n])
            x.scatter_(1, first[:, None], -math.inf)
    return logp, lse, ent, ids, top


def _exact_backward(s):
    """Row by row the Jacobian's product: d logp_t/dz_v = [v = t] - p_v, d lse/dz_v = p_v,
    dH/dz_v = -p_v (log p_v + H); lse and the entropy are the inputs that the call is given."""
    T, V = s["logits"].shape
    out = torch.empty(T, V, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // V)
    for r in range(0, T, step):
        n = min(step, T - r)
        x = _rows64(s, r, n)
        gone = torch.isneginf(x) | torch.isneginf(s["lse"][r:r + n].double())[:, None]
        logp = (x * s["inv_temp"] - s["lse"][r:r + n].double()[:, None]).masked_fill_(gone, -1e6)
        p = logp.exp()
        d = -s["grad_entropy"][r:r + n].double()[:, None] * p * (logp + s["entropy"][r:r + n].double()[:, None])
        if s["grad_lse"] is not None:
            d += s["grad_lse"][r:r + n].double()[:, None] * p
        pairs = [(s["targets"][r:r + n].long(), s["grad_logp"][r:r + n].double())]
        if s["grad_top"] is not None:
            pairs += [(s["top_ids"][r:r + n, k].long(), s["grad_top"][r:r + n, k].double())
                      for k in range(s["top_ids"].shape[1])]
        weight = torch.zeros(n, dtype=torch.float64, device="cuda")
        for v, w in pairs:
            row = ((v >= 0) & (v < V)).nonzero()[:, 0]
            d[row, v[row]] += w[row]
            weight[row] += w[row]
        d -= weight[:, None] * p
        out[r:r + n] = d.mul_(s["inv_temp"]).masked_fill_(gone, 0.0)
    return out


def _exact_linear(s):
    N, K = s["codes"].shape
    group = torch.arange(K, device="cuda") // s["group"]
    x = s["x"].double()
    y = torch.empty(x.shape[0], N, dtype=torch.float64, device="cuda")
    step = 16384
    for r in range(0, N, step):
        w = s["codes"][r:r + step].double()
        w -= 8.0 if s["zeros"] is None else s["zeros"][r:r + step].double().index_select(1, group)
        w *= s["scales"][r:r + step].double().index_select(1, group)
        y[:, r:r + step] = torch.mm(x, w.t())
    return y


def _exact_quantize(s):
    """The scales alone: the values stand on the rounded scales, and whole zero points are
    compared as they are."""
    W, group = s["W"], s["group"]
    cols = []
    for k in range(0, W.shape[1], group):
        w = W[:, k:k + group].double()
        if s["zeros"]:
            cols.append((w.amax(1).clamp(min=0) - w.amin(1).clamp(max=0)) / 15)
        else:
            cols.append(torch.maximum(w.amax(1), -w.amin(1)) / 7)
    scales = torch.stack(cols, 1)
    return (None, scales, None) if s["zeros"] else (None, scales)


def work(case):
    """Bytes: each input read once, each output written once; operations: of the formulas."""
    if case["op"] in ("logprobs", "backward"):
        T, V, size = case["T"], case["V"], SIZES[case["dtype"]]
        bits = T * ((V + 31) // 32) * 4 if case["masked"] else 0
        if case["op"] == "logprobs":
            return {"bytes": T * V * size + bits + T * 16 + T * case["top_k"] * 8, "flops": 6 * T * V}
        row = 20 + case["top_k"] * 8 + (4 if case["top_k"] else 0)
        return {"bytes": 2 * T * V * size + bits + T * row, "flops": 7 * T * V}
    N, K = case["N"], case["K"]
    G = (K + case["group"] - 1) // case["group"]
    meta = N * G * (3 if case["zeros"] else 2)
    if case["op"] == "linear":
        T = case["T"]
        return {"bytes": N * K // 2 + meta + T * K * 2 + T * N * SIZES[case["out"]], "flops": 2 * T * N * K}
    return {"bytes": 4 * N * K + meta, "flops": 4 * N * K}
