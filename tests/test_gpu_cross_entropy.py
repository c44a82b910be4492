"""GPU tests of the cross entropy (loss and gradients) against plain implementations in 64 bits.

Tolerances.  A logit sums H exact products of bf16 numbers on the tensor core, 16 to an
instruction; each of its additions loses at most 2^-22 of the magnitudes added so far (it may cut
instead of rounding), the instruction's own sum included.  The loss takes parts of 512 k, which
fp32 additions join, the gradient's logits all of H: with A = inv_temp sum |h||W| (a row's largest)
  loss:     |z - z64| <= A ((32 + 16) 2^-22 + (H/512 + 1) 2^-24) =: E
  gradient: |z - z64| <= A (H/16 + 16) 2^-22                     =: G
The log-sum-exp moves by at most E, and its own fp32 steps (exponentials of arguments rounded to
2^-23 of their size, a tree of additions of positive numbers, one logarithm) by at most
2^-19 (1 + |lse|).  The loss adds the target's logit (E), smoothing's mean (E and an fp32 sum of
V numbers in chunks of 128, tiles and lanes: 2^-19 of the mean magnitude) and z_loss lse^2.
In the gradients p is off by a relative G + 2^-18, and the products' sums lose 2^-22 per instruction
of 16, 2^-12 in all for the sizes here.  For grad_h the gradient with respect to the logits is
rounded to bf16 (2^-8 at most) but for the target's element, which is kept; for grad_W to fp16
(2^-11), h is not, and what lies 2^-39 below the largest product of a row's gradient and hidden
state may be lost.  With P := |a| (p (1 + 2 l lse) + e / V) and D := P + |a| (1 - e) [target]:
  |grad_h - grad_h64| <= inv_temp (2^-8 P + (2^-11 + G) D) |W|
  |grad_W - grad_W64| <= inv_temp ((2^-10 + G) D^T |h| + T 2^-36 max D max |h|)
(2^-11 in each for the terms above), and the output's rounding, 2^-8 for bf16."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import invariant_token_logprob_gb300 as rlk
    rlk.lib()
    rlk.take_device_errors()


def make(T, H, V, seed=0, weighted=True, scale=1.3):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, H, generator=g) * (scale / math.sqrt(H))).bfloat16()
    h = torch.randn(T, H, generator=g).bfloat16()
    t = torch.randint(0, V, (T,), generator=g).to(torch.int32)
    if T > 3:
        t[1] = -100
        t[T // 2] = V - 1
        t[2] = 0
    w = torch.rand(T, generator=g) + 0.5 if weighted else None
    if weighted and T > 4:
        w[3] = 0
    return h, W, t, w


class Ref:
    """Everything in 64 bits, on the device of its inputs."""

    def __init__(self, h, W, t, w, inv_temp, e, l, lse=None):
        it = float(np.float32(inv_temp))
        T, V = h.shape[0], W.shape[0]
        self.h, self.W, self.it, self.e, self.l = h.double(), W.double(), it, float(np.float32(e)), float(np.float32(l))
        self.z = self.h @ self.W.T * it
        self.lse = torch.logsumexp(self.z, 1) if lse is None else lse.double()
        inside = (t >= 0) & (t < V)
        self.t = t.long().clamp(0, V - 1)
        self.zt = self.z.gather(1, self.t[:, None])[:, 0]
        self.w = torch.where(inside, torch.ones(T, device=h.device) if w is None else w, torch.zeros(T, device=h.device)).double()
        nll = self.lse - (1 - self.e) * self.zt - self.e * self.z.mean(1) + self.l * self.lse ** 2
        self.row = torch.where(self.w != 0, self.w * nll, torch.zeros_like(nll))
        self.total = self.w.sum()
        A = (self.h.abs() @ self.W.abs().T).amax(1) * it
        self.E = A * (48 * 2.0 ** -22 + (h.shape[1] / 512 + 1) * 2.0 ** -24)
        self.G = A * (h.shape[1] / 16 + 16) * 2.0 ** -22

    def loss_bound(self):
        rows = 2 * self.E * (1 + 2 * self.l * self.lse.abs()) + 2.0 ** -19 * (
            1 + self.lse.abs() * (1 + 2 * self.l * self.lse.abs()) + self.zt.abs() + self.e * self.z.abs().mean(1))
        return rows * self.w

    def value(self, reduction):
        if reduction == "none":
            return self.row
        s = self.row.sum()
        return s if reduction == "sum" else (s / self.total if self.total > 0 else s * 0)

    def grads(self, g, reduction):
        """(grad_h, its bound), (grad_W, its bound), without the outputs' rounding."""
        a = g.double() * self.w
        if reduction == "mean":
            a = a / self.total if self.total > 0 else a * 0
        p = torch.exp(self.z - self.lse[:, None])
        up = p * (1 + 2 * self.l * self.lse)[:, None]
        hit = torch.zeros_like(p).scatter_(1, self.t[:, None], 1 - self.e)
        V = p.shape[1]
        dz = a[:, None] * (up - hit - self.e / V)
        P = a.abs()[:, None] * (up.abs() + self.e / V)
        D = P + a.abs()[:, None] * hit
        it, G = self.it, self.G[:, None]
        floor = p.shape[0] * 2.0 ** -36 * (D.amax(1) * self.h.abs().amax(1)).max()
        return ((it * dz @ self.W, it * (2.0 ** -8 * P + (2.0 ** -11 + G) * D) @ self.W.abs()),
                (it * dz.T @ self.h, it * (((2.0 ** -10 + G) * D).T @ self.h.abs() + floor)))


def within(got, want, bound, rounding=0.0, what=""):
    off = (got.double() - want).abs() - bound - rounding * want.abs()
    assert torch.isfinite(got).all(), what
    assert off.max() <= 0, f"{what}: over the bound by {off.max():.3g} at {int(off.argmax())}"


SHAPES = [(1, 64, 1), (1, 8, 33), (2, 72, 500), (17, 256, 1024), (128, 136, 257), (129, 520, 511), (300, 264, 5003),
          (257, 64, 32761)]


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("e,l,it", [(0.0, 0.0, 1.0), (0.1, 1e-3, 1 / 0.7)])
@pytest.mark.parametrize("shape", SHAPES)
def test_loss_and_gradients(shape, e, l, it, reduction):
    import invariant_token_logprob_gb300 as rlk
    T, H, V = shape
    h, W, t, w = (None if x is None else x.cuda() for x in make(T, H, V, T + V, weighted=e > 0 or reduction == "sum"))
    opts = dict(inv_temp=it, label_smoothing=e, z_loss=l, reduction=reduction)
    r = rlk.cross_entropy(h, W, t, w, **opts)
    ref = Ref(h, W, t, w, it, e, l)
    bound = ref.loss_bound()
    within(r.lse, ref.lse, ref.E + 2.0 ** -19 * (1 + ref.lse.abs()), what="lse")
    assert abs(float(r.total) - float(ref.total)) <= 2.0 ** -20 * float(ref.total)
    if reduction == "none":
        within(r.loss, ref.row, bound + 2.0 ** -23 * ref.row.abs(), what="loss")
    else:
        scale = 1.0 if reduction == "sum" else 1 / max(float(ref.total), 1e-30)
        tol = (bound.sum() + 2.0 ** -19 * ref.row.abs().sum()) * scale
        assert abs(float(r.loss) - float(ref.value(reduction))) <= float(tol)
    g = torch.randn(T, generator=torch.Generator().manual_seed(1)).cuda() if reduction == "none" else torch.tensor(
        0.7, device="cuda")
    ref = Ref(h, W, t, w, it, e, l, lse=r.lse)
    (gh, bh), (gW, bW) = ref.grads(g, reduction)
    for dtype, half in ((torch.bfloat16, 2.0 ** -8), (torch.float32, 2.0 ** -24)):
        a, b = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, grad_dtype=dtype, **opts)
        assert a.dtype == b.dtype == dtype
        within(a, gh, bh * (1 + half), half, f"grad_h {dtype}")
        within(b, gW, bW * (1 + half), half, f"grad_W {dtype}")
        only_h = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, grad_dtype=dtype, need_W=False, **opts)
        only_W = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, grad_dtype=dtype, need_h=False, **opts)
        assert only_h[1] is None and only_W[0] is None
        assert torch.equal(only_h[0], a) and torch.equal(only_W[1], b)
    start = torch.randn(V, H, generator=torch.Generator().manual_seed(2)).cuda()
    acc = start.clone()
    _, same = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, need_h=False, grad_W=acc, **opts)
    assert same is acc and torch.equal(acc, start + b)  # one fp32 addition each
    assert rlk.take_device_errors() == (0, 0)


@pytest.mark.parametrize("T,H,V", [(2048, 64, 100000), (1100, 72, 150777), (4096, 256, 40001)])
def test_pieces_of_the_vocabulary(T, H, V):
    """More than one piece, the last one short; every column counts exactly once."""
    import invariant_token_logprob_gb300 as rlk
    h, W, t, w = (x.cuda() for x in make(T, H, V, 5))
    opts = dict(label_smoothing=0.1, z_loss=1e-4)
    r = rlk.cross_entropy(h, W, t, w, **opts)
    g = torch.tensor(1.0, device="cuda")
    size = rlk.cross_entropy_backward_workspace_size(T, H, V)
    assert size < 4 * T * V  # (not the whole dz and its transpose)
    gh, gW = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, **opts)
    ref = Ref(h, W, t, w, 1.0, 0.1, 1e-4, lse=r.lse)
    (wh, bh), (wW, bW) = ref.grads(g, "mean")
    within(gh, wh, bh * (1 + 2.0 ** -8), 2.0 ** -8, "grad_h")
    within(gW, wW, bW * (1 + 2.0 ** -8), 2.0 ** -8, "grad_W")
    again = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, **opts)
    assert torch.equal(gh, again[0]) and torch.equal(gW, again[1])
    # a poisoned workspace: nothing is read that the call has not written
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    again = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, workspace=ws, **opts)
    assert torch.equal(gh, again[0]) and torch.equal(gW, again[1])


@pytest.mark.parametrize("T,H,V", [(8192, 64, 32001), (16384, 72, 331), (8199, 136, 1105)])
def test_bands_of_rows_behind_a_short_tile(T, H, V):
    """More rows than a band of row tiles (4096), so that tiles follow the vocabulary's last one, which
    has an odd number of chunks of 32 entries in a half: no staged block of the transposed gradient is
    written before the store from it has read it.  Repeated calls give the same bits."""
    import invariant_token_logprob_gb300 as rlk
    h, W, t, w = (x.cuda() for x in make(T, H, V, 7))
    opts = dict(label_smoothing=0.1, z_loss=1e-4)
    r = rlk.cross_entropy(h, W, t, w, **opts)
    g = torch.tensor(1.0, device="cuda")
    gh, gW = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, **opts)
    ref = Ref(h, W, t, w, 1.0, 0.1, 1e-4, lse=r.lse)
    (wh, bh), (wW, bW) = ref.grads(g, "mean")
    within(gh, wh, bh * (1 + 2.0 ** -8), 2.0 ** -8, "grad_h")
    within(gW, wW, bW * (1 + 2.0 ** -8), 2.0 ** -8, "grad_W")
    for _ in range(10):
        again = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, **opts)
        assert torch.equal(gh, again[0]) and torch.equal(gW, again[1])
    assert rlk.take_device_errors() == (0, 0)


@pytest.mark.parametrize("reduction", ["mean", "none"])
@pytest.mark.parametrize("T,H,V", SHAPES + [(130, 1032, 50001), (64, 256, 20000), (2048, 64, 100000), (1100, 72, 150777),
                                            (8192, 64, 32001)])
def test_adding_to_a_gradient_beside_grad_h(T, H, V, reduction):
    """grad_W added to a given fp32 tensor with grad_h wanted in the same call, bf16 and fp32, of one piece
    of the vocabulary and of several: grad_h as without adding, one fp32 addition per element of grad_W."""
    import invariant_token_logprob_gb300 as rlk
    h, W, t, w = (x.cuda() if x is not None else None for x in make(T, H, V, T + H, weighted=T > 3))
    opts = dict(inv_temp=1.25, label_smoothing=0.1, z_loss=1e-4, reduction=reduction)
    r = rlk.cross_entropy(h, W, t, w, **opts)
    gen = torch.Generator().manual_seed(3)
    g = torch.randn(T, generator=gen).cuda() if reduction == "none" else torch.tensor(0.3, device="cuda")
    start = torch.randn(V, H, generator=gen).cuda() * 1e-3
    full = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, grad_dtype=torch.float32, **opts)
    for dtype in (torch.bfloat16, torch.float32):
        alone = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, grad_dtype=dtype, **opts)
        acc = start.clone()
        gh, same = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, grad_dtype=dtype, grad_W=acc, **opts)
        assert same is acc and gh.dtype == dtype
        assert torch.equal(gh, alone[0]) and torch.equal(acc, start + full[1])
    assert rlk.take_device_errors() == (0, 0)


def test_row_bits_do_not_depend_on_the_batch():
    import invariant_token_logprob_gb300 as rlk
    for H in (256, 1032):
        h, W, t, _ = (None if x is None else x.cuda() for x in make(300, H, 5003, 3, weighted=False))
        lp, lse, _ = rlk.logprob(h, W, t, 0.8)
        opts = dict(inv_temp=0.8, reduction="none")
        r = rlk.cross_entropy(h, W, t, **opts)
        ref = Ref(h, W, t, None, 0.8, 0.0, 0.0)
        within(r.lse, lse.double(), ref.E + ref.G + 2.0 ** -19 * (1 + lse.double().abs()), what="the log probability's lse")
        s = rlk.cross_entropy(h, W, t, label_smoothing=0.2, z_loss=1e-3, **opts)
        assert torch.equal(s.lse, r.lse)
        for n in (1, 7, 128, 200):  # single rows and both launch shapes
            for o, full in ((dict(), r), (dict(label_smoothing=0.2, z_loss=1e-3), s)):
                part = rlk.cross_entropy(h[:n].contiguous(), W, t[:n].contiguous(), **opts, **o)
                assert torch.equal(part.loss, full.loss[:n]) and torch.equal(part.lse, full.lse[:n])


def test_long_sums_stay_near():
    """Logits that add up to one side over a long H, where cut additions would show: the loss keeps
    fp32's nearness."""
    import invariant_token_logprob_gb300 as rlk
    g = torch.Generator().manual_seed(0)
    T, H, V = 64, 8192, 600
    W = (torch.rand(V, H, generator=g) / 64).bfloat16().cuda()
    h = torch.rand(T, H, generator=g).bfloat16().cuda()
    t = torch.randint(0, V, (T,), generator=g).to(torch.int32).cuda()
    r = rlk.cross_entropy(h, W, t, reduction="none")
    ref = Ref(h, W, t, None, 1.0, 0.0, 0.0)
    assert ((r.lse.double() - ref.lse).abs() / ref.lse).max() < 1e-6  # 32 cuts of 2^-24 and the rest


@pytest.mark.parametrize("spread", [0, 20, 60])
def test_gradients_of_rows_far_apart(spread):
    """Incoming gradients, hidden states and weights' rows that lie many powers of two apart, and
    rows of zeros: every row keeps its own nearness."""
    import invariant_token_logprob_gb300 as rlk
    T, H, V = 140, 72, 515
    h, W, t, _ = (None if x is None else x.cuda() for x in make(T, H, V, 6, weighted=False))
    g = torch.Generator().manual_seed(spread)
    rows = (2.0 ** torch.randint(-spread // 2, spread // 2 + 1, (T, 1), generator=g)).cuda()
    grad = torch.randn(T, generator=g).cuda() * (2.0 ** torch.randint(-spread, spread + 1, (T,), generator=g)).cuda()
    grad[4] = 0
    h[5] = 0
    h = torch.where(rows > 1, h, h * rows).bfloat16()  # (large ones would make one-hot softmaxes alone)
    opts = dict(label_smoothing=0.1, reduction="none")
    r = rlk.cross_entropy(h, W, t, **opts)
    ref = Ref(h, W, t, None, 1.0, 0.1, 0.0, lse=r.lse)
    (wh, bh), (wW, bW) = ref.grads(grad, "none")
    gh, gW = rlk.cross_entropy_backward(h, W, t, r.lse, grad, **opts)
    within(gh, wh, bh * (1 + 2.0 ** -8) + 1e-38, 2.0 ** -8, "grad_h")
    within(gW, wW, bW * (1 + 2.0 ** -8) + 1e-38, 2.0 ** -8, "grad_W")


@pytest.mark.parametrize("grad,hidden", [(2.0 ** -100, 1.0), (2.0 ** -112, 1.0), (1.0, 2.0 ** -100),
                                         (2.0 ** -4, 2.0 ** -116), (2.0 ** 90, 1.0), (2.0 ** -120, 2.0 ** 20)])
def test_gradients_near_the_ends_of_the_range(grad, hidden):
    """Incoming gradients and hidden states near the ends of fp32's range: powers of two that go in
    come out.  Numbers below 2^-126 may be lost at each step: of the softmax's part of a gradient
    (times |W| or |h|), of h under the power that lifts it and of the result."""
    import invariant_token_logprob_gb300 as rlk
    T, H, V = 130, 72, 300
    h, W, t, _ = (None if x is None else x.cuda() for x in make(T, H, V, 16, weighted=False))
    h = (h.float() * hidden).bfloat16()
    if hidden > 1:
        W = (W.float() / hidden).bfloat16()
    g = torch.tensor(grad, device="cuda")
    r = rlk.cross_entropy(h, W, t, reduction="sum")
    ref = Ref(h, W, t, None, 1.0, 0.0, 0.0, lse=r.lse)
    (wh, bh), (wW, bW) = ref.grads(g, "sum")
    gh, gW = rlk.cross_entropy_backward(h, W, t, r.lse, g, reduction="sum", grad_dtype=torch.float32)
    least = 2.0 ** -126
    within(gh, wh, bh + least * (2 + W.double().abs().sum(0)), what="grad_h")
    within(gW, wW, bW + least * (2 + 2 * h.double().abs().sum(0)), what="grad_W")


def test_rows_that_do_not_count():
    """Ignored targets, weights of 0 and targets outside the vocabulary, with any logits."""
    import invariant_token_logprob_gb300 as rlk
    h, W, t, w = (x.cuda() for x in make(40, 64, 700, 9))
    t[5], t[6], w[7] = -1, 700, 0
    opts = dict(label_smoothing=0.1, z_loss=1e-2)
    r = rlk.cross_entropy(h, W, t, w, reduction="none", **opts)
    assert rlk.take_device_errors() == (0, 1)
    idle = (t < 0) | (t >= 700) | (w == 0)
    assert (r.loss[idle] == 0).all() and (r.loss[~idle] != 0).all()
    keep = (~idle).nonzero()[:, 0]
    few = rlk.cross_entropy(h[keep], W, t[keep], w[keep], **opts)
    assert abs(float(few.total) - float(r.total)) <= 2.0 ** -20 * float(r.total)
    g = torch.tensor(1.0, device="cuda")
    m = rlk.cross_entropy(h, W, t, w, **opts)
    rlk.take_device_errors()
    lse = m.lse.clone()
    lse[idle] = float("nan")  # what such a row's logits gave does not matter
    gh, gW = rlk.cross_entropy_backward(h, W, t, lse, g, m.total, w, **opts)
    assert (gh[idle] == 0).all() and torch.isfinite(gW).all()
    padded = h.clone()
    padded[idle] = float("nan")  # nor what it holds
    again = rlk.cross_entropy(padded, W, t, w, **opts)
    rlk.take_device_errors()
    assert torch.equal(again.loss, m.loss) and torch.equal(again.lse[~idle], m.lse[~idle])
    ph, pW = rlk.cross_entropy_backward(padded, W, t, lse, g, m.total, w, **opts)
    assert torch.equal(ph, gh) and torch.equal(pW, gW)
    nothing = torch.full_like(t, -100)
    for reduction in ("mean", "sum"):
        z = rlk.cross_entropy(h, W, nothing, w, reduction=reduction, **opts)
        assert float(z.loss) == 0 and float(z.total) == 0
        gh, gW = rlk.cross_entropy_backward(h, W, nothing, z.lse, g, z.total, w, reduction=reduction, **opts)
        assert (gh == 0).all() and (gW == 0).all()
    big = h.clone()
    big[0] = 3e38  # logits beyond fp32: the row's own loss alone is not finite
    r2 = rlk.cross_entropy(big, W, t, w, reduction="none", **opts)
    rlk.take_device_errors()
    assert torch.equal(r2.loss[1:], r.loss[1:])


def test_no_rows():
    import invariant_token_logprob_gb300 as rlk
    h, W, t, _ = (None if x is None else x.cuda() for x in make(4, 64, 100, 0))
    r = rlk.cross_entropy(h[:0], W, t[:0])
    assert float(r.loss) == 0 and float(r.total) == 0 and r.lse.shape == (0,)
    assert rlk.cross_entropy(h[:0], W, t[:0], reduction="none").loss.shape == (0,)
    g = torch.tensor(1.0, device="cuda")
    gh, gW = rlk.cross_entropy_backward(h[:0], W, t[:0], r.lse, g, r.total)
    assert gh.shape == (0, 64) and (gW == 0).all()
    acc = torch.ones(100, 64, device="cuda")
    rlk.cross_entropy_backward(h[:0], W, t[:0], r.lse, g, r.total, grad_W=acc)
    assert (acc == 1).all()


def test_gradient_against_differences():
    """Along random directions d: central differences of the loss in 64 bits, whose error is of
    third order in the step, against the gradients' products with d, each element of which may
    be off by its bound."""
    import invariant_token_logprob_gb300 as rlk
    h, W, t, w = (x.cuda() for x in make(33, 72, 301, 4))
    e, l, it = 0.1, 1e-2, 1.25
    opts = dict(inv_temp=it, label_smoothing=e, z_loss=l)
    r = rlk.cross_entropy(h, W, t, w, **opts)
    g = torch.tensor(1.0, device="cuda")
    gh, gW = rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, **opts)
    ref = Ref(h, W, t, w, it, e, l, lse=r.lse)
    (wh, bh), (wW, bW) = ref.grads(g, "mean")
    gen = torch.Generator().manual_seed(0)
    for _ in range(4):
        dh = torch.randn(h.shape, generator=gen).cuda().double()
        dW = torch.randn(W.shape, generator=gen).cuda().double()
        step = 1e-4
        up = Ref(h.double() + step * dh, W.double() + step * dW, t, w, it, e, l).value("mean")
        dn = Ref(h.double() - step * dh, W.double() - step * dW, t, w, it, e, l).value("mean")
        slope = float((up - dn) / (2 * step))
        got = float((gh.double() * dh).sum() + (gW.double() * dW).sum())
        tol = float(((bh * (1 + 2.0 ** -8) + 2.0 ** -8 * wh.abs()) * dh.abs()).sum() +
                    ((bW * (1 + 2.0 ** -8) + 2.0 ** -8 * wW.abs()) * dW.abs()).sum())
        assert abs(got - slope) <= tol + 1e-5


def test_training_step_in_a_graph():
    """Loss and backward pass under autograd, captured as torch asks for (warmed up on a side stream,
    the eager graphs gone) and replayed on other inputs."""
    import invariant_token_logprob_gb300 as rlk
    h, W, t, w = (x.cuda() for x in make(150, 136, 3001, 18))
    opts = dict(label_smoothing=0.05, z_loss=1e-4)
    hp, Wp = h.clone().requires_grad_(), W.clone().requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            hp.grad = Wp.grad = None
            rlk.differentiable_cross_entropy(hp, Wp, t, w, **opts).loss.backward()
    torch.cuda.current_stream().wait_stream(s)
    first = hp.grad, Wp.grad
    hp.grad = Wp.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        loss = rlk.differentiable_cross_entropy(hp, Wp, t, w, **opts).loss
        loss.backward()
    graph.replay()
    assert torch.equal(hp.grad, first[0]) and torch.equal(Wp.grad, first[1])
    other = h.flip(1).contiguous()
    with torch.no_grad():
        hp.copy_(other)
    graph.replay()
    e = rlk.cross_entropy(other, W, t, w, **opts)
    gh, gW = rlk.cross_entropy_backward(other, W, t, e.lse, torch.tensor(1.0, device="cuda"), e.total, w, **opts)
    assert torch.equal(loss, e.loss) and torch.equal(hp.grad, gh) and torch.equal(Wp.grad, gW)


def test_autograd_step_and_graph():
    """The loss under autograd, twice, then captured in a graph and replayed on other inputs, and
    the explicit calls on a stream of their own with given workspaces: all the same bits."""
    import invariant_token_logprob_gb300 as rlk
    h, W, t, w = (x.cuda() for x in make(200, 136, 3001, 8))
    opts = dict(label_smoothing=0.05, z_loss=1e-4)
    hp, Wp = h.clone().requires_grad_(), W.clone().requires_grad_()
    r = rlk.differentiable_cross_entropy(hp, Wp, t, w, **opts)
    assert not r.lse.requires_grad and not r.total.requires_grad
    (r.loss * 2).backward()
    e = rlk.cross_entropy(h, W, t, w, **opts)
    two = torch.tensor(2.0, device="cuda")
    gh, gW = rlk.cross_entropy_backward(h, W, t, e.lse, two, e.total, w, **opts)
    assert torch.equal(r.loss, e.loss) and torch.equal(hp.grad, gh) and torch.equal(Wp.grad, gW)
    only = rlk.differentiable_cross_entropy(h, Wp, t, w, **opts).loss
    (gW2,) = torch.autograd.grad(only * 2, (Wp,))
    assert torch.equal(gW2, gW)
    with pytest.raises(RuntimeError, match="first derivatives"):
        l = rlk.differentiable_cross_entropy(hp, W, t, w, **opts).loss
        (g1,) = torch.autograd.grad(l, (hp,), create_graph=True)
        g1.float().sum().backward()
    s = torch.cuda.Stream()
    ws1 = torch.empty(rlk.cross_entropy_workspace_size(200, 136, 3001), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(rlk.cross_entropy_backward_workspace_size(200, 136, 3001), dtype=torch.uint8, device="cuda")
    hs = h.clone()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        a = rlk.cross_entropy(hs, W, t, w, workspace=ws1, stream=s, **opts)
        return a, rlk.cross_entropy_backward(hs, W, t, a.lse, two, a.total, w, workspace=ws2, stream=s, **opts)
    with torch.cuda.stream(s):
        a, (x, y) = step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            ga, (gx, gy) = step()
        hs.copy_(h.flip(0))
        graph.replay()
    s.synchronize()
    assert torch.equal(a.loss, e.loss) and torch.equal(x, gh) and torch.equal(y, gW)
    f = rlk.cross_entropy(h.flip(0).contiguous(), W, t, w, **opts)
    fh, fW = rlk.cross_entropy_backward(h.flip(0).contiguous(), W, t, f.lse, two, f.total, w, **opts)
    assert torch.equal(ga.loss, f.loss) and torch.equal(gx, fh) and torch.equal(gy, fW)


def test_reads_and_writes_stay_inside():
    """Operands in the middle of poisoned memory, workspaces of the size asked for with a guard
    behind: results unchanged, guards untouched."""
    import invariant_token_logprob_gb300 as rlk
    T, H, V = 131, 72, 1023
    h, W, t, w = (x.cuda() for x in make(T, H, V, 2))
    opts = dict(label_smoothing=0.1)
    e = rlk.cross_entropy(h, W, t, w, **opts)
    g = torch.tensor(1.0, device="cuda")
    gh, gW = rlk.cross_entropy_backward(h, W, t, e.lse, g, e.total, w, **opts)

    def between(x):
        buf = torch.full((x.numel() + 128,), float("nan") if x.is_floating_point() else 7, dtype=x.dtype, device="cuda")
        v = buf[64:64 + x.numel()].view(x.shape)
        v.copy_(x)
        return v
    ins = [between(x) for x in (h, W, t, w)]

    def guarded(n):
        buf = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
        return buf, buf[:n]
    b1, w1 = guarded(rlk.cross_entropy_workspace_size(T, H, V))
    b2, w2 = guarded(rlk.cross_entropy_backward_workspace_size(T, H, V))
    r = rlk.cross_entropy(*ins, workspace=w1, **opts)
    x, y = rlk.cross_entropy_backward(*ins[:3], r.lse, g, r.total, ins[3], workspace=w2, **opts)
    assert torch.equal(r.loss, e.loss) and torch.equal(x, gh) and torch.equal(y, gW)
    assert (b1[w1.numel():] == 0xAB).all() and (b2[w2.numel():] == 0xAB).all()
    for off in (16, 48, 240):  # a workspace at any 16-byte boundary
        b2, _ = guarded(w2.numel() + off)
        x, y = rlk.cross_entropy_backward(*ins[:3], r.lse, g, r.total, ins[3], workspace=b2[off:off + w2.numel()], **opts)
        assert torch.equal(x, gh) and torch.equal(y, gW)
        assert (b2[:off] == 0xAB).all() and (b2[off + w2.numel():] == 0xAB).all()


def test_refusals():
    import invariant_token_logprob_gb300 as rlk
    h, W, t, w = (x.cuda() for x in make(8, 64, 100, 0))
    r = rlk.cross_entropy(h, W, t, w)
    g = torch.tensor(1.0, device="cuda")
    with pytest.raises(ValueError, match="reduction"):
        rlk.cross_entropy(h, W, t, w, reduction="max")
    with pytest.raises(TypeError):
        rlk.cross_entropy(h.half(), W, t, w)
    with pytest.raises(ValueError):
        rlk.cross_entropy(h, W[:, :32], t, w)
    with pytest.raises(ValueError):
        rlk.cross_entropy(h, W, t, w[:4])
    with pytest.raises(ValueError, match="contiguous"):
        rlk.cross_entropy(h.t().contiguous().t(), W, t, w)
    for bad in (dict(label_smoothing=1.0), dict(label_smoothing=-0.1), dict(z_loss=float("nan")), dict(inv_temp=0.0)):
        with pytest.raises(rlk.RlkError):
            rlk.cross_entropy(h, W, t, w, **bad)
        with pytest.raises(rlk.RlkError):
            rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, **bad)
    with pytest.raises(ValueError, match="total"):
        rlk.cross_entropy_backward(h, W, t, r.lse, g, None, w)
    with pytest.raises(ValueError):
        rlk.cross_entropy_backward(h, W, t, r.lse, g, None, w, reduction="none")
    with pytest.raises(TypeError):
        rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, grad_W=torch.zeros_like(W))
    with pytest.raises(TypeError, match="grad_dtype"):
        rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, grad_dtype=torch.float16)
    with pytest.raises(rlk.RlkError, match="workspace"):
        rlk.cross_entropy(h, W, t, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(rlk.RlkError, match="workspace"):
        rlk.cross_entropy_backward(h, W, t, r.lse, g, r.total, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
