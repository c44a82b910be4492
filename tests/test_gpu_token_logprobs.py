"""GPU tests of token_logprobs (log probabilities, entropy and top alternatives from
logits) and its gradient, against a plain implementation in 64 bits.

Tolerances, derived from the arithmetic (u = 2^-24, the fp32 unit roundoff):
  S = sum e^{z-m}: every term is an exp2 with relative error <= 2^-22 and a rounded
      argument, summed along chains of at most V/256 + 32 additions:
      rel(S) <= eS = (V/256 + 32) u + 2^-20
  lse     <= eS + 4 u |lse|
  logp    <= eS + 8 u (1 + |z_t - m| + log V)         (top alternatives too)
  entropy <= 3 (1 + log V) eS                         (|U/S| <= log V)
  grad    <= tol = 1.01 inv_temp [ p (|A| + |g_H| |lp + H|) (8 u (|z| + |lse|) + 2^-20) + 4 u
             (|g_logp| + sum |g_top|) ] before its one rounding, which is monotonic: the
             output lies between the rounded ends of the formula's value -+ tol
Ids are exact.  Invariance is bitwise."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IT = float(np.float32(1 / 0.7))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import invariant_token_logprob_gb300 as rlk
    rlk.lib()
    rlk.take_device_errors()


def pack_bits(keep):
    """bool [T, V] -> int32 words [T, ceil(V/32)] (numpy)."""
    T, V = keep.shape
    words = (V + 31) // 32
    b = np.zeros((T, words * 32), dtype=np.uint8)
    b[:, :V] = keep
    return np.packbits(b, axis=1, bitorder="little").view(np.int32)


def ref_forward(x, targets, it, top_k, keep=None):
    """The definition in 64 bits; x float64 [T, V], row by row."""
    T, V = x.shape
    out = dict(logp=np.zeros(T), lse=np.zeros(T), entropy=np.zeros(T),
               top_ids=np.full((T, top_k), -1), top_logp=np.full((T, top_k), -np.inf), zspan=np.zeros(T))
    for t in range(T):
        ok = x[t] != -np.inf
        if keep is not None:
            ok &= keep[t]
        v = np.nonzero(ok)[0]
        tg = targets[t]
        if v.size == 0:
            out["lse"][t] = -np.inf
            out["logp"][t] = -np.inf if 0 <= tg < V else 0.0
            continue
        z = x[t, v] * it
        m = z.max()
        logs = math.log(np.exp(z - m).sum())
        lp = (z - m) - logs  # not z - lse: log S would be lost beside a huge m
        out["lse"][t] = m + logs
        out["entropy"][t] = -(np.exp(lp) * lp).sum()
        if 0 <= tg < V:
            out["logp"][t] = (x[t, tg] * it - m) - logs if ok[tg] else -np.inf
            if ok[tg]:
                out["zspan"][t] = m - x[t, tg] * it
        order = v[np.lexsort((v, -x[t, v]))][:top_k]
        out["top_ids"][t, :order.size] = order
        out["top_logp"][t, :order.size] = (x[t, order] * it - m) - logs
    return out


def check_forward(got, ref, V, it, what=""):
    eS = (V / 256 + 32) * U + 2.0 ** -20
    logv = math.log(max(2, V))
    lp, lse, ent, ids, top = [x.cpu().numpy().astype(np.float64) if x.dtype.is_floating_point
                              else x.cpu().numpy() for x in got]

    def near(a, b, tol, name):
        inf = np.isinf(b)
        assert np.array_equal(a[inf], b[inf]), f"{what}: {name} at infinities"
        assert np.all(np.isfinite(a[~inf])), f"{what}: {name} not finite"
        bad = np.abs(a[~inf] - b[~inf]) > np.broadcast_to(tol, b.shape)[~inf]
        assert not bad.any(), f"{what}: {name}: {np.abs(a[~inf] - b[~inf]).max():.3g}"

    near(lse, ref["lse"], eS + 4 * U * np.abs(np.where(np.isinf(ref["lse"]), 0, ref["lse"])), "lse")
    near(lp, ref["logp"], eS + 8 * U * (1 + ref["zspan"] + logv), "logp")
    near(ent, ref["entropy"], np.full_like(ent, 3 * (1 + logv) * eS), "entropy")
    assert np.array_equal(ids, ref["top_ids"]), f"{what}: ids"
    span = np.abs(np.where(np.isinf(ref["top_logp"]), 0, ref["top_logp"]))
    near(top, ref["top_logp"], eS + 8 * U * (1 + span + 2 * logv), "top_logp")


def make(T, V, dtype, seed, it=1.0, masked=False, pad=0, offset=0, std=2.5):
    """logits (a view with `pad` columns behind and `offset` before each row), targets, keep."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, V, generator=g) * std
    hot = torch.randint(0, V, (T, min(4, V)), generator=g)
    x.scatter_add_(1, hot, torch.rand(T, hot.shape[1], generator=g) * 8 + 2)
    buf = torch.zeros(T, offset + V + pad, dtype=DTYPES[dtype], device="cuda")
    buf.fill_(float("nan"))
    logits = buf[:, offset:offset + V]
    logits.copy_(x.to(DTYPES[dtype]))
    targets = torch.where(torch.rand(T, generator=g) < 0.6, hot[:, 0],
                          torch.randint(0, V, (T,), generator=g)).to(torch.int32)
    if T > 3:
        targets[1] = -1
    keep = None
    if masked:
        keep = torch.rand(T, V, generator=g) < torch.rand(T, 1, generator=g)
        keep.scatter_(1, hot[:, :2], True)
        if T > 2:
            keep[T // 2] = False
            keep[0] = False
            keep[0, V // 3] = True
        logits.masked_fill_((torch.rand(T, V, generator=g) < 0.05).cuda() & ~keep.cuda(), float("nan"))
        logits.masked_fill_((torch.rand(T, V, generator=g) < 0.02).cuda() & ~keep.cuda(), float("inf"))
    return logits, targets.cuda(), keep


def bits_of(keep):
    return None if keep is None else torch.from_numpy(pack_bits(keep.numpy())).cuda()


def call(logits, targets, top_k, keep, it, **kw):
    import invariant_token_logprob_gb300 as rlk
    r = rlk.token_logprobs(logits, targets, top_k=top_k, allowed=bits_of(keep), inv_temp=it, **kw)
    rlk.check_device_error()
    return r


def x64(logits):
    return logits.float().cpu().numpy().astype(np.float64)


SHAPES = [(1, 1), (1, 7), (2, 31), (3, 33), (5, 255), (4, 256), (3, 257), (2, 1000), (7, 2049),
          (3, 4097), (2, 32768), (9, 32761), (2, 50001)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_matches_64_bits(shape, dtype):
    T, V = shape
    for k, (masked, pad, offset, it) in enumerate([(False, 0, 0, 1.0), (True, 0, 0, IT),
                                                   (False, 3, 1, 0.5), (True, 5, 3, 1.0)]):
        logits, tg, keep = make(T, V, dtype, 100 * V + k, masked=masked, pad=pad, offset=offset)
        for top_k in (0, 1, 5, 32):
            got = call(logits, tg, top_k, keep, it)
            ref = ref_forward(x64(logits), tg.cpu().numpy(), it, top_k,
                              None if keep is None else keep.numpy())
            check_forward(got, ref, V, it, f"{shape} {dtype} {k} top_k={top_k}")


@pytest.mark.parametrize("T,V,dtype,top_k", [(1, 151936, "fp32", 20), (2, 151936, "bf16", 32),
                                             (33, 151937, "fp16", 5), (200, 32768, "bf16", 20),
                                             (1300, 5003, "fp16", 8), (1, 1000003, "fp32", 32)])
def test_forward_at_model_sizes(T, V, dtype, top_k):
    logits, tg, keep = make(T, V, dtype, V + T, masked=T < 100)
    got = call(logits, tg, top_k, keep, IT)
    rows = np.arange(T) if T * V < 2e7 else np.unique(np.r_[0, T // 2, T - 1, 7])
    ref = ref_forward(x64(logits)[rows], tg.cpu().numpy()[rows], IT, top_k,
                      None if keep is None else keep.numpy()[rows])
    check_forward([x[torch.from_numpy(rows).cuda()] for x in got], ref, V, IT)


def test_ties_and_orders():
    """Equal logits keep the order of their indices, also where all are equal, where +0 and
    -0 meet, and for rows sorted either way (the most candidates in a run of columns)."""
    V = 70001
    rows = [torch.zeros(V), torch.arange(V).float(), -torch.arange(V).float(),
            (torch.arange(V) % 7).float(), torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0),
            torch.where(torch.arange(V) > V - 10, 1.0, 0.0),
            torch.full((V,), float(torch.finfo(torch.float32).min))]
    big = torch.zeros(V)
    big[300:2300] = torch.arange(2000).float() + 1.0
    rows.append(big)
    strided = torch.zeros(V)  # large values at a fixed distance, in runs of eight
    idx = (torch.arange(0, V - 8, 256)[:, None] + torch.arange(8)).reshape(-1)
    strided[idx] = 5.0 + (torch.arange(idx.numel()) % 977) / 977.0
    rows.append(strided)
    x = torch.stack(rows)
    tg = torch.tensor([V - 1, V - 1, 0, 6, 1, V - 1, 5, 2299, 0], dtype=torch.int32)
    for top_k in (1, 20, 32):
        got = call(x.cuda(), tg.cuda(), top_k, None, 1.0)
        ref = ref_forward(x.double().numpy(), tg.numpy(), 1.0, top_k)
        assert np.array_equal(got.top_ids.cpu().numpy(), ref["top_ids"]), top_k
        fine = torch.tensor([0, 3, 4, 5, 6, 8])
        check_forward([a[fine.cuda()] for a in got],
                      {k: v[fine.numpy()] for k, v in ref.items()}, V, 1.0)


def test_many_candidates_in_few_places():
    """All large logits lie where one lane of one strip reads them: every element of those
    places is a candidate, more than any buffer of candidates holds."""
    for V, dtype in ((151936, "fp32"), (600000, "fp32"), (151936, "bf16")):
        x = torch.zeros(1, V)
        strip = ((V + 63) // 64 + 7) // 8 * 8
        lane = torch.arange(32)
        base = torch.arange(0, strip, 256)
        for s in range(2):
            idx = (s * strip + base[:, None, None] + 8 * lane[None, :, None] + torch.arange(8)).reshape(-1)
            idx = idx[idx < min((s + 1) * strip, V)]
            x[0, idx] = 4.0 + torch.rand(idx.numel(), generator=torch.Generator().manual_seed(s))
        x = x.to(DTYPES[dtype])
        tg = torch.zeros(1, dtype=torch.int32)
        got = call(x.cuda(), tg.cuda(), 32, None, 1.0)
        ref = ref_forward(x.double().numpy(), tg.numpy(), 1.0, 32)
        check_forward(got, ref, V, 1.0, f"{V} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_special_values(dtype):
    dt = DTYPES[dtype]
    V = 3000
    low = torch.finfo(dt).min
    g = torch.Generator().manual_seed(5)
    x = torch.randn(12, V, generator=g)
    x[0] = -math.inf                      # nothing left
    x[1, 1:] = -math.inf                  # one token
    x[2, : V // 2] = -math.inf            # half, the target among the missing
    x[3] = low                            # all at the type's lowest value
    x[4, 10:] = low                       # masked by the lowest value
    x[5, 7] = math.nan
    x[6, 7] = math.inf
    x[7] = 0.0
    x[8, ::2] = -math.inf
    x[9] = torch.finfo(dt).max / 4
    x[10, 5] = 60000.0                    # one token with everything
    x[11, V - 3:] = -math.inf
    x = x.to(dt).cuda()
    tg = torch.tensor([3, 0, 5, 1, 2, 7, 9, 3, 1, 2, 5, V - 1], dtype=torch.int32, device="cuda")
    got = call(x, tg, 6, None, 1.0)
    fine = [0, 1, 2, 4, 7, 8, 10, 11]
    with np.errstate(invalid="ignore"):  # the rows with NaN and inf
        ref = ref_forward(x64(x), tg.cpu().numpy(), 1.0, 6)
    check_forward([a[torch.tensor(fine).cuda()] for a in got], {k: v[fine] for k, v in ref.items()}, V, 1.0)
    for r in (3, 9):  # huge equal logits: a uniform row
        assert abs(float(got.logp[r]) + math.log(V)) <= 1e-5 * math.log(V)
        assert abs(float(got.entropy[r]) - math.log(V)) <= 1e-4
        assert got.top_ids[r].tolist() == list(range(6))
    for r in (5, 6):
        assert all(math.isnan(float(a[r])) for a in (got.logp, got.lse, got.entropy))
        assert torch.isnan(got.top_logp[r]).all()
    y = x64(x)[5]
    y[7] = -np.inf
    assert got.top_ids[5].tolist() == list(np.lexsort((np.arange(V), -y))[:6])
    assert int(got.top_ids[6, 0]) == 7


def test_target_out_of_range_is_counted():
    import invariant_token_logprob_gb300 as rlk
    logits, tg, _ = make(6, 500, "fp32", 3)
    tg = torch.tensor([0, -5, 500, 499, 2 ** 31 - 1, -1], dtype=torch.int32, device="cuda")
    r = rlk.token_logprobs(logits, tg)
    bits, rows = rlk.take_device_errors()
    assert (bits, rows) == (0, 2)
    lp = r.logp.cpu().numpy()
    assert lp[1] == lp[2] == lp[4] == lp[5] == 0 and lp[0] < 0 and lp[3] < 0
    assert rlk.take_device_errors() == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [151936, 32761])
def test_row_bits_do_not_depend_on_the_batch(V, dtype):
    """The same row alone, in small and in large batches, at other alignments and strides."""
    T = 700
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(T, V, generator=g, device="cuda") * 3).to(DTYPES[dtype])
    tg = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    full = [a.cpu() for a in call(x, tg, 20, None, IT)]

    def same(rows, got, what):
        for name, a, b in zip(("logp", "lse", "entropy", "ids", "top"), full, got):
            a, b = a[rows].contiguous(), b.cpu().contiguous()
            assert torch.equal(a.view(torch.int32), b.view(torch.int32)), (what, name)

    for n in (1, 2, 5, 17, 19, 40, 76, 77, 152, 153, 300, 304, 305, 608, 609):
        rows = torch.arange(T - n, T)
        same(rows, call(x[T - n:].clone(), tg[T - n:].clone(), 20, None, IT), f"T={n}")
    for offset in range(1, 8):
        buf = torch.empty(3, V + 8 + offset, dtype=x.dtype, device="cuda")
        view = buf[:, offset:offset + V]
        view.copy_(x[5:8])
        same(torch.arange(5, 8), call(view, tg[5:8].clone(), 20, None, IT), f"offset {offset}")
    no_top = call(x[:9].clone(), tg[:9].clone(), 0, None, IT)
    same(torch.arange(9), no_top[:3], "without alternatives")
    all_bits = torch.full((9, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    import invariant_token_logprob_gb300 as rlk
    same(torch.arange(9), rlk.token_logprobs(x[:9].clone(), tg[:9].clone(), 20, all_bits, IT), "mask of ones")


def test_streams_outputs_and_graph():
    import invariant_token_logprob_gb300 as rlk
    logits, tg, keep = make(4, 5000, "bf16", 9, masked=True)
    want = call(logits, tg, 5, keep, 1.0)
    bits = bits_of(keep)
    out = [torch.empty_like(a) for a in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rlk.token_logprobs(logits, tg, 5, bits, out=out, stream=s)
        g = torch.cuda.CUDAGraph()
        for a in out:
            a.zero_()
        with torch.cuda.graph(g, stream=s):
            rlk.token_logprobs(logits, tg, 5, bits, out=out, stream=s)
        g.replay()
    s.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 elements behind the first."""
    V, T = 1000, 3
    stride = (1 << 32) // 2 + 24
    buf = torch.empty(stride * (T - 1) + V, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (T, V), (stride, 1))
    g = torch.Generator(device="cuda").manual_seed(1)
    x.copy_(torch.randn(T, V, generator=g, device="cuda") * 3)
    tg = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    import invariant_token_logprob_gb300 as rlk
    r = rlk.token_logprobs(x, tg, 4)
    dense = rlk.token_logprobs(x.contiguous(), tg, 4)
    for a, b in zip(r, dense):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    ones = torch.ones(T, device="cuda")
    want = rlk.token_logprobs_backward(x.contiguous(), tg, dense.lse, grad_logp=ones)
    rlk.token_logprobs_backward(x, tg, r.lse, grad_logp=ones, out=x)
    assert torch.equal(x, want)


# ---------------------------------------------------------------- gradient
def ref_backward(x, targets, it, lse, ent, g, ids=None, keep=None):
    """The formula in 64 bits and the tolerance of the header, for [T, V]."""
    T, V = x.shape
    grad, tol = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        ok = x[t] != -np.inf
        if keep is not None:
            ok &= keep[t]
        if not ok.any() or lse[t] == -np.inf:
            continue
        z = np.where(ok, x[t], 0.0) * it
        lp = z - lse[t]
        p = np.exp(lp)
        gl = g["logp"][t] if 0 <= targets[t] < V else 0.0
        G = gl + (sum(w for i, w in zip(ids[t], g["top"][t]) if 0 <= i < V) if ids is not None else 0.0)
        a = g["lse"][t] - G
        d = p * (a - g["entropy"][t] * (lp + ent[t]))
        mag = np.zeros(V)
        if 0 <= targets[t] < V:
            d[targets[t]] += gl
            mag[targets[t]] += abs(gl)
        if ids is not None:
            for i, w in zip(ids[t], g["top"][t]):
                if 0 <= i < V:
                    d[i] += w
                    mag[i] += abs(w)
        sum_abs = abs(gl) + abs(g["lse"][t]) + (np.abs(g["top"][t]).sum() if ids is not None else 0.0)
        tol[t] = it * (p * (sum_abs + abs(g["entropy"][t]) * np.abs(lp + ent[t]))
                       * (8 * U * (np.abs(z) + abs(lse[t])) + 2.0 ** -20)
                       + p * abs(g["entropy"][t]) * 8 * U * (np.abs(z) + abs(lse[t]) + ent[t])
                       + 4 * U * mag)
        grad[t] = np.where(ok, d * it, 0.0)
        tol[t] = np.where(ok, tol[t], 0.0)
    return grad, tol


def beyond(got, want, tol, dtype):
    """How far `got` lies outside [want - 1.01 tol, want + 1.01 tol] rounded to its type."""
    lo, hi = (torch.from_numpy(want + sign * 1.01 * tol).to(DTYPES[dtype]).double().numpy() for sign in (-1, 1))
    return max(0.0, float(np.max(np.maximum(lo - got, got - hi))))


def grads(T, top_k, seed):
    g = torch.Generator().manual_seed(seed)
    return dict(logp=torch.randn(T, generator=g), lse=torch.randn(T, generator=g),
                entropy=torch.randn(T, generator=g), top=torch.randn(T, top_k, generator=g))


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 33), (4, 257), (7, 2049), (5, 5003), (2, 32768)])
def test_backward_matches_the_formula(shape, dtype):
    import invariant_token_logprob_gb300 as rlk
    T, V = shape
    for k, (masked, pad, offset, it, top_k) in enumerate([(False, 0, 0, 1.0, 0), (True, 0, 0, IT, 5),
                                                          (False, 3, 1, 0.5, 32), (True, 5, 3, 1.0, 0)]):
        logits, tg, keep = make(T, V, dtype, 7 * V + k, masked=masked, pad=pad, offset=offset)
        bits = bits_of(keep)
        r = rlk.token_logprobs(logits, tg, top_k, bits, it)
        g = grads(T, top_k, k)
        c = {n: v.cuda() for n, v in g.items()}
        top = dict(top_ids=r.top_ids, grad_top=c["top"]) if top_k else {}
        want, tol = ref_backward(x64(logits), tg.cpu().numpy(), it, f64(r.lse), f64(r.entropy),
                                 {n: f64(v) for n, v in g.items()}, r.top_ids.cpu().numpy() if top_k else None,
                                 None if keep is None else keep.numpy())

        def check(got, what):
            got = f64(got)
            far = beyond(got, want, tol, dtype)
            assert far == 0, f"{shape} {dtype} {k} {what}: {far:.3g} beyond the tolerance"

        got = rlk.token_logprobs_backward(logits, tg, r.lse, r.entropy, c["logp"], c["lse"], c["entropy"],
                                          allowed=bits, inv_temp=it, **top)
        check(got, "new tensor")
        buf = torch.full((T, V + 7), 3.0, dtype=DTYPES[dtype], device="cuda")
        rlk.token_logprobs_backward(logits, tg, r.lse, r.entropy, c["logp"], c["lse"], c["entropy"],
                                    allowed=bits, inv_temp=it, out=buf[:, 5:5 + V], **top)
        assert torch.equal(buf[:, 5:5 + V], got)
        assert bool((buf[:, :5] == 3).all()) and bool((buf[:, 5 + V:] == 3).all())
        rlk.token_logprobs_backward(logits, tg, r.lse, r.entropy, c["logp"], c["lse"], c["entropy"],
                                    allowed=bits, inv_temp=it, out=logits, **top)
        assert torch.equal(logits, got), "in place"


def test_backward_parts_and_ignored_rows():
    """Each gradient alone; ignored targets and ids of -1 count as nothing; a target that is
    also an alternative takes both."""
    import invariant_token_logprob_gb300 as rlk
    T, V, it = 6, 900, IT
    logits, tg, keep = make(T, V, "fp32", 77, masked=True)
    tg[2], tg[4] = -3, V
    bits = bits_of(keep)
    r = rlk.token_logprobs(logits, tg, 32, bits, it)
    rlk.take_device_errors()
    tg[5] = r.top_ids[5, 3]
    zero = {n: torch.zeros_like(v) for n, v in grads(T, 32, 0).items()}
    for name in ("logp", "lse", "entropy", "top"):
        g = dict(zero, **{name: grads(T, 32, 4)[name]})
        c = {n: v.cuda() for n, v in g.items()}
        kw = {"logp": dict(grad_logp=c["logp"]), "lse": dict(grad_lse=c["lse"]),
              "entropy": dict(grad_entropy=c["entropy"], entropy=r.entropy),
              "top": dict(grad_top=c["top"], top_ids=r.top_ids)}[name]
        got = f64(rlk.token_logprobs_backward(logits, tg, r.lse, allowed=bits, inv_temp=it, **kw))
        want, tol = ref_backward(x64(logits), tg.cpu().numpy(), it, f64(r.lse), f64(r.entropy),
                                 {n: f64(v) for n, v in g.items()}, r.top_ids.cpu().numpy(), keep.numpy())
        assert beyond(got, want, tol, "fp32") == 0, name
    both = dict(grad_logp=torch.ones(T, device="cuda"), grad_top=torch.ones(T, 32, device="cuda"),
                top_ids=r.top_ids)
    got = f64(rlk.token_logprobs_backward(logits, tg, r.lse, allowed=bits, inv_temp=it, **both))
    g = dict(zero, logp=torch.ones(T), top=torch.ones(T, 32))
    want, tol = ref_backward(x64(logits), tg.cpu().numpy(), it, f64(r.lse), f64(r.entropy),
                             {n: f64(v) for n, v in g.items()}, r.top_ids.cpu().numpy(), keep.numpy())
    assert beyond(got, want, tol, "fp32") == 0


def test_backward_special_rows():
    import invariant_token_logprob_gb300 as rlk
    V = 500
    x = torch.randn(5, V)
    x[0] = -math.inf
    x[1, 1:] = -math.inf
    x[2, 3] = math.nan
    x[3, 10:] = torch.finfo(torch.float32).min
    x = x.cuda()
    tg = torch.tensor([0, 0, 1, 2, 3], dtype=torch.int32, device="cuda")
    r = rlk.token_logprobs(x, tg)
    one = torch.ones(5, device="cuda")
    d = rlk.token_logprobs_backward(x, tg, r.lse, r.entropy, one, None, one)
    assert bool((d[0] == 0).all()) and bool(torch.isnan(d[2]).all())
    assert float(d[1].abs().max()) == 0.0  # a certain token
    assert bool(torch.isfinite(d[3]).all()) and bool((d[3, 10:] == 0).all())


def test_backward_against_differences():
    """Central differences of the 64-bit forward (step 1e-5: their error, about 1e-9, is far
    below the gradient's tolerance) for a random mix of all outputs, through autograd."""
    import invariant_token_logprob_gb300 as rlk
    T, V, it, top_k = 4, 40, 0.8, 4
    it = float(np.float32(it))
    logits, tg, keep = make(T, V, "fp32", 21, masked=True)
    tg[1] = int(np.nonzero(keep[1].numpy())[0][0])
    logits = torch.nan_to_num(logits, nan=0.0, posinf=0.0).contiguous()
    bits = bits_of(keep)
    x = logits.clone().requires_grad_()
    out = rlk.differentiable_token_logprobs(x, tg, top_k, bits, it)
    w = grads(T, top_k, 9)
    w["lse"][T // 2] = 0.0  # the row without tokens has lse -inf
    there = torch.isfinite(out.top_logp)
    loss = ((torch.where(torch.isfinite(out.logp), out.logp, 0.0) * w["logp"].cuda()).sum()
            + (torch.where(torch.isfinite(out.lse), out.lse, 0.0) * w["lse"].cuda()).sum()
            + (out.entropy * w["entropy"].cuda()).sum()
            + (torch.where(there, out.top_logp, 0.0) * w["top"].cuda()).sum())
    loss.backward()
    assert not out.top_ids.requires_grad
    ids = out.top_ids.cpu().numpy()
    base = x64(logits)

    def value(y, t):
        r = ref_forward(y[None], tg.cpu().numpy()[t:t + 1], it, 0, keep.numpy()[t:t + 1])
        if np.isinf(r["lse"][0]):
            return 0.0
        v = r["lse"][0] * float(w["lse"][t]) + r["entropy"][0] * float(w["entropy"][t])
        if np.isfinite(r["logp"][0]):
            v += r["logp"][0] * float(w["logp"][t])
        return v + sum((y[i] * it - r["lse"][0]) * float(w["top"][t, j])
                       for j, i in enumerate(ids[t]) if i >= 0)

    h = 1e-5
    got = f64(x.grad)
    for t in range(T):
        for v in range(V):
            up, dn = base[t].copy(), base[t].copy()
            up[v] += h
            dn[v] -= h
            want = (value(up, t) - value(dn, t)) / (2 * h)
            assert abs(got[t, v] - want) <= 1e-7 + 2e-5 * max(1.0, abs(want)), (t, v, got[t, v], want)


def test_autograd_skips_what_is_not_asked():
    import invariant_token_logprob_gb300 as rlk
    logits, tg, _ = make(5, 300, "bf16", 2)
    x = logits.clone().requires_grad_()
    r = rlk.differentiable_token_logprobs(x, tg)
    (-r.logp.mean()).backward()
    want = rlk.token_logprobs_backward(logits, tg, r.lse.detach(),
                                       grad_logp=torch.full((5,), -0.2, device="cuda"))
    assert x.grad.dtype == torch.bfloat16 and torch.equal(x.grad, want)


def test_refusals():
    import invariant_token_logprob_gb300 as rlk
    x, tg, _ = make(4, 100, "fp32", 1)
    bits = torch.zeros(4, 4, dtype=torch.int32, device="cuda")
    ok = rlk.token_logprobs(x, tg, 3, bits)
    for bad, err in [(dict(logits=x.double()), TypeError), (dict(logits=x.cpu()), ValueError),
                     (dict(logits=x[0]), ValueError), (dict(logits=x.t()), ValueError),
                     (dict(logits=x[:1].expand(4, 100)), ValueError),
                     (dict(logits=x[:, ::2], allowed=None), ValueError),
                     (dict(targets=tg.long()), TypeError), (dict(targets=tg[:2]), ValueError),
                     (dict(targets=tg.cpu()), ValueError), (dict(top_k=-1), ValueError),
                     (dict(top_k=33), ValueError), (dict(allowed=bits[:, :3].contiguous()), ValueError),
                     (dict(allowed=bits.bool()), TypeError), (dict(allowed=bits[:2]), ValueError),
                     (dict(inv_temp=0.0), rlk.RlkError), (dict(inv_temp=float("nan")), rlk.RlkError),
                     (dict(inv_temp=float("inf")), rlk.RlkError), (dict(inv_temp=-1.0), rlk.RlkError),
                     (dict(out=(ok.logp, ok.lse, ok.entropy, ok.top_ids[:, :2], ok.top_logp)), ValueError),
                     (dict(out=(ok.logp[:2], ok.lse, ok.entropy, ok.top_ids, ok.top_logp)), ValueError)]:
        kw = dict(logits=x, targets=tg, top_k=3, allowed=bits)
        kw.update(bad)
        with pytest.raises(err):
            rlk.token_logprobs(**kw)
    one = torch.ones(4, device="cuda")
    for bad, err in [(dict(grad_entropy=one), ValueError), (dict(grad_top=ok.top_logp), ValueError),
                     (dict(grad_top=ok.top_logp, top_ids=ok.top_ids[:, :2].contiguous()), ValueError),
                     (dict(grad_logp=one[:2]), ValueError), (dict(grad_logp=one.half()), TypeError),
                     (dict(lse=one[:3]), ValueError), (dict(out=x.half()), ValueError),
                     (dict(out=x[:2]), ValueError), (dict(inv_temp=0.0), rlk.RlkError)]:
        kw = dict(logits=x, targets=tg, lse=ok.lse)
        kw.update(bad)
        with pytest.raises(err):
            rlk.token_logprobs_backward(**kw)
    e = rlk.token_logprobs(x[:0], tg[:0], 3)
    assert e.logp.shape == (0,) and e.top_ids.shape == (0, 3)
    assert rlk.token_logprobs_backward(x[:0], tg[:0], ok.lse[:0]).shape == (0, 100)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V,pad,offset", [(33, 0, 0), (2049, 3, 1), (5008, 0, 0), (70003, 5, 3)])
def test_backward_is_zero_at_missing_tokens_whatever_comes_in(V, pad, offset, dtype):
    """Infinite and NaN gradients, factors that overflow, a NaN lse: masked tokens and tokens at
    -inf stay 0; where the row itself is NaN every other token is."""
    import invariant_token_logprob_gb300 as rlk
    T = 9
    x, tg, keep = make(T, V, dtype, V, masked=True, pad=pad, offset=offset)
    g = torch.Generator().manual_seed(V)
    gone = (torch.rand(T, V, generator=g) < 0.2)
    gone[:, 0] = False
    keep[:, 0] = True
    keep[T // 2] = False
    x.masked_fill_(gone.cuda(), -math.inf)
    x[7, 0] = math.nan  # allowed: the row is NaN
    tg[1] = 0
    bits = bits_of(keep)
    r = rlk.token_logprobs(x, tg, 3, bits)
    inf, nan, big = math.inf, math.nan, 3e38
    c = dict(grad_logp=torch.tensor([inf, nan, 1, 1, inf, -inf, 1, 1, big]),
             grad_lse=torch.tensor([0.0, 0, 0, inf, nan, 0, 1, 1, -big]),
             grad_entropy=torch.tensor([0.0, 0, big, 0, inf, nan, 1, 1, 1e37]),
             grad_top=torch.zeros(T, 3))
    c["grad_top"][6, 0] = nan
    c = {n: v.cuda() for n, v in c.items()}
    got = rlk.token_logprobs_backward(x, tg, r.lse, r.entropy, top_ids=r.top_ids, allowed=bits, **c)
    missing = gone | ~keep
    assert bool((got.cpu()[missing] == 0).all())
    assert bool(missing[T // 2].all())  # (a row without tokens)
    for row in (1, 5, 6, 7):
        assert bool(torch.isnan(got[row].cpu()[~missing[row]]).all()), row
    rlk.token_logprobs_backward(x, tg, r.lse, r.entropy, top_ids=r.top_ids, allowed=bits, out=x, **c)
    assert torch.equal(torch.isnan(x), torch.isnan(got)) and torch.equal(torch.nan_to_num(x), torch.nan_to_num(got))


def test_special_targets_in_special_rows():
    """In a row that a NaN makes NaN, a missing target keeps -inf, an ignored one 0 and places
    left over -inf; rows at the type's lowest value whose z leave fp32 count as empty."""
    import invariant_token_logprob_gb300 as rlk
    V = 300
    x = torch.randn(5, V, generator=torch.Generator().manual_seed(1))
    keep = torch.ones(5, V, dtype=torch.bool)
    x[:4, 7] = math.nan
    keep[:4, 9:] = False
    x[1, 3] = -math.inf
    x[4] = torch.finfo(torch.float32).min
    tg = torch.tensor([200, 3, -1, 2, 5], dtype=torch.int32)
    r = [a.cpu() for a in call(x.cuda(), tg.cuda(), 12, keep, 2.0)]
    logp, lse, entropy, ids, top = r
    assert torch.isnan(lse[:4]).all() and torch.isnan(entropy[:4]).all()
    assert logp[0] == -math.inf and logp[1] == -math.inf and logp[2] == 0 and torch.isnan(logp[3])
    for t, n in ((0, 8), (1, 7), (2, 8), (3, 8)):  # the tokens that are not NaN
        assert bool((ids[t, :n] >= 0).all()) and bool(torch.isnan(top[t, :n]).all())
        assert bool((ids[t, n:] == -1).all()) and bool((top[t, n:] == -math.inf).all())
    assert lse[4] == -math.inf and entropy[4] == 0 and logp[4] == -math.inf
    assert ids[4].tolist() == list(range(12)) and bool((top[4] == -math.inf).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [5, 257, 40001])
def test_forward_at_the_ends_of_inv_temp(V, dtype):
    """A temperature near 0 leaves the largest logit's tokens, equally likely; one near fp32's
    largest value leaves a uniform row."""
    T = 3
    x = (torch.arange(V) * 37 % V % 64).float().repeat(T, 1)
    x[1] *= -1
    x[2] += 0.5
    x = x.to(DTYPES[dtype])
    tg = torch.tensor([0, 0, int(x[2].float().argmax())], dtype=torch.int32)
    for it in (1e30, 2.3e38, 2.5e38, 3.4e38):
        got = [a.cpu() for a in call(x.cuda(), tg.cuda(), 2, None, it)]
        best = x.float().amax(1, keepdim=True)
        n = (x.float() == best).sum(1)
        logn = torch.log(n.double()).float()
        hit = (x.float() == best)[torch.arange(T), tg.long()]
        assert torch.allclose(got[2], logn, atol=1e-5), (it, got[2], logn)
        assert torch.allclose(got[0][hit], -logn[hit], atol=1e-5), it
        assert bool((got[0][~hit] < -1e25).all())
        assert not torch.isnan(got[4]).any() and torch.allclose(got[4][:, 0], -logn, atol=1e-5)
        assert not torch.isnan(got[1]).any()
    for it in (1e-44, 1e-39, 1e-36):
        got = [a.cpu() for a in call(x.cuda(), tg.cuda(), 2, None, it)]
        want = math.log(V)
        for a, w in ((got[0], -want), (got[1], want), (got[2], want), (got[4][:, 0], -want)):
            assert torch.allclose(a, torch.full_like(a, w), atol=1e-4, rtol=1e-5), (it, a, w)


@pytest.mark.parametrize("V,dtype", [(151936, "fp32"), (600000, "fp32"), (151936, "bf16"), (300001, "fp16")])
@pytest.mark.parametrize("order", ["up", "down", "any", "equal"])
def test_many_candidates_where_one_lane_reads_them(V, dtype, order):
    """Strip s gives its lane l the elements 256 s + 8 l + 16384 n + (0..7): all large logits lie
    in one lane's place, in one strip's, or in the same lanes of all strips, where every token
    is a candidate, more than the lists hold; in rows for one CTA and for clusters."""
    i = torch.arange(V)
    strip, lane = i // 256 % 64, i // 8 % 32
    places = [(strip == 3) & (lane == 9), strip == 0, (strip == 62) | (strip == 17), lane == 31,
              (strip < 40) & (lane < 7)]
    x = torch.zeros(len(places), V)
    g = torch.Generator().manual_seed(V)
    for r, p in enumerate(places):
        n = int(p.sum())
        step = {"up": torch.arange(n), "down": -torch.arange(n), "any": torch.randperm(n, generator=g),
                "equal": torch.zeros(n, dtype=torch.long)}[order]
        x[r, p] = 4.0 + step.float() * (4.0 / n)
    x = x.to(DTYPES[dtype])
    tg = torch.zeros(len(places), dtype=torch.int32)
    ref = ref_forward(x.double().numpy(), tg.numpy(), 1.0, 32)
    for copies in (1, 8, 40):  # clusters of eight down to one CTA per row
        got = call(x.cuda().repeat(copies, 1), tg.cuda().repeat(copies), 32, None, 1.0)
        for c in {0, copies - 1}:
            rows = slice(c * len(places), (c + 1) * len(places))
            check_forward([a[rows] for a in got], ref, V, 1.0, f"{V} {dtype} {order} {copies}")


def bits(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [151936, 32761])
def test_masked_row_bits_and_gradient_bits_do_not_depend_on_the_batch(V, dtype):
    """Masked rows, and the gradient of all outputs: the same rows alone, in other batches, at
    other alignments and strides, of the logits and of the gradient, and in place."""
    import invariant_token_logprob_gb300 as rlk
    T, top_k = 320, 8
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(T, V, generator=g, device="cuda") * 3).to(DTYPES[dtype])
    x[5, ::3] = -math.inf
    tg = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    allowed = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, (V + 31) // 32), generator=g, device="cuda", dtype=torch.int32)
    allowed[T - 3] = 0
    allowed[T - 4] = 1 << 5
    c = {n: v.cuda() for n, v in grads(T, top_k, 3).items()}

    def grad(r, logits, sl, mask, **kw):
        return rlk.token_logprobs_backward(
            logits, tg[sl], r.lse, r.entropy, grad_logp=c["logp"][sl], grad_lse=c["lse"][sl], grad_entropy=c["entropy"][sl],
            top_ids=r.top_ids, grad_top=c["top"][sl], allowed=mask, inv_temp=IT, **kw)

    for mask in (allowed, None):
        full = rlk.token_logprobs(x, tg, top_k, mask, IT)
        full_grad = grad(full, x, slice(0, T), mask)
        for n in (1, 2, 3, 7, 19, 38, 39, 76, 153, 304):
            sl = slice(T - n, T)
            part = None if mask is None else mask[sl]
            r = rlk.token_logprobs(x[sl], tg[sl], top_k, part, IT)
            for a, b in zip(r, full):
                assert torch.equal(bits(a), bits(b[sl])), (n, "forward")
            assert torch.equal(bits(grad(r, x[sl], sl, part)), bits(full_grad[sl])), (n, "gradient")
        sl = slice(T - 5, T)
        part = None if mask is None else mask[sl]
        for off_in, off_out in ((0, 1), (1, 0), (3, 5), (7, 7), (2, 6)):
            buf = torch.empty(5, V + 9, dtype=x.dtype, device="cuda")
            view = buf[:, off_in:off_in + V]
            view.copy_(x[sl])
            r = rlk.token_logprobs(view, tg[sl], top_k, part, IT)
            for a, b in zip(r, full):
                assert torch.equal(bits(a), bits(b[sl])), (off_in, "forward")
            out = torch.empty(5, V + 11, dtype=x.dtype, device="cuda")[:, off_out:off_out + V]
            grad(r, view, sl, part, out=out)
            assert torch.equal(bits(out), bits(full_grad[sl])), (off_in, off_out, "gradient")
            grad(r, view, sl, part, out=view)
            assert torch.equal(bits(view), bits(full_grad[sl])), (off_in, "in place")
    rlk.check_device_error()
