"""GPU tests of the 4-bit weight operators: quantize_w4, dequantize_w4, linear_w4 and the
decode step logprob_w4, against plain implementations.

Quantising and reading back are exact (the same fp32 operations in numpy).  linear_w4
against the product in 64 bits: every product of a 16-bit x and a whole number up to 15 is
exact in fp32, so with A = sum_g s |sum of the group's |products|| only the additions round.
The tensor core's additions lose at most 2^-22 of the partial sum's magnitude each (they
may cut instead of rounding), a group makes at most 8 of them after its first instruction's
own sum of 16, and the groups and parts of K add with u = 2^-24 each over at most
ceil(K/32) + 16 steps:
  |y - y64| <= A (24 * 2^-22 + (K/32 + 16) 2^-24)
before the one rounding to the output type, which is monotonic: the output lies between the
rounded ends of that interval.
Row bits across batch sizes are equal."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import invariant_token_logprob_gb300 as rlk
    rlk.lib()


def weight(N, K, dtype, seed, std=0.02):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(N, K, generator=g) * std).to(DTYPES[dtype])


def ref_quantize(W, group, asymmetric):
    """(codes uint8 [N, K], scales, zeros) by the definition, in fp32."""
    N, K = W.shape
    G = -(-K // group)
    w = torch.zeros(N, G * group)
    w[:, :K] = W.float()
    w = w.view(N, G, group)
    if asymmetric:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        s = ((hi - lo) / 15).to(W.dtype)
    else:
        s = (w.abs().amax(2) / 7).to(W.dtype)
    s = torch.where(s == 0, torch.ones_like(s), s)
    f = s.float()[:, :, None]
    if asymmetric:
        z = torch.round(-lo[:, :, None] / f).clamp(0, 15)
        q = (torch.round(w / f) + z).clamp(0, 15)
        zeros = z[:, :, 0].to(torch.uint8)
    else:
        q = torch.round(w / f).clamp(-7, 7) + 8
        zeros = None
    return q.view(N, -1)[:, :K].to(torch.uint8), s, zeros


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("asymmetric", [False, True])
@pytest.mark.parametrize("shape", [(1, 32, 32), (3, 64, 128), (5, 160, 64), (129, 416, 128),
                                   (1000, 2080, 64), (77, 4096, 128), (10, 5120, 32)])
def test_quantize_and_read_back(shape, asymmetric, dtype):
    import invariant_token_logprob_gb300 as rlk
    N, K, group = shape
    W = weight(N, K, dtype, N + K)
    W[0, :group] = 0
    if N > 2:
        W[1] = W[1].abs()
        W[2] = 1e-7 if dtype == "fp16" else 1e-40
    codes, scales, zeros = rlk.quantize_w4(W.cuda(), group, asymmetric)
    q, s, z = ref_quantize(W, group, asymmetric)
    assert torch.equal(scales.cpu(), s)
    assert (zeros is None) == (z is None) and (z is None or torch.equal(zeros.cpu(), z))
    assert torch.equal(rlk.unpack_w4(codes).cpu(), q)
    assert torch.equal(rlk.pack_w4(q.cuda()), codes)
    sf = s.float().repeat_interleave(group, 1)[:, :K]
    zf = 8.0 if z is None else z.float().repeat_interleave(group, 1)[:, :K]
    values = (q.float() - zf) * sf
    assert torch.equal(rlk.dequantize_w4(codes, scales, zeros, group, torch.float32).cpu(), values)
    assert torch.equal(rlk.dequantize_w4(codes, scales, zeros, group).cpu(), values.to(W.dtype))
    err = (values - W.float()).abs()
    assert bool((err <= 0.57 * sf + 2 ** -24).all())  # half a step, and the scale's rounding


def test_quantize_every_step_of_the_grid():
    """Every multiple of an eighth of a step, ties included, for scales of every binade."""
    import invariant_token_logprob_gb300 as rlk
    rows = []
    for e in range(-100, 100, 3):
        x = torch.arange(-56, 57).float() / 8
        rows.append(torch.nn.functional.pad(x, (0, 15)) * 2.0 ** e)
    W = torch.stack(rows).to(torch.bfloat16)
    for asym in (False, True):
        codes, scales, zeros = rlk.quantize_w4(W.cuda(), 128, asym)
        q, s, z = ref_quantize(W, 128, asym)
        assert torch.equal(scales.cpu(), s) and torch.equal(rlk.unpack_w4(codes).cpu(), q)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantize_every_maximum(dtype):
    """Every finite positive value of the type as a group's maximum (subnormal ones too): the
    scales' rounding, and codes at whole and half steps of them."""
    import invariant_token_logprob_gb300 as rlk
    top = torch.arange(1, 0x7f80 if dtype == "bf16" else 0x7c00, dtype=torch.int32).to(torch.int16)
    m = top.view(DTYPES[dtype])
    f = torch.linspace(-1, 1, 31)
    f[15] = 0.0
    W = torch.cat([m.float()[:, None], m.float()[:, None] * f], 1).to(DTYPES[dtype])
    for asym in (False, True):
        codes, scales, zeros = rlk.quantize_w4(W.cuda(), 32, asym)
        q, s, z = ref_quantize(W, 32, asym)
        assert torch.equal(scales.cpu(), s), asym
        assert torch.equal(rlk.unpack_w4(codes).cpu(), q), asym
        assert z is None or torch.equal(zeros.cpu(), z)


def make(T, N, K, group, dtype, zeros, seed):
    """Codes over the whole range, scales over some binades, zero points of every value."""
    g = torch.Generator().manual_seed(seed)
    G = -(-K // group)
    q = torch.randint(0, 16, (N, K), generator=g).to(torch.uint8)
    s = (torch.rand(N, G, generator=g) + 0.5) * 2.0 ** torch.randint(-9, -3, (N, G), generator=g)
    z = torch.randint(0, 16, (N, G), generator=g).to(torch.uint8) if zeros else None
    x = torch.randn(T, K, generator=g)
    return x.to(DTYPES[dtype]), q, s.to(DTYPES[dtype]), z


def ref_linear(x, q, s, z, group):
    """(product, sum of magnitudes) in 64 bits."""
    K = q.shape[1]
    d = "cuda"
    sf = s.to(d).double().repeat_interleave(group, 1)[:, :K]
    zf = 8.0 if z is None else z.to(d).double().repeat_interleave(group, 1)[:, :K]
    w = (q.to(d).double() - zf) * sf
    xd = x.to(d).double()
    return (xd @ w.t()).cpu().numpy(), (xd.abs() @ w.abs().t()).cpu().numpy()


def check_linear(y, x, q, s, z, group, out, what=""):
    want, mag = ref_linear(x, q, s, z, group)
    K = q.shape[1]
    tol = mag * (24 * 2.0 ** -22 + (K / 32 + 16) * 2.0 ** -24)
    lo, hi = (torch.from_numpy(want + sign * tol).to(DTYPES[out]).double().numpy() for sign in (-1, 1))
    got = y.double().cpu().numpy()
    far = np.maximum(lo - got, got - hi)
    assert np.all(far <= 0), f"{what}: {far.max():.3g} beyond the tolerance"


@pytest.mark.parametrize("dtype,out,zeros", [("bf16", "fp32", False), ("bf16", "bf16", True),
                                             ("fp16", "fp32", True), ("fp16", "fp16", False)])
@pytest.mark.parametrize("shape", [(1, 1, 32, 32), (1, 128, 128, 128), (2, 129, 160, 64), (3, 255, 4096, 128),
                                   (5, 1000, 2080, 64), (8, 300, 96, 32), (9, 513, 1056, 32),
                                   (16, 256, 4128, 128), (17, 130, 512, 128), (31, 77, 5120, 64),
                                   (33, 200, 1024, 32), (64, 384, 4096, 128), (65, 100, 992, 64),
                                   (130, 50, 256, 128), (300, 140, 320, 32)])
def test_linear_matches_64_bits(shape, dtype, out, zeros):
    import invariant_token_logprob_gb300 as rlk
    T, N, K, group = shape
    x, q, s, z = make(T, N, K, group, dtype, zeros, T * N + K)
    y = rlk.linear_w4(x.cuda(), rlk.pack_w4(q.cuda()), s.cuda(), None if z is None else z.cuda(), group,
                      out_dtype=DTYPES[out])
    rlk.check_device_error()
    check_linear(y, x, q, s, z, group, out, str(shape))


def test_linear_exact_products():
    """Whole numbers small enough for every partial sum to be exact: the result is the
    integer product, for every group size, with all zero points."""
    import invariant_token_logprob_gb300 as rlk
    for T, N, K, group in ((1, 300, 1024, 32), (7, 131, 608, 64), (20, 260, 1152, 128), (64, 129, 352, 32)):
        g = torch.Generator().manual_seed(K)
        q = torch.randint(0, 16, (N, K), generator=g).to(torch.uint8)
        G = -(-K // group)
        z = torch.randint(0, 16, (N, G), generator=g).to(torch.uint8)
        s = 2.0 ** torch.randint(-1, 2, (N, G), generator=g)
        x = torch.randint(-4, 5, (T, K), generator=g).float()
        want = x.double() @ ((q.double() - z.double().repeat_interleave(group, 1)[:, :K])
                             * s.double().repeat_interleave(group, 1)[:, :K]).t()
        for dt in (torch.bfloat16, torch.float16):
            y = rlk.linear_w4(x.to(dt).cuda(), rlk.pack_w4(q.cuda()), s.to(dt).cuda(), z.cuda(), group)
            assert torch.equal(y.double().cpu(), want), (T, N, K, group, dt)


@pytest.mark.parametrize("N,K,group", [(5000, 4096, 128), (1024, 2080, 64), (40000, 1024, 32)])
def test_row_bits_do_not_depend_on_the_batch(N, K, group):
    import invariant_token_logprob_gb300 as rlk
    T = 200
    x, q, s, z = make(T, N, K, group, "bf16", True, 3)
    codes, s, z, x = rlk.pack_w4(q.cuda()), s.cuda(), z.cuda(), x.cuda()
    full = rlk.linear_w4(x, codes, s, z, group)
    for n in (1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 128, 129):
        part = rlk.linear_w4(x[T - n:].clone(), codes, s, z, group)
        assert torch.equal(part.view(torch.int32), full[T - n:].view(torch.int32)), n
    again = rlk.linear_w4(x, codes, s, z, group)
    assert torch.equal(again.view(torch.int32), full.view(torch.int32))
    nan = x.clone()
    nan[0] = float("nan")
    mixed = rlk.linear_w4(nan, codes, s, z, group)
    assert bool(torch.isnan(mixed[0]).all())
    assert torch.equal(mixed[1:].view(torch.int32), full[1:].view(torch.int32)), "rows mix"


def test_linear_reads_nothing_beyond_its_operands():
    """NaN around x and outputs around y: rows and columns beyond the operands stay out."""
    import invariant_token_logprob_gb300 as rlk
    T, N, K, group = 3, 131, 416, 64
    x, q, s, z = make(T, N, K, group, "fp16", True, 5)
    xb = torch.full((T + 8, K), float("nan"), dtype=torch.float16, device="cuda")
    xb[:T] = x.cuda()
    yb = torch.full((T + 8, N), 7.0, device="cuda")
    rlk.linear_w4(xb[:T], rlk.pack_w4(q.cuda()), s.cuda(), z.cuda(), group, out=yb[:T])
    check_linear(yb[:T], x, q, s, z, group, "fp32")
    assert bool((yb[T:] == 7).all())


def test_decode_step_in_a_graph_and_on_a_stream():
    """logprob_w4: the head's product, then log probabilities, entropy and alternatives."""
    import invariant_token_logprob_gb300 as rlk
    from test_gpu_token_logprobs import check_forward, ref_forward
    T, V, K = 5, 3001, 512
    W = weight(V, K, "bf16", 4, 0.05).cuda()
    codes, scales, _ = rlk.quantize_w4(W)
    h = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    tg = torch.tensor([0, 5, -1, 3000, 17], dtype=torch.int32, device="cuda")
    r = rlk.logprob_w4(h, codes, scales, tg, top_k=6)
    logits = rlk.linear_w4(h, codes, scales)
    check_forward(r, ref_forward(logits.double().cpu().numpy(), tg.cpu().numpy(), 1.0, 6), V, 1.0)
    buf = torch.empty(T, V, device="cuda")
    out = [torch.zeros_like(a) for a in r]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rlk.logprob_w4(h, codes, scales, tg, top_k=6, logits=buf, out=out, stream=s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rlk.logprob_w4(h, codes, scales, tg, top_k=6, logits=buf, out=out, stream=s)
        for a in out:
            a.zero_()
        for _ in range(3):
            g.replay()
    s.synchronize()
    rlk.check_device_error()
    for a, b in zip(out, r):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_refusals():
    import invariant_token_logprob_gb300 as rlk
    T, N, K, group = 2, 40, 256, 64
    x, q, s, z = make(T, N, K, group, "bf16", True, 1)
    x, c, s, z = x.cuda(), rlk.pack_w4(q.cuda()), s.cuda(), z.cuda()
    rlk.linear_w4(x, c, s, z, group)
    for bad, err in [(dict(x=x.half()), TypeError), (dict(x=x.float()), TypeError), (dict(x=x.cpu()), ValueError),
                     (dict(x=x[:, :224].contiguous()), ValueError), (dict(x=x[0]), ValueError),
                     (dict(codes=c.long()), TypeError), (dict(codes=c[:, :24].contiguous()), ValueError),
                     (dict(scales=s.float()), TypeError), (dict(scales=s[:, :3].contiguous()), ValueError),
                     (dict(zeros=z.int()), TypeError), (dict(zeros=z[:5]), ValueError), (dict(group=48), ValueError),
                     (dict(group=128), ValueError), (dict(out_dtype=torch.float16), TypeError),
                     (dict(out=torch.empty(T, N + 1, device="cuda")), ValueError)]:
        kw = dict(x=x, codes=c, scales=s, zeros=z, group=group)
        kw.update(bad)
        with pytest.raises(err):
            rlk.linear_w4(**kw)
    W = weight(N, K, "bf16", 2).cuda()
    for bad, err in [(dict(W=W.float()), TypeError), (dict(W=W[:, :40].contiguous()), ValueError),
                     (dict(W=W.cpu()), ValueError), (dict(W=W.t()), ValueError), (dict(group=16), ValueError),
                     (dict(out=(c, s, z), asymmetric=False), ValueError)]:
        kw = dict(W=W, group=group)
        kw.update(bad)
        with pytest.raises(err):
            rlk.quantize_w4(**kw)
    with pytest.raises(TypeError):
        rlk.dequantize_w4(c, s, z, group, torch.float16)
    with pytest.raises(ValueError):
        rlk.pack_w4(q.int().cuda())
    with pytest.raises(rlk.RlkError):  # x not on a 16-byte boundary
        flat = torch.zeros(T * K + 1, dtype=torch.bfloat16, device="cuda")
        rlk.linear_w4(flat[1:].view(T, K), c, s, z, group)
    assert rlk.linear_w4(x[:0], c, s, z, group).shape == (0, N)
    assert rlk.linear_w4(x, c[:0], s[:0], z[:0], group).shape == (T, 0)


@pytest.mark.parametrize("T,N,K,group", [(1, 130, 1024, 128), (3, 258, 128, 128), (20, 130, 256, 128),
                                         (64, 1154, 768, 128), (9, 163, 32, 32), (2, 32002, 1024, 128)])
def test_linear_with_few_groups_per_row(T, N, K, group):
    """Few groups per row and a few rows behind a multiple of 128: the words copied for the
    scales and zero points of a tile's last rows span more rows than are left."""
    import invariant_token_logprob_gb300 as rlk
    for zeros in (False, True):
        x, q, s, z = make(T, N, K, group, "bf16", zeros, N + K)
        y = rlk.linear_w4(x.cuda(), rlk.pack_w4(q.cuda()), s.cuda(), None if z is None else z.cuda(), group)
        rlk.check_device_error()
        check_linear(y, x, q, s, z, group, "fp32", str((T, N, K, group, zeros)))


def test_zero_points_off_a_word():
    """A view into a packed buffer: read back as it is, refused by the product."""
    import invariant_token_logprob_gb300 as rlk
    T, N, K, group = 2, 40, 256, 64
    x, q, s, z = make(T, N, K, group, "bf16", True, 11)
    x, c, s, z = x.cuda(), rlk.pack_w4(q.cuda()), s.cuda(), z.cuda()
    flat = torch.zeros(z.numel() + 4, dtype=torch.uint8, device="cuda")
    want = rlk.dequantize_w4(c, s, z, group)
    y = rlk.linear_w4(x, c, s, z, group)
    for off in (1, 2, 3, 4):
        view = flat[off:off + z.numel()].view_as(z)
        view.copy_(z)
        assert torch.equal(rlk.dequantize_w4(c, s, view, group), want)
        if off < 4:
            with pytest.raises(rlk.RlkError):
                rlk.linear_w4(x, c, s, view, group)
        else:
            assert torch.equal(rlk.linear_w4(x, c, s, view, group), y)


@pytest.mark.parametrize("mode", [1, 2])
def test_bounded_wait_runs_out_and_context_survives(mode):
    """No copy is issued, or no stage is consumed after every copy was issued: the wait that
    runs out is reported, every teardown wait ends in time, and the next call is right."""
    import ctypes
    import time

    import invariant_token_logprob_gb300 as rlk
    x, q, s, _ = make(1, 128, 1024, 128, "bf16", False, mode)
    x, codes, s = x.cuda(), rlk.pack_w4(q.cuda()), s.cuda()
    y = torch.full((1, 128), 7.0, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rlk.check_device_error()

    def selftest(m):
        return rlk.lib().rlk_selftest_wait_timeout_w4(*(ctypes.c_void_p(t.data_ptr()) for t in (x, codes, s, y)),
                                                      m, stream)

    assert selftest(0) == 1 and selftest(3) == 1
    t0 = time.time()
    assert selftest(mode) == 0
    assert rlk.take_device_errors() == (1, 0)  # a wait ran out, and no teardown wait did
    assert 1.0 < time.time() - t0 < 30.0
    assert bool((y == 7).all())
    rlk.check_device_error()
    rlk.linear_w4(x, codes, s, out=y)
    check_linear(y, x.cpu(), q, s.cpu(), None, 128, "fp32")
