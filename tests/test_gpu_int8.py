"""GPU tests of the 8-bit integer operators: quantize_int8, dequantize_int8, linear_int8 and the
decode step logprob_int8.

Everything here is exact: quantising and reading back are single fp32 operations, done again in
numpy; the product's sum is one of whole numbers, taken here in 64 bits, and what follows it (one
rounding to fp32, two fp32 products, one rounding to the output type) is done again step by step."""
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
    rlk.take_device_errors()


def normal(rows, K, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, K, generator=g) * std).to(DTYPES[dtype])


def ref_quantize(x):
    """(codes int8, scales f32) by the definition, numpy's fp32 divisions."""
    x = x.float().numpy()
    s = np.abs(x).max(1) / np.float32(127)
    s = np.where(s == 0, np.float32(1), s).astype(np.float32)
    q = np.clip(np.rint((x / s[:, None]).astype(np.float32)), -127, 127)
    return torch.from_numpy(q.astype(np.int8)), torch.from_numpy(s)


def ref_linear(qx, sx, qw, sw, out):
    """The product in whole numbers (float64 holds them: |sum| < 2^31), then the steps in fp32."""
    sums = qx.double() @ qw.double().T
    assert float(sums.abs().max()) < 2.0 ** 31
    return ((sums.float() * sx[:, None]) * sw[None]).to(DTYPES[out])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 16), (3, 32), (1, 4096), (7, 5152), (2050, 4096), (2049, 2064), (5000, 112),
                                   (2100, 1040), (3, 32768), (2, 70000)])
def test_quantize_and_read_back(shape, dtype):
    import invariant_token_logprob_gb300 as rlk
    rows, K = shape
    x = normal(rows, K, dtype, rows + K)
    x[0, :] *= 30
    if rows > 2:
        x[1] = 0
        x[2] = x[2].abs() * (1e-6 if dtype == "fp16" else 1e-38)
    codes, scales = rlk.quantize_int8(x.cuda())
    q, s = ref_quantize(x)
    assert torch.equal(scales.cpu(), s) and torch.equal(codes.cpu(), q)
    for out in ("fp32", "bf16", "fp16"):
        y = rlk.dequantize_int8(codes, scales, out_dtype=DTYPES[out])
        assert torch.equal(y.cpu(), (q.float() * s[:, None]).to(DTYPES[out]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantize_every_maximum(dtype):
    """Every positive finite number as a row's maximum, next to numbers around the ties of its
    grid and random ones below it: the quotients are IEEE's, so the codes are the definition's."""
    import invariant_token_logprob_gb300 as rlk
    top = torch.arange(1, 0x7F80 if dtype == "bf16" else 0x7C00, dtype=torch.int16).view(DTYPES[dtype]).cuda()
    steps = (torch.arange(-127, 127, device="cuda") + 0.5) / 127
    u = torch.rand(len(top), 2 * 256 - 254 - 1, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 2 - 1
    x = (top.float()[:, None] * torch.cat([torch.ones(len(top), 1, device="cuda"), steps.expand(len(top), -1), u], 1))
    x = torch.minimum(torch.maximum(x, -top.float()[:, None]), top.float()[:, None]).to(DTYPES[dtype]).contiguous()
    assert x.shape[1] == 512
    codes, scales = rlk.quantize_int8(x)
    s = x.float().abs().amax(1) / torch.full((), 127.0, device="cuda")  # (a plain number would be multiplied)
    s = torch.where(s == 0, torch.ones_like(s), s)
    assert torch.equal(scales, s)
    # a quotient of fp32 numbers in 64 bits, rounded to 32, is the fp32 quotient
    q = torch.round((x.double() / s.double()[:, None]).float()).clamp(-127, 127)
    assert torch.equal(codes.float(), q)


SHAPES = [(1, 1, 16), (1, 128, 128), (2, 129, 160), (3, 255, 4096), (5, 1009, 2080), (8, 300, 5152), (9, 300, 1040),
          (13, 5119, 5152), (16, 640, 256), (17, 200, 1024), (33, 257, 1040), (64, 4096, 4096), (65, 130, 2064),
          (100, 1, 4096), (192, 384, 512), (193, 129, 272), (300, 1000, 3088), (513, 777, 96), (1, 151936, 64)]


@pytest.mark.parametrize("x,out", [("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "bf16"), ("int8", "fp32")])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_is_exact(shape, x, out):
    import invariant_token_logprob_gb300 as rlk
    T, N, K = shape
    qw, sw = ref_quantize(normal(N, K, "bf16", N + K, 0.02))
    if x == "int8":
        g = torch.Generator().manual_seed(T)
        qx = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8)
        sx = torch.rand(T, generator=g) + 0.1
        y = rlk.linear_int8(qx.cuda(), qw.cuda(), sw.cuda(), x_scales=sx.cuda(), out_dtype=DTYPES[out])
    else:
        a = normal(T, K, x, T + K)
        a[0, 0] = 9
        qx, sx = ref_quantize(a)
        y = rlk.linear_int8(a.cuda(), qw.cuda(), sw.cuda(), out_dtype=DTYPES[out])
    assert torch.equal(y.cpu(), ref_linear(qx, sx, qw, sw, out))
    assert rlk.take_device_errors() == (0, 0)


@pytest.mark.parametrize("T", [1, 8, 9, 40, 200])
@pytest.mark.parametrize("K", [1024, 1040, 8208, 131056])
def test_largest_sums(T, K):
    """Codes of -128 and 127 everywhere, rows that stay at the sums' ends (up to 128^2 K, next to
    2^31) and rows that cross 0 and powers of two by single steps."""
    import invariant_token_logprob_gb300 as rlk
    N = 131
    g = torch.Generator().manual_seed(K)
    qw = torch.randint(0, 2, (N, K), generator=g, dtype=torch.int8) * 127 - 128 * torch.randint(0, 2, (N, K), generator=g, dtype=torch.int8)
    qw[0], qw[1] = -128, 127
    qw[2, ::2], qw[2, 1::2] = -128, 127
    qw[3] = 127
    qw[3, K // 2:] = -127
    qx = torch.full((T, K), -128, dtype=torch.int8)
    if T > 2:
        qx[1] = 127
        qx[2, K - 16:] = 1
        qx[T - 1] = torch.randint(-128, 128, (K,), generator=g, dtype=torch.int8)
    one = torch.ones(max(T, N))
    y = rlk.linear_int8(qx.cuda(), qw.cuda(), one[:N].cuda(), x_scales=one[:T].cuda())
    sums = (qx.double().cuda() @ qw.double().cuda().T)
    assert torch.equal(y, sums.float())  # one rounding
    assert rlk.take_device_errors() == (0, 0)


def test_row_bits_do_not_depend_on_the_batch():
    import invariant_token_logprob_gb300 as rlk
    N, K = 1000, 2080
    qw, sw = (a.cuda() for a in ref_quantize(normal(N, K, "bf16", 1, 0.02)))
    x = normal(260, K, "bf16", 2).cuda()
    y = rlk.linear_int8(x, qw, sw)
    for n in (1, 2, 8, 9, 16, 31, 64, 65, 128, 200):
        assert torch.equal(rlk.linear_int8(x[:n], qw, sw), y[:n]), n
    assert torch.equal(rlk.linear_int8(x, qw[100:300].contiguous(), sw[100:300].contiguous()), y[:, 100:300])


@pytest.mark.parametrize("T,N,K", [(1, 512, 4096), (3, 20000, 1040), (150, 1000, 2064)])
def test_codes_written_by_the_call_before(T, N, K):
    """Two weights in turn, quantised into the same codes and multiplied at once, without a wait and
    from a graph: every product is of the codes that were written last."""
    import invariant_token_logprob_gb300 as rlk
    g = torch.Generator().manual_seed(T)
    W = [torch.randn(N, K, generator=g).bfloat16().cuda() for _ in range(2)]
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    want = [rlk.linear_int8(x, *rlk.quantize_int8(w)) for w in W]
    assert not torch.equal(*want)
    buffers = rlk.quantize_int8(W[0])
    out = [torch.empty_like(want[0]) for _ in range(20)]
    workspace = torch.empty(rlk.lib().rlk_linear_int8_workspace_size(T, K), dtype=torch.uint8, device="cuda")

    def run():
        for i, o in enumerate(out):
            rlk.quantize_int8(W[i % 2], out=buffers)
            rlk.linear_int8(x, *buffers, out=o, workspace=workspace)
    run()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(out))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    for o in out:
        o.zero_()
    graph.replay()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(out))


def test_reads_and_writes_stay_inside():
    """Operands in the middle of poisoned memory, an output and a workspace with guards behind."""
    import invariant_token_logprob_gb300 as rlk
    for T, N, K in [(1, 130, 160), (9, 257, 1040), (70, 131, 528), (300, 129, 272)]:
        qw, sw = ref_quantize(normal(N, K, "bf16", 1, 0.02))
        x = normal(T, K, "bf16", 3)
        want = ref_linear(*ref_quantize(x), qw, sw, "fp32")

        def between(t):
            buf = torch.full((t.numel() + 256,), float("nan") if t.is_floating_point() else 77, dtype=t.dtype, device="cuda")
            v = buf[128:128 + t.numel()].view(t.shape)
            v.copy_(t)
            return v
        buf = torch.full((T * N + 512,), -5.0, device="cuda")
        n = rlk.lib().rlk_linear_int8_workspace_size(T, K)
        ws = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
        rlk.linear_int8(between(x), between(qw), between(sw), out=buf[:T * N].view(T, N), workspace=ws[:n])
        assert torch.equal(buf[:T * N].view(T, N).cpu(), want)
        assert (buf[T * N:] == -5).all() and (ws[n:] == 0xAB).all()


def test_decode_step_in_a_graph_and_on_a_stream():
    import invariant_token_logprob_gb300 as rlk
    V, H = 3001, 528
    qw, sw = (a.cuda() for a in ref_quantize(normal(V, H, "bf16", 1, 0.05)))
    tg = torch.randint(0, V, (20,), dtype=torch.int32).cuda()
    for T in (1, 20):
        h = normal(T, H, "bf16", T).cuda()
        t = tg[:T].contiguous()
        want = rlk.logprob_int8(h, qw, sw, t, top_k=5)
        ref = rlk.token_logprobs(rlk.linear_int8(h, qw, sw), t, top_k=5)
        assert all(torch.equal(a, b) for a, b in zip(want, ref))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = rlk.logprob_int8(h, qw, sw, t, top_k=5, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        hs = h.clone()
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                out = rlk.logprob_int8(hs, qw, sw, t, top_k=5)
            hs.copy_(h * 2)
            graph.replay()
        s.synchronize()
        want = rlk.logprob_int8(h * 2, qw, sw, t, top_k=5)
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_train_then_roll_out():
    """The operators together: a step on the cross entropy, the new head quantised, and the log
    probabilities that it answers with against the loss of the values it stands for."""
    import invariant_token_logprob_gb300 as rlk
    g = torch.Generator().manual_seed(0)
    T, H, V = 48, 256, 1500
    W = (torch.randn(V, H, generator=g) / 16).bfloat16().cuda().requires_grad_()
    h = torch.randn(T, H, generator=g).bfloat16().cuda()
    t = torch.randint(0, V, (T,), generator=g).to(torch.int32).cuda()
    rlk.differentiable_cross_entropy(h, W, t).loss.backward()
    new = (W.detach().float() - 0.5 * W.grad.float()).bfloat16()
    codes, scales = rlk.quantize_int8(new)
    r = rlk.logprob_int8(h, codes, scales, t)
    qx, sx = ref_quantize(h.cpu())
    z = ref_linear(qx, sx, codes.cpu(), scales.cpu(), "fp32").double()
    want = z.gather(1, t.cpu().long()[:, None])[:, 0] - torch.logsumexp(z, 1)
    # (fp32 exponentials, sums and one logarithm behind exact logits)
    assert (r.logp.cpu().double() - want).abs().max() <= 2.0 ** -18 * (1 + want.abs().max())


def test_empty_and_refusals():
    import invariant_token_logprob_gb300 as rlk
    qw, sw = (a.cuda() for a in ref_quantize(normal(10, 32, "bf16", 1)))
    x = normal(2, 32, "bf16", 3).cuda()
    assert rlk.linear_int8(x[:0], qw, sw).shape == (0, 10)
    assert rlk.linear_int8(x, qw[:0], sw[:0]).shape == (2, 0)
    assert rlk.quantize_int8(x[:0])[0].shape == (0, 32)
    with pytest.raises(rlk.RlkError, match="align"):
        rlk.quantize_int8(torch.zeros(2, 24, device="cuda"))
    with pytest.raises(TypeError):
        rlk.quantize_int8(torch.zeros(2, 32, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        rlk.linear_int8(x[:, :16].contiguous(), qw, sw)
    with pytest.raises(ValueError, match="contiguous"):
        rlk.linear_int8(normal(2, 64, "bf16", 3).cuda()[:, ::2], qw, sw)
    with pytest.raises(ValueError, match="x_scales"):
        rlk.linear_int8(qw[:2], qw, sw)
    with pytest.raises(ValueError, match="x_scales"):
        rlk.linear_int8(x, qw, sw, x_scales=sw[:2])
    with pytest.raises(TypeError):
        rlk.linear_int8(x, qw.to(torch.uint8), sw)
    with pytest.raises(ValueError, match="scales"):
        rlk.linear_int8(x, qw, sw[:5])
    with pytest.raises(rlk.RlkError, match="workspace"):
        rlk.linear_int8(x, qw, sw, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        rlk.dequantize_int8(qw, sw, out_dtype=torch.int32)


@pytest.mark.parametrize("mode", [1, 2])
def test_bounded_wait_runs_out_and_context_survives(mode):
    """No copy is issued, or no stage is consumed after every copy was issued: the wait that runs
    out is reported, every teardown wait ends in time, and the next call is right."""
    import ctypes
    import time

    import invariant_token_logprob_gb300 as rlk
    qx, sx = ref_quantize(normal(1, 512, "bf16", 1))
    qw, sw = ref_quantize(normal(128, 512, "bf16", 2))
    x, xs, w, s = qx.half().cuda(), sx.cuda(), qw.cuda(), sw.cuda()
    y = torch.full((1, 128), 7.0, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rlk.check_device_error()

    def selftest(m):
        return rlk.lib().rlk_selftest_wait_timeout_int8(*(ctypes.c_void_p(t.data_ptr()) for t in (x, xs, w, s, y)), m,
                                                        stream)

    assert selftest(0) == 1 and selftest(3) == 1
    t0 = time.time()
    assert selftest(mode) == 0
    assert rlk.take_device_errors() == (1, 0)  # a wait ran out, and no teardown wait did
    assert 1.0 < time.time() - t0 < 30.0
    assert bool((y == 7).all())
    rlk.check_device_error()
    assert torch.equal(rlk.linear_int8(qx.cuda(), w, s, x_scales=xs).cpu(), ref_linear(qx, sx, qw, sw, "fp32"))


CAPTURE = """
import torch
import invariant_token_logprob_gb300 as rlk
g = torch.Generator().manual_seed(0)
N, K = 300, 528
codes, scales = rlk.quantize_int8(torch.randn(N, K, generator=g).cuda())
rows = [1, 17, 40, 100, 192, 193, 200, 256, 257, 300, 400]
xs = [torch.randint(-127, 128, (T, K), generator=g, dtype=torch.int8).cuda() for T in rows]
ss = [torch.rand(T, generator=g).cuda() for T in rows]
for dtype in (torch.float32, torch.bfloat16, torch.float16):
    call = lambda i: rlk.linear_int8(xs[i], codes, scales, ss[i], out_dtype=dtype)
    call(%d)  # the only call of this type before
    graphs = []
    for i in range(len(rows)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(i)
        graphs.append((graph, out))
    for graph, _ in graphs:
        graph.replay()
    for i, (_, out) in enumerate(graphs):
        assert torch.equal(out, call(i)), rows[i]
assert rlk.take_device_errors() == (0, 0)
print("captured")
"""


@pytest.mark.parametrize("first", [0, 9])
def test_one_call_of_a_type_before_a_capture(first):
    """In a process of its own: one eager call per output type, of 1 or 300 rows, then captures with other
    numbers of rows, the first calls with those."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE % first], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
