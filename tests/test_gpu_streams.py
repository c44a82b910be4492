"""GPU tests of calls on a stream that is not the current one: what a call allocates itself,
temporaries and outputs, is memory of the stream that it runs on, so no other stream's work
is given a block that the call still writes to or reads."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import invariant_token_logprob_gb300 as rlk
    rlk.lib()


def owner(t):
    """The stream (its address) whose memory a tensor lies in, by the allocator's own account."""
    p = t.data_ptr()
    for seg in torch.cuda.memory._snapshot()["segments"]:
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def held(stream):
    """Bytes of the stream's memory, free blocks included."""
    return sum(seg["total_size"] for seg in torch.cuda.memory._snapshot()["segments"]
               if seg["stream"] == stream.cuda_stream)


def problem(V=40000, K=512, T=64):
    import invariant_token_logprob_gb300 as rlk
    g = torch.Generator(device="cuda").manual_seed(3)
    W = (torch.randn(V, K, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    h = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    tg = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    return W, h, tg, rlk.quantize_w4(W)


def test_decode_step_allocates_its_logits_on_its_stream():
    import invariant_token_logprob_gb300 as rlk
    W, h, tg, (codes, scales, _) = problem()
    T, V = h.shape[0], W.shape[0]
    want = rlk.logprob_w4(h, codes, scales, tg, top_k=4)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got, rest = [], []
    for _ in range(8):
        s.wait_stream(torch.cuda.current_stream())
        got.append(rlk.logprob_w4(h, codes, scales, tg, top_k=4, stream=s))
        # whatever the allocator gives to the current stream now is not the step's logits
        rest.append(torch.full((T, V), float("nan"), device="cuda"))
    s.synchronize()
    assert held(s) >= 4 * T * V
    rlk.check_device_error()
    for r in got:
        assert all(owner(a) == s.cuda_stream for a in r)
        for a, b in zip(r, want):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_outputs_and_workspaces_belong_to_their_stream():
    import invariant_token_logprob_gb300 as rlk
    W, h, tg, (codes, scales, _) = problem(V=2048, K=256, T=8)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    logits = rlk.linear_w4(h, codes, scales)
    lse, ones = torch.logsumexp(logits, 1), torch.ones(8, device="cuda")
    packed, ps = rlk.quantize_fp8_weight(W)
    torch.cuda.synchronize()
    calls = {
        "linear_w4": lambda **k: rlk.linear_w4(h, codes, scales, **k),
        "dequantize_w4": lambda **k: rlk.dequantize_w4(codes, scales, **k),
        "quantize_w4": lambda **k: rlk.quantize_w4(W, asymmetric=True, **k),
        "token_logprobs": lambda **k: rlk.token_logprobs(logits, tg, 3, **k),
        "token_logprobs_backward": lambda **k: rlk.token_logprobs_backward(
            logits, tg, lse, grad_logp=ones, **k),
        "logprob": lambda **k: rlk.logprob(h, W, tg, **k),
        "logprob_entropy": lambda **k: rlk.logprob_entropy(h, W, tg, **k),
        "logprob_fp8": lambda **k: rlk.logprob_fp8(h, packed, ps, tg, **k),
        "consistency_stats_async": lambda **k: rlk.consistency_stats_async(ones, ones, **k),
    }
    for name, call in calls.items():
        want = call()
        s.wait_stream(torch.cuda.current_stream())
        got = call(stream=s)
        s.synchronize()
        for a, b in zip(*((r if isinstance(r, tuple) else (r,)) for r in (got, want))):
            assert owner(a) == s.cuda_stream, name
            assert owner(b) == torch.cuda.current_stream().cuda_stream, name
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    assert rlk.linear_w4(h[:0], codes, scales, stream=s).shape == (0, 2048)
    rlk.check_device_error()
