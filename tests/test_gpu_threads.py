"""GPU test: calls from a host thread that has made no CUDA call before, with every buffer given,
as autograd's worker thread makes them when all its memory comes from a cache."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_first_call_of_a_thread():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import invariant_token_logprob_gb300 as rlk
    g = torch.Generator().manual_seed(0)
    T, H, V = 9, 64, 500
    h = torch.randn(T, H, generator=g).bfloat16().cuda()
    W = torch.randn(V, H, generator=g).bfloat16().cuda()
    t = torch.randint(0, V, (T,), generator=g).to(torch.int32).cuda()
    want = rlk.logprob(h, W, t)
    ws = torch.empty(rlk.workspace_size(T, H, V), dtype=torch.uint8, device="cuda")
    out = tuple(torch.empty_like(x) for x in want)
    torch.cuda.synchronize()
    failed = []

    def call():
        try:
            rlk.logprob_ws(h, W, t, ws, out=out, stream=torch.cuda.default_stream())
        except Exception as e:
            failed.append(e)
    thread = threading.Thread(target=call)
    thread.start()
    thread.join()
    assert not failed, failed
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
