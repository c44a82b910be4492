"""GPU tests of the workspaces that the binding keeps for small calls: calls of two threads on one
stream, of one thread on two streams, and calls next to captured graphs do not share one."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def made():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import invariant_token_logprob_gb300 as rlk
    g = torch.Generator().manual_seed(0)
    codes, scales = rlk.quantize_int8(torch.randn(700, 512, generator=g).cuda())
    xs = [torch.randn(T, 512, generator=g).bfloat16().cuda() for T in (1, 3, 20, 40)]
    want = [rlk.linear_int8(x, codes, scales, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
            for x in xs]
    torch.cuda.synchronize()
    return codes, scales, xs, want


def test_threads_on_one_stream(made):
    import invariant_token_logprob_gb300 as rlk
    codes, scales, xs, want = made
    stream = torch.cuda.Stream()
    bad = []

    def work(k):
        with torch.cuda.stream(stream):
            for i in range(200):
                j = (i + k) % len(xs)
                got = rlk.linear_int8(xs[j], codes, scales)
                stream.synchronize()
                if not torch.equal(got, want[j]):
                    bad.append((k, i))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:5]


def test_streams_of_one_thread(made):
    import invariant_token_logprob_gb300 as rlk
    codes, scales, xs, want = made
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for i in range(40):
        with torch.cuda.stream(streams[i % 4]):
            got.append(rlk.linear_int8(xs[(i // 4) % 4], codes, scales))
        if i % 3 == 0:
            got.append(rlk.linear_int8(xs[(i // 4) % 4], codes, scales, stream=streams[(i + 1) % 4]))
    torch.cuda.synchronize()
    k = 0
    for i in range(40):
        for _ in range(2 if i % 3 == 0 else 1):
            assert torch.equal(got[k], want[(i // 4) % 4]), (i, k)
            k += 1


def test_graphs_and_eager_calls(made):
    """Two graphs captured on one stream and replayed on two at once, next to eager calls there."""
    import invariant_token_logprob_gb300 as rlk
    codes, scales, xs, want = made
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for x in xs:
            rlk.linear_int8(x, codes, scales)
        for x in xs[2:]:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs = [rlk.linear_int8(x, codes, scales) for _ in range(10)]
            graphs.append((g, outs))
    s.synchronize()
    other = torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(s):
            graphs[0][0].replay()
            eager = rlk.linear_int8(xs[1], codes, scales)
        with torch.cuda.stream(other):
            graphs[1][0].replay()
            eager2 = rlk.linear_int8(xs[0], codes, scales)
        torch.cuda.synchronize()
        assert torch.equal(eager, want[1]) and torch.equal(eager2, want[0])
        for (g, outs), w in zip(graphs, want[2:]):
            assert all(torch.equal(o, w) for o in outs)


def test_streams_that_torch_has_not_made(made):
    """A stream given by its address alone may be gone, and its address another stream's, by the next call:
    no workspace is kept for it; torch's own streams have one each."""
    import invariant_token_logprob_gb300 as rlk
    codes, scales, xs, want = made
    rlk._scratch.__dict__.clear()
    own = torch.cuda.Stream()
    other = torch.cuda.ExternalStream(torch.cuda.Stream().cuda_stream)
    for stream in (other, own, torch.cuda.default_stream()):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            got = [rlk.linear_int8(x, codes, scales) for x in xs]
            got += [rlk.linear_int8(x, codes, scales, stream=stream) for x in xs]
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, 2 * want))
    got = [rlk.linear_int8(x, codes, scales, stream=other) for x in xs]
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert {raw for _, raw in rlk._scratch.__dict__} == {own.cuda_stream, 0}
