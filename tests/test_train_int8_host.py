"""Host-only checks of the cross entropy and the 8-bit integer entry points: bad arguments are
refused before a device is touched, empty problems are answered, a machine without a supported
GPU reports a status, and the backward's cut of the vocabulary holds for every shape."""
import ctypes
import os
import subprocess

import pytest
import torch

import invariant_token_logprob_gb300 as rlk

A16 = ctypes.c_void_p(1 << 20)
A4 = ctypes.c_void_p((1 << 20) + 4)
A2 = ctypes.c_void_p((1 << 20) + 2)
BIG = 1 << 60


@pytest.fixture(scope="module")
def L():
    from invariant_token_logprob_gb300 import _build
    _build.build()
    return rlk.lib()


def loss(L, h=A16, W=A16, t=A16, w=None, T=4, H=64, V=100, it=1.0, e=0.0, z=0.0, red=0, out=A16, lse=A16, total=A16,
         ws=A16, size=BIG):
    return L.rlk_cross_entropy(h, W, t, w, T, H, V, it, e, z, red, out, lse, total, ws, size, None)


def grad(L, h=A16, W=A16, t=A16, w=None, lse=A16, g=A16, total=A16, T=4, H=64, V=100, it=1.0, e=0.0, z=0.0, red=0,
         gh=A16, hd=0, gW=A16, wd=0, acc=0, ws=A16, size=BIG):
    return L.rlk_cross_entropy_backward(h, W, t, w, lse, g, total, T, H, V, it, e, z, red, gh, hd, gW, wd, acc, ws,
                                        size, None)


SHARED = [(dict(T=-1), 1), (dict(H=0), 1), (dict(V=0), 1), (dict(V=1 << 31), 1), (dict(T=1 << 31), 1), (dict(it=0.0), 1),
          (dict(it=float("nan")), 1), (dict(e=1.0), 1), (dict(e=-0.5), 1), (dict(e=float("nan")), 1), (dict(z=-1.0), 1),
          (dict(z=float("inf")), 1), (dict(red=3), 1), (dict(red=-1), 1), (dict(h=None), 1), (dict(W=None), 1),
          (dict(t=None), 1), (dict(lse=None), 1), (dict(H=60), 2), (dict(h=A4), 2), (dict(W=A4), 2), (dict(t=A2), 2),
          (dict(w=A2), 2), (dict(lse=A2), 2), (dict(total=A2), 2), (dict(ws=None), 5), (dict(ws=A4), 2), (dict(size=16), 5)]


@pytest.mark.parametrize("kw,expect", SHARED + [(dict(out=None), 1), (dict(total=None), 1), (dict(out=A2), 2)])
def test_loss_refusals(L, kw, expect):
    assert loss(L, **kw) == expect


@pytest.mark.parametrize("kw,expect", SHARED + [(dict(g=None), 1), (dict(total=None), 1), (dict(hd=1), 1), (dict(wd=3), 1),
                                                (dict(acc=1), 1), (dict(gh=A4), 2), (dict(gW=A4), 2), (dict(g=A2), 2)])
def test_gradient_refusals(L, kw, expect):
    assert grad(L, **kw) == expect


def linear(L, x=A16, xd=0, xs=None, c=A16, s=A16, T=2, N=10, K=64, y=A16, yd=2, ws=A16, size=BIG):
    return L.rlk_linear_int8(x, xd, xs, c, s, T, N, K, y, yd, ws, size, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(xd=4), 1), (dict(xd=-1), 1), (dict(yd=3), 1), (dict(T=-1), 1), (dict(N=-1), 1), (dict(K=0), 1), (dict(K=56), 2),
    (dict(K=131072), 1), (dict(N=1 << 31), 1), (dict(T=1 << 30, N=1 << 20), 1), (dict(x=None), 1), (dict(c=None), 1),
    (dict(s=None), 1), (dict(y=None), 1), (dict(xd=3), 1), (dict(xs=A16), 1), (dict(x=A4), 2), (dict(c=A4), 2),
    (dict(s=A2), 2), (dict(y=A2), 2), (dict(xd=3, xs=A2), 2), (dict(ws=None), 5), (dict(ws=A4), 2), (dict(size=100), 5),
])
def test_linear_refusals(L, kw, expect):
    assert linear(L, **kw) == expect


def test_quantize_refusals(L):
    q, d = L.rlk_quantize_int8, L.rlk_dequantize_int8
    assert q(A16, 3, 4, 64, A16, A16, None) == 1 and q(A16, 0, 4, 72, A16, A16, None) == 2
    assert q(None, 0, 4, 64, A16, A16, None) == 1 and q(A4, 0, 4, 64, A16, A16, None) == 2
    assert q(A16, 0, 1 << 30, 1 << 20, A16, A16, None) == 1 and q(None, 0, 0, 64, None, None, None) == 0
    assert d(A16, A16, 4, 64, A16, 3, None) == 1 and d(A16, A16, 4, 64, None, 0, None) == 1
    assert d(A16, A16, 4, 64, A4, 0, None) == 2 and d(None, None, 0, 64, None, 0, None) == 0


def test_empty_problems_and_no_gpu(L):
    assert grad(L, T=0, h=None, W=None, t=None, gW=None, ws=None) == 0
    assert linear(L, T=0, x=None, y=None) == 0 and linear(L, N=0, c=None, s=None, x=None, y=None) == 0
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the gpu tests")
    assert loss(L) == grad(L) == linear(L) == 3 and loss(L, T=0, h=None, W=None, t=None, ws=None) == 3
    assert L.rlk_quantize_int8(A16, 0, 4, 64, A16, A16, None) == 3
    assert L.rlk_dequantize_int8(A16, A16, 4, 64, A16, 0, None) == 3


def test_wait_selftest_refusals(L):
    f = L.rlk_selftest_wait_timeout_int8
    assert f(A16, A16, A16, A16, A16, 0, None) == 1 and f(A16, A16, A16, A16, A16, 3, None) == 1
    assert f(None, A16, A16, A16, A16, 1, None) == 1 and f(A16, A16, A16, A16, None, 2, None) == 1
    assert f(A4, A16, A16, A16, A16, 1, None) == 2 and f(A16, A16, A16, A16, A2, 1, None) == 2
    if not torch.cuda.is_available():
        assert f(A16, A16, A16, A16, A16, 1, None) == 3


def test_binding_refuses_cpu_tensors():
    b = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rlk.cross_entropy(b, b, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        rlk.quantize_int8(b)
    with pytest.raises(ValueError, match="CUDA"):
        rlk.linear_int8(b, torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2))


PLAN = r"""
#include <cstdio>
#include <cstdlib>
#include "rlk_ce_plan.h"
using namespace rlk;
static int fail(const char* what, long T, long H, long V) { std::printf("%s T=%ld H=%ld V=%ld\n", what, T, H, V); return 1; }
int main() {
    const long Ts[] = {1, 2, 7, 64, 128, 129, 300, 441, 442, 1000, 4096, 4097, 16384, 32768, 100003, 1 << 20};
    const long Vs[] = {1, 63, 64, 255, 256, 257, 500, 32761, 50001, 151936, 250000, 1000003, 20000000};
    const long Hs[] = {8, 64, 1032, 4096, 5120, 16384};
    for (long T : Ts) for (long V : Vs) for (long H : Hs) {
        const CePlan p = ce_plan(T, H, V);
        if (p.rows <= 0 || p.rows % 256 || p.pieces != ce_cdiv(V, p.rows)) return fail("pieces", T, H, V);
        if (p.rows > 256 && 4 * p.rows * T > kCeBytes) return fail("bytes", T, H, V);
        if (p.parts < 1 || p.parts > kCeMaxParts) return fail("parts", T, H, V);
        const long part = ce_part_rows(p);
        if (part % 64 || part * p.parts < p.rows) return fail("part rows", T, H, V);
        // every piece's ranges are the first piece's first ones, and fit the sums' space
        const long first = V < p.rows ? V : p.rows, written = ce_cdiv(first, part);
        if (written > p.parts) return fail("written", T, H, V);
        long covered = 0;
        for (long v0 = 0; v0 < V && v0 < 100 * p.rows; v0 += p.rows) {
            const long rows = V - v0 < p.rows ? V - v0 : p.rows;
            if (ce_cdiv(ce_cdiv(rows, 64), part / 64) > written) return fail("ranges", T, H, V);
            covered += rows;
        }
        if (V <= 100 * p.rows && covered != V) return fail("covered", T, H, V);
        const CeLayout l = ce_layout(T, H, p);
        if (l.dzt % 256 || l.sums % 256 || l.h % 256 || l.rows % 256 || l.tops % 256 || l.top % 256 ||
            l.h - l.sums < size_t(p.parts) * T * H * 4 || l.rows - l.h < size_t(T) * H * 2 ||
            l.tops - l.rows < size_t(T) * 32 || l.top - l.tops < size_t(T) * 4 || l.bytes - l.top < 4 || l.dzt < size_t(T) * p.rows * 2 ||
            l.sums - l.dzt < size_t(p.rows) * ce_row_stride(T) * 2)
            return fail("layout", T, H, V);
    }
    return 0;
}
"""


INT8_PLAN = r"""
#include <cstdio>
#include <initializer_list>
#include "rlk_int8_plan.h"
using namespace rlk;
int main() {
    for (int room : {16, 32, 64, 128, 192}) {
        const size_t stages = size_t(int8_stages(room)) * int8_stage_bytes(room);
        if (int8_smem_bytes(room) > 227 * 1024 || int8_tmem_cols(room) > 512 || int8_warps(room) > 32 ||
            int8_stage_bytes(room) % 1024 || size_t(room + kInt8MaxParts) * kInt8TileN * 4 > stages)
            return std::printf("room %d\n", room), 1;
    }
    for (long T : {1, 7, 16, 17, 32, 33, 64, 65, 128, 129, 192, 193, 300, 385, 4096, 100000})
        for (long N : {1, 127, 128, 129, 5119, 151936})
            for (long K : {16, 128, 144, 1024, 4096, 5152, 131056}) {
                const Int8Plan p = int8_plan(T, N, K, 152);
                const bool ok = long(p.chunks) * p.rows >= T && long(p.chunks - 1) * p.rows < T &&
                                p.rows <= p.mma_n && p.mma_n <= p.room && p.mma_n % 16 == 0 && p.room <= 192 &&
                                long(p.tiles) * 128 >= N && long(p.stages) * 128 >= K && p.parts >= 1 &&
                                p.parts <= kInt8MaxParts && p.parts <= p.stages;
                if (!ok) return std::printf("T=%ld N=%ld K=%ld\n", T, N, K), 1;
            }
    return 0;
}
"""


@pytest.mark.parametrize("source", [PLAN, INT8_PLAN], ids=["vocabulary", "int8"])
def test_plans(tmp_path, source):
    src = tmp_path / "plan.cpp"
    src.write_text(source)
    csrc = os.path.join(os.path.dirname(rlk.__file__), "csrc")
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", csrc, str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


REFUSED_SHAPES = [(-1, 64, 100), (0, 64, 100), (4, 64, 0), (4, 0, 100), (1 << 31, 64, 100), (4, 64, 1 << 31), (4, 1 << 31, 100),
                  (4, 64, 1 << 60), (1 << 60, 64, 100), (1 << 62, 1 << 62, 1 << 62), (1 << 30, 64, 1 << 20),
                  ((1 << 31) - 1, (1 << 31) - 8, 1), (1, (1 << 31) - 8, (1 << 31) - 1)]


@pytest.mark.timeout(60)
@pytest.mark.parametrize("T,H,V", REFUSED_SHAPES)
def test_no_workspace_for_refused_shapes(L, T, H, V):
    """Sizes that the calls refuse: the queries answer 0, at once."""
    assert L.rlk_cross_entropy_workspace_size(T, H, V) == 0
    assert L.rlk_cross_entropy_backward_workspace_size(T, H, V) == 0
    if T != 0:
        assert loss(L, T=T, H=H, V=V) == grad(L, T=T, H=H, V=V) == 1


@pytest.mark.parametrize("T,H,V", [(1, 8, (1 << 31) - 1), (1 << 20, 8192, 250000), ((1 << 31) - 1, 8, 1), (32768, 16384, 1 << 20)])
def test_largest_shapes_have_a_workspace(L, T, H, V):
    """What the loss keeps: 12 bytes per row and half tile, 8 per row; the gradient at least its dz and
    its transpose's smallest piece, and h in fp16."""
    halves = 2 * ((V + 255) // 256)
    assert L.rlk_cross_entropy_workspace_size(T, H, V) >= 12 * T * halves + 8 * T
    assert L.rlk_cross_entropy_backward_workspace_size(T, H, V) >= T * 256 * 4 + 6 * T * H


@pytest.mark.parametrize("T,K", [(-1, 64), (0, 64), (4, 0), (1 << 31, 16), (4, 131072), (1 << 62, 1 << 62), (1 << 30, 4096)])
def test_no_workspace_for_refused_products(L, T, K):
    assert L.rlk_linear_int8_workspace_size(T, K) == 0
    if T != 0:
        assert linear(L, T=T, K=K) != 0
    assert L.rlk_linear_int8_workspace_size(13, 131056) >= 13 * 131056 * 2 + 13 * 4


@pytest.mark.parametrize("it,taken", [(2.358e38, True), (2.37e38, False), (3.4e38, False), (1e-45, True)])
def test_largest_inverse_temperature(L, it, taken):
    """The kernels' exponentials take logits times inv_temp log2 e, which has to be finite in fp32: behind
    it every logit would be infinite or NaN, a row of zeros too."""
    assert (grad(L, T=0, it=it, h=None, gW=None) == 0) == taken
    assert loss(L, it=it, h=None) == grad(L, it=it, h=None) == 1
    if not taken:
        assert loss(L, T=0, it=it) == 1
    if not torch.cuda.is_available():
        assert (loss(L, it=it) == 3) == (grad(L, it=it) == 3) == taken
