"""Host check of the arithmetic by which the product with a 4-bit weight cuts its work
(csrc/rlk_w4_plan.h), compiled by the host compiler: no word copied without a check of its own
lies outside the scales or the zero points."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "invariant_token_logprob_gb300", "csrc")
SOURCE = r"""
#include "rlk_w4_plan.h"
extern "C" {
// Over all tiles and chunks of an [n][g] array whose chunks start at multiples of `step` groups:
// the most bytes that words of a chunk held to lie inside reach behind the array (<= 0: none).
long long worst_overrun(int n, int g, int size, int step) {
    long long worst = -(1ll << 60);
    for (int n0 = 0; n0 < n; n0 += rlk::kW4TileN)
        for (int first = 0; first < g; first += step) {
            const long long from = (long long)n0 * g + first;
            if (!rlk::w4_chunk_inside(from, g, n, size)) continue;
            for (int r = 0; r < rlk::kW4TileN; ++r)
                for (int w = 0; w < rlk::w4_chunk_words(size); ++w) {
                    const long long end = rlk::w4_chunk_word(from, r, g, size, w) + 4 - (long long)n * g * size;
                    if (end > worst) worst = end;
                }
        }
    return worst;
}
// Chunks held to lie inside, and chunks that do.
int counts(int n, int g, int size, int* held) {
    int inside = 0;
    *held = 0;
    for (int n0 = 0; n0 < n; n0 += rlk::kW4TileN)
        for (int first = 0; first < g; first += rlk::kW4ScaleGroups) {
            const long long from = (long long)n0 * g + first;
            *held += rlk::w4_chunk_inside(from, g, n, size);
            inside += rlk::w4_chunk_word(from, rlk::kW4TileN - 1, g, size, rlk::w4_chunk_words(size) - 1) + 4 <=
                      (long long)n * g * size;
        }
    return inside;
}
int parts_of_k(int n, int k) { return rlk::w4_parts_of_k((n + 127) / 128, (k + 255) / 256); }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "no host compiler"
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"), "-o",
                    str(d / "plan.so")], check=True)
    L = ctypes.CDLL(str(d / "plan.so"))
    L.worst_overrun.restype = ctypes.c_longlong
    return L


@pytest.mark.parametrize("size", [1, 2])
def test_unchecked_words_lie_inside_the_arrays(plan, size):
    for g in (1, 2, 3, 4, 5, 7, 8, 9, 11, 12, 15, 16, 17, 31, 32, 33, 40, 81):
        for n in (1, 127, 128, 129, 130, 131, 133, 140, 157, 162, 163, 165, 255, 258, 260, 291, 300, 385):
            over = plan.worst_overrun(n, g, size, 2)
            assert over <= 0, (n, g, size, over)


@pytest.mark.parametrize("n,k,group", [(32002, 1024, 128), (50178, 768, 128), (130, 256, 128), (130, 1024, 128),
                                       (258, 128, 128), (131, 416, 64)])
def test_few_groups_per_row(plan, n, k, group):
    g = -(-k // group)
    assert plan.worst_overrun(n, g, 2, 1) <= 0 and plan.worst_overrun(n, g, 1, 1) <= 0


def test_every_chunk_that_lies_inside_is_held_to(plan):
    """The unchecked form is the fast one: it is taken wherever it may be."""
    held = ctypes.c_int(0)
    for n, g in ((151936, 32), (151936, 64), (5120, 40), (1000, 9), (4096, 1), (129, 32)):
        for size in (1, 2):
            assert plan.counts(n, g, size, ctypes.byref(held)) == held.value, (n, g, size)


def test_tensor_memory_is_fenced_behind_every_wait():
    """tcgen05 accesses are ordered behind what a barrier's phase reports (other tcgen05 work
    of the issuing warp among it) only by a fence after the wait.  No run can show a missing
    one, so the source is read: between each access and the wait before it there is one."""
    text = open(os.path.join(CSRC, "rlk_w4_linear.cu")).read()
    body = re.sub(r"//[^\n]*", "", text[text.index("linear_w4_kernel("):])
    accesses = [m.start() for m in re.finditer(r"\b(tmem_st16|add_products|umma_f16_tmem_a)\b", body)]
    assert len(accesses) >= 3
    for at in accesses:
        wait = max(body.rfind("warp_wait(", 0, at), body.rfind("wait_bounded(", 0, at))
        assert "tc_fence_after_sync()" in body[wait:at], body[wait:at][:200]


def test_copies_are_waited_for_whoever_gives_up():
    """The producer's drain of its last copies stands under no condition: a consumer's wait may
    run out after the last copy was issued, and the copies must not land in the shared memory
    of the CTA that comes next.  (No run can show it without writing over that memory.)"""
    text = open(os.path.join(CSRC, "rlk_w4_linear.cu")).read()
    body = re.sub(r"//[^\n]*", "", text[text.index("linear_w4_kernel("):])
    producer = body[body.index("if (warp == 0) {"):body.index("} else if (warp == 1) {")]
    tail = producer[producer.rindex("++issued;"):]
    drain = tail.index("wait_drain(")
    assert "issued" in tail[tail.index("for ("):drain]
    assert not re.search(r"if \(!ok\)", tail[:drain])


@pytest.mark.parametrize("n,k,parts", [(151936, 4096, 1), (32768, 4096, 1), (40000, 1024, 1), (19584, 4096, 2),
                                       (5119, 5152, 3), (5000, 4096, 3), (4864, 4096, 4), (4096, 4096, 4),
                                       (1024, 2080, 5), (128, 4096, 8), (128, 256, 1)])
def test_cut_of_k_is_pinned(plan, n, k, parts):
    """The cut decides the order of a row's sums, hence its bits: a function of the weight's
    shape, the same on every device."""
    assert plan.parts_of_k(n, k) == parts


def test_cut_of_k_does_not_ask_the_device():
    text = open(os.path.join(CSRC, "rlk_w4_linear.cu")).read()
    assert re.search(r"w4_parts_of_k\(int\(tiles\), p\.num_stages\);", text)
