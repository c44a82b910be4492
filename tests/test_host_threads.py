"""Host check: what the launchers of the kernels on logits and 4-bit weights remember between
calls (which kernel may have how much shared memory) is safe to touch from several threads;
the binding's calls run without Python's lock."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "invariant_token_logprob_gb300", "csrc")


@pytest.mark.parametrize("name", ["rlk_token_logprobs.cu", "rlk_w4_linear.cu", "rlk_w4.cu"])
def test_host_side_records_are_atomic(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for line in re.findall(r"\n\s+static (?!_|constexpr|const |__device__)[^\n(]*;", text):
        assert "std::atomic" in line, line
