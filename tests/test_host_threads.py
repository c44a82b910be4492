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


@pytest.mark.parametrize("name", ["rlk_lmhead.cu", "rlk_lmhead_fp8b.cu", "rlk_bwd_gemm.cu", "rlk_cross_entropy.cu",
                                  "rlk_int8.cu", "rlk_int8_linear.cu"])
def test_records_outside_functions_are_atomic(name):
    """The same for what stands outside of functions, and for the members of structs that do."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    records = re.findall(r"\n(?:static )?([A-Za-z_][\w:<>]*) (g_\w+)\[[^;\n]*;", text)
    for kind, variable in records:
        struct = re.search(r"struct %s \{(.*?)\n\};" % re.escape(kind), text, re.S)
        members = re.findall(r"\n\s+([^\n;]+);", struct.group(1)) if struct else [kind]
        for member in members:
            assert "std::atomic" in member, (variable, member)
    for line in re.findall(r"\n\s+static (?!_|constexpr|const |__device__)[^\n(]*;", text):
        assert "std::atomic" in line, line
