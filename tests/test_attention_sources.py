"""Rules of the attention operators' kernel sources that no output shows (CPU)."""
import os
import re

import pytest

import fake_quant_numerics_gb300 as fq

CSRC = os.path.join(os.path.dirname(fq.__file__), "csrc")


@pytest.mark.parametrize("name", ["kernels_kvsplit.cu", "kernels_kvattn.cu", "kernels_rope.cu", "kernels_kvcache.cu"])
def test_warp_exchanges_do_not_hang_on_conditions(name):
    """An exchange over a full warp behind && or || or ?: is left out by the lanes whose
    condition fails, and the others wait for them without end."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for statement in re.split(r"[;{}]", text):
        first = re.search(r"&&|\|\||\?", statement)
        for m in re.finditer(r"__(shfl\w*|ballot|any|all)_sync", statement):
            assert not first or m.start() < first.start(), " ".join(statement.split())


@pytest.mark.parametrize("name,kernels", [("kernels_kvattn.cu", ["k_kv_join"]), ("kernels_rope.cu", ["k_rope_join"])])
def test_chained_kernels_read_what_others_write_coherently(name, kernels):
    """The kernels that are launched while the call's first one runs read its results
    behind the wait, and not through the read-only path."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for k in kernels:
        body = text[text.index(k + "("):]
        body = body[:body.index("\n}\n")]
        assert "pdl_wait" in body and "__ldg" not in body and "__restrict__" not in body
        assert body.index("pdl_wait") < body.index("ws." if "ws." in body else "parts[")
