"""Rules that every kernel source keeps about single issuing lanes, TMEM bases and setmaxnreg, read from the sources: a
kernel that breaks one may fault, so none is run to show it."""
import os
import re

import pytest

from attention_kl_divergence_streamkl_gb300 import build as B

SOURCES = sorted(f for f in os.listdir(B.CSRC) if f.endswith(".cu"))
TENSOR = [f for f in SOURCES if "tmem_alloc(" in open(os.path.join(B.CSRC, f)).read()]


def code(name):
    text = open(os.path.join(B.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def test_the_tensor_core_kernels_are_found():
    assert {"fwd.cu", "bwd.cu", "bwd_tc.cu", "bwd_mutual.cu", "attn_fwd.cu", "attn_bwd.cu", "attn_bwd_fused.cu"} <= set(TENSOR)


@pytest.mark.parametrize("name", TENSOR)
def test_a_tmem_base_is_checked_and_not_kept(name):
    """Every allocation of all 512 columns is looked at by whole_tmem behind the set-up barrier and before setmaxnreg, and
    addresses follow from the constant."""
    text = code(name)
    allocations = [m.start() for m in re.finditer(r"tmem_alloc\(", text)]
    assert not re.search(r"tmem = \*", text)
    for at, end in zip(allocations, allocations[1:] + [len(text)]):
        block = text[at:end]
        check = block.index("whole_tmem(")
        assert "constexpr uint32_t tmem = 0;" in block
        deal = re.search(r"setmaxnreg_\w+(<\w+>)?\(", block)
        assert deal is None or check < deal.start()


@pytest.mark.parametrize("name", [f for f in SOURCES if "mbar_init(" in code(f) and f != "api.cu"])
def test_one_elected_lane_issues(name):
    """Copies, products and arrivals come from a lane that elect.sync chose, never from a branch on the lane's number whose
    other lanes may run on."""
    text = code(name)
    for m in re.finditer(r"if \((?:lane|threadIdx\.x) == 0\)\s*(\{(?:[^{}]|\{[^{}]*\})*\}|[^;{]*;)", text):
        assert not re.search(r"mbar_|tma_|mma_|bulk|tcgen05", m.group(1)), m.group(0)[:80]
    assert "elect_one()" in text or "arrive_one(" in text


@pytest.mark.parametrize("name", [f for f in TENSOR if "seq_len(" in code(f) and "setmaxnreg" in code(f)])
def test_lengths_have_arrived_before_registers_are_dealt_out(name):
    """A block that reads its sequence's lengths from memory uses them in the set-up barrier: no load is in flight when
    setmaxnreg runs."""
    text = code(name)
    for m in re.finditer(r"tmem_alloc\(", text):
        block = text[m.start():]
        assert "setup_barrier(ql, kl);" in block[:block.index("setmaxnreg")]
    assert name in ("attn_fwd.cu", "attn_bwd.cu", "attn_bwd_fused.cu")
