"""The rules of test_kernel_sources.py about TMEM bases and single issuing lanes, for the kernels whose blocks come in pairs and
for the headers; and that a source which breaks them is found."""
import os
import re

import pytest

from attention_kl_divergence_streamkl_gb300 import build as B

FILES = sorted(f for f in os.listdir(B.CSRC) if f.endswith((".cu", ".cuh")))
ALLOC = re.compile(r"\btmem_alloc(?:_pair)?\(")


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(B.CSRC, name)).read())


PAIRS = [f for f in FILES if f.endswith(".cu") and "tmem_alloc_pair(" in code(f)]


def base_is_checked_and_constant(text):
    """Every allocation is followed, before another and before setmaxnreg, by whole_tmem and the constant base."""
    assert not re.search(r"tmem = \*", text)
    at = [m.start() for m in ALLOC.finditer(text)]
    assert at
    for a, b in zip(at, at[1:] + [len(text)]):
        block = text[a:b]
        assert "whole_tmem(" in block and "constexpr uint32_t tmem = 0;" in block
        check = block.index("whole_tmem(")
        barrier = block.index("__syncthreads();")
        deal = re.search(r"setmaxnreg_\w+(<\w+>)?\(", block)
        assert barrier < check and (deal is None or check < deal.start())


def one_lane_issues(text):
    for m in re.finditer(r"if \((?:lane|threadIdx\.x)(?: == 0|\))\s*(\{(?:[^{}]|\{[^{}]*\})*\}|[^;{]*;)", text):
        assert not re.search(r"mbar_|tma_|mma_|bulk_|tcgen05", m.group(1)), m.group(0)[:80]


def test_the_pairs_kernels_are_found():
    assert "vocab_xent.cu" in PAIRS


@pytest.mark.parametrize("name", PAIRS)
def test_a_pairs_tmem_base_is_checked_and_not_kept(name):
    base_is_checked_and_constant(code(name))


@pytest.mark.parametrize("name", PAIRS + [f for f in FILES if f.endswith(".cuh")])
def test_one_elected_lane_issues(name):
    one_lane_issues(code(name))


@pytest.mark.parametrize("name", PAIRS)
def test_both_blocks_are_set_up_before_and_done_after(name):
    """The cluster's barrier stands between the set-up and the first use of the other block's memory, and before the end."""
    text = code(name)
    for m in re.finditer(r"\btmem_alloc_pair\(", text):
        block = text[m.start():]
        block = block[:block.index("tmem_dealloc_pair(")]
        assert block.count("cluster_sync();") == 2
        assert block.index("cluster_sync();") < block.index("whole_tmem(") and block.rindex("cluster_sync();") > block.rindex("__syncthreads();")


def test_sources_that_break_a_rule_are_found():
    text = code("vocab_xent.cu")
    for wrong in (text.replace("whole_tmem(", "look("), text.replace("constexpr uint32_t tmem = 0;", "const uint32_t tmem = *slot;"),
                  text.replace("tmem_alloc_pair(", "setmaxnreg_dec<40>(); tmem_alloc_pair(", 1).replace("whole_tmem(", "setmaxnreg_inc<96>(); whole_tmem(", 1)):
        assert wrong != text
        with pytest.raises((AssertionError, ValueError)):
            base_is_checked_and_constant(wrong)
    with pytest.raises(AssertionError):
        one_lane_issues("if (lane == 0) mbar_arrive(full);")
