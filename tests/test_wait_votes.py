"""Bounded waits that a whole warp makes are decided by a vote.

mbar_wait returns false when it runs out or another warp gave up. Lanes of one warp poll at their own times, so at that moment
some may have seen the barrier's phase and others not. What follows such a wait in these kernels (tensor-memory loads, full-mask
shuffles, __syncwarp) needs the whole warp, so a lane that leaves by itself would make the others wait without a limit. It cannot be
provoked without holding up a GPU; the sources are read instead: a wait is made by lane 0 alone, or its result is voted on."""

import os
import re

import pytest

import rmsnorm_linear_projection_fold_b200 as fn

CSRC = os.path.join(os.path.dirname(fn.__file__), "csrc")
VOTE = "__all_sync(0xffffffffu, "


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _unvoted(code):
    """Calls of mbar_wait or mbar_wait_cluster that neither stand in a block of lane 0 (or thread 0) nor are voted on."""
    found, blocks, last = [], [], 0
    for m in re.finditer(r"[{};]|\bmbar_wait(_cluster)?\(", code):
        if m.group() == "{":
            blocks.append(code[last:m.start()])
        elif m.group() == "}":
            blocks.pop()
        elif m.group() != ";":
            head = " ".join(blocks) + code[last:m.start()]
            if not re.search(r"(lane|threadIdx\.x) == 0\b", head) and not re.search(re.escape(VOTE) + r"([^;{}]*&& )?$", code[last:m.start()]):
                found.append(code[:m.start()].count("\n") + 1)
            continue
        last = m.end()
    return found


def test_the_reader_sees_an_unvoted_wait():
    assert _unvoted("void f() { if (lane == 0) { mbar_wait(a, 0, f); } }") == []
    assert _unvoted("void f() { bool ok = " + VOTE + "mbar_wait(a, 0, f)); }") == []
    assert _unvoted("void f() { bool ok = " + VOTE + "mbar_wait(a, 0, f) && mbar_wait(b, 0, f)); }") == []
    assert _unvoted("void f() { bool ok = " + VOTE + "mbar_wait(a, 0, f)) || mbar_wait(b, 0, f); }") == [1]
    assert _unvoted("void f() {\n if (!mbar_wait_cluster(a, 0, f)) return; }") == [2]


@pytest.mark.parametrize("name", ["pair_gemm.cuh", "decode_int8.cuh", "decode_int8_cluster.cuh", "cross_entropy_small.cuh"])
def test_waits_of_whole_warps_are_voted_on(name):
    code = _code(name)
    assert "mbar_wait" in code and _unvoted(code) == []


def test_every_epilogue_warp_of_the_cluster_decode_reports_its_own_wait():
    """A rank's partial sums come from eight warps, whose waits may end differently: each has a word of its own, and a sum counts
    as incomplete if any of them is set."""
    code = _code("decode_int8_cluster.cuh")
    assert re.search(r"dsmem_addr\(failed \+ rank \* 8 \+ w,", code)
    assert re.search(r"failed \+ kI8cMaxRanks \* 8\b", code) and "lane + 32 < 8 * ranks" in code


def test_a_loss_whose_product_gave_up_is_not_joined_from_what_lies_in_the_workspace():
    """The CTA-pair product sets a word of the workspace when it leaves tiles unfinished; the row pass before it clears that word and
    the join after it writes NaN where it is set."""
    product, head, host = (_code(n) for n in ("pair_gemm.cuh", "cross_entropy.cuh", "api_cross_entropy.cuh"))
    assert re.search(r"if \(!ok && lane == 0 && p0\.failed != nullptr\) atomicExch\(p0\.failed, 1u\)", product)
    join = head[head.index(" k_ce_join("):head.index("struct __align__(16) CeRow")]
    assert re.search(r"grid_dep_wait\(\);.* gave_up = __ldcg\(failed\);.*ce_join_row<.*if \(gave_up != 0u[^;]*\) loss\[row\] = lse\[row\] = "
                     r"__int_as_float\(0x7fc00000\)", join, re.S)
    assert "launch_rstd(x, rstd, p.failed," in host


@pytest.mark.parametrize("name", ["decode_tc.cuh", "decode_fp8.cuh", "fused_gemm.cuh", "fused_gemm_pair.cuh", "postnorm_pair.cuh",
                                  "postnorm_split.cuh"])
def test_waits_of_whole_warps_are_voted_on_in_the_projections(name):
    code = _code(name)
    assert "mbar_wait" in code and _unvoted(code) == []
