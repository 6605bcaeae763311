"""How the 4-bit product's kernel waits (of its source; a wait that runs out is not to be provoked on a GPU).

A wait ends by its own lane's clock, so whatever is for whole warps may only follow a wait that the warp has voted on."""

import os
import re

import speculative_decoding_head_gb300 as pkg


def test_warps_go_on_or_give_up_as_one():
    src = open(os.path.join(os.path.dirname(pkg.__file__), "csrc", "k_fp4_linear.cu")).read()
    alone = re.findall(r"mbar_wait\(.*?;", src)
    assert len(re.findall(r"mbar_wait_warp\(", src)) >= 8
    # one lane alone waits only for what is in flight when the kernel has given up already
    assert alone and all(w.endswith("&never);") for w in alone), alone


def test_the_vote_is_of_the_whole_warp():
    src = open(os.path.join(os.path.dirname(pkg.__file__), "csrc", "tc_ptx.cuh")).read()
    body = re.search(r"bool mbar_wait_warp\(.*?\n}", src, re.S).group(0)
    assert "__all_sync(0xFFFFFFFFu, mbar_wait(" in body
