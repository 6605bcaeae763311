"""How the 4-bit product's kernel waits (of its source; a wait that runs out is not to be provoked on a GPU).

A wait ends by its own lane's clock, so whatever is for whole warps may only go by a wait that the warp has voted on."""

import os
import re

import speculative_decoding_head_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def test_warps_go_on_or_give_up_as_one():
    src = open(os.path.join(CSRC, "k_fp4_linear.cu")).read()
    assert len(re.findall(r"mbar_wait_warp\(", src)) >= 6
    for m in re.finditer(r"[^\n;{}]*\bmbar_wait\(.*?;", src):
        wait = m.group(0).strip()
        # one lane alone for what is in flight when the kernel has given up, a wait inside a vote, and U's boxes
        assert (wait.endswith("&never);") or wait.startswith("ok = __all_sync(0xFFFFFFFFu, ok && tc::mbar_wait(")
                or "ok = ok && tc::mbar_wait(bar(&bars.ufull" in wait), wait
    # between a wait for U's box, which each lane remembers for itself, and the next vote no lane goes by it
    put = src[src.index("auto put = ["):src.index("float wf_next")]
    assert len(re.findall(r"\bok\b", put)) == 2, "put() only takes `ok` along"


def test_the_vote_is_of_the_whole_warp():
    src = open(os.path.join(CSRC, "tc_ptx.cuh")).read()
    body = re.search(r"bool mbar_wait_warp\(.*?\n}", src, re.S).group(0)
    assert "__all_sync(0xFFFFFFFFu, mbar_wait(" in body
