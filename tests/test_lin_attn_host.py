"""CPU checks of what the linear-attention kernels' sources have to hold and no run can
show without a fault."""
import os
import re

from kda_prefill_gb300 import build as kbuild

SOURCE = open(os.path.join(kbuild.CSRC, "kda_lin_walk.cu")).read()


def body(name):
    """The text of a function of the walk's source, comments left out."""
    text = re.sub(r"//[^\n]*", "", SOURCE)
    start = text.index("{", re.search(r"\bvoid\s+(__launch_bounds__\([^)]*\)\s+)?" + name + r"\(", text).end())
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]


def test_every_way_out_of_the_state_role_waits_for_its_stores():
    """A state leaves for the pool by an asynchronous copy from shared memory that is still
    under way when the next item begins.  The role returns from its loops when a wait has
    given up, so the wait for the copies stands behind the role, before the warp joins the
    others and the CTA's shared memory goes."""
    role = body("state_role")
    assert "bulk_commit()" in role and re.search(r"wait_all\([^;]*\)\)? return;", role)
    kernel = re.sub(r"\s+", " ", body("kda_lin_walk"))
    after = kernel[re.search(r"state_role<P, Local>\([^;]*\);", kernel).end():]
    assert after.startswith(" if (x.lane == 0) bulk_wait_all();"), after[:80]


def test_the_other_stores_are_read_before_their_role_can_return():
    """The output rows' copies: nothing can return between a copy and the wait for it."""
    role = body("out_role")
    copies = [m.end() for m in re.finditer(r"bulk_commit\(\);", role)]
    assert copies
    for at in copies:
        rest = role[at:]
        wait = rest.index("bulk_wait_read_all();")
        assert "return" not in rest[:wait]
