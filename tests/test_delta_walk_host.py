"""CPU checks of what the gated delta rule's sources have to hold and no run can show
without a fault or a hang."""
import os
import re

import pytest

from kda_prefill_gb300 import build as kbuild

SOURCES = ["kda_delta_step.cu", "kda_delta_chunk.cu", "kda_delta_walk.cu", "kda_qk_norm_rope.cu"]


def source(name):
    with open(os.path.join(kbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SOURCES)
def test_no_endless_wait(name):
    text = source(name)
    assert not re.search(r"while\s*\(\s*(true|1|!)|for\s*\(\s*;\s*;", text)
    assert not re.search(r"__trap|\bassert\s*\(|brkpt|nanosleep", text)


def test_waits_of_the_walk_are_looked_at():
    """Each wait's result decides whether the role goes on; a wait that gives up tells the others."""
    text = source("kda_delta_walk.cu")
    body = text[text.index("__device__ __forceinline__ bool wait("):]
    body = body[:body.index("\n}")]
    assert "i < kWaitLimit" in body and "abort_flag() = 1" in body and "abort_flag())) return false" in body
    for m in re.finditer(r"(?<![\w.])(mbar_)?wait\(", text):
        line = text[text.rfind("\n", 0, m.start()) + 1:text.index("\n", m.start())]
        assert re.search(r"if \(|bool ok|ok = |&& ok|return |__syncthreads_and|bool wait\(|mbar_wait\(full", line), line


def test_registers_of_the_roles():
    """setmaxnreg draws on what the launch gave: the roles' shares may not exceed it."""
    text = source("kda_delta_walk.cu")
    const = {k: int(v) for k, v in re.findall(r"constexpr int (k\w+) = (\d+);", text)}
    split = [int(x) for x in re.findall(r"setmaxnreg\.\w+\.sync\.aligned\.u32 (\d+);", text)]
    assert len(split) == 3 and const["kThreads"] == 768
    warps = (const["kMakers"], const["kWriters"], const["kThreads"] // 32 - const["kMakers"] - const["kWriters"])
    launch = 65536 // const["kThreads"] // 8 * 8
    assert sum(32 * w * r for w, r in zip(warps, split)) <= const["kThreads"] * launch
    assert all(w % 4 == 0 for w in warps)
