"""Every hand-off of a tensor-memory accumulator between threads carries its tcgen05 fences, read from the kernels'
sources: PTX orders the tcgen05 operations of two threads only when fence::before_thread_sync stands ahead of the
first one's arrival (tcgen05.commit implies it for MMAs) and fence::after_thread_sync behind the other one's wait."""
import os
import re

import pytest

from int8_fully_quantized_b200 import build_lib

# accumulator (and scale-column) barriers; `full` / `empty` of the shared-memory ring order no tensor memory
BARRIERS = r"(?:tfull|tempty|acc_full|acc_empty|sf_full)"
EVENTS = [
    ("wait", re.compile(r"\bmbar_(?:try_)?wait(?:_often)?(?:<\w+>)?\(\s*&" + BARRIERS + r"\[")),
    ("arrive", re.compile(r"\bmbar_arrive(?:_if)?\(\s*&" + BARRIERS + r"\[")),
    ("after", re.compile(r"\btc_fence_after\(")),
    ("before", re.compile(r"\btc_fence_before\(")),
    ("access", re.compile(r"\b(?:tmem_ld\w*|tmem_st\w*|mma_\w+|block)\(")),   # `block`: a sum warp's load and use of one accumulator
]
KERNELS = [("gemm.cu", "gemm_i8_kernel"), ("gemm.cu", "gemm_i8_s32_kernel"), ("mxfp8.cu", "mxf8_gemm_kernel")]


def body(name, kernel):
    text = open(os.path.join(build_lib.CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    at = re.search(r"__global__[^;{]*\b" + kernel + r"\s*\(", text).end()
    i = start = text.index("{", at)
    depth = 0
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[start:i]


def events(text):
    found = sorted((m.start(), what) for what, pattern in EVENTS for m in pattern.finditer(text))
    return [what for _, what in found]


def unfenced(seq):
    """Indexes of accesses not fenced from the wait before them and of arrivals not fenced from the access before."""
    bad, waited, used = [], False, False
    for i, what in enumerate(seq):
        if what == "wait":
            waited = True
        elif what == "after":
            waited = False
        elif what == "before":
            used = False
        elif what == "access":
            if waited:
                bad.append(i)
            used = True
        elif what == "arrive" and used:
            bad.append(i)
    return bad


def test_the_reader_sees_missing_fences():
    assert unfenced(["wait", "after", "access", "before", "arrive"]) == []
    assert unfenced(["wait", "access", "before", "arrive"]) == [1]
    assert unfenced(["wait", "after", "access", "arrive"]) == [3]


@pytest.mark.parametrize("name,kernel", KERNELS)
def test_hand_offs_are_fenced(name, kernel):
    seq = events(body(name, kernel))
    assert seq.count("wait") >= 2 and seq.count("arrive") >= 1 and "access" in seq
    assert unfenced(seq) == [], seq


def test_scale_columns_are_fenced():
    """The warps that rewrite a stage's scale columns in tensor memory learn from the stage's `full` barrier that the
    MMAs which read them are done (their commit freed the stage for the producer, whose copies complete `full`)."""
    text = body("mxfp8.cu", "mxf8_gemm_kernel").replace("&full[", "&sf_full[")
    seq = events(text)
    assert unfenced(seq) == [], seq
