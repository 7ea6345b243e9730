"""What the operators' sources have to keep to and no run can show (CPU only).

A load through the read-only path (__ldg) is defined only for memory that stays as it is while the
kernel runs; the compiler may move it behind a store of the same kernel, or repeat it there.  So a
tensor that a call may name as input and output at once is read by plain loads."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "recurrent_vision_backbone_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", text)


def body(text, name):
    """The function or kernel `name` with its braces."""
    i = text.index("{", re.search(r"\b%s\(" % name, text).end())
    depth, j = 0, i
    while True:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
        if depth == 0:
            return text[i:j]


def read_only_loads(text):
    """The arguments of the loads through the read-only path (load_raw and ld16 are such)."""
    found = []
    for m in re.finditer(r"(?:__ldg|\bload_raw(?:<\w+>)?|\bld16)\(", text):
        depth, j = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[j], 0)
            j += 1
        found.append(text[m.end():j - 1])
    return found


def test_carried_rows_of_the_convolution():
    """final_state may be init_state: no read-only load of init_state, by its name or through a
    pointer that may stand for it."""
    text = source("causal_conv.cuh")
    assert "a.init" in text
    loads = read_only_loads(text)
    for name in ["a.init"] + re.findall(r"\*\s*(\w+)\s*=[^;]*a\.init\b", text):
        assert not [a for a in loads if re.search(r"(?<![\w.])%s\b" % re.escape(name), a)], name


@pytest.mark.parametrize("kernel", ["group_norm_results_kernel", "group_norm_apply_kernel"])
def test_rows_of_a_norm_in_place(kernel):
    """out may be x: the kernels that write out read x by plain loads."""
    loads = read_only_loads(body(source("group_norm.cu"), kernel))
    assert loads   # the parameters
    assert not [a for a in loads if re.search(r"(?<![\w.])a\.x\b", a)]


def test_error_words_are_taken_in_one_step():
    """Kernels of other streams may set an error bit at any time: a word is cleared by the exchange that
    reads it, never by a copy after it."""
    for name in sorted(os.listdir(CSRC)):
        assert not re.search(r"cudaMemcpy(?:To|From)Symbol(?:Async)?\([^;]*error_word", source(name)), name
