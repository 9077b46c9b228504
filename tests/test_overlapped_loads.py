"""Kernels that are launched to overlap the one before them read what that one writes by ordinary loads, read here from
the sources: the read-only path (__ldg, a const __restrict__ parameter) is for data that does not change while the kernel
lives, and a load through it may be moved in front of the wait for the kernel before."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_softmax_attention_fa_gb300", "csrc")


def block(text, *markers):
    """The braces behind the last of the markers, each looked for inside the block of the one before, with what stands
    between marker and brace (a function's parameters)."""
    for marker in markers:
        at = re.search(marker, text)
        assert at, marker
        depth, i = 0, text.index("{", at.end())
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        text = text[at.start():i]
    return text


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def read_only_loads(text):
    """The arguments of the loads through the read-only path."""
    out = []
    for at in re.finditer(r"\b(?:__ldg|ldg_f4)\(", text):
        depth, i = 1, at.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        out.append(text[at.end():i - 1])
    return out


# file, where in it, and the names of what the kernel before writes
PACKED = [
    ("fa_bwd.cu", (r"struct BwdWork<CAUSAL, true> ",), ("sched",)),
    ("fa_bwd.cu", (r"int bwd_total_items\(",), ("sched",)),
    ("fa_bwd.cu", (r"auto fetch_ld = ", r"if constexpr \(RAG\)"), ("from", "lse2", "D")),
    ("fa_bwd256_ragged.cu", (r"auto fetch_ld = ",), ("from", "lse2", "D")),
    ("fa_packed.cu", (r"void __launch_bounds__\(256\) packed_kv_sum_kernel\(",), ("src", "kv_part", "sched")),
]


@pytest.mark.parametrize("name,where,written", PACKED, ids=lambda x: x if isinstance(x, str) else None)
def test_packed_backward(name, where, written):
    text = block(source(name), *where)
    for arg in read_only_loads(text):
        assert not set(written) & set(re.findall(r"\w+", arg)), arg


JOINING = [
    ("fa_fwd.cu", r"void __launch_bounds__\(256\) fwd_combine_kernel\(", ("o_part", "lse_part", "src")),
    ("fa_norm_rope.cu", r"void __launch_bounds__\(1024\) norm_rope_dw_kernel\(", ("part",)),
    ("fa_fwd_kv8.cu", r"kv8_combine_kernel\(", ("part", "part_ml")),
    ("fa_fwd_kv8_tile.cu", r"kv8_tile_combine_kernel\(", ("part", "part_ml", "run")),
]


@pytest.mark.parametrize("name,where,written", JOINING, ids=lambda x: x if isinstance(x, str) and "." in x else None)
def test_joining_kernels(name, where, written):
    text = block(source(name), where)
    for arg in read_only_loads(text):
        assert not set(written) & set(re.findall(r"\w+", arg)), arg
    for parameter in re.findall(r"const [\w ]+\* *__restrict__ (\w+)", text):
        assert parameter not in written, parameter
