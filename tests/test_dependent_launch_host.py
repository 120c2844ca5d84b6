"""Kernels that are launched as dependents read what their predecessor writes by ordinary loads.

A dependent launch starts while its predecessor still runs, so that what that one writes is not
read-only for the kernel's whole life, which __ldg asks for. The race does not show in results (it
depends on what the compiler moves and what a cache holds), so the sources are checked."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "memory_efficient_attention_b200", "csrc")


def read(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(src, name):
    """The braces after the definition of `name`."""
    start = re.search(r"\b%s\s*\([^;{]*\)\s*\{" % name, src).end() - 1
    depth = 0
    for i in range(start, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[start:i + 1]
    raise AssertionError(name)


def ldg_arguments(text):
    out = []
    for m in re.finditer(r"__ldg\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        out.append(text[m.end():i - 1])
    return out


# What the kernel launched before writes (block choice, split kernels, eviction's selection), in the
# kernels that depend on it and the functions that they read it through. None: the predecessor is
# the caller's, and may have written every input.
DEPENDENTS = [
    ("decode_sm100.cuh", "mea_decode_split_kernel", None),
    ("decode_sm100.cuh", "dec_selected_keys", None),
    ("decode_sm100.cuh", "mea_selected_merge_kernel", ("ws_o", "ws_lse")),
    ("decode_sm100.cuh", "mea_decode_weights_kernel", ("ws_o", "ws_lse", "ws_s")),
    ("decode_sm100.cuh", "dec_merge", ("ws_o", "ws_lse", "ws_s")),
    ("cache_sm100.cuh", "mea_evict_copy_kernel", ("kept", "out_weights", "out_cu")),
    ("tree_sm100.cuh", "mea_tree_merge_kernel", ("ws_o", "ws_lse")),
    ("weights_sm100.cuh", "mea_weights_merge_kernel", ("ws",)),
]


@pytest.mark.parametrize("unit,name,written", DEPENDENTS, ids=[n for _, n, _ in DEPENDENTS])
def test_no_read_only_loads_of_what_the_predecessor_writes(unit, name, written):
    for arg in ldg_arguments(body(read(unit), name)):
        assert written is not None, f"{name}: __ldg({arg})"
        assert not re.search(r"\bp\.(%s)\b" % "|".join(written), arg), f"{name}: __ldg({arg})"


def test_every_dependent_launch_is_in_the_table():
    names = {n for _, n, _ in DEPENDENTS}
    for unit in sorted(os.listdir(CSRC)):
        if unit.endswith(".cu"):
            for kern in re.findall(r"launch_dependent\(\s*(?:mea::)?(\w+)", read(unit)):
                assert kern in names or kern == "kern", (unit, kern)
