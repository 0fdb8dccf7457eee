"""Properties of the kernels' sources that no run shows."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "turboquant_kv_cache_tq_gb300", "csrc")


def _sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            with open(os.path.join(CSRC, name)) as f:
                yield name, f.read()


def test_dynamic_shared_memory_states_its_alignment():
    """Dynamic shared memory follows a kernel's static arrays: without an
    alignment of its own it starts wherever they happen to end, and 16-byte
    accesses to it work by luck."""
    found = 0
    for name, text in _sources():
        for line in re.findall(r"extern __shared__[^;]*;", text):
            found += 1
            align = re.search(r"__align__\((\d+)\)", line)
            assert align and int(align.group(1)) >= 16, (name, line)
    assert found >= 6


def test_device_helpers_of_the_ragged_caches_have_callers():
    text = dict(_sources())
    everything = "".join(text.values())
    for name in ("tq_ragged.cuh", "tq_ragged_tiles.cuh", "tq_tcgen05.cuh", "tq_tree_attention.cuh"):
        for helper in re.findall(r"__forceinline__ [\w:<> ]*?(\w+)\(", text[name]):
            if helper not in ("TileUnit", "operator"):  # (a constructor)
                assert len(re.findall(r"\b%s\b" % helper, everything)) > 1, (name, helper)


def test_calls_on_ragged_caches_cannot_throw():
    """Below a C entry point an exception ends the process: no containers,
    strings, locks or allocations that throw."""
    text = dict(_sources())
    for name in ("tq_ragged.cuh", "tq_ragged_tiles.cuh", "tq_tcgen05.cuh", "tq_tree_attention.cuh", "tq_tree_attention.cu",
                 "tq_attention_weights.cu", "tq_evict.cu"):
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", text[name], flags=re.S)
        assert not re.search(r"std::(vector|string|map|function|mutex|lock_guard)|\bnew\b|\bthrow\b", code), name
