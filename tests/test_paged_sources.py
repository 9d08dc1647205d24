"""Rules of the paged cache's CUDA sources that a wrong build need not show in its results."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "io_aware_attention_fa2_gb300", "csrc")


def sources():
    """File name -> text without comments."""
    out = {}
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            text = open(os.path.join(CSRC, name)).read()
            out[name] = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    return out


CHAINED = [name for name, text in sources().items() if "launch_chained" in text]


def test_the_chained_kernels_are_found():
    assert set(CHAINED) == {"fa_paged.cu", "fa_paged.cuh", "fa_paged_decode.cu",
                            "fa_key_weights.cu"}


@pytest.mark.parametrize("name", CHAINED)
def test_inputs_of_chained_kernels_are_not_declared_read_only(name):
    """A kernel that is launched while the one before it still writes its inputs must not let the
    compiler load them through the non-coherent path or above the wait."""
    text = sources()[name]
    for word in ("__restrict__", "__ldg", ".nc", "restrict"):
        assert word not in text, word


@pytest.mark.parametrize("name", CHAINED)
def test_loads_past_l1_keep_their_place(name):
    """The move's loads must stay behind its wait and in front of its cluster barrier: they are
    assembly that is volatile and clobbers memory, not intrinsics without a promised order."""
    text = sources()[name]
    assert not re.search(r"__ld(cg|ca|cs|cv|lu)\b", text)
    for asm in re.findall(r"asm[^;]*?\(\s*\"ld\.global.*?\);", text, flags=re.S):
        assert asm.startswith("asm volatile") and '"memory"' in asm, asm


@pytest.mark.parametrize("name", [n for n in CHAINED if n.endswith(".cu")])
def test_every_chained_kernel_waits(name):
    """Every kernel of these files is launched so, and waits for the one before it."""
    text = sources()[name]
    assert text.count("__global__") == text.count("  wait_prerequisites();")


def test_dynamic_shared_memory_is_aligned():
    """A dynamic shared array is declared with the alignment of its widest access (16 bytes), or
    its base is rounded up by hand."""
    found = 0
    for name, text in sources().items():
        for line in re.findall(r"extern __shared__[^;]*;", text):
            found += 1
            if "smem_raw" in line:
                assert "(smem_raw) + 1023u) & ~1023u" in text, name
            else:
                assert "__align__(16)" in line, (name, line)
    assert found >= 5


def test_launches_report_their_own_status():
    """No launch of the cache's files asks for the last error, which an earlier call may have
    left: the error query would then fail after it has cleared the word."""
    for name in CHAINED:
        text = sources()[name]
        assert "<<<" not in text and "cudaGetLastError" not in text, name
