"""CPU checks of the few-token kernels' sources for what no result shows."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "activation_sparse_feedforward_amd", "csrc")
SOURCES = ("few_token.hpp", "k_linear4.hip", "k_moe.hip", "k_weights.hip")


def _code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SOURCES)
def test_lanes_hand_over_through_lds_between_fences(name):
    """A wave barrier orders no memory: it stands between a release and an acquire fence wherever it is used."""
    fenced = re.compile(r'__builtin_amdgcn_fence\(__ATOMIC_RELEASE, "wavefront"\);\s*'
                        r'__builtin_amdgcn_wave_barrier\(\);\s*'
                        r'__builtin_amdgcn_fence\(__ATOMIC_ACQUIRE, "wavefront"\);')
    assert "__builtin_amdgcn_wave_barrier" not in fenced.sub("", _code(name))


def test_what_is_stored_to_in_16_bytes_is_aligned_to_16():
    """LDS that 16-byte vectors go to says so itself; the compiler's placing of variables is not relied on."""
    code = _code("k_moe.hip")
    assert "reinterpret_cast<u32x4_t*>(l.taken)" in code
    assert re.search(r"struct alignas\(16\) WaveList \{\s*uint8_t taken\[", code)
    for name in SOURCES:
        for line in _code(name).splitlines():
            if re.search(r"__shared__.*\bchar lds\[", line):
                assert "__align__(16)" in line, (name, line)


@pytest.mark.parametrize("name", [n for n in SOURCES if n.endswith(".hip")])
def test_kernels_handed_lds_at_launch_ask_for_it(name):
    """More than 64 KB of LDS, the kernel's own included, is asked for in one place that every such launch goes through:
    launch() itself is for kernels that are handed none."""
    code = _code(name)
    assert "hipFuncSetAttribute" not in code and "<<<" not in code
    handed = re.findall(r"void (\w+_kernel)\(\w+ a\) \{(?:(?!\n\}).)*?extern __shared__", code, re.S)
    assert handed == {"k_linear4.hip": ["linear4_kernel"], "k_moe.hip": ["moe_up_kernel", "moe_down_kernel"],
                      "k_weights.hip": []}[name]
    for kernel in handed:
        assert re.search(rf"launch_lds<&{kernel}<", code)
        assert not re.search(rf"launch\({kernel}<", code)


def test_down_kernel_for_few_tokens_fetches_no_further_ahead_than_a_wave_has_blocks():
    """The launcher's limit on (pair, block)s, over the kernel's waves, is what a wave fetches at once: a longer body
    would be code that no call reaches."""
    code = _code("k_moe.hip")
    assert re.search(r"blocks <= few_blocks<E>\(\)", code)
    kernel = code[code.index("void moe_down_few_kernel"):code.index("hipError_t go_route")]
    assert re.findall(r"template run<(.*)>\(x,", kernel) == ["few_blocks<E>() / kFewWaves"]
