"""The experts' shared tiles wait for DMAs by counting the loads issued behind them:
the compiled order, from the assembly of the source."""
import os
import re
import subprocess

import pytest

from int8_mixed_precision_outlier_amd import build


def memory_operations(assembly, kernel):
    """For each instance of a kernel its memory instructions in order: 'd' a DMA into
    LDS, 'w' another vector load, '|' a barrier with the vmcnt of the wait right
    before it ('' without one)."""
    found, name, wait = {}, None, ""
    for line in assembly.splitlines():
        m = re.match(r"(_ZN\S*%s\S*):" % kernel, line)
        if m:
            name = m.group(1)
            found[name] = []
            continue
        word = line.split(";")[0].split()
        if name is None or not word or not re.match(r"[a-z]", word[0]):
            continue
        if word[0] == "s_barrier":
            found[name].append("|" + wait)
        elif word[0].startswith("buffer_load"):
            found[name].append("d" if word[-1] == "lds" else "w")
        elif word[0].startswith("global_load") or word[0].startswith("buffer_store"):
            found[name].append("o")
        m = re.search(r"s_waitcnt.*vmcnt\((\d+)\)", line)
        wait = m.group(1) if m else ""
        if word[0] == "s_endpgm":
            name = None
    return found


def test_parser():
    text = ("_ZN1k_a:\n\tbuffer_load_dwordx4 v1, s[0:3], 0 offen lds\n\tbuffer_load_dwordx4 v[1:4], v5, s[0:3], 0 offen nt\n"
            "\ts_waitcnt vmcnt(1)\n\t;;#ASMSTART\n\ts_barrier\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier\n\ts_endpgm\n")
    assert memory_operations(text, "k_a") == {"_ZN1k_a": ["d", "w", "|1", "|"]}


@pytest.mark.skipif(not any(c and os.path.exists(c) for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc")),
                    reason="needs hipcc")
def test_dmas_are_in_front_of_the_loads_that_the_waits_count(tmp_path):
    out = tmp_path / "moe_experts.s"
    subprocess.run([build.hipcc(), *build.common_flags(), "--cuda-device-only", "-S", os.path.join(build.CSRC, "moe_experts.hip"),
                    "-o", str(out)], check=True, capture_output=True, timeout=300)
    kernels = memory_operations(out.read_text(), "k_moe_wide")
    assert len(kernels) == 3  # first product of both types, second product
    for name, ops in kernels.items():
        counted = 0
        for i, op in enumerate(ops):
            if op[0] == "|" and op[1:] not in ("", "0"):
                n = int(op[1:])
                assert ops[i - n:i] == ["w"] * n, (name, i, ops[max(0, i - 16):i + 1])
                counted += 1
        assert counted >= 12, (name, counted)  # a first tile and two steps for 1 to 4 blocks of tokens
