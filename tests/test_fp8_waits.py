"""The 8-bit float tiles' main loops wait for the copies that they read.

A loop's copies into LDS run on across its barrier, and a wait that counts
the newer memory operations (vmcnt) lets the earlier ones finish: the copies
that the iteration before issued behind its barrier.  The count in the source
holds only where the compiler leaves the newer ones before the wait, and none
but copies behind it: read here from the assembly of the compiled loops."""
import os
import re
import subprocess

import pytest

from expert_ffn_layer_router_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc") and not os.environ.get("HIPCC"),
                                reason="hipcc not installed")
MEMORY = ("buffer_", "global_", "flat_", "scratch_")


def _loops(assembly):
    """Of each tile kernel the blocks that multiply and pass a barrier: lists of instructions."""
    for name in re.findall(r"^(_ZN\S+fp8_tile_kernel\S+):", assembly, re.M):
        body = assembly[assembly.index(f"\n{name}:"):]
        for block in re.split(r"\n(?=\.LBB)", body[:body.index(".Lfunc_end")]):
            lines = [line.strip() for line in block.split("\n")]
            if sum(line.startswith("v_mfma") for line in lines) >= 16 and "s_barrier" in lines:
                yield name, lines


def test_waits_cover_the_copies(tmp_path):
    out = tmp_path / "tile.s"
    subprocess.run([build._hipcc(), *build.HIPCC_FLAGS, "--cuda-device-only", "-S", "-o", str(out),
                    os.path.join(build.CSRC, "fp8_tile.hip")], check=True, stdout=subprocess.PIPE,
                   stderr=subprocess.STDOUT)
    names = []
    for name, lines in _loops(out.read_text()):
        names.append(name)
        assert lines.count("s_barrier") == 1, name
        barrier = lines.index("s_barrier")
        wait = max(i for i in range(barrier) if lines[i].startswith("s_waitcnt vmcnt"))
        newer = sum(line.startswith(MEMORY) for line in lines[:wait])
        assert int(re.search(r"vmcnt\((\d+)\)", lines[wait]).group(1)) <= newer, name
        behind = [line for line in lines[wait:] if line.startswith(MEMORY)]
        assert behind and all(re.search(r"\blds\b", line) for line in behind), name
    assert len(set(names)) == len(names) == 6
