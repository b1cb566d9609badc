"""What the assembly of the bf16 tile and adapter kernels as built has to show.
Needs hipcc and no GPU.

The tile product's loads into LDS are written in assembly and set m0 without naming it
(the compiler does not allow it to be named).  That is right as long as the compiler
itself keeps nothing in m0 there: no instruction of its own may read or write it.  No
kernel spills registers: the tile product counts the loads that may be in flight."""
import os
import re
import subprocess

import pytest

from sparse_gemm_layers_amd import build as B

SOURCES = ["gated.hip", "lora.hip"]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """source -> {mangled name: assembly of that kernel, with its statistics}, compiled when asked for."""
    done = {}

    def of(source):
        if not os.path.exists(B.HIPCC):
            pytest.skip("hipcc not available")
        if source not in done:
            asm = tmp_path_factory.mktemp("asm") / "device.s"
            r = subprocess.run([B.HIPCC, *B.CFLAGS, *B.SRC_FLAGS.get(source, []), "--cuda-device-only", "-S",
                                os.path.join(B.CSRC, source), "-o", str(asm)], capture_output=True, text=True)
            assert r.returncode == 0, r.stderr
            parts = re.split(r"^(?=_Z\w+:)", asm.read_text(), flags=re.M)[1:]
            done[source] = {p.split(":", 1)[0]: p for p in parts}
        return done[source]

    return of


@pytest.mark.timeout(300)
@pytest.mark.parametrize("source", SOURCES)
def test_no_spills(source, kernels):
    bad = []
    for name, f in kernels(source).items():
        scratch = re.search(r"; ScratchSize: (\d+)", f)
        assert scratch, name
        if int(scratch.group(1)):
            bad.append(f"{name}: {scratch.group(1)} bytes a lane")
    assert not bad, "\n".join(bad)


@pytest.mark.timeout(300)
def test_m0_is_the_loads_alone(kernels):
    tiles = 0
    for name, f in kernels("gated.hip").items():
        body = f.split(".Lfunc_end", 1)[0]
        loads = body.count("offen lds")
        outside = re.sub(r";;#ASMSTART.*?;;#ASMEND", "", body, flags=re.S)
        assert not re.search(r"\bm0\b", outside), name
        assert not re.search(r"buffer_load\w* .*\blds\b", outside), name
        assert len(re.findall(r"s_add_u32 m0,", body)) == loads, name
        tiles += loads > 0
    assert tiles >= 8


@pytest.mark.timeout(300)
def test_no_wait_for_all_loads_in_the_tile_loop(kernels):
    """Where a tile kernel multiplies or loads into LDS, only the waits that count loads."""
    seen = 0
    for name, f in kernels("gated.hip").items():
        body = f.split(".Lfunc_end", 1)[0]
        if "offen lds" not in body:
            continue
        for block in re.split(r"^(?=\.LBB)", body, flags=re.M):
            if "v_mfma" in block:
                outside = re.sub(r";;#ASMSTART.*?;;#ASMEND", "", block, flags=re.S)
                assert "vmcnt" not in outside, name
                seen += 1
    assert seen >= 8
