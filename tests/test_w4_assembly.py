"""What the assembly of the 4-bit kernels as built has to show.  Needs hipcc and no GPU.

Few-rows kernels: a wave's part of LDS is refilled by loads that write LDS
themselves, and such a write is not ordered against the wave's own LDS reads.  So
no read may be outstanding where a refill is issued: along every path, the most LDS
operations that may be in flight (lgkmcnt) is zero at each load into LDS.

All of them: no registers are spilled to memory; the waits count loads, and spills
count among those."""
import os
import re
import subprocess

import pytest

from sparse_gemm_layers_amd import build as B

KERNELS = {"gemm_w4a16.hip": ("k_w4_rows",), "moe_mlp.hip": ("k_moe_gate_up_rows", "k_moe_down_join")}
CAP = 64


def outstanding(lines):
    """Instructions of one function -> [(line, text, most LDS operations in flight)] of its loads into LDS."""
    starts, blocks, cur = {}, [], None
    for n, line in enumerate(lines):
        text = line.split(";")[0].strip()
        label = re.match(r"^([.\w$]+):", text)
        if label or cur is None:
            cur = []
            blocks.append(cur)
            if label:
                starts[label.group(1)] = len(blocks) - 1
                continue
        if not text or text.startswith("."):
            continue
        cur.append((n, text))
        if text.startswith(("s_branch", "s_cbranch", "s_endpgm")):
            cur = None
    after = []
    for i, b in enumerate(blocks):
        last = b[-1][1] if b else ""
        nxt = [] if last.startswith(("s_branch", "s_endpgm")) or i + 1 == len(blocks) else [i + 1]
        if last.startswith(("s_branch", "s_cbranch")):
            nxt.append(starts[last.split()[1]])
        after.append(nxt)

    def run(i, have, sink=None):
        for n, text in blocks[i]:
            op = text.split()[0]
            if op.startswith("ds_"):
                have = min(have + 1, CAP)
            elif op == "s_waitcnt":
                m = re.search(r"lgkmcnt\((\d+)\)", text)
                if m:
                    have = min(have, int(m.group(1)))
                else:
                    assert "vmcnt" in text or "expcnt" in text, text     # no bare immediates
            elif op.startswith("buffer_load") and text.split()[-1] == "lds" and sink is not None:
                sink.append((n, text, have))
        return have

    state = [0] + [-1] * (len(blocks) - 1)
    todo = [0]
    while todo:
        i = todo.pop()
        out = run(i, state[i])
        for j in after[i]:
            if out > state[j]:
                state[j] = out
                todo.append(j)
    found = []
    for i, s in enumerate(state):
        if s >= 0:
            run(i, s, found)
    return found


def test_the_check_itself():
    loop = ["ds_read_b128 v[0:3], v9", "s_waitcnt lgkmcnt(0)", ".L1:", "buffer_load_dwordx4 v1, s[0:3], 0 offen lds",
            "ds_read_b128 v[0:3], v9", "s_cbranch_scc0 .L1", "s_endpgm"]
    assert [h for _, _, h in outstanding(loop)] == [CAP]                 # the read of the pass before
    loop.insert(5, "s_waitcnt vmcnt(0) lgkmcnt(0)")
    assert [h for _, _, h in outstanding(loop)] == [0]
    one = ["ds_read_b32 v0, v9", "ds_read_b32 v1, v9", "s_waitcnt lgkmcnt(1)", "buffer_load_dword v1, s[0:3], 0 offen lds",
           "buffer_load_dword v1, v2, s[0:3], 0 offen"]
    assert [h for _, _, h in outstanding(one)] == [1]


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
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
@pytest.mark.parametrize("source", sorted(KERNELS))
def test_no_read_in_flight_at_a_refill(source, functions):
    seen, bad = set(), []
    for name, f in functions(source).items():
        which = [k for k in KERNELS[source] if k in name]
        if not which:
            continue
        refills = outstanding(f.split(".Lfunc_end", 1)[0].splitlines()[1:])
        assert refills, f"{name}: no load into LDS found"
        seen.update(which)
        worst = max(h for _, _, h in refills)
        if worst:
            bad.append(f"{name}: {sum(h > 0 for _, _, h in refills)} of {len(refills)} refills, up to {worst} reads in flight")
    assert seen == set(KERNELS[source])
    assert not bad, "\n".join(bad)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("source", ["gemm_w4a16.hip", "moe_mlp.hip", "moe_route.hip"])
def test_no_spills(source, functions):
    bad = []
    for name, f in functions(source).items():
        scratch = re.search(r"; ScratchSize: (\d+)", f)
        assert scratch, name
        if int(scratch.group(1)):
            bad.append(f"{name}: {scratch.group(1)} bytes a lane")
    assert not bad, "\n".join(bad)
