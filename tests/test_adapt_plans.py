"""The GPU tests' cases reach every way that the calls go: asked of the library, no GPU needed."""
import pytest

import sparse_gemm_layers_amd as sg
import test_gpu_gated_ways as gated
import test_gpu_lora_ways as lora


def test_gated_forward_ways_are_reached():
    ways = {(16, 16), (64, 32), (128, 64), (256, 64), (256, 128)}
    for size, way in gated.FORWARD:
        assert sg.gated_gemm_plan(*size[:3]) == way, size
    assert {way for _, way in gated.FORWARD} == ways
    # sums longer than any ring of blocks (five of 64)
    assert all(size[2] > 8 * 64 for size, _ in gated.FORWARD)
    seen = {sg.gated_gemm_plan(T, 8 * f, 64) for T in (1, 16, 17, 40, 100, 200, 300, 500, 1000, 3000) for f in range(1, 2000, 7)}
    assert seen == ways


def test_gated_backward_ways_are_reached():
    for T, F, D, dw, way in gated.BACKWARD:
        assert gated.backward_way(T, F, D, dw) == way, (T, F, D, dw)
    assert {(dw, way) for *_, dw, way in gated.BACKWARD} == {(d, (t, p)) for d in (True, False) for t in (128, 256)
                                                             for p in (True, False)}


def lora_sizes():
    return [(T, K, N, r, L) for T in (1, 40, 64, 65, 100, 300, 500, 511, 512, 700, 1500, 2048, 2049, 4100, 9000)
            for K, N in ((72, 136), (1032, 72), (72, 1032), (1032, 2056), (4096, 4096), (14336, 4096))
            for r in (8, 16, 24, 32, 40, 64, 72, 128, 200, 256) for L in (1, 2, 20)]


def test_adapter_ways_are_reached():
    for size, forward, backward in lora.CASES:
        assert lora.forward_way(*size[:5]) == forward and lora.backward_way(*size[:5]) == backward, size
    assert {f for _, f, _ in lora.CASES} == {lora.forward_way(*s) for s in lora_sizes()}

    def ways(b):
        tokens, ranks, v, u, sum_ranks, parts = b
        return {("first launch", tokens, ranks), ("parts of dy . B", v), ("parts of x . A^T", u),
                ("sums", sum_ranks, parts > 1)}

    reached = set().union(*(ways(b) for *_, b in lora.CASES))
    assert reached == set().union(*(ways(lora.backward_way(*s)) for s in lora_sizes()))


@pytest.mark.parametrize("bad", [(0, 8, 8, 8, 1), (1, 12, 8, 8, 1), (1, 8, 12, 8, 1), (1, 8, 8, 264, 1), (1, 8, 8, 8, 65536)])
def test_adapter_plans_refuse_what_the_calls_refuse(bad):
    for call in (sg.lora_gemm_plan, sg.lora_gemm_backward_plan):
        with pytest.raises(sg.SgError):
            call(*bad)


@pytest.mark.parametrize("bad", [(0, 8, 8), (1, 12, 8), (1, 8, 12), (1 << 31, 8, 8)])
def test_plans_refuse_what_the_calls_refuse(bad):
    for call in (sg.gated_gemm_plan, sg.gated_gemm_backward_plan):
        with pytest.raises(sg.SgError):
            call(*bad)


def test_plan_and_workspace_agree():
    for T, F, D in [c[:3] for c, _ in gated.FORWARD] + [c[:3] for c in gated.BACKWARD]:
        need = [4 * p * T * D if p > 1 else 0 for p in (sg.gated_gemm_backward_plan(T, F, D, dw)[1] for dw in (True, False))]
        assert sg.gated_gemm_backward_workspace(T, F, D) == max(need)
