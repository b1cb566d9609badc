"""The GPU tests' cases reach every way that the calls go: asked of the library, no GPU needed."""
import pytest

import sparse_gemm_layers_amd as sg
import test_gpu_gated_ways as gated


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


@pytest.mark.parametrize("bad", [(0, 8, 8), (1, 12, 8), (1, 8, 12), (1 << 31, 8, 8)])
def test_plans_refuse_what_the_calls_refuse(bad):
    for call in (sg.gated_gemm_plan, sg.gated_gemm_backward_plan):
        with pytest.raises(sg.SgError):
            call(*bad)


def test_plan_and_workspace_agree():
    for T, F, D in [c[:3] for c, _ in gated.FORWARD] + [c[:3] for c in gated.BACKWARD]:
        need = [4 * p * T * D if p > 1 else 0 for p in (sg.gated_gemm_backward_plan(T, F, D, dw)[1] for dw in (True, False))]
        assert sg.gated_gemm_backward_workspace(T, F, D) == max(need)
