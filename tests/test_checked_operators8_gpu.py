"""The bounds-checked build and the calls on 8-bit rows: whole layers count
nothing, ranges outside the buffers are skipped and counted."""
import pytest
import torch

from tests.test_checked_gpu import epxc  # noqa: F401  (the binding bound to the checked library)
from tests.test_experts8_gpu import gen, int8, kept_guard, kept_untouched, kept_values, scales32
from tests.test_experts_gpu import guard, make_rows, rand, untouched

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8_rows", [False, True])
def test_whole_layer_without_violations(epxc, int8_rows):  # noqa: F811
    from tests.test_layer8_gpu import Kept, check_gradients
    epxc.epx_checked_violations()
    lay = Kept(epxc, 128, 16, 4, 288, 160, seed=3, int8=int8_rows)
    lay.forward()
    lay.backward()
    torch.cuda.synchronize()
    assert epxc.epx_checked_violations() == 0
    check_gradients(lay)


def test_bad_ranges_are_skipped_and_counted(epxc):  # noqa: F811
    g = gen(32)
    off, cnt, R, N, K = [0, -1, 60, 20], [10, 5, 5, 8], 64, 64, 96
    good, kept = [0, 0, 0, 20], [10, 0, 0, 8]
    rows = make_rows(epxc, off, cnt, R)
    calls = []
    out, dx, act = guard(R, N), guard(R, 2 * N), guard(R, N)
    codes, scales = kept_guard(R, 2 * N)
    x, w, sx, sw = int8(g, R, K), int8(g, 4, 2 * N, K), scales32(g, R), scales32(g, 4, 2 * N)
    calls.append(lambda: epxc.epx_expert_gemm_int8(rows, x, sx, w, sw, out, act=epxc.ACT_SWIGLU, preact_codes=codes,
                                                   preact_scales=scales))
    bx, bw = rand(g, R, K), rand(g, 4, 2 * N, K, std=0.1)
    calls.append(lambda: epxc.epx_expert_gemm_keep8(rows, bx, bw, out, codes, scales))
    dy, w2 = rand(g, R, K), rand(g, 4, K, N, std=0.1)
    pc, ps = kept_values(g, R, 2 * N)
    calls.append(lambda: epxc.epx_expert_gemm_dgrad_kept8(rows, dy, w2, pc, ps, dx, act_out=act))
    xc, xs = kept_values(g, R, K)
    dw = guard(4, 2 * N, K, dtype=torch.float32)
    calls.append(lambda: epxc.epx_expert_gemm_wgrad_kept8(rows, rand(g, R, 2 * N), xc, xs, dw))
    for i, call in enumerate(calls):
        epxc.epx_checked_violations()
        call()
        torch.cuda.synchronize()
        assert epxc.epx_checked_violations() > 0, i
    for t in (out, dx, act):
        untouched(t, good, kept, "rows")
    kept_untouched(codes, scales, good, kept)
    assert not dw[1:3].any()
