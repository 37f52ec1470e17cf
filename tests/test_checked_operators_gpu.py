"""The bounds-checked build and the experts' row ranges: ranges inside the
buffers count nothing, ranges outside are skipped and counted."""
import pytest
import torch

from tests import experts_reference as ref
from tests.test_checked_gpu import epxc  # noqa: F401  (the binding bound to the checked library)
from tests.test_experts_gpu import gen, guard, make_rows, rand, untouched

pytestmark = pytest.mark.gpu


def run(epxc, off, cnt, R, good):  # noqa: F811
    g = gen(31)
    N, K = 136, 200
    rows = make_rows(epxc, off, cnt, R)
    n = len(cnt)
    x, w, dy = rand(g, R, K), rand(g, n, N, K, std=K ** -0.5), rand(g, R, N)
    out, dx, dw = guard(R, N), guard(R, K), guard(n, N, K, dtype=torch.float32)
    epxc.epx_checked_violations()
    epxc.epx_expert_gemm(rows, x, w, out)
    epxc.epx_expert_gemm_dgrad(rows, dy, w, dx)
    epxc.epx_expert_gemm_wgrad(rows, dy, x, dw)
    kept = [c if e in good else 0 for e, c in enumerate(cnt)]
    safe = [o if e in good else 0 for e, o in enumerate(off)]
    count = epxc.epx_checked_violations()
    ref.close(out, *ref.product(x.double(), w.double(), safe, kept), ref.BF16, "out")
    ref.close(dx, *ref.product(dy.double(), w.double().transpose(1, 2), safe, kept), ref.BF16, "dx")
    untouched(out, safe, kept, "out")
    return count


def test_good_ranges_count_nothing(epxc):  # noqa: F811
    assert run(epxc, [0, 7, 7, 40], [7, 0, 33, 24], 64, (0, 1, 2, 3)) == 0


def test_bad_ranges_are_skipped_and_counted(epxc):  # noqa: F811
    assert run(epxc, [0, -1, 60, 20], [10, 5, 5, 8], 64, (0, 3)) > 0


def test_whole_layer_without_violations(epxc):  # noqa: F811
    from tests.test_layer_gpu import Layer
    epxc.epx_checked_violations()
    lay = Layer(epxc, 128, 16, 4, 264, 136, seed=3)
    lay.forward()
    lay.backward()
    torch.cuda.synchronize()
    assert epxc.epx_checked_violations() == 0
