"""scaled_gemm_norm_quantize without a GPU: bad arguments are refused on the host."""
import pytest

from fp8_scaled_gemm_sm_gb300 import binding, build

A = 1 << 20  # addresses that nothing looks at


@pytest.fixture(scope="module")
def call():
    build.build()
    L = binding.lib()

    def call(mode=1, dt=0, x=A, res=2 * A, kept=3 * A, w=4 * A, eps=1e-6, R=4, C=256, q=5 * A, scale=6 * A):
        return L.scaled_gemm_norm_quantize(mode, dt, x, res, kept, w, eps, R, C, q, scale, None)

    return call


@pytest.mark.parametrize("bad,status", [
    (dict(mode=4), 1), (dict(mode=-1), 1), (dict(dt=2), 1), (dict(R=-1), 1), (dict(C=-16), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=2.0 ** 61), 1), (dict(C=32784), 2), (dict(C=264), 2), (dict(mode=0, C=260), 2), (dict(mode=2, C=192), 2), (dict(mode=3, C=48), 2), (dict(R=1 << 31), 2),
    (dict(x=None), 1), (dict(w=None), 1), (dict(q=None), 1), (dict(scale=None), 1), (dict(kept=None), 1),
    (dict(x=A + 8), 3), (dict(res=2 * A + 4), 3), (dict(kept=3 * A + 2), 3), (dict(w=4 * A + 8), 3), (dict(q=5 * A + 8), 3), (dict(scale=6 * A + 4), 3),
    (dict(kept=A + 512), 1), (dict(kept=2 * A + 512), 1), (dict(kept=4 * A), 1), (dict(q=A), 1), (dict(q=3 * A), 1), (dict(scale=5 * A), 1),
    (dict(scale=4 * A), 1), (dict(mode=0, dt=1, q=A), 1),
])
def test_refusals(call, bad, status):
    assert call(**bad) == status


def test_nothing_to_do(call):
    assert call(R=0) == 0 and call(C=0) == 0


def test_rows_counted_in_32_bits(call):
    far = 1 << 50  # buffers of that many rows do not overlap
    assert call(mode=0, R=(1 << 31) - 1, C=8, x=far, res=None, kept=None, w=2 * far, q=3 * far, scale=None) == 2
