"""The workspace of a linear call: one for some rows serves fewer, whichever way each of them runs (no GPU)."""
import pytest

from int4_group_affine_b200 import (MoeError, QTensor, moe_affine_linear, moe_affine_linear_dx,
                                    moe_affine_linear_dx_workspace_bytes, moe_affine_linear_workspace_bytes)

A, B, C, D, S, WS = (0x10000000 * i for i in (1, 2, 3, 4, 5, 6))  # aligned addresses that nothing reads


@pytest.fixture(scope="module", autouse=True)
def built():
    from int4_group_affine_b200 import build
    build.build()


def _w(N, K, bits=4, group=64):
    q = QTensor()
    q.packed, q.scales, q.biases, q.n, q.out, q.in_, q.bits, q.group = A, B, C, 1, N, K, bits, group
    return q


@pytest.mark.parametrize("K", [2048, 2880, 4096, 5120, 8192, 16384, 65536])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32)])
def test_sizes_never_fall_for_narrow_matrices(K, bits, group):
    """Few outputs: from some number of rows on the codes are the faster way again, and the largest workspace that fewer
    rows needed is still asked for."""
    for N in list(range(1, 65)) + [100]:
        W, top = _w(N, K, bits, group), 0
        for T in list(range(0, 16386, 41)) + [16384, 16385, 17000]:
            size = moe_affine_linear_workspace_bytes(W, T)
            assert size >= top, (N, K, T, size, top)
            top = size


@pytest.mark.parametrize("N", [64, 1000, 4099, 131072])
@pytest.mark.parametrize("K", [32, 96, 128, 512, 2048])
def test_input_gradient_sizes_never_fall(N, K):
    top = 0
    for T in list(range(0, 5000, 17)) + [16384, 16385, 100000]:
        size = moe_affine_linear_dx_workspace_bytes(_w(N, K, 4, 32), T)
        assert size >= top, (N, K, T, size, top)
        top = size


@pytest.mark.parametrize("N,K", [(16, 2048), (4, 8192), (1, 8192), (15, 5120), (300, 256)])
def test_a_workspace_for_many_rows_is_taken_by_fewer(N, K):
    """What the size function says for T is enough for every call of fewer rows.  The calls are stopped by a missing y,
    which is looked at after the workspace."""
    W = _w(N, K)
    for f, size in ((moe_affine_linear, moe_affine_linear_workspace_bytes),
                    (moe_affine_linear_dx, moe_affine_linear_dx_workspace_bytes)):
        for most in (17, 300, 1797, 3073, 12600, 17000):
            nb = size(W, most)
            for T in range(1, most + 1, 61):
                with pytest.raises(MoeError) as e:
                    f(W, S, T, None, WS, nb, stream=0)
                assert e.value.status == 1, (T, most)
            with pytest.raises(MoeError) as e:
                f(W, S, most, D, WS, 255, stream=0)
            assert e.value.status == 4
