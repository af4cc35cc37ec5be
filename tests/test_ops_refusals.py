"""What the linear, grouped and SwiGLU entry points refuse, on the host and before anything is enqueued (no GPU)."""
import pytest

from int4_group_affine_b200 import (MoeError, QTensor, moe_affine_linear, moe_affine_linear_dx,
                                    moe_affine_linear_dx_workspace_bytes, moe_affine_linear_workspace_bytes,
                                    moe_grouped_matmul, moe_grouped_matmul_dw, moe_grouped_matmul_dx, moe_swiglu,
                                    moe_swiglu_grad)

A, B, C, D, S = (0x10000000 * i for i in (1, 2, 3, 4, 5))  # aligned addresses that nothing reads


@pytest.fixture(scope="module", autouse=True)
def built():
    from int4_group_affine_b200 import build
    build.build()


def _status(f, *args):
    with pytest.raises(MoeError) as e:
        f(*args, stream=0)
    return e.value.status


def _w(**kw):
    q = QTensor()
    v = dict(packed=A, scales=B, biases=C, n=1, out=100, in_=256, bits=4, group=64)
    v.update(kw)
    for k, x in v.items():
        setattr(q, k, x)
    return q


@pytest.mark.parametrize("change,status", [
    (dict(packed=None), 1), (dict(scales=None), 1), (dict(biases=None), 1), (dict(packed=A + 8), 1), (dict(n=2), 1),
    (dict(out=0), 1), (dict(in_=0), 1), (dict(in_=250), 1), (dict(bits=2), 1), (dict(group=48), 1), (dict(group=0), 1),
    (dict(group=512), 1), (dict(in_=65536 + 64), 2), (dict(out=(1 << 24) + 1), 2)])
def test_linear_refuses_a_matrix(change, status):
    for f, size in ((moe_affine_linear, moe_affine_linear_workspace_bytes),
                    (moe_affine_linear_dx, moe_affine_linear_dx_workspace_bytes)):
        assert _status(f, _w(**change), S, 4, D, 0x60000000, 1 << 40) == status
        assert size(_w(**change), 4) == 0


def test_linear_refuses_arguments():
    w = _w()
    for f, size in ((moe_affine_linear, moe_affine_linear_workspace_bytes),
                    (moe_affine_linear_dx, moe_affine_linear_dx_workspace_bytes)):
        need = size(w, 4)
        assert need >= 256 and need % 256 == 0 and size(w, -1) == 0
        assert size(w, 1 << 26) > 0 and size(w, (1 << 26) + 1) == 0
        assert _status(f, w, S, (1 << 26) + 1, D, 0x60000000, 1 << 60) == 2
        assert _status(f, w, S, 2 ** 31 - 1, D, 0x60000000, 1 << 60) == 2
        ws = 0x60000000
        assert _status(f, w, S, -1, D, ws, need) == 1
        assert _status(f, w, None, 4, D, ws, need) == 1
        assert _status(f, w, S, 4, None, ws, need) == 1
        assert _status(f, w, S, 4, S, ws, need) == 1
        assert _status(f, w, S, 4, D, None, need) == 4
        assert _status(f, w, S, 4, D, ws + 16, need) == 4
        assert _status(f, w, S, 4, D, ws, need - 1) == 4
        f(w, S, 0, D, ws, need, stream=0)  # no rows: nothing is enqueued
    assert _status(moe_affine_linear, w, S + 2, 4, D, 0x60000000, 1 << 30) == 1     # x on 16 bytes
    assert _status(moe_affine_linear_dx, w, S, 4, D + 2, 0x60000000, 1 << 30) == 1  # dx on 16 bytes


@pytest.mark.parametrize("N,K", [(100, 8192), (384, 4096), (4096, 2048), (1003, 256), (131072, 64), (3001, 1024),
                                 (1 << 20, 2048), (1 << 22, 64)])
def test_linear_workspace_for_some_rows_serves_fewer(N, K):
    for f in (moe_affine_linear_workspace_bytes, moe_affine_linear_dx_workspace_bytes):
        sizes = [f(_w(out=N, in_=K), T) for T in list(range(0, 1100, 7)) + [1500, 2048, 5000]]
        assert sizes == sorted(sizes), (N, K)


def _parts(T, J, terms, at_once=74):
    """fp32 values of a split sum's parts on a 148-multiprocessor device: as many parts as there are pairs of
    multiprocessors to a tile of 256 x 256, of at least four steps of 64 terms each."""
    tiles, steps = -(-J // 256) * -(-T // 256), -(-terms // 64)
    want = max(1, min(at_once // tiles, steps // 4))
    per = -(-steps // want) * 64
    splits = -(-terms // per)
    return splits * T * J if splits > 1 else 0


@pytest.mark.parametrize("T", [1, 50, 255, 256, 257, 500, 513, 1000, 3000])
@pytest.mark.parametrize("N,K", [(3001, 1024), (100001, 256), (4096, 2048), (520, 8192), (264, 320), (1 << 20, 2048), (1 << 24, 64)])
def test_linear_workspace_holds_the_parts(T, N, K):
    w = _w(out=N, in_=K)
    pitch = -(-N // 8) * 8
    need = 256 + 2 * N * K + (2 * T * pitch if pitch != N else 0) + 4 * _parts(T, K, N)
    assert moe_affine_linear_dx_workspace_bytes(w, T) >= need
    if moe_affine_linear_workspace_bytes(w, T) > 256:  # (few rows go by the codes)
        assert moe_affine_linear_workspace_bytes(w, T) >= 256 + 2 * N * K + 4 * _parts(T, N, K)


GOOD = dict(dtype=0, a=A, off=B, w=C, M=10, G=3, N=16, K=32, out=D, st=S)
BAD = [(dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(dtype=2), 2), (dict(a=None), 1), (dict(w=None), 1),
       (dict(out=None), 1), (dict(st=None), 1), (dict(off=None), 1), (dict(M=-1), 1), (dict(G=0), 1), (dict(N=0), 1),
       (dict(K=0), 1), (dict(G=16385), 2), (dict(N=65537), 2), (dict(K=65537), 2), (dict(a=A + 1), 1),
       (dict(M=(1 << 26) + 1), 2), (dict(M=2 ** 31 - 1), 2),
       (dict(w=C + 1), 1), (dict(out=D + 1), 1), (dict(off=B + 2), 1), (dict(st=S + 2), 1), (dict(out=A), 1),
       (dict(out=C), 1)]


@pytest.mark.parametrize("change,status", BAD)
def test_grouped_refuses(change, status):
    v = dict(GOOD, **change)
    size = (v["M"], v["G"], v["N"], v["K"])
    for f in (moe_grouped_matmul, moe_grouped_matmul_dx):
        assert _status(f, v["dtype"], v["a"], v["off"], v["w"], *size, v["out"], v["st"]) == status
    out_dtype = v["dtype"] if v["dtype"] in (0, 1) else 0
    assert _status(moe_grouped_matmul_dw, v["dtype"], v["a"], v["w"], v["off"], *size, out_dtype, 0, v["out"],
                   v["st"]) == status


def test_grouped_weight_gradient_refuses_its_own():
    size = (10, 3, 16, 32)
    assert _status(moe_grouped_matmul_dw, 0, A, C, B, *size, 1, 0, D, S) == 1      # fp16 output of bf16 rows
    assert _status(moe_grouped_matmul_dw, 0, A, C, B, *size, 0, 2, D, S) == 1      # accumulate is 0 or 1
    assert _status(moe_grouped_matmul_dw, 0, A, C, B, *size, 2, 0, D + 2, S) == 1  # fp32 output on 4 bytes


def test_no_rows_is_a_no_op():
    for f in (moe_grouped_matmul, moe_grouped_matmul_dx):
        f(0, None, B, None, 0, 3, 16, 32, None, S, stream=0)
    moe_grouped_matmul_dw(0, None, None, B, 0, 3, 16, 32, 0, 1, D, S, stream=0)
    moe_swiglu(0, None, None, None, 0, 0, 16, None, stream=0)
    moe_swiglu_grad(0, None, None, None, None, 0, 0, 16, None, None, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), 1), (dict(dtype=2), 2), (dict(gu=None), 1), (dict(M=-1), 1), (dict(I=0), 1), (dict(I=65537), 2),
    (dict(M=(1 << 26) + 1), 2), (dict(M=2 ** 31 - 1), 2), (dict(G=0), 1), (dict(G=16385), 2), (dict(w=B + 2), 1), (dict(off=C + 2), 1), (dict(gu=A + 1), 1),
    (dict(out=None), 1), (dict(out=A), 1), (dict(out=D + 1), 1)])
def test_swiglu_refuses(change, status):
    v = dict(dtype=0, gu=A, w=B, off=C, G=3, M=10, I=16, out=D)
    v.update(change)
    assert _status(moe_swiglu, v["dtype"], v["gu"], v["w"], v["off"], v["G"], v["M"], v["I"], v["out"]) == status
    assert _status(moe_swiglu_grad, v["dtype"], v["gu"], v["w"], S, v["off"], v["G"], v["M"], v["I"], v["out"],
                   None) == status


def test_swiglu_grad_refuses_its_own():
    assert _status(moe_swiglu_grad, 0, A, B, None, C, 3, 10, 16, D, None) == 1  # no dh
    assert _status(moe_swiglu_grad, 0, A, B, S, C, 3, 10, 16, S, None) == 1     # dgu on dh
    assert _status(moe_swiglu_grad, 0, A, B, S, C, 3, 10, 16, D, B) == 1        # dw on w


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The binding takes contiguous tensors of the current device only (stand-in tensors: no GPU is needed)."""
    import int4_group_affine_b200 as m

    class Tensor:
        def __init__(self, device, contiguous=True):
            self.device, self.contiguous = device, contiguous

        def get_device(self):
            return self.device

        def is_contiguous(self):
            return self.contiguous

        def data_ptr(self):
            return A

    monkeypatch.setattr(m, "_device", lambda: 0)
    for bad, why in ((Tensor(1), "cuda:1"), (Tensor(-1), "CUDA"), (Tensor(0, False), "contiguous")):
        with pytest.raises(ValueError, match=why):
            moe_swiglu(0, bad, None, None, 0, 4, 16, D, stream=0)
        with pytest.raises(ValueError, match=why):
            moe_swiglu(0, Tensor(0), bad, None, 0, 4, 16, D, stream=0)
