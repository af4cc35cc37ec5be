"""The binding of the linear, grouped and SwiGLU entry points refuses tensors that are too short for the call's sizes or of
another type than its type code, before anything is enqueued (stand-in tensors: no GPU is needed)."""
import math

import pytest

import int4_group_affine_b200 as m

torch = pytest.importorskip("torch")
A = 0x10000000
BF, HF, F32, I32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8


class Tensor:
    """A contiguous tensor of device 0 at an address of its own that nothing reads."""
    made = 0

    def __init__(self, dtype, *shape):
        Tensor.made += 1
        self.dtype, self.nbytes, self.at = dtype, math.prod(shape) * dtype.itemsize, A * (Tensor.made % 4096 + 1)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


@pytest.fixture(autouse=True)
def _here(monkeypatch):
    from int4_group_affine_b200 import build
    build.build()
    monkeypatch.setattr(m, "_device", lambda: 0)


def _w(T, N, K):
    q = m.QTensor()
    q.packed, q.scales, q.biases, q.n, q.out, q.in_, q.bits, q.group = A, 2 * A, 3 * A, 1, N, K, 4, 32
    return q


# every call with its tensors: (type, shape) in the order of the arguments, a call that takes them, and which of them may be
# given as raw bits; each call is made with one argument that the library itself refuses (a missing status, y or h, so
# nothing is enqueued) once its tensors have passed
T, M, G, N, K, I = 5, 6, 3, 40, 64, 24
CALLS = {
    "linear": ([(BF, T, K), (U8, 1 << 20)], lambda x, ws: m.moe_affine_linear(_w(T, N, K), x, T, None, ws, 1 << 20, stream=0)),
    "linear y": ([(BF, T, N)], lambda y: m.moe_affine_linear(_w(T, N, K), None, T, y, A, 1 << 20, stream=0)),
    "linear_dx": ([(BF, T, N), (U8, 1 << 20)],
                  lambda dy, ws: m.moe_affine_linear_dx(_w(T, N, K), dy, T, None, ws, 1 << 20, stream=0)),
    "linear_dx dx": ([(BF, T, K)], lambda dx: m.moe_affine_linear_dx(_w(T, N, K), None, T, dx, A, 1 << 20, stream=0)),
    "grouped": ([(BF, M, K), (I32, G + 1), (BF, G, N, K), (BF, M, N)],
                lambda x, o, w, y: m.moe_grouped_matmul(0, x, o, w, M, G, N, K, y, None, stream=0)),
    "grouped status": ([(I32, 1)], lambda st: m.moe_grouped_matmul(0, None, A, A, M, G, N, K, A, st, stream=0)),
    "grouped fp16": ([(HF, M, K), (I32, G + 1), (HF, G, N, K), (HF, M, N)],
                     lambda x, o, w, y: m.moe_grouped_matmul(1, x, o, w, M, G, N, K, y, None, stream=0)),
    "grouped_dx": ([(BF, M, N), (I32, G + 1), (BF, G, N, K), (BF, M, K)],
                   lambda dy, o, w, dx: m.moe_grouped_matmul_dx(0, dy, o, w, M, G, N, K, dx, None, stream=0)),
    "grouped_dw": ([(BF, M, N), (BF, M, K), (I32, G + 1), (F32, G, N, K)],
                   lambda dy, x, o, dw: m.moe_grouped_matmul_dw(0, dy, x, o, M, G, N, K, 2, 0, dw, None, stream=0)),
    "grouped_dw bf16": ([(BF, M, N), (BF, M, K), (I32, G + 1), (BF, G, N, K)],
                        lambda dy, x, o, dw: m.moe_grouped_matmul_dw(0, dy, x, o, M, G, N, K, 0, 1, dw, None, stream=0)),
    "swiglu": ([(BF, M, 2 * I), (F32, M), (I32, G + 1)], lambda gu, w, o: m.moe_swiglu(0, gu, w, o, G, M, I, None, stream=0)),
    "swiglu h": ([(HF, M, I)], lambda h: m.moe_swiglu(1, None, None, None, 0, M, I, h, stream=0)),
    "swiglu_grad": ([(BF, M, 2 * I), (F32, M), (BF, M, I), (I32, G + 1), (F32, M)],
                    lambda gu, w, dh, o, dw: m.moe_swiglu_grad(0, gu, w, dh, o, G, M, I, None, dw, stream=0)),
    "swiglu_grad dgu": ([(HF, M, 2 * I)], lambda dgu: m.moe_swiglu_grad(1, None, None, None, None, 0, M, I, dgu, None, stream=0)),
}


@pytest.mark.parametrize("name", CALLS)
def test_short_tensors_and_other_types_are_refused(name):
    specs, call = CALLS[name]
    make = lambda: [Tensor(t, *s) for t, *s in specs]  # noqa: E731
    with pytest.raises(m.MoeError) as e:  # right ones get as far as the library
        call(*make())
    assert e.value.status == 1
    for i, (t, *shape) in enumerate(specs):
        args = make()
        args[i].nbytes -= t.itemsize
        with pytest.raises(ValueError, match="bytes"):
            call(*args)
        args = make()
        args[i].nbytes += 1000  # (a longer one will do)
        with pytest.raises(m.MoeError):
            call(*args)
        if t is U8:
            continue
        args = make()
        args[i] = Tensor(torch.float64, *shape)
        with pytest.raises(ValueError, match="float64"):
            call(*args)
        if t in (BF, HF):
            args[i] = Tensor(HF if t is BF else BF, *shape)
            with pytest.raises(ValueError, match="float16"):
                call(*args)
            for bits in (torch.int16, torch.uint16):
                args[i] = Tensor(bits, *shape)
                with pytest.raises(m.MoeError):
                    call(*args)


def test_sizes_of_more_than_32_bits():
    """2^26 rows of 65536: the bytes are counted in whole numbers of any size."""
    x = Tensor(BF, 1 << 26, 64)
    with pytest.raises(ValueError, match="8796093022208"):
        m.moe_grouped_matmul(0, x, None, None, 1 << 26, 1, 8, 65536, None, None, stream=0)
