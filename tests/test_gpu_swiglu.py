"""GPU parity of SwiGLU on stacked rows and its gradient against 64 bits."""
import pytest

from tests.gpu_helpers import need_cuda
from tests.op_helpers import DTYPES, HALF, assert_within, swiglu_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    need_cuda()


def _m():
    import int4_group_affine_b200 as m
    return m


# fp32 arithmetic before the one rounding: the exponential (2 ulp, and 1.5 |g| units of 2^-24 for the rounding of its
# argument -|g| log2 e and of log2 e), sigmoid's addition and division, up to five products and 1 + g (1 - s), whose
# two terms can cancel (|1 + g (1 - s)| against 1 + |g| (1 - s)): 16 + 1.5 |g| units of 2^-24 of the terms'
# magnitudes bound them.
def _rel(gu):
    g = gu[:, :gu.shape[1] // 2].double().abs().nan_to_num()
    return (16 + 1.5 * g) * 2.0 ** -24


def _data(seed, M, I, dtype, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gu = (torch.randn((M, 2 * I), generator=g, device="cuda") * scale).to(DTYPES[dtype])
    dh = torch.randn((M, I), generator=g, device="cuda").to(DTYPES[dtype])
    return gu, torch.rand(M, generator=g, device="cuda"), dh


def _terms(gu, w, dh):
    """Magnitudes of dgu's terms before they cancel."""
    I = gu.shape[1] // 2
    g, u, d = gu[:, :I].double(), gu[:, I:].double(), dh.double()
    w = torch.ones(len(gu), dtype=torch.float64, device=gu.device) if w is None else w.double()
    s = torch.sigmoid(g)
    return torch.cat([(w[:, None] * d * u).abs() * s * (1 + g.abs() * (1 - s)), (w[:, None] * d * g).abs() * s], 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,I,off,weights", [
    (1, 1, None, True), (3, 7, None, False), (5, 8, [1, 2, 4], True), (64, 512, [0, 64], True), (33, 100, [3, 30], True),
    (17, 1001, None, True), (9, 2048, [0, 0], True), (2, 4104, None, True), (700, 16, [5, 100, 690], False)])
def test_forward_and_gradient(dtype, M, I, off, weights):
    m = _m()
    gu, w, dh = _data(M + I, M, I, dtype)
    w = w if weights else None
    code = m.DT_BF16 if dtype == "bf16" else m.DT_F16
    od, G = (None, 0) if off is None else (torch.tensor(off, dtype=torch.int32, device="cuda"), len(off) - 1)
    r = slice(0, M) if off is None else slice(off[0], off[-1])
    out = [slice(0, r.start), slice(r.stop, M)]
    if off is not None:  # rows of no group are not read
        for o in out:
            gu[o], dh[o] = float("nan"), float("nan")
    tiny = 2.0 ** -24 if dtype == "fp16" else 0.0  # half a step of the smallest fp16 values

    h = torch.full((M, I), 7.0, dtype=DTYPES[dtype], device="cuda")
    m.moe_swiglu(code, gu, w, od, G, M, I, h)
    ref = swiglu_ref(gu, w)
    assert_within(h[r], ref[r], (HALF[dtype] + _rel(gu)[r]) * 1.001 * ref[r].abs() + tiny, "h")
    assert all(bool((h[o] == 7.0).all()) for o in out)

    dgu = torch.full((M, 2 * I), 7.0, dtype=DTYPES[dtype], device="cuda")
    dw = torch.full((M,), 7.0, dtype=torch.float32, device="cuda")
    m.moe_swiglu_grad(code, gu, w, dh, od, G, M, I, dgu, dw)
    rgu, rdw, mag = swiglu_ref(gu, w, dh)
    assert_within(dgu[r], rgu[r], HALF[dtype] * 1.001 * rgu[r].abs() + _rel(gu).repeat(1, 2)[r] * _terms(gu, w, dh)[r] + tiny, "dgu")
    assert_within(dw[r], rdw[r], ((_rel(gu).max() if len(gu) else 0) + (I / 32 + 16) * 2.0 ** -24) * mag[r], "dw")
    assert all(bool((dgu[o] == 7.0).all()) and bool((dw[o] == 7.0).all()) for o in out)

    same = torch.full_like(dgu, 7.0)
    m.moe_swiglu_grad(code, gu, w, dh, od, G, M, I, same, None)  # dw not wanted
    torch.cuda.synchronize()
    assert torch.equal(same, dgu)


def test_extremes():
    """Saturated gates: silu(g) is g or 0, its slope 1 or 0; no overflow of the exponential shows."""
    m = _m()
    g = torch.tensor([[-120.0, 120.0, -3e4, 3e4, 0.0, -0.0, 88.5, -88.5]], device="cuda")
    gu = torch.cat([g, torch.full_like(g, 2.0)], 1).bfloat16()
    dh = torch.ones((1, 8), dtype=torch.bfloat16, device="cuda")
    h = torch.empty((1, 8), dtype=torch.bfloat16, device="cuda")
    dgu = torch.empty((1, 16), dtype=torch.bfloat16, device="cuda")
    m.moe_swiglu(m.DT_BF16, gu, None, None, 0, 1, 8, h)
    m.moe_swiglu_grad(m.DT_BF16, gu, None, dh, None, 0, 1, 8, dgu, None)
    torch.cuda.synchronize()
    ref = swiglu_ref(gu, None)
    rgu = swiglu_ref(gu, None, dh)[0]
    # below fp32's smallest normal value results may be flushed
    assert_within(h, ref, 1.01 * HALF["bf16"] * ref.abs() + 2.0 ** -125)
    assert_within(dgu, rgu, 1.01 * HALF["bf16"] * rgu.abs() + 200 * 2.0 ** -126)


def test_gradient_against_differences():
    """Central differences of the 64-bit form in a random direction against the kernel's gradients: the third
    derivative of silu is below 0.7, so a step of 1e-4 leaves under 1e-8 of the direction's cube."""
    m = _m()
    M, I, e = 6, 40, 1e-4
    gu, w, dh = _data(3, M, I, "fp16", 1.0)
    dgu = torch.empty((M, 2 * I), dtype=torch.float16, device="cuda")
    dw = torch.empty(M, dtype=torch.float32, device="cuda")
    m.moe_swiglu_grad(m.DT_F16, gu, w, dh, None, 0, M, I, dgu, dw)
    gen = torch.Generator(device="cuda").manual_seed(4)
    v = torch.randn((M, 2 * I), generator=gen, device="cuda").double()
    vw = torch.randn(M, generator=gen, device="cuda").double()
    f = lambda t: (swiglu_ref(gu.double() + t * v, w.double() + t * vw) * dh.double()).sum(1)  # noqa: E731
    by_diff = (f(e) - f(-e)) / (2 * e)
    by_grad = (dgu.double() * v).sum(1) + dw.double() * vw
    tol = 1.1 * HALF["fp16"] * (dgu.double() * v).abs().sum(1) + 1e-6 * (1 + (v.abs() ** 3).sum(1) * 10)
    assert_within(by_grad, by_diff, tol)
