"""The linear, grouped and SwiGLU operators where element offsets of matrices, results and activations pass 32 bits, and
at the limits of their sizes.  Whole numbers: the sums are exact, and the results have to be theirs, rounded once."""
import pytest

from tests.gpu_helpers import need_cuda
from tests.op_helpers import HALF, assert_within, packed, qtensor, swiglu_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    need_cuda()
    yield
    torch.cuda.empty_cache()


def _m():
    import int4_group_affine_b200 as m
    return m


def _whole(g, *shape):
    v = torch.empty(shape, dtype=torch.int8, device="cuda").random_(-2, 3, generator=g)
    return v.bfloat16()


@pytest.mark.parametrize("N,K", [(1024, 2048), (1023, 2047)])
def test_matrices_past_32_bits(N, K):
    """1100 matrices of 2 M elements; rows in the first and the last groups."""
    m = _m()
    G, sizes = 1100, {0: 3, 1: 70, 1022: 1, 1025: 33, 1098: 5, 1099: 130}
    off = torch.zeros(G + 1, dtype=torch.int32)
    for e, n in sizes.items():
        off[e + 1] = n
    off = off.cumsum(0, dtype=torch.int32).cuda()
    M = sum(sizes.values())
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy, W = _whole(g, M, K), _whole(g, M, N), _whole(g, G, N, K)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    m.moe_grouped_matmul(m.DT_BF16, x, off, W, M, G, N, K, y, st)
    m.moe_grouped_matmul_dx(m.DT_BF16, dy, off, W, M, G, N, K, dx, st)
    want, at = {}, 0
    for e, n in sizes.items():
        a, b, w = x[at:at + n].double(), dy[at:at + n].double(), W[e].double()
        assert torch.equal(y[at:at + n], (a @ w.t()).bfloat16()) and torch.equal(dx[at:at + n], (b @ w).bfloat16())
        want[e] = (b.t() @ a).bfloat16()
        at += n
    dw = W.fill_(7.0)
    m.moe_grouped_matmul_dw(m.DT_BF16, dy, x, off, M, G, N, K, m.DT_BF16, 0, dw, st)
    for e in range(G):
        assert torch.equal(dw[e], want[e]) if e in want else not bool(dw[e].any())
    assert int(st.item()) == 0


@pytest.mark.parametrize("T", [1, 16, 130])
def test_the_tallest_matrix(T):
    """2^24 outputs; with 130 rows the results' offsets pass 2^31."""
    m = _m()
    N, K = 1 << 24, 32
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    s = torch.randint(1, 3, (N, 1), generator=g, device="cuda").bfloat16()
    b = torch.randint(-8, 1, (N, 1), generator=g, device="cuda").bfloat16()
    q = qtensor(m, (w, s, b), N, K, 4, 32)
    x, dy1 = _whole(g, T, K), _whole(g, 2, N)
    dy1 *= (torch.rand(N, generator=g, device="cuda") < 0.01) | (torch.arange(N, device="cuda") >= N - 40)
    nb = max(m.moe_affine_linear_workspace_bytes(q, T), m.moe_affine_linear_dx_workspace_bytes(q, 2))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    m.moe_workspace_init(ws, nb)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_affine_linear(q, x, T, y, ws, nb)
    dx = torch.empty((2, K), dtype=torch.bfloat16, device="cuda")
    m.moe_affine_linear_dx(q, dy1, 2, dx, ws, nb)
    shift, ref = 4 * torch.arange(8, device="cuda", dtype=torch.int32), torch.zeros((2, K), dtype=torch.float64, device="cuda")
    for n in range(0, N, 1 << 20):
        r = slice(n, n + (1 << 20))
        mat = ((w[r][:, :, None] >> shift) & 15).reshape(-1, K).float() * s[r].float() + b[r].float()
        assert torch.equal(y[:, r], (x.float() @ mat.t()).bfloat16())  # (whole numbers below 2^24: exact in 32 bits)
        ref += dy1[:, r].double() @ mat.double()
    assert torch.equal(dx, ref.bfloat16()) and m.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("I", [65536, 65535])
def test_activations_past_32_bits(I):
    """The widest rows, 17000 of them: offsets of gate and up pass 2^31.  fp32 arithmetic before one rounding, 30 units of
    2^-24 with gates below 9 in magnitude."""
    m = _m()
    M = 17000
    g = torch.Generator(device="cuda").manual_seed(3)
    gu = torch.zeros((M, 2 * I), dtype=torch.bfloat16, device="cuda")
    rows = [0, 16383, 16384, 16385, M - 2]
    for r in rows:
        gu[r] = torch.randn(2 * I, generator=g, device="cuda").bfloat16()
    w = torch.rand(M, generator=g, device="cuda")
    off = torch.tensor([0, M - 1], dtype=torch.int32, device="cuda")
    h = torch.full((M, I), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_swiglu(m.DT_BF16, gu, w, off, 1, M, I, h)
    rel = HALF["bf16"] + 30 * 2.0 ** -24
    ref = swiglu_ref(gu[rows], w[rows])
    assert_within(h[rows], ref, rel * 1.001 * ref.abs())
    assert bool((h[M - 1] == 7.0).all()) and not bool(h[1:16383].any())
    dh = h.normal_(generator=g)
    dgu, dw = torch.full_like(gu, 7.0), torch.full((M,), 7.0, device="cuda")
    m.moe_swiglu_grad(m.DT_BF16, gu, w, dh, off, 1, M, I, dgu, dw)
    rgu, rdw, mag = swiglu_ref(gu[rows], w[rows], dh[rows])
    gate = gu[rows][:, :I].double().abs().repeat(1, 2)
    slack = (dh[rows].double().abs() * w[rows].double()[:, None]).repeat(1, 2) * 8 * (1 + gate) * 40 * 2.0 ** -24
    assert_within(dgu[rows], rgu, HALF["bf16"] * 1.001 * rgu.abs() + slack)
    assert_within(dw[rows], rdw, (30 + I / 256 + 16) * 2.0 ** -24 * mag)
    assert bool((dgu[M - 1] == 7.0).all()) and float(dw[M - 1]) == 7.0 and not bool(dgu[1:16383, :I].any())
