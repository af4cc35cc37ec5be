"""GPU parity of the linear layers in the affine format, forward and input gradient, against 64 bits."""
import pytest

from tests.gpu_helpers import need_cuda
from tests.op_helpers import HALF, assert_within, packed, qtensor, sum_err

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    need_cuda()


def _m():
    import int4_group_affine_b200 as m
    return m


def _ws(m, nb):
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    m.moe_workspace_init(ws, nb)
    return ws


def _rows(seed, T, n):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, n), generator=g, device="cuda").bfloat16()


def _forward_tol(x, s, q, b, bits, group):
    """The larger of the two ways a call may run.  Whole codes: the products' magnitudes with the largest code (what x
    loses as fp16, 2^-35 of a unit's largest value a term, is far below these), one rounding per group and term.  The
    matrix in bf16: half a step of every weight."""
    xa, K = x.double().abs(), x.shape[1]
    code = 2 ** bits - 1
    whole = xa @ (s * code + b.abs()).t()
    w = s * q + b
    tol_codes = sum_err(K + 16 * (K // group) + 128, whole)
    tol_matrix = HALF["bf16"] * (xa @ w.abs().t()) + sum_err(K, xa @ w.abs().t())
    return torch.maximum(tol_codes, tol_matrix), w


# (T, N, K, bits, group): single tokens, every token count around the row tiles, odd outputs, group counts that no
# vector of four divides, one group, groups of 96 and 128, the largest inputs
CASES = [(1, 512, 2048, 4, 64), (1, 1, 32, 4, 32), (1, 17, 64, 4, 64), (2, 31, 96, 4, 32), (3, 100, 192, 4, 96),
         (5, 33, 128, 8, 64), (7, 64, 320, 4, 64), (8, 130, 2048, 4, 32), (9, 65, 1056, 8, 32), (13, 1003, 1056, 8, 32),
         (16, 48, 384, 4, 128), (17, 257, 512, 4, 64), (33, 128, 256, 4, 32), (64, 96, 640, 8, 64),
         (65, 72, 448, 4, 64), (100, 51, 96, 4, 32), (129, 136, 1024, 4, 64), (300, 264, 576, 8, 32),
         (1, 40, 65536, 4, 64), (3, 24, 32768, 8, 64), (2, 24, 65536, 8, 64), (5, 19, 65536, 8, 32), (17, 16, 8192, 4, 64), (2, 4099, 256, 4, 64),
         (200, 100, 8192, 4, 64), (150, 40, 65536, 4, 64), (256, 384, 4096, 8, 32), (257, 300, 2304, 4, 128),
         (16384, 3, 32, 4, 32), (70001, 1, 64, 8, 64)]


@pytest.mark.parametrize("T,N,K,bits,group", CASES)
def test_forward(T, N, K, bits, group):
    m = _m()
    t, (s, q, b) = packed(T + N, N, K, bits, group)
    W = qtensor(m, t, N, K, bits, group)
    x = _rows(K, T, K)
    nb = m.moe_affine_linear_workspace_bytes(W, T)
    ws = _ws(m, nb)
    y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_affine_linear(W, x, T, y, ws, nb)
    torch.cuda.synchronize()
    tol, w = _forward_tol(x, s, q, b, bits, group)
    ref = x.double() @ w.t()
    assert_within(y[:T], ref, HALF["bf16"] * ref.abs() + 1.01 * tol)
    assert bool((y[T] == 7.0).all()) and m.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("T,N,K,bits,group", [(1, 512, 256, 4, 64), (3, 17, 64, 4, 32), (70, 136, 320, 8, 64),
                                              (129, 1000, 96, 4, 32), (40, 1003, 128, 4, 64), (257, 264, 2048, 4, 64),
                                              (50, 30011, 128, 4, 64), (300, 5000, 64, 8, 32), (1, 4099, 320, 4, 32),
                                              (500, 3001, 1024, 4, 64)])
def test_input_gradient(T, N, K, bits, group):
    m = _m()
    t, (s, q, b) = packed(T + N, N, K, bits, group)
    W = qtensor(m, t, N, K, bits, group)
    dy = _rows(K, T, N)
    nb = m.moe_affine_linear_dx_workspace_bytes(W, T)
    ws = _ws(m, nb)
    dx = torch.full((T + 1, K), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_affine_linear_dx(W, dy, T, dx, ws, nb)
    torch.cuda.synchronize()
    w = s * q + b
    ref, mag = dy.double() @ w, dy.double().abs() @ w.abs()
    assert_within(dx[:T], ref, HALF["bf16"] * ref.abs() + 1.01 * (HALF["bf16"] * mag + sum_err(N, mag)))
    assert bool((dx[T] == 7.0).all()) and m.moe_get_device_status(ws) == 0


def test_input_gradient_against_differences():
    """<dy, y(v)> = <dx, v> for the linear map, up to the roundings of y, of dx and of the bf16 matrix."""
    m = _m()
    T, N, K = 40, 72, 128
    t, (s, q, b) = packed(5, N, K, 4, 64)
    W = qtensor(m, t, N, K, 4, 64)
    v, dy = _rows(1, T, K), _rows(2, T, N)
    nb = max(m.moe_affine_linear_workspace_bytes(W, T), m.moe_affine_linear_dx_workspace_bytes(W, T))
    ws = _ws(m, nb)
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    dx = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    m.moe_affine_linear(W, v, T, y, ws, nb)
    m.moe_affine_linear_dx(W, dy, T, dx, ws, nb)
    torch.cuda.synchronize()
    a, c = float((dy.double() * y.double()).sum()), float((dx.double() * v.double()).sum())
    mag = float((dy.double().abs() @ (s * q + b).abs() * v.double().abs()).sum())
    assert abs(a - c) <= mag * 4.1 * HALF["bf16"]  # y, dx and the matrix on either side: one half step each


def test_one_token_of_many_is_that_token():
    """The rows of a batch do not touch each other: a NaN token leaves the others finite and unchanged."""
    m = _m()
    N, K = 72, 256
    t, _ = packed(6, N, K, 4, 64)
    W = qtensor(m, t, N, K, 4, 64)
    for T in (2, 9, 20, 140):
        nb = m.moe_affine_linear_workspace_bytes(W, T)
        ws = _ws(m, nb)
        x = _rows(3, T, K)
        y0 = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        y1 = torch.empty_like(y0)
        m.moe_affine_linear(W, x, T, y0, ws, nb)
        x[1] = float("nan")
        m.moe_affine_linear(W, x, T, y1, ws, nb)
        torch.cuda.synchronize()
        keep = torch.arange(T, device="cuda") != 1
        assert torch.equal(y0[keep], y1[keep]) and bool(y1[1].isnan().all())


def test_graph_and_stream():
    """Captured on a side stream and replayed on new inputs; the largest and the smallest T share a workspace."""
    m = _m()
    N, K = 264, 512
    t, (s, q, b) = packed(7, N, K, 4, 64)
    W = qtensor(m, t, N, K, 4, 64)
    nb = m.moe_affine_linear_workspace_bytes(W, 300)
    ws = _ws(m, nb)
    x1, x2 = _rows(4, 1, K), _rows(5, 300, K)
    y1 = torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    y2 = torch.empty((300, N), dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            m.moe_affine_linear(W, x1, 1, y1, ws, nb)
            m.moe_affine_linear(W, x2, 300, y2, ws, nb)
        x1.copy_(_rows(6, 1, K))
        x2.copy_(_rows(7, 300, K))
        gr.replay()
        gr.replay()
    torch.cuda.synchronize()
    for x, y in ((x1, y1), (x2, y2)):
        tol, w = _forward_tol(x, s, q, b, 4, 64)
        ref = x.double() @ w.t()
        assert_within(y, ref, HALF["bf16"] * ref.abs() + 1.01 * tol)
    assert m.moe_get_device_status(ws) == 0


def test_input_gradient_through_a_million_outputs():
    """All products positive and every weight a bf16 number, so that only the sums err: parts of up to 8192 terms by
    sum_err's 1.3e-4 of the result, the fp32 additions of 128 of them by 128 / 2 roundings, 4e-6, then half a bf16 step.
    (4.9e-4 covers them; in one part a sum so long would be off by more.)"""
    m = _m()
    N, K, T = 1 << 20, 64, 3
    g = torch.Generator(device="cuda").manual_seed(6)
    w = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, K // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    s, b = (torch.full((N, K // 32), v, device="cuda", dtype=torch.bfloat16) for v in (2.0 ** -4, 1.0))
    dy = (0.5 + torch.rand((T, N), generator=g, device="cuda")).bfloat16()
    dx = torch.empty((T, K), device="cuda", dtype=torch.bfloat16)
    q = qtensor(m, (w, s, b), N, K, 4, 32)
    nb = m.moe_affine_linear_dx_workspace_bytes(q, T)
    ws = _ws(m, nb)
    m.moe_affine_linear_dx(q, dy, T, dx, ws, nb)
    codes = (w[:, :, None] >> (4 * torch.arange(8, device="cuda", dtype=torch.int32))) & 15
    ref = dy.double() @ (codes.reshape(N, K).double() / 16 + 1)
    assert m.moe_get_device_status(ws) == 0
    step = torch.exp2(torch.floor(torch.log2(ref))) * 2.0 ** -7
    assert_within(dx, ref, step / 2 + (4.9e-4 + 16 * 2.0 ** -23) * ref, "dx of many outputs")


@pytest.mark.parametrize("bits,group", [(4, 32), (4, 64), (8, 64)])
def test_rows_and_terms_of_very_different_magnitudes(bits, group):
    """Tokens from 2^-120 to 2^120 and terms up to 2^40 apart within a row, beside zeros and subnormals; half a step of
    the smallest bf16 numbers is 2^-134."""
    m = _m()
    T, N, K = 9, 70, 512
    t, (s, q, b) = packed(8, N, K, bits, group)
    W = qtensor(m, t, N, K, bits, group)
    g = torch.Generator(device="cuda").manual_seed(9)
    p = torch.randint(-40, 1, (T, K), generator=g, device="cuda") + torch.arange(T, device="cuda")[:, None] * 30 - 120
    x = (_rows(9, T, K).double() * torch.exp2(p.double())).bfloat16()
    x[3] = 0
    x[4, :group] = 0
    x[0, ::7] = 2.0 ** -130
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    nb = m.moe_affine_linear_workspace_bytes(W, T)
    m.moe_affine_linear(W, x, T, y, _ws(m, nb), nb)
    tol, w = _forward_tol(x, s, q, b, bits, group)
    ref = x.double() @ w.t()
    assert_within(y, ref, HALF["bf16"] * ref.abs() + 1.01 * tol + 2.0 ** -134, "magnitudes")
    assert bool((y[3] == 0).all())


@pytest.mark.parametrize("T,N,K,bits,group", [(1, 100, 1024, 4, 64), (9, 4800, 512, 8, 64), (2, 5000, 1024, 4, 256)])
def test_scales_and_biases_at_any_address(T, N, K, bits, group):
    """Scales and biases that start on an odd 16-bit element give the same bits as aligned ones."""
    m = _m()
    t, _ = packed(10, N, K, bits, group)
    x, out = _rows(11, T, K), []
    for shift in (0, 1):
        moved = []
        for v in t[1:]:
            room = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")
            room[shift:shift + v.numel()] = v.flatten()
            moved.append(room[shift:])
        W = qtensor(m, (t[0], *moved), N, K, bits, group)
        nb = m.moe_affine_linear_workspace_bytes(W, T)
        y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        m.moe_affine_linear(W, x, T, y, _ws(m, nb), nb)
        out.append(y)
    assert torch.equal(*out)
