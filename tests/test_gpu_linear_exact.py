"""The linear layers on inputs whose sums are exact, and within bounds made for the way each call runs.

Exact: the rows hold 0, 1 and -1, the scales are 1/2 or 1 and the biases whole numbers, so every product is a multiple of
1/2 and every partial sum below 2^14 * 264, 2^14 * 528 < 2^24 such steps (a row has at most 2^14 terms that are not zero).
No fp32 addition rounds or truncates then, whatever its order, and the result has to be the exact sum rounded to bf16: one
lost or doubled term that shows in 8 bits is found.  Sparse rows, with terms at the start, at the end and in between, keep
most sums small enough to be bf16 numbers themselves.

A call runs over the whole codes where its workspace holds the status word alone (256 bytes), else over the matrix, each
weight of it rounded to bf16 once; the reference takes the same operands."""
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


def _whole_matrix(seed, N, K, bits, group):
    """Random codes, scales 1/2 or 1, biases -8 .. 8, and the matrix in 64 bits."""
    (words, s, b), (_, q, _) = packed(seed, N, K, bits, group)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    s = (torch.randint(1, 3, s.shape, generator=g, device="cuda") * 0.5).bfloat16()
    b = torch.randint(-8, 9, b.shape, generator=g, device="cuda").bfloat16()
    rep = lambda v: v.double().repeat_interleave(group, 1)  # noqa: E731
    return (words, s, b), rep(s) * q + rep(b)


def _sparse(seed, T, n, most=1 << 14):
    """Rows of 0, 1 and -1: row by row a dense one (of at most `most` terms), one of some 16 terms anywhere, one of the
    last terms alone and one of the first."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randint(0, 2, (T, n), generator=g, device="cuda") * 2 - 1).float()
    t = torch.arange(T, device="cuda")[:, None]
    k = torch.arange(n, device="cuda")[None]
    rare = torch.rand((T, n), generator=g, device="cuda") < min(1.0, 16 / n)
    keep = torch.where(t % 4 == 0, rare | (k >= n - 5), torch.where(t % 4 == 1, k < most, torch.where(
        t % 4 == 2, k >= n - 1 - t % 7, k <= t % 9)))
    return (x * keep).bfloat16()


# (T, N, K, bits, group): both ways through a forward, the lengths at which units, quads, steps, padding and split sums end
FORWARD = [(1, 512, 2048, 4, 64), (1, 1, 32, 4, 32), (1, 17, 64, 4, 64), (2, 31, 96, 4, 32), (3, 100, 192, 4, 96),
           (5, 33, 128, 8, 64), (7, 64, 320, 4, 64), (8, 130, 2048, 4, 32), (13, 1003, 1056, 8, 32), (16, 48, 384, 4, 128),
           (17, 257, 512, 4, 64), (33, 128, 256, 4, 32), (64, 104, 640, 8, 64), (65, 136, 448, 4, 64), (129, 136, 1024, 4, 64),
           (300, 264, 576, 8, 32), (1, 40, 65536, 4, 64), (3, 24, 32768, 8, 64), (4, 24, 65536, 8, 64), (5, 19, 65536, 8, 32),
           (4, 40, 65504, 4, 32), (4, 24, 32736, 8, 32), (17, 128, 8192, 4, 64), (4, 4099, 256, 4, 64), (200, 100, 8192, 4, 64),
           (150, 104, 65536, 4, 64), (256, 384, 4096, 8, 32), (257, 300, 2304, 4, 128), (16384, 3, 32, 4, 32), (20001, 8, 64, 8, 64),
           (4, 20000, 2880, 4, 96), (9, 10000, 352, 8, 32)]


def _forward(m, t, N, K, bits, group, x):
    T = len(x)
    W = qtensor(m, t, N, K, bits, group)
    nb = m.moe_affine_linear_workspace_bytes(W, T)
    ws = _ws(m, nb)
    y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_affine_linear(W, x, T, y, ws, nb)
    torch.cuda.synchronize()
    assert bool((y[T] == 7.0).all()) and m.moe_get_device_status(ws) == 0
    return y[:T], nb > 256


@pytest.mark.parametrize("T,N,K,bits,group", FORWARD)
def test_forward_of_whole_numbers(T, N, K, bits, group):
    t, w = _whole_matrix(T + N, N, K, bits, group)
    x = _sparse(K, T, K)
    y, matrix = _forward(_m(), t, N, K, bits, group, x)
    if matrix:
        w = w.bfloat16().double()
    assert torch.equal(y, (x.double() @ w.t()).bfloat16())


@pytest.mark.parametrize("T,N,K,bits,group", FORWARD)
def test_forward_within_the_bound_of_its_way(T, N, K, bits, group):
    """Over the codes: a unit's tensor-core sum (64 terms at most, sum_err), the sum of its x (11 additions), two fused
    multiply-adds a unit, up to 8 parts, all of the products' magnitudes; an x below 2^-27 of its unit's largest is off by
    2^-35 of that.  Over the matrix: bf16 weights are the operands; parts of 8192 terms, and up to 147 split ones added."""
    t, (s, q, b) = packed(T + N, N, K, bits, group)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    y, matrix = _forward(_m(), t, N, K, bits, group, x)
    w, xa = s * q + b, x.double().abs()
    if matrix:
        w = w.bfloat16().double()
        mag = xa @ w.abs().t()
        tol = sum_err(min(K, 8192), mag) + (147 + K / 8192) * 2.0 ** -24 * mag
    else:
        mag = xa @ (s * q + b.abs()).t()
        tol = sum_err(64, mag) + (11 + 2 * K / 32 + 8) * 2.0 ** -24 * mag
        tol += 2.0 ** -35 * xa.amax(1, keepdim=True) * (s * q).sum(1)[None]
    ref = x.double() @ w.t()
    assert_within(y, ref, HALF["bf16"] * (ref.abs() + tol) + tol)


GRADIENT = [(1, 512, 256, 4, 64), (4, 17, 64, 4, 32), (70, 136, 320, 8, 64), (129, 1000, 96, 4, 32), (40, 1003, 128, 4, 64),
            (257, 264, 2048, 4, 64), (50, 30011, 128, 4, 64), (300, 5000, 64, 8, 32), (4, 4099, 320, 4, 32), (4, 1, 32, 8, 32),
            (500, 3001, 1024, 4, 64), (5, 65537, 64, 4, 64), (4, 100003, 96, 8, 32)]


def _gradient(m, t, N, K, bits, group, dy):
    T = len(dy)
    W = qtensor(m, t, N, K, bits, group)
    nb = m.moe_affine_linear_dx_workspace_bytes(W, T)
    ws = _ws(m, nb)
    dx = torch.full((T + 1, K), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_affine_linear_dx(W, dy, T, dx, ws, nb)
    torch.cuda.synchronize()
    assert bool((dx[T] == 7.0).all()) and m.moe_get_device_status(ws) == 0
    return dx[:T]


@pytest.mark.parametrize("T,N,K,bits,group", GRADIENT)
def test_input_gradient_of_whole_numbers(T, N, K, bits, group):
    t, w = _whole_matrix(T + N, N, K, bits, group)
    dy = _sparse(K, T, N)
    dx = _gradient(_m(), t, N, K, bits, group, dy)
    assert torch.equal(dx, (dy.double() @ w.bfloat16().double()).bfloat16())


@pytest.mark.parametrize("T,N,K,bits,group", GRADIENT)
def test_input_gradient_within_its_bound(T, N, K, bits, group):
    t, (s, q, b) = packed(T + N, N, K, bits, group)
    g = torch.Generator(device="cuda").manual_seed(K)
    dy = torch.randn((T, N), generator=g, device="cuda").bfloat16()
    dx = _gradient(_m(), t, N, K, bits, group, dy)
    w = (s * q + b).bfloat16().double()
    ref, mag = dy.double() @ w, dy.double().abs() @ w.abs()
    tol = sum_err(min(N, 8192), mag) + (147 + N / 8192) * 2.0 ** -24 * mag
    assert_within(dx, ref, HALF["bf16"] * (ref.abs() + tol) + tol)


@pytest.mark.parametrize("T,N,K", [(1, 2048, 512), (40, 136, 256), (300, 264, 2048), (2048, 512, 1024)])
def test_the_same_bits_again(T, N, K):
    """The same call, other calls between: the sums' order is fixed."""
    m = _m()
    t, _ = packed(1, N, K, 4, 64)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn((T, n), generator=g, device="cuda").bfloat16() for n in (K, N))
    y, dx = _forward(m, t, N, K, 4, 64, x)[0], _gradient(m, t, N, K, 4, 64, dy)
    for _ in range(3):
        _forward(m, t, N, K, 4, 64, -x)
        assert torch.equal(y, _forward(m, t, N, K, 4, 64, x)[0])
        assert torch.equal(dx, _gradient(m, t, N, K, 4, 64, dy))
