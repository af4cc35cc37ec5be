"""The products grouped by expert on inputs whose sums are exact, and the weight gradients' long sums.

Exact: rows and matrices of small whole numbers, so few or so sparse that every partial sum is a whole number below 2^24:
no fp32 addition rounds or truncates, whatever its order, and the result has to be the exact sum rounded once."""
import pytest

from tests.gpu_helpers import need_cuda
from tests.op_helpers import DTYPES, HALF, assert_within, grouped_ref, offsets_of, sum_err

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    need_cuda()


def _m():
    import int4_group_affine_b200 as m
    return m


def _call(kind, dtype, off, M, N, K, x=None, W=None, dy=None, out_dtype=None, old=None):
    m = _m()
    G = len(off) - 1
    code = {"bf16": m.DT_BF16, "fp16": m.DT_F16, "fp32": m.DT_F32}
    st, od = torch.zeros(1, dtype=torch.int32, device="cuda"), off.cuda()
    shape = {"fwd": (M, N), "dx": (M, K), "dw": (G, N, K)}[kind]
    out = torch.full(shape, 7.0, dtype=DTYPES[out_dtype or dtype], device="cuda") if old is None else old.clone()
    if kind == "fwd":
        m.moe_grouped_matmul(code[dtype], x, od, W, M, G, N, K, out, st)
    elif kind == "dx":
        m.moe_grouped_matmul_dx(code[dtype], dy, od, W, M, G, N, K, out, st)
    else:
        m.moe_grouped_matmul_dw(code[dtype], dy, x, od, M, G, N, K, code[out_dtype or dtype], int(old is not None), out, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return out


def _whole(g, shape, top, dtype, dense=1.0):
    v = torch.randint(-top, top + 1, shape, generator=g, device="cuda").float()
    if dense < 1.0:
        v *= torch.rand(shape, generator=g, device="cuda") < dense
    return v.to(DTYPES[dtype])


# (rows of each group, N, K): sums that end inside a step of 16, 32, 64 or 128 terms and just behind one, split weight
# gradients and long ones
SHAPES = [([1], 8, 8), ([3, 0, 5], 24, 40), ([0, 1, 255, 256, 257, 0], 136, 72), ([17] * 40, 16, 264), ([511, 700], 264, 520),
          ([100, 33], 384, 1000), ([33, 1, 64], 130, 65528), ([40, 0, 3], 65528, 136), ([5, 70, 0, 1], 51, 75), ([130], 129, 257),
          ([2, 1], 1, 1), ([1, 0, 66], 7, 2049), ([20, 3], 33, 65535), ([3, 9], 65533, 35), ([5000, 130], 40, 200), ([4097, 31], 51, 75)]


@pytest.mark.parametrize("kind", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dg_%dx%d" % (len(s[0]), s[1], s[2]))
def test_whole_numbers(kind, dtype, shape):
    """Terms of at most 9 (16-bit results of at most 2^16 sums of 9 stay below fp16's largest by the terms' random signs; the
    matrices of long sums are mostly zeros)."""
    sizes, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(N + K)
    off = offsets_of(sizes, 2)
    M, terms = int(off[-1]) + 3, {"fwd": K, "dx": N, "dw": max(sizes)}[kind]
    dense = min(1.0, 2000 / terms)
    x, dy = _whole(g, (M, K), 3, dtype, dense), _whole(g, (M, N), 3, dtype, dense)
    W = _whole(g, (len(sizes), N, K), 3, dtype) if kind != "dw" else None
    for t in (x, dy):  # rows of no group
        t[:2] = float("nan")
        t[int(off[-1]):] = float("nan")
    got = _call(kind, dtype, off, M, N, K, x, W, dy)
    ref = grouped_ref(kind, off, x, W, dy)[0]
    if kind != "dw":
        ref[:2] = ref[int(off[-1]):] = 7.0
    assert torch.equal(got, ref.to(got.dtype))
    if kind == "dw":
        assert torch.equal(_call(kind, dtype, off, M, N, K, x, W, dy, "fp32"), ref.float())
        old = _whole(g, got.shape, 100, "fp32")
        assert torch.equal(_call(kind, dtype, off, M, N, K, x, W, dy, "fp32", old), (ref + old.double()).float())
        old = _whole(g, got.shape, 100, dtype)
        assert torch.equal(_call(kind, dtype, off, M, N, K, x, W, dy, dtype, old), (ref + old.double()).to(got.dtype))


# Weight gradients whose tiles fill the device, so that no tile's rows are shared between blocks: long groups among 200
# short ones; widths of one and of two bands of 128 columns, and rows that are no multiple of 16 bytes.
MANY = [0, 1, 2, 3] * 25
LONG = [(MANY + [20000] + MANY, 64, 64), (MANY + [9000, 8192, 8193] + MANY, 40, 264), (MANY + [16500] + MANY, 51, 75),
        (MANY + [513, 1024, 3000, 512] + MANY, 136, 264), (MANY + [513, 1024, 3000] + MANY, 33, 130)]


def _ids(s):
    return "%dx%d_%d" % (s[1], s[2], max(s[0]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", LONG, ids=_ids)
def test_long_groups_of_whole_numbers(dtype, shape):
    sizes, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(N)
    off = offsets_of(sizes, 1)
    M = int(off[-1]) + 2
    x, dy = _whole(g, (M, K), 3, dtype, 0.3), _whole(g, (M, N), 3, dtype, 0.3)
    x[0] = dy[0] = x[-2:] = dy[-2:] = float("nan")
    ref = grouped_ref("dw", off, x=x, dy=dy)[0]
    for out_dtype in (dtype, "fp32"):
        assert torch.equal(_call("dw", dtype, off, M, N, K, x, None, dy, out_dtype), ref.to(DTYPES[out_dtype]))
        old = _whole(g, ref.shape, 100, out_dtype)
        got = _call("dw", dtype, off, M, N, K, x, None, dy, out_dtype, old)
        assert torch.equal(got, (ref + old.double()).to(DTYPES[out_dtype]))


@pytest.mark.parametrize("dtype,out_dtype", [("fp16", "fp16"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp32")])
@pytest.mark.parametrize("shape", LONG, ids=_ids)
def test_long_groups_of_one_sign(dtype, out_dtype, shape):
    """All products positive.  16-bit results: parts of at most 8192 terms (sum_err, 1.3e-4 of the result), added in fp32.
    fp32 ones: parts of at most 512 (sum_err, 8.6e-6), at most 40 additions, 40 * 2^-24."""
    sizes, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(N)
    off = offsets_of(sizes, 0)
    M = int(off[-1])
    mk = lambda n: (0.05 + 0.1 * torch.rand((M, n), generator=g, device="cuda")).to(DTYPES[dtype])  # noqa: E731
    x, dy = mk(K), mk(N)
    ref, mag, n = grouped_ref("dw", off, x=x, dy=dy)
    got = _call("dw", dtype, off, M, N, K, x, None, dy, out_dtype)
    tol = sum_err(min(n, 512 if out_dtype == "fp32" else 8192), mag) + 40 * 2.0 ** -24 * mag
    assert_within(got, ref, tol + HALF[out_dtype] * (ref + tol) + (2.0 ** -25 if out_dtype == "fp16" else 0))
    assert torch.equal(got, _call("dw", dtype, off, M, N, K, x, None, dy, out_dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", LONG + [([5000], 16, 264), ([3000, 2000], 51, 75)], ids=_ids)
def test_gradients_are_added_once(dtype, shape):
    """accumulate in fp32: the sum of the rows is complete before it meets the earlier gradient, which is 1000 times as large
    as a part of the sum: one rounding of the new value, half a step, whatever the number of parts; beside it the sum's own
    error.  (Part by part onto it, 3000 rows and more are several steps off.)"""
    sizes, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(K)
    off = offsets_of(sizes, 0)
    M = int(off[-1])
    mk = lambda n: (0.005 + 0.01 * torch.rand((M, n), generator=g, device="cuda")).to(DTYPES[dtype])  # noqa: E731
    x, dy = mk(K), mk(N)
    old = 1000 + 16 * torch.rand((len(sizes), N, K), generator=g, device="cuda")
    ref, mag, n = grouped_ref("dw", off, x=x, dy=dy)
    want = ref + old.double()
    got = _call("dw", dtype, off, M, N, K, x, None, dy, "fp32", old)
    tol = sum_err(min(n, 512), mag) + 40 * 2.0 ** -24 * mag
    assert_within(got, want, 2.0 ** -15 + tol)  # (a step of [512, 1024) is 2^-14)
