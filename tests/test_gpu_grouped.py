"""GPU parity of the products grouped by expert: forward, row gradient and weight gradient against 64 bits."""
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


def _case(seed, sizes, N, K, dtype, first=0, tail=0):
    """x, dy, W, offsets for groups of `sizes` rows; the rows before the first and behind the last are NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    off = offsets_of(sizes, first)
    M = int(off[-1]) + tail
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(DTYPES[dtype])  # noqa: E731
    x, dy, W = mk(M, K), mk(M, N), mk(len(sizes), N, K) * 0.1
    for t in (x, dy):
        t[:first] = float("nan")
        t[int(off[-1]):] = float("nan")
    return x, dy, W, off, M


def _run(kind, dtype, x, dy, W, off, M, G, N, K, out_dtype=None, accumulate=0, out=None, stream=None, null_off=False):
    m = _m()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    od = off.cuda() if off is not None else None
    code = {"bf16": m.DT_BF16, "fp16": m.DT_F16, "fp32": m.DT_F32}
    if out is None:
        shape = {"fwd": (M, N), "dx": (M, K), "dw": (G, N, K)}[kind]
        out = torch.full(shape, 7.0, dtype=DTYPES[out_dtype or dtype], device="cuda")
    if kind == "fwd":
        m.moe_grouped_matmul(code[dtype], x, od, W, M, G, N, K, out, st, stream)
    elif kind == "dx":
        m.moe_grouped_matmul_dx(code[dtype], dy, od, W, M, G, N, K, out, st, stream)
    else:
        m.moe_grouped_matmul_dw(code[dtype], dy, x, od, M, G, N, K, code[out_dtype or dtype], accumulate, out, st,
                                stream)
    torch.cuda.synchronize()
    return out, int(st.item())


def _check(kind, dtype, sizes, N, K, first=0, tail=0, out_dtype=None, seed=0):
    x, dy, W, off, M = _case(seed, sizes, N, K, dtype, first, tail)
    out, st = _run(kind, dtype, x, dy, W, off, M, len(sizes), N, K, out_dtype)
    assert st == 0
    ref, mag, n = grouped_ref(kind, off, x, W, dy)
    tol = HALF[out_dtype or dtype] * ref.abs() + 1.01 * sum_err(min(n, 512) + n // 64 if out_dtype == "fp32" else n, mag)
    tol += 2.0 ** -25 if (out_dtype or dtype) == "fp16" else 0  # half a step of the smallest fp16 values
    if kind != "dw":  # rows of no group keep what they held
        for r in (slice(0, first), slice(int(off[-1]), M)):
            assert bool((out[r] == 7.0).all())
            ref[r], tol[r] = 7.0, 0.0
    assert_within(out, ref, tol, "%s %s %dx%d" % (kind, dtype, N, K))


# (rows of each group, N, K): one row, odd sizes, empty groups, group ends inside tiles and on their edges, tiles
# wider than the matrix, sums shorter than a step
SHAPES = [
    ([1], 16, 16),
    ([1], 8, 8),
    ([3, 0, 5], 24, 40),
    ([64, 128, 0, 0, 129], 128, 64),
    ([0, 1, 255, 256, 257, 0], 136, 72),
    ([17] * 40, 16, 256),           # adapter-sized: many groups, few outputs
    ([2, 0, 3, 1] * 12, 256, 16),
    ([511, 700], 264, 520),
    ([100, 33], 384, 1000),
    ([5, 70, 0, 1], 51, 75),        # rows that are no multiple of 16 bytes
    ([130], 129, 257),
    ([2, 1], 1, 1),
    ([1, 0, 66], 7, 2048),
]


@pytest.mark.parametrize("kind", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dg_%dx%d" % (len(s[0]), s[1], s[2]))
def test_against_64_bits(kind, dtype, shape):
    _check(kind, dtype, *shape, first=3, tail=5)


@pytest.mark.parametrize("shape", [([3, 0, 5], 24, 40), ([700, 1200, 0, 31], 136, 264), ([1500], 51, 75)],
                         ids=["small", "long", "odd"])
def test_weight_gradient_in_fp32(shape):
    _check("dw", "bf16", *shape, first=1, tail=2, out_dtype="fp32")


@pytest.mark.parametrize("N,K", [(136, 264), (51, 75)])
@pytest.mark.parametrize("out_dtype", ["fp32", "bf16"])
def test_weight_gradient_accumulates(N, K, out_dtype):
    sizes = [40, 0, 600]
    x, dy, W, off, M = _case(3, sizes, N, K, "bf16")
    g = torch.Generator(device="cuda").manual_seed(9)
    old = torch.randn((3, N, K), generator=g, device="cuda").to(DTYPES[out_dtype])
    out, st = _run("dw", "bf16", x, dy, W, off, M, 3, N, K, out_dtype, 1, old.clone())
    ref, mag, n = grouped_ref("dw", off, x, W, dy)
    want = ref + old.double()
    assert st == 0 and bool((out[1] == old[1]).all())  # the group without rows
    assert_within(out, want, HALF[out_dtype] * want.abs() + 1.01 * sum_err(n, mag + old.double().abs()))


@pytest.mark.parametrize("N,K", [(64, 128), (33, 50)])
def test_one_group_without_offsets(N, K):
    x, dy, W, off, M = _case(4, [77], N, K, "bf16")
    for kind in ("fwd", "dx", "dw"):
        out, st = _run(kind, "bf16", x, dy, W, None, M, 1, N, K)
        ref, mag, n = grouped_ref(kind, off, x, W, dy)
        assert st == 0
        assert_within(out, ref, HALF["bf16"] * ref.abs() + 1.01 * sum_err(n, mag), kind)


@pytest.mark.parametrize("N,K", [(64, 128), (33, 50)])
def test_no_rows(N, K):
    """All groups empty: nothing is written but the weight gradient's zeros; M = 0 with no rows at all too."""
    x, dy, W, off, M = _case(5, [0, 0, 0], N, K, "bf16", first=2, tail=70)
    for kind in ("fwd", "dx"):
        out, st = _run(kind, "bf16", x, dy, W, off, M, 3, N, K)
        assert st == 0 and bool((out == 7.0).all())
    out, st = _run("dw", "bf16", x, dy, W, off, M, 3, N, K)
    assert st == 0 and bool((out == 0.0).all())
    out, st = _run("dw", "bf16", None, None, None, offsets_of([0, 0, 0]), 0, 3, N, K)
    assert st == 0 and bool((out == 0.0).all())


@pytest.mark.parametrize("N,K", [(64, 128), (33, 50)])
@pytest.mark.parametrize("bad", [[0, 50, 20, 90], [-5, 10, 40, 90], [0, 30, 60, 1000], [80, 70, 60, 50]])
def test_bad_offsets_are_flagged_and_clamped(N, K, bad):
    """Every row belongs to at most one group (the running maximum of the clamped offsets), and the status is raised."""
    M = 90
    x, dy, W, _, _ = _case(6, [30, 30, 30], N, K, "bf16")
    fixed, top = [], 0
    for v in bad:
        top = max(top, min(max(v, 0), M))
        fixed.append(top)
    for kind in ("fwd", "dx", "dw"):
        out, st = _run(kind, "bf16", x, dy, W, torch.tensor(bad, dtype=torch.int32), M, 3, N, K)
        assert st == 5
        ref, mag, n = grouped_ref(kind, fixed, x, W, dy)
        tol = HALF["bf16"] * ref.abs() + 1.01 * sum_err(n, mag)
        if kind != "dw":
            for r in (slice(0, fixed[0]), slice(fixed[-1], M)):
                ref[r], tol[r] = 7.0, 0.0
        assert_within(out, ref, tol, kind)


@pytest.mark.parametrize("N,K", [(128, 192), (30, 77)])
def test_a_nan_row_stays_in_its_row_and_group(N, K):
    sizes = [37, 64, 21]
    x, dy, W, off, M = _case(7, sizes, N, K, "bf16")
    x[40] = float("nan")
    dy[40] = float("inf")
    y, _ = _run("fwd", "bf16", x, dy, W, off, M, 3, N, K)
    dx, _ = _run("dx", "bf16", x, dy, W, off, M, 3, N, K)
    dw, _ = _run("dw", "bf16", x, dy, W, off, M, 3, N, K)
    ok = torch.ones(M, dtype=torch.bool, device="cuda")
    ok[40] = False
    assert bool(y[40].isnan().all()) and bool(y[ok].isfinite().all())
    assert not bool(dx[40].isfinite().any()) and bool(dx[ok].isfinite().all())
    assert bool(dw[1].isnan().all()) and bool(dw[[0, 2]].isfinite().all())


@pytest.mark.parametrize("N,K", [(128, 192), (30, 77)])
def test_unaligned_addresses(N, K):
    """Operands and outputs that start 2 bytes past a 16-byte boundary."""
    sizes = [37, 0, 90]
    x, dy, W, off, M = _case(8, sizes, N, K, "bf16")

    def shift(t):
        b = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        v = b[1:1 + t.numel()].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 16 == 2
        return v

    for kind, shape in (("fwd", (M, N)), ("dx", (M, K)), ("dw", (3, N, K))):
        out = shift(torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda"))
        _, st = _run(kind, "bf16", shift(x), shift(dy), shift(W), off, M, 3, N, K, out=out)
        ref, mag, n = grouped_ref(kind, off, x, W, dy)
        assert st == 0
        assert_within(out, ref, HALF["bf16"] * ref.abs() + 1.01 * sum_err(n, mag), kind)


def test_results_repeat_and_do_not_depend_on_other_groups():
    """Bitwise: the same call twice, and a group's rows alone against the same rows among others."""
    sizes, N, K = [300, 5, 0, 77, 130], 264, 512
    x, dy, W, off, M = _case(10, sizes, N, K, "bf16")
    for kind in ("fwd", "dx", "dw"):
        a, _ = _run(kind, "bf16", x, dy, W, off, M, 5, N, K)
        b, _ = _run(kind, "bf16", x, dy, W, off, M, 5, N, K)
        assert torch.equal(a, b)
    whole, _ = _run("fwd", "bf16", x, dy, W, off, M, 5, N, K)
    r = slice(int(off[3]), int(off[4]))
    alone, _ = _run("fwd", "bf16", x[r].contiguous(), None, W[3:4].contiguous(), offsets_of([77]), 77, 1, N, K)
    assert torch.equal(whole[r], alone)


@pytest.mark.parametrize("kind", ["fwd", "dx", "dw"])
def test_element_offsets_past_32_bits(kind):
    """The groups' rows lie behind more than 2^31 elements of rows."""
    K, N = 2048, 2048
    M = (1 << 31) // K + 300
    sizes = [100, 0, 120]
    first = M - 225
    off = offsets_of(sizes, first)
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    rows = torch.randn((220, K), generator=g, device="cuda").bfloat16()
    x[first:first + 220] = rows
    W = (torch.randn((3, N, K), generator=g, device="cuda") * 0.1).bfloat16()
    small = [0, 100, 100, 220]
    if kind == "dw":
        out, st = _run("dw", "bf16", x, x, None, off, M, 3, N, K)
        ref, mag, n = grouped_ref("dw", small, rows, None, rows)
    else:
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        _, st = _run(kind, "bf16", x, x, W, off, M, 3, N, K, out=out)
        out = out[first:first + 220]
        ref, mag, n = grouped_ref(kind, small, rows, W, rows)
    assert st == 0
    assert_within(out, ref, HALF["bf16"] * ref.abs() + 1.01 * sum_err(n, mag), kind)


def test_graph_replay_with_new_offsets_and_two_streams():
    """A captured call follows the offsets' new values; two graphs on two streams at once do not disturb each other."""
    m = _m()
    N, K, G, M = 128, 256, 4, 400
    x, dy, W, off, _ = _case(12, [100] * 4, N, K, "bf16")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    offs = [off.cuda(), off.cuda()]
    ys = [torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dws = [torch.empty((G, N, K), dtype=torch.float32, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=streams[i]):
                m.moe_grouped_matmul(m.DT_BF16, x, offs[i], W, M, G, N, K, ys[i], st[i:i + 1])
                m.moe_grouped_matmul_dw(m.DT_BF16, dy, x, offs[i], M, G, N, K, m.DT_F32, 0, dws[i], st[i:i + 1])
        graphs.append(gr)
    new = [[0, 10, 10, 300, 400], [0, 399, 400, 400, 400]]
    for i in range(2):
        offs[i].copy_(torch.tensor(new[i], dtype=torch.int32))
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0]
    for i in range(2):
        ref, mag, n = grouped_ref("fwd", new[i], x, W, dy)
        assert_within(ys[i], ref, HALF["bf16"] * ref.abs() + 1.01 * sum_err(n, mag))
        ref, mag, n = grouped_ref("dw", new[i], x, W, dy)
        assert_within(dws[i], ref, HALF["fp32"] * ref.abs() + 1.01 * sum_err(n, mag))


def test_gradients_against_differences():
    """<dy, y(x + e v) - y(x - e v)> / 2e = <dx, v> and the same for W: the products are linear, so the difference is
    exact up to the roundings of the outputs (bounded by half a step of each)."""
    sizes, N, K, e = [9, 0, 30], 40, 24, 0.5
    x, dy, W, off, M = _case(13, sizes, N, K, "fp16")
    v = (torch.randint(-2, 3, x.shape, device="cuda") * 0.25).half()
    V = (torch.randint(-2, 3, W.shape, device="cuda") * 0.25).half()
    dx, _ = _run("dx", "fp16", x, dy, W, off, M, 3, N, K)
    dw, _ = _run("dw", "fp16", x, dy, W, off, M, 3, N, K, "fp32")
    for grad, direction, run in (
            (dx, v, lambda t: _run("fwd", "fp16", v * t, dy, W, off, M, 3, N, K)[0]),
            (dw, V, lambda t: _run("fwd", "fp16", x, dy, V * t, off, M, 3, N, K)[0])):
        up, dn = run(e).double(), run(-e).double()
        d = dy.double()
        by_diff = float((d * (up - dn)).sum() / (2 * e))
        by_grad = float((grad.double() * direction.double()).sum())
        tol = float((d.abs() * (up.abs() + dn.abs())).sum()) / (2 * e) * HALF["fp16"] * 1.1
        tol += float((grad.double().abs() * direction.double().abs()).sum()) * HALF["fp16"] * 1.1
        assert abs(by_diff - by_grad) <= tol, (by_diff, by_grad, tol)


@pytest.mark.parametrize("kind", ["fwd", "dx", "dw"])
def test_more_groups_than_a_block_tabulates(kind):
    """2500 groups, most of them empty or of one row: (expert, adapter) pairs."""
    g = torch.Generator().manual_seed(14)
    sizes = (torch.randint(0, 4, (2500,), generator=g) * (torch.rand(2500, generator=g) > 0.5)).tolist()
    sizes[1300] = 300
    _check(kind, "bf16", sizes, 40, 48, first=2, tail=3)


def test_on_a_given_stream():
    """The stream argument: work follows what that stream did before."""
    m = _m()
    sizes, N, K = [50, 0, 70], 128, 256
    x, dy, W, off, M = _case(15, sizes, N, K, "bf16")
    s = torch.cuda.Stream()
    xs = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2000000)
        xs.copy_(x)
    out, st = _run("fwd", "bf16", xs, dy, W, off, M, 3, N, K, stream=s)
    ref, mag, n = grouped_ref("fwd", off, x, W, dy)
    assert st == 0
    assert_within(out, ref, HALF["bf16"] * ref.abs() + 1.01 * sum_err(n, mag))


@pytest.mark.parametrize("N,K", [(8, 8), (9, 7)])
def test_very_many_rows_of_one_sign_in_16_bits(N, K):
    """A million rows of one expert, all products positive, to fp16.  Parts of at most 8192
    terms err by sum_err's 1.3e-4 of the result, the fp32 additions of at most 2048 parts, whose partial sums average
    half of the whole, by 2048 / 2 * 2^-24 = 6e-5 at most: 2.5e-4 covers both.  In one part a sum so long would be
    off by several half steps."""
    M = 1 << 20
    g = torch.Generator(device="cuda").manual_seed(5)
    mk = lambda n: (0.05 + 0.1 * torch.rand((M, n), generator=g, device="cuda")).half()  # noqa: E731
    x, dy = mk(K), mk(N)
    off = offsets_of([3, M - 10, 0, 7])
    out, st = _run("dw", "fp16", x, dy, None, off, M, 4, N, K)
    assert st == 0
    ref, mag, n = grouped_ref("dw", off, x=x, dy=dy)
    step = torch.exp2(torch.floor(torch.log2(ref.clamp(min=2.0 ** -14)))) * 2.0 ** -10
    assert_within(out, ref, step / 2 + (2.5e-4 + 8 * 2.0 ** -23) * mag + 2.0 ** -25, "dw of many rows")


@pytest.mark.parametrize("kind,N,K", [("fwd", 24, 65536), ("dx", 65536, 24), ("fwd", 9, 65535), ("dx", 65535, 9)])
def test_the_longest_sums_of_one_sign(kind, N, K):
    """As above for the widest matrices: parts of at most 8192 terms, 8 to 128 of them."""
    g = torch.Generator(device="cuda").manual_seed(6)
    mk = lambda *s: (0.05 + 0.1 * torch.rand(s, generator=g, device="cuda")).half()  # noqa: E731
    off = offsets_of([5, 0, 300, 1])
    M = int(off[-1])
    x, dy, W = mk(M, K), mk(M, N), mk(4, N, K)
    out, st = _run(kind, "fp16", x, dy, W, off, M, 4, N, K)
    assert st == 0
    ref, mag, n = grouped_ref(kind, off, x, W, dy)
    step = torch.exp2(torch.floor(torch.log2(ref.clamp(min=2.0 ** -14)))) * 2.0 ** -10
    assert_within(out, ref, step / 2 + (sum_err(8192, 1) + 64 * 2.0 ** -24) * mag + 2.0 ** -25, "long sums")


@pytest.mark.parametrize("sizes", [[5000], [2100, 0, 1, 4000], [1024, 1030], [300, 290]])
@pytest.mark.parametrize("N,K", [(16, 264), (51, 75), (130, 8)])
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("fp16", "fp32"), ("bf16", "fp32")])
def test_weight_gradients_of_few_tiles_and_many_rows(sizes, N, K, dtype, out_dtype):
    """Blocks that share a tile's rows: rows before and behind the groups are NaN, accumulation adds once, and the
    result is the same again."""
    _check("dw", dtype, sizes, N, K, first=2, tail=3, out_dtype=out_dtype, seed=11)
    x, dy, W, off, M = _case(12, sizes, N, K, dtype)
    once, _ = _run("dw", dtype, x, dy, W, off, M, len(sizes), N, K, out_dtype)
    old = torch.randn(once.shape, generator=torch.Generator(device="cuda").manual_seed(13), device="cuda").to(once.dtype)
    outs = [_run("dw", dtype, x, dy, W, off, M, len(sizes), N, K, out_dtype, 1, old.clone())[0] for _ in range(2)]
    assert torch.equal(*outs)
    ref, mag, n = grouped_ref("dw", off, x=x, dy=dy)
    ref += old.double()
    tol = HALF[out_dtype] * ref.abs() + 1.01 * sum_err(min(n, 512) + n // 64, mag) + 2.0 ** -24 * (mag + old.double().abs())
    assert_within(outs[0], ref, tol if out_dtype == "fp32" else tol + 1.01 * sum_err(n, mag), "added")
