"""The linear, grouped and SwiGLU operators together, as a program uses them: an unquantised expert layer forward and
backward on the library's own routing, and adapters trained over a packed base.

The bounds are propagated: every stored 16-bit value may be off by half a step of its type (HALF), every sum by its
accumulation (sum_err), and an operator passes on what its inputs may be off by, |W| times it for a product and the
derivative's magnitude times it for SwiGLU; products of two such errors are covered by the factor 1.1."""
import pytest

from tests.gpu_helpers import need_cuda
from tests.op_helpers import HALF, assert_within, packed, qtensor, sum_err

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
H16 = HALF["bf16"]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    need_cuda()


def _m():
    import int4_group_affine_b200 as m
    return m


def _randn(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


class Bounded:
    """A value in 64 bits and how far the stored 16-bit one may be off it."""

    def __init__(self, v, e):
        self.v, self.e = v, e

    def stored(self):
        return Bounded(self.v, self.e + H16 * (self.v.abs() + self.e))

    def __matmul__(self, w):  # w exact
        n = self.v.shape[-1]
        return Bounded(self.v @ w, (self.e @ w.abs() + sum_err(n, (self.v.abs() + self.e) @ w.abs())))


def _exact(t):
    return Bounded(t.double(), torch.zeros_like(t, dtype=torch.float64))


@pytest.mark.parametrize("T,H,E,K,I", [(5, 64, 8, 2, 32), (150, 128, 16, 4, 72), (33, 256, 4, 3, 40)])
def test_expert_layer_forward_and_backward(T, H, E, K, I):
    m = _m()
    dev = "cuda"
    # the library's routing: an 8-bit router, the jobs sorted by expert
    rt, (s, q, b) = packed(1, E, H, 8, 32)
    router = qtensor(m, rt, E, H, 8, 32)
    x = _randn(2, T, H)
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    w = torch.empty((T, K), device=dev)
    logits = torch.empty((T, E), device=dev)
    m.moe_router_topk(x, router, None, None, T, H, E, K, idx, w, None, logits)
    nb = m.moe_index_workspace_bytes(T, K, E, 0)
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    m.moe_workspace_init(ws, nb)
    J = T * (K + 1)  # the shared expert's jobs come last: rows behind the groups used here
    counts, offs = torch.empty(E + 1, dtype=torch.int32, device=dev), torch.empty(E + 2, dtype=torch.int32, device=dev)
    perm = torch.empty((J, 4), dtype=torch.int32, device=dev)
    m.moe_index_build(idx, None, T, K, E, 0, counts, offs, perm, ws, nb)
    tok, kk = perm[:, 0].long(), perm[:, 1].long()
    routed = kk < K
    R = T * K
    roww = torch.where(routed, w[tok, kk.clamp(max=K - 1)], 0.0).contiguous()
    pos = torch.empty((T, K), dtype=torch.int32, device=dev)
    pos[tok[:R], kk[:R]] = torch.arange(R, dtype=torch.int32, device=dev)
    ones = torch.ones((T, K), device=dev)

    Wgu, Wd = _randn(3, E, 2 * I, H, std=0.15), _randn(4, E, H, I, std=0.2)
    xr = x[tok].contiguous()
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    nan = lambda *shape: torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev)  # noqa: E731
    gu, h, yr = nan(J, 2 * I), nan(J, I), nan(J, H)
    m.moe_grouped_matmul(m.DT_BF16, xr, offs, Wgu, J, E, 2 * I, H, gu, st)
    m.moe_swiglu(m.DT_BF16, gu, roww, offs, E, J, I, h)
    m.moe_grouped_matmul(m.DT_BF16, h, offs, Wd, J, E, H, I, yr, st)
    y = nan(T, H)
    m.moe_ep_combine(yr, pos, ones, None, None, T, K, H, y)

    dy = _randn(5, T, H)
    dyr = dy[tok].contiguous()
    dh, dgu, dxr = nan(J, I), nan(J, 2 * I), nan(J, H)
    droww = torch.full((J,), float("nan"), device=dev)
    dWgu, dWd = torch.empty((E, 2 * I, H), device=dev), torch.empty((E, H, I), device=dev)
    m.moe_grouped_matmul_dw(m.DT_BF16, dyr, h, offs, J, E, H, I, m.DT_F32, 0, dWd, st)
    m.moe_grouped_matmul_dx(m.DT_BF16, dyr, offs, Wd, J, E, H, I, dh, st)
    m.moe_swiglu_grad(m.DT_BF16, gu, roww, dh, offs, E, J, I, dgu, droww)
    m.moe_grouped_matmul_dw(m.DT_BF16, dgu, xr, offs, J, E, 2 * I, H, m.DT_F32, 0, dWgu, st)
    m.moe_grouped_matmul_dx(m.DT_BF16, dgu, offs, Wgu, J, E, 2 * I, H, dxr, st)
    dx = nan(T, H)
    m.moe_ep_combine(dxr, pos, ones, None, None, T, K, H, dx)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool(yr[R:].isnan().all()) and bool(dxr[R:].isnan().all()) and bool(droww[R:].isnan().all())

    # the same in 64 bits by autograd
    g64 = lambda t: t.double().detach().requires_grad_(True)  # noqa: E731
    x64, Wgu64, Wd64, w64 = g64(x), g64(Wgu), g64(Wd), g64(w)
    rows, ref_h = [], []
    for j in range(R):
        t, k, e = int(tok[j]), int(kk[j]), int(perm[j, 3])
        z = Wgu64[e] @ x64[t]
        hj = w64[t, k] * torch.nn.functional.silu(z[:I]) * z[I:]
        rows.append(Wd64[e] @ hj)
        ref_h.append(hj)
    y64 = torch.zeros((T, H), dtype=torch.float64, device=dev).index_add(0, tok[:R], torch.stack(rows))
    (y64 * dy.double()).sum().backward()

    # the bounds, job by job
    exp = perm[:R, 3].long()
    by = lambda W: W.double()[exp]  # noqa: E731  [R, ., .]
    lin = lambda a, W: Bounded(torch.bmm(W, a.v[..., None])[..., 0],  # noqa: E731
                               torch.bmm(W.abs(), a.e[..., None])[..., 0]
                               + sum_err(W.shape[2], torch.bmm(W.abs(), (a.v.abs() + a.e)[..., None])[..., 0]))
    z = lin(_exact(xr[:R]), by(Wgu)).stored()
    gv, uv, ge, ue = z.v[:, :I], z.v[:, I:], z.e[:, :I], z.e[:, I:]
    sg = torch.sigmoid(gv)
    silu, slope = gv * sg, sg * (1 + gv * (1 - sg))
    slope_max, curve = 1.1, 0.5  # |silu'| <= 1.0999, |silu''| <= 0.5
    rw = roww[:R].double()[:, None]
    hb = Bounded(rw * silu * uv, rw * (slope_max * ge * uv.abs() + silu.abs() * ue) + 2.0 ** -20 * (rw * silu * uv).abs())
    hb = hb.stored()
    yb = lin(hb, by(Wd)).stored()
    cmb = lambda v: torch.zeros((T, v.shape[1]), dtype=torch.float64, device=dev).index_add(0, tok[:R], v)  # noqa: E731
    ytol = cmb(yb.e) + 2.0 ** -20 * cmb(yb.v.abs())
    assert_within(y, y64.detach(), 1.1 * (ytol + H16 * (y64.detach().abs() + ytol)), "y")

    dhb = lin(_exact(dyr[:R]), by(Wd).transpose(1, 2).contiguous()).stored()
    d, de = dhb.v, dhb.e
    dg = Bounded(rw * d * uv * slope, rw * ((de * uv.abs() + d.abs() * ue) * slope_max + (d * uv).abs() * curve * ge)
                 + 2.0 ** -18 * (rw * d * uv).abs() * (1 + gv.abs()))
    du = Bounded(rw * d * silu, rw * (de * silu.abs() + d.abs() * slope_max * ge) + 2.0 ** -18 * (rw * d * silu).abs())
    dz = Bounded(torch.cat([dg.v, du.v], 1), torch.cat([dg.e, du.e], 1)).stored()
    dwr = (d * silu * uv).sum(1)
    dwr_e = ((de * (silu * uv).abs() + (d * uv).abs() * slope_max * ge + (d * silu).abs() * ue).sum(1)
             + 2.0 ** -16 * (d * silu * uv).abs().sum(1))
    assert_within(droww[:R], w64.grad[tok[:R], kk[:R]], 1.1 * dwr_e, "routing weights")
    assert torch.allclose(dwr, w64.grad[tok[:R], kk[:R]], rtol=1e-9, atol=1e-12)
    dxb = lin(dz, by(Wgu).transpose(1, 2).contiguous()).stored()
    xtol = cmb(dxb.e) + 2.0 ** -20 * cmb(dxb.v.abs())
    assert_within(dx, x64.grad, 1.1 * (xtol + H16 * (x64.grad.abs() + xtol)), "dx")

    def outer(a, c):  # sums over each expert's rows of a c^T
        v = torch.zeros((E, a.v.shape[1], c.v.shape[1]), dtype=torch.float64, device=dev)
        e, mag = torch.zeros_like(v), torch.zeros_like(v)
        for g in range(E):
            r = exp == g
            av, ae, cv, ce = a.v[r], a.e[r], c.v[r], c.e[r]
            v[g] = av.t() @ cv
            mag[g] = (av.abs() + ae).t() @ (cv.abs() + ce)
            e[g] = ae.t() @ (cv.abs() + ce) + av.abs().t() @ ce + sum_err(int(r.sum()), mag[g])
        return Bounded(v, e)
    for got, want, a, c in ((dWd, Wd64.grad, _exact(dyr[:R]), hb), (dWgu, Wgu64.grad, dz, _exact(xr[:R]))):
        o = outer(a, c)
        assert_within(got, want, 1.1 * o.e + HALF["fp32"] * want.abs(), "weights")


@pytest.mark.parametrize("T,N,K,r,A", [(7, 72, 128, 8, 2), (140, 264, 256, 16, 3), (300, 136, 192, 24, 1)])
def test_adapters_over_a_packed_base(T, N, K, r, A):
    """y = W x + B_a (A_a x) for tokens sorted by adapter, and the gradients of x, A and B; W stays packed."""
    m = _m()
    dev = "cuda"
    t, (s, q, b) = packed(11, N, K, 4, 64)
    W = qtensor(m, t, N, K, 4, 64)
    w64 = s * q + b
    x, dy = _randn(12, T, K), _randn(13, T, N)
    FA, FB = _randn(14, A, r, K, std=0.1), _randn(15, A, N, r, std=0.1)
    cuts = [0] + sorted(int(v) for v in torch.randint(0, T + 1, (A - 1,), generator=torch.Generator().manual_seed(T)))
    cuts.append(T)
    off = torch.tensor(cuts, dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    nb = max(m.moe_affine_linear_workspace_bytes(W, T), m.moe_affine_linear_dx_workspace_bytes(W, T))
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    m.moe_workspace_init(ws, nb)
    new = lambda *sh: torch.empty(sh, dtype=torch.bfloat16, device=dev)  # noqa: E731
    y0, v, y1 = new(T, N), new(T, r), new(T, N)
    m.moe_affine_linear(W, x, T, y0, ws, nb)
    m.moe_grouped_matmul(m.DT_BF16, x, off, FA, T, A, r, K, v, st)
    m.moe_grouped_matmul(m.DT_BF16, v, off, FB, T, A, N, r, y1, st)
    dx0, dv, dx1 = new(T, K), new(T, r), new(T, K)
    dA, dB = torch.zeros((A, r, K), device=dev), torch.zeros((A, N, r), device=dev)
    m.moe_affine_linear_dx(W, dy, T, dx0, ws, nb)
    m.moe_grouped_matmul_dx(m.DT_BF16, dy, off, FB, T, A, N, r, dv, st)
    m.moe_grouped_matmul_dx(m.DT_BF16, dv, off, FA, T, A, r, K, dx1, st)
    m.moe_grouped_matmul_dw(m.DT_BF16, dy, v, off, T, A, N, r, m.DT_F32, 1, dB, st)
    m.moe_grouped_matmul_dw(m.DT_BF16, dv, x, off, T, A, r, K, m.DT_F32, 1, dA, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and m.moe_get_device_status(ws) == 0

    xd, dyd = x.double(), dy.double()
    matrix = lambda a, wt: H16 * (a.abs() @ wt.abs())  # noqa: E731  the packed base as bf16
    yb = _exact(x) @ w64.t()
    y = Bounded(yb.v, yb.e + matrix(xd, w64.t()) + 2.0 ** -14 * (xd.abs() @ (s * 300 + b.abs()).t())).stored()
    assert_within(y0, y.v, 1.1 * y.e, "base")
    db = _exact(dy) @ w64
    d = Bounded(db.v, db.e + matrix(dyd, w64)).stored()
    assert_within(dx0, d.v, 1.1 * d.e, "base dx")
    for a in range(A):
        r0 = slice(cuts[a], cuts[a + 1])
        if cuts[a] == cuts[a + 1]:
            assert bool((dA[a] == 0).all()) and bool((dB[a] == 0).all())
            continue
        Ad, Bd = FA[a].double(), FB[a].double()
        vb = (_exact(x[r0]) @ Ad.t()).stored()
        yb = (vb @ Bd.t()).stored()
        dvb = (_exact(dy[r0]) @ Bd).stored()
        dxb = (dvb @ Ad).stored()
        n = cuts[a + 1] - cuts[a]
        for got, want, what in ((v[r0], vb, "Ax"), (y1[r0], yb, "delta"), (dv[r0], dvb, "dv"), (dx1[r0], dxb, "dx")):
            assert_within(got, want.v, 1.1 * want.e, what)
        mag = dyd[r0].abs().t() @ (vb.v.abs() + vb.e)
        assert_within(dB[a], dyd[r0].t() @ vb.v, 1.1 * (dyd[r0].abs().t() @ vb.e + sum_err(n, mag)), "dB")
        mag = (dvb.v.abs() + dvb.e).t() @ xd[r0].abs()
        assert_within(dA[a], dvb.v.t() @ xd[r0], 1.1 * (dvb.e.t() @ xd[r0].abs() + sum_err(n, mag)), "dA")


@pytest.mark.parametrize("T", [1, 40])
def test_a_chain_of_calls_without_waiting(T):
    """Each call reads what the call before wrote, the layer's own forward among them: the same bits whether the host
    waits after every call, after none, or replays the chain as a graph (kernels set themselves up beside the one they
    depend on)."""
    from int4_group_affine_b200.layer import DeviceLayer
    from synth import workloads
    from tests.helpers import quantize_layer
    m = _m()
    d = DeviceLayer.from_host(workloads.TINY, quantize_layer(workloads.moe_weights(workloads.TINY, seed=3)))
    H, rounds = d.H, 6
    ws, nb = d.workspace(T)
    lt, _ = packed(4, H, H, 4, 32, std=H ** -0.5)
    lin = qtensor(m, lt, H, H, 4, 32)
    lb = max(m.moe_affine_linear_workspace_bytes(lin, T), m.moe_affine_linear_dx_workspace_bytes(lin, T))
    lws = torch.empty(lb, dtype=torch.uint8, device="cuda")
    m.moe_workspace_init(lws, lb)
    W = _randn(5, 2, 2 * H, H, std=H ** -0.5)
    off = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = _randn(6, T, H)
    a, b, gu = (torch.empty((T, n), dtype=torch.bfloat16, device="cuda") for n in (H, H, 2 * H))
    dw = torch.empty((2, 2 * H, H), device="cuda")

    def chain(wait):
        def call(f, *args):
            f(*args)
            if wait:
                torch.cuda.synchronize()
        a.copy_(x)
        for _ in range(rounds):
            call(m.moe_rmsnorm, a, T, H, 1e-30, b)  # (the layer's outputs are small: without it the values die out)
            call(m.moe_ffn_forward, d.L, b, None, T, a, ws, nb)
            call(m.moe_rmsnorm, a, T, H, 1e-30, b)
            call(m.moe_grouped_matmul, m.DT_BF16, b, off, W, T, 2, 2 * H, H, gu, st)
            call(m.moe_grouped_matmul_dw, m.DT_BF16, gu, b, off, T, 2, 2 * H, H, m.DT_F32, 0, dw, st)
            call(m.moe_swiglu, m.DT_BF16, gu, None, off, 2, T, H, a)
            call(m.moe_affine_linear, lin, a, T, b, lws, lb)
            call(m.moe_grouped_matmul, m.DT_BF16, b, off, W, T, 2, 2 * H, H, gu, st)
            call(m.moe_grouped_matmul_dx, m.DT_BF16, gu, off, W, T, 2, 2 * H, H, b, st)
            call(m.moe_affine_linear_dx, lin, b, T, a, lws, lb)

    chain(True)
    want = [t.clone() for t in (a, dw)]
    assert bool(want[0].isfinite().all()) and bool((want[0] != 0).any())
    for _ in range(3):
        chain(False)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, (a, dw)))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            chain(False)
        for _ in range(3):
            a.zero_()
            dw.zero_()
            g.replay()
            s.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(want, (a, dw)))
    assert int(st.item()) == 0 and m.moe_get_device_status(ws) == 0 and m.moe_get_device_status(lws) == 0
