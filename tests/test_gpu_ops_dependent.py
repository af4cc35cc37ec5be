"""Operators that set themselves up beside the kernel they depend on read what that kernel has written: rows, weights per row,
scales and whole matrices that a grouped product leaves behind, for kernels of every kind, bit for bit what they read after
a wait."""
import pytest

from tests.gpu_helpers import need_cuda
from tests.op_helpers import packed, qtensor

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    need_cuda()


def _m():
    import int4_group_affine_b200 as m
    return m


@pytest.mark.parametrize("what", ["swiglu", "swiglu_grad", "linear", "linear_dx", "grouped", "scales", "offsets"])
@pytest.mark.parametrize("n", [102, 128, 130, 1024])
@pytest.mark.parametrize("T", [12, 700])
def test_what_the_kernel_ahead_wrote(what, n, T):
    """y = W x by moe_grouped_matmul (whole numbers, two sets of rows in turn, so what was there before differs), and the
    operator on y straight behind it."""
    m = _m()
    g = torch.Generator(device="cuda").manual_seed(n + T)
    mk = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").bfloat16()  # noqa: E731
    K, bf = 1024, m.DT_BF16
    xs, W = [mk(T, K), mk(T, K)], mk(1, n, K) * 0.125
    y, st = torch.empty((T, n), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    if what in ("linear", "linear_dx", "scales"):
        N, Kl = {"linear": (264, n // 32 * 32), "linear_dx": (n, 320), "scales": (300, n // 32 * 32)}[what]
        if what == "linear" and n % 32:
            pytest.skip("rows of whole groups")
        t, _ = packed(1, N, Kl, 4, 32)
        Q = qtensor(m, t, N, Kl, 4, 32)
        size = m.moe_affine_linear_dx_workspace_bytes if what == "linear_dx" else m.moe_affine_linear_workspace_bytes
        nb = size(Q, T)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        m.moe_workspace_init(ws, nb)
    out = {}
    new = lambda name, *s, t=torch.bfloat16: out.setdefault(name, torch.empty(s, dtype=t, device="cuda"))  # noqa: E731
    W2, dh, rows = mk(1, 136, n), mk(T, n // 2), mk(T, 320)

    def run():
        if what == "swiglu":
            m.moe_swiglu(bf, y, None, off, 1, T, n // 2, new("h", T, n // 2))
        elif what == "swiglu_grad":
            m.moe_swiglu_grad(bf, y, None, dh, off, 1, T, n // 2, new("d", T, n), new("w", T, t=torch.float32))
        elif what == "linear":
            m.moe_affine_linear(Q, y, T, new("y", T, N), ws, nb)
        elif what == "linear_dx":
            m.moe_affine_linear_dx(Q, y, T, new("x", T, Kl), ws, nb)
        elif what == "scales":  # the matrix's scales and biases are the rows just written
            Q.scales = Q.biases = y.data_ptr()
            m.moe_affine_linear(Q, xl, T, new("y", T, N), ws, nb)
        elif what == "grouped":
            m.moe_grouped_matmul(bf, y, off, W2, T, 1, 136, n, new("y", T, 136), st)
            m.moe_grouped_matmul_dw(bf, y, rows, off, T, 1, n, 320, m.DT_F32, 0, new("dw", 1, n, 320, t=torch.float32), st)
        else:  # offsets: written by the index kernels between two products
            m.moe_index_build(idx, None, T, 1, 8, 0, counts, offs, perm, iws, inb)
            m.moe_grouped_matmul(bf, y, offs, W8, T, 8, 72, n, new("y", T, 72), st)
    if what == "scales":
        if T * n < N * Kl // 32:
            pytest.skip("too few values")
        xl = mk(T, Kl)
    if what == "offsets":
        idx = torch.randint(0, 8, (T, 1), generator=g, device="cuda", dtype=torch.int32)
        counts, offs = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (9, 10))
        perm = torch.empty((2 * T, 4), dtype=torch.int32, device="cuda")
        inb = m.moe_index_workspace_bytes(T, 1, 8, 0)
        iws = torch.empty(inb, dtype=torch.uint8, device="cuda")
        m.moe_workspace_init(iws, inb)
        W8 = mk(8, 72, n)
        idx2 = [idx.clone(), (idx + 3) % 8]

    def chain(i, wait):
        if what == "offsets":
            idx.copy_(idx2[i])
        m.moe_grouped_matmul(bf, xs[i], off, W, T, 1, n, K, y, st)
        if wait:
            torch.cuda.synchronize()
        run()
    want = []
    for i in range(2):
        chain(i, True)
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
    assert any(not torch.equal(want[0][k], want[1][k]) for k in out)
    for k in range(20):
        i = k % 2
        for _ in range(3):
            chain(1 - i, False)
            chain(i, False)
        torch.cuda.synchronize()
        for name, v in out.items():
            assert torch.equal(v.view(torch.uint8), want[i][name].view(torch.uint8)), (name, k)
    assert int(st.item()) == 0
