"""Pairs of blocks and clusters that end: what they send each other (reports of multiplied stages, of accumulators that were
read, sums in shared memory) has arrived before either ends, so blocks of the next call, which use the same shared memory
for something else, find their own barriers and sums.  Short calls of all kinds, back to back and on two streams."""
import pytest

from tests.gpu_helpers import need_cuda

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    need_cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_short_calls_back_to_back(dtype):
    import int4_group_affine_b200 as m
    t = torch.bfloat16 if dtype == "bf16" else torch.float16
    code = m.DT_BF16 if dtype == "bf16" else m.DT_F16
    g = torch.Generator(device="cuda").manual_seed(1)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(t)  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = []
    # one stage and many (the ring's length and one more and less), one tile a pair and several, few and many rows
    for sizes, N, K in (([1], 256, 64), ([5, 60], 512, 320), ([70], 264, 384), ([300, 0, 9], 1024, 448), ([33] * 40, 384, 136),
                        ([2] * 64, 512, 512), ([700, 31], 16, 264), ([2000], 40, 72)):
        off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        M, G = sum(sizes), len(sizes)
        x, dy, W = whole(M, K), whole(M, N), whole(G, N, K)
        new = lambda *s: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        y, dx, dw = new(M, N), new(M, K), torch.empty((G, N, K), device="cuda")
        args = (M, G, N, K)
        calls += [(m.moe_grouped_matmul, (code, x, off, W, *args), y), (m.moe_grouped_matmul_dx, (code, dy, off, W, *args), dx),
                  (m.moe_grouped_matmul_dw, (code, dy, x, off, *args, m.DT_F32, 0), dw)]
        for e in range(G):
            r = slice(int(off[e]), int(off[e + 1]))
            a, b, w = x[r].double(), dy[r].double(), W[e].double()
            y[r], dx[r], dw[e] = (a @ w.t()).to(t), (b @ w).to(t), (b.t() @ a).float()
    want = [out.clone() for _, _, out in calls]  # (whole numbers: the sums are exact)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rounds in range(8):
        for _, _, out in calls:
            out.fill_(7.0)
        torch.cuda.synchronize()
        for k in range(6):
            for i, (f, args, out) in enumerate(calls):
                f(*args, out, st, stream=streams[i % 2 if rounds % 2 else 0])
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        for (f, _, out), w in zip(calls, want):
            assert torch.equal(out, w), f.__name__
