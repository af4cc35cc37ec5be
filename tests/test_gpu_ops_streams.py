"""The operators where streams meet and where threads call at once: a dependent kernel behind an event of another stream,
captured and not, and calls from several threads on streams of their own."""
import threading

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


@pytest.mark.parametrize("captured", [False, True])
def test_streams_meet(captured):
    """Two products on two streams, and behind the event that joins them operators on both results: first on the other
    stream's, which a kernel that waited for its own stream's product alone would read too early."""
    m = _m()
    T, K, I = 2048, 2048, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").bfloat16()  # noqa: E731
    xs = [whole(T, K), whole(T, K)]
    x, W, Ws, W2 = whole(T, K), whole(8, 2 * I, K) * 0.125, whole(1, 2 * I, K) * 0.125, whole(1, 72, 2 * I)
    off1 = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    off8 = torch.tensor([0] + [T] * 8, dtype=torch.int32, device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    new = lambda n: torch.empty((T, n), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y1, y2, z, h1, h2 = new(2 * I), new(2 * I), new(72), new(I), new(I)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    bf = m.DT_BF16

    def work(wait):
        step = torch.cuda.synchronize if wait else (lambda: None)
        fork = torch.cuda.Event()
        fork.record(a)
        b.wait_event(fork)
        m.moe_grouped_matmul(bf, x, off8, W, T, 8, 2 * I, K, y2, st[:1], stream=b)
        for _ in range(3):  # (the other stream's result comes late, and changes on the way)
            m.moe_grouped_matmul(bf, y2, off1, W2, T, 1, 72, 2 * I, z, st[:1], stream=b)
            m.moe_grouped_matmul(bf, x, off8, W, T, 8, 2 * I, K, y2, st[:1], stream=b)
        step()
        m.moe_grouped_matmul(bf, x, off1, Ws, T, 1, 2 * I, K, y1, st[1:], stream=a)
        step()
        join = torch.cuda.Event()
        join.record(b)
        a.wait_event(join)
        m.moe_swiglu(bf, y2, None, None, 0, T, I, h2, stream=a)
        step()
        m.moe_swiglu(bf, y1, None, None, 0, T, I, h1, stream=a)
        step()

    want = []
    for v in xs:
        x.copy_(v)
        torch.cuda.synchronize()
        work(True)
        want.append((h1.clone(), h2.clone()))
    assert not torch.equal(want[0][1], want[1][1])
    torch.cuda.synchronize()
    if captured:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=a):
            work(False)
        run = gr.replay
    else:
        def run():
            work(False)
    for k in range(20):
        with torch.cuda.stream(a):
            x.copy_(xs[k % 2])
            run()
        torch.cuda.synchronize()
        assert torch.equal(h1, want[k % 2][0]) and torch.equal(h2, want[k % 2][1]), k
    assert st.tolist() == [0, 0]


def test_threads_call_at_once():
    """Four threads, each with its stream, workspace and results, on the same matrices: every operator's first call among
    them (attributes of a kernel are set by whoever comes first)."""
    m = _m()
    N, K, T = 264, 512, 40
    t, _ = packed(1, N, K, 4, 64)
    Q = qtensor(m, t, N, K, 4, 64)
    g = torch.Generator(device="cuda").manual_seed(2)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    x, dy, W, gu = mk(T, K), mk(T, N), mk(3, N, K), mk(T, 2 * 100)
    xb, dyb = x.bfloat16(), dy.bfloat16()
    off = torch.tensor([0, 7, 7, T], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    results, errors = [None] * 5, []

    def call(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                st = torch.zeros(1, dtype=torch.int32, device="cuda")
                nb = max(m.moe_affine_linear_workspace_bytes(Q, T), m.moe_affine_linear_dx_workspace_bytes(Q, T))
                ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
                m.moe_workspace_init(ws, nb)
                new = lambda *sh, t=torch.float16: torch.zeros(sh, dtype=t, device="cuda")  # noqa: E731
                y, dx, dw, h = new(T, N), new(T, K), new(3, N, K, t=torch.float32), new(T, 100)
                yl, dxl = new(T, N, t=torch.bfloat16), new(T, K, t=torch.bfloat16)
                for _ in range(30):
                    m.moe_grouped_matmul(m.DT_F16, x, off, W, T, 3, N, K, y, st)
                    m.moe_grouped_matmul_dx(m.DT_F16, dy, off, W, T, 3, N, K, dx, st)
                    m.moe_grouped_matmul_dw(m.DT_F16, dy, x, off, T, 3, N, K, m.DT_F32, 0, dw, st)
                    m.moe_swiglu(m.DT_F16, gu, None, None, 0, T, 100, h)
                    m.moe_affine_linear(Q, xb, T, yl, ws, nb)
                    m.moe_affine_linear_dx(Q, dyb, T, dxl, ws, nb)
                s.synchronize()
                assert int(st.item()) == 0 and m.moe_get_device_status(ws) == 0
                results[i] = (y, dx, dw, h, yl, dxl)
        except BaseException as e:  # noqa: BLE001 (reported by the test below)
            errors.append(e)

    threads = [threading.Thread(target=call, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    call(4)
    for i in range(4):
        assert all(torch.equal(u, v) for u, v in zip(results[i], results[4]))
