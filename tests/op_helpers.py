"""Plain 64-bit forms of the linear, grouped and SwiGLU operators, and the error bounds their tests use.

Bounds.  `HALF[t]` is the largest relative error of one rounding to type t.  A tensor-core sum of n products adds
16 of them per step into an fp32 accumulator; each addition errs by at most one unit of the last place of a partial
sum (2^-23 of it, the accumulation may truncate), and no partial sum exceeds the sum of the products' magnitudes A:
at most (n / 16 + 1) steps plus 16 inner terms' alignment, taken as (n / 8 + 8) * 2^-23 * A."""
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {t: torch.finfo(d).eps / 2 for t, d in DTYPES.items()}


def sum_err(n, A):
    return (n / 8 + 8) * 2.0 ** -23 * A


def assert_within(got, want, tol, what=""):
    """|got - want| <= tol element by element (got any float type, want and tol fp64)."""
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    if bool(bad.any()):
        i = int((d - tol).flatten().nan_to_num(nan=float("inf")).argmax())
        raise AssertionError("%s: %d of %d off; worst at %d: got %r, want %r, off by %.3e, allowed %.3e" % (
            what, int(bad.sum()), bad.numel(), i, got.flatten()[i].item(), want.flatten()[i].item(),
            d.flatten()[i].item(), tol.flatten()[i].item()))


def offsets_of(sizes, first=0):
    return torch.tensor([first] + [first + int(v) for v in torch.tensor(sizes).cumsum(0)], dtype=torch.int32)


def grouped_ref(kind, off, x=None, W=None, dy=None, G=None):
    """(result, sum of the products' magnitudes, longest sum) in 64 bits; rows of no group are zero."""
    off = [int(v) for v in off]
    G = len(off) - 1
    if kind == "dw":
        out = torch.zeros((G, dy.shape[1], x.shape[1]), dtype=torch.float64, device=x.device)
    else:
        src = x if kind == "fwd" else dy
        out = torch.zeros((src.shape[0], W.shape[1] if kind == "fwd" else W.shape[2]), dtype=torch.float64,
                          device=src.device)
    mag, n = torch.zeros_like(out), 0
    for g in range(G):
        r = slice(off[g], off[g + 1])
        if off[g] >= off[g + 1]:
            continue
        if kind == "fwd":
            a, b, at = x[r].double(), W[g].double().t(), r
        elif kind == "dx":
            a, b, at = dy[r].double(), W[g].double(), r
        else:
            a, b, at = dy[r].double().t(), x[r].double(), g
        out[at], mag[at] = a @ b, a.abs() @ b.abs()
        n = max(n, a.shape[1])
    return out, mag, n


def packed(seed, N, K, bits, group, device="cuda", std=0.02):
    """Random packed words, scales and biases with the ranges of N(0, std) weights, and s, q, b in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 2 ** bits, (N, K), generator=g)
    s = (std * 5 / (2 ** bits - 1) * (0.6 + 0.8 * torch.rand((N, K // group), generator=g))).bfloat16()
    b = (-std * 2.5 * (0.6 + 0.8 * torch.rand((N, K // group), generator=g))).bfloat16()
    per = 32 // bits
    u = (q.view(N, K // per, per) << (torch.arange(per) * bits)).sum(2)
    words = torch.where(u >= 1 << 31, u - (1 << 32), u).to(torch.int32)
    rep = lambda v: v.double().repeat_interleave(group, 1)  # noqa: E731
    return (words.to(device), s.to(device), b.to(device)), (rep(s).to(device), q.double().to(device),
                                                           rep(b).to(device))


def qtensor(m, t, N, K, bits, group):
    q = m.QTensor()
    q.packed, q.scales, q.biases = (v.data_ptr() for v in t)
    q.n, q.out, q.in_, q.bits, q.group = 1, N, K, bits, group
    return q


def swiglu_ref(gu, w, dh=None):
    """h, or (dgu, dw), in 64 bits; w None: ones."""
    I = gu.shape[1] // 2
    g, u = gu[:, :I].double(), gu[:, I:].double()
    w = torch.ones(gu.shape[0], dtype=torch.float64, device=gu.device) if w is None else w.double()
    s = torch.sigmoid(g)
    if dh is None:
        return w[:, None] * g * s * u
    d = dh.double()
    return (torch.cat([w[:, None] * d * u * s * (1 + g * (1 - s)), w[:, None] * d * g * s], 1),
            (d * g * s * u).sum(1), (d * g * s * u).abs().sum(1))
