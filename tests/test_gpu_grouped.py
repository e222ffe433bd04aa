"""Products grouped by expert against the definition in 64 bits.

Tolerances, per element, from the arithmetic: a product's terms are summed in
fp32 in k / 16 instructions, each adding at most 2^-23 of the running sum of
magnitudes (and a few times that inside the instruction), so the sum is off by
at most (k / 16 + 8) 2^-23 sum |x| |w|; the result is rounded once to its
type, half a step eps / 2 of its value (fp16: plus half a step 2^-25 of its
subnormals). alpha and beta add two fp32 roundings.
"""

import numpy as np
import pytest
import torch

from newton_schulz_10_b200 import muon as mu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def offsets_of(counts, first=0):
    return torch.tensor(np.cumsum([first, *counts]), dtype=torch.int32, device="cuda")


def padded(t, extra=8):
    """The same values with rows that are `extra` (and up to a 16-byte step) wider in memory, NaN behind."""
    width = (t.shape[-1] + extra + 7) // 8 * 8
    wide = torch.full((*t.shape[:-1], width), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def draw(shape, std, dtype, seed, pad=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(shape, generator=g, device="cuda") * std
    t = t.to(dtype)
    return padded(t) if pad or shape[-1] % 8 else t


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, magnitude, terms, dtype):
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    tol = half_step(dtype) * want.abs() + (1 + half_step(dtype)) * (terms / 16 + 8) * 2.0 ** -23 * magnitude + tiny
    off = (got.double() - want).abs()
    worst = (off / tol.clamp_min(1e-300)).max().item() if off.numel() else 0.0
    assert bool((off <= tol).all()), f"{worst:.3g} times the tolerance"


def rows_ref(x, w, off, transpose):
    """(rows, product, sum of magnitudes) per expert"""
    o = off.tolist()
    for e in range(len(o) - 1):
        r = slice(o[e], o[e + 1])
        W = w[e].double()
        W = W.T if transpose else W
        yield r, x[r].double() @ W, x[r].double().abs() @ W.abs()


COUNTS = {
    "one_token": [1],
    "decode": [1, 0, 1, 2, 0, 0, 1, 3],
    "tiles": [31, 32, 33, 0, 64, 65, 1],
    "wide": [255, 256, 257, 0, 513, 1],
    "skewed": [0, 0, 1100, 3, 0, 17, 0],
    "long": [1300, 700],
}
SIZES = {"small": (64, 64), "ragged": (200, 136), "odd": (77, 91), "narrow": (5, 3), "wide": (640, 1032)}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("counts", list(COUNTS))
def test_rows_products(cuda, counts, size, dtype):
    n, k = SIZES[size]
    c = COUNTS[counts]
    d = DT[dtype]
    off = offsets_of(c, first=3)
    total = 3 + sum(c) + 5
    x, w, dy = draw((total, k), 1.0, d, 1), draw((len(c), n, k), 0.1, d, 2), draw((total, n), 1.0, d, 3)
    # rows of no expert hold NaN: none of it may reach a result
    x[:3], x[total - 5:], dy[:3], dy[total - 5:] = (float("nan"),) * 4
    y = draw((total, n), 1.0, d, 4)
    dx = draw((total, k), 1.0, d, 5)
    y0, dx0 = y.clone(), dx.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert mu.grouped_matmul(x, w, off, out=y, dev_status=status) is y
    assert mu.grouped_matmul_dx(dy, w, off, out=dx, dev_status=status) is dx
    for r, want, mag in rows_ref(x, w, off, True):
        close(y[r], want, mag, k, d)
    for r, want, mag in rows_ref(dy, w, off, False):
        close(dx[r], want, mag, n, d)
    for out, before in ((y, y0), (dx, dx0)):
        assert torch.equal(out[:3], before[:3]) and torch.equal(out[total - 5:], before[total - 5:])
    assert int(status.item()) == mu.OK


def dw_ref(dy, x, off, alpha, beta, old):
    o = off.tolist()
    want, mag = [], []
    for e in range(len(o) - 1):
        r = slice(o[e], o[e + 1])
        want.append(alpha * (dy[r].double().T @ x[r].double()))
        mag.append(abs(alpha) * (dy[r].double().abs().T @ x[r].double().abs()))
    want, mag = torch.stack(want), torch.stack(mag)
    if beta:
        want = want + beta * old.double()
    return want, mag


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("alpha,beta", [(1.0, 0.0), (0.5, 0.95)])
def test_weight_gradient(cuda, counts, size, dtype, out, alpha, beta):
    n, k = SIZES[size]
    c = COUNTS[counts]
    d = DT[dtype]
    o = torch.float32 if out == "f32" else d
    off = offsets_of(c, first=3)
    total = 3 + sum(c) + 5
    x, dy = draw((total, k), 1.0, d, 6), draw((total, n), 1.0, d, 7)
    x[:3], x[total - 5:], dy[:3], dy[total - 5:] = (float("nan"),) * 4
    dw = draw((len(c), n, k), 1.0, o, 8)
    old = dw.clone()
    if beta == 0.0:
        dw.fill_(float("nan"))  # not read
    wide = dw._base if dw._base is not None else None
    mu.grouped_matmul_dw(dy, x, off, out=dw, alpha=alpha, beta=beta)
    want, mag = dw_ref(dy, x, off, alpha, beta, old)
    tol = half_step(o) * want.abs() + 2.0 ** -22 * (want.abs() + abs(beta) * old.double().abs())
    tol += 1.01 * (max(c) / 16 + 8) * 2.0 ** -23 * mag + (2.0 ** -25 if o == torch.float16 else 0.0)
    off_by = (dw.double() - want).abs()
    assert bool((off_by <= tol).all()), (off_by / tol.clamp_min(1e-300)).max().item()
    if wide is not None:
        assert bool(wide[..., k:].isnan().all())  # nothing behind the rows is written


@pytest.mark.parametrize("dtype", list(DT))
def test_neighbours_do_not_mix(cuda, dtype):
    """NaN and infinities of one expert stay in its own rows and its own gradient."""
    d = DT[dtype]
    c = [37, 50, 70]
    off = offsets_of(c)
    x, w, dy = draw((157, 72), 1.0, d, 1), draw((3, 80, 72), 1.0, d, 2), draw((157, 80), 1.0, d, 3)
    y, dx = mu.grouped_matmul(x, w, off), mu.grouped_matmul_dx(dy, w, off)
    dw = mu.grouped_matmul_dw(dy, x, off)
    x[37], x[86], dy[50], w[1, 3] = float("nan"), float("inf"), float("-inf"), float("nan")
    y2, dx2 = mu.grouped_matmul(x, w, off), mu.grouped_matmul_dx(dy, w, off)
    dw2 = mu.grouped_matmul_dw(dy, x, off)
    keep = torch.cat([torch.arange(37), torch.arange(87, 157)]).cuda()
    assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
    assert torch.equal(dw2[[0, 2]], dw[[0, 2]])
    assert bool(y2[37].isnan().all()) and bool(y2[38, 3].isnan()) and not bool(y2[38, :3].isnan().any())


@pytest.mark.parametrize("experts,tokens", [(1024, 5000), (1000, 40), (2, 0), (1, 4097)])
def test_many_and_few_experts(cuda, experts, tokens):
    g = torch.Generator().manual_seed(experts)
    c = torch.bincount(torch.randint(0, experts, (tokens,), generator=g), minlength=experts).tolist()
    off = offsets_of(c)
    d = torch.bfloat16
    x, w, dy = draw((tokens, 40), 1.0, d, 1), draw((experts, 24, 40), 1.0, d, 2), draw((tokens, 24), 1.0, d, 3)
    y, dx, dw = mu.grouped_matmul(x, w, off), mu.grouped_matmul_dx(dy, w, off), mu.grouped_matmul_dw(dy, x, off)
    e = torch.repeat_interleave(torch.arange(experts), torch.tensor(c, dtype=torch.int64)).cuda()
    want = torch.einsum("tk,tnk->tn", x.double(), w.double()[e])
    close(y, want, torch.einsum("tk,tnk->tn", x.double().abs(), w.double()[e].abs()), 40, d)
    want = torch.einsum("tn,tnk->tk", dy.double(), w.double()[e])
    close(dx, want, torch.einsum("tn,tnk->tk", dy.double().abs(), w.double()[e].abs()), 24, d)
    outer = dy.double()[:, :, None] * x.double()[:, None, :]
    want = torch.zeros(experts, 24, 40, dtype=torch.float64, device="cuda").index_add_(0, e, outer)
    mag = torch.zeros_like(want).index_add_(0, e, outer.abs())
    assert bool(((dw.double() - want).abs() <= 2.0 ** -24 * want.abs() + (max(c) / 16 + 8) * 2.0 ** -23 * mag).all())


def test_views_of_larger_tensors(cuda):
    """Column blocks of x and y, row blocks of a fused weight (gate and up), a slice of the experts."""
    d = torch.bfloat16
    c = [70, 0, 33]
    off = offsets_of(c)
    X, Y = draw((103, 256), 1.0, d, 1), draw((103, 320), 1.0, d, 2)
    W = draw((5, 2 * 96, 128), 0.1, d, 3)
    x, y, up = X[:, 64:192], Y[:, 160:256], W[1:4, 96:]
    before = Y.clone()
    mu.grouped_matmul(x, up, off, out=y)
    for r, want, mag in rows_ref(x, up, off, True):
        close(y[r], want, mag, 128, d)
    assert torch.equal(Y[:, :160], before[:, :160]) and torch.equal(Y[:, 256:], before[:, 256:])
    G = torch.zeros((5, 2 * 96, 128), dtype=torch.float32, device="cuda")
    mu.grouped_matmul_dw(y, x, off, out=G[1:4, 96:])
    want, mag = dw_ref(y, x, off, 1.0, 0.0, None)
    assert bool(((G[1:4, 96:].double() - want).abs() <= 2.0 ** -24 * want.abs() + 20 * 2.0 ** -23 * mag).all())
    G[1:4, 96:] = 0
    assert not bool(G.any())


def test_graph_replay_reads_new_offsets(cuda):
    d = torch.bfloat16
    x, w, dy = draw((300, 128), 1.0, d, 1), draw((4, 96, 128), 0.1, d, 2), draw((300, 96), 1.0, d, 3)
    off = offsets_of([100, 100, 50, 50])
    y, dx = torch.zeros((300, 96), dtype=d, device="cuda"), torch.zeros((300, 128), dtype=d, device="cuda")
    dw, ws = torch.zeros((4, 96, 128), device="cuda"), mu.workspace(mu.grouped_workspace_size(4))

    def calls():
        mu.grouped_matmul(x, w, off, out=y)
        mu.grouped_matmul_dx(dy, w, off, out=dx)
        mu.grouped_matmul_dw(dy, x, off, out=dw, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for counts in ([100, 100, 50, 50], [0, 7, 260, 1], [300, 0, 0, 0], [0, 0, 0, 0]):
        off.copy_(offsets_of(counts))
        for t in (y, dx, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw)]
        for t in (y, dx, dw):
            t.zero_()
        calls()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, dx, dw)):
            assert torch.equal(a, b)
        r = sum(counts)
        assert not bool(y[r:].any()) and not bool(dx[r:].any())


def test_on_another_stream_and_repeated(cuda):
    """A call on a stream of its own sees what that stream wrote; the same call twice gives the same bits."""
    d = torch.float16
    x, w, off = draw((500, 264), 1.0, d, 1), draw((6, 320, 264), 0.1, d, 2), offsets_of([90, 0, 200, 10, 150, 50])
    want = mu.grouped_matmul(x, w, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x2 = torch.zeros_like(x)
    with torch.cuda.stream(s):
        x2.copy_(x)
        got = mu.grouped_matmul(x2, w, off)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(mu.grouped_matmul(x, w, off), want)


@pytest.mark.parametrize("bad", [[0, 30, 20, 40], [0, 10, 20, 41], [-1, 10, 20, 30], [0, 10, 2 ** 31 - 1, 40], [40, 30, 20, 10]])
def test_bad_offsets_are_reported(cuda, bad):
    """Entries out of range or decreasing: an error in the status word, nothing outside the matrices touched."""
    d = torch.bfloat16
    X, Y = draw((60, 64), 1.0, d, 1), draw((60, 64), 1.0, d, 2)
    w = draw((3, 64, 64), 0.1, d, 3)
    x, y = X[10:50], Y[10:50]
    before = Y.clone()
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for call in (lambda s: mu.grouped_matmul(x, w, off, out=y, dev_status=s), lambda s: mu.grouped_matmul_dx(x, w, off, out=y, dev_status=s),
                 lambda s: mu.grouped_matmul_dw(x, x, off, dev_status=s)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(status)
        assert int(status.item()) == mu.ERR_INVALID_ARG
    assert torch.equal(Y[:10], before[:10]) and torch.equal(Y[50:], before[50:])


def test_gradients_against_differences(cuda):
    """loss = sum(y * c): its differences along random directions of x and W are the products with dx and dW.
    The loss is linear in each, so a central difference has no error but the roundings of y (bf16, half a step of
    each of its values, random: 2^-8 sqrt(sum (c y)^2) a side would be large against a small step; the step is as
    large as the inputs) and of dx."""
    d = torch.float16
    c = [40, 0, 21]
    off = offsets_of(c)
    x, w, cot = draw((61, 96), 1.0, d, 1), draw((3, 80, 96), 0.1, d, 2), draw((61, 80), 1.0, d, 3)
    dx, dw = mu.grouped_matmul_dx(cot, w, off), mu.grouped_matmul_dw(cot, x, off)
    ux, uw = draw((61, 96), 1.0, d, 4), draw((3, 80, 96), 0.1, d, 5)

    def loss(x_, w_):
        return (mu.grouped_matmul(x_, w_, off).double() * cot.double()).sum().item()

    # exact in fp16: x +- u halves are rounded, so differentiate along the rounded points
    for a, b, grad in (((x + ux, w), (x - ux, w), dx), ((x, w + uw), (x, w - uw), dw)):
        delta = (a[0].double() - b[0].double(), a[1].double() - b[1].double())
        slope = (grad.double() * (delta[0] if grad is dx else delta[1])).sum().item()
        ya, yb = mu.grouped_matmul(*a, off).double(), mu.grouped_matmul(*b, off).double()
        # half a step of every y and of every dx, all of one sign at worst
        tol = 2.0 ** -11 * ((ya.abs() + yb.abs()) * cot.double().abs()).sum().item()
        if grad is dx:
            tol += 2.0 ** -11 * (dx.double().abs() * delta[0].abs()).sum().item()
        assert abs(loss(*a) - loss(*b) - slope) <= 1.01 * tol


def test_long_sums_keep_fp32(cuda):
    """Thousands of rows in one expert: parts of 512 rows, each losing at most 2^-24 of its running sum in each of its
    32 instructions. A sum of random signs grows like a square root, so the running sum is 2/3 of the part's on
    average, and a truncation loses half a step on average: 32 * 2^-24 * 2/3 * 1/2 of the part, and less than that of
    the whole once parts add up: below 2^-20. The additions of parts are rounded to nearest, 2^-24 each."""
    d = torch.bfloat16
    c = [5000, 1024, 1025, 3, 2049]
    total = sum(c)
    off = offsets_of(c)
    x, dy = draw((total, 72), 1.0, d, 1), draw((total, 264), 1.0, d, 2)
    old = draw((5, 264, 72), 1.0, torch.float32, 3)
    for beta in (0.0, 0.95):
        dw = old.clone()
        mu.grouped_matmul_dw(dy, x, off, out=dw, beta=beta)
        want, _ = dw_ref(dy, x, off, 1.0, beta, old)
        for e in range(5):
            assert (dw[e].double() - want[e]).norm() <= 2.0 ** -20 * want[e].norm()


@pytest.mark.parametrize("rows", [512, 16384])
def test_short_device_wait_is_reported(cuda, rows):
    """A wait bound of nothing: every role stops, copies and products in flight are drained, the context stays usable.
    A wait looks twice (and each look lasts up to the hardware's own limit) before it reads the clock, so a product of
    a few k-blocks (dx here, and dW in its parts of 768 rows) may end in time; one over 8192 columns, tens of
    microseconds, cannot."""
    d = torch.bfloat16
    off = offsets_of([300, rows - 300])
    x, w, dy = draw((rows, 8192), 1.0, d, 1), draw((2, 512, 8192), 0.02, d, 2), draw((rows, 512), 1.0, d, 3)
    calls = [(lambda st: mu.grouped_matmul(x, w, off, dev_status=st), True), (lambda st: mu.grouped_matmul_dx(dy, w, off, dev_status=st), False),
             (lambda st: mu.grouped_matmul_dw(dy, x, off, dev_status=st), False)]
    for call, surely in calls:
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mu.set_wait_timeout_ns(1)
        try:
            call(status)
            torch.cuda.synchronize()
        finally:
            mu.set_wait_timeout_ns(0)
        assert int(status.item()) == mu.ERR_TIMEOUT or (not surely and int(status.item()) == mu.OK)
        status.zero_()
        call(status)
        assert int(status.item()) == mu.OK
    for r, want, mag in rows_ref(x, w, off, True):
        close(mu.grouped_matmul(x, w, off)[r], want, mag, 8192, d)


def test_weight_gradient_on_another_stream_without_a_workspace(cuda):
    """The workspace that the call makes for itself belongs to the stream that uses it."""
    d = torch.bfloat16
    x, dy, off = draw((5000, 256), 1.0, d, 1), draw((5000, 256), 1.0, d, 2), offsets_of([3000, 2000])
    want = mu.grouped_matmul_dw(dy, x, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(8):
        out = torch.zeros((2, 256, 256), device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        mu.grouped_matmul_dw(dy, x, off, out=out, stream=s)
        torch.full((6_000_000,), float("nan"), device="cuda")  # would land in a workspace freed on this stream
        got.append(out)
    raw = torch.zeros((2, 256, 256), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    mu.grouped_matmul_dw(dy, x, off, out=raw, stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(g, want) for g in got) and torch.equal(raw, want)


@pytest.mark.parametrize("counts", [[2000, 1000, 0, 500], [0, 0, 3500, 0]])
def test_graph_replay_of_cut_sums(cuda, counts):
    """Few tiles over many rows: the sums are cut into parts; a captured call follows the offsets it finds."""
    d = torch.float16
    x, dy = draw((3500, 72), 1.0, d, 1), draw((3500, 136), 1.0, d, 2)
    off = offsets_of([875, 875, 875, 875])
    dw, ws = draw((4, 136, 72), 1.0, torch.float32, 3), mu.workspace(mu.grouped_workspace_size(4))
    old = dw.clone()
    mu.grouped_matmul_dw(dy, x, off, out=dw, beta=0.5, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mu.grouped_matmul_dw(dy, x, off, out=dw, beta=0.5, ws=ws)
    off.copy_(offsets_of(counts))
    dw.copy_(old)
    graph.replay()
    torch.cuda.synchronize()
    want, mag = dw_ref(dy, x, off, 1.0, 0.5, old)
    assert bool(((dw.double() - want).abs() <= 2.0 ** -22 * (want.abs() + old.double().abs()) + (max(counts) / 16 + 8) * 2.0 ** -23 * mag).all())


def test_two_calls_at_once(cuda):
    """Two streams, each with its own outputs and workspace, on the same inputs."""
    d = torch.bfloat16
    x, dy, w = draw((3000, 512), 1.0, d, 1), draw((3000, 384), 1.0, d, 2), draw((5, 384, 512), 0.05, d, 3)
    off = offsets_of([700, 0, 1500, 300, 500])
    want = (mu.grouped_matmul(x, w, off), mu.grouped_matmul_dx(dy, w, off), mu.grouped_matmul_dw(dy, x, off))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((mu.grouped_matmul(x, w, off), mu.grouped_matmul_dx(dy, w, off), mu.grouped_matmul_dw(dy, x, off)))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("which", ["y", "dx", "dw"])
def test_results_on_another_stream_are_its_own(cuda, which):
    """A result that a call makes for itself does not take memory that this stream still reads."""
    d = torch.bfloat16
    x, w, off = draw((512, 256), 1.0, d, 1), draw((2, 256, 256), 0.1, d, 2), offsets_of([300, 212])
    call = {"y": lambda **k: mu.grouped_matmul(x, w, off, **k), "dx": lambda **k: mu.grouped_matmul_dx(x, w, off, **k),
            "dw": lambda **k: mu.grouped_matmul_dw(x, x, off, **k)}[which]
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        old = torch.ones_like(want)
        s.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(20_000_000)  # this stream is some milliseconds behind
        read = old.clone()
        del old
        got = call(stream=stream)
        torch.cuda.synchronize()
        assert bool((read == 1).all()) and torch.equal(got, want)


@pytest.mark.parametrize("bad", [[0, 40, 0, 40], [0, 30, 20, 40], [-1, 10, 20, 30], [0, 10, 20, 41]])
def test_bad_offsets_leave_the_rows_alone(cuda, bad):
    d = torch.float16
    x, w = draw((40, 64), 1.0, d, 1), draw((3, 64, 64), 0.1, d, 2)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for call in (mu.grouped_matmul, mu.grouped_matmul_dx):
        y, status = torch.full_like(x, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        call(x, w, off, out=y, dev_status=status)
        assert int(status.item()) == mu.ERR_INVALID_ARG and bool((y == 7.0).all())


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("k", [40, 64, 91, 200, 1032])
def test_many_tiles_with_an_odd_number_of_blocks(cuda, k, dtype, out):
    """Several tiles a CTA pair, whose last one leaves each storing warp an odd number of 32-column blocks (1 or 3; none
    for one half of the warps at k = 1032), with empty, short and long experts in turn: the blocks of a tile may not
    overwrite those of the tile before while they are being stored. Repeated, since that would depend on timing."""
    d = DT[dtype]
    o = torch.float32 if out == "f32" else d
    n, c = 1024, [0, 1, 0, 0, 70, 1600, 33, 0] * 8
    off = offsets_of(c)
    total = sum(c)
    x, dy = draw((total, k), 1.0, d, 1), draw((total, n), 1.0, d, 2)
    first = mu.grouped_matmul_dw(dy, x, off, out=draw((len(c), n, k), 1.0, o, 3))
    at = off.tolist()
    for e in range(len(c)):
        r = slice(at[e], at[e + 1])
        want, mag = dy[r].double().T @ x[r].double(), dy[r].double().abs().T @ x[r].double().abs()
        tol = (half_step(o) + 2.0 ** -22) * want.abs() + 1.01 * (c[e] / 16 + 8) * 2.0 ** -23 * mag
        tol += 2.0 ** -25 if o == torch.float16 else 0.0
        assert bool(((first[e].double() - want).abs() <= tol).all()), e
    ws, again = mu.workspace(mu.grouped_workspace_size(len(c))), draw((len(c), n, k), 1.0, o, 4)
    for _ in range(20):
        again.fill_(float("nan"))
        mu.grouped_matmul_dw(dy, x, off, out=again, ws=ws)
        assert torch.equal(again, first)


def test_as_many_rows_as_fit_32_bits(cuda):
    """2^31 - 513 rows, nearly all of them one expert's: the same 2^20 rows of x and dy over and over."""
    d = torch.bfloat16
    total, block, width = 2 ** 31 - 513, 1 << 20, 8
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 4 * 2 * width * total:
        pytest.skip("needs 140 GB")
    base_x, base_dy, w = draw((block, width), 1.0, d, 1), draw((block, width), 1.0, d, 2), draw((3, width, width), 0.5, d, 3)
    cut = [0, 5, total - 70, total - 7]
    off = torch.tensor(cut, dtype=torch.int32, device="cuda")
    x, dy, out = (torch.empty((total, width), dtype=d, device="cuda") for _ in range(3))
    for t, base in ((x, base_x), (dy, base_dy)):
        for r in range(0, total, block):
            t[r:r + block] = base[:total - r]
    for call, src, transpose in ((mu.grouped_matmul, x, True), (mu.grouped_matmul_dx, dy, False)):
        out[total - 7:] = 3.0
        call(src, w, off, out=out)
        assert bool((out[total - 7:] == 3.0).all())
        for e in range(3):
            W = w[e].double().T if transpose else w[e].double()
            for r in range(cut[e], cut[e + 1], block * 300 + 12345):  # here and there, and the end
                for a in (r, max(cut[e], cut[e + 1] - 4096)):
                    rows = slice(a, min(a + 4096, cut[e + 1]))
                    close(out[rows], src[rows].double() @ W, src[rows].double().abs() @ W.abs(), width, d)
    del out
    dw = mu.grouped_matmul_dw(dy, x, off)
    whole = base_dy.double().T @ base_x.double()
    left = total % block
    want = (total // block) * whole + base_dy[:left].double().T @ base_x[:left].double()
    ends = [dy[a:b].double().T @ x[a:b].double() for a, b in ((0, 5), (total - 70, total - 7))]
    tail = dy[total - 7:].double().T @ x[total - 7:].double()
    want = torch.stack([ends[0], want - ends[0] - ends[1] - tail, ends[1]])
    # sums of at most 768 rows as elsewhere; then at most 2^28 / 768 additions of them, rounded to nearest (half a step of a
    # sum that is largest at the end), and one for each of at most 16 parts
    adds = (total / 16 + 64) / 768 + 16
    mag = torch.stack([ends[0].abs(), (total // block + 1) * (base_dy.double().abs().T @ base_x.double().abs()), ends[1].abs()])
    mag[0], mag[2] = dy[:5].double().abs().T @ x[:5].double().abs(), dy[total - 70:total - 7].double().abs().T @ x[total - 70:total - 7].double().abs()
    tol = (768 / 16 + 8) * 2.0 ** -23 * mag + adds * 2.0 ** -24 * want.abs().max()
    assert bool(((dw.double() - want).abs() <= tol).all())
    assert ((dw[1].double() - want[1]).norm() <= 0.05 * want[1].norm())
    del x, dy
    torch.cuda.empty_cache()
