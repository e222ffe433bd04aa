"""The update of stacks of matrices against its formulas in 64 bits.

Tolerances of O are the framework's own, relative in the Frobenius norm:
1e-4 for two fp16 planes (the bound of the fp32 paths: every rounding of that
chain is 2^-11 of the fp16 chain's, which stays below 1e-2; its sums' own
roundings come on top and grow with their length: measured 1e-5 up to n = 256,
about the largest here, and 1e-4 at 4096) and for fp32, 2e-2 for bf16 and fp16. An element of O is then off by at most tol ||O||_F. The
update adds one rounding to W's type (half a step) and two fp32 roundings of
the sum's terms (2^-23 of each).
"""

import math

import pytest
import torch

from newton_schulz_10_b200 import muon as mu

pytestmark = pytest.mark.gpu

ABC = (3.4445, -4.7750, 2.0315)
TOL = {mu.F16X2: 1e-4, mu.F32: 1e-4, mu.BF16: 2e-2, mu.F16: 2e-2}
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def polar(X, eps=1e-7, T=5):
    a, b, c = ABC
    X = X.double()
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT if tall else X
    norm = X.square().sum((-2, -1), keepdim=True).sqrt()
    X = torch.where(norm > 0, X / (norm + eps), torch.zeros_like(X))
    for _ in range(T):
        A = X @ X.mT
        X = a * X + (b * A + c * A @ A) @ X
    return X.mT if tall else X


def gauss(shape, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def spectrum(shape, seed, std=1.0):
    """Strong directions over noise, 16 to 1."""
    c, r, m = shape
    k = max(1, min(r, m) // 16)
    low = gauss((c, r, k), seed) @ gauss((c, k, m), seed + 1)
    return (low * (4.0 / math.sqrt(k)) + 0.25 * gauss(shape, seed + 2)) * std


LAYOUTS = ("dense", "padded", "beside", "gap")


def laid_out(t, layout):
    """The same values as a view of a wider tensor of NaN, and that tensor."""
    c, r, m = t.shape
    if layout == "dense":
        return t.clone(), None
    if layout == "padded":  # rows 5 elements wider, 3 rows between matrices
        wide = torch.full((c, r + 3, m + 5), float("nan"), dtype=t.dtype, device=t.device)
        view = wide[:, :r, :m]
    elif layout == "beside":  # column blocks of one matrix
        wide = torch.full((r, c * m + 7), float("nan"), dtype=t.dtype, device=t.device)
        view = wide[:, :c * m].view(r, c, m).permute(1, 0, 2)
    else:  # rows 8 elements wider: aligned vectors with a gap
        wide = torch.full((c, r, (m + 15) // 8 * 8), float("nan"), dtype=t.dtype, device=t.device)
        view = wide[:, :, :m]
    view.copy_(t)
    return view, wide


def rel(a, b):
    return ((a.double() - b).norm() / b.norm().clamp_min(1e-300)).item()


SHAPES = [(1, 1, 1), (3, 1, 40), (2, 40, 1), (3, 64, 64), (5, 33, 200), (4, 200, 33), (2, 130, 257), (12, 64, 768), (2, 520, 264)]


@pytest.mark.parametrize("compute", [mu.F16X2, mu.BF16, mu.F16, mu.F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_orthogonalised_update(cuda, shape, compute):
    """W = 0, lr scale = -1: the new W is O itself."""
    M = spectrum(shape, 11, 1e-3) if compute in (mu.F16X2, mu.F32) else gauss(shape, 11, 1e-3)
    W = torch.zeros(shape, device="cuda")
    step = mu.stack_step([mu.Stack(W, M.clone())], mu.stack_params(lr=1.0, scale=-1.0, ns=mu.ns_params(compute=compute)))
    want = polar(M)
    assert step.device_status() == mu.OK
    for i in range(shape[0]):
        assert rel(W[i], want[i]) <= TOL[compute], i


# matrices that fit on chip, at the edges of the cluster's split: one to eight
# CTAs, the last with few or no columns, both orientations, more matrices than SMs
SMALL = [(1, 128, 2048), (1, 2048, 128), (3, 100, 1000), (40, 16, 2048), (2, 2047, 127), (300, 128, 128), (1, 65, 129),
         (5, 128, 257), (7, 513, 33), (20, 31, 1025), (160, 5, 300)]


@pytest.mark.parametrize("compute", [mu.F16X2, mu.BF16, mu.F16])
@pytest.mark.parametrize("shape", SMALL, ids=str)
def test_small_matrices(cuda, shape, compute):
    M = spectrum(shape, 13, 1e-3) if compute == mu.F16X2 else gauss(shape, 13, 1e-3)
    W0, G = gauss(shape, 14, 0.02), gauss(shape, 15, 1e-3)
    W, Mv = W0.clone(), M.clone()
    p = mu.stack_params(nesterov=True, weight_decay=0.1, scale=-3.0, ns=mu.ns_params(compute=compute))
    before = mu.kernel_launch_count()
    step = mu.StackStep([mu.Stack(W, Mv, G)], p)
    step()
    assert mu.kernel_launch_count() - before == 1
    assert step.device_status() == mu.OK
    check_update(W0, M, G, W, Mv, None, p, TOL[compute])
    want = polar(G.double() + p.mu * Mv.double())
    O = (W.double() - (1 - p.lr * p.weight_decay) * W0.double()) / (3.0 * p.lr)
    for i in range(0, shape[0], 17):
        # W's roundings, three half steps of values below 0.125 (2^-28 each), come back divided by 0.06, beside
        # elements of O of about 0.9 / sqrt(max)
        assert rel(O[i], want[i]) <= TOL[compute] + 3 * 2.0 ** -27 / 0.06 / 0.9 * math.sqrt(max(shape[1:])), i


def test_short_device_wait_is_reported(cuda):
    """A wait bound of nothing: an error in the status word, the context usable, and the right result afterwards."""
    W0, M = gauss((3, 100, 400), 16, 0.02), gauss((3, 100, 400), 17)
    step = mu.StackStep([mu.Stack(W0.clone(), M.clone())], mu.stack_params(ns=mu.ns_params(compute=mu.F16X2)))
    mu.set_wait_timeout_ns(1)
    try:
        step()
        torch.cuda.synchronize()
    finally:
        mu.set_wait_timeout_ns(0)
    assert step.device_status() in (mu.OK, mu.ERR_TIMEOUT)
    again = mu.stack_step([mu.Stack(torch.zeros_like(W0), M.clone())], mu.stack_params(lr=1.0, scale=-1.0, ns=mu.ns_params(compute=mu.F16X2)))
    assert again.device_status() == mu.OK
    assert rel(again.stacks[0].W, polar(M)) <= 1e-4


@pytest.mark.parametrize("gram,compute", [(True, mu.F16), (True, mu.BF16), (True, mu.F32)])
def test_gram_chain(cuda, gram, compute):
    M = gauss((3, 96, 300), 12, 1e-3)
    W = torch.zeros_like(M)
    mu.stack_step([mu.Stack(W, M.clone())], mu.stack_params(lr=1.0, scale=-1.0, ns=mu.ns_params(gram=True, compute=compute)))
    assert rel(W, polar(M)) <= TOL[compute]


def check_update(W0, M0, G, W, M, copy, p, tol):
    lr, wd, sc = p.lr, p.weight_decay, p.scale
    m = M0.double() if G is None else p.mu * M0.double() + G.double()
    assert bool(((M.double() - m).abs() <= 2.0 ** -23 * m.abs() + 2.0 ** -149).all())
    X = G.double() + p.mu * M.double() if p.nesterov else M.double()
    O = polar(X)
    want = (1 - lr * wd) * W0.double() - lr * sc * O
    norm = O.square().sum((-2, -1), keepdim=True).sqrt()
    base = 2.0 ** -22 * (W0.double().abs() + abs(lr * sc) * O.abs()) + abs(lr * sc) * tol * norm
    for got in (W, copy):
        if got is None:
            continue
        tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
        assert bool(((got.double() - want).abs() <= 1.01 * (torch.finfo(got.dtype).eps / 2 * want.abs() + base) + tiny).all())


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("w,g,copy,nesterov,decay", [("f32", "f32", None, False, 0.0), ("f32", "bf16", "bf16", True, 0.1),
                                                     ("bf16", "bf16", None, True, 0.1), ("f16", "f16", "bf16", False, 0.3),
                                                     ("f32", None, "f16", False, 0.1), ("bf16", "f32", None, True, 0.0)])
@pytest.mark.parametrize("shape", [(3, 48, 80), (4, 37, 21), (2, 24, 4100)], ids=str)
@pytest.mark.parametrize("compute", [mu.F16X2, mu.BF16])
def test_whole_update(cuda, shape, w, g, copy, nesterov, decay, layout, compute):
    W0, M0 = gauss(shape, 21, 0.02, DT[w]), gauss(shape, 22, 1e-2)
    G = gauss(shape, 23, 1e-2, DT[g]) if g else None
    (W, Wb), (M, Mb) = laid_out(W0, layout), laid_out(M0, layout)
    Gv, Gb = laid_out(G, layout) if g else (None, None)
    C, Cb = laid_out(torch.zeros(shape, dtype=DT[copy], device="cuda"), layout) if copy else (None, None)
    p = mu.stack_params(mu=0.9, lr=0.01, weight_decay=decay, scale=3.0, nesterov=nesterov, ns=mu.ns_params(compute=compute))
    behind = [(b, b.isnan().sum()) for b in (Wb, Mb, Cb) if b is not None]
    step = mu.stack_step([mu.Stack(W, M, Gv, C)], p)
    assert step.device_status() == mu.OK
    check_update(W0, M0, G, W, M, C, p, TOL[compute])
    for b, n in behind:
        assert torch.equal(b.isnan().sum(), n)  # nothing between the rows is written
    if g:
        assert torch.equal(Gv, G)


def test_several_stacks_and_empty_ones(cuda):
    """More stacks than one launch's shape groups, some empty, each as if alone."""
    shapes = [(2, 40, 24), (0, 8, 8), (3, 24, 40), (1, 64, 200), (4, 0, 16), (1, 200, 64), (2, 96, 96), (1, 17, 5), (2, 3, 0)]
    for compute in (mu.F16X2, mu.BF16):
        p = mu.stack_params(nesterov=True, weight_decay=0.1, ns=mu.ns_params(compute=compute))
        a = [mu.Stack(gauss(s, 31, 0.02), gauss(s, 32), gauss(s, 33)) for s in shapes]
        b = [mu.Stack(k.W.clone(), k.M.clone(), k.G) for k in a]
        step = mu.stack_step(a, p)
        assert step.device_status() == mu.OK
        for x, y in zip(a, b):
            mu.stack_step([y], p)
            assert torch.equal(x.M, y.M)
            # a tile width or a split of K that goes by the launch's size may order the sums differently
            if x.W.numel():
                assert rel(x.W, y.W.double()) <= (1e-6 if compute == mu.F16X2 else 1e-4)


@pytest.mark.parametrize("compute", [mu.F16X2, mu.BF16, mu.F16])
def test_zero_small_and_large_matrices(cuda, compute):
    """A matrix of zeros is left alone (with eps 0 too), a tiny or huge one is orthogonalised like any other."""
    M = gauss((5, 48, 64), 41)
    M[1] = 0
    M[2] *= 1e-6
    M[3] *= 1e15 if compute == mu.BF16 else 1e30
    M[4] = 0
    M[4, 3, 5] = 2.0
    for eps in (1e-7, 0.0):
        W = torch.ones_like(M)
        step = mu.stack_step([mu.Stack(W, M.clone())], mu.stack_params(lr=1.0, scale=-1.0, ns=mu.ns_params(compute=compute, norm_eps=eps)))
        assert step.device_status() == mu.OK
        assert bool((W[1] == 1).all())
        want = polar(M, eps)
        for i in (0, 2, 3, 4):
            # 1 + O in fp32: half a step of 1 an element beside O's own error
            assert (W[i].double() - 1 - want[i]).norm() <= TOL[compute] * want[i].norm() + 2.0 ** -23 * math.sqrt(48 * 64)


def test_nonfinite_matrix_is_reported_and_stays_alone(cuda):
    M = gauss((3, 40, 56), 51)
    W, ref = gauss(M.shape, 52), None
    p = mu.stack_params(ns=mu.ns_params(compute=mu.F16X2))
    good = W.clone()
    mu.stack_step([mu.Stack(good, M.clone())], p)
    M2 = M.clone()
    M2[1, 3, 7] = float("nan")
    W2 = W.clone()
    step = mu.stack_step([mu.Stack(W2, M2)], p)
    assert step.device_status() == mu.ERR_NONFINITE
    assert torch.equal(W2[0], good[0]) and torch.equal(W2[2], good[2])


def test_overflowing_polynomial_is_reported(cuda):
    W, M = torch.zeros((2, 64, 64), device="cuda"), gauss((2, 64, 64), 53)
    for compute in (mu.F16X2, mu.F16):
        step = mu.stack_step([mu.Stack(W.clone(), M.clone())],
                             mu.stack_params(ns=mu.ns_params(compute=compute, coeffs=(3000.0, 0.0, 0.0))))
        assert step.device_status() == mu.ERR_NONFINITE


def test_repeated_gradient_and_single_matrix(cuda):
    """G may be one matrix for the whole stack (stride 0); a padded single matrix is a stack of one."""
    g = gauss((1, 32, 48), 61)
    W0, M0 = gauss((4, 32, 48), 62, 0.02), gauss((4, 32, 48), 63)
    W, M = W0.clone(), M0.clone()
    p = mu.stack_params(nesterov=True, ns=mu.ns_params(compute=mu.F16X2))
    mu.stack_step([mu.Stack(W, M, g.expand(4, 32, 48))], p)
    check_update(W0, M0, g.expand(4, 32, 48), W, M, None, p, TOL[mu.F16X2])


def test_graph_replay_and_two_steps(cuda):
    shapes = [(3, 64, 96), (2, 100, 40)]
    p = mu.stack_params(nesterov=True, weight_decay=0.1, ns=mu.ns_params(compute=mu.F16X2))

    def make():
        return [mu.Stack(gauss(s, 71, 0.02), gauss(s, 72), gauss(s, 73, dtype=torch.bfloat16), gauss(s, 74, dtype=torch.bfloat16)) for s in shapes]

    a, b = make(), make()
    eager, captured = mu.StackStep(a, p), mu.StackStep(b, p)
    warm = mu.StackStep(make(), p)
    warm()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    for _ in range(2):
        eager()
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x.W, y.W) and torch.equal(x.M, y.M) and torch.equal(x.copy, y.copy)


@pytest.mark.parametrize("shape", [(3, 96, 160), (3, 160, 288)], ids=str)
def test_agrees_with_the_matrix_step(cuda, shape):
    """Plain fp32 tensors: the same update as muon_step, matrix by matrix. Larger matrices run the same chain of products
    there and here (the row sums are added in another order, so the scale may differ in its last bit); small ones run on
    chip with other roundings, each side within the type's tolerance of the exact update, so within twice of each other."""
    for compute in (mu.BF16, mu.F16):
        tol = 1e-3 if min(shape[1:]) > 128 else 2 * TOL[compute]
        W, M, G = gauss(shape, 81, 0.02), gauss(shape, 82), gauss(shape, 83)
        a = [(W[i].clone(), M[i].clone(), G[i].clone()) for i in range(3)]
        ns = mu.ns_params(compute=compute)
        mu.muon_step(a, mu.step_params(mu=0.95, lr=0.02, ns=ns))
        W0 = W.clone()
        mu.stack_step([mu.Stack(W, M, G)], mu.stack_params(mu=0.95, lr=0.02, ns=ns))
        for i in range(3):
            assert torch.equal(M[i], a[i][1])
            assert rel(W[i] - W0[i], (a[i][0] - W0[i]).double()) <= tol


@pytest.mark.parametrize("copy", [None, "bf16"])
def test_expert_layer_step(cuda, copy):
    """Together: forward, both gradients (the weights' into the momentum), update of the expert stack."""
    d = torch.bfloat16
    counts = [70, 0, 131, 7]
    off = torch.tensor([0, 70, 70, 201, 208], dtype=torch.int32, device="cuda")
    n, k = 96, 136
    W0 = gauss((4, n, k), 91, 0.05)
    W, M = W0.clone(), gauss((4, n, k), 92, 1e-2)
    M[1] = 0  # the expert without rows never had any
    M0 = M.clone()
    w = W.to(d)
    x, dy = gauss((208, k), 93, dtype=d), gauss((208, n), 94, 1e-2, dtype=d)
    p = mu.stack_params(mu=0.9, lr=0.01, weight_decay=0.1, scale=2.0, ns=mu.ns_params(compute=mu.F16X2))
    step = mu.StackStep([mu.Stack(W, M, None, w if copy else None)], p)
    y, dx = mu.grouped_matmul(x, w, off), mu.grouped_matmul_dx(dy, w, off)
    w_used = w.clone()
    step.accumulate(0, dy, x, off)
    step()
    assert step.device_status() == mu.OK
    m = 0.9 * M0.double()
    for e in range(4):
        r = slice(int(off[e]), int(off[e + 1]))
        assert rel(y[r], x[r].double() @ w_used[e].double().T) <= 2.0 ** -8 if counts[e] else True
        assert rel(dx[r], dy[r].double() @ w_used[e].double()) <= 2.0 ** -8 if counts[e] else True
        m[e] += dy[r].double().T @ x[r].double()
    # p.mu is 0.9 in fp32; sums of up to 131 products and two roundings
    assert (M.double() - m).norm() <= 2.0 ** -21 * m.norm() + (131 / 16 + 8) * 2.0 ** -23 * (dy.double().abs().T @ x.double().abs()).norm()
    assert bool((M[1] == 0).all())
    check_update(W0, M.clone(), None, W, M, w if copy else None, p, TOL[mu.F16X2])
    if copy:
        assert not torch.equal(w, w_used)


def test_on_another_stream(cuda):
    p = mu.stack_params(nesterov=True, ns=mu.ns_params(compute=mu.F16X2))
    W, M, G = gauss((3, 80, 120), 95, 0.02), gauss((3, 80, 120), 96), gauss((3, 80, 120), 97)
    W1, M1 = W.clone(), M.clone()
    mu.stack_step([mu.Stack(W1, M1, G)], p)
    W2, M2, G2 = W.clone(), M.clone(), torch.zeros_like(G)
    step = mu.StackStep([mu.Stack(W2, M2, G2)], p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        G2.copy_(G)
        step()
    s.synchronize()
    assert torch.equal(W1, W2) and torch.equal(M1, M2)


def test_two_updates_at_once(cuda):
    """Two streams, each with its own tensors and workspace: small matrices on chip and larger ones by the chain."""
    p = mu.stack_params(nesterov=True, weight_decay=0.1, ns=mu.ns_params(compute=mu.F16X2))
    shapes = [(6, 64, 200), (2, 200, 330)]

    def make():
        return [mu.Stack(gauss(s, 101, 0.02), gauss(s, 102), gauss(s, 103)) for s in shapes]

    ref = make()
    for _ in range(3):
        mu.stack_step(ref, p)
    sets = [make() for _ in range(2)]
    steps = [mu.StackStep(s, p) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s, step in zip(streams, steps):
            step(stream=s)
    torch.cuda.synchronize()
    for stacks in sets:
        for a, b in zip(stacks, ref):
            assert torch.equal(a.W, b.W) and torch.equal(a.M, b.M)


def test_accumulate_needs_no_gradient_and_nesterov_needs_one(cuda):
    W, M, G = gauss((2, 16, 24), 1), gauss((2, 16, 24), 2), gauss((2, 16, 24), 3)
    off = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    dy, x = gauss((5, 16), 4, dtype=torch.bfloat16), gauss((5, 24), 5, dtype=torch.bfloat16)
    with pytest.raises(mu.MuonError) as err:
        mu.StackStep([mu.Stack(W, M, G)], mu.stack_params()).accumulate(0, dy, x, off)
    assert err.value.code == mu.ERR_INVALID_ARG
    with pytest.raises(mu.MuonError) as err:
        mu.StackStep([mu.Stack(W, M)], mu.stack_params(nesterov=True))()
    assert err.value.code == mu.ERR_INVALID_ARG


def test_workspace_of_a_step_on_another_stream(cuda):
    """stack_step makes its workspace for the stream it runs on: the result may be dropped at once, and memory freed on
    this stream is not written while this stream still reads it."""
    p = mu.stack_params(nesterov=True, ns=mu.ns_params(compute=mu.BF16))
    shape = (3, 200, 300)
    M, G, W = gauss(shape, 95), gauss(shape, 96), gauss(shape, 97, 0.02)
    want, m = W.clone(), M.clone()
    size = mu.stack_step([mu.Stack(want, m, G)], p).ws.numel()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        w, m = W.clone(), M.clone()
        old = torch.ones(size, dtype=torch.uint8, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(20_000_000)  # this stream is some milliseconds behind
        read = old.clone()
        del old
        mu.stack_step([mu.Stack(w, m, G)], p, stream=stream)
        torch.cuda.synchronize()
        assert bool((read == 1).all()) and torch.equal(w, want)
        w, m = W.clone(), M.clone()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        mu.stack_step([mu.Stack(w, m, G)], p, stream=stream)
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # would land in a workspace freed on this stream
        torch.cuda.synchronize()
        assert torch.equal(w, want)


def test_accumulate_on_two_streams(cuda):
    """Each stream has its own workspace, kept while the step lives."""
    x, dy = gauss((4000, 128), 1, dtype=torch.bfloat16), gauss((4000, 128), 2, dtype=torch.bfloat16)
    off = torch.tensor([0, 3000, 4000], dtype=torch.int32, device="cuda")
    M = torch.zeros((2, 128, 128), device="cuda")
    step = mu.StackStep([mu.Stack(torch.zeros_like(M), M)], mu.stack_params())
    want = torch.zeros_like(M)
    s = torch.cuda.Stream()
    for stream in (None, s, None, s.cuda_stream):
        mu.grouped_matmul_dw(dy, x, off, out=want, beta=step.params.mu)
        s.wait_stream(torch.cuda.current_stream())
        step.accumulate(0, dy, x, off, stream=stream)
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(M, want)
    assert len(step._grouped_ws[0]) == 2


@pytest.mark.parametrize("compute", [mu.F16X2, mu.BF16, mu.F16])
@pytest.mark.parametrize("shape", [(1, 16, 2048), (9, 16, 1030), (40, 2048, 16), (12, 64, 768), (3, 100, 1000), (1, 128, 2048)], ids=str)
def test_clusters_repeat_their_results(cuda, shape, compute):
    """The CTAs of a cluster pass rows of A to one another and then write B' in their place: no peer may receive B' for A.
    Repeated beside another stream's traffic, since that would depend on timing: the same bits every time, and right."""
    M = spectrum(shape, 111, 1e-3) if compute == mu.F16X2 else gauss(shape, 111, 1e-3)
    W = torch.zeros(shape, device="cuda")
    step = mu.StackStep([mu.Stack(W, M)], mu.stack_params(lr=1.0, scale=-1.0, ns=mu.ns_params(compute=compute)))
    before = mu.kernel_launch_count()
    step()
    assert mu.kernel_launch_count() - before == 1 and step.device_status() == mu.OK
    want = polar(M)
    for i in range(shape[0]):
        assert rel(W[i], want[i]) <= TOL[compute], i
    first, other = W.clone(), torch.cuda.Stream()
    a, b = torch.zeros(1 << 24, device="cuda"), torch.zeros(1 << 24, device="cuda")
    torch.cuda.synchronize()
    for i in range(60):
        if i % 4 == 0:
            with torch.cuda.stream(other):
                b.copy_(a)
        W.zero_()
        step()
        assert torch.equal(W, first), i


@pytest.mark.parametrize("own_word", [False, True])
@pytest.mark.parametrize("bad", [[0, 40, 20, 60], [0, 20, 40, 61], [-1, 20, 40, 60]])
def test_deferred_errors_of_accumulate(cuda, bad, own_word):
    """Offsets out of order leave the momentum unspecified: reported where the step's errors are, and not forgotten by
    the step that follows."""
    dy, x = gauss((60, 24), 1, dtype=torch.bfloat16), gauss((60, 40), 2, dtype=torch.bfloat16)
    good = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device="cuda")
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    M = torch.zeros((3, 24, 40), device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda") if own_word else None
    step = mu.StackStep([mu.Stack(torch.zeros_like(M), M)], mu.stack_params(dev_status=word))

    def status():
        if not own_word:
            return step.device_status()
        code = int(word.item())
        word.zero_()
        return code

    side = torch.cuda.Stream()
    for stream in (None, side):
        for table, code in ((good, mu.OK), (off, mu.ERR_INVALID_ARG), (good, mu.OK)):
            M.zero_()
            side.wait_stream(torch.cuda.current_stream())
            step.accumulate(0, dy, x, table, stream=stream)
            torch.cuda.current_stream().wait_stream(side)
            if code != mu.OK:
                M.zero_()  # unspecified, NaN perhaps; the step has errors of its own to tell
            step()
            assert status() == code
            assert status() == mu.OK


def test_workspaces_and_status_words_of_calls(cuda):
    """A workspace on the host or in pieces is refused; one of another element type counts its bytes; a status word
    lives as long as the parameters that hold its address."""
    import gc
    import weakref
    M, x, off = gauss((2, 16, 24), 1), gauss((5, 24), 2, dtype=torch.bfloat16), torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    need = mu.grouped_workspace_size(2)
    pieces = torch.empty((need // 4 + 1, 8), dtype=torch.uint8, device="cuda")[:, :4]
    for ws in (torch.empty(need, dtype=torch.uint8), pieces):
        for call in (lambda: mu.grouped_matmul_dw(x, x, off, ws=ws), lambda: mu.StackStep([mu.Stack(M.clone(), M.clone())], mu.stack_params(), ws=ws)):
            with pytest.raises(mu.MuonError) as err:
                call()
            assert err.value.code == mu.ERR_INVALID_ARG
    want = mu.grouped_matmul_dw(x, x, off)
    assert torch.equal(mu.grouped_matmul_dw(x, x, off, ws=torch.empty(need // 4 + 1, dtype=torch.float32, device="cuda")), want)
    a, b = M.clone(), M.clone()
    size = mu.stack_step([mu.Stack(a, M.clone())]).ws.numel()
    step = mu.StackStep([mu.Stack(b, M.clone())], mu.stack_params(), ws=torch.empty(size // 2 + 1, dtype=torch.float16, device="cuda"))
    step()
    assert step.device_status() == mu.OK and torch.equal(a, b)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    alive, p = weakref.ref(word), mu.stack_params(dev_status=word)
    step = mu.StackStep([mu.Stack(b, M.clone())], p)
    del word, p
    gc.collect()
    assert alive() is not None
    step()
    assert int(alive().item()) == mu.OK


@pytest.mark.parametrize("compute", [mu.F16X2, mu.BF16, mu.F16, mu.F32])
@pytest.mark.parametrize("shape", [(6, 136, 300), (6, 300, 136)], ids=str)
def test_range_of_the_chain(cuda, shape, compute):
    """Matrices too large for the chip: zeros are left alone (with eps 0 too), a tiny or huge matrix is orthogonalised like
    any other, down to entries whose squares leave fp32's range. bf16's range ends at a norm of 1e18."""
    M = gauss(shape, 121)
    M[1] = 0
    M[2] *= 1e-6
    M[3] *= 1e15 if compute == mu.BF16 else 1e30
    M[4] = 0
    M[4, 3, 5] = 2.0
    for eps, tiny in ((1e-7, 1e-21), (0.0, 1e-16), (0.0, 1e-21), (0.0, 1e-25), (0.0, 1e-33)):
        M[5] = gauss(shape[1:], 122) * tiny
        W = torch.ones_like(M)
        step = mu.stack_step([mu.Stack(W, M.clone())], mu.stack_params(lr=1.0, scale=-1.0, ns=mu.ns_params(compute=compute, norm_eps=eps)))
        assert step.device_status() == mu.OK, (eps, tiny)
        assert bool((W[1] == 1).all())
        want = polar(M, eps)
        for i in (0, 2, 3, 4, 5):
            # 1 + O in fp32: half a step of 1 an element beside O's own error
            off = (W[i].double() - 1 - want[i]).norm()
            assert off <= TOL[compute] * want[i].norm() + 2.0 ** -23 * math.sqrt(shape[1] * shape[2]), (eps, tiny, i)


def test_large_bf16_matrix_is_reported(cuda):
    """The chain's bf16 operands are stored unscaled: norms from 1e18 on may be reported (from 1e20 on they are)."""
    M = gauss((2, 200, 300), 123)
    M[1] *= 1e20
    W = torch.zeros_like(M)
    step = mu.stack_step([mu.Stack(W, M.clone())], mu.stack_params(lr=1.0, scale=-1.0, ns=mu.ns_params(compute=mu.BF16)))
    assert step.device_status() == mu.ERR_NONFINITE
    assert rel(W[0], polar(M[0])) <= TOL[mu.BF16]


@pytest.mark.parametrize("compute", [mu.F16X2, mu.BF16, mu.F16, mu.F32])
def test_nonfinite_matrix_stays_alone_in_the_chain(cuda, compute):
    M = gauss((3, 200, 300), 124)
    W = gauss(M.shape, 125)
    p = mu.stack_params(ns=mu.ns_params(compute=compute))
    good = W.clone()
    assert mu.stack_step([mu.Stack(good, M.clone())], p).device_status() == mu.OK
    for bad in (float("nan"), float("inf")):
        M2, W2 = M.clone(), W.clone()
        M2[1, 3, 7] = bad
        assert mu.stack_step([mu.Stack(W2, M2)], p).device_status() == mu.ERR_NONFINITE
        assert torch.equal(W2[0], good[0]) and torch.equal(W2[2], good[2])


@pytest.mark.parametrize("compute", [mu.F16, mu.BF16, mu.F32])
@pytest.mark.parametrize("shape", [(3, 64, 200), (2, 130, 257), (2, 257, 130), (2, 24, 1000), (2, 520, 264), (1, 1, 40)], ids=str)
def test_gram_chain_of_other_shapes(cuda, shape, compute):
    """By the Gram iteration, which the on-chip form does not take; the last matrix is zeros. In bf16 its own storage points
    miss 2e-2: rounding R, Q and Z where the chain stores them, and nothing else, gives 1.5e-2 to 2.5e-2 (a single row) on
    gaussian matrices of these shapes; twice that is allowed."""
    M = gauss(shape, 126, 1e-3)
    if shape[0] > 1:
        M[-1] = 0
    W = torch.zeros_like(M)
    step = mu.stack_step([mu.Stack(W, M.clone())], mu.stack_params(lr=1.0, scale=-1.0, ns=mu.ns_params(gram=True, compute=compute)))
    assert step.device_status() == mu.OK
    tol = 5e-2 if compute == mu.BF16 else TOL[compute]
    want = polar(M)
    for i in range(shape[0]):
        assert rel(W[i], want[i]) <= tol if want[i].any() else not bool(W[i].any()), i


@pytest.mark.parametrize("shape", [(8, 520, 1030), (8, 1030, 520), (32, 264, 776), (12, 776, 264), (3, 1000, 1000), (1, 1536, 2050)], ids=str)
def test_two_planes_of_larger_stacks(cuda, shape):
    """More tiles than one wave of the smallest holds: CTA pairs on 256 and 128 columns, several tiles a pair, several chunks
    a storing warp, ragged edges. Besides the tolerance for small matrices the sums' own roundings count: the accumulator
    loses up to 2^-23 of its running sum in each instruction of 16 columns, half of that on average, and 2/3 of the final
    sum stands in it on average, so a product over K columns is off by K / 16 * 2^-23 / 3 of itself. The first product
    (K = the longer side) and the last (the shorter) enter O about once each step, the n x n one through B, and a step
    passes on what it gets with a factor of at most 3.44 (its slope at 0) and about 1 near the end: five steps, allowed
    once each with factor 2."""
    longer, shorter = max(shape[1:]), min(shape[1:])
    M = spectrum(shape, 131, 1e-3)
    W0, G = gauss(shape, 132, 0.02), spectrum(shape, 133, 1e-3)
    W, Mv = W0.clone(), M.clone()
    C = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    p = mu.stack_params(nesterov=True, weight_decay=0.1, scale=-3.0, ns=mu.ns_params(compute=mu.F16X2))
    step = mu.stack_step([mu.Stack(W, Mv, G, C)], p)
    assert step.device_status() == mu.OK
    tol = TOL[mu.F16X2] + 5 * 2 * (longer + 2 * shorter) / 16 * 2.0 ** -23 / 3
    check_update(W0, M, G, W, Mv, C, p, tol)
    want = polar(G.double() + p.mu * Mv.double())
    O = (W.double() - (1 - p.lr * p.weight_decay) * W0.double()) / (3.0 * p.lr)
    for i in range(shape[0]):
        # W's three roundings (of values below 0.125) as in test_small_matrices
        assert rel(O[i], want[i]) <= tol + 3 * 2.0 ** -27 / 0.06 / 0.9 * math.sqrt(longer), i


def test_status_of_stacks_without_elements(cuda):
    """Nothing is computed, and the status is not what happened to be in the workspace."""
    dirty = torch.full((4096,), 7, dtype=torch.uint8, device="cuda")
    for stacks in ([], [(0, 8, 8)], [(2, 0, 8), (3, 8, 0)]):
        step = mu.StackStep([mu.Stack(gauss(s, 1), gauss(s, 2), gauss(s, 3)) for s in stacks], mu.stack_params(), ws=dirty.clone())
        step()
        assert step.device_status() == mu.OK


@pytest.mark.parametrize("kind", ["gauss", "spectrum"])
@pytest.mark.parametrize("shape", [(1, 4096, 4096), (1, 256, 16384), (2, 2048, 1024)], ids=str)
def test_two_planes_of_long_sums(cuda, shape, kind):
    """The largest matrices, with the tolerance of test_two_planes_of_larger_stacks: here most of it is the sums' own."""
    longer, shorter = max(shape[1:]), min(shape[1:])
    M = (gauss if kind == "gauss" else spectrum)(shape, 141, 1e-3)
    W = torch.zeros_like(M)
    step = mu.stack_step([mu.Stack(W, M)], mu.stack_params(lr=1.0, scale=-1.0, ns=mu.ns_params(compute=mu.F16X2)))
    assert step.device_status() == mu.OK
    want = polar(M)
    for i in range(shape[0]):
        assert rel(W[i], want[i]) <= TOL[mu.F16X2] + 5 * 2 * (longer + 2 * shorter) / 16 * 2.0 ** -23 / 3, i
