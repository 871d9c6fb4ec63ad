"""Layer norm, forward and backward, against 64-bit formulas.

Tolerances, in units u = 2^-24 (half a step of fp32): a thread adds at most 32
of a row's elements in a chain and at most 5 + 16 partial results are merged,
so a row sum is off by at most 64 u times the mean magnitude of its terms (the
merge's own products and quotients, at most 8 u a level, included), and the
relative error of the variance by as much.  A column sum over R rows is off by
at most (R + 16) u times the sum of its terms' magnitudes.  Rounding a result
to bf16 adds 2^-8 of it.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def M():
    import sparse_moe_layer_limited_b200 as M
    return M


def make(R, d, dtype, seed=0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(R, d) * torch.exp(r(R, 1)) + shift).to(dtype)
    return x, 1 + 0.5 * r(d), r(d), r(R, d).to(dtype)


def forward(M, x, w, b, eps):
    R = x.shape[0]
    y = torch.empty_like(x)
    mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    M.moe_layer_norm(x, w, b, eps, y, mean, rstd)
    return y, mean, rstd


def rounding(v, dtype):
    return v.abs() * (2.0 ** -8 if dtype == BF else U)


def check_forward(x, w, b, eps, y, mean, rstd):
    xd = x.double()
    mu = xd.mean(1, keepdim=True)
    var = (xd - mu).square().mean(1, keepdim=True)
    rs = (var + eps).rsqrt()
    z = (xd - mu) * rs
    want = z * w.double() + (0 if b is None else b.double())
    top = xd.abs().mean(1, keepdim=True)
    assert ((mean[:, None].double() - mu).abs() <= 64 * U * top + 1e-30).all()
    # the variance's error relative to itself, and the error of the centred terms
    rel = 64 * U * (1 + top * rs)
    assert ((rstd[:, None].double() - rs).abs() <= rel * rs).all()
    t = (64 * U * (top + xd.abs()) * rs + rel * z.abs()) * w.double().abs()
    t = t + 2 * U * (want.abs() + (0 if b is None else b.double().abs()))
    t = t + rounding(want.abs() + t, x.dtype)
    bad = (y.double() - want).abs() > t
    assert not bad.any(), float(((y.double() - want).abs() / t).max())


SIZES = [(1, 1), (3, 7), (5, 32), (1, 250), (9, 256), (4, 500), (130, 512), (2, 1001), (64, 1024),
         (3, 1030), (7, 2048), (2, 2049), (33, 4096), (1, 7168), (2, 8191), (300, 8192), (5, 9999),
         (2, 16384), (3000, 64)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,d", SIZES)
def test_forward_and_backward(M, R, d, dtype):
    x, w, b, dy = make(R, d, dtype)
    eps = 1e-5
    y, mean, rstd = forward(M, x, w, b, eps)
    check_forward(x, w, b, eps, y, mean, rstd)
    y2, *_ = forward(M, x, w, None, eps)
    check_forward(x, w, None, eps, y2, mean, rstd)
    dx = torch.empty_like(x)
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(M.layer_norm_workspace_size(R, d), dtype=torch.uint8, device="cuda")
    M.moe_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    g, rs = dy.double(), rstd[:, None].double()
    z = (x.double() - mean[:, None].double()) * rs
    h = g * w.double()
    m1, m2 = h.mean(1, keepdim=True), (h * z).mean(1, keepdim=True)
    want = rs * (h - m1 - z * m2)
    t = 64 * U * rs * (h.abs() + h.abs().mean(1, keepdim=True)
                       + z.abs() * (h * z).abs().mean(1, keepdim=True) + (z * m2).abs())
    t = t + rounding(want.abs() + t, dtype)
    bad = (dx.double() - want).abs() > t
    assert not bad.any(), float(((dx.double() - want).abs() / t).max())
    assert ((dw.double() - (g * z).sum(0)).abs() <= (R + 16) * U * (g * z).abs().sum(0) + 1e-30).all()
    assert ((db.double() - g.sum(0)).abs() <= (R + 16) * U * g.abs().sum(0) + 1e-30).all()
    # without dbias, and the same bits on a second call
    dx2, dw2 = torch.empty_like(x), torch.empty(d, device="cuda")
    M.moe_layer_norm_backward(dy, x, w, mean, rstd, dx2, dw2, None, ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_a_large_common_offset_does_not_cancel(M):
    x, w, b, _ = make(40, 1777, F32, seed=3, shift=3.0e4)
    check_forward(x, w, b, 1e-5, *forward(M, x, w, b, 1e-5))


def test_constant_rows_and_non_finite_rows(M):
    x, w, b, _ = make(6, 640, F32, seed=4)
    x[1] = 2.5
    x[3, 17] = float("nan")
    x[4, 3] = float("inf")
    y, mean, rstd = forward(M, x, w, b, 1e-5)
    assert torch.equal(y[1], b) and rstd[1].item() == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    assert y[3].isnan().all() and y[4].isnan().all()
    keep = [0, 1, 2, 5]
    check_forward(x[keep], w, b, 1e-5, y[keep], mean[keep], rstd[keep])


def test_gradient_against_differences(M):
    """Central differences of the 64-bit forward along random directions, step 2^-13: their own
    error is of the order of step^2 (below 1e-6 of the terms' size here)."""
    R, d, eps = 3, 96, 1e-3
    x, w, b, dy = make(R, d, F32, seed=5)
    _, mean, rstd = forward(M, x, w, b, eps)
    dx, dw, db = torch.empty_like(x), torch.empty(d).cuda(), torch.empty(d).cuda()
    ws = torch.empty(M.layer_norm_workspace_size(R, d), dtype=torch.uint8, device="cuda")
    M.moe_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)

    def loss(xx, ww, bb):
        mu = xx.mean(1, keepdim=True)
        rs = ((xx - mu).square().mean(1, keepdim=True) + eps).rsqrt()
        return (dy.double() * ((xx - mu) * rs * ww + bb)).sum()
    xd, wd, bd = x.double(), w.double(), b.double()
    h = 2.0 ** -13
    g = torch.Generator(device="cuda").manual_seed(6)
    for _ in range(4):
        vx = torch.randn(R, d, generator=g, device="cuda").double()
        vw = torch.randn(d, generator=g, device="cuda").double()
        vb = torch.randn(d, generator=g, device="cuda").double()
        num = (loss(xd + h * vx, wd + h * vw, bd + h * vb)
               - loss(xd - h * vx, wd - h * vw, bd - h * vb)) / (2 * h)
        parts = [(dx.double() * vx), (dw.double() * vw), (db.double() * vb)]
        got = sum(p.sum() for p in parts)
        size = sum(p.abs().sum() for p in parts)
        assert abs(got - num) <= 1e-5 * size


def test_no_rows(M):
    d = 40
    w = torch.ones(d, device="cuda")
    e = torch.empty(0, d, device="cuda")
    m = torch.empty(0, device="cuda")
    M.moe_layer_norm(e, w, None, 1e-5, e, m, m)
    dw, db = torch.full((d,), 3.0, device="cuda"), torch.full((d,), 3.0, device="cuda")
    ws = torch.empty(max(1, M.layer_norm_workspace_size(0, d)), dtype=torch.uint8, device="cuda")
    M.moe_layer_norm_backward(e, e, w, m, m, e, dw, db, ws)
    assert (dw == 0).all() and (db == 0).all()


def test_side_stream_and_graph(M):
    R, d = 50, 1536
    x, w, b, dy = make(R, d, BF, seed=7)
    side = torch.cuda.Stream()
    y = torch.empty_like(x)
    mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    M.moe_layer_norm(x, w, b, 1e-5, y, mean, rstd, stream=side)
    side.synchronize()
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty(d).cuda(), torch.empty(d).cuda()
    ws = torch.empty(M.layer_norm_workspace_size(R, d), dtype=torch.uint8, device="cuda")
    M.moe_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    kept = dx.clone(), dw.clone(), db.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_layer_norm(x, w, b, 1e-5, y, mean, rstd)
        M.moe_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    for t in (y, dx, dw, db):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip((dx, dw, db), kept):
        assert torch.equal(a, c)


def test_two_host_threads_with_rows_of_different_widths(M):
    """Calls of one process at the same time, on streams of their own."""
    import threading
    cases, errors = [], []
    for d in (1032, 6144, 7680):
        x, w, b, dy = make(40, d, BF, seed=d)
        cases.append((x, w, b, dy, *forward(M, x, w, b, 1e-5)))
    torch.cuda.synchronize()

    def work(x, w, b, dy, y, mean, rstd):
        try:
            st = torch.cuda.Stream()
            got = [torch.empty_like(t) for t in (y, mean, rstd)]
            dx, dw = torch.empty_like(x), torch.empty_like(w)
            ws = torch.empty(M.layer_norm_workspace_size(*x.shape), dtype=torch.uint8,
                             device="cuda")
            for _ in range(3000):
                M.moe_layer_norm(x, w, b, 1e-5, *got, stream=st)
                M.moe_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, None, ws, stream=st)
            st.synchronize()
            assert all(torch.equal(g, t) for g, t in zip(got, (y, mean, rstd)))
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
