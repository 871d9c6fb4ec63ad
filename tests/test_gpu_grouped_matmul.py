"""Grouped matmul by expert (forward, input and weight gradient) and the
block-scaled FP8 matmul against plain 64-bit products.

Tolerances: a sum of K products in fp32 is off by at most K steps of 2^-23 of
the sum of the products' magnitudes (tensor cores may drop the bits below a
step, so a whole step, not half, per addition); one rounding to bf16 adds
2^-8 of the value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def M():
    import sparse_moe_layer_limited_b200 as M
    return M


@pytest.fixture()
def ws(M):
    w = torch.zeros(M.matmul_workspace_size(), dtype=torch.uint8, device="cuda")
    yield w
    assert M.moe_read_device_status(w) == 0


def offsets_of(counts, lead=0):
    o = torch.zeros(len(counts) + 1, dtype=torch.int64)
    o[1:] = torch.tensor(counts).cumsum(0)
    return (o + lead).to(torch.int32).cuda()


def rand(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tol(mag, want, K, dtype):
    t = mag * (K * 2.0 ** -23)
    if dtype == BF:
        t = t + (want.abs() + t) * 2.0 ** -8
    return t


def close(got, want, mag, K):
    bad = (got.double() - want).abs() > tol(mag, want, K, got.dtype) + 1e-30
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()))


# counts per expert, rows before the first and behind the last expert, n, k
RAGGED = [
    ([1], 0, 0, 8, 8),
    ([5, 0, 131, 1], 3, 7, 72, 40),
    ([0, 0, 0], 0, 9, 64, 64),
    ([128, 256, 64], 0, 0, 256, 192),
    ([33, 0, 97, 129, 200, 31], 0, 5, 264, 520),
    ([1] * 40 + [0] * 20 + [2] * 4, 1, 0, 136, 328),
    ([700], 0, 0, 1000, 72),
    # few rows, a long contraction in either direction: split over clusters
    ([3], 0, 0, 40, 4104), ([1, 0, 17], 0, 2, 2056, 1032), ([64], 0, 0, 136, 2048),
    ([65, 2], 1, 1, 520, 1024),
]


def expected(mode, a, b, counts, lead, n, k):
    """64-bit result and the sum of the products' magnitudes."""
    R = a.shape[0]
    ad, bd = a.double(), b.double()
    if mode == "dw":
        want = torch.zeros(len(counts), n, k, dtype=F64, device="cuda")
    else:
        want = torch.zeros(R, n if mode == "fwd" else k, dtype=F64, device="cuda")
    mag = torch.zeros_like(want)
    r = lead
    for e, c in enumerate(counts):
        s = slice(r, r + c)
        if mode == "dw":
            want[e] = ad[s].t() @ bd[s]
            mag[e] = ad[s].abs().t() @ bd[s].abs()
        else:
            w = bd[e].t() if mode == "fwd" else bd[e]
            want[s] = ad[s] @ w
            mag[s] = ad[s].abs() @ w.abs()
        r += c
    return want, mag


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("mode", ["fwd", "dx"])
@pytest.mark.parametrize("counts,lead,behind,n,k", RAGGED)
def test_rows_times_weight(M, ws, mode, dtype, counts, lead, behind, n, k):
    g = gen(1)
    R, E = lead + sum(counts) + behind, len(counts)
    cin, cout = (k, n) if mode == "fwd" else (n, k)
    a = rand(g, R, cin, dtype=dtype)
    a[:lead] = float("nan")
    a[R - behind:R] = float("nan")
    w = rand(g, E, n, k, dtype=dtype)
    out = torch.full((R, cout), 7.0, dtype=dtype, device="cuda")
    f = M.moe_grouped_matmul if mode == "fwd" else M.moe_grouped_matmul_dx
    f(a, offsets_of(counts, lead), w, out, ws)
    want, mag = expected(mode, a, w, counts, lead, n, k)
    own = slice(lead, R - behind)
    close(out[own], want[own], mag[own], cin)
    assert (out[:lead] == 7.0).all() and (out[R - behind:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,lead,behind,n,k", RAGGED)
def test_weight_gradient(M, ws, dtype, counts, lead, behind, n, k):
    g = gen(2)
    R, E = lead + sum(counts) + behind, len(counts)
    dy, x = rand(g, R, n, dtype=dtype), rand(g, R, k, dtype=dtype)
    for t in (dy, x):   # rows of nobody, in the same blocks as an expert's last rows
        t[:lead] = float("nan")
        t[R - behind:R] = float("inf")
    dw = torch.full((E, n, k), 7.0, dtype=dtype, device="cuda")
    M.moe_grouped_matmul_dw(dy, x, offsets_of(counts, lead), dw, ws)
    want, mag = expected("dw", dy, x, counts, lead, n, k)
    close(dw, want, mag, max(counts))


# few output tiles and many rows (their contraction is split over clusters), and
# tiles enough for the others
@pytest.mark.parametrize("counts,lead,behind,n,k", [
    ([5001], 0, 0, 8, 8), ([600], 1, 3, 136, 264), ([1500, 0, 37, 2103], 3, 5, 72, 40),
    ([0, 0, 4500], 0, 9, 264, 136), ([9000, 1], 2, 0, 128, 1032), ([64 * 40 + 1], 5, 70, 40, 2056),
    ([777] * 5, 0, 0, 128, 128), ([129, 0, 1000, 33], 7, 2, 1032, 1160)])
def test_weight_gradient_of_many_rows(M, ws, counts, lead, behind, n, k):
    g = gen(23)
    R = lead + sum(counts) + behind
    dy, x = rand(g, R, n, dtype=BF), rand(g, R, k, dtype=BF)
    for t in (dy, x):
        t[:lead] = float("nan")
        t[R - behind:R] = float("nan")
    dw = torch.full((len(counts), n, k), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_matmul_dw(dy, x, offsets_of(counts, lead), dw, ws)
    close(dw, *expected("dw", dy, x, counts, lead, n, k), max(counts))
    again = torch.empty_like(dw)
    for _ in range(3):
        M.moe_grouped_matmul_dw(dy, x, offsets_of(counts, lead), again, ws)
        assert torch.equal(again, dw)


def test_split_weight_gradients_and_bad_offsets(M):
    """The other experts' gradients stay right; the bad one's are zeros."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    g = gen(24)
    dy, x = rand(g, 3000, 40, dtype=BF), rand(g, 3000, 72, dtype=BF)
    off = torch.tensor([0, 1400, 1200, 3000], dtype=torch.int32, device="cuda")
    dw = torch.full((3, 40, 72), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_matmul_dw(dy, x, off, dw, ws)
    assert (dw[1] == 0).all() and M.moe_read_device_status(ws) != 0
    for e, s in ((0, slice(0, 1400)), (2, slice(1200, 3000))):
        a, b = dy[s].double(), x[s].double()
        close(dw[e], a.t() @ b, a.abs().t() @ b.abs(), 1800)


@pytest.mark.parametrize("mode", ["fwd", "dx"])
@pytest.mark.parametrize("counts,m", [
    ([512] * 32, 2048),                                   # 222 units of two tiles, 34 in the last
    ([257 + 8 * e for e in range(31)] + [0, 3], 2048),    # round: the last experts' are cut
    ([511, 1, 0, 700, 260] * 8 + [300], 1288), ([8190], 5000)])
def test_units_cut_in_the_last_round(M, ws, mode, counts, m):
    g = gen(25)
    n, k = (m, 72) if mode == "fwd" else (72, m)
    R, off = sum(counts) + 2, offsets_of(counts, 1)
    a, w = rand(g, R, 72, dtype=BF), rand(g, len(counts), n, k, dtype=BF)
    out = torch.full((R, m), 7.0, dtype=BF, device="cuda")
    (M.moe_grouped_matmul if mode == "fwd" else M.moe_grouped_matmul_dx)(a, off, w, out, ws)
    want, mag = expected(mode, a, w, counts, 1, n, k)
    close(out[1:-1], want[1:-1], mag[1:-1], 72)
    assert (out[0] == 7.0).all() and (out[-1] == 7.0).all()


def test_fp32_takes_any_width(M, ws):
    g = gen(3)
    counts, n, k = [3, 0, 66, 130], 37, 101
    R, off = sum(counts), offsets_of(counts)
    x, dy, w = rand(g, R, k), rand(g, R, n), rand(g, 4, n, k)
    y, dx, dw = torch.empty(R, n).cuda(), torch.empty(R, k).cuda(), torch.empty(4, n, k).cuda()
    M.moe_grouped_matmul(x, off, w, y, ws)
    M.moe_grouped_matmul_dx(dy, off, w, dx, ws)
    M.moe_grouped_matmul_dw(dy, x, off, dw, ws)
    close(y, *expected("fwd", x, w, counts, 0, n, k), k)
    close(dx, *expected("dx", dy, w, counts, 0, n, k), n)
    close(dw, *expected("dw", dy, x, counts, 0, n, k), 130)


def test_large_fp32_tile(M, ws):
    """Enough output tiles for the 128 x 128 fp32 kernel."""
    g = gen(4)
    counts, n, k = [600, 1, 655], 4100, 76
    R, off = sum(counts), offsets_of(counts)
    x, w = rand(g, R, k), rand(g, 3, n, k)
    y = torch.empty(R, n, device="cuda")
    M.moe_grouped_matmul(x, off, w, y, ws)
    close(y, *expected("fwd", x, w, counts, 0, n, k), k)
    dw = torch.empty(3, n, k, device="cuda")
    M.moe_grouped_matmul_dw(y, x, off, dw, ws)
    close(dw, *expected("dw", y, x, counts, 0, n, k), 655)


def test_gradients_against_differences(M, ws):
    """<dy, y(x + h) - y(x)> in 64 bits equals <dx, h> (the product is linear in x and in w), up to
    the gradients' own error bound."""
    g = gen(5)
    counts, n, k = [9, 70], 24, 40
    R, off = sum(counts), offsets_of(counts)
    x, dy, w = rand(g, R, k), rand(g, R, n), rand(g, 2, n, k)
    dx, dw = torch.empty(R, k).cuda(), torch.empty(2, n, k).cuda()
    M.moe_grouped_matmul_dx(dy, off, w, dx, ws)
    M.moe_grouped_matmul_dw(dy, x, off, dw, ws)

    def loss(xx, ww):
        return (dy.double() * expected("fwd", xx, ww, counts, 0, n, k)[0]).sum()
    hx, hw = rand(g, R, k).double(), rand(g, 2, n, k).double()
    for grad, h, diff, K, mag in (
            (dx, hx, loss(x.double() + hx, w) - loss(x, w), n, expected("dx", dy, w, counts, 0, n, k)[1]),
            (dw, hw, loss(x, w.double() + hw) - loss(x, w), 70, expected("dw", dy, x, counts, 0, n, k)[1])):
        bound = (tol(mag, grad.double(), K, F32) * h.abs()).sum()
        assert abs((grad.double() * h).sum() - diff) <= bound + 1e-9 * abs(diff)


def test_an_expert_does_not_see_its_neighbours(M, ws):
    """Infinities in one expert's rows and weights stay in its own results."""
    g = gen(6)
    counts, n, k = [50, 3, 77], 136, 72
    R, off = sum(counts), offsets_of(counts)
    x, dy, w = (rand(g, R, k, dtype=BF), rand(g, R, n, dtype=BF), rand(g, 3, n, k, dtype=BF))
    x[50:53] = float("inf")
    dy[50:53] = float("nan")
    w[1] = float("nan")
    y, dx, dw = (torch.empty(R, n, dtype=BF).cuda(), torch.empty(R, k, dtype=BF).cuda(),
                 torch.empty(3, n, k, dtype=BF).cuda())
    M.moe_grouped_matmul(x, off, w, y, ws)
    M.moe_grouped_matmul_dx(dy, off, w, dx, ws)
    M.moe_grouped_matmul_dw(dy, x, off, dw, ws)
    for t in (y, dx):
        assert t[:50].isfinite().all() and t[53:].isfinite().all() and t[50:53].isnan().all()
    assert dw[0].isfinite().all() and dw[2].isfinite().all() and dw[1].isnan().all()


def test_no_rows(M, ws):
    off = offsets_of([0, 0])
    w = torch.zeros(2, 16, 24, dtype=BF, device="cuda")
    e = lambda c: torch.empty(0, c, dtype=BF, device="cuda")  # noqa: E731
    M.moe_grouped_matmul(e(24), off, w, e(16), ws)
    M.moe_grouped_matmul_dx(e(16), off, w, e(24), ws)
    dw = torch.full_like(w, 3.0)
    M.moe_grouped_matmul_dw(e(16), e(24), off, dw, ws)
    assert (dw == 0).all()


def test_rows_that_belong_to_nobody(M, ws):
    """Many rows, no owner: nothing is written but the (zero) weight gradients, on the kernels for
    many rows too."""
    R, E, n, k = 40000, 3, 512, 64
    off = torch.full((E + 1,), 17, dtype=torch.int32, device="cuda")
    x = torch.full((R, k), float("nan"), dtype=BF, device="cuda")
    w = torch.ones(E, n, k, dtype=BF, device="cuda")
    y = torch.full((R, n), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_matmul(x, off, w, y, ws)
    assert (y == 7.0).all()
    dx = torch.full((R, k), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_matmul_dx(y, off, w, dx, ws)
    assert (dx == 7.0).all()
    M.moe_grouped_matmul_dw(y, x, off, w, ws)
    assert (w == 0).all()
    q = torch.zeros(R, k, dtype=E4M3, device="cuda")
    wq = torch.zeros(E, n, k, dtype=E4M3, device="cuda")
    M.moe_matmul_fp8(q, torch.ones(1, R, device="cuda"), off, wq, torch.ones(E, 4, 1, device="cuda"),
                     y, ws)
    assert (y == 7.0).all()


@pytest.mark.parametrize("rows_each", [1, 40])
def test_the_most_experts(M, ws, rows_each):
    g = gen(21)
    counts = [rows_each * (e % 3) for e in range(384)]
    R, n, k = sum(counts), 264, 72
    off = offsets_of(counts)
    x, dy, w = rand(g, R, k, dtype=BF), rand(g, R, n, dtype=BF), rand(g, 384, n, k, dtype=BF)
    y, dx, dw = (torch.empty(R, n, dtype=BF).cuda(), torch.empty(R, k, dtype=BF).cuda(),
                 torch.empty(384, n, k, dtype=BF).cuda())
    M.moe_grouped_matmul(x, off, w, y, ws)
    M.moe_grouped_matmul_dx(dy, off, w, dx, ws)
    M.moe_grouped_matmul_dw(dy, x, off, dw, ws)
    close(y, *expected("fwd", x, w, counts, 0, n, k), k)
    close(dx, *expected("dx", dy, w, counts, 0, n, k), n)
    close(dw, *expected("dw", dy, x, counts, 0, n, k), max(counts))


def test_large_graph_replays(M, ws):
    """The kernels for many rows, first reached inside a capture, replayed with other inputs."""
    g = gen(22)
    counts, n, k = [900, 0, 1300, 411], 1024, 640
    off, R = offsets_of(counts), sum(counts)
    x, w = rand(g, R, k, dtype=BF), rand(g, 4, n, k, dtype=BF)
    y, dw = torch.empty(R, n, dtype=BF, device="cuda"), torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_grouped_matmul(x, off, w, y, ws)
        M.moe_grouped_matmul_dw(y, x, off, dw, ws)
    for _ in range(2):
        x.copy_(rand(g, R, k, dtype=BF))
        graph.replay()
        torch.cuda.synchronize()
        close(y, *expected("fwd", x, w, counts, 0, n, k), k)
        close(dw, *expected("dw", y, x, counts, 0, n, k), max(counts))


def test_bad_offsets_are_reported_and_skipped(M):
    g = gen(7)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x, w = rand(g, 40, 16, dtype=BF), rand(g, 3, 24, 16, dtype=BF)
    off = torch.tensor([0, 10, 5, 40], dtype=torch.int32, device="cuda")   # expert 1 runs backwards
    y = torch.full((40, 24), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_matmul(x, off, w, y, ws)
    torch.cuda.synchronize()
    assert M.moe_read_device_status(ws, clear=True) == 4
    off = torch.tensor([0, 10, 41, 12], dtype=torch.int32, device="cuda")  # past the last row
    y.fill_(7.0)
    M.moe_grouped_matmul(x, off, w, y, ws)
    want, mag = expected("fwd", x[:10], w[:1], [10], 0, 24, 16)
    close(y[:10], want, mag, 16)
    assert (y[10:] == 7.0).all()
    assert M.moe_read_device_status(ws, clear=True) == 4
    dw = torch.full((3, 24, 16), 7.0, dtype=BF, device="cuda")
    M.moe_grouped_matmul_dw(rand(g, 40, 24, dtype=BF), x, off, dw, ws)
    assert (dw[1:] == 0).all() and M.moe_read_device_status(ws, clear=True) == 4


def test_long_rows_pass_32_bit_offsets(M, ws):
    """Output elements past 2^31: the last rows are the last expert's."""
    n, k = 40960, 8
    R = (1 << 31) // n + 200
    g = gen(8)
    x = torch.zeros(R, k, dtype=BF, device="cuda")
    x[-150:] = rand(g, 150, k, dtype=BF)
    w = rand(g, 2, n, k, dtype=BF)
    y = torch.empty(R, n, dtype=BF, device="cuda")
    M.moe_grouped_matmul(x, offsets_of([R - 150, 150]), w, y, ws)
    want, mag = expected("fwd", x[-150:], w[1:], [150], 0, n, k)
    close(y[-150:], want, mag, k)
    assert not y[0].any() and not y[R - 151].any()


@pytest.mark.parametrize("kind", ["fwd", "dx", "dw", "fp8"])
def test_short_contractions_of_many_ragged_units(M, ws, kind):
    """Units that end within microseconds of each other, full row blocks (stored by bulk copies)
    next to ragged ones (stored by the threads): a staging buffer handed on too early shows as
    32 x 32 blocks of another tile's values, in some runs only."""
    g = gen(20)
    counts, n, k = [674, 633, 680, 632, 678, 659], 4152, 168
    if kind == "fp8":
        n, k = 4152, 80
    off, R, E = offsets_of(counts), sum(counts), len(counts)
    if kind == "dx":
        n, k = k, n
    x, dy, w = rand(g, R, k, dtype=BF), rand(g, R, n, dtype=BF), rand(g, E, n, k, dtype=BF)
    if kind == "fp8":
        qa, sa = torch.empty(R, k, dtype=E4M3, device="cuda"), torch.empty(1, R, device="cuda")
        qw = torch.empty(E, n, k, dtype=E4M3, device="cuda")
        sw = torch.empty(E, -(-n // 128), 1, device="cuda")
        M.moe_quantize_rows_fp8(x, qa, sa)
        M.moe_quantize_blocks_fp8(w, qw, sw)
        out = torch.empty(R, n, dtype=BF, device="cuda")
        call = lambda: M.moe_matmul_fp8(qa, sa, off, qw, sw, out, ws)  # noqa: E731
        want, mag = expected("fwd", dequant_rows(qa, sa), dequant_blocks(qw, sw), counts, 0, n, k)
        K = k + 2
    elif kind == "dw":
        out = torch.empty(E, n, k, dtype=BF, device="cuda")
        call = lambda: M.moe_grouped_matmul_dw(dy, x, off, out, ws)  # noqa: E731
        want, mag = expected("dw", dy, x, counts, 0, n, k)
        K = max(counts)
    else:
        out = torch.empty(R, n if kind == "fwd" else k, dtype=BF, device="cuda")
        f = M.moe_grouped_matmul if kind == "fwd" else M.moe_grouped_matmul_dx
        a = x if kind == "fwd" else dy
        call = lambda: f(a, off, w, out, ws)  # noqa: E731
        want, mag = expected(kind, a, w, counts, 0, n, k)
        K = k if kind == "fwd" else n
    first = None
    for _ in range(60):
        out.fill_(7.0)
        call()
        if first is None:
            first = out.clone()
            close(first, want, mag, K)
        assert torch.equal(out, first)


def test_side_stream_and_graphs_sharing_a_workspace(M, ws):
    g = gen(9)
    counts, n, k = [17, 200], 128, 256
    off = offsets_of(counts)
    w = rand(g, 2, n, k, dtype=BF)
    xs = [rand(g, 217, k, dtype=BF) for _ in range(2)]
    ys = [torch.empty(217, n, dtype=BF, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.moe_grouped_matmul(xs[0], off, w, ys[0], ws, stream=side)
    side.synchronize()
    close(ys[0], *expected("fwd", xs[0], w, counts, 0, n, k), k)
    graphs = []
    for x, y in zip(xs, ys):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            M.moe_grouped_matmul(x, off, w, y, ws)
        graphs.append(graph)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):      # both at once
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        close(y, *expected("fwd", x, w, counts, 0, n, k), k)


# ---- FP8 -------------------------------------------------------------------------------

def quant_rows_reference(x, fmt):
    """The quantiser's definition: fp32 amax / top, codes round(v * (top * (1 / amax))).  (The scale
    divides by a tensor: torch divides by a Python number by multiplying with its reciprocal.)"""
    top = 448.0 if fmt == E4M3 else 57344.0
    tops = torch.full((x.shape[0],), top, device="cuda")
    R, C = x.shape
    codes = torch.empty(R, C, dtype=fmt, device="cuda")
    scales = torch.empty(-(-C // 128), R, device="cuda")
    for b in range(scales.shape[0]):
        t = x[:, 128 * b:128 * b + 128].float()
        amax = t.abs().amax(1)
        inv = torch.where(amax > 0, top * amax.reciprocal(), 0.0)
        codes[:, 128 * b:128 * b + 128] = (t * inv[:, None]).clamp(-top, top).to(fmt)
        scales[b] = torch.where(amax > 0, amax / tops, 1.0)
    return codes, scales


@pytest.mark.parametrize("fmt", [E4M3, E5M2], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("R,C", [(1, 16), (3, 128), (17, 144), (130, 1008), (2, 4096)])
def test_row_quantiser(M, fmt, R, C):
    g = gen(10)
    x = rand(g, R, C, dtype=BF)
    x[0, :16] = 0
    x[R - 1] = x[R - 1] * 1e-6
    x[R // 2, :] = 0
    codes = torch.empty(R, C, dtype=fmt, device="cuda")
    ld = R + 3
    scales = torch.full((-(-C // 128), ld), 9.0, device="cuda")
    M.moe_quantize_rows_fp8(x, codes, scales)
    wc, wsc = quant_rows_reference(x, fmt)
    assert torch.equal(codes.view(torch.uint8), wc.view(torch.uint8))
    assert torch.equal(scales[:, :R], wsc) and (scales[:, R:] == 9.0).all()


@pytest.mark.parametrize("fmt", [E4M3, E5M2], ids=["e4m3", "e5m2"])
def test_quantiser_at_the_ends_of_the_range(M, fmt):
    """Tiny tiles (the inverse would overflow), NaN and infinity."""
    x = torch.zeros(5, 256, dtype=BF, device="cuda")
    x[0, 3] = 1e-38                     # zeros beside it stay zeros
    x[1] = 2.0 ** -100
    x[2, 5] = float("nan")              # the only non-zero of its tile
    x[3] = 1.0
    x[3, 130] = float("inf")
    x[4] = 3.3e38
    codes = torch.empty(5, 256, dtype=fmt, device="cuda")
    scales = torch.empty(2, 5, device="cuda")
    M.moe_quantize_rows_fp8(x, codes, scales)
    top = 448.0 if fmt == E4M3 else 57344.0
    c = codes.float()
    assert c[0, 4:].eq(0).all() and c[0, 3].isfinite() and scales.T[0].isfinite().all()
    assert (c[1] == top).all() and (scales[:, 1] == 2.0 ** -100 / top).all()
    assert c[2, 5].isnan() and c[2, :5].eq(0).all() and c[2, 6:].eq(0).all()
    assert (c[3, :128] == top).all()
    v = c[3, 128:].double() * scales[1, 3].double()
    assert v.isnan().all()              # an infinite tile has no finite values
    assert (c[4] == top).all() and scales[:, 4].isfinite().all()


@pytest.mark.parametrize("E,n,k", [(1, 1, 16), (2, 128, 128), (3, 200, 272), (1, 129, 1040)])
def test_block_quantiser(M, E, n, k):
    g = gen(11)
    w = rand(g, E, n, k, dtype=BF)
    w[0, :128, :128] = 0
    codes = torch.empty(E, n, k, dtype=E4M3, device="cuda")
    scales = torch.empty(E, -(-n // 128), -(-k // 128), device="cuda")
    M.moe_quantize_blocks_fp8(w, codes, scales)
    for e in range(E):
        for i in range(scales.shape[1]):
            for j in range(scales.shape[2]):
                t = w[e, 128 * i:128 * i + 128, 128 * j:128 * j + 128].float()
                amax = t.abs().max()
                top = torch.full((), 448.0, device="cuda")
                s = amax / top if amax > 0 else torch.ones((), device="cuda")
                inv = top * amax.reciprocal() if amax > 0 else 0.0
                c = (t * inv).clamp(-448, 448).to(E4M3)
                got = codes[e, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                assert torch.equal(got.contiguous().view(torch.uint8),
                                   c.contiguous().view(torch.uint8))
                assert scales[e, i, j] == s


def dequant_rows(q, s):
    R, C = q.shape
    return q.float().double() * s[:, :R].double().repeat_interleave(128, 0)[:C].t()


def dequant_blocks(q, s):
    E, n, k = q.shape
    return q.float().double() * s.double().repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]


FP8_CASES = [
    (None, 7, 144, 10000), (None, 64, 1000, 2064),
    (None, 1, 16, 16), (None, 1, 129, 128), (None, 130, 264, 144), (None, 33, 257, 528),
    (None, 300, 512, 1040), ([5, 0, 131, 1], 0, 72, 48), ([0, 64, 257, 3, 0, 31], 0, 400, 656),
]


@pytest.mark.parametrize("counts,rows,n,k", FP8_CASES)
@pytest.mark.parametrize("fmt", [E4M3, E5M2], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("mode", ["fwd", "dx"])
def test_fp8_matmul(M, ws, mode, fmt, counts, rows, n, k):
    if mode == "dx":
        n = (n + 15) // 16 * 16
    g = gen(12)
    cs = counts or [rows]
    lead, behind = (0, 0) if counts is None else (2, 5)
    R, E = lead + sum(cs) + behind, len(cs)
    cin, cout = (k, n) if mode == "fwd" else (n, k)
    a, w = rand(g, R, cin, dtype=BF), rand(g, E, n, k, dtype=BF, scale=0.1)
    qa = torch.empty(R, cin, dtype=fmt, device="cuda")
    sa = torch.full((-(-cin // 128), R + 1), float("nan"), device="cuda")
    qw = torch.empty(E, n, k, dtype=E4M3, device="cuda")
    sw = torch.empty(E, -(-n // 128), -(-k // 128), device="cuda")
    M.moe_quantize_rows_fp8(a, qa, sa)
    M.moe_quantize_blocks_fp8(w, qw, sw)
    sa[:, :lead] = float("nan")                     # scales of rows that belong to nobody
    sa[:, lead + sum(cs):] = float("nan")
    out = torch.full((R, cout), 7.0, dtype=BF, device="cuda")
    f = M.moe_matmul_fp8 if mode == "fwd" else M.moe_matmul_fp8_dx
    f(qa, sa, None if counts is None else offsets_of(cs, lead), qw, sw, out, ws)
    want, mag = expected(mode, dequant_rows(qa, sa), dequant_blocks(qw, sw), cs, lead, n, k)
    own = slice(lead, R - behind)
    # two more roundings per slice: the scales' product and the multiply-add
    close(out[own], want[own], mag[own], cin + 2)
    assert (out[:lead] == 7.0).all() and (out[R - behind:] == 7.0).all()


def test_fp8_reads_the_dispatch_layout(M, ws):
    """Codes and scales as moe_dispatch writes them (E4M3 mode) feed the product by expert."""
    from synth import CONFIGS, gen as sg
    from tests import support as S
    cfg = CONFIGS[3].with_(T=200, d=256, N=8, K=2, G=2, topG=1, f=256)
    s = S.moe_shape(cfg)
    Rw, b = sg.make_router(cfg), sg.make_bias(cfg)
    x, _ = S.tie_free_x(cfg, Rw, b)
    W = S.device_weights(cfg)
    layer = M.MoELayer(s, torch.from_numpy(Rw).cuda(), torch.from_numpy(b).cuda(), W["w13"],
                       W["w2"], W["w13_scales"], W["w2_scales"], gamma=0.0)
    layer.forward(S.to_dev_x(x, cfg))
    y = torch.empty(cfg.T * cfg.K, 2 * cfg.f, dtype=BF, device="cuda")
    w13 = layer.w13.view(cfg.N + 1, 2 * cfg.f, cfg.d)[:cfg.N].contiguous()
    s13 = layer.w13_scales.view(cfg.N + 1, 2 * cfg.f // 128, cfg.d // 128)[:cfg.N].contiguous()
    M.moe_matmul_fp8(layer.x_perm, layer.x_perm_scales, layer.offsets, w13, s13, y, ws)
    counts = layer.counts.tolist()
    want, mag = expected("fwd", dequant_rows(layer.x_perm, layer.x_perm_scales),
                         dequant_blocks(w13, s13), counts, 0, 2 * cfg.f, cfg.d)
    close(y, want, mag, cfg.d + 2)
