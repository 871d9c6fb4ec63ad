"""The operators around the fused expert FFN used together, as a user's layer
would: the norm in front of MoELayer, the experts out of grouped products, and
a normed dense FP8 projection with its gradients."""
import numpy as np
import pytest
import torch

from synth import CONFIGS, gen
from tests import support as S

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def M():
    import sparse_moe_layer_limited_b200 as M
    return M


def layer_inputs(T=300, bias=True):
    cfg = CONFIGS[1].with_(T=T, d=256, N=8, K=2, G=2, topG=1, f=256)
    Rw, b = gen.make_router(cfg), gen.make_bias(cfg)
    W = S.device_weights(cfg)
    x = S.to_dev_x(gen.make_x(cfg, 0, 0), cfg)
    g = torch.Generator(device="cuda").manual_seed(3)
    nw = 1 + 0.2 * torch.randn(cfg.d, generator=g, device="cuda")
    nb = 0.1 * torch.randn(cfg.d, generator=g, device="cuda") if bias else None
    return cfg, torch.from_numpy(Rw).cuda(), torch.from_numpy(b).cuda(), W, x, nw, nb, g


@pytest.mark.parametrize("bias", [True, False])
def test_the_layer_with_a_norm_is_the_norm_then_the_layer(M, bias):
    cfg, Rw, b, W, x, nw, nb, g = layer_inputs(bias=bias)
    s = S.moe_shape(cfg)
    normed = M.MoELayer(s, Rw, b.clone(), W["w13"], W["w2"], gamma=1e-3, norm_w=nw, norm_b=nb)
    plain = M.MoELayer(s, Rw, b.clone(), W["w13"], W["w2"], gamma=1e-3)
    xn = torch.empty_like(x)
    mean, rstd = torch.empty(cfg.T, device="cuda"), torch.empty(cfg.T, device="cuda")
    M.moe_layer_norm(x, nw, nb, 1e-5, xn, mean, rstd)
    assert torch.equal(normed.forward(x), plain.forward(xn))
    assert torch.equal(normed.topk_idx, plain.topk_idx) and torch.equal(normed.bias, plain.bias)
    # backward: the layer's, then the norm's
    w13t = torch.empty(cfg.N + 1, cfg.d, 2 * cfg.f, dtype=BF, device="cuda")
    w2t = torch.empty(cfg.N + 1, cfg.f, cfg.d, dtype=BF, device="cuda")
    M.moe_transpose_weights(s, W["w13"], W["w2"], w13t, w2t)
    dy = torch.randn(cfg.T, cfg.d, generator=g, device="cuda").to(BF)
    a, p = normed.backward(x, dy, w13t, w2t), plain.backward(xn, dy, w13t, w2t)
    dx, dw, db = torch.empty_like(x), torch.empty_like(nw), torch.empty_like(nw)
    ws = torch.empty(M.layer_norm_workspace_size(cfg.T, cfg.d), dtype=torch.uint8, device="cuda")
    M.moe_layer_norm_backward(p["dx"], x, nw, mean, rstd, dx, dw, db, ws)
    assert torch.equal(a["dx"], dx) and torch.equal(a["dnorm_w"], dw)
    assert ("dnorm_b" in a) == bias and (not bias or torch.equal(a["dnorm_b"], db))
    for k in ("drouter", "dgate", "dw13", "dw2"):
        assert torch.equal(a[k], p[k]), k
    # captured: the same step from one graph launch, from a fresh buffer's contents
    buf = x.clone()
    normed.bias.copy_(b)
    normed.capture(buf, update_bias=False)
    normed.bias.copy_(b)
    buf.copy_(x.flip(0))
    y = normed.replay().clone()
    normed.bias.copy_(b)
    assert torch.equal(y, normed.forward(x.flip(0).contiguous(), update_bias=False))
    assert normed.device_status() == 0 and normed.backward_status() == 0


def unpack13(w13, f):
    """[E, 2f, d] packed -> W1, W3 [E, f, d]."""
    E, _, d = w13.shape
    w = w13.view(E, f // 128, 2, 128, d)
    return w[:, :, 0].reshape(E, f, d).contiguous(), w[:, :, 1].reshape(E, f, d).contiguous()


def test_the_routed_experts_from_grouped_products(M):
    """x W1^T, x W3^T, silu(.) * ., h W2^T by expert on the dispatched rows, and the gradients of
    the last product, against the layer's fused kernels.  Both sides round h and y to bf16 once;
    g and u are rounded here only, and one rounding of either moves h by at most about 2^-8 of it
    (silu's relative slope is below 1.1 for g > 0 and stays below 1 + |g| elsewhere), so outputs
    agree to a few bf16 steps of the root mean square."""
    cfg, Rw, b, W, x, *_ , g = layer_inputs()
    s = S.moe_shape(cfg)
    layer = M.MoELayer(s, Rw, b, W["w13"], W["w2"], gamma=0.0)
    layer.forward(x)
    w1, w3 = unpack13(W["w13"].view(cfg.N + 1, 2 * cfg.f, cfg.d)[:cfg.N].contiguous(), cfg.f)
    w2 = W["w2"].view(cfg.N + 1, cfg.d, cfg.f)[:cfg.N].contiguous()
    R = cfg.T * cfg.K
    gate, up = (torch.empty(R, cfg.f, dtype=BF, device="cuda") for _ in range(2))
    M.moe_grouped_matmul(layer.x_perm, layer.offsets, w1, gate, layer.ws)
    M.moe_grouped_matmul(layer.x_perm, layer.offsets, w3, up, layer.ws)
    h = (torch.nn.functional.silu(gate.float()) * up.float()).to(BF)
    y = torch.empty(R, cfg.d, dtype=BF, device="cuda")
    M.moe_grouped_matmul(h, layer.offsets, w2, y, layer.ws)
    rel = S.rel_fro(y.float().cpu().numpy(), layer.y_perm.float().cpu().numpy())
    assert rel <= 4 * 2.0 ** -8, rel
    dy = torch.randn(R, cfg.d, generator=g, device="cuda").to(BF)
    dh, dw2 = torch.empty_like(h), torch.empty_like(w2)
    M.moe_grouped_matmul_dx(dy, layer.offsets, w2, dh, layer.ws)
    M.moe_grouped_matmul_dw(dy, h, layer.offsets, dw2, layer.ws)
    o = layer.offsets.tolist()
    for e in range(cfg.N):
        r = slice(o[e], o[e + 1])
        want = dy[r].double() @ w2[e].double()
        # K products of magnitude sum m in fp32: K 2^-23 m, and one rounding to bf16
        m = dy[r].double().abs() @ w2[e].double().abs()
        assert ((dh[r].double() - want).abs() <= 2.0 ** -8 * want.abs() + (cfg.d + 2) * 2.0 ** -23 * m).all()
        want = dy[r].double().t() @ h[r].double()
        m = dy[r].double().abs().t() @ h[r].double().abs()
        n = max(1, o[e + 1] - o[e])
        assert ((dw2[e].double() - want).abs() <= 2.0 ** -8 * want.abs() + (n + 2) * 2.0 ** -23 * m).all()
    assert layer.device_status() == 0


def test_a_normed_fp8_projection_and_its_gradients(M):
    """LN -> E4M3 rows -> product; backward: E5M2 rows -> input gradient -> LN backward, and the
    weight gradient in bf16 (one expert that owns all rows).  Each step against 64 bits on the
    step's own inputs; the whole against the unquantised chain, within the formats' half steps:
    relative 2^-4 (E4M3 rows and weights) or 2^-3 (E5M2) per element, which average out over a row,
    so 2^-4 and 2^-3 bound the results' relative error with room."""
    g = torch.Generator(device="cuda").manual_seed(5)
    T, d, n = 517, 768, 400
    x = (torch.randn(T, d, generator=g, device="cuda") * 3 + 1).to(BF)
    nw = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    w = (torch.randn(1, n, d, generator=g, device="cuda") / d ** 0.5).to(BF)
    ws = torch.zeros(M.matmul_workspace_size(), dtype=torch.uint8, device="cuda")
    E4, E5, f32 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float32
    emp = lambda *sh, dt=f32: torch.empty(*sh, dtype=dt, device="cuda")  # noqa: E731
    wq, wsc = emp(1, n, d, dt=E4), emp(1, -(-n // 128), -(-d // 128))
    M.moe_quantize_blocks_fp8(w, wq, wsc)
    xn, mean, rstd = emp(T, d, dt=BF), emp(T), emp(T)
    M.moe_layer_norm(x, nw, None, 1e-5, xn, mean, rstd)
    xq, xs = emp(T, d, dt=E4), emp(-(-d // 128), T)
    M.moe_quantize_rows_fp8(xn, xq, xs)
    y = emp(T, n, dt=BF)
    M.moe_matmul_fp8(xq, xs, None, wq, wsc, y, ws)
    want = xn.double() @ w[0].double().t()
    assert S.rel_fro(y.double().cpu().numpy(), want.cpu().numpy()) <= 2.0 ** -4
    dy = torch.randn(T, n, generator=g, device="cuda").to(BF)
    dq, ds = emp(T, n, dt=E5), emp(-(-n // 128), T)
    M.moe_quantize_rows_fp8(dy, dq, ds)
    dxn, dw = emp(T, d, dt=BF), emp(1, n, d, dt=BF)
    M.moe_matmul_fp8_dx(dq, ds, None, wq, wsc, dxn, ws)
    M.moe_grouped_matmul_dw(dy, xn, None, dw, ws)
    dx, dnw = emp(T, d, dt=BF), emp(d)
    lws = emp(M.layer_norm_workspace_size(T, d), dt=torch.uint8)
    M.moe_layer_norm_backward(dxn, x, nw, mean, rstd, dx, dnw, None, lws)
    # autograd in 64 bits on the unquantised chain
    x64, w64, g64 = x.double().requires_grad_(), w[0].double().requires_grad_(), nw.double().requires_grad_()
    torch.nn.functional.layer_norm(x64, (d,), g64, None, 1e-5).matmul(w64.t()).backward(dy.double())
    for got, ref, tol in ((dx, x64.grad, 2.0 ** -3), (dw[0], w64.grad, 2.0 ** -7), (dnw, g64.grad, 2.0 ** -3)):
        assert S.rel_fro(got.double().cpu().numpy(), ref.cpu().numpy()) <= tol
    assert M.moe_read_device_status(ws) == 0
    assert np.isfinite(y.float().cpu().numpy()).all()


def test_calls_on_several_streams_at_once(M):
    """Every operator on its own stream, all sharing one status workspace, many times over: the
    results are those of calls made one after another."""
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *sh, dt=BF: torch.randn(*sh, generator=g, device="cuda").to(dt)  # noqa: E731
    ws = torch.zeros(M.matmul_workspace_size(), dtype=torch.uint8, device="cuda")
    counts = [300, 0, 41, 513, 7, 260]
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    R, E, n, k = sum(counts), len(counts), 1160, 392
    x, dy, w = rnd(R, k), rnd(R, n), rnd(E, n, k)
    x32, w32 = x.float(), w.float()
    E4 = torch.float8_e4m3fn
    xq, xs = torch.empty(R, 400, dtype=E4, device="cuda"), torch.empty(4, R, device="cuda")
    x400, w400 = rnd(R, 400), rnd(E, n, 400)
    wq = torch.empty(E, n, 400, dtype=E4, device="cuda")
    wsc = torch.empty(E, -(-n // 128), 4, device="cuda")
    M.moe_quantize_blocks_fp8(w400, wq, wsc)
    few = rnd(3, k)
    d = 1536
    nx, nw, ndy = rnd(700, d), rnd(d, dt=torch.float32), rnd(700, d)
    mean, rstd = torch.empty(700, device="cuda"), torch.empty(700, device="cuda")
    lws = torch.empty(M.layer_norm_workspace_size(700, d), dtype=torch.uint8, device="cuda")
    e = lambda *sh, dt=BF: torch.empty(*sh, dtype=dt, device="cuda")  # noqa: E731
    y, dx, dw, y32, y8, yf = (e(R, n), e(R, k), e(E, n, k), e(R, n, dt=torch.float32), e(R, n),
                              e(3, n))
    ny, ndx, ndw = e(700, d), e(700, d), e(d, dt=torch.float32)

    def fp8(st):
        M.moe_quantize_rows_fp8(x400, xq, xs, st)
        M.moe_matmul_fp8(xq, xs, off, wq, wsc, y8, ws, st)

    def norm(st):
        M.moe_layer_norm(nx, nw, None, 1e-5, ny, mean, rstd, st)
        M.moe_layer_norm_backward(ndy, nx, nw, mean, rstd, ndx, ndw, None, lws, st)
    jobs = [(lambda st: M.moe_grouped_matmul(x, off, w, y, ws, st), [y]),
            (lambda st: M.moe_grouped_matmul_dx(dy, off, w, dx, ws, st), [dx]),
            (lambda st: M.moe_grouped_matmul_dw(dy, x, off, dw, ws, st), [dw]),
            (lambda st: M.moe_grouped_matmul(x32, off, w32, y32, ws, st), [y32]),
            (lambda st: M.moe_grouped_matmul(few, None, w[:1], yf, ws, st), [yf]),
            (fp8, [y8]), (norm, [ny, ndx, ndw])]
    alone = []
    for job, outs in jobs:
        job(None)
        alone.append([t.clone() for t in outs])
        for t in outs:
            t.fill_(3.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(25):
        for (job, _o), st in zip(jobs, streams):
            job(st)
    torch.cuda.synchronize()
    for (_j, outs), want in zip(jobs, alone):
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    assert M.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("dtype", [1, 3], ids=["bf16", "e4m3"])
def test_bad_offsets_on_a_layers_workspace_do_not_disturb_the_layer(M, dtype):
    """Any workspace serves the products.  Bad offsets leave their bit in the layer's status word;
    the layer's own kernels, whose waits are long here, still finish."""
    cfg = CONFIGS[dtype].with_(T=2048, d=1024, N=16, K=4, G=4, topG=2, f=512)
    s = S.moe_shape(cfg)
    Rw, b = torch.from_numpy(gen.make_router(cfg)).cuda(), torch.from_numpy(gen.make_bias(cfg)).cuda()
    W = S.device_weights(cfg)
    x = S.to_dev_x(gen.make_x(cfg, 0, 0), cfg)
    layer = M.MoELayer(s, Rw, b, W["w13"], W["w2"], W.get("w13_scales"), W.get("w2_scales"), gamma=0.0)
    want = layer.forward(x).clone()
    g = torch.Generator(device="cuda").manual_seed(12)
    rows, w = (torch.randn(*sh, generator=g, device="cuda").to(BF) for sh in ((40, 64), (3, 32, 64)))
    off = torch.tensor([0, 10, 5, 40], dtype=torch.int32, device="cuda")
    for _ in range(20):
        M.moe_grouped_matmul(rows, off, w, torch.empty(40, 32, dtype=BF, device="cuda"), layer.ws)
        layer.y.zero_()
        assert torch.equal(layer.forward(x), want)
        assert layer.device_status() == 4      # MOE_DEV_BAD_INDEX, and nothing else
