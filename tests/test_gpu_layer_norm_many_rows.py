"""Layer norm where a CTA takes many rows: the ring's slots are refilled and their
barriers' phases turn, the register kernels load the next row while one is
reduced, and the column sums run over many rows of a thread.  Bounds as in
test_gpu_layer_norm.py (they hold for any number of rows)."""
import threading

import pytest
import torch

from synth import CONFIGS, gen
from tests import support as S
from tests import test_gpu_layer_norm as T

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    import sparse_moe_layer_limited_b200 as M
    return M


def by_copies(d, dtype):
    """Rows of whole 16-byte pieces up to 32 KB go through the ring of bulk copies."""
    size = 2 if dtype == BF else 4
    return d * size % 16 == 0 and d * size <= 32768


# rows for at least a dozen to a CTA: the ring holds 6 (3 in the backward of wide rows), and a CTA
# of 32 x t threads is one of 16 / t on an SM
RING = [(12000, 40), (16000, 1032), (9000, 2048), (9000, 3000), (4000, 5000), (4000, 7000),
        (5000, 7168), (2500, 8192), (2500, 12296), (2500, 16384)]
RING32 = [(16000, 36), (12000, 1028), (5000, 2052), (4000, 4096), (4000, 5004), (2500, 7168),
          (2500, 8192)]
# at least two rows to a group of threads
REGISTERS = [(20000, 33), (12000, 250), (10000, 511), (12000, 1001), (6000, 2047), (6000, 3001),
             (4000, 6001), (1500, 9999), (1500, 16383)]


@pytest.mark.parametrize("R,d,dtype", [(*s, BF) for s in RING] + [(*s, F32) for s in RING32])
def test_rows_through_the_ring(M, R, d, dtype):
    assert by_copies(d, dtype) and R >= 148 * 16
    T.test_forward_and_backward(M, R, d, dtype)


@pytest.mark.parametrize("R,d,dtype", [(*s, t) for s in REGISTERS for t in (BF, F32)]
                         + [(1500, 12000, F32), (1500, 16384, F32)])
def test_rows_through_registers(M, R, d, dtype):
    assert not by_copies(d, dtype)
    T.test_forward_and_backward(M, R, d, dtype)


@pytest.mark.parametrize("R", [40, 2500])
@pytest.mark.parametrize("d", [40, 1032, 4096, 5000, 7168, 8188])
def test_a_large_common_offset_does_not_cancel(M, d, R):
    x, w, b, _ = T.make(R, d, F32, seed=3, shift=3.0e4)
    T.check_forward(x, w, b, 1e-5, *T.forward(M, x, w, b, 1e-5))
    # The variance itself.  Squares are summed around a mean m' that is off by at most e = 64 u times
    # the mean magnitude (the bound on a row sum), and sum (x - m')^2 / n = var + (m' - m)^2, so that
    # part is at most e^2; two parts whose means are each off by e and differ by D are merged with
    # (D +- 2 e)^2 in place of D^2 and D is at most the spread, so at most 4 e sqrt(var) + 4 e^2;
    # the fp32 sums and rsqrt add 128 u of the variance.  (Here e is 0.115 and the standard deviations
    # 0.02 to 20; differences of squares would be off by u 9e8 = 54.)
    var = x.double().var(1, unbiased=False)
    _, _, rstd = T.forward(M, x, w, b, 0.0)
    e = 64 * T.U * x.double().abs().mean(1)
    bound = 128 * T.U * var + 4 * e * var.sqrt() + 5 * e.square()
    assert ((rstd.double() ** -2 - var).abs() <= bound).all()


def test_two_host_threads_get_their_own_gradients(M):
    """Calls of one process at the same time, on streams of their own, rows of different widths."""
    cases, errors = [], []
    for d in (1032, 6144, 7680):
        x, w, b, dy = T.make(2400, d, BF, seed=d)
        y, mean, rstd = T.forward(M, x, w, b, 1e-5)
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
        ws = torch.empty(M.layer_norm_workspace_size(*x.shape), dtype=torch.uint8, device="cuda")
        M.moe_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
        cases.append((x, w, b, dy, mean, rstd, (y, dx, dw, db)))
    torch.cuda.synchronize()

    def work(x, w, b, dy, mean, rstd, want):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                got = [torch.empty_like(t) for t in want]
                m, r = torch.empty_like(mean), torch.empty_like(rstd)
                ws = torch.empty(M.layer_norm_workspace_size(*x.shape), dtype=torch.uint8,
                                 device="cuda")
                for _ in range(8):
                    for t in got:
                        t.fill_(3.0)
                    for _ in range(40):
                        M.moe_layer_norm(x, w, b, 1e-5, got[0], m, r)
                        M.moe_layer_norm_backward(dy, x, w, mean, rstd, *got[1:], ws)
                    st.synchronize()
                    assert all(torch.equal(g, t) for g, t in zip(got, want))
                    assert torch.equal(m, mean) and torch.equal(r, rstd)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_a_graph_writes_the_forward_too(M):
    x, w, b, dy = T.make(3000, 1536, BF, seed=7)
    want = T.forward(M, x, w, b, 1e-5)
    y, mean, rstd = (torch.empty_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_layer_norm(x, w, b, 1e-5, y, mean, rstd)
    for _ in range(2):
        for t in (y, mean, rstd):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((y, mean, rstd), want))


@pytest.mark.parametrize("cfg_id", [0, 3], ids=["fp32", "e4m3"])
@pytest.mark.parametrize("bias", [True, False])
def test_a_layer_of_another_type_with_a_norm(M, cfg_id, bias):
    cfg = CONFIGS[cfg_id]
    if cfg_id == 3:
        cfg = cfg.with_(T=300, d=256, N=8, K=2, G=2, topG=1, f=256)
    s = S.moe_shape(cfg)
    Rw, b = torch.from_numpy(gen.make_router(cfg)).cuda(), torch.from_numpy(gen.make_bias(cfg)).cuda()
    W = S.device_weights(cfg)
    x = S.to_dev_x(gen.make_x(cfg, 0, 0), cfg)
    g = torch.Generator(device="cuda").manual_seed(4)
    nw = 1 + 0.2 * torch.randn(cfg.d, generator=g, device="cuda")
    nb = 0.1 * torch.randn(cfg.d, generator=g, device="cuda") if bias else None
    args = (W["w13"], W["w2"], W["w13_scales"], W["w2_scales"])
    normed = M.MoELayer(s, Rw, b.clone(), *args, gamma=1e-3, norm_w=nw, norm_b=nb)
    plain = M.MoELayer(s, Rw, b.clone(), *args, gamma=1e-3)
    xn = torch.empty_like(x)
    mean, rstd = torch.empty(cfg.T, device="cuda"), torch.empty(cfg.T, device="cuda")
    M.moe_layer_norm(x, nw, nb, 1e-5, xn, mean, rstd)
    assert torch.equal(normed.forward(x), plain.forward(xn))
    assert torch.equal(normed.topk_idx, plain.topk_idx) and torch.equal(normed.bias, plain.bias)
    assert normed.device_status() == 0
