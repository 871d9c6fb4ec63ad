"""The bounded waits of the grouped and FP8 matmuls: a time-out on record in the
status word makes the other waits give up.  Such a call has no result, but it
ends, and after the word is cleared the next call is right again."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def M():
    import sparse_moe_layer_limited_b200 as M
    return M


def rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


def offsets_of(counts):
    return torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()


def bf16_call(M, op, counts, n, k):
    R, E = sum(counts), len(counts)
    off, x, dy, w = offsets_of(counts), rand(1, R, k), rand(2, R, n), rand(3, E, n, k)
    if op == "dw":
        out = torch.empty(E, n, k, dtype=BF, device="cuda")
        return out, lambda ws: M.moe_grouped_matmul_dw(dy, x, off, out, ws)
    out = torch.empty(R, n if op == "fwd" else k, dtype=BF, device="cuda")
    if op == "fwd":
        return out, lambda ws: M.moe_grouped_matmul(x, off, w, out, ws)
    return out, lambda ws: M.moe_grouped_matmul_dx(dy, off, w, out, ws)


def fp8_call(M, op, counts, n, k):
    R, E = sum(counts), len(counts)
    cin, cout = (k, n) if op == "fp8_fwd" else (n, k)
    a, w = rand(4, R, cin), rand(5, E, n, k)
    qa, sa = torch.empty(R, cin, dtype=E4M3, device="cuda"), torch.empty(-(-cin // 128), R).cuda()
    qw = torch.empty(E, n, k, dtype=E4M3, device="cuda")
    sw = torch.empty(E, -(-n // 128), -(-k // 128), device="cuda")
    M.moe_quantize_rows_fp8(a, qa, sa)
    M.moe_quantize_blocks_fp8(w, qw, sw)
    out = torch.empty(R, cout, dtype=BF, device="cuda")
    f = M.moe_matmul_fp8 if op == "fp8_fwd" else M.moe_matmul_fp8_dx
    off = offsets_of(counts)
    return out, lambda ws: f(qa, sa, off, qw, sw, out, ws)


@pytest.mark.parametrize("op,counts,n,k", [
    ("fwd", [3, 0, 40], 1032, 4104), ("fwd", [1], 264, 7168),          # few rows, split and not
    ("fwd", [600, 0, 411, 33], 2056, 2048), ("dx", [600, 0, 411, 33], 1032, 4104),
    ("fwd", [511, 300] * 20, 4096, 1024), ("dx", [511, 300] * 20, 1024, 4096),  # two row tiles a unit
    ("dw", [9000], 136, 264),                                          # split over clusters
    ("dw", [1001, 0, 777, 64], 2056, 1032), ("dw", [130] * 40, 1024, 1024),
    ("fp8_fwd", [7], 1000, 4096), ("fp8_dx", [7], 4096, 1008),
    ("fp8_fwd", [700, 0, 129, 640], 2049, 2064), ("fp8_dx", [700, 0, 129, 640], 2064, 2048)])
def test_a_recorded_time_out(M, op, counts, n, k):
    out, call = (fp8_call if op.startswith("fp8") else bf16_call)(M, op, counts, n, k)
    ws = torch.zeros(M.matmul_workspace_size(), dtype=torch.uint8, device="cuda")
    out.fill_(3.0)
    call(ws)
    torch.cuda.synchronize()
    assert M.moe_read_device_status(ws) == 0
    want = out.clone()
    for _ in range(3):
        ws.view(torch.int32)[0] = 1          # MOE_DEV_WAIT_TIMEOUT
        call(ws)
        torch.cuda.synchronize()
        assert M.moe_read_device_status(ws, clear=True) == 1
        out.fill_(3.0)
        call(ws)
        torch.cuda.synchronize()
        assert M.moe_read_device_status(ws) == 0 and torch.equal(out, want)


def test_a_contraction_that_takes_longer_than_the_limit(M):
    """One of 80 experts owns 700 million rows: one pair of CTAs adds them, for some 2.7 s, and the
    warps that wait for it must not give up after 2.  All but 400 rows are zeros, so the sum has 400
    terms: at most 400 steps of 2^-23 of the terms' magnitudes, and one rounding to bf16."""
    R, E, c = 700_000_005, 80, 8
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    dy, x = (torch.zeros(R, c, dtype=BF, device="cuda") for _ in range(2))
    at = torch.cat([torch.arange(0, R, R // 390 + 1, device="cuda"),
                    torch.arange(R - 17, R, device="cuda")])[-400:]
    dy[at], x[at] = rand(6, len(at), c), rand(7, len(at), c)
    off = torch.full((E + 1,), R, dtype=torch.int32, device="cuda")
    off[0] = 0
    dw = torch.full((E, c, c), 7.0, dtype=BF, device="cuda")
    ws = torch.zeros(M.matmul_workspace_size(), dtype=torch.uint8, device="cuda")
    M.moe_grouped_matmul_dw(dy, x, off, dw, ws)
    assert M.moe_read_device_status(ws) == 0
    a, b = dy[at].double(), x[at].double()
    want, mag = a.t() @ b, a.abs().t() @ b.abs()
    err = mag * 400 * 2.0 ** -23
    err = err + (want.abs() + err) * 2.0 ** -8
    assert ((dw[0].double() - want).abs() <= err).all() and (dw[1:] == 0).all()
    del dy, x
    torch.cuda.empty_cache()
