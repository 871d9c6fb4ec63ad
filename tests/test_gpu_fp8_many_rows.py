"""The FP8 matmul at sizes beyond the few-row kernel, against 64-bit products:
odd and even numbers of 128-wide slices, more units than CTAs, output rows that
do not start on 16 bytes, ragged rows, both row formats.

Rows and weights have a power of two of their own for every scaled tile, so that
a scale taken from another tile shows.  Tolerances as in
test_gpu_grouped_matmul.py: a whole fp32 step per addition and two more for the
scales' product and the multiply-add, and one rounding to bf16."""
import pytest
import torch

from tests.test_gpu_grouped_matmul import (BF, E4M3, E5M2, close, dequant_blocks, dequant_rows,
                                           expected, gen, offsets_of, rand)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import sparse_moe_layer_limited_b200 as M
    return M


def few_rows(R, E, cols):
    """The rule that gives a call to the few-row kernel: units of at most 64 rows by 128 columns
    that all fit on the SMs at once."""
    tiles = -(-R // 64) if E == 1 else R // 64 + min(R, E)
    return tiles * -(-cols // 128) <= torch.cuda.get_device_properties(0).multi_processor_count


def tiles_of_their_own_size(t, g, rows, cols):
    """t [.., n, k] times a power of two, 2^-4 to 2^4, for each block of rows x cols."""
    n, k = t.shape[-2:]
    e = torch.randint(-4, 5, (*t.shape[:-2], -(-n // rows), -(-k // cols)), generator=g, device="cuda")
    f = torch.exp2(e.float()).repeat_interleave(rows, -2)[..., :n, :].repeat_interleave(cols, -1)[..., :k]
    return (t.float() * f).to(t.dtype)


@pytest.mark.parametrize("fmt", [E4M3, E5M2], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("counts,lead,behind,n,k", [
    ([1300], 0, 0, 1041, 1040),                                 # 9 slices
    ([1300], 0, 0, 1040, 2048), ([9000], 0, 0, 1024, 144),      # 16 and 2
    ([4100], 0, 0, 2099, 1168), ([20000], 0, 0, 520, 16),
    ([0, 700, 129, 31, 1, 640], 3, 7, 1168, 1296),              # 11 slices, 75 units
    ([0, 3000, 129, 31, 1, 2000, 515], 1, 2, 2319, 400),        # more units than SMs
    ([33 * e for e in range(60)], 0, 5, 272, 1040)])
@pytest.mark.parametrize("mode", ["fwd", "dx"])
def test_many_rows(M, mode, counts, lead, behind, n, k, fmt):
    if mode == "dx":
        n, k = (k + 15) // 16 * 16, (n + 15) // 16 * 16         # the same output and contraction
    g = gen(30)
    R, E = lead + sum(counts) + behind, len(counts)
    cin, cout = (k, n) if mode == "fwd" else (n, k)
    assert not few_rows(R, E, cout)
    a = tiles_of_their_own_size(rand(g, R, cin, dtype=BF), g, 1, 128)
    w = tiles_of_their_own_size(rand(g, E, n, k, dtype=BF, scale=0.1), g, 128, 128)
    qa = torch.empty(R, cin, dtype=fmt, device="cuda")
    sa = torch.full((-(-cin // 128), R + 3), float("nan"), device="cuda")
    qw = torch.empty(E, n, k, dtype=E4M3, device="cuda")
    sw = torch.empty(E, -(-n // 128), -(-k // 128), device="cuda")
    M.moe_quantize_rows_fp8(a, qa, sa)
    M.moe_quantize_blocks_fp8(w, qw, sw)
    sa[:, :lead] = float("nan")
    sa[:, R - behind:] = float("nan")
    ws = torch.zeros(M.matmul_workspace_size(), dtype=torch.uint8, device="cuda")
    out = torch.full((R, cout), 7.0, dtype=BF, device="cuda")
    f = M.moe_matmul_fp8 if mode == "fwd" else M.moe_matmul_fp8_dx
    f(qa, sa, offsets_of(counts, lead) if E > 1 else None, qw, sw, out, ws)
    want, mag = expected(mode, dequant_rows(qa, sa), dequant_blocks(qw, sw), counts, lead, n, k)
    own = slice(lead, R - behind)
    close(out[own], want[own], mag[own], cin + 2)
    assert (out[:lead] == 7.0).all() and (out[R - behind:] == 7.0).all()
    again = torch.full_like(out, 7.0)
    for _ in range(3):
        f(qa, sa, offsets_of(counts, lead) if E > 1 else None, qw, sw, again, ws)
        assert torch.equal(again, out)
    assert M.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("fmt", [E4M3, E5M2], ids=["e4m3", "e5m2"])
def test_many_rows_keep_infinities_and_nan_to_their_rows(M, fmt):
    """Non-finite rows (their scales included) and an expert's non-finite weight scales stay in
    their own results."""
    g = gen(31)
    counts, n, k = [700, 300, 900], 1032, 656
    R, off = sum(counts), offsets_of(counts)
    assert not few_rows(R, 3, n)
    a, w = rand(g, R, k, dtype=BF), rand(g, 3, n, k, dtype=BF)
    a[5] = float("inf")
    a[1200, 300] = float("nan")
    qa, sa = torch.empty(R, k, dtype=fmt, device="cuda"), torch.empty(-(-k // 128), R, device="cuda")
    qw = torch.empty(3, n, k, dtype=E4M3, device="cuda")
    sw = torch.empty(3, -(-n // 128), -(-k // 128), device="cuda")
    M.moe_quantize_rows_fp8(a, qa, sa)
    M.moe_quantize_blocks_fp8(w, qw, sw)
    sw[1] = float("nan")
    out = torch.empty(R, n, dtype=BF, device="cuda")
    ws = torch.zeros(M.matmul_workspace_size(), dtype=torch.uint8, device="cuda")
    M.moe_matmul_fp8(qa, sa, off, qw, sw, out, ws)
    bad = torch.zeros(R, dtype=torch.bool, device="cuda")
    bad[5] = bad[1200] = True
    bad[700:1000] = True
    assert out[bad].isnan().all() and out[~bad].isfinite().all()
    assert M.moe_read_device_status(ws) == 0
