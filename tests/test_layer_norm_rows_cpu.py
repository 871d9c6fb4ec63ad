"""MoELayer with a norm in front: the calls that read normalised rows refuse
others, before anything is launched (no GPU here)."""
import pytest
import torch

import sparse_moe_layer_limited_b200 as M
from sparse_moe_layer_limited_b200 import build


@pytest.fixture(scope="module", autouse=True)
def library():
    import os
    if not os.path.exists(build.LIB_PATH):
        build.build()


def layer(norm, gather=False, fused=False):
    s = M.shape(T=16, d=256, N=8, K=2, G=2, topG=1, f=256, dtype=M.DTYPE_BF16)
    z = lambda *sh, dt=torch.float32: torch.zeros(*sh, dtype=dt)  # noqa: E731
    bf = torch.bfloat16
    return M.MoELayer(s, z(8, 256), z(8), z(9, 512, 256, dt=bf), z(9, 256, 256, dt=bf),
                      gather=gather, fused_combine=fused, norm_w=torch.ones(256) if norm else None)


@pytest.mark.parametrize("how", [{}, dict(gather=True), dict(fused=True)])
@pytest.mark.parametrize("call", ["experts", "experts_and_combine"])
def test_rows_before_the_norm_are_refused(call, how):
    m = layer(True, **how)
    with pytest.raises(ValueError, match="norm"):
        getattr(m, call)(torch.zeros(16, 256, dtype=torch.bfloat16))
    # the rows after it pass this check, and so do any without a norm: the next one names the device
    for m, x in ((m, m.x_norm), (layer(False, **how), torch.zeros(16, 256, dtype=torch.bfloat16))):
        with pytest.raises(Exception) as e:
            getattr(m, call)(x)
        assert "norm(x)" not in str(e.value)


def test_rows_after_the_norm_are_refused():
    m = layer(True)
    dy = torch.zeros(16, 256, dtype=torch.bfloat16)
    for call in (m.norm, m.route, m.forward, lambda x: m.backward(x, dy, None, None)):
        with pytest.raises(ValueError, match="before the norm"):
            call(m.x_norm)
    with pytest.raises(Exception) as e:
        m.forward(dy)
    assert "before the norm" not in str(e.value)
