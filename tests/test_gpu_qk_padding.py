"""GPU: a padded token's outputs and gradients are zero whatever the norm's
weights hold, as they are whatever the token's buffers hold."""
import pytest
import torch

from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu
TABLE = 40


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("t,hq,hk,d,rot,G", [(5, 3, 1, 64, 64, 16), (6, 4, 2, 128, 128, 128), (4, 5, 3, 80, 48, 16),
                                             (600, 8, 8, 256, 128, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_weights_that_are_not_finite(t, hq, hk, d, rot, G, interleaved):
    coat = lib()
    g = torch.Generator().manual_seed(t + d)
    x = torch.randn(t, hq + hk, d, generator=g).bfloat16().to(DEV)
    dy = torch.randn(t, hq + hk, d, generator=g).bfloat16().to(DEV)
    cos, sin = [torch.randn(TABLE, rot // 2, generator=g).to(DEV) for _ in range(2)]
    pos = torch.randint(0, TABLE, (t,), generator=g)
    pos[1], pos[-1] = -1, TABLE
    dead = ((pos < 0) | (pos >= TABLE)).to(DEV)
    pos = pos.to(DEV)
    good = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    wq, wk = good.clone(), good.clone()
    wq[3], wq[d // 2], wq[d - 1] = float("inf"), float("nan"), -float("inf")
    wk[:] = float("nan")
    ws = torch.empty(coat.qk_norm_rope_bwd_workspace(t, hq + hk, d), dtype=torch.uint8, device=DEV)

    def run(wq, wk):
        dx = torch.full_like(x, 7.0)
        o = dict(codes=torch.full((t, hq + hk, d), 0x55, dtype=torch.uint8, device=DEV),
                 scales=torch.full((t, hq + hk, d // G), 7.0, device=DEV), rstd=torch.full((t, hq + hk), 7.0, device=DEV))
        qo, ko = [torch.full((t, h, d), 7.0, dtype=torch.bfloat16, device=DEV) for h in (hq, hk)]
        coat.qk_norm_rope(x[:, :hq], x[:, hq:], wq, wk, 1e-5, cos, sin, pos, qo, ko, interleaved=interleaved,
                          group_size=G, **o)
        dw = torch.full((2, d), 7.0, device=DEV)
        coat.qk_norm_rope_bwd(dy[:, :hq], dy[:, hq:], *o.values(), wq, wk, cos, sin, pos, dx[:, :hq], dx[:, hq:], dw[0],
                              dw[1], workspace=ws, interleaved=interleaved, group_size=G)
        return (qo, ko, dx, *o.values()), dw

    written, dw = run(wq, wk)
    for v in written:
        assert (v[dead] == 0).all()
    assert written[0][~dead].isnan().any() and written[1][~dead].isnan().any()   # the weights do reach the others
    # the weights' gradients do not read the weights
    assert torch.equal(dw, run(good, good)[1]) and dw.isfinite().all()
