"""GPU: the activation operators where offsets pass 32 bits (arrays over 4 GiB)
and where one call's rows are another's: the last rows of a long call equal a
call on those rows alone, bit for bit."""
import pytest
import torch

from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu
LAST = 96


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def filled(rows, cols, seed, dtype=torch.bfloat16):
    """Rows of zeros but for the last ones."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.zeros(rows, cols, dtype=dtype, device=DEV)
    x[-LAST:] = torch.randn(LAST, cols, device=DEV, generator=g).to(dtype)
    return x


def test_norm():
    coat = lib()
    rows, cols, G = 1_100_000, 2048, 128   # 4.5 GB of BF16
    x = filled(rows, cols, 0)
    w = torch.randn(cols, device=DEV).bfloat16()

    def forward(x):
        n = x.shape[0]
        o = dict(y=torch.empty_like(x), codes=torch.empty(n, cols, dtype=torch.uint8, device=DEV),
                 scales=torch.empty(n, cols // G, device=DEV), rstd=torch.empty(n, device=DEV))
        coat.rms_norm(x, w, 1e-5, group_size=G, **o)
        return o

    def backward(x, o):
        dx, dw = torch.empty_like(x), torch.empty(cols, device=DEV)
        ws = torch.empty(coat.rms_norm_bwd_workspace(*x.shape), dtype=torch.uint8, device=DEV)
        coat.rms_norm_bwd(x, o["codes"], o["scales"], o["rstd"], w, dx, dw, workspace=ws, group_size=G)
        return dx

    big, small = forward(x), forward(x[-LAST:].contiguous())
    for k in big:
        assert torch.equal(big[k][-LAST:], small[k]), k
    assert torch.equal(backward(x, big)[-LAST:], backward(x[-LAST:].contiguous(), small))


def test_swiglu():
    coat = lib()
    rows, cols, G = 600_000, 2048, 64      # 4.9 GB of gates and ups
    x = filled(rows, 2 * cols, 1)

    def run(x):
        n = x.shape[0]
        o = (torch.empty(n, cols, dtype=torch.bfloat16, device=DEV), torch.empty(n, 2 * cols, dtype=torch.uint8, device=DEV),
             torch.empty(n, 2 * cols // G, device=DEV), torch.empty_like(x))
        coat.swiglu(o[1], o[2], gate_up=x, h=o[0], group_size=G)
        coat.swiglu_bwd(o[0], o[1], o[2], o[3], group_size=G)
        return o

    for a, b in zip(run(x), run(x[-LAST:].contiguous())):
        assert torch.equal(a[-LAST:], b)


def test_qk():
    coat = lib()
    t, hq, hk, d = 180_000, 64, 16, 128    # packed rows of 96 heads: 4.4 GB
    qkv = filled(t, (hq + 2 * hk) * d, 2)
    w = torch.randn(2, d, device=DEV).bfloat16()
    table = torch.randn(2, 50, d // 2, device=DEV)
    pos = torch.arange(t, device=DEV) % 50

    def run(qkv, pos):
        n = qkv.shape[0]
        q, k = qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        o = dict(q_out=torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV),
                 k_out=torch.empty(n, hk, d, dtype=torch.bfloat16, device=DEV),
                 codes=torch.empty(n, hq + hk, d, dtype=torch.uint8, device=DEV),
                 scales=torch.empty(n, hq + hk, 1, device=DEV), rstd=torch.empty(n, hq + hk, device=DEV))
        coat.qk_norm_rope(q, k, w[0], w[1], 1e-5, table[0], table[1], pos, **o)
        coat.qk_norm_rope_bwd(o["q_out"], o["k_out"], o["codes"], o["scales"], o["rstd"], w[0], w[1], table[0],
                              table[1], pos, q, k)   # the gradients over the inputs
        return (*o.values(), q, k)

    small = run(qkv[-LAST:].clone(), pos[-LAST:].clone())
    for a, b in zip(run(qkv, pos), small):
        assert torch.equal(a[-LAST:], b)


@pytest.mark.parametrize("n,k", [(2048, 128), (4096, 4096)])
def test_weight_grad(n, k):
    """Small integers, so that the order of the sums does not matter."""
    coat = lib()
    rows = (1 << 32) // (2 * n) + 5000
    g = torch.Generator(device=DEV).manual_seed(3)
    dy = torch.zeros(rows, n, dtype=torch.bfloat16, device=DEV)
    dy[-LAST:] = torch.randint(-8, 9, (LAST, n), device=DEV, generator=g).bfloat16()
    codes = torch.zeros(rows, k, dtype=torch.uint8, device=DEV)
    codes[-LAST:] = torch.randint(-8, 9, (LAST, k), device=DEV, generator=g).float().to(torch.float8_e4m3fn).view(torch.uint8)

    def run(dy, codes):
        dw = torch.empty(n, k, device=DEV)
        ws = torch.empty(coat.weight_grad_workspace(dy.shape[0], n, k), dtype=torch.uint8, device=DEV)
        coat.weight_grad(dy, codes, 1.0, dw, workspace=ws)
        return dw

    assert torch.equal(run(dy, codes), run(dy[-LAST:].contiguous(), codes[-LAST:].contiguous()))


def test_residual_in_place():
    """residual_out may be the residual itself, at every kind of row length."""
    coat = lib()
    for cols in (512, 4096, 8192, 16384, 32768):
        x, r = [torch.randn(40, cols, device=DEV).bfloat16() for _ in range(2)]
        w = torch.randn(cols, device=DEV).bfloat16()
        out, y, y2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        coat.rms_norm(x, w, 1e-5, residual=r, residual_out=out, y=y)
        coat.rms_norm(x, w, 1e-5, residual=r, residual_out=r, y=y2)
        assert torch.equal(r, out) and torch.equal(y, y2)
