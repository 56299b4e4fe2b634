"""e4m3 products whose rows, weights or outputs lie beyond 2^31 and 2^32 bytes
and elements, and the most rows: a sample of rows and outputs against 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from moe_util import DEV, HALF, TINY, U, blocks, ints, product  # noqa: E402
from test_gemm_e4m3 import E4M3, call, qg  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def far_codes(shape, seed):
    """Any codes but NaN, made on the device."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = t.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randint(0, 0x70, part.shape, generator=g, device=DEV, dtype=torch.uint8))
        part |= torch.randint(0, 2, part.shape, generator=g, device=DEV, dtype=torch.uint8) << 7
    return t.view(E4M3)


def far_scales(shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.exp(torch.rand(shape, generator=g, device=DEV) * 4.6 - 9.2)


def near(y, want, mag, i, yt):
    """The f32 additions that test_gemm_e4m3_sums counts, and the output's rounding."""
    slack = (265 + blocks(i)) * U * mag
    return bool(((y.double() - want).abs() <= slack + HALF[yt] * (want.abs() + slack) + TINY[yt]).all())


@pytest.mark.parametrize("m,i,o", [(400001, 8192, 130), (400001, 8191, 20), (300007, 128, 8200), (300007, 120, 8200),
                                   (65535 * 64, 16, 24), (65535 * 64, 8, 24), (3, 16384, 270000), (100, 16384, 270000)])
def test_far_dense(qg, m, i, o):  # noqa: F811
    x, w = far_codes((m, i), 1), far_codes((1, o, i), 2)
    xs, ws = far_scales((m, blocks(i)), 3), far_scales((1, blocks(o), blocks(i)), 4)
    y = torch.full((m, o), 7.0, dtype=torch.bfloat16, device=DEV)
    qg.check(call(qg, y, x, xs, w, ws))
    # the first and last rows and outputs, and the ones around 2^31 and 2^32 bytes of the rows, weights and outputs
    rows = sorted({r for b in (0, m, 2 ** 31 // i, 2 ** 32 // i, 2 ** 31 // (2 * o), 2 ** 32 // (2 * o)) for r in range(b - 40, b + 40)
                   if 0 <= r < m})
    outs = sorted({n for b in (0, o, 2 ** 31 // i, 2 ** 32 // i) for n in range(b - 40, b + 40) if 0 <= n < o})
    scale = ws[0].repeat_interleave(128, 0)[:o][outs].repeat_interleave(128, 1)[:, :i].double()
    wd = w[0].view(torch.uint8)[outs].view(E4M3).double() * scale
    xd = x.view(torch.uint8)[rows].view(E4M3).double() * xs[rows].double().repeat_interleave(128, 1)[:, :i]
    assert near(y[rows][:, outs], xd @ wd.t(), xd.abs() @ wd.abs().t(), i, "bf16")


@pytest.mark.parametrize("i,per", [(16384, 1), (16384, 200), (16376, 1)])
def test_far_experts(qg, i, per):  # noqa: F811
    experts, o = 40, 8192                                     # 5.4 GB of weights
    bounds = [per * e for e in range(experts + 1)]
    m = bounds[-1]
    x, w = far_codes((m, i), 1), far_codes((experts, o, i), 2)
    xs, ws = far_scales((m, blocks(i)), 3), far_scales((experts, blocks(o), blocks(i)), 4)
    y = torch.full((m, o), 7.0, device=DEV)
    qg.check(call(qg, y, x, xs, w, ws, ints(bounds)))
    for e in (0, 15, 16, 31, 32, experts - 1):
        a, b = bounds[e], bounds[e + 1]
        for o0 in (0, o - 256):
            want, mag = product(x[a:b], xs[a:b], w[e:e + 1, o0:o0 + 256], ws[e:e + 1, o0 // 128:o0 // 128 + 2], [0, b - a])
            assert near(y[a:b, o0:o0 + 256], want, mag, i, "f32"), (e, o0)
