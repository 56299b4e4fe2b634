"""Tables of offsets that decrease or leave the rows: one rule in every kernel
of the e4m3 products, which rows are written and with whose weights, row by row
against 64 bits, and the error word."""
import pytest

torch = pytest.importorskip("torch")

from moe_util import DEV, blocks, guarded, ints, product, unharmed  # noqa: E402
from test_gemm_e4m3 import call, codes, held, qg, scales  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def ranges(table, m):
    """Expert e's rows go from the largest of offsets[0 .. e] to the largest of offsets[0 .. e + 1], each held to [0, m]."""
    most, out = min(max(table[0], 0), m), []
    for hi in table[1:]:
        to = max(most, min(max(hi, 0), m))
        out.append((most, to))
        most = to
    return out


def check_table(qg, table, m, i, o, bad=True):  # noqa: F811
    e = len(table) - 1
    x, w = codes((m, i), 1, 20.0), codes((e, o, i), 2, 20.0)
    xs, ws = scales((m, blocks(i)), 3, False), scales((e, blocks(o), blocks(i)), 4, False)
    y = guarded((m, o), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws, ints(table)))
    assert qg.qg_device_status() == (qg.QG_OK, qg.QG_EEXPERT if bad else qg.QG_OK)
    assert qg.qg_device_status() == (qg.QG_OK, qg.QG_OK)
    none = torch.ones(m, dtype=torch.bool, device=DEV)
    for g, (a, b) in enumerate(ranges(table, m)):
        if a == b:
            continue
        none[a:b] = False
        want, mag = product(x[a:b], xs[a:b], w[g:g + 1], ws[g:g + 1], [0, b - a])
        assert held(y[a:b], want, mag, "f32"), g
    assert bool((y[none] == 7).all()) and unharmed(y)


# 271 elements: the general kernel; 256 by 128 outputs: few tokens a tile; 1040 by 1300 and 75 times the rows: many
@pytest.mark.parametrize("i,o,times", [(271, 128, 1), (256, 128, 1), (271, 70, 5), (1040, 1300, 75)])
@pytest.mark.parametrize("table", [[0, 10, 5, 30], [-5, 10, 20, 30], [0, 10, 20, 99], [40, 50, 2 ** 31 - 1, -2 ** 31],
                                   [30, 10, 40, 20], [20, 0, 0, 33], [-3, -2, -1, 40], [0, 40, 0, 40], [-2 ** 31, 2 ** 31 - 1, 0, 3]])
def test_every_kernel_holds_a_table_alike(qg, table, i, o, times):  # noqa: F811
    most = 2 ** 31 - 1
    check_table(qg, [v if abs(v) >= most else v * times for v in table], 40 * times, i, o)
