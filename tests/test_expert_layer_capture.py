"""The expert-layer example's warm-up and capture: they wait for what the
current stream still has to do, and the program runs."""
import sys

import pytest

torch = pytest.importorskip("torch")

from test_expert_layer import ex, make, randn, slots  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def test_warm_up_waits_for_the_current_stream(ex):  # noqa: F811
    x, (_, ids, weights) = randn(3, 70, 400).bfloat16(), slots(70, 3, 6, 4, 0.1)
    want, out = torch.empty_like(x), torch.empty_like(x)
    make(ex)(want, x, ids, weights)
    layer, late_x, late_ids, late_weights = make(ex), torch.zeros_like(x), torch.zeros_like(ids), torch.zeros_like(weights)
    torch.cuda.Stream()                                       # the process's first one takes as long as the wait below
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                            # some 50 ms before the inputs are there
    for late, t in ((late_x, x), (late_ids, ids), (late_weights, weights)):
        late.copy_(t)
    graph = ex.capture(layer, out, late_x, late_ids, late_weights)
    assert torch.equal(out, want)                             # of the warm-up: a capture runs nothing
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


SMALL = ["expert_layer.py", "--tokens", "130", "--experts", "12", "--top", "4", "--hidden", "256", "--width", "144"]


def test_the_program_reports_the_device_status(ex, monkeypatch):  # noqa: F811
    import weight_only_quantized_i4g_gb300 as qg
    monkeypatch.setattr(sys, "argv", SMALL)
    layer = make(ex)
    layer.offsets.copy_(torch.tensor([0, 9, 5, 12, 12, 12, 12]))                 # decreases
    n = layer.rows
    qg.check(qg.qgemm_e4m3_moe(qg.QG_FMT_FP8B128, layer.gu, qg.QG_BF16, layer.x, layer.x_scale, layer.up, layer.up_scale,
                               layer.offsets, layer.E, n, layer.H, 2 * layer.F))
    with pytest.raises(qg.QGError):
        ex.main()
    assert qg.qg_device_status() == (qg.QG_OK, qg.QG_OK)


def test_the_program_runs(ex, monkeypatch, capsys):  # noqa: F811
    monkeypatch.setattr(sys, "argv", SMALL)
    ex.main()
    assert "130 tokens, 12 experts" in capsys.readouterr().out
