"""layer.py refuses a result that lies over an input: kernels write it while they still read."""
import pytest

torch = pytest.importorskip("torch")


def test_results_over_inputs_are_refused():
    from mixture_experts_layer_35_amd.layer import _apart
    flat = torch.zeros(4000)
    x, w = flat[:600].view(10, 60), flat[600:1600].view(2, 10, 50)
    wide = torch.zeros(20, 100)
    bad = [(x, (w, x)), (flat[599:899].view(10, 30), (x,)), (flat[1590:2000], (x, w)), (wide[:, 30:60], (wide[:, :31],)),
           (wide[:, :31], (wide[:, 30:60],)), (wide[5:, 50:], (wide[:, 20:60],)), (wide[:, 10:20], (wide,)), (wide[3:4], (wide[:4],)),
           (wide.view(-1)[:600].view(10, 60), (wide[:, 60:],)), (x.view(torch.bfloat16)[:, :60], (x,)),
           (wide[::2, :61], (wide[:, 60:],)), (wide[::3], (wide[::2],))]
    for out, inputs in bad:
        with pytest.raises(ValueError, match="shares memory"):
            _apart("out", out, *inputs)
    fine = [(flat[1600:2200].view(10, 60), (x, w)), (wide[:, 60:], (wide[:, :60], x)), (wide[:, :60], (wide[:, 60:],)),
            (wide[3:, 40:60], (wide[:, :40], wide[:, 60:])), (wide[10:], (wide[:10],)), (flat[:0].view(0, 5), (x,)), (x, (flat[:0],)),
            (x.view(torch.bfloat16)[:, 60:], (x.view(torch.bfloat16)[:, :60],)), (wide[::2, :60], (wide[:, 60:],)),
            (wide[::2], (wide[1::2],)), (wide[::3, 70:], (wide[::2, :70],))]
    for out, inputs in fine:
        _apart("out", out, *inputs)
