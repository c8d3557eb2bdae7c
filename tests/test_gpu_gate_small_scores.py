"""moe_gate_backward where the chosen scores lie near the smallest floats: the weights are shares of their sum, and so
is the gradient, whatever the sum's size."""
import math

import pytest

import _definitions as ref
from test_gpu_gate import reference_gradient

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
TINY = 2.0 ** -149


def both(z, bias, K, score, scale, dw, ds, dtype="fp32"):
    import mixture_experts_layer_35_amd as moe
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    T, E = z.shape
    rule = moe.make_gate_rule(T, E, K, score=score, routed_scale=scale, logits=dtype)
    z = z.cuda()
    idx, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    moe.moe_gate(rule, z, E, None if bias is None else bias.cuda(), None, idx, w)
    dz = torch.empty((T, E), device="cuda", dtype=z.dtype)
    moe.moe_gate_backward(rule, z, E, idx, w, dw.cuda(), None if ds is None else ds.cuda(), dz, E)
    return idx.long().cpu(), w.double().cpu(), dz.double().cpu()


def check(z, idx, w, dz, dw, ds, softmax, scale):
    """Shares are quotients of scores that are held to 2^-23 of themselves or half of the smallest float: their
    relative error, and that of the mean they weigh, is below 8 times the two together; terms of a row are scale * |g|
    and s * |dscores|, 2^-20 of the largest as elsewhere."""
    z, dw = z.double(), dw.double()
    ds = None if ds is None else ds.double()
    s, _ = ref.scores(z, softmax)
    chosen = s.gather(1, idx)
    want = ref.weigh(chosen, True, scale)
    rel = 8 * (2.0 ** -23 + TINY / chosen.amin(1, keepdim=True))
    assert ((w - want).abs() <= rel * want).all()
    grad = reference_gradient(z, idx, w, dw, ds, softmax, True, scale)
    term = scale * dw.abs().amax(1, keepdim=True)
    tol = (8 * 2.0 ** -20 + rel) * term
    if ds is not None:
        tol = tol + 8 * 2.0 ** -20 * (s * ds.abs()).amax(1, keepdim=True)
    err = (dz - grad).abs()
    assert torch.isfinite(dz).all() and (err <= tol).all(), float((err / tol).max())
    assert w.shape[1] == 1 or float(grad.abs().max()) > 0.01          # the gradient is nothing like as small as the scores


@pytest.mark.parametrize("E", [16, 64, 200])
@pytest.mark.parametrize("K", [1, 4])
@pytest.mark.parametrize("aux", [False, True])
@pytest.mark.parametrize("T", [5, 5000])
def test_softmax_far_below_the_largest_logit(E, K, aux, T):
    # the bias takes the expert with the largest logit out of the choice; what is chosen lies 88 to 93 below it
    torch.manual_seed(E + K)
    z = torch.rand(T, E) * 5 - 93
    z[:, 3] = 0.0
    bias = torch.zeros(E)
    bias[3] = -math.inf
    dw, ds = torch.randn(T, K), torch.randn(T, E) if aux else None
    idx, w, dz = both(z, bias, K, "softmax", 2.5, dw, ds)
    check(z, idx, w, dz, dw, ds, True, 2.5)
    if K == 1:
        assert (w == 2.5).all()                                # a share of one, and no gradient of its own
        assert aux or (dz == 0).all()


@pytest.mark.parametrize("K", [1, 2, 8])
@pytest.mark.parametrize("aux", [False, True])
def test_sigmoid_of_logits_near_minus_88(K, aux):
    torch.manual_seed(K)
    T, E = 70, 48
    z = -torch.rand(T, E) * 1.5 - 87
    dw, ds = torch.randn(T, K) * 4, torch.randn(T, E) if aux else None
    idx, w, dz = both(z, None, K, "sigmoid", 2.5, dw, ds)
    check(z, idx, w, dz, dw, ds, False, 2.5)
