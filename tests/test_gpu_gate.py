"""moe_gate and moe_gate_backward against the definition in 64 bits.

Tolerances.  A score is a few fp32 roundings from its value: exp within 1 ulp of a
result that is then added to 1 or summed, a reciprocal and a product, together under
4 * 2^-23 of the score; a renormalised weight divides two such numbers, under 2^-20.  A
choice value adds a bias of at most 1: under 5e-7 absolute.  Two choices may therefore
swap where the definition has them within 1e-6, and nowhere else."""
import math

import pytest

import _definitions as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

W_TOL = 2.0 ** -20
C_TOL = 1e-6
INF = math.inf


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_35_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


def rows_of(z, pad, offset=0, fill=math.nan):
    """z on the GPU as the leading columns of a wider buffer that starts `offset` elements late."""
    T, E = z.shape
    flat = torch.full((offset + T * (E + pad),), fill, dtype=z.dtype, device="cuda")
    view = flat[offset:].view(T, E + pad)[:, :E]
    view.copy_(z)
    return view


def call(moe, z, bias, G, M, K, score="sigmoid", group="top2", renorm=True, scale=1.0, scores=False, stream=None):
    T, E = z.shape
    rule = moe.make_gate_rule(T, E, K, score=score, n_groups=G, topk_groups=M, group_score=group, renormalize=renorm,
                              routed_scale=scale, logits="fp32" if z.dtype == torch.float32 else "bf16")
    idx = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), -7.0, device="cuda")
    s = torch.full((T, E), -7.0, device="cuda") if scores else None
    moe.moe_gate(rule, z, z.stride(0) if T > 1 else max(E, z.stride(0)), bias, s, idx, w, stream)
    return rule, idx, w, s


def check_choice(idx, w, z, bias, G, M, K, score, group, renorm, scale):
    """The GPU's choice and weights against the definition on the same logits (float64, CPU)."""
    T, E = z.shape
    ridx, rw, c, best = ref.gate(z, bias, G, M, K, score == "softmax", group == "max", renorm, scale)
    idx, w = idx.long().cpu(), w.double().cpu()
    assert ((idx >= 0) & (idx < E)).all()
    assert (idx.sort(1).values.diff(dim=1) > 0).all(), "a token's experts are distinct"
    same = (idx == ridx).all(1)
    if not same.all():
        # where the choice differs, the slots' choice values agree to the tolerance, or two groups are a near tie
        for t in torch.nonzero(~same).flatten().tolist():
            g = best[t].sort(descending=True).values
            near = M < G and (g[M - 1] - g[M]).abs() <= 2 * C_TOL
            assert near or ((c[t, idx[t]] - c[t, ridx[t]]).abs() <= C_TOL).all(), (t, idx[t], ridx[t])
        assert same.double().mean() > 0.98 or T < 64
    torch.testing.assert_close(w[same], rw[same], rtol=W_TOL, atol=2.0 ** -126)


CASES = [
    # T, E, G, M, K, score, group, bias, renorm, scale, dtype, pad
    (1, 256, 8, 4, 8, "sigmoid", "top2", True, True, 1.0, "fp32", 0),
    (333, 256, 8, 4, 8, "sigmoid", "top2", True, True, 2.5, "fp32", 0),
    (333, 256, 8, 4, 8, "softmax", "max", False, False, 16.0, "bf16", 3),
    (97, 256, 64, 9, 32, "sigmoid", "top2", True, True, 1.0, "bf16", 8),
    (65, 64, 64, 33, 17, "softmax", "top2", True, True, 1.0, "fp32", 4),     # one expert a group
    (70, 1, 1, 1, 1, "softmax", "max", False, True, 1.0, "fp32", 0),
    (70, 2, 1, 1, 1, "sigmoid", "max", True, False, 1.0, "bf16", 1),
    (70, 33, 1, 1, 32, "softmax", "max", True, True, 1.0, "fp32", 0),
    (129, 60, 1, 1, 4, "softmax", "max", False, True, 1.0, "fp32", 0),
    (129, 60, 4, 2, 6, "softmax", "top2", True, False, 1.0, "bf16", 0),
    (50, 160, 8, 3, 6, "softmax", "max", False, False, 16.0, "fp32", 0),
    (50, 129, 3, 2, 5, "sigmoid", "top2", False, True, 1.0, "fp32", 7),
    (31, 511, 7, 3, 10, "softmax", "top2", True, True, 1.0, "fp32", 0),
    (31, 513, 1, 1, 8, "sigmoid", "max", True, True, 1.0, "bf16", 0),
    (19, 1024, 32, 5, 32, "sigmoid", "top2", True, True, 1.0, "fp32", 0),
    (5, 1021, 1, 1, 3, "softmax", "max", True, True, 1.0, "fp32", 0),
    (3, 24, 3, 1, 8, "sigmoid", "top2", True, True, 1.0, "fp32", 0),         # K fills the kept group
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_gate_against_the_definition(moe, case):
    T, E, G, M, K, score, group, has_bias, renorm, scale, dtype, pad = case
    torch.manual_seed(E * 7 + T)
    z = torch.randn(T, E) * 2
    z = z.to(torch.bfloat16) if dtype == "bf16" else z
    bias = torch.rand(E) * 0.2 - 0.1 if has_bias else None
    dz = rows_of(z, pad)
    rule, idx, w, s = call(moe, dz, bias.cuda() if has_bias else None, G, M, K, score, group, renorm, scale, True)
    torch.cuda.synchronize()
    check_choice(idx, w, z.double(), bias.double() if has_bias else None, G, M, K, score, group, renorm, scale)
    want, _ = ref.scores(z.double(), score == "softmax")
    torch.testing.assert_close(s.double().cpu(), want, rtol=W_TOL, atol=2.0 ** -126)


@pytest.mark.parametrize("E,G,M,K", [(256, 8, 4, 8), (64, 1, 1, 6), (96, 12, 5, 7), (1024, 4, 2, 9)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_go_to_the_lower_index(moe, E, G, M, K, score):
    # logits on a coarse grid: equal ones score equal bits, different ones differ by far more than a rounding
    torch.manual_seed(E + K)
    z = torch.randint(-2, 3, (200, E)).float() * 0.5
    _, idx, w, _ = call(moe, z.cuda(), None, G, M, K, score, "max")
    ridx, rw, _, _ = ref.gate(z.double(), None, G, M, K, score == "softmax", True, True, 1.0)
    assert (idx.cpu().long() == ridx).all()
    torch.testing.assert_close(w.double().cpu(), rw, rtol=W_TOL, atol=0.0)


@pytest.mark.parametrize("offset,pad,dtype", [(0, 1, "fp32"), (1, 0, "fp32"), (3, 5, "bf16"), (4, 4, "bf16"), (2, 2, "fp32")])
def test_unaligned_rows_give_the_same_bits(moe, offset, pad, dtype):
    torch.manual_seed(offset + 10 * pad)
    z = torch.randn(77, 136).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    _, i0, w0, s0 = call(moe, z.cuda(), None, 4, 2, 5, "softmax", scores=True)
    _, i1, w1, s1 = call(moe, rows_of(z, pad, offset), None, 4, 2, 5, "softmax", scores=True)
    assert (i0 == i1).all() and (w0 == w1).all() and (s0 == s1).all()


def masked_rows(E, K):
    torch.manual_seed(E)
    z = torch.randn(12, E)
    z[0] = -INF                                   # nothing in use
    z[1] = math.nan
    z[2, : E - 2] = -INF                          # two experts in use, fewer than K
    z[3, 1:] = -INF                               # one
    z[4, ::2] = math.nan
    z[5] = torch.finfo(torch.float32).min         # the lowest finite value everywhere
    z[6, : E // 2] = torch.finfo(torch.float32).min
    z[7, E // 3] = INF                            # a single +infinity
    z[8, ::3] = INF                               # several
    z[9] = 1e30
    z[10] = -1e30
    z[11, : E // 2] = -INF                        # the first groups out of use
    return z


@pytest.mark.parametrize("E,G,M,K", [(64, 1, 1, 6), (64, 8, 4, 6), (256, 8, 4, 8), (40, 4, 2, 5)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_masks_infinities_and_nan(moe, E, G, M, K, score, renorm, dtype):
    z = masked_rows(E, K).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    _, idx, w, s = call(moe, z.cuda(), None, G, M, K, score, "top2", renorm, 1.5, True)
    idx, w, s = idx.cpu(), w.cpu(), s.cpu()
    assert torch.isfinite(w).all() and torch.isfinite(s).all()
    check_choice(idx, w, z.double(), None, G, M, K, score, "top2", renorm, 1.5)
    for t in (0, 1):                              # a row without experts still names distinct ones, at weight 0
        assert (w[t] == 0).all() and idx[t].tolist() == list(range(K))
    assert (s[~(z.float() > -INF)] == 0).all()
    # the gradient of such rows is finite, and 0 where the expert is out of use
    rule = moe.make_gate_rule(12, E, K, score=score, n_groups=G, topk_groups=M, renormalize=renorm, routed_scale=1.5,
                              logits=dtype)
    dz = torch.full((12, E), 7.0, dtype=z.dtype, device="cuda")
    ds = torch.randn(12, E, device="cuda")
    ds[~(z.cuda().float() > -INF)] = math.nan     # what the caller holds at a masked place does not count
    moe.moe_gate_backward(rule, z.cuda(), E, idx.cuda(), w.cuda(), torch.randn(12, K, device="cuda"), ds, dz, E)
    got = dz.float().cpu()
    assert torch.isfinite(got).all()
    assert (got[~(z.float() > -INF)] == 0).all()


def test_bias_of_minus_infinity_and_nan_takes_an_expert_out(moe):
    torch.manual_seed(3)
    z = torch.randn(50, 48)
    bias = torch.zeros(48)
    bias[5], bias[7] = -INF, math.nan
    _, idx, w, _ = call(moe, z.cuda(), bias.cuda(), 1, 1, 8)
    check_choice(idx, w, z.double(), bias.double(), 1, 1, 8, "sigmoid", "top2", True, 1.0)
    assert not ((idx == 5) | (idx == 7)).any()


def reference_gradient(z, idx, w, dw, ds, softmax, renorm, scale):
    """autograd in 64 bits through the scores of the chosen experts (the weights' zeros stay out)."""
    z = z.clone().requires_grad_(True)
    dead = ~(z.detach() > -INF)
    safe = torch.where(dead, torch.zeros_like(z), z)
    if softmax:
        s = torch.softmax(torch.where(dead, torch.full_like(z, -1e300), safe), 1)
    else:
        s = torch.sigmoid(safe)
    s = torch.where(dead, torch.zeros_like(s), s)
    sel = torch.where(w != 0, s.gather(1, idx), torch.zeros(()).double())
    out = sel / sel.sum(1, keepdim=True).clamp(min=1e-300) if renorm else sel
    loss = (out * scale * dw).sum() + ((s * ds).sum() if ds is not None else 0.0)
    loss.backward()
    return z.grad


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("aux", [False, True])
def test_gradient_against_the_formula(moe, case, aux):
    T, E, G, M, K, score, group, has_bias, renorm, scale, dtype, pad = case
    torch.manual_seed(E * 3 + T)
    z = torch.randn(T, E)
    if E > K + 1:
        z[:, E - 1] = -INF
    z = z.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    bias = (torch.rand(E) * 0.2 - 0.1).cuda() if has_bias else None
    dz = rows_of(z, pad)
    rule, idx, w, _ = call(moe, dz, bias, G, M, K, score, group, renorm, scale)
    dw = torch.randn(T, K, device="cuda")
    ds = torch.randn(T, E, device="cuda") if aux else None
    got = rows_of(torch.zeros(T, E, dtype=z.dtype), pad, fill=3.0)
    moe.moe_gate_backward(rule, dz, E + pad, idx, w, dw, ds, got, E + pad)
    want = reference_gradient(z.double(), idx.long().cpu(), w.double().cpu(), dw.double().cpu(),
                              ds.double().cpu() if aux else None, score == "softmax", renorm, scale)
    # terms of a row: at most scale * max|g| / D in ds_j (D >= the largest chosen s) or dscores; fp32 over sums of
    # E terms: 2^-20 of the row's largest term; a bf16 result rounds by 2^-9 of itself
    s, _ = ref.scores(z.double(), score == "softmax")
    top = s.gather(1, idx.long().cpu()).amax(1, keepdim=True)
    # each ds_j multiplies an s_j <= top, and D >= top
    term = scale * dw.double().abs().amax(1, keepdim=True).cpu() * (torch.ones_like(top) if renorm else top)
    if aux:
        term = term + (s * ds.double().abs().cpu()).amax(1, keepdim=True)
    tol = 8 * 2.0 ** -20 * term + (2.0 ** -8 * want.abs() if dtype == "bf16" else 0.0)
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    if pad and T > 1:                              # the padding of dlogits is untouched
        assert (got.as_strided((T - 1, pad), (E + pad, 1), got.storage_offset() + E) == 3.0).all()


@pytest.mark.parametrize("score,renorm,G,M", [("sigmoid", True, 4, 2), ("sigmoid", False, 1, 1), ("softmax", True, 4, 2),
                                              ("softmax", False, 1, 1)])
def test_gradient_against_differences(moe, score, renorm, G, M):
    # token t of the batch moves logit t alone: two forward calls give every central difference of one row
    E, K, h = 48, 5, 2.0 ** -7
    torch.manual_seed(11)
    z = torch.randperm(E).float() * 0.125 - 3.0    # 1/8 apart, so that a step of 1/128 moves no choice
    base = z.repeat(E, 1).cuda()
    step = torch.eye(E, device="cuda") * h
    dw, ds = torch.randn(K, device="cuda").double(), torch.randn(E, device="cuda").double()
    losses, idxs = [], []
    for sign in (1, -1):
        _, idx, w, s = call(moe, base + sign * step, None, G, M, K, score, "max", renorm, 2.0, True)
        losses.append((w.double() * dw).sum(1) + (s.double() * ds).sum(1))
        idxs.append(idx)
    assert (idxs[0] == idxs[1]).all()
    numeric = ((losses[0] - losses[1]) / (2 * h)).cpu()
    rule, idx, w, _ = call(moe, base[:1].contiguous(), None, G, M, K, score, "max", renorm, 2.0)
    got = torch.empty((1, E), device="cuda")
    moe.moe_gate_backward(rule, base[:1].contiguous(), E, idx, w, dw.float()[None].contiguous(),
                          ds.float()[None].contiguous(), got, E)
    # third derivatives of both scores are below 1/2 here times weights of order 10: h^2/6 * 10 = 1e-4; fp32 losses of
    # order 10 over 2h: 64 * 10 * 2^-24 = 4e-5
    assert (got[0].double().cpu() - numeric).abs().max() < 3e-4


def test_no_tokens(moe):
    z = torch.empty((0, 32), device="cuda")
    rule = moe.make_gate_rule(0, 32, 4)
    e = torch.empty(0, device="cuda")
    assert moe.moe_gate(rule, z, 32, None, None, e, e) == 0
    assert moe.moe_gate_backward(rule, z, 32, e, e, e, None, e, 32) == 0


def test_more_than_2_to_31_logits(moe):
    T, E, K = (1 << 21) + 5, 1024, 2
    z = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    z[T - 1, 1000], z[T - 1, 30], z[1, 7] = 3.0, 2.0, 1.0
    _, idx, w, _ = call(moe, z, None, 1, 1, K, "sigmoid")
    assert idx[T - 1].tolist() == [1000, 30] and idx[1].tolist() == [7, 0] and idx[T - 2].tolist() == [0, 1]
    rule = moe.make_gate_rule(T, E, K, logits="bf16")
    dw = torch.ones((T, K), device="cuda")
    dw[:, 0] = 2.0
    dz = torch.full_like(z, 9.0)
    moe.moe_gate_backward(rule, z, E, idx, w, dw, None, dz, E)
    last = dz[T - 1].float()
    assert last[1000] > 0 and last[30] < 0 and torch.count_nonzero(last) == 2
    assert torch.count_nonzero(dz[T - 2].float()) == 2


def test_streams_and_graph_replays(moe):
    torch.manual_seed(5)
    T, E, K = 300, 96, 6
    z = torch.randn(T, E, device="cuda")
    bias = torch.rand(E, device="cuda") * 0.1
    rule = moe.make_gate_rule(T, E, K, n_groups=8, topk_groups=4)
    idx, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    dw, dz = torch.randn(T, K, device="cuda"), torch.empty((T, E), device="cuda")

    def both(stream):
        moe.moe_gate(rule, z, E, bias, None, idx, w, stream)
        moe.moe_gate_backward(rule, z, E, idx, w, dw, None, dz, E, stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both(side)
    for k in range(4):
        z.copy_(torch.randn(T, E, device="cuda") + k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (idx, w, dz)]
        for t in (idx, w, dz):
            t.zero_()
        both(None)
        torch.cuda.synchronize()
        assert all((a == b).all() for a, b in zip(got, (idx, w, dz)))
