"""The top-k router and its gradient against their definitions in 64 bits.

Weights: exp of an argument rounded once (relative error |l| * 2^-24) and good to 2 ulp, a
sum of at most 1024 such terms over 32 lanes (at most 37 additions in a row) and a few
roundings: relative error at most (range + 64) * 2^-23, range the span of the logits."""
import numpy as np
import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu
FMAX = float(np.finfo(np.float32).max)
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SOFT, SIGM = moe.MOE_SCORE_SOFTMAX, moe.MOE_SCORE_SIGMOID


def scores(l, scoring):
    if scoring == SIGM:
        return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    top = l.max(1, keepdims=True)
    e = np.where(l > -np.inf, np.exp(l - np.where(np.isfinite(top), top, 0)), 0.0)
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def reference(logits, topk, scoring, renorm, scale, bias=None):
    l = logits.double().cpu().numpy()
    l = np.minimum(np.where(np.isnan(l), -np.inf, l), FMAX)
    s = scores(l, scoring)
    key = l if bias is None else np.where(l > -np.inf, s + bias.double().cpu().numpy(), -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :topk]
    live = np.take_along_axis(key, ids, 1) > -np.inf
    w = np.where(live, np.take_along_axis(s, ids, 1), 0.0)
    if renorm:
        lc = np.where(live, np.take_along_axis(l, ids, 1), -np.inf)
        # the ratio of the scores, whatever their size: a softmax over the logs of the scores
        log_s = lc if scoring == SOFT else np.where(live, np.minimum(lc, 0) - np.log1p(np.exp(-np.abs(lc))), -np.inf)
        w = scores(log_s, SOFT) * live
    return w * scale, np.where(live, ids, -1), key


def check_forward(logits, topk, scoring, renorm, scale, bias=None, ids_dtype=torch.int32):
    ids = torch.empty(logits.shape[0], topk, dtype=ids_dtype, device="cuda")
    w, ids = moe.moe_router_topk(logits, topk, scoring, renorm, scale, bias, topk_ids=ids)
    rw, rid, key = reference(logits, topk, scoring, renorm, scale, bias)
    keep = np.ones(len(rid), bool)
    if bias is not None:  # biased scores that fp32 cannot tell apart may come in either order
        top = -np.sort(-key, axis=1)[:, :topk + 1]
        with np.errstate(invalid="ignore"):
            gap = -np.diff(top, axis=1)
        keep = np.nan_to_num(gap, nan=1.0).min(1, initial=1.0) > 1e-6
        assert keep.mean() > 0.9
    assert np.array_equal(ids.cpu().numpy()[keep], rid[keep])
    got = w.double().cpu().numpy()
    fin = logits.float()[torch.isfinite(logits.float()) & (logits.float().abs() < 1e30)]
    span = float(fin.max() - fin.min()) if fin.numel() else 0.0
    tol = (span + 64) * 2.0 ** -23 * np.abs(rw) + 1e-37
    assert np.isfinite(got).all()
    assert (np.abs(got - rw) <= tol)[keep].all(), np.abs(got - rw)[keep].max()


@pytest.mark.parametrize("M,E,topk", [(1, 1, 1), (1, 128, 8), (7, 5, 5), (33, 32, 1), (64, 60, 4), (100, 128, 8),
                                      (5, 1024, 32), (9, 1000, 17), (40, 257, 8), (1000, 64, 6), (13, 512, 32), (3, 33, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scoring,renorm", [(SOFT, True), (SOFT, False), (SIGM, True), (SIGM, False)])
def test_choice_and_weights(M, E, topk, dtype, scoring, renorm):
    g = torch.Generator(device="cuda").manual_seed(M * E + topk)
    logits = (3 * torch.randn(M, E, device="cuda", generator=g)).to(dtype)
    check_forward(logits, topk, scoring, renorm, 1.75)


@pytest.mark.parametrize("scoring,renorm", [(SOFT, True), (SOFT, False), (SIGM, True), (SIGM, False)])
def test_masks_ties_and_extremes(scoring, renorm):
    inf, nan = float("inf"), float("nan")
    low = -FMAX
    rows = [[0.0] * 8, [-0.0, 0.0] * 4, [1, 2, 2, 1, 2, 0, 0, 2], [-inf] * 8, [nan] * 8, [nan, 1, -inf, 2, nan, -inf, -inf, -inf],
            [low] * 8, [low, 1, low, low, 2, low, low, low], [inf, 0, 1, 2, 3, 4, 5, 6], [inf, inf, 0, -inf, 0, 0, 0, 0],
            [-200, -300, -201, -202, -400, -200, -210, -1000], [90, 80, 70, 60, 50, 40, 30, 100], [-inf, -inf, 0, -inf, -inf, -inf, -inf, -inf]]
    check_forward(torch.tensor(rows, device="cuda"), 4, scoring, renorm, 2.0)
    check_forward(torch.tensor(rows, device="cuda"), 8, scoring, renorm, 1.0, ids_dtype=torch.int64)


@pytest.mark.parametrize("E,topk", [(128, 8), (120, 5), (8, 8), (64, 1), (136, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scoring,renorm", [(SOFT, True), (SOFT, False), (SIGM, True), (SIGM, False)])
def test_large_batches(E, topk, dtype, scoring, renorm):
    """Many tokens, with ties (few distinct values), signed zeros, masks and NaN among them."""
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(20011, E, device="cuda", generator=g)
    logits[:5000] = (logits[:5000] * 2).round() / 2
    logits[1000:2000] *= torch.where(torch.rand(1000, E, device="cuda", generator=g) < 0.5, 0.0, 1.0)
    logits[3000:7000].masked_fill_(torch.rand(4000, E, device="cuda", generator=g) < 0.4, -float("inf"))
    logits[6000:8000].masked_fill_(torch.rand(2000, E, device="cuda", generator=g) < 0.1, float("nan"))
    logits[8000:8010] = -float("inf")
    check_forward(logits.to(dtype), topk, scoring, renorm, 1.0)
    check_forward(logits.to(dtype), topk, scoring, renorm, 0.5, ids_dtype=torch.int64)


@pytest.mark.parametrize("scoring,renorm", [(SOFT, True), (SOFT, False), (SIGM, True), (SIGM, False)])
@pytest.mark.parametrize("E", [16, 100, 256])
def test_bias_moves_the_choice_only(scoring, renorm, E):
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(200, E, device="cuda", generator=g)
    bias = 0.3 * torch.randn(E, device="cuda", generator=g)
    bias[1], bias[3] = -float("inf"), float("nan")
    logits[0, 2:9] = -float("inf")
    safe = bias.clone()
    safe[3] = -float("inf")                         # what a NaN counts as
    w, ids = moe.moe_router_topk(logits, 6, scoring, renorm, 1.0, bias)
    assert not ((ids == 1) | (ids == 3)).any()
    w2, ids2 = moe.moe_router_topk(logits, 6, scoring, renorm, 1.0, safe)
    assert torch.equal(w, w2) and torch.equal(ids, ids2)
    check_forward(logits, 6, scoring, renorm, 1.0, safe)


def grad_reference(l, ids, g, scoring, renorm, scale):
    """d logits by the formulas, in 64 bits (numpy)."""
    s = scores(l, scoring)
    live = ids >= 0
    i = np.where(live, ids, 0)
    q = np.where(live, np.take_along_axis(s, i, 1), 0.0)
    g = np.where(live, g, 0.0) * scale
    d = np.zeros_like(l)
    rows = np.arange(len(l))[:, None].repeat(ids.shape[1], 1)
    if renorm:
        S = np.maximum(q.sum(1, keepdims=True), 1e-300)
        g = (g - (g * q).sum(1, keepdims=True) / S) / S
    if scoring == SOFT:
        np.add.at(d, (rows[live], ids[live]), (q * g)[live])
        return d - s * (q * g).sum(1, keepdims=True)
    np.add.at(d, (rows[live], ids[live]), (g * q * (1 - q))[live])
    return d


@pytest.mark.parametrize("M,E,topk", [(1, 1, 1), (1, 128, 8), (7, 5, 5), (64, 60, 4), (33, 128, 8), (9, 1000, 17),
                                      (5, 1024, 32), (40, 257, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scoring,renorm", [(SOFT, True), (SOFT, False), (SIGM, True), (SIGM, False)])
def test_gradient(M, E, topk, dtype, scoring, renorm):
    rng = torch.Generator(device="cuda").manual_seed(M + E)
    logits = (2 * torch.randn(M, E, device="cuda", generator=rng)).to(dtype)
    if E > 8:
        logits[0, :3] = -float("inf")
    _, ids = moe.moe_router_topk(logits, topk, scoring, renorm, 1.5)
    if topk > 2:
        ids[-1, 1] = -1                              # an empty slot
    g = torch.randn(M, topk, device="cuda", generator=rng)
    d = moe.moe_router_topk_backward(logits, ids, g, scoring, renorm, 1.5)
    d64 = moe.moe_router_topk_backward(logits, ids.long(), g, scoring, renorm, 1.5)
    assert torch.equal(d, d64)
    ref = grad_reference(logits.double().cpu().numpy(), ids.cpu().numpy(), g.double().cpu().numpy(), scoring, renorm, 1.5)
    # the difference g - sum q g of terms up to 1.5 max|g|, each good to (range + 64) * 2^-23
    big = 1.5 * g.abs().max().item() * topk ** 0.5
    tol = U[dtype] * np.abs(ref) + (20 + 64) * 2.0 ** -22 * big + (2.0 ** -25 if dtype == torch.float16 else 0)
    assert (np.abs(d.double().cpu().numpy() - ref) <= tol).all()
    inplace = logits.clone()
    moe.moe_router_topk_backward(inplace, ids, g, scoring, renorm, 1.5, d_logits=inplace)
    assert torch.equal(inplace, d)


@pytest.mark.parametrize("scoring,renorm", [(SOFT, True), (SOFT, False), (SIGM, True), (SIGM, False)])
def test_gradient_against_differences(scoring, renorm):
    rng = np.random.default_rng(4)
    l = rng.standard_normal((6, 40)).astype(np.float32)
    logits = torch.from_numpy(l).cuda()
    _, ids = moe.moe_router_topk(logits, 5, scoring, renorm, 1.25)
    g = torch.randn(6, 5, device="cuda")
    d = moe.moe_router_topk_backward(logits, ids, g, scoring, renorm, 1.25).double().cpu().numpy()
    i, gn = ids.cpu().numpy(), g.double().cpu().numpy()

    def loss(l):  # the choice is fixed
        w = np.take_along_axis(scores(l, scoring), i, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return 1.25 * (w * gn).sum()
    u, h = rng.standard_normal(l.shape), 1e-5
    num = (loss(l + h * u) - loss(l - h * u)) / (2 * h)
    # differences: h^2 * third derivatives (below 1e-8 here) and the loss's rounding / h
    assert abs(num - (d * u).sum()) <= 1e-5 * np.abs(d * u).sum() + 1e-8


def test_fully_masked_rows_have_no_gradient():
    logits = torch.full((3, 64), -float("inf"), device="cuda")
    w, ids = moe.moe_router_topk(logits, 4)
    assert (ids == -1).all() and not w.any()
    for renorm in (False, True):
        assert not moe.moe_router_topk_backward(logits, ids, torch.ones(3, 4, device="cuda"), renormalize=renorm).any()


def test_unaligned_logits():
    base = torch.randn(128 * 50 + 1, device="cuda")
    logits = base[1:].view(50, 128)
    check_forward(logits, 8, SOFT, True, 1.0)
    h = base.bfloat16()[1:].view(50, 128)
    check_forward(h, 8, SIGM, False, 1.0)
