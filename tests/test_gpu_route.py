"""The router and its backward on the GPU against the definitions in 64 bits.

Tolerances.  A weight is a quotient of exponentials and sums in fp32: the
argument z - max is off by 2^-24 of its size (|z| <= 40 here: 2.4e-6 of the
exponential), expf by 2 ulp, a sum of at most 2048 terms (64 in sequence, then
a tree of 5) by 70 * 2^-24 = 4.2e-6, the divisions by an ulp each.  Twice that
sum is below 2e-5.  A gradient is a difference of such terms, so the same
bound holds against the size of its terms, not of their difference.
"""
import numpy as np
import pytest
import torch

import combine_ep_plan_gb300 as ep

pytestmark = pytest.mark.gpu

RTOL = 2e-5
NEAR = 1e-5  # 64-bit scores closer than this (and not equal) may come in either order


def scores64(z, score):
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-z))
    else:
        m = z.max(1, keepdim=True).values
        e = torch.exp(z - torch.where(torch.isinf(m), 0.0, m))
        e = torch.where(torch.isneginf(z) | torch.isnan(z), 0.0, e)
        t = e.sum(1, keepdim=True)
        s = torch.where(t > 0, e / t, 0.0)
    return torch.where(torch.isneginf(z) | torch.isnan(z), 0.0, s)


def select64(z, score, k, bias, G, TG):
    """-> (idx [T,k] with -1, rows whose order is certain)."""
    T, E = z.shape
    off = torch.isneginf(z) | torch.isnan(z)
    exact = bias is None and G == TG  # by the logits themselves: no rounding
    by = z if exact else scores64(z, score) + (0.0 if bias is None else bias.double())
    by = torch.where(off, -torch.inf, by)
    sure = torch.ones(T, dtype=torch.bool)
    idx = torch.full((T, k), -1)
    for t in range(T):
        row = by[t].tolist()
        allowed = list(range(E))
        if G != TG:
            per = E // G
            group = []
            for g in range(G):
                top = sorted((v for v in row[g * per:(g + 1) * per] if v > -np.inf), reverse=True)[:2]
                group.append(sum(top) if top else -np.inf)
            order = sorted(range(G), key=lambda g: (-group[g], g))
            a, b = group[order[TG - 1]], group[order[TG]]
            if a != b and a - b < NEAR:
                sure[t] = False
            allowed = [e for g in order[:TG] for e in range(g * per, (g + 1) * per)]
        live = sorted((e for e in allowed if row[e] > -np.inf), key=lambda e: (-row[e], e))
        for i in range(min(k, len(live))):
            idx[t, i] = live[i]
            if i + 1 < len(live) and row[live[i]] != row[live[i + 1]] and row[live[i]] - row[live[i + 1]] < NEAR:
                sure[t] = sure[t] and exact
    return idx, sure


def weights64(z, idx, score, renorm, scale):
    s = scores64(z, score)
    w = torch.where(idx < 0, 0.0, s.gather(1, idx.clamp(min=0)))
    if renorm:
        if score == "softmax":  # over the chosen logits: no underflow
            zk = torch.where(idx < 0, -torch.inf, z.gather(1, idx.clamp(min=0)))
            m = zk.max(1, keepdim=True).values
            w = torch.exp(zk - torch.where(torch.isinf(m), 0.0, m))
        t = w.sum(1, keepdim=True)
        w = torch.where(t > 0, w / t, 0.0)
    return w * scale


def draw_logits(T, E, dtype, seed, masked=0.0, grid=None):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * 2
    if grid:
        z = torch.round(z * grid) / grid  # equal logits on purpose
    z = z.clamp(-20, 20)
    if masked:
        z[torch.rand(T, E, generator=g) < masked] = -torch.inf
    return z.to(dtype)


SHAPES = [(1, 1, 1), (1, 8, 8), (3, 7, 3), (33, 64, 6), (5, 100, 4), (17, 128, 8), (40, 129, 16), (70, 256, 6),
          (9, 257, 2), (11, 512, 8), (6, 513, 1), (4, 2048, 16), (1030, 24, 5), (4101, 60, 7), (4098, 128, 4), (4099, 250, 3),
          (4097, 300, 9)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route(T, E, k, dtype, score):
    for case, (biased, renorm, masked, grid) in enumerate([(False, True, 0.0, None), (False, False, 0.4, 4),
                                                           (True, True, 0.1, None), (True, False, 0.0, None)]):
        z = draw_logits(T, E, dtype, 100 * E + case, masked, grid)
        bias = torch.randn(E, generator=torch.Generator().manual_seed(case)) * 0.1 if biased else None
        idx, w = ep.route(z.cuda(), k, score, bias.cuda() if biased else None, renormalize=renorm, scale=2.5)
        assert idx.dtype == torch.int64 and w.dtype == torch.float32
        want, sure = select64(z.double(), score, k, bias, 1, 1)
        if not biased:
            assert sure.all()
        assert sure.float().mean() > 0.8 or T < 20
        assert torch.equal(idx.cpu()[sure], want[sure])
        w64 = weights64(z.double(), idx.cpu(), score, renorm, 2.5)
        assert torch.allclose(w.cpu().double(), w64, rtol=RTOL, atol=1e-30)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 6, 6), (67, 9, 8), (130, 64, 6), (33, 72, 8), (5000, 128, 8), (50, 250, 7),
                                   (21, 256, 1), (19, 260, 8), (4500, 512, 8), (9, 520, 4), (7, 2048, 8)])
def test_route_bf16_as_fp32(T, E, k, renorm, score):
    """bf16 logits give the choice of the same numbers in fp32: ties, masked
    rows, NaN, infinities, both zeros, rows that are not aligned."""
    lowest = torch.finfo(torch.bfloat16).min
    g = torch.Generator().manual_seed(T + E)
    wide = torch.round(torch.randn(T, E + 3, generator=g) * 4) / 2  # many ties, and zeros of both signs
    kind = torch.rand(T, E + 3, generator=g)
    for i, v in enumerate((-torch.inf, torch.nan, -torch.nan, lowest, -lowest)):
        wide[(kind > 0.05 * i) & (kind < 0.05 * (i + 1) - (0.045 if v == -lowest else 0.0))] = v
    wide[T // 2] = -torch.inf
    wide = wide.to(torch.bfloat16).cuda()
    for z in (wide[:, 1:1 + E], wide[:, :E].contiguous()):
        idx, w = ep.route(z, k, score, renormalize=renorm)
        want, weights = ep.route(z.float(), k, score, renormalize=renorm)
        assert torch.equal(idx, want)
        assert torch.allclose(w, weights, rtol=2 * RTOL, atol=1e-30)
        assert (idx[T // 2] == -1).all() and (w[T // 2] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,TG,k", [(256, 8, 4, 8), (64, 8, 1, 6), (160, 8, 3, 6), (96, 3, 2, 5), (32, 32, 5, 4),
                                      (2048, 32, 7, 16), (30, 15, 2, 4), (8, 2, 1, 8), (24, 24, 24, 3)])
def test_route_groups(E, G, TG, k, score):
    for masked, T in ((0.0, 150), (0.3, 150), (0.1, 4103)):
        z = draw_logits(T, E, torch.float32, E + G, masked)
        bias = torch.randn(E, generator=torch.Generator().manual_seed(G)) * 0.1
        for b in (None, bias):
            idx, w = ep.route(z.cuda(), k, score, None if b is None else b.cuda(), G, TG)
            want, sure = select64(z.double(), score, k, b, G, TG)
            assert sure.float().mean() > 0.5
            assert torch.equal(idx.cpu()[sure], want[sure])
            assert torch.allclose(w.cpu().double(), weights64(z.double(), idx.cpu(), score, True, 1.0), rtol=RTOL,
                                  atol=1e-30)


def test_route_ties_go_to_the_lowest_index():
    z = torch.zeros(5, 200)
    z[1, 150:] = 1.0
    z[2, ::2] = -0.0  # equal to +0
    z[3, 199] = 3.0
    z[3, 7] = 3.0
    idx, w = ep.route(z.cuda(), 4)
    assert idx.cpu().tolist() == [[0, 1, 2, 3], [150, 151, 152, 153], [0, 1, 2, 3], [7, 199, 0, 1], [0, 1, 2, 3]]
    assert torch.equal(w.cpu()[0], torch.full((4,), 0.25))
    idx, _ = ep.route(z.cuda()[:1], 3, num_groups=10, topk_groups=2)
    assert idx.cpu().tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masked_and_non_finite_rows(score, renorm):
    lowest = torch.finfo(torch.float32).min
    z = torch.full((7, 64), -torch.inf)
    z[1, 5] = 1.0                     # one expert
    z[2] = torch.nan                  # none
    z[3, :] = lowest                  # a mask by the type's lowest value: all equal, all available
    z[4] = lowest
    z[4, 60] = 2.0
    z[5, 3] = torch.nan
    z[5, 9] = -200.0                  # a sigmoid that underflows
    z[6, 2], z[6, 4] = torch.inf, 1.0
    idx, w = ep.route(z.cuda(), 3, score, renormalize=renorm)
    idx, w = idx.cpu(), w.cpu()
    assert idx[:6].tolist() == [[-1] * 3, [5, -1, -1], [-1] * 3, [0, 1, 2], [60, 0, 1], [9, -1, -1]]
    assert idx[6].tolist() == [2, 4, -1]
    assert w[0].tolist() == [0] * 3 and w[2].tolist() == [0] * 3
    if renorm:
        assert w[1].tolist() == [1, 0, 0]
        assert w[4].tolist() == [1, 0, 0]
        assert w[5].tolist() == ([1, 0, 0] if score == "softmax" else [0, 0, 0])
        if score == "softmax":
            assert torch.allclose(w[3], torch.full((3,), 1 / 3))
    if score == "softmax":
        assert torch.isnan(w[6, 0])
    elif not renorm:
        assert w[6].tolist()[0] == 1.0
    grad = ep.route_backward(z.cuda()[:6], idx.cuda()[:6], torch.ones(6, 3).cuda(), score, renormalize=renorm).cpu()
    assert torch.isfinite(grad).all()
    assert (grad[0] == 0).all() and (grad[2] == 0).all()
    assert (grad[torch.isinf(z[:6]) | torch.isnan(z[:6])] == 0).all()


def test_route_strided_rows_outputs_and_streams():
    wide = torch.randn(50, 300).cuda()
    z = wide[:, 17:17 + 130]
    idx = torch.empty(50, 4, dtype=torch.int64).cuda()
    w = torch.empty(50, 4).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = ep.route(z, 4, topk_idx=idx, topk_weights=w, stream=s)
    s.synchronize()
    assert a is idx and b is w
    want, weights = ep.route(z.contiguous(), 4)
    assert torch.equal(idx, want) and torch.equal(w, weights)
    g = torch.randn(50, 4).cuda()
    assert torch.equal(ep.route_backward(z, idx, g), ep.route_backward(z.contiguous(), idx, g))
    empty = ep.route(z[:0], 4)
    assert empty[0].shape == (0, 4) and ep.route_backward(z[:0], empty[0], empty[1]).shape == (0, 130)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route_backward(T, E, k, dtype, renorm, score):
    z = draw_logits(T, E, dtype, 7 * E + k, 0.2)
    idx, _ = ep.route(z.cuda(), k, score, renormalize=renorm)
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(E))
    got = ep.route_backward(z.cuda(), idx, g.cuda(), score, renorm, 2.5).cpu()
    assert got.dtype == dtype and got.shape == (T, E)
    i = idx.cpu()

    def loss(v):  # 64-bit forward for a fixed selection
        return (weights64(v, i, score, renorm, 2.5) * g.double()).sum(1)

    v = torch.where(torch.isneginf(z), -1e4, z.double()).requires_grad_(True)
    loss(v).sum().backward()
    want = torch.where(torch.isneginf(z), 0.0, v.grad)
    size = 2.5 * g.abs().double().sum(1, keepdim=True)  # bounds each term of the row's gradient
    eps = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert ((got.double() - want).abs() <= RTOL * size + eps * want.abs()).all()
    # differences: along a random direction; the truncation error is h^2/6 times a third derivative of order `size`
    d = torch.where(torch.isneginf(z), 0.0, torch.randn(T, E, generator=torch.Generator().manual_seed(k)).double())
    h, base = 1e-4, v.detach()
    slope = (loss(base + h * d) - loss(base - h * d)) / (2 * h)
    along = (got.double() * d).sum(1)
    room = (RTOL * size[:, 0] + 1e-6 * size[:, 0]) * d.abs().sum(1) + eps * (want * d).abs().sum(1)
    assert ((slope - along).abs() <= room).all()


def test_route_backward_ignores_entries_outside():
    z = torch.randn(2, 40).cuda()
    idx = torch.tensor([[3, -1, 40], [1 << 40, 5, -7]]).cuda()
    got = ep.route_backward(z, idx, torch.ones(2, 3).cuda(), "sigmoid", False).cpu()
    assert (got != 0).sum(1).tolist() == [1, 1] and got[0, 3] > 0 and got[1, 5] > 0


def test_route_feeds_plan_and_combine_feeds_backward():
    """Router, plan, dispatch, combine and both backwards: the gradient of the
    logits through the whole layer against 64 bits."""
    T, E, k, H = 96, 16, 3, 64
    z = draw_logits(T, E, torch.float32, 5).cuda()
    z[7] = -torch.inf  # a token without experts
    idx, w = ep.route(z, k, "sigmoid", scale=1.5)
    h = ep.plan(idx, 4, E)
    x = torch.randn(T, H).to(torch.bfloat16).cuda()
    y, _ = ep.dispatch(h, x)
    out = ep.combine(h, y, w)
    grad_out = torch.randn(T, H).to(torch.bfloat16).cuda()
    _, grad_w = ep.combine_backward(h, grad_out, y, w)
    h.check()
    grad = ep.route_backward(z, idx, grad_w, "sigmoid", True, 1.5)
    assert (out[7] == 0).all() and (grad[7] == 0).all()
    gw = (grad_out.double() * x.double()).sum(1, keepdim=True).expand(-1, k).cpu()
    v = torch.where(torch.isneginf(z), -1e4, z.double()).cpu().requires_grad_(True)
    (weights64(v, idx.cpu(), "sigmoid", True, 1.5) * gw).sum().backward()
    size = 1.5 * gw.abs().sum(1, keepdim=True)
    live = torch.arange(T) != 7  # the reference's own gradient is 0/0 there
    assert ((grad.cpu().double() - v.grad).abs() <= 2 * RTOL * size + 1e-6)[live].all()
    # experts that differ, so that the slots' gradients do too
    y = (y.float() * torch.randn(len(y), 1, device="cuda")).to(torch.bfloat16)
    _, grad_w = ep.combine_backward(h, grad_out, y, w)
    grad = ep.route_backward(z, idx, grad_w, "sigmoid", True, 1.5)
    gw = (grad_out.double()[:, None] * y.double()[h.field("slot").long().clamp(min=0)]).sum(2).cpu()
    v.grad = None
    (weights64(v, idx.cpu(), "sigmoid", True, 1.5) * gw).sum().backward()
    size = 1.5 * gw.abs().sum(1, keepdim=True)
    assert ((grad.cpu().double() - v.grad).abs() <= 2 * RTOL * size + 1e-6)[live].all()
    assert grad[live.cuda()].abs().max() > 0.1
    h.destroy()


def test_route_refusals():
    z = torch.randn(4, 16).cuda()
    with pytest.raises(ep.EPError):
        ep.route(z, 17)
    with pytest.raises(ep.EPError):
        ep.route(z, 0)
    with pytest.raises(ep.EPError):
        ep.route(z, 2, num_groups=3)
    with pytest.raises(ep.EPError):
        ep.route(z, 2, num_groups=4, topk_groups=5)
    with pytest.raises(ValueError):
        ep.route(z, 2, "relu")
    with pytest.raises(ValueError):
        ep.route(z.t(), 2)
    with pytest.raises(ValueError):
        ep.route(z.cpu(), 2)
    with pytest.raises(TypeError):
        ep.route(z.half(), 2)
    with pytest.raises(ValueError):
        ep.route(z, 2, bias=torch.zeros(15).cuda())
    with pytest.raises(ValueError):
        ep.route(z, 2, topk_idx=torch.empty(4, 3, dtype=torch.int64).cuda())
    idx, w = ep.route(z, 2)
    with pytest.raises(ValueError):
        ep.route_backward(z, idx, w[:3].contiguous())
    with pytest.raises(TypeError):
        ep.route_backward(z, idx.int(), w)
    with pytest.raises(TypeError):
        ep.route_backward(z, idx, w, grad_logits=torch.empty(4, 16, dtype=torch.bfloat16).cuda())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G", [(64, 8), (30, 5), (256, 8), (520, 4)])
@pytest.mark.parametrize("T", [5, 4100])
def test_route_groups_without_bias_go_by_the_logits(T, E, G, dtype):
    """Inside the groups that compete, experts whose scores round to the same
    number (a softmax far below its maximum, a saturated sigmoid) still go by
    their logits, an expert masked by the type's lowest value last."""
    per, lowest = E // G, torch.finfo(dtype).min
    g = torch.Generator().manual_seed(E)
    order = torch.randperm(2 * per, generator=g)  # of the two groups that win
    for score, top, step in (("softmax", 0.0, -128.0), ("sigmoid", 40.0, 2.0)):
        z = torch.full((T, E), -200.0 if score == "softmax" else -30.0)
        place = torch.cat([torch.arange(per) + per * (G - 1), torch.arange(per) + per])
        if score == "softmax":  # one expert at the top of each group, the others' scores underflow
            z[:, place] = step - 0.5 * order.float()
            z[:, place[0]], z[:, place[per]] = top, -0.5
            z[:, place[1]] = lowest
        else:                   # all of them round to 1
            z[:, place] = top + step * order.float()
        z = z.to(dtype)
        k = min(6, 2 * per - 1)
        idx, w = ep.route(z.cuda(), k, score, num_groups=G, topk_groups=2)
        row = z[0].double()
        want = sorted(place.tolist(), key=lambda e: (-float(row[e]), e))[:k]
        assert (idx.cpu() == torch.tensor(want)).all(), score
        assert torch.allclose(w.cpu().double(), weights64(z.double(), idx.cpu(), score, True, 1.0), rtol=RTOL, atol=1e-30)
        # a softmax of +inf leaves nobody, as before
        z[0, 3] = torch.inf
        idx, _ = ep.route(z.cuda(), k, score, num_groups=G, topk_groups=2)
        assert score == "sigmoid" or (idx[0] == -1).all()
