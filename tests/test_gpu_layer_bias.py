"""fp4_route: a bias of -inf (or NaN) takes an expert out of the choice."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F = pytest.importorskip("bit_floating_point_amd")
DEV = "cuda"


def say(*a):
    print(*a, flush=True)


def reference(logits, k, score, bias, groups, top_groups, group_top):
    """In 64 bits; experts are usable where logit and key are finite or the key is +inf."""
    T, E = logits.shape
    l = logits.double()
    ok = torch.isfinite(l)
    p = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(torch.where(ok, l, -math.inf), 1)
    p = torch.where(ok, p, 0.0).nan_to_num(0.0)
    key = torch.where(ok, p + bias.double(), -math.inf)
    key = torch.where(key > -math.inf, key, -math.inf)  # NaN too
    if groups > 1:
        best = key.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :group_top]
        total = torch.where(best[:, :, 0] == -math.inf, -math.inf, torch.where(best == -math.inf, 0.0, best).sum(2))
        order = total.argsort(dim=1, descending=True, stable=True)[:, :top_groups]
        keep = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(keep.repeat_interleave(E // groups, 1), key, -math.inf)
    value, idx = key.sort(dim=1, descending=True, stable=True)
    value, idx = value[:, :k], idx[:, :k]
    none = value == -math.inf
    w = torch.where(none, 0.0, p.gather(1, idx))
    w = torch.where(w.sum(1, keepdim=True) > 0, w / w.sum(1, keepdim=True), 0.0)
    return torch.where(none, -1, idx).int(), w, torch.where(none, E, idx).view(-1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top", [(1, 8, 6, 1, 1, 1), (7, 64, 8, 1, 1, 1), (300, 64, 8, 8, 3, 2),
                                                               (90, 256, 8, 8, 2, 1), (50, 700, 32, 1, 1, 1)])
def test_bias_takes_experts_out(T, E, k, groups, top_groups, group_top, score):
    say("bias", T, E, k, groups, score)
    g = torch.Generator()
    g.manual_seed(T + E)
    # sigmoid scores 1/2 or below 1e-13, softmax scores of equal logits: the biases, far apart
    # for binary32, decide
    l = torch.where(torch.rand(T, E, generator=g) < 0.5, 0.0, -32.0) if score == "sigmoid" else torch.full((T, E), 0.5)
    l[torch.rand(T, E, generator=g) < 0.05] = -math.inf
    bias = torch.rand(E, generator=g) * 8 - 4
    out = torch.rand(E, generator=g) < 0.6  # too few are left for some tokens
    bias[out] = -math.inf
    bias[1] = math.nan
    bias[2] = -math.nan if E == 64 else bias[2]
    if groups > 1:
        bias[:E // groups] = -math.inf  # a whole group
    got = F.fp4_route(l.to(DEV), k, score=score, bias=bias.to(DEV), groups=groups, top_groups=top_groups, group_top=group_top)
    idx, w, flat = reference(l, k, score, bias, groups, top_groups, group_top)
    assert torch.equal(got.experts.cpu(), idx)
    # (the routing weights' bound with logits within 32 of the largest)
    assert ((got.weights.cpu().double() - w).abs() <= (2 * 32 + 40) * 2.0 ** -24 * w + 1e-37).all()
    slots = torch.sort(flat, stable=True).indices
    assert torch.equal(got.slots.cpu().long(), slots)
    assert torch.equal(got.offsets.cpu().long(), torch.searchsorted(flat[slots], torch.arange(E + 1)))


def test_no_expert_is_left():
    r = F.fp4_route(torch.zeros(40, 16, device=DEV), 2, bias=torch.full((16,), -math.inf, device=DEV))
    assert (r.experts == -1).all() and not r.weights.any() and not r.offsets.any()
    assert torch.equal(r.slots.cpu(), torch.arange(80, dtype=torch.int32))


def test_positive_infinity_is_chosen_first():
    bias = torch.zeros(16, device=DEV)
    bias[11] = math.inf
    r = F.fp4_route(torch.randn(40, 16, device=DEV), 2, score="sigmoid", bias=bias)
    assert (r.experts[:, 0] == 11).all()
