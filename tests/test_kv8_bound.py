"""The error bound of tests/_kv8_bound.py says something: it takes the right
output rounded to fp32, and refuses outputs with a step, a flush or a team's
share left out, on rows of every length that the GPU tests use."""
import pytest
import torch

from tests import _kv8_bound as A

D = 128


def _head(T, G, mean, seed):
    g = torch.Generator().manual_seed(seed)
    spread = lambda: torch.exp(0.5 * torch.randn((1, D), generator=g))  # noqa: E731
    k, v = (torch.randn((T, D), generator=g) * spread() for _ in range(2))
    q = (torch.randn((G, D), generator=g) * spread()).bfloat16().double()
    sv = torch.exp2(torch.ceil(torch.log2((v + mean).abs().amax() / 448.0))).double().expand(T, 1)
    return q, k.double(), (v + mean).double(), sv


def _without(q, k, v, gone, sums_only):
    """The output with tokens `gone` left out (sums_only: of the sums over values, not of those of p)."""
    x = q @ k.T / D ** 0.5
    p = torch.softmax(x, -1)
    p2 = p.clone()
    p2[:, gone] = 0.0
    return (p2 @ v) / (1.0 if sums_only else p2.sum(-1, keepdim=True))


@pytest.mark.parametrize("T,G,mean", [(20011, 4, 0.0), (65537, 4, 0.0), (131072, 4, 0.0), (131072, 4, 1.0),
                                      (150000, 2, 0.0), (150001, 8, 1.0)])
def test_bound_refuses_missing_tokens(T, G, mean):
    q, k, v, sv = _head(T, G, mean, T + G)
    S = A.stretch([T], 8, G, False, 148)
    seen = torch.ones(T, dtype=torch.bool)
    ref, tol = A.head(q, k, v, sv, seen, False, S)
    assert A.worst(ref.float(), ref, tol) < 0.1
    assert A.worst(torch.zeros_like(ref), ref, tol) > 10
    assert float(((ref.abs() > tol).double().mean())) > 0.9  # zeros fail nearly everywhere
    for first in (0, T // 2 // 32 * 32, T - 32):
        step = slice(first, first + 32)
        assert A.worst(_without(q, k, v, step, False), ref, tol) > 1
        assert A.worst(_without(q, k, v, step, True), ref, tol) > 1
    for n in (16 * 32, S * 32):  # one flush's sums; one team's share
        gone = slice(T // 3 // 32 * 32, T // 3 // 32 * 32 + n)
        assert A.worst(_without(q, k, v, gone, True), ref, tol) > 4
        assert A.worst(_without(q, k, v, gone, False), ref, tol) > 1


def test_bound_refuses_probabilities_scaled_by_a_page_without_weight():
    """Probabilities as two fp16 halves: scaled by the largest p times value
    scale they keep to the bound, by the largest value scale alone they do not."""
    q, k, v, sv = _head(96, 4, 0.0, 1)
    R = 20
    k[64:] = 0.0
    k[:64, 0] += 60.0 * D ** 0.5  # with q's channel 0 of 1: some 60 nats above the last page
    q[:, 0] = 1.0
    v, sv = v.clone(), sv.clone()
    v[64:] *= 2.0 ** R
    sv[64:] *= 2.0 ** R
    ref, tol = A.head(q, k, v, sv, torch.ones(96, dtype=torch.bool), False, 1)
    x = q @ k.T / D ** 0.5
    p = torch.exp(x - x.amax(-1, keepdim=True))

    def halves(top):
        y = (p * sv.T / top * 2.0 ** 6).float()
        hi = y.half()
        y = hi.double() + (y - hi.float()).half().double()
        return (y @ (v / sv)) * top / 2.0 ** 6 / p.sum(-1, keepdim=True)

    own = torch.exp2(torch.ceil(torch.log2((p * sv.T).amax(-1, keepdim=True))))
    assert A.worst(halves(own), ref, tol) < 1
    assert A.worst(halves(sv.max()), ref, tol) > 1
