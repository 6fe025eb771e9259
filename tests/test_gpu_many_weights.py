"""Stacking, stacking with clipping, and unstacking of more weights than one launch takes (80), of any number that
one launch takes, and of lists whose launches end by size (2^16 workgroups of 16 KiB of tiles): copies, so every
bit is compared; the clipping factor is a power of two."""
import random

import pytest
import torch

import matrix_inverse_roots_amd as dash
from gpu_helpers import DEV
from test_gpu_norm import randn

pytestmark = pytest.mark.gpu


def ragged(count, B, seed):
    """Weights of less than a tile, of whole tiles and with edge tiles, in buffers with room between their rows."""
    rng = random.Random(seed)
    side = lambda: rng.choice((1, 3, B - 1, B, B + 1, rng.randrange(1, 3 * B), 2 * B))
    shapes = [(side(), side()) for _ in range(count)]
    return [randn(seed + i, r, c + -c % 4 + 4 * rng.randrange(3))[:, :c] for i, (r, c) in enumerate(shapes)]


def tiles(W, B):
    r, c = -(-W.shape[0] // B), -(-W.shape[1] // B)
    W = torch.nn.functional.pad(W, (0, c * B - W.shape[1], 0, r * B - W.shape[0]))
    return W.reshape(r, B, c, B).permute(0, 2, 1, 3).reshape(r * c, B, B)


def check(weights, B):
    sizes = [-(-w.shape[0] // B) * -(-w.shape[1] // B) for w in weights]
    G = torch.full((sum(sizes) + 1, B, B), 7.0, device=DEV)

    def stacked(factor):
        at = 0
        for i, (w, k) in enumerate(zip(weights, sizes)):
            assert torch.equal(G[at:at + k], tiles(w, B) * factor), i
            at += k
        assert bool((G[at] == 7).all())

    dash.dash_stack(weights, B, G[:-1])
    stacked(1.0)
    outs = [torch.full((w.shape[0] + 2, w.stride(0) + 8), -5.0, device=DEV) for w in weights]
    views = [o[1:1 + w.shape[0], 4:4 + w.shape[1]] for o, w in zip(outs, weights)]
    dash.dash_unstack(G[:-1], B, views)
    for i, (o, v, w) in enumerate(zip(outs, views, weights)):
        assert torch.equal(v, w), i
        v.fill_(-5.0)
        assert bool((o == -5).all()), i
    del outs, views
    norm = torch.full((1,), 8.0, device=DEV)
    for grads in (weights, dash.grad_list(weights)):
        G[:-1].fill_(7.0)
        dash.dash_stack_clip(grads, B, norm, 2.0, G[:-1])
        stacked(0.25)


@pytest.mark.parametrize("B", [64, 192])
@pytest.mark.parametrize("count", [64, 65, 70, 79, 80, 81, 170])
def test_many_weights(count, B):
    check(ragged(count, B, 1000 * count), B)


@pytest.mark.parametrize("first", [(16384, 16384), (16384 - 64, 16384), (16320, 16450)])
def test_launches_that_end_by_size(first):
    """The first weight fills a launch, nearly fills it, or passes it with edge tiles; small ragged ones follow."""
    B = 64
    big = randn(1, first[0], first[1] + -first[1] % 4)[:, :first[1]]
    check([big] + ragged(75, B, 2) + [big[:9000]] + ragged(30, B, 3), B)


@pytest.mark.parametrize("B", [64, 192])
def test_norms_that_are_not_finite(B):
    """An infinite norm makes finite elements 0 and others NaN, and the padding stays 0; a NaN norm makes every element
    of every tile NaN, the padding's too."""
    weights = ragged(20, B, 4)
    weights[3][0, 0] = float("inf")
    n = sum(-(-w.shape[0] // B) * -(-w.shape[1] // B) for w in weights)
    G = torch.full((n, B, B), 7.0, device=DEV)
    dash.dash_stack_clip(weights, B, torch.full((1,), float("inf"), device=DEV), 1.0, G)
    want = torch.cat([tiles(w * 0.0, B) for w in weights])
    assert torch.equal(G.isnan(), want.isnan()) and int(G.isnan().sum()) == 1
    assert not bool(G[~G.isnan()].any())
    dash.dash_stack_clip(weights, B, torch.full((1,), float("nan"), device=DEV), 1.0, G)
    assert bool(G.isnan().all())
