"""The global gradient norm and clipping (in place, and into tiles) against 64-bit arithmetic, and the chain
from a layer's norm to the clipped tiles.

Tolerances, u = 2^-24.  A norm: squares in pieces of at most 8 elements carry 8 roundings of one sign's sum,
64 bits from there; the root halves that and its own rounding adds u: 5u, 6u with the second order.  The factor
max_norm / norm and the product carry u each, the stored value half a step of its type (or half of its least
magnitude)."""
import math
import random

import numpy as np
import pytest
import torch

import matrix_inverse_roots_amd as dash
import mx_ref as ref
from gpu_helpers import DEV
from test_gpu_norm import LEAST, NAMES, TYPES, U, half, randn

pytestmark = pytest.mark.gpu


def grads_of(seed, shapes, types, pad=0):
    """Tensors of these shapes, one after the other in a buffer of each type with `pad` elements between (and
    between the rows of matrices); the buffers too."""
    rng = random.Random(seed)
    kinds = [rng.choice(types) for _ in shapes]
    size = {t: 64 for t in types}
    for s, t in zip(shapes, kinds):
        rows, cols = (1, s) if isinstance(s, int) else s
        size[t] += rows * (cols + pad) + pad
    flat = {t: randn(seed + i, size[t], dtype=t) for i, t in enumerate(types)}
    at, out = {t: pad for t in types}, []
    for s, t in zip(shapes, kinds):
        if isinstance(s, int):
            out.append(flat[t][at[t]:at[t] + s])
            at[t] += s + pad
        else:
            out.append(flat[t].as_strided(s, (s[1] + pad, 1), at[t]))
            at[t] += s[0] * (s[1] + pad) + pad
    return out, flat


def norm(grads, per_tensor=True):
    out = torch.full((1,), -1.0, device=DEV)
    norms = torch.full((len(grads),), -1.0, device=DEV) if per_tensor else None
    dash.dash_grad_norm(grads, out, norms=norms, ws=dash.grad_norm_workspace(grads, device=DEV))
    torch.cuda.synchronize()
    return out, norms


def close(got, want, tol):
    return abs(float(got) - want) <= tol * want


LISTS = {
    "one element": [1],
    "an empty one": [0],
    "empty ones between": [0, 5, (0, 7), (7, 0), 3, 0],
    "around a piece": [1, 3, 4, 5, 7, 8, 9, 15, 16, 17],
    "a layer": [(64, 200), (200, 64), 64, 200, (1, 33), (33, 1), (5, 3)],
    "around a workgroup's share": [16383, 16384, 16385, 32767, 32768, 32769, 65537],
    "slices of matrices": [(100, 129), (257, 64), (3, 5000), (5000, 3)],
    "eighty and one": [7] * 81,
    "a thousand": [1 + i * i % 977 for i in range(1000)],
    "large": [1 << 24, (4096, 4097), 3],
}


@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("name", LISTS)
def test_norm(name, pad):
    for types in ([torch.float32], [torch.bfloat16], [torch.float16], TYPES):
        grads, _ = grads_of(1, LISTS[name], types, pad)
        want = [float(g.double().square().sum().sqrt()) for g in grads]
        got, norms = norm(grads)
        assert close(got, math.sqrt(sum(w * w for w in want)), 6 * U)
        assert all(close(g, w, 6 * U) for g, w in zip(norms.tolist(), want))
        # described once, without the tensors' own norms: the same bits
        again, _ = norm(dash.grad_list(grads), False)
        assert torch.equal(again, got)


def test_no_gradients():
    got, _ = norm([], False)
    assert float(got) == 0.0
    dash.dash_grad_clip([], got, 1.0)


@pytest.mark.parametrize("dtype,scales", [(torch.float32, (1e-38, 1e-30, 1e-12, 1e18, 1e30, 1e38)),
                                          (torch.bfloat16, (1e-38, 1e-30, 1e-12, 1e18, 1e30, 1e38)),
                                          (torch.float16, (1e-7, 1e-5, 1e4))], ids=["fp32", "bf16", "fp16"])
def test_norm_beyond_the_squares_range(dtype, scales):
    """Elements whose squares leave fp32's range, alone and beside ordinary ones and zeros."""
    for s in scales:
        g = (randn(5, 3000).clamp(-3, 3).double() * s).to(dtype)
        g[100:900] = 0
        for grads in ([g], [g, randn(6, 500, dtype=dtype)], [torch.cat((g, randn(7, 77, dtype=dtype)))[1:]]):
            want = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
            # (subnormal results have a step of 2^-149)
            got = float(norm(grads)[0])
            if want < 3.4e38:
                assert abs(got - want) <= 6 * U * want + 2.0**-150, s
            else:
                assert got == float("inf")


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
def test_norm_of_what_is_not_finite(dtype):
    for bad in (float("nan"), float("inf"), -float("inf")):
        for at in (0, 7, 1000, 2999):
            grads = [randn(8 + i, 3000, dtype=dtype) for i in range(3)]
            grads[1][at] = bad
            got, norms = norm(grads)
            want = float("nan") if math.isnan(bad) else float("inf")
            for v in (float(got), float(norms[1])):
                assert math.isnan(v) if math.isnan(want) else v == want
            assert math.isfinite(float(norms[0])) and math.isfinite(float(norms[2]))


def test_norm_past_32_bits():
    """A tensor of over 2^32 elements, and rows that start beyond 2^32 elements."""
    g = torch.zeros((1 << 32) + 1000, dtype=torch.bfloat16, device=DEV)
    g[0], g[1 << 31], g[-1] = 2.0, 3.0, 6.0
    got, norms = norm([g, g[:5], g.view(-1)[:70000 * 61000].view(70000, 61000)[:, 60999:]])
    assert float(norms[0]) == 7.0 and float(norms[1]) == 2.0 and float(norms[2]) == 0.0
    g[69999 * 61000 + 60999] = 5.0
    tail = g[:70000 * 61000].view(70000, 61000)[:, 60990:]
    assert float(norm([tail])[0]) == 5.0
    dash.dash_grad_clip([tail], torch.full((1,), 5.0, device=DEV), 2.5)
    assert float(g[69999 * 61000 + 60999]) == 2.5 and float(g[-1]) == 6.0


@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("name", LISTS)
def test_clip(name, pad):
    for types in ([torch.float32], [torch.bfloat16], [torch.float16], TYPES):
        grads, flat = grads_of(2, LISTS[name], types, pad)
        before = {t: f.clone() for t, f in flat.items()}
        inside = {t: torch.zeros_like(f, dtype=torch.bool) for t, f in flat.items()}
        for g in grads:
            inside[g.dtype].as_strided(g.shape, g.stride(), g.storage_offset()).fill_(True)
        total, _ = norm(grads)
        v = float(total)
        if v:
            dash.dash_grad_clip(grads, total, 2 * v)  # nothing to clip: the same bits
            dash.dash_grad_clip(grads, total, v)
        assert all(torch.equal(flat[t], before[t]) for t in flat)
        dash.dash_grad_clip(grads, total, 0.37 * v)
        c = 0.37 * v / v if v else 1.0
        # (0.37 v enters as fp32: u more)
        for t in flat:
            want = torch.where(inside[t], before[t].double() * c, before[t].double())
            tol = torch.where(inside[t], (3 * U + half(t)) * want.abs() + LEAST[t], torch.zeros_like(want))
            assert bool(((flat[t].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
def test_large_lists(dtype):
    """Lists beyond the caches' size, which are read and written past them, with odd pieces among them."""
    n = 3 * 2**26 if dtype != torch.float32 else 3 * 2**25
    flat = randn(11, n, scale=1e-3, dtype=dtype)
    old = flat.clone()
    grads = [flat[:5], flat[5:n // 2 - 3], flat[n // 2:n // 2 + 4097 * 1000].view(1000, 4097)[:, 1:4090],
             flat[n // 2 + 4097 * 1000:n - 1]]
    total, norms = norm(grads)
    want = [math.sqrt(sum(float(p.double().square().sum()) for p in g.split(1 << 24 if g.dim() == 1 else 1000)))
            for g in grads]
    assert close(total, math.sqrt(sum(w * w for w in want)), 6 * U)
    assert all(close(g, w, 6 * U) for g, w in zip(norms.tolist(), want))
    dash.dash_grad_clip(grads, total, 0.5 * float(total))  # (the factor is exact)
    inside = torch.zeros(n, dtype=torch.bool, device=DEV)
    for g in grads:
        inside.as_strided(g.shape, g.stride(), g.storage_offset()).fill_(True)
    assert torch.equal(flat, torch.where(inside, old * 0.5, old))


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
def test_clip_by_any_norm(dtype):
    inf, nan = float("inf"), float("nan")
    for value, most, factor in ((0.0, 0.0, 1), (5.0, 0.0, 0), (1.0, inf, 1), (inf, inf, 1), (inf, 1.0, 0), (nan, 1.0, nan),
                                (nan, inf, nan), (4.0, 1.0, 0.25), (1e-40, 1.0, 1)):
        g = randn(9, 1000, dtype=dtype)
        g[3], g[4] = inf, nan
        old = g.clone()
        dash.dash_grad_clip([g], torch.tensor([value], device=DEV), most)
        want = old if factor == 1 else (old.float() * factor).to(dtype)
        assert torch.equal(g.isnan(), want.isnan())
        assert torch.equal(g[~g.isnan()], want[~want.isnan()])


def test_interleaved_slices():
    """Column slices of one buffer are gradients of their own."""
    wide = randn(10, 50, 300)
    old = wide.clone()
    parts = [wide[:, :100], wide[:, 100:101], wide[:, 150:300]]
    total, _ = norm(parts)
    dash.dash_grad_clip(parts, total, float(total) * 0.5)
    c = wide / old
    assert bool(((c[:, :101] - 0.5).abs() < 1e-6).all()) and bool(((c[:, 150:] - 0.5).abs() < 1e-6).all())
    assert torch.equal(wide[:, 101:150], old[:, 101:150])
    for bad in ([wide, wide[:, :3]], [parts[0], wide[:, 99:120]], [parts[0], parts[0]], [wide[3], parts[2]]):
        with pytest.raises(dash.DashError):
            dash.dash_grad_clip(bad, total, 1.0)


@pytest.mark.parametrize("B", [64, 192])
def test_clip_into_tiles(B):
    shapes = [(1, 1), (64, 64), (65, 63), (200, 130), (3, 700), (700, 3), (192, 384)] * 6  # (over one launch's)
    grads = [randn(20 + i, r, -(-c // 4) * 4)[:, :c] for i, (r, c) in enumerate(shapes)]
    old = [g.clone() for g in grads]
    total, _ = norm(grads)
    n = sum(-(-r // B) * -(-c // B) for r, c in shapes)
    G, plain = (torch.full((n, B, B), 7.0, device=DEV) for _ in range(2))
    dash.dash_stack(grads, B, plain)
    for most in (float(total) * 2, float("inf")):
        G.fill_(7.0)
        dash.dash_stack_clip(grads, B, total, most, G)
        assert torch.equal(G, plain)
    most = 0.25 * float(total)
    dash.dash_stack_clip(dash.grad_list(grads), B, total, most, G)
    want = plain.double() * 0.25
    assert bool(((G.double() - want).abs() <= 3 * U * want.abs()).all())
    assert all(torch.equal(a, b) for a, b in zip(grads, old))
    total.fill_(float("nan"))
    dash.dash_stack_clip(grads, B, total, most, G)
    assert bool(G[1].isnan().all())


def test_wrong_tensors_are_refused():
    x, total = torch.zeros((8, 64), device=DEV), torch.zeros(1, device=DEV)
    for bad in (x.int(), x.t(), x.double(), x[:, ::2], torch.zeros((2, 8, 64), device=DEV)[:, :, :32]):
        with pytest.raises(ValueError):
            dash.grad_list([x, bad])
        with pytest.raises(ValueError):
            dash.dash_grad_clip([bad], total, 1.0)
    with pytest.raises(ValueError):
        dash.dash_grad_clip([x], total.double(), 1.0)
    with pytest.raises(ValueError):
        dash.dash_grad_norm([x, x], total, norms=torch.zeros(1, device=DEV), ws=dash.grad_norm_workspace([x, x]))
    with pytest.raises(ValueError):
        dash.dash_stack_clip([x.bfloat16()], 64, total, 1.0, torch.zeros((1, 64, 64), device=DEV))
    with pytest.raises(ValueError):
        dash.dash_stack_clip(dash.grad_list([x.bfloat16()]), 64, total, 1.0, torch.zeros((1, 64, 64), device=DEV))
    with pytest.raises(dash.DashError):
        dash.dash_grad_norm([x], total)  # no workspace


# ------------------------------------------------------------------------------------------------
# Together: norm -> product -> gradient tiles -> norm of all gradients -> clipped statistics
# ------------------------------------------------------------------------------------------------

FMT, B = dash.DASH_MX_E4M3, 64


class Layer:
    """y = norm(x + res) gain, z = y W^T, and what its training step keeps."""

    def __init__(self, T, n, out):
        self.T, self.n, self.out = T, n, out
        bf = dict(dtype=torch.bfloat16, device=DEV)
        self.x, self.res, self.dz = torch.empty((T, n), **bf), torch.empty((T, n), **bf), torch.empty((T, out), **bf)
        self.dy, self.dh, self.dx = (torch.empty((T, n), **bf) for _ in range(3))
        self.gain = torch.empty(n, device=DEV)
        self.h, self.y = torch.empty((T, n), **bf), torch.empty((T, n), **bf)
        self.codes, self.scales = dash.mx_buffers(1, T, n, FMT, device=DEV)
        self.rstd, self.dgain = torch.empty(T, device=DEV), torch.empty(n, device=DEV)
        tiles = -(-out // B) * -(-n // B)
        self.G = torch.empty((tiles, B, B), device=DEV)
        self.pieces = torch.empty((-(-n // B), B), device=DEV)
        self.gws = dash.grad_stack_mx_workspace(T, out, n, torch.bfloat16, device=DEV)
        self.bws = dash.rmsnorm_backward_workspace(T, n, device=DEV)
        self.grads = dash.grad_list([self.G, self.dgain])
        self.nws = dash.grad_norm_workspace(self.grads, device=DEV)
        self.total, self.norms = torch.empty(1, device=DEV), torch.empty(2, device=DEV)
        self.A, self.L = torch.zeros((2 * tiles, B, B), device=DEV), torch.zeros((-(-n // B), B, B), device=DEV)

    def fill(self, seed):
        for i, (t, s) in enumerate(((self.x, 1.0), (self.res, 2.0), (self.dz, 0.01), (self.dy, 0.01), (self.dh, 0.01))):
            t.copy_(randn(seed + i, *t.shape, scale=s))
        self.gain.copy_(1 + randn(seed + 9, self.n, scale=0.2))

    def step(self, most):
        T, n = self.T, self.n
        dash.dash_rmsnorm(self.x, T, n, 1e-5, res=self.res, gain=self.gain, h=self.h, y=self.y, fmt=FMT, codes=self.codes,
                          scales=self.scales, rstd=self.rstd)
        dash.dash_grad_stack_mx(self.dz, self.codes, self.scales, FMT, T, self.out, n, B, self.G, ws=self.gws)
        dash.dash_rmsnorm_backward(self.dy, self.h, self.rstd, T, n, self.dx, gain=self.gain, dh=self.dh,
                                   dgain=self.dgain, ws=self.bws)
        dash.dash_grad_norm(self.grads, self.total, norms=self.norms, ws=self.nws)
        dash.dash_grad_clip(self.grads, self.total, most)
        dash.dash_update_stats(self.G, self.G.shape[0], B, 0.5, self.A)
        dash.dash_stack_vec([self.dgain], B, self.pieces)
        dash.dash_update_stats_vec(self.pieces, self.pieces.shape[0], B, 0.5, self.L)

    OUT = ("h", "y", "codes", "scales", "rstd", "G", "dx", "dgain", "total", "norms", "A", "L")

    def results(self):
        torch.cuda.synchronize()
        return {k: getattr(self, k).clone() for k in self.OUT}

    def reset(self):
        self.A.zero_()
        self.L.zero_()


def equal(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_the_operators_together():
    """Each stage against 64 bits on what the stage before it left."""
    T, n, out = 700, 200, 150
    s = Layer(T, n, out)
    s.fill(300)
    h = s.x.double() + s.res.double()
    rstd = ((h * h).mean(1) + 1e-5) ** -0.5
    y = h * rstd[:, None] * s.gain.double()
    s.step(0.1)
    assert bool(((s.y.double() - y).abs() <= (10 * U + half(torch.bfloat16)) * y.abs() + 2.0**-133).all())
    Q = torch.from_numpy(ref.values(s.codes.cpu().numpy(), s.scales.cpu().numpy(), n, FMT)[0]).to(DEV)
    assert bool(((Q - y).abs() <= 0.0626 * y.abs() + 2.0**-10 * y.abs().max() / 200).all())
    W = s.dz.double().t().contiguous() @ Q
    mag = s.dz.double().abs().t().contiguous() @ Q.abs()
    xhat = s.h.double() * s.rstd.double()[:, None]
    dg = (s.dy.double() * xhat).sum(0)
    total = float(torch.sqrt((W * W).sum() + (dg * dg).sum()))
    assert total > 0.1 and abs(float(s.total) - total) <= 1e-4 * total
    assert abs(float(s.norms[1]) - float(dg.norm())) <= 1e-4 * float(dg.norm())
    c = 0.1 / float(s.total)
    tiles = torch.from_numpy(ref.tiles((W * c).cpu().numpy(), B)).to(DEV)
    tol = torch.from_numpy(ref.tiles((c * (T + 264) * U * mag).cpu().numpy(), B)).to(DEV)
    assert bool(((s.G.double() - tiles).abs() <= tol).all())
    after = float(torch.sqrt(s.G.double().square().sum() + s.dgain.double().square().sum()))
    assert abs(after - 0.1) <= 1e-6
    N = s.G.shape[0]
    G = s.G.double()
    stat = torch.cat([0.5 * G @ G.transpose(1, 2).contiguous(), 0.5 * G.transpose(1, 2).contiguous() @ G])
    assert float((s.A.double() - stat).norm()) <= 1e-5 * float(stat.norm()) and stat.shape[0] == 2 * N
    p = torch.nn.functional.pad(s.dgain, (0, -n % B)).view(-1, B).double()
    stat = 0.5 * p[:, :, None] * p[:, None, :]
    assert float((s.L.double() - stat).norm()) <= 1e-5 * float(stat.norm())


def test_on_another_stream_and_two_at_once():
    layers = [Layer(600, 264, 130) for _ in range(2)]
    want = []
    for i, s in enumerate(layers):
        s.fill(310 + 20 * i)
        s.step(0.05)
        want.append(s.results())
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s in layers:
            s.reset()
        torch.cuda.synchronize()
        for s, st in zip(layers, streams):
            with torch.cuda.stream(st):
                s.step(0.05)
        for s, w in zip(layers, want):
            equal(s.results(), w)


def test_captured_steps_replay():
    """A captured step, replayed on new inputs between eager ones, equals them every time; two graphs share
    their workspaces."""
    s, e = Layer(530, 200, 70), Layer(530, 200, 70)
    t = Layer(1100, 72, 130)
    shared = torch.empty(max(w.numel() for w in (s.bws, t.bws)), dtype=torch.uint8, device=DEV)
    s.bws = t.bws = shared
    s.nws = t.nws = torch.empty(max(w.numel() for w in (s.nws, t.nws)), dtype=torch.uint8, device=DEV)
    graphs = []
    for k in (s, t):
        k.fill(400)
        k.step(0.05)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            k.step(0.05)
        graphs.append(g)
    other = Layer(1100, 72, 130)
    for seed in (410, 420, 430, 440):
        for k, eager, g in zip((s, t), (e, other), graphs):
            for m in (k, eager):
                m.fill(seed)
                m.reset()
            g.replay()
            eager.step(0.05)
            equal(k.results(), eager.results())


def test_descriptors_stay_with_the_call():
    """The host's descriptors are read before the call returns: changing them afterwards changes nothing."""
    grads = [randn(500 + i, 1 << 20) for i in range(90)]
    want = float(norm(grads)[0])
    lst = dash.grad_list(grads)
    total = torch.empty(1, device=DEV)
    ws = dash.grad_norm_workspace(lst, device=DEV)
    dash.dash_grad_norm(lst, total, ws=ws)
    for i in range(90):
        lst.array[i].ptr, lst.array[i].cols = 1 << 20, 0
    assert float(total) == want
    assert np.isfinite(want)
