"""What a list of gradients that is described once stands for (no GPU: host tensors in the place of the GPU's, and a
library that takes the calls' arguments down)."""
import ctypes

import pytest
import torch

import matrix_inverse_roots_amd as dash
from matrix_inverse_roots_amd import _lib

NORM, STACK = 1 << 24, 2 << 24


class Calls:
    """The library's entry points: every call succeeds and leaves its descriptors in `last`."""

    def __getattr__(self, name):
        def call(arr, n, *rest):
            self.last = [(arr[i].ptr, arr[i].rows, arr[i].cols, arr[i].ld) for i in range(n)]
            if name.endswith("_workspace"):
                ctypes.cast(rest[0], ctypes.POINTER(ctypes.c_size_t))[0] = 1
            return 0

        return call


@pytest.fixture
def calls(monkeypatch):
    _lib._torch()
    calls = Calls()
    monkeypatch.setattr(_lib, "library", lambda: calls)
    monkeypatch.setattr(_lib._Args, "_tensor", lambda self, t, name: isinstance(t, torch.Tensor))
    return calls


def every_call(lst):
    yield lambda: dash.dash_grad_norm(lst, NORM, stream=0)
    yield lambda: dash.dash_grad_norm_workspace(lst)
    yield lambda: dash.dash_grad_clip(lst, NORM, 1.0, stream=0)
    yield lambda: dash.dash_stack_clip(lst, 64, NORM, 1.0, STACK, stream=0)


def gradients():
    return [torch.zeros(8, 64), torch.zeros(70, 132)[:, :130], torch.zeros(3, 4)]


def test_the_tensors_themselves(calls):
    ts = gradients()
    lst = dash.grad_list(ts)
    for call in every_call(lst):
        call()
        assert [p for p, *_ in calls.last] == [t.data_ptr() for t in ts]
    ts[0].add_(1)  # (their values may change)
    for call in every_call(lst):
        call()


def test_other_memory_is_refused(calls):
    def data(t):
        t.data = torch.zeros_like(t)

    def set_(t):
        t.set_(torch.zeros(t.numel()).view(t.shape))

    def resized(t):  # (as sharded training frees a parameter)
        t.untyped_storage().resize_(0)

    def shifted(t):
        t.data = t.data[1:]

    def grown(t):
        t.resize_(1000, 1000)

    for change in (data, set_, resized, shifted, grown):
        for i in range(3):
            ts = gradients()
            lst = dash.grad_list(ts)
            for call in every_call(lst):
                call()
            change(ts[i])
            for call in every_call(lst):
                with pytest.raises(ValueError, match=r"\[%d\] has other memory" % i):
                    call()
            for call in every_call(dash.grad_list(ts)) if change not in (resized, grown) else ():
                call()


def test_the_memory_stays(calls):
    """A list keeps what its descriptors point to, so that nothing else can come to lie there."""
    t = torch.zeros(1 << 16)
    lst = dash.grad_list([t])
    at = t.data_ptr()
    t.data = torch.zeros(1 << 16)
    held = [torch.zeros(1 << 16) for _ in range(50)]
    assert all(h.data_ptr() != at for h in held)
    with pytest.raises(ValueError):
        dash.dash_grad_clip(lst, NORM, 1.0, stream=0)


def test_other_sizes_in_the_same_memory(calls):
    """Tiles are refused, whether the list has been used for tiles before or not.  Norm and clipping take what the list
    was made of."""
    for used in (False, True):
        for change in (lambda t: t.resize_(8, 4), lambda t: t.resize_(64, 256), lambda t: t.resize_(255, 256)):
            ts = [torch.zeros(64, 64), torch.zeros(256, 256)]
            lst = dash.grad_list(ts)
            if used:
                dash.dash_stack_clip(lst, 64, NORM, 1.0, STACK, stream=0)
            change(ts[1])
            with pytest.raises(ValueError, match="other sizes"):
                dash.dash_stack_clip(lst, 64, NORM, 1.0, STACK, stream=0)
            dash.dash_grad_clip(lst, NORM, 1.0, stream=0)
            assert calls.last == [(ts[0].data_ptr(), 1, 4096, 4096), (ts[1].data_ptr(), 1, 65536, 65536)]


def test_tiles_are_those_of_the_description(calls):
    """A weight that is transposed in place, after or before the list's first tiles: the stack has to hold the tiles that
    are launched."""
    for used in (False, True):
        t = torch.zeros(64, 250)
        lst = dash.grad_list([t])
        if used:
            dash.dash_stack_clip(lst, 192, NORM, 1.0, STACK, stream=0)
        t.t_()
        for B, tiles in ((192, 2), (64, 4), (192, 2)):
            with pytest.raises(ValueError, match="G_stack"):
                dash.dash_stack_clip(lst, B, NORM, 1.0, torch.zeros(tiles * B * B - 1), stream=0)
            dash.dash_stack_clip(lst, B, NORM, 1.0, torch.zeros(tiles * B * B), stream=0)
            assert calls.last == [(t.data_ptr(), 64, 250, 250)]
