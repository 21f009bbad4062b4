"""The bound for the routing gradient tells mistakes from roundings: a plain fp32 evaluation is
inside it, gradients without one of their terms are not (on the CPU)."""
import numpy as np
import pytest
import torch

import moe_reference as ref
from moe_reference import close
from route_tolerance import route_backward_tolerance


def inputs(T, E, k):
    g = torch.Generator().manual_seed(E + k)
    x = 1.5 * torch.randn((T, E), generator=g)
    ids = x.topk(k, dim=1).indices.to(torch.int32).numpy().astype(np.int64)
    ids[0, 0] = -1
    return x.double().numpy(), ids, torch.randn((T, k), generator=g).double().numpy()


def plain(dw, x, ids, sigmoid_score, renorm):
    """The formulas in fp32 (numpy)."""
    f = np.float32
    x, here = x.astype(f), ids >= 0
    at = np.where(here, ids, 0)
    g = np.where(here, dw.astype(f), f(0))
    sel = np.take_along_axis(x, at, 1)
    d = np.zeros_like(x)
    if sigmoid_score:
        s, rest = f(1) / (f(1) + np.exp(-sel)), f(1) / (f(1) + np.exp(sel))
        s = np.where(here, s, f(0))
        if renorm:
            total = s.sum(1, keepdims=True) + f(1e-20)
            g = (g - (g * s).sum(1, keepdims=True) / total) / total
        mine = g * s * rest
    elif renorm:
        w = np.where(here, np.exp(sel - np.where(here, sel, f(-1e9)).max(1, keepdims=True)), f(0))
        w = w / w.sum(1, keepdims=True)
        mine = w * (g - (w * g).sum(1, keepdims=True))
    else:
        p = np.exp(x - x.max(1, keepdims=True))
        p = p / p.sum(1, keepdims=True)
        mine = np.take_along_axis(p, at, 1) * g
        d = -p * mine.sum(1, keepdims=True)
    assert mine.dtype == f and d.dtype == f
    for t, j in zip(*np.nonzero(here)):
        d[t, ids[t, j]] += mine[t, j]
    return d.astype(np.float64)


@pytest.mark.parametrize("E,k", [(8, 2), (33, 4), (160, 6), (256, 8), (500, 10), (1024, 32)])
@pytest.mark.parametrize("sigmoid_score,renorm", [(False, False), (False, True), (True, False),
                                                  (True, True)])
def test_bound(E, k, sigmoid_score, renorm):
    x, ids, dw = inputs(40, E, k)
    want = ref.route_backward(dw, x, ids, sigmoid_score, renorm, 1.0)
    tol = route_backward_tolerance(dw, x, ids, sigmoid_score, renorm, 1.0, torch.float32, want)
    got = plain(dw, x, ids, sigmoid_score, renorm)
    close(got, want, tol, "the fp32 form")
    chosen = np.zeros(x.shape, bool)
    for t, j in zip(*np.nonzero(ids >= 0)):
        chosen[t, ids[t, j]] = True
    if not sigmoid_score and not renorm:
        # what the experts that were not chosen share: nearly every value can be told from 0
        assert (tol < 0.01 * np.abs(want))[~chosen].mean() > 0.99
        with pytest.raises(AssertionError):
            close(np.where(chosen, want, 0.0), want, tol, "zeros for the others")
        with pytest.raises(AssertionError):
            close(want * (1 + 1e-4 * ~chosen), want, tol, "others off by 1e-4")
    else:
        assert not want[~chosen].any() and not tol[~chosen].max() > 1e-40
    if k > 1:
        with pytest.raises(AssertionError):
            close(want * (1 + 1e-4 * chosen), want, tol, "the chosen off by 1e-4")
