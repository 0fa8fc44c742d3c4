"""The plain forms of dropout, layer norm, router and embedding themselves (no
GPU): known answers, and gradients against differences of the forward pass."""
import numpy as np
import pytest
import torch

import step_reference as ref

D = torch.float64


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, words):
    assert [int(w) for w in ref.philox(counter, key)] == list(words)


@pytest.mark.parametrize("p", [0.05, 0.1, 0.5, 0.9])
def test_the_factors_share_and_mean(p):
    f = ref.drop_factor(256, 1024, p, 77, 5, 3)
    n, q = f.numel(), ref.cut_of(p) / 65536
    kept = (f > 0).double().mean().item()
    assert abs(kept - (1 - q)) < 5 * np.sqrt(q * (1 - q) / n)
    assert abs(f.mean().item() - 1) < 5 * np.sqrt(q / (1 - q) / n)
    # rows, columns, sites and steps are independent of each other
    for other in (ref.drop_factor(256, 1024, p, 77, 5, 4), ref.drop_factor(256, 1024, p, 77, 6, 3),
                  ref.drop_factor(256, 1024, p, 78, 5, 3), f.roll(1, 0), f.roll(1, 1), f.roll(8, 1)):
        both = ((f > 0) & (other > 0)).double().mean().item()
        assert abs(both - (1 - q) ** 2) < 6 * np.sqrt((1 - q) ** 2 / n)


def differences(f, x, h=1e-5):
    """Central differences of the scalar f by every element of x."""
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = f().item()
        flat[i] = keep - h
        out[i] = (up - f().item()) / (2 * h)
        flat[i] = keep
    return g


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=D)


def test_layer_norm_gradients_are_those_of_differences():
    rows, H = 3, 7
    u, res, w, b = randn(rows, H, seed=1), randn(rows, H, seed=2), randn(H, seed=3), randn(H, seed=4)
    dy, dr = randn(rows, H, seed=5), randn(rows, H, seed=6)
    factor = ref.drop_factor(rows, H, 0.3, 9, 1, 2)

    def layer():
        return ref.LayerNorm(u, res, w, b, 1e-5, 0.5, factor).forward()

    def value():
        n = layer()
        return (n.y * dy).sum() + (n.out * dr).sum()
    n = layer()
    got = n.backward(dy, dr, n.out, n.mean, n.rstd)
    for name, x in (("du", u), ("dres", res), ("dweight", w), ("dbias", b)):
        assert torch.allclose(got[name][0], differences(value, x), atol=1e-6), name


@pytest.mark.parametrize("normalize", [False, True])
def test_router_gradient_is_that_of_differences(normalize):
    T, E, K = 5, 6, 3
    x, dw = randn(T, E, seed=1), randn(T, K, seed=2)
    x[1, 2] = -np.inf
    mask = torch.tensor([1, 1, 0, 1, 1])

    def value():
        r = ref.Router(x, mask, K, normalize, 0.7, 0.2).forward()
        return 1.5 * r.loss + (r.weights * dw).sum()
    got = ref.Router(x, mask, K, normalize, 0.7, 0.2).forward().backward(dw, 1.5)[0]
    finite = torch.isfinite(x)
    want = torch.zeros_like(x)
    for t, e in finite.nonzero().tolist():
        keep = x[t, e].item()
        x[t, e] = keep + 1e-5
        up = value().item()
        x[t, e] = keep - 1e-5
        want[t, e] = (up - value().item()) / 2e-5
        x[t, e] = keep
    assert torch.allclose(got, want, atol=1e-6)


def test_embedding_gradient_is_that_of_differences():
    table, d = randn(4, 3, seed=1), randn(6, 3, seed=2)
    idx = torch.tensor([2, -1, 0, 2, 9, 2])
    got = ref.embedding_backward(idx, d, 4, 1.7)[0]
    assert torch.allclose(got, differences(lambda: (ref.embedding(idx, table, 1.7)[0] * d).sum(), table),
                          atol=1e-6)
