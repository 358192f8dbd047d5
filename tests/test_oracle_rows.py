"""Oracle self-tests of dropout and layer norm: the generator against the
vectors published with it, the mask's layout and rate, the norm's gradients
against torch autograd in float64 and against differences."""

import numpy as np
import pytest
import torch

from oracle import dropout, dropout_gain, dropout_keep, layernorm, layernorm_grads, philox4x32


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, words):
    assert tuple(int(w) for w in philox4x32(counter, key)) == words


def test_mask_layout():
    """Row i's group j uses counter offset + i * ceil(cols / 8) + j; element e
    of it bits 16 e .. 16 e + 15."""
    rows, cols, seed, offset, p = 3, 19, 0x123456789ABCDEF0, (1 << 32) - 2, 0.3
    keep = dropout_keep(rows, cols, p, seed, offset)
    for i in range(rows):
        for c in range(cols):
            n = offset + i * 3 + c // 8
            w = philox4x32((n & 0xFFFFFFFF, n >> 32, 0, 0), (seed & 0xFFFFFFFF, seed >> 32))
            bits = sum(int(x) << (32 * k) for k, x in enumerate(w))
            assert keep[i, c] == ((bits >> (16 * (c % 8)) & 0xFFFF) >= round(65536 * p))


def test_rate_and_ends():
    n = 1 << 16
    assert dropout_keep(1, n, 0.0, 7).all() and not dropout_keep(1, n, 1.0, 7).any()
    # 5 standard deviations of a binomial count
    assert abs(dropout_keep(1, n, 0.1, 7).sum() - 0.9 * n) < 5 * np.sqrt(0.09 * n)
    assert dropout_gain(1.0) == 0.0 and dropout_gain(0.5) == 2.0
    x = np.full((1, 64), np.inf)
    assert set(np.unique(dropout(x, 0.5, 3))) == {0.0, np.inf}
    assert (dropout_keep(1, n, 0.5, 7) != dropout_keep(1, n, 0.5, 8)).any()


def test_norm_against_autograd_and_differences():
    r = np.random.default_rng(5)
    x, dy, w, b = r.normal(2, 3, (4, 9)), r.normal(size=(4, 9)), r.normal(size=9), r.normal(size=9)
    tx, tw, tb = (torch.tensor(a, requires_grad=True) for a in (x, w, b))
    ty = torch.nn.functional.layer_norm(tx, (9,), tw, tb, 1e-5)
    ty.backward(torch.tensor(dy))
    y, mean, rstd = layernorm(x, w, b, 1e-5)
    dx, dw, db = layernorm_grads(dy, x, mean, rstd, w)
    for got, ref in ((y, ty.detach()), (dx, tx.grad), (dw, tw.grad), (db, tb.grad)):
        np.testing.assert_allclose(got, ref.numpy(), rtol=1e-10, atol=1e-12)
    step = 1e-6
    for i, j in ((0, 0), (3, 8), (2, 4)):
        e = np.zeros_like(x)
        e[i, j] = step
        diff = ((layernorm(x + e, w, b)[0] - layernorm(x - e, w, b)[0]) * dy).sum() / (2 * step)
        assert abs(diff - dx[i, j]) < 1e-7
