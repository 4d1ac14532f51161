"""The 64-bit references of the behaviour-history operators against published
vectors, differences and closed forms (CPU)."""
import numpy as np
import pytest
import torch

import history_ref as R


def test_philox_published_vectors():
    assert R.philox4x32([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert R.philox4x32([R.MASK] * 4, [R.MASK] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_keep_mask_share_and_factor():
    n, p = 40000, 0.3
    keep, f = R.keep_mask(n, p, 12345, (1 << 63) + 17)
    cut = int(p * 65536 + 0.5)
    want = 1 - cut / 65536
    # five standard deviations of a binomial share
    assert abs(keep.mean() - want) < 5 * np.sqrt(want * (1 - want) / n)
    assert abs(f * want - 1) < 1e-12
    assert not R.keep_mask(64, 1.0, 3, 4)[0].any() and R.keep_mask(64, 0.0, 3, 4)[0].all()


def _differences(f, x, step=1e-6):
    g = torch.zeros_like(x)
    flat, gf = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + step
        a = f()
        flat[i] = keep - step
        b = f()
        flat[i] = keep
        gf[i] = (a - b) / (2 * step)
    return g


def test_embed_grad_against_differences():
    g = torch.Generator().manual_seed(1)
    T = torch.randn(5, 4, generator=g, dtype=torch.float64)
    tok = torch.tensor([0, 3, 3, -1, 4, 7, 0])
    dout = torch.randn(7, 4, generator=g, dtype=torch.float64)
    want = _differences(lambda: (R.embed(T, tok, 2.5) * dout).sum(), T)
    assert torch.allclose(R.embed_grad(tok, dout, 5, 2.5)[0], want, atol=1e-8)


@pytest.mark.parametrize("p", [0.0, 0.4])
def test_addnorm_grad_against_differences(p):
    g = torch.Generator().manual_seed(2)
    n, d = 3, 7
    x, res, dy, dh = (torch.randn(n, d, generator=g, dtype=torch.float64) for _ in range(4))
    w = torch.randn(d, generator=g, dtype=torch.float64)
    keep, f = R.keep_mask(n * d, p, 9, 10)
    keep = torch.from_numpy(keep).view(n, d)

    def loss():
        h, y, _ = R.addnorm(x, res, w, 1e-3, keep, f)
        return (y * dy).sum() + (h * dh).sum()

    h, _, r = R.addnorm(x, res, w, 1e-3, keep, f)
    dx, dres, dw = R.addnorm_grad(dy, dh, h, w, r, keep, f)
    for got, var in ((dx, x), (dres, res), (dw, w)):
        assert torch.allclose(got, _differences(loss, var), atol=1e-6)


def test_linattn_grad_against_differences():
    g = torch.Generator().manual_seed(3)
    off = [0, 3, 3, 8]
    H, dk, dv = 2, 3, 4
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do = rnd(8, H, dk), rnd(8, H, dk), rnd(8, H, dv), rnd(8, H, dv)
    S0, dS = rnd(3, H, dk, dv), rnd(3, H, dk, dv)
    lam = torch.tensor([0.9, 0.3], dtype=torch.float64)

    def loss():
        o, S = R.linattn(q, k, v, off, lam, 0.7, S0)
        return (o * do).sum() + (S * dS).sum()

    got = R.linattn_grad(q, k, v, do, off, lam, 0.7, S0, dS)
    for a, var in zip(got, (q, k, v, S0)):
        assert torch.allclose(a, _differences(loss, var), atol=1e-6)


def test_linattn_equals_its_double_sum():
    g = torch.Generator().manual_seed(4)
    T, dk, dv = 9, 4, 5
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v = rnd(T, 1, dk), rnd(T, 1, dk), rnd(T, 1, dv)
    t = torch.arange(T)
    D = torch.where(t[:, None] >= t, 0.8 ** (t[:, None] - t).double(), 0.0)
    want = ((q[:, 0] @ k[:, 0].T) * D) @ v[:, 0] * 0.5
    assert torch.allclose(R.linattn(q, k, v, [0, T], torch.tensor([0.8], dtype=torch.float64), 0.5)[0][:, 0], want)
