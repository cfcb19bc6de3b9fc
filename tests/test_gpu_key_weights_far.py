"""Key weights where the scores and the lse are large: the weight is of their difference, and no rounding may be of
their own size.

Queries and keys are small integers and the scale is a power of two, so every score is exact in fp32, whatever the
order of its sum.  With u = 2^-24 and x = z - lse of the lse as given, a weight e^x has: the rounding of the difference,
u |x|; the constant log2 e and the product with it, u |x| each; the hardware's exp2, 2 u, and its argument's last step,
which is among those.  A position's sum of R terms adds (R + 64) u of itself (64: the joins of lanes and waves, and
what the terms below 2^-126 lose):
    |w - ref| <= 1.01 (sum e^x (3 u |x| + 4 u) + (R + 64) u sum e^x) + 1e-37.
The bound of longcache.py, for scores that are not exact, allows 4 u |lse| on top, which the order of steps that this
file excludes (the lse rounded as lse log2 e, then subtracted) stays within."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L

U = L.U


def _inputs(rng, T, Hq, H, D, n):
    """Integers: q [T, Hq, D], K [n, H, D] with scores of some 1,400 of which many lie within 10, and the fp32 lse over the keys."""
    g = Hq // H
    base = rng.integers(3, 9, (H, D)) * rng.choice([-1, 1], (H, D))
    q = np.repeat(base, g, 0)[None] + rng.integers(-1, 2, (T, Hq, D))
    K = np.tile(4 * np.sign(base), (n, 1, 1))
    K = np.where(rng.random((n, H, D)) < 2 / D, 3 * np.sign(base), K)
    z = np.einsum("thgd,nhd->thgn", q.reshape(T, H, g, D).astype(np.float64), K.astype(np.float64)).reshape(T, Hq, n)
    scale = 64.0 / D
    z *= scale
    top = z.max(2, keepdims=True)
    lse = (top[..., 0] + np.log(np.exp(z - top).sum(2))).astype(np.float32)
    return q, K, z, lse, scale


def _bound(z, lse):
    x = z - lse.astype(np.float64)[..., None]
    p = np.exp(x)
    ref = p.sum((0, 1))
    return ref, 1.01 * ((p * (3 * U * np.abs(x) + 4 * U)).sum((0, 1)) + (x.shape[0] * x.shape[1] + 64) * U * ref) + 1e-37


def test_the_bound_tells_the_orders_apart():
    """In fp32 on the host: the difference first is within the bound, the lse times log2 e first is not."""
    f = np.float32
    q, K, z, lse, scale = _inputs(np.random.default_rng(0), 3, 4, 2, 128, 500)
    assert np.abs(lse).min() > 1000
    ref, tol = _bound(z, lse)
    log2e = f(1.44269504088896341)
    z32 = z.astype(f)
    good = np.exp2((z32 - lse[..., None]) * log2e).astype(np.float64).sum((0, 1))
    assert (np.abs(good - ref) <= tol).all()
    far = np.exp2((z * np.float64(log2e) - (lse * log2e)[..., None].astype(np.float64)).astype(f)).astype(np.float64).sum((0, 1))
    assert (np.abs(far - ref) > tol).mean() > 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("T,Hq,H,D", [(1, 4, 1, 64), (3, 4, 2, 128), (9, 10, 5, 64), (2, 8, 8, 256), (40, 2, 1, 32)])
@pytest.mark.parametrize("n,room", [(500, 0), (1500, 1 << 17)])
def test_large_scores(dev, dt, T, Hq, H, D, n, room):
    rng = np.random.default_rng(T + D + n)
    q, K, z, lse, scale = _inputs(rng, T, Hq, H, D, n)
    P = 16
    cols = -(-n // P)
    k, ks = L.empty_cache(dev, dt, cols, P, H, D)
    table = rng.permutation(cols).astype(np.int32)
    pos = np.arange(n)
    rows = (torch.from_numpy(table[pos // P].astype(np.int64)).to(dev), torch.from_numpy(pos % P).to(dev))
    assert np.array_equal(L.put(k, ks, torch.ones(H, device=dev), rows, K.astype(np.float64)), K)
    wide = np.full((1, max(cols, room // P)), -1, np.int32)
    wide[0, :cols] = table
    w = torch.full((1, wide.shape[1] * P), 9.0, device=dev)
    ds.key_weights(L.dev_of(q[None].astype(np.float32), dev).to(L.BF16), L.dev_of(lse[None], dev), k, L.dev_of(wide, dev),
                   torch.tensor([n], dtype=torch.int32, device=dev), w, decay=0.0, scale=scale, k_scale=ks)
    torch.cuda.synchronize()
    assert ds.device_error() == 0
    ref, tol = _bound(z, lse)
    got = w[0, :n].double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])
    assert (w[0, n:] == 9).all()
