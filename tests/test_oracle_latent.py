"""Pins the latent-attention oracle: against brute force over the definition, against the
E4M3 grid, and its gradients against central differences."""
import numpy as np
import pytest

import oracle
from oracle import e4m3, latent


def _rand(rng, *shape):
    return oracle.round_bf16(rng.standard_normal(shape).astype(np.float32))


@pytest.mark.parametrize("width", [256, 512])
def test_cache_rows_hold_the_nearest_codes(width):
    rng = np.random.default_rng(1)
    x = _rand(rng, 9, width + 64) * np.exp2(rng.integers(-20, 20, (9, 1))).astype(np.float32)
    x[3, :128] = 0
    rows = latent.cache_rows(x, True)
    assert rows.shape == (9, latent.row_bytes(width, True)) and rows.shape[1] % 16 == 0
    v = latent.cache_values(rows, width)
    assert np.array_equal(v[:, width:], x[:, width:].astype(np.float64))
    grid = np.concatenate([e4m3.finite_values(), -e4m3.finite_values()])
    for r in range(9):
        for g in range(width // 128):
            t = x[r, 128 * g:128 * (g + 1)].astype(np.float64)
            top = np.abs(t).max()
            s = 1.0 if top == 0 else next(2.0 ** k for k in range(-126, 120) if top / 2.0 ** k <= 448)
            near = np.abs(t[:, None] / s - grid[None, :]).min(1) * s
            assert np.allclose(np.abs(v[r, 128 * g:128 * (g + 1)] - t), near, rtol=1e-12, atol=0)
    # a value read back is a bf16 number
    assert np.array_equal(oracle.round_bf16(v.astype(np.float32)).astype(np.float64), v)
    b = latent.cache_rows(x, False)
    assert np.array_equal(latent.cache_values(b, width), x.astype(np.float64))


def test_attend_is_the_definition():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((4, 6)), rng.standard_normal((5, 6)), rng.standard_normal((5, 3))
    out, lse, p, mag = latent.attend(q, k, v, 0.7, np.array([5, 3, 1, 0]))
    for i, n in enumerate((5, 3, 1, 0)):
        w = [np.exp(0.7 * sum(q[i, d] * k[j, d] for d in range(6))) for j in range(n)]
        if n == 0:
            assert np.all(out[i] == 0) and lse[i] == -np.inf and np.all(p[i] == 0)
            continue
        assert np.isclose(lse[i], np.log(sum(w)))
        for c in range(3):
            assert np.isclose(out[i, c], sum(w[j] * v[j, c] for j in range(n)) / sum(w))
            assert np.isclose(mag[i, c], sum(w[j] * abs(v[j, c]) for j in range(n)) / sum(w))


def test_absorbed_is_expanded_with_the_projections_folded_in():
    """scores (W c) . q = c . (W^T q) and values U c: the two forms agree."""
    rng = np.random.default_rng(3)
    H, R, D, n = 3, 256, 64, 11
    c, kr = rng.standard_normal((n, R)), rng.standard_normal((n, 64))
    wk, wv = rng.standard_normal((H, D, R)) / 16, rng.standard_normal((H, D, R)) / 16
    q = rng.standard_normal((2, H, D + 64))
    kv = np.concatenate([np.einsum("nr,hdr->nhd", c, wk), np.einsum("nr,hdr->nhd", c, wv)], 2)
    ref, lse, _ = latent.expanded(q, kv, kr, [0, 2], [0, n], 0.1, True)
    qa = np.concatenate([np.einsum("thd,hdr->thr", q[:, :, :D], wk), q[:, :, D:]], 2)
    out, lse2, _ = latent.absorbed(qa[None], [np.concatenate([c, kr], 1)], R, 0.1)
    assert np.allclose(np.einsum("thr,hdr->thd", out[0], wv), ref)
    assert np.allclose(lse2[0].T, lse)


def test_seen_keys():
    assert latent.seen_keys(3, 5, True).tolist() == [3, 4, 5]
    assert latent.seen_keys(5, 3, True).tolist() == [0, 0, 1, 2, 3]
    assert latent.seen_keys(2, 3, False).tolist() == [3, 3]


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_against_differences(causal):
    rng = np.random.default_rng(4)
    H, D = 2, 64
    cu_q, cu_k = [0, 3, 3, 7], [0, 2, 5, 9]
    args = [rng.standard_normal((7, H, D + 64)), rng.standard_normal((9, H, 2 * D)), rng.standard_normal((9, 64))]
    g = rng.standard_normal((7, H, D))
    (grads, bounds) = latent.expanded_backward(*args, cu_q, cu_k, 0.1, causal, g)
    f = lambda a: (latent.expanded(*a, cu_q, cu_k, 0.1, causal)[0] * g).sum()
    for i in range(3):
        assert np.all(bounds[i] >= np.abs(grads[i]) * 0.999 - 1e-12)
        for _ in range(6):
            d = rng.standard_normal(args[i].shape)
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
            assert np.isclose((f(up) - f(down)) / 2e-5, (grads[i] * d).sum(), rtol=1e-6, atol=1e-6)
