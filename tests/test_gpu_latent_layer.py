"""The latent-attention driver: chunked prefill, decoding and a training step, against the
float64 oracle on the same weights (needs an MI355X).

The driver rounds the expansion (or the folded query and the latent output) to bf16 beside
what the kernels round, so results are compared by norm: three or four bf16 roundings of
2^-9 rms each, the scores' one amplified by their spread of about two: below 1.5e-2.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import latent

pytestmark = pytest.mark.gpu
H, R, D, P = 4, 512, 128, 16


def rand(rng, *shape, s=1.0):
    return oracle.round_bf16((s * rng.standard_normal(shape)).astype(np.float32))


def bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda", torch.bfloat16)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def close(got, ref, tol=1.5e-2):
    return np.linalg.norm(got - ref) <= tol * np.linalg.norm(ref)


@pytest.fixture
def setup():
    import deepseekmoe_routing_fp8_amd as lib
    rng = np.random.default_rng(21)
    wk, wv = rand(rng, H, R, D, s=R ** -0.5), rand(rng, H, R, D, s=R ** -0.5)
    return lib, rng, wk, wv


def reference(rows, q, wk, wv, upto):
    """Attention of query token i over rows[:upto[i]] in float64."""
    kv = np.concatenate([np.einsum("nr,hrd->nhd", rows[:, :R], wk), np.einsum("nr,hrd->nhd", rows[:, :R], wv)], 2)
    out = np.zeros((len(q), H, D))
    for h in range(H):
        k = np.concatenate([kv[:, h, :D], rows[:, R:]], 1)
        out[:, h] = latent.attend(q[:, h].astype(np.float64), k, kv[:, h, D:], (D + 64) ** -0.5, np.array(upto))[0]
    return out


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_chunked_prefill_then_decode(setup, kind):
    lib, rng, wk, wv = setup
    a = lib.LatentAttention(H, bf(wk), bf(wv), cache=kind, n_pages=24, page_size=P, max_seqs=3)
    lens, rows = [0, 0], [np.zeros((0, R + 64)), np.zeros((0, R + 64))]

    def seen(x):   # what the cache holds of new rows
        return latent.cache_values(latent.cache_rows(x, kind == "fp8"), R)
    for counts in ([37, 5], [20, 64]):      # two chunks; the second attends to the first too
        x, q = rand(rng, sum(counts), R + 64), rand(rng, sum(counts), H, D + 64)
        out = host(a.prefill([0, 2], counts, bf(x), bf(q)))
        at = 0
        for i, n in enumerate(counts):
            rows[i] = np.concatenate([rows[i], seen(x[at:at + n])])
            ref = reference(rows[i], q[at:at + n], wk, wv, [lens[i] + 1 + j for j in range(n)])
            assert close(out[at:at + n], ref)
            lens[i] += n
            at += n
    for Sq in (1, 1, 3):                    # decoding, then drafted tokens
        x, q = rand(rng, 2, Sq, R + 64), rand(rng, 2, Sq, H, D + 64)
        out = host(a.decode([0, 2], bf(x), bf(q)))
        for i in range(2):
            rows[i] = np.concatenate([rows[i], seen(x[i])])
            ref = reference(rows[i], q[i], wk, wv, [lens[i] + 1 + j for j in range(Sq)])
            assert close(out[i], ref)
            lens[i] += Sq
    assert [a.lens[0], a.lens[2]] == lens
    used = 24 - len(a.free)
    a.release(0)
    assert len(a.free) == 24 - used + -(-lens[0] // P)
    with pytest.raises(RuntimeError):
        a.prefill([1], [24 * P], bf(rand(rng, 24 * P, R + 64)), bf(rand(rng, 24 * P, H, D + 64)))
    before = (list(a.lens), [list(p) for p in a.pages], list(a.free))
    for seqs, counts in (([1, 1], [1, 1]), ([3], [2]), ([1], [3]), ([0, 1], [2])):   # twice, out of range, too few rows
        with pytest.raises(ValueError):
            a.prefill(seqs, counts, bf(rand(rng, 2, R + 64)), bf(rand(rng, 2, H, D + 64)))
    assert before == (a.lens, a.pages, a.free)


def test_training_step(setup):
    lib, rng, wk, wv = setup
    a = lib.LatentAttention(H, bf(wk), bf(wv))
    counts = [30, 1, 17]
    T, cu = sum(counts), np.concatenate([[0], np.cumsum(counts)])
    x, q, g = rand(rng, T, R + 64), rand(rng, T, H, D + 64), rand(rng, T, H, D)
    out = host(a.attend_train(counts, bf(x), bf(q)))
    dq, drows, dw = (host(t) for t in a.backward(bf(g)))
    kv = np.concatenate([np.einsum("nr,hrd->nhd", x[:, :R], wk), np.einsum("nr,hrd->nhd", x[:, :R], wv)], 2)
    ref, _, _ = latent.expanded(q, kv, x[:, R:], cu, cu, (D + 64) ** -0.5, True)
    assert close(out, ref)
    (rq, rkv, rr), _ = latent.expanded_backward(q, kv, x[:, R:], cu, cu, (D + 64) ** -0.5, True, g)
    w = np.concatenate([wk, wv], 2)
    assert close(dq, rq, 3e-2)
    assert close(drows, np.concatenate([np.einsum("nhd,hrd->nr", rkv, w), rr], 1), 3e-2)
    assert close(dw, np.einsum("nr,nhd->rhd", x[:, :R].astype(np.float64), rkv), 3e-2)
