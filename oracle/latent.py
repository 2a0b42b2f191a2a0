"""Oracle of the latent attention and its cache (float64 unless a step fixes float32). Test
infrastructure only: see the package docstring for who may call this.

Passages followed: the MLA pseudocode of the 2kiu.com digest and the MLA snippet of the
lpnh.cn guide (keys and values from one cached latent vector a token, a rotary key shared
by the heads); the cache codes follow the power-of-two 1x128 quantiser of ``moe.py``.

Beside each result come the sums of absolute terms that the rounding bounds of the tests
are built on: a kernel rounds each softmax weight (and each score gradient) to bf16, an
error of at most 2^-8 of every term.
"""
from __future__ import annotations

import numpy as np

from .backward import round_bf16
from .e4m3 import decode
from .moe import quantize_1x128_pow2

ROPE = 64


def row_bytes(latent: int, fp8: bool) -> int:
    """Bytes of a cache row: codes, rotary key in bf16, a float scale per 128 codes, padded
    to 16; or all in bf16."""
    return -(-(latent + 2 * ROPE + 4 * (latent // 128)) // 16) * 16 if fp8 else 2 * (latent + ROPE)


def bf16_bits(v: np.ndarray) -> np.ndarray:
    return (round_bf16(v.astype(np.float32)).view(np.uint32) >> 16).astype(np.uint16)


def cache_rows(x: np.ndarray, fp8: bool):
    """Cache rows of x [n, latent + ROPE] float32: bytes [n, row_bytes] (pad bytes zero)
    when fp8, else bf16 bits [n, latent + ROPE]."""
    n, latent = x.shape[0], x.shape[1] - ROPE
    if not fp8:
        return bf16_bits(x)
    codes, scales = quantize_1x128_pow2(np.ascontiguousarray(x[:, :latent], np.float32))
    rows = np.zeros((n, row_bytes(latent, True)), np.uint8)
    rows[:, :latent] = codes
    rows[:, latent:latent + 2 * ROPE] = bf16_bits(x[:, latent:]).view(np.uint8).reshape(n, 2 * ROPE)
    rows[:, latent + 2 * ROPE:latent + 2 * ROPE + 4 * (latent // 128)] = \
        np.ascontiguousarray(scales, np.float32).view(np.uint8).reshape(n, 4 * (latent // 128))
    return rows


def cache_values(rows: np.ndarray, latent: int) -> np.ndarray:
    """float64 values [n, latent + ROPE] of cache rows."""
    if rows.dtype == np.uint16:
        return (rows.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    n = rows.shape[0]
    scales = np.ascontiguousarray(rows[:, latent + 128:latent + 128 + 4 * (latent // 128)]).view(np.float32)
    c = decode(rows[:, :latent]).astype(np.float64) * np.repeat(scales.astype(np.float64), 128, axis=1)
    rope = np.ascontiguousarray(rows[:, latent:latent + 128]).view(np.uint16)
    return np.concatenate([c.reshape(n, latent), cache_values(rope, 0)], 1)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, seen: np.ndarray):
    """Softmax attention of query rows q over keys k and values v; row i sees the first
    seen[i] keys. -> (out, lse, P, sum of P |v|); a row that sees nothing is zero, lse -inf."""
    s = scale * (q @ k.T)
    s[np.arange(k.shape[0])[None, :] >= np.asarray(seen)[:, None]] = -np.inf
    top = s.max(1, initial=-np.inf)
    base = np.where(np.isinf(top), 0.0, top)
    e = np.exp(s - base[:, None])
    l = e.sum(1)
    p = e / np.where(l == 0, 1.0, l)[:, None]
    with np.errstate(divide="ignore"):
        lse = base + np.log(l)
    return p @ v, lse, p, p @ np.abs(v)


def absorbed(q: np.ndarray, contexts, latent: int, scale: float):
    """q [B, Sq, H, latent + ROPE], contexts: values [len, latent + ROPE] of each sequence
    -> (out [B, Sq, H, latent], lse [B, Sq, H], sums of absolute terms like out)."""
    B, S, H, _ = q.shape
    out, mag = np.zeros((B, S, H, latent)), np.zeros((B, S, H, latent))
    lse = np.full((B, S, H), -np.inf)
    for b, ctx in enumerate(contexts):
        for s in range(S):
            seen = max(0, len(ctx) - (S - 1 - s))
            out[b, s], lse[b, s], _, mag[b, s] = attend(q[b, s].astype(np.float64), ctx, ctx[:, :latent], scale,
                                                        np.full(H, seen))
    return out, lse, mag


def seen_keys(nq: int, nk: int, causal: bool) -> np.ndarray:
    """Keys that each of nq queries sees: the last query sees all of them."""
    if not causal:
        return np.full(nq, nk)
    return np.clip(np.arange(nq) + nk - nq + 1, 0, nk)


def expanded(q, kv, k_rope, cu_q, cu_k, scale: float, causal: bool):
    """q [Tq, H, D + ROPE], kv [Tk, H, 2 D], k_rope [Tk, ROPE] -> (out [Tq, H, D],
    lse [H, Tq], sums of absolute terms like out)."""
    H, D = q.shape[1], kv.shape[2] // 2
    out, mag = np.zeros((q.shape[0], H, D)), np.zeros((q.shape[0], H, D))
    lse = np.full((H, q.shape[0]), -np.inf)
    for b in range(len(cu_q) - 1):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        seen = seen_keys(rq.stop - rq.start, rk.stop - rk.start, causal)
        for h in range(H):
            k = np.concatenate([kv[rk, h, :D], k_rope[rk]], 1).astype(np.float64)
            out[rq, h], lse[h, rq], _, mag[rq, h] = attend(q[rq, h].astype(np.float64), k,
                                                           kv[rk, h, D:].astype(np.float64), scale, seen)
    return out, lse, mag


def expanded_backward(q, kv, k_rope, cu_q, cu_k, scale: float, causal: bool, dout):
    """-> ((dq, dkv, dk_rope), bounds): the gradients of sum(out * dout), and for each of
    them the rounding bound in units of 2^-8: the sums of absolute terms (dS rounded, P
    rounded) plus the effect of D = rowsum(dout * out) formed from a rounded out, whose
    error is at most sum |dout| (|out| + sum P |v|)."""
    H, D = q.shape[1], kv.shape[2] // 2
    grads = [np.zeros(np.shape(t), np.float64) for t in (q, kv, k_rope)]
    bounds = [np.zeros(np.shape(t), np.float64) for t in (q, kv, k_rope)]
    for b in range(len(cu_q) - 1):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        seen = seen_keys(rq.stop - rq.start, rk.stop - rk.start, causal)
        for h in range(H):
            qh, g = q[rq, h].astype(np.float64), dout[rq, h].astype(np.float64)
            k = np.concatenate([kv[rk, h, :D], k_rope[rk]], 1).astype(np.float64)
            v = kv[rk, h, D:].astype(np.float64)
            o, _, p, mag = attend(qh, k, v, scale, seen)
            ds = p * (g @ v.T - (g * o).sum(1)[:, None]) * scale
            # an error of D shifts ds by p times it
            dd = np.abs(ds) + scale * p * (np.abs(g) * (np.abs(o) + mag)).sum(1)[:, None]
            grads[0][rq, h], bounds[0][rq, h] = ds @ k, dd @ np.abs(k)
            dk, bk = ds.T @ qh, dd.T @ np.abs(qh)
            grads[1][rk, h] = np.concatenate([dk[:, :D], p.T @ g], 1)
            bounds[1][rk, h] = np.concatenate([bk[:, :D], p.T @ np.abs(g)], 1)
            grads[2][rk] += dk[:, D:]
            bounds[2][rk] += bk[:, D:]
    return tuple(grads), tuple(bounds)
