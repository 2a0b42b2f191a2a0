"""Latent attention and its cache against the float64 oracle (needs an MI355X).

Cache bytes and read-back values must match exactly. Attention outputs are compared
element by element with bounds from the arithmetic, derived before any run:
  * a softmax weight is rounded to bf16 before its product, a relative error of at most
    u = 2^-8 (half a unit in the last of 8 significant bits), so out is off by at most u * sum P |v|; the output's own rounding adds
    u * |out|; FP32 scores, exponentials and sums (at most 576 products a score, scores
    below 64) stay under 2^-12 of the same sums;
  * lse sums the unrounded weights: 2^-18 * (1 + |lse|), from FP32 scores;
  * a gradient's terms carry one bf16 rounding (P or dS) and the rounding of D through the
    rounded out; the oracle returns their sum, used with u, plus u * |gradient| for the
    output's rounding and 2^-11 of the sum for FP32 (scores, lse and dO V^T).
"""
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import latent

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
DEV = "cuda"


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def lib():
    import deepseekmoe_routing_fp8_amd as m
    assert torch.cuda.is_available()
    return m


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def bf(a):
    return dev(a.astype(np.float32), torch.bfloat16)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def rand(rng, *shape, s=1.0):
    return oracle.round_bf16((s * rng.standard_normal(shape)).astype(np.float32))


def assert_within(got, ref, bound, what):
    assert np.all(np.isfinite(got)), what
    worst = np.max(np.abs(got - ref) / np.maximum(bound, 1e-30)) if got.size else 0.0
    say(f"  {what}: at most {worst:.3f} of the bound")
    assert worst <= 1.0, what


def out_bound(ref, mag, bf16=True):
    return (U + 2.0 ** -12) * mag + (U * np.abs(ref) if bf16 else 0) + 1e-30


def assert_lse(got, ref):
    empty = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got[~empty] - ref[~empty]) <= 2.0 ** -18 * (1 + np.abs(ref[~empty])))


# ---------------------------------------------------------------------------------------
# cache
# ---------------------------------------------------------------------------------------
def latents(rng, n, width):
    x = rng.standard_normal((n, width + 64)).astype(np.float32) * np.exp2(rng.integers(-3, 4, (n, 1))).astype(np.float32)
    return x


def edge_rows(width):
    """All-zero tiles, one outlier, subnormals, the largest values, ties of the E4M3 grid."""
    x = np.zeros((6, width + 64), np.float32)
    x[1, 3] = 1e4
    x[1, 4:128] = 1e-3
    x[2, :width] = np.linspace(-1e-38, 1e-38, width)
    x[3, :width] = np.linspace(-3e38, 3e38, width)
    ties = (oracle.finite_values()[:-1] + oracle.finite_values()[1:]) / 2
    x[4, :126] = ties[:126]
    x[4, 126] = 448.0
    x[5, ::2] = -0.0
    return x


@pytest.mark.parametrize("width", [512, 256])
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
def test_cache_write_and_read_back(lib, width, kind, xt):
    rng = np.random.default_rng(width + len(kind))
    fp8 = kind == "fp8"
    x = np.concatenate([latents(rng, 77, width), edge_rows(width)])
    if xt == torch.bfloat16:
        x = oracle.round_bf16(x)
    n, page, n_pages = len(x), 5, 40
    cfg = lib.make_latent_config(4, latent=width, cache=kind)
    # rows of a wider tensor
    wide = torch.full((n, width + 64 + 40), 7.0, dtype=xt, device=DEV)
    wide[:, 16:16 + width + 64] = dev(x, xt)
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    slots[[5, 11]] = [-1, n_pages * page]   # skipped
    rowb = lib.moe_latent_cache_row_bytes(cfg)
    if fp8:
        cache = torch.full((n_pages, page, rowb), 0xA5, dtype=torch.uint8, device=DEV)
    else:
        cache = torch.full((n_pages, page, width + 64), -3.0, dtype=torch.bfloat16, device=DEV)
    before = cache.clone()
    lib.moe_latent_cache_write(cfg, wide[:, 16:16 + width + 64], dev(slots), cache)
    ref = latent.cache_rows(x, fp8)
    kept = (slots >= 0) & (slots < n_pages * page)
    got = cache.reshape(n_pages * page, -1).cpu()
    got = got.numpy() if fp8 else got.view(torch.int16).numpy().view(np.uint16)
    used = width + 128 + 4 * (width // 128) if fp8 else width + 64
    assert np.array_equal(got[slots[kept]][:, :used], ref[kept][:, :used])
    others = np.ones(n_pages * page, bool)
    others[slots[kept]] = False
    assert torch.equal(cache.reshape(n_pages * page, -1)[dev(others)], before.reshape(n_pages * page, -1)[dev(others)])

    # three sequences over shuffled pages, one empty, from given starts
    table = rng.permutation(n_pages)[:30].astype(np.int32).reshape(3, 10)
    table[2, 4] = n_pages        # no such page: zero rows
    table[2, 5] = -1
    starts, counts = np.array([3, 0, 1], np.int32), [31, 0, 49]
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n_out = int(cu[-1]) + 4      # rows outside every sequence: zero
    out = torch.full((n_out, width + 64), 9.0, dtype=torch.bfloat16, device=DEV)
    lib.moe_latent_cache_read(cfg, cache, dev(table), dev(cu), starts=dev(starts), out=out)
    values = latent.cache_values(got, width)
    want = np.zeros((n_out, width + 64))
    for b in range(3):
        for i in range(counts[b]):
            p = starts[b] + i
            pg = table[b, p // page]
            if 0 <= pg < n_pages:
                want[cu[b] + i] = values[pg * page + p % page]
    with np.errstate(over="ignore", invalid="ignore"):
        want = oracle.round_bf16(want.astype(np.float32))
    written = np.zeros(n_pages * page, bool)
    written[slots[kept]] = True
    ok = np.ones(n_out, bool)    # rows that were written (the others hold no cache row), or are zero
    for b in range(3):
        for i in range(counts[b]):
            p = starts[b] + i
            pg = table[b, p // page]
            ok[cu[b] + i] = not 0 <= pg < n_pages or written[pg * page + p % page]
    assert np.array_equal(host(out)[ok], want.astype(np.float64)[ok])
    assert ok.sum() > 20
    again = lib.moe_latent_cache_read(cfg, cache, dev(table), dev(cu), starts=dev(starts), n_out=n_out)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_cache_offsets_past_32_bits(lib):
    """A cache of more than 4 GiB: rows at its end."""
    rng = np.random.default_rng(9)
    cfg = lib.make_latent_config(16)
    page, n_pages = 64, 120_000                  # 5.0 GB of rows
    cache = torch.empty((n_pages, page, 656), dtype=torch.uint8, device=DEV)
    x = rand(rng, 100, 576)
    first = n_pages * page - 100
    slots = np.arange(first, first + 100).astype(np.int32)
    lib.moe_latent_cache_write(cfg, bf(x), dev(slots), cache)
    table = dev(np.array([[n_pages - 2, n_pages - 1]], np.int32))
    got = lib.moe_latent_cache_read(cfg, cache, table, dev(np.array([0, 100], np.int32)),
                                    starts=dev(np.array([28], np.int32)), n_out=100)
    ref = latent.cache_values(latent.cache_rows(x, True), 512)
    assert np.array_equal(host(got), ref)
    q = rand(rng, 1, 1, 16, 576)
    cache[n_pages - 2, :28] = 0                  # rows before them: zeros
    cache[n_pages - 2, :28, 640:656] = torch.tensor([1.0] * 4).view(torch.uint8).to(DEV)
    out, lse = lib.moe_latent_attn_absorbed(cfg, bf(q), cache, table, dev(np.array([128], np.int32)), 0.07)
    ctx = np.concatenate([np.zeros((28, 576)), ref])
    r, rl, mag = latent.absorbed(q, [ctx], 512, 0.07)
    assert_within(host(out), r, out_bound(r, mag), "out")
    assert_lse(host(lse), rl)


# ---------------------------------------------------------------------------------------
# absorbed form
# ---------------------------------------------------------------------------------------
def paged(rng, lib, cfg, kind, width, lens, page, poison=True):
    """A cache that holds the sequences over shuffled pages; every other row is NaN."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 2
    order = rng.permutation(n_pages)[:sum(need)].astype(np.int32)
    table = np.full((len(lens), max(max(need), 1)), n_pages - 1, np.int32)
    if kind == "fp8":
        rows = np.full((n_pages * page, latent.row_bytes(width, True)), 0x7F if poison else 0, np.uint8)
        if poison:
            rows[:, width:] = 0xFF
    else:
        rows = np.full((n_pages * page, width + 64), 0x7FC0 if poison else 0, np.uint16)
    ctx, at = [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        x = rand(rng, n, width + 64)
        r = latent.cache_rows(x, kind == "fp8")
        pos = np.arange(n)
        rows[table[b, pos // page] * page + pos % page] = r
        ctx.append(latent.cache_values(r, width) if n else np.zeros((0, width + 64)))
    t = torch.from_numpy(rows if kind == "fp8" else rows.view(np.int16)).to(DEV)
    if kind != "fp8":
        t = t.view(torch.bfloat16)
    return t.reshape(n_pages, page, -1), dev(table), ctx


LENS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 200]
ABSORBED = [(1, 1, 512, "fp8", 64, [1]), (1, 1, 512, "bf16", 64, [300]), (5, 1, 512, "fp8", 1, LENS),
            (16, 1, 512, "fp8", 64, LENS), (16, 1, 512, "bf16", 7, LENS), (16, 2, 512, "fp8", 64, LENS),
            (17, 1, 512, "bf16", 64, LENS), (16, 3, 512, "bf16", 48, LENS), (16, 4, 512, "fp8", 48, LENS),
            (33, 1, 512, "fp8", 16, LENS), (128, 1, 512, "fp8", 64, LENS), (128, 1, 512, "bf16", 64, LENS),
            (130, 1, 512, "fp8", 64, [70, 0, 129]), (128, 3, 512, "bf16", 48, [2, 130, 65]),
            (16, 64, 512, "fp8", 64, [10, 100]), (8, 1, 256, "fp8", 64, LENS), (24, 1, 256, "bf16", 64, LENS),
            (64, 1, 256, "fp8", 5, LENS), (100, 2, 256, "bf16", 64, LENS), (16, 1, 512, "fp8", 64, [20000]),
            (8, 1, 512, "bf16", 64, [9000, 1, 0, 5000]), (128, 1, 512, "fp8", 64, [5000, 33, 1200]),
            (64, 1, 512, "fp8", 64, [3000, 7]), (16, 1, 512, "fp8", 64, [0, 0, 0])]


@pytest.mark.parametrize("H,Sq,width,kind,page,lens", ABSORBED)
def test_absorbed(lib, H, Sq, width, kind, page, lens):
    say(f"absorbed H={H} Sq={Sq} latent={width} {kind} page={page} lens={lens[:4]}..")
    rng = np.random.default_rng(H * 1000 + Sq + page)
    cfg = lib.make_latent_config(H, latent=width, cache=kind)
    cache, table, ctx = paged(rng, lib, cfg, kind, width, lens, page)
    q = rand(rng, len(lens), Sq, H, width + 64) * np.exp2(rng.integers(0, 2, (1, 1, H, 1))).astype(np.float32)
    args = (cfg, bf(q), cache, table, dev(np.array(lens, np.int32)), 0.07)
    out, lse = lib.moe_latent_attn_absorbed(*args)
    ref, rl, mag = latent.absorbed(q, ctx, width, np.float32(0.07))
    assert_within(host(out), ref, out_bound(ref, mag), "out")
    assert_lse(host(lse), rl)
    out32, lse32 = lib.moe_latent_attn_absorbed(*args, out_dtype=torch.float32)
    assert torch.equal(lse32, lse) and torch.equal(out32.to(torch.bfloat16), out)


@pytest.mark.parametrize("H,Sq,width,kind,B", [(16, 1, 512, "fp8", 64), (16, 1, 512, "fp8", 65), (8, 2, 256, "bf16", 200),
                                               (128, 1, 512, "bf16", 130), (4, 1, 512, "fp8", 513),
                                               (16, 1, 256, "fp8", 1300)])
def test_absorbed_many_sequences(lib, H, Sq, width, kind, B):
    """More sequences than lanes, than threads of a workgroup and than workgroups; lengths
    from none up, with runs of empty sequences and some long ones."""
    say(f"absorbed H={H} Sq={Sq} latent={width} {kind} B={B}")
    rng = np.random.default_rng(B)
    cfg = lib.make_latent_config(H, latent=width, cache=kind)
    lens = rng.integers(0, 100, B)
    lens[rng.random(B) < 0.3] = 0
    lens[B // 3: B // 3 + 12] = 0
    lens[[0, 7, B - 1]] = 0, 900, 400
    cache, table, ctx = paged(rng, lib, cfg, kind, width, [int(n) for n in lens], 16)
    q = rand(rng, B, Sq, H, width + 64)
    out, lse = lib.moe_latent_attn_absorbed(cfg, bf(q), cache, table, dev(lens.astype(np.int32)), 0.07)
    ref, rl, mag = latent.absorbed(q, ctx, width, np.float32(0.07))
    assert_within(host(out), ref, out_bound(ref, mag), "out")
    assert_lse(host(lse), rl)


def test_absorbed_lengths_and_pages_out_of_range(lib):
    """Lengths past the table are clamped, negative ones are empty; a page outside the pool
    reads as zero rows."""
    rng = np.random.default_rng(3)
    cfg = lib.make_latent_config(16)
    lens = [128, 128, 100, 128]
    cache, table, ctx = paged(rng, lib, cfg, "fp8", 512, lens, 64)
    table[3, 0] = 1 << 20
    ctx[3] = np.concatenate([np.zeros((64, 576)), ctx[3][64:]])
    q = rand(rng, 4, 1, 16, 576)
    out, lse = lib.moe_latent_attn_absorbed(cfg, bf(q), cache, table,
                                            dev(np.array([1000, -7, 100, 128], np.int32)), 0.07)
    ctx[1] = ctx[1][:0]
    ref, rl, mag = latent.absorbed(q, ctx, 512, np.float32(0.07))
    assert_within(host(out), ref, out_bound(ref, mag), "out")
    assert_lse(host(lse), rl)


def test_absorbed_large_scores_stay_finite(lib):
    """Scores of thousands, and rows whose scores differ by more than FP32's exponent range."""
    rng = np.random.default_rng(5)
    cfg = lib.make_latent_config(16, cache="bf16")
    cache, table, ctx = paged(rng, lib, cfg, "bf16", 512, [150], 64)
    q = rand(rng, 1, 1, 16, 576, s=60.0)
    out, lse = lib.moe_latent_attn_absorbed(cfg, bf(q), cache, table, dev(np.array([150], np.int32)), 1.0)
    ref, rl, mag = latent.absorbed(q, ctx, 512, 1.0)
    assert np.abs(rl).max() > 2000
    # scores of some thousands carry FP32 errors of 2^-24 * sum |q k|, below 2^-8 here
    e = np.expm1(2.0 ** -24 * 8 * np.abs(q[0, 0].astype(np.float64)) @ np.abs(ctx[0]).T).max()
    assert_within(host(out), ref, out_bound(ref, mag) + 2 * e * mag, "out")


# ---------------------------------------------------------------------------------------
# expanded form and its gradients
# ---------------------------------------------------------------------------------------
def packed(rng, H, D, nq, nk):
    cu = lambda v: np.concatenate([[0], np.cumsum(v)]).astype(np.int32)
    Tq, Tk = sum(nq), sum(nk)
    return (rand(rng, Tq, H, D + 64), rand(rng, Tk, H, 2 * D), rand(rng, Tk, 64), cu(nq), cu(nk), rand(rng, Tq, H, D))


EXPANDED = [(1, 128, [1], [1], True), (3, 128, [64], [64], True), (2, 128, [65, 1, 130], [65, 1, 130], True),
            (5, 128, [0, 127, 0, 33], [0, 127, 0, 33], True), (2, 128, [128, 20], [129, 300], True),
            (2, 128, [40, 7], [10, 0], True), (2, 128, [33, 5], [70, 0], False), (1, 128, [0, 3], [50, 3], True),
            (8, 128, [300], [300], True), (3, 64, [65, 1, 200], [65, 1, 200], True),
            (2, 64, [31, 0, 100], [64, 9, 191], False), (9, 64, [129], [257], True),
            (1, 128, [700], [700], True), (1, 64, [520], [1100], False),
            (128, 128, [500, 260], [500, 300], True), (96, 64, [1100, 3], [300, 70], False)]


@pytest.mark.parametrize("H,D,nq,nk,causal", EXPANDED)
def test_expanded_and_its_gradients(lib, H, D, nq, nk, causal):
    say(f"expanded H={H} D={D} queries={nq} keys={nk} causal={causal}")
    rng = np.random.default_rng(H * 100 + D + sum(nq))
    q, kv, kr, cu_q, cu_k, g = packed(rng, H, D, nq, nk)
    cfg = lib.make_latent_config(H, nope=D, v_dim=D)
    scale = np.float32(0.11)
    args = (cfg, bf(q), bf(kv), bf(kr), dev(cu_q), dev(cu_k), float(scale))
    out, lse = lib.moe_latent_attn_expanded(*args, causal=causal)
    ref, rl, mag = latent.expanded(q, kv, kr, cu_q, cu_k, scale, causal)
    assert_within(host(out), ref, out_bound(ref, mag), "out")
    assert_lse(host(lse), rl)
    out32, lse32 = lib.moe_latent_attn_expanded(*args, causal=causal, out_dtype=torch.float32)
    assert torch.equal(lse32, lse) and torch.equal(out32.to(torch.bfloat16), out)

    grads, bounds = latent.expanded_backward(q, kv, kr, cu_q, cu_k, scale, causal, g)
    got = lib.moe_latent_attn_expanded_backward(*args, out, lse, bf(g), causal=causal)
    got32 = lib.moe_latent_attn_expanded_backward(*args, out, lse, bf(g), causal=causal, grad_dtype=torch.float32)
    for name, a, a32, r, b in zip(("dq", "dkv", "dk_rope"), got, got32, grads, bounds):
        assert_within(host(a), r, (U + 2.0 ** -11) * b + U * np.abs(r), name)
        assert torch.equal(a32.to(torch.bfloat16), a)
    for a, c in zip(got, lib.moe_latent_attn_expanded_backward(*args, out, lse, bf(g), causal=causal)):
        assert torch.equal(a.view(torch.int16), c.view(torch.int16))   # no order-dependent sums


def test_gradients_against_differences(lib):
    """The kernels' gradients along random directions against central differences of the
    float64 forward: each direction's error is bounded by the gradients' bounds."""
    rng = np.random.default_rng(12)
    q, kv, kr, cu_q, cu_k, g = packed(rng, 2, 128, [20, 9], [25, 9])
    cfg = lib.make_latent_config(2)
    args = (cfg, bf(q), bf(kv), bf(kr), dev(cu_q), dev(cu_k), 0.1)
    out, lse = lib.moe_latent_attn_expanded(*args)
    got = lib.moe_latent_attn_expanded_backward(*args, out, lse, bf(g), grad_dtype=torch.float32)
    _, bounds = latent.expanded_backward(q, kv, kr, cu_q, cu_k, 0.1, True, g)
    f = lambda a: (latent.expanded(*a, cu_q, cu_k, np.float32(0.1), True)[0] * g).sum()
    base = [q.astype(np.float64), kv.astype(np.float64), kr.astype(np.float64)]
    for i in range(3):
        for _ in range(4):
            d = rng.standard_normal(base[i].shape)
            up, down = list(base), list(base)
            up[i], down[i] = base[i] + 1e-4 * d, base[i] - 1e-4 * d
            slope = (f(up) - f(down)) / 2e-4
            assert abs(slope - (host(got[i]) * d).sum()) <= ((U + 2.0 ** -11) * bounds[i] * np.abs(d)).sum() + 1e-4


def test_another_sequences_nan_stays_there(lib):
    """A sequence's NaN and infinite keys and values reach no other sequence, in either
    direction, nor do the rows past the last sequence."""
    rng = np.random.default_rng(13)
    q, kv, kr, cu_q, cu_k, g = packed(rng, 2, 128, [50, 40, 70], [50, 40, 70])
    cfg = lib.make_latent_config(2)
    pad = lambda a: np.concatenate([a, np.full((9,) + a.shape[1:], np.nan, np.float32)])
    q2, kv2, kr2, g2 = pad(q), pad(kv), pad(kr), pad(g)
    kv2[50:90], kr2[55] = np.inf, np.nan
    clean = (cfg, bf(q), bf(kv), bf(kr), dev(cu_q), dev(cu_k), 0.1)
    dirty = (cfg, bf(q2), bf(kv2), bf(kr2), dev(cu_q), dev(cu_k), 0.1)
    out, lse = lib.moe_latent_attn_expanded(*clean)
    keep = np.r_[0:50, 90:160]
    o2 = torch.full((169, 2, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    l2 = torch.full((2, 169), 6.0, device=DEV)
    lib.moe_latent_attn_expanded(*dirty, out=o2, lse=l2)
    assert torch.equal(o2[keep], out[keep]) and torch.equal(l2[:, keep], lse[:, keep])
    assert (o2[160:] == 5).all() and (l2[:, 160:] == 6).all()    # rows of no sequence
    a = lib.moe_latent_attn_expanded_backward(*clean, out, lse, bf(g))
    b = lib.moe_latent_attn_expanded_backward(*dirty, o2, l2, bf(g2))
    for x, y in zip(a, b):
        assert torch.equal(x[keep], y[keep])


def test_expanded_offsets_past_32_bits(lib):
    """Keys and queries that start more than 4 GiB into their tensors."""
    rng = np.random.default_rng(14)
    H, n = 128, 90_000                    # 5.9 GB of kv, 4.4 GB of q
    q = torch.empty((n, H, 192), dtype=torch.bfloat16, device=DEV)
    kv = torch.empty((n, H, 256), dtype=torch.bfloat16, device=DEV)
    kr = torch.empty((n, 64), dtype=torch.bfloat16, device=DEV)
    a, b, c = rand(rng, 70, H, 192), rand(rng, 70, H, 256), rand(rng, 70, 64)
    q[-70:], kv[-70:], kr[-70:] = bf(a), bf(b), bf(c)
    cu = dev(np.array([n - 70, n], np.int32))
    out = torch.empty((n, H, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((H, n), device=DEV)
    cfg = lib.make_latent_config(H)
    lib.moe_latent_attn_expanded(cfg, q, kv, kr, cu, cu, 0.1, out=out, lse=lse)
    ref, rl, mag = latent.expanded(a, b, c, [0, 70], [0, 70], np.float32(0.1), True)
    assert_within(host(out[-70:]), ref, out_bound(ref, mag), "out")
    assert_lse(host(lse[:, -70:]), rl)


# ---------------------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------------------
def test_calls_on_another_stream(lib):
    rng = np.random.default_rng(15)
    q, kv, kr, cu_q, cu_k, g = packed(rng, 4, 128, [100], [100])
    cfg = lib.make_latent_config(4)
    args = (cfg, bf(q), bf(kv), bf(kr), dev(cu_q), dev(cu_k), 0.1)
    out, lse = lib.moe_latent_attn_expanded(*args)
    grads = lib.moe_latent_attn_expanded_backward(*args, out, lse, bf(g))
    gd = bf(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = lib.moe_latent_attn_expanded(*args, stream=side)
    g2 = lib.moe_latent_attn_expanded_backward(*args, o2, l2, gd, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, o2) and all(torch.equal(x, y) for x, y in zip(grads, g2))


def test_decode_step_in_a_graph(lib):
    """A token appended and attended to inside a captured graph, replayed over changing
    inputs with eager work between, equals the eager calls every time."""
    rng = np.random.default_rng(16)
    cfg = lib.make_latent_config(16)
    B, page = 3, 16
    cache = torch.zeros((12, page, 656), dtype=torch.uint8, device=DEV)
    table = dev(rng.permutation(12).astype(np.int32).reshape(3, 4))
    lens = torch.zeros((B,), dtype=torch.int32, device=DEV)
    x = torch.zeros((B, 576), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((B, 1, 16, 576), dtype=torch.bfloat16, device=DEV)
    slots = torch.zeros((B,), dtype=torch.int32, device=DEV)
    out = torch.empty((B, 1, 16, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((B, 1, 16), device=DEV)
    ws = torch.empty((lib.moe_latent_attn_absorbed_workspace_bytes(cfg, B, 1),), dtype=torch.uint8, device=DEV)

    def step():
        lib.moe_latent_cache_write(cfg, x, slots, cache)
        lib.moe_latent_attn_absorbed(cfg, q, cache, table, lens, 0.07, out=out, lse=lse, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    cache.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    mirror = torch.zeros_like(cache)
    for n in range(1, 40):
        x.copy_(bf(rand(rng, B, 576)))
        q.copy_(bf(rand(rng, B, 1, 16, 576)))
        pos = n - 1
        slots.copy_(table[:, pos // page] * page + pos % page)
        lens.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        got = (out.clone(), lse.clone())
        lib.moe_latent_cache_write(cfg, x, slots, mirror)
        ref = lib.moe_latent_attn_absorbed(cfg, q, mirror, table, lens, 0.07)
        assert torch.equal(cache, mirror)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), n


def test_prefill_and_decode_agree(lib):
    """The two forms on the same tokens: the cached latents read back, expanded by key and
    value projections and attended to by the expanded form, against the absorbed form with
    the projections folded in. Both within the rounding of their bf16 steps."""
    rng = np.random.default_rng(17)
    H, n, R, D = 16, 90, 512, 128
    cfg = lib.make_latent_config(H)
    x = rand(rng, n, R + 64)
    cache = torch.zeros((3, 32, 656), dtype=torch.uint8, device=DEV)
    table = dev(np.array([[2, 0, 1]], np.int32))
    pos = np.arange(n)
    slots = np.array([2, 0, 1])[pos // 32] * 32 + pos % 32
    lib.moe_latent_cache_write(cfg, bf(x), dev(slots.astype(np.int32)), cache)
    cu = dev(np.array([0, n], np.int32))
    rows = lib.moe_latent_cache_read(cfg, cache, table, cu, n_out=n)
    wk, wv = rand(rng, H, D, R, s=R ** -0.5), rand(rng, H, D, R, s=R ** -0.5)
    q = rand(rng, n, H, D + 64)
    c = host(rows)
    kv = np.concatenate([np.einsum("nr,hdr->nhd", c[:, :R], wk), np.einsum("nr,hdr->nhd", c[:, :R], wv)], 2)
    kv = oracle.round_bf16(kv.astype(np.float32))
    out, _ = lib.moe_latent_attn_expanded(cfg, bf(q), bf(kv), rows[:, R:].contiguous(), cu, cu, 192 ** -0.5)
    qa = np.concatenate([np.einsum("hd,hdr->hr", q[-1, :, :D], wk), q[-1, :, D:]], 1)
    lat, _ = lib.moe_latent_attn_absorbed(cfg, bf(oracle.round_bf16(qa.astype(np.float32)))[None, None], cache, table,
                                          dev(np.array([n], np.int32)), 192 ** -0.5)
    folded = np.einsum("hr,hdr->hd", host(lat)[0, 0], wv)
    a, b = host(out)[-1], folded
    # bf16 roundings of kv, q and the latent output: scores off by about 2^-9 * sqrt(576) / 8
    assert np.linalg.norm(a - b) / np.linalg.norm(a) < 2e-2
