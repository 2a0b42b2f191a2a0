"""Host-side checks of the latent-attention entry points: every refusal comes back with its
documented status before any launch (no GPU needed)."""
import ctypes

import pytest

OK, NULL, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def m():
    import os

    import __graft_entry__
    b = __graft_entry__._builder()
    if not os.path.exists(b.LIB):
        b.build()
    import deepseekmoe_routing_fp8_amd as lib
    return lib


P = ctypes.c_void_p
fake, odd = P(0x1000), P(0x1008)   # never dereferenced


def cfg_of(m, **kw):
    base = dict(n_heads=8, latent=512, rope=64, nope=128, v_dim=128, cache_kind=1)
    base.update(kw)
    return m.moe_latent_config(*[base[f] for f, _ in m.moe_latent_config._fields_])


BAD = [(dict(n_heads=0), SHAPE), (dict(n_heads=1025), SHAPE), (dict(latent=0), SHAPE), (dict(rope=-1), SHAPE),
       (dict(latent=384), UNSUPPORTED), (dict(rope=32), UNSUPPORTED), (dict(nope=64), UNSUPPORTED),
       (dict(nope=96, v_dim=96), UNSUPPORTED), (dict(cache_kind=2), UNSUPPORTED)]


def calls(m, c, **kw):
    """Every entry point with valid arguments but for ``kw``; none may get past its checks
    unless a check is missing."""
    L, r = m._lib, ctypes.byref(c) if c is not None else None
    a = dict(T=4, x=fake, xt=1, ldx=576, slots=fake, cache=fake, n_slots=64, n_pages=4, page=16, table=fake, B=2,
             max_pages=3, cu=fake, n_out=5, out=fake, Sq=1, q=fake, lengths=fake, scale=0.1, ot=1, lse=fake,
             ws=fake, ws_bytes=1 << 40, Tq=5, Tk=6, kv=fake, kr=fake, dout=fake, dq=fake, dkv=fake, dkr=fake)
    a.update(kw)
    g = a.__getitem__
    return {
        "write": lambda: L.moe_latent_cache_write(r, g("T"), g("x"), g("xt"), g("ldx"), g("slots"), g("cache"),
                                                  g("n_slots"), None),
        "read": lambda: L.moe_latent_cache_read(r, g("cache"), g("n_pages"), g("page"), g("table"), g("B"),
                                                g("max_pages"), g("cu"), None, g("n_out"), g("out"), None),
        "absorbed": lambda: L.moe_latent_attn_absorbed(r, g("B"), g("Sq"), g("q"), g("cache"), g("n_pages"),
                                                       g("page"), g("table"), g("max_pages"), g("lengths"),
                                                       g("scale"), g("out"), g("ot"), g("lse"), g("ws"),
                                                       g("ws_bytes"), None),
        "expanded": lambda: L.moe_latent_attn_expanded(r, g("B"), g("Tq"), g("Tk"), g("q"), g("kv"), g("kr"),
                                                       g("cu"), g("cu"), g("scale"), 1, g("out"), g("ot"),
                                                       g("lse"), None),
        "backward": lambda: L.moe_latent_attn_expanded_backward(
            r, g("B"), g("Tq"), g("Tk"), g("q"), g("kv"), g("kr"), g("cu"), g("cu"), g("scale"), 1, g("out"),
            g("lse"), g("dout"), g("dq"), g("dkv"), g("dkr"), g("ot"), g("ws"), g("ws_bytes"), None),
    }


@pytest.mark.parametrize("bad,status", BAD)
def test_configurations_are_checked_by_every_call(m, bad, status):
    c = cfg_of(m, **bad)
    for name, f in calls(m, c).items():
        assert f() == status, name
    assert m._lib.moe_latent_cache_row_bytes(ctypes.byref(c)) == 0
    assert m._lib.moe_latent_attn_absorbed_workspace_bytes(ctypes.byref(c), 1, 1) == 0
    assert m._lib.moe_latent_attn_expanded_backward_workspace_bytes(ctypes.byref(c), 1, 1) == 0


def test_null_configuration(m):
    for name, f in calls(m, None).items():
        assert f() == NULL, name


CHECKS = [
    ("write", dict(T=-1), SHAPE), ("write", dict(ldx=575), SHAPE), ("write", dict(n_slots=-1), SHAPE),
    ("write", dict(xt=2), DTYPE), ("write", dict(x=None), NULL), ("write", dict(slots=None), NULL),
    ("write", dict(cache=None), NULL), ("write", dict(x=odd), UNSUPPORTED), ("write", dict(cache=odd), UNSUPPORTED),
    ("write", dict(ldx=577), UNSUPPORTED), ("write", dict(xt=0, ldx=578), UNSUPPORTED),
    ("write", dict(T=0, x=None), OK), ("write", dict(n_slots=0, cache=None), OK),
    ("read", dict(n_pages=-1), SHAPE), ("read", dict(page=0), SHAPE), ("read", dict(B=-1), SHAPE),
    ("read", dict(n_out=-1), SHAPE), ("read", dict(n_pages=1 << 30, page=4), SHAPE), ("read", dict(out=None), NULL),
    ("read", dict(cu=None), NULL), ("read", dict(table=None), NULL), ("read", dict(cache=None), NULL),
    ("read", dict(out=odd), UNSUPPORTED), ("read", dict(n_out=0, out=None), OK),
    ("absorbed", dict(Sq=0), SHAPE), ("absorbed", dict(Sq=65), SHAPE), ("absorbed", dict(B=-1), SHAPE),
    ("absorbed", dict(B=65536), SHAPE), ("absorbed", dict(page=0), SHAPE), ("absorbed", dict(max_pages=-1), SHAPE),
    ("absorbed", dict(max_pages=1 << 28), SHAPE), ("absorbed", dict(scale=0.0), SHAPE),
    ("absorbed", dict(scale=-1.0), SHAPE), ("absorbed", dict(scale=float("nan")), SHAPE),
    ("absorbed", dict(scale=float("inf")), SHAPE), ("absorbed", dict(ot=2), DTYPE), ("absorbed", dict(q=None), NULL),
    ("absorbed", dict(lengths=None), NULL), ("absorbed", dict(out=None), NULL), ("absorbed", dict(lse=None), NULL),
    ("absorbed", dict(table=None), NULL), ("absorbed", dict(cache=None), NULL), ("absorbed", dict(q=odd), UNSUPPORTED),
    ("absorbed", dict(cache=odd), UNSUPPORTED), ("absorbed", dict(ws=odd), UNSUPPORTED),
    ("absorbed", dict(ws=None), WORKSPACE), ("absorbed", dict(ws_bytes=1000), WORKSPACE),
    ("absorbed", dict(B=0, q=None), OK), ("absorbed", dict(B=65535, max_pages=0x7fffff0, page=16), UNSUPPORTED),
    ("expanded", dict(B=-1), SHAPE), ("expanded", dict(Tq=-1), SHAPE), ("expanded", dict(Tk=1 << 31), SHAPE),
    ("expanded", dict(scale=0.0), SHAPE), ("expanded", dict(ot=9), DTYPE), ("expanded", dict(q=None), NULL),
    ("expanded", dict(kv=None), NULL), ("expanded", dict(kr=None), NULL), ("expanded", dict(cu=None), NULL),
    ("expanded", dict(out=None), NULL), ("expanded", dict(lse=None), NULL), ("expanded", dict(q=odd), UNSUPPORTED),
    ("expanded", dict(kv=odd), UNSUPPORTED), ("expanded", dict(out=odd), UNSUPPORTED),
    ("expanded", dict(Tq=0, q=None), OK), ("expanded", dict(B=0), OK),
    ("backward", dict(B=-1), SHAPE), ("backward", dict(Tk=-1), SHAPE), ("backward", dict(scale=-0.5), SHAPE),
    ("backward", dict(ot=5), DTYPE), ("backward", dict(dout=None), NULL), ("backward", dict(dq=None), NULL),
    ("backward", dict(dkv=None), NULL), ("backward", dict(dkr=None), NULL), ("backward", dict(lse=None), NULL),
    ("backward", dict(dq=odd), UNSUPPORTED), ("backward", dict(dout=odd), UNSUPPORTED),
    ("backward", dict(ws=None), WORKSPACE), ("backward", dict(ws_bytes=100), WORKSPACE),
    ("backward", dict(B=0), OK),
]


@pytest.mark.parametrize("name,kw,status", CHECKS)
def test_refusals(m, name, kw, status):
    assert calls(m, cfg_of(m), **kw)[name]() == status


def test_workspace_sizes(m):
    L, c = m._lib, cfg_of(m)
    need = L.moe_latent_attn_absorbed_workspace_bytes(ctypes.byref(c), 2, 1)
    assert need > 0
    assert calls(m, c, ws_bytes=need - 1)["absorbed"]() == WORKSPACE
    assert L.moe_latent_attn_absorbed_workspace_bytes(ctypes.byref(c), 2, 65) == 0
    assert L.moe_latent_attn_absorbed_workspace_bytes(ctypes.byref(c), 70000, 1) == 0
    b = L.moe_latent_attn_expanded_backward_workspace_bytes(ctypes.byref(c), 5, 6)
    assert b >= 5 * 8 * 4 + 6 * 64 * 4
    assert calls(m, c, ws_bytes=b - 1)["backward"]() == WORKSPACE
    assert m.moe_latent_cache_row_bytes(c) == 656
    assert m.moe_latent_cache_row_bytes(cfg_of(m, latent=256)) == 400
    assert m.moe_latent_cache_row_bytes(cfg_of(m, cache_kind=0)) == 1152


def test_binding_refuses_host_tensors_and_unknown_caches(m):
    import torch
    c = m.make_latent_config(8)
    with pytest.raises(m.MoEError):
        m.make_latent_config(8, cache="int8")
    with pytest.raises(m.MoEError):
        m.moe_latent_cache_write(c, torch.zeros(2, 576), torch.zeros(2, dtype=torch.int32),
                                 torch.zeros(1, 16, 656, dtype=torch.uint8))
    with pytest.raises(m.MoEError):
        m.moe_latent_attn_absorbed(c, torch.zeros(2, 576), torch.zeros(1, 16, 656, dtype=torch.uint8),
                                   torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 0.1)
