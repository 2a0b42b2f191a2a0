"""Measured cases of the latent-attention operators.

A token's keys and values are one latent vector c (``latent`` wide, shared by every head)
and one rotary key (``rope`` wide). The operators are

- ``cache``: write new tokens' (c, rotary key) rows into a paged cache, as bf16 or as E4M3
  codes with a power-of-two scale per 128 values, and read whole contexts back as bf16;
- ``absorbed``: attention of one or a few query tokens a sequence over that cache, with the
  key and value projections absorbed into the query and the output;
- ``expanded``: attention over per-head keys and values expanded from the latents, packed
  sequences of any length, causal or not;
- ``train``: the expanded form with its backward (the rotary key is shared by the heads, so
  its gradient is their sum).

``run`` computes them by elementary operations in 32 bits (``own`` False) or by the calls of
deepseekmoe_routing_fp8_amd (``own`` True).
"""
import math
import random

import torch

own = False

LOG2_448 = (9, 0.875)   # 448 = 0.875 * 2^9


# -- cases ------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a handful of short chats: every sequence appends its token
        dict(name="cache_step", op="cache", kind="fp8", seqs=7, new_lo=1, new_hi=1, ctx_lo=0,
             ctx_hi=250, page=64, latent=512, x="bf16"),
        # a prefill chunk of 4096 tokens: the chunk is written, and the whole contexts are
        # read back for the expansion to keys and values
        dict(name="cache_chunk", op="cache", kind="fp8", seqs=8, new_lo=512, new_hi=512,
             ctx_lo=100, ctx_hi=16000, page=64, latent=512, x="bf16"),
        # the same with an unquantised cache, ragged chunks and an odd page
        dict(name="cache_chunk_bf16", op="cache", kind="bf16", seqs=33, new_lo=1, new_hi=301,
             ctx_lo=1, ctx_hi=4000, page=48, latent=512, x="bf16"),
        # one user, one token, one of eight tensor-parallel ranks' heads: latency
        dict(name="absorbed_one", op="absorbed", kind="fp8", seqs=1, tokens=1, heads=16,
             len_lo=777, len_hi=777, page=64, latent=512),
        # a serving batch on one of eight ranks: few heads, the cache's bytes bound it
        dict(name="absorbed_rank", op="absorbed", kind="bf16", seqs=128, tokens=1, heads=16,
             len_lo=500, len_hi=8192, page=64, latent=512),
        # a data-parallel rank's batch with all heads, one slot of the batch unused
        dict(name="absorbed_heads", op="absorbed", kind="fp8", seqs=64, tokens=1, heads=128,
             len_lo=0, len_hi=8192, page=64, latent=512),
        # two drafted tokens verified beside the last one, a page that ends inside a tile
        dict(name="absorbed_drafts", op="absorbed", kind="bf16", seqs=31, tokens=3, heads=128,
             len_lo=2, len_hi=4097, page=48, latent=512),
        # short prompts on few heads, a single-token one among them
        dict(name="expanded_short", op="expanded", seqs=5, q_lo=1, q_hi=257, ctx_lo=0, ctx_hi=0,
             heads=8, head=128, causal=True),
        # the 4096-token prefill step, all heads, one document
        dict(name="expanded_prefill", op="expanded", seqs=1, q_lo=4096, q_hi=4096, ctx_lo=0,
             ctx_hi=0, heads=128, head=128, causal=True),
        # chunked prefill: new tokens attend to an earlier context as well
        dict(name="expanded_context", op="expanded", seqs=4, q_lo=300, q_hi=700, ctx_lo=1000,
             ctx_hi=8000, heads=32, head=128, causal=True),
        # a training step of a small model on short documents
        dict(name="train_short", op="train", seqs=6, q_lo=1, q_hi=500, ctx_lo=0, ctx_hi=0,
             heads=10, head=64, causal=True),
        # a training step over 4096 tokens in two documents, all heads
        dict(name="train_step", op="train", seqs=2, q_lo=1900, q_hi=2196, ctx_lo=0, ctx_hi=0,
             heads=128, head=128, causal=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("cache", "absorbed", "absorbed", "expanded", "train"))
    kind = rng.choice(("fp8", "bf16"))
    latent = rng.choice((512, 512, 512, 256))
    page = rng.choice((1, 16, 48, 64, 64, 100, 128))
    if op == "cache":
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 1, 60000 // seqs)
        new = _log(rng, 1, max(1, min(hi, 4096 // seqs)))
        return dict(op=op, kind=kind, seqs=seqs, new_lo=rng.choice((1, new)), new_hi=new,
                    ctx_lo=0, ctx_hi=hi, page=page, latent=latent, x=rng.choice(("bf16", "bf16", "f32")))
    if op == "absorbed":
        while True:
            seqs, heads, tokens = _log(rng, 1, 128), _log(rng, 1, 128), rng.choice((1, 1, 1, 2, 3, 4))
            if rng.random() < 0.6:
                heads = rng.choice((8, 16, 32, 64, 128))
            hi = _log(rng, 1, 32000)
            # no more cached rows, and no more products, than the largest listed case may have
            if seqs * hi <= 300_000 and seqs * hi * heads * tokens <= 25_000_000:
                break
        return dict(op=op, kind=kind, seqs=seqs, tokens=tokens, heads=heads,
                    len_lo=rng.choice((0, 1, max(1, hi // 2), hi)), len_hi=hi, page=page, latent=latent)
    while True:
        seqs, heads, hi = _log(rng, 1, 16), _log(rng, 1, 128), _log(rng, 1, 4096)
        if rng.random() < 0.5:
            heads = rng.choice((8, 32, 64, 128))
        ctx = rng.choice((0, 0, _log(rng, 1, 8000)))
        if seqs * hi * (hi + 2 * ctx) * heads <= 600_000_000 and seqs * (hi + ctx) * heads <= 1_000_000:
            break
    return dict(op=op, seqs=seqs, q_lo=rng.choice((1, max(1, hi // 2), hi)), q_hi=hi, ctx_lo=0,
                ctx_hi=ctx, heads=heads, head=rng.choice((128, 128, 64)),
                causal=rng.random() < 0.8)


def _ragged(n, lo, hi, salt):
    """n lengths in [lo, hi], the ends among them, the same for the same case."""
    r = random.Random(f"{n},{lo},{hi},{salt}")
    v = [hi, lo][:n] + [r.randint(lo, hi) for _ in range(n - 2)]
    r.shuffle(v)
    return v


def _sizes(case):
    """The lengths of the case's sequences: (new tokens, tokens before them) a sequence."""
    n = case["seqs"]
    if case["op"] == "cache":
        return _ragged(n, case["new_lo"], case["new_hi"], "new"), _ragged(n, case["ctx_lo"], case["ctx_hi"], "ctx")
    if case["op"] == "absorbed":
        return [case["tokens"]] * n, _ragged(n, case["len_lo"], case["len_hi"], "len")
    return _ragged(n, case["q_lo"], case["q_hi"], "q"), _ragged(n, case["ctx_lo"], case["ctx_hi"], "ctx")


# -- inputs -----------------------------------------------------------------------------
def _row_bytes(latent):
    """codes, 64 bf16 of rotary key, a float scale per 128 codes, padded to 16 bytes."""
    return (latent + 2 * 64 + 4 * (latent // 128) + 15) // 16 * 16


def _scores_like(shape, gen, heads_dim, width):
    """Queries whose scaled scores against unit keys spread by about two, by head between
    one and four."""
    q = torch.randn(shape, generator=gen, device="cuda")
    gain_shape = [1] * len(shape)
    gain_shape[heads_dim] = shape[heads_dim]
    gain = torch.exp2(2 * torch.rand(gain_shape, generator=gen, device="cuda"))
    return (q * gain * (math.sqrt(192) / math.sqrt(width))).to(torch.bfloat16)


def _latents(n, latent, gen):
    """Normalised latents with a channel weight and a few strong channels, and rotary keys."""
    w = 0.5 + torch.rand((latent,), generator=gen, device="cuda")
    w[torch.randint(0, latent, (4,), generator=gen, device="cuda")] *= 4
    c = torch.randn((n, latent), generator=gen, device="cuda")
    return torch.cat([c * torch.rsqrt((c * c).mean(1, keepdim=True)) * w,
                      torch.randn((n, 64), generator=gen, device="cuda")], 1)


def _pages(lens, page, gen):
    """A page table over a pool whose pages the sequences hold in no order."""
    need = [-(-l // page) for l in lens]
    total = sum(need) + 3
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, total


def _slots(table, page, b, start, n):
    """Row numbers in the pool of positions start..start+n-1 of sequence b."""
    pos = torch.arange(start, start + n, device=table.device)
    return table[b].long()[pos // page] * page + pos % page


def _plain_encode(x, kind, latent):
    """Cache rows of x [n, latent + 64]."""
    if kind == "bf16":
        return x.to(torch.bfloat16)
    n = x.shape[0]
    v = x[:, :latent].float().reshape(n, latent // 128, 128)
    amax = v.abs().amax(2)
    m, e = torch.frexp(amax)
    k = e - LOG2_448[0] + (m > LOG2_448[1]).to(e.dtype)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), k.clamp(min=-126)), torch.ones_like(amax))
    codes = (v / scale[:, :, None]).reshape(n, latent).to(torch.float8_e4m3fn)
    row = torch.zeros((n, _row_bytes(latent)), dtype=torch.uint8, device=x.device)
    row[:, :latent] = codes.view(torch.uint8)
    row[:, latent:latent + 128] = x[:, latent:].to(torch.bfloat16).contiguous().view(torch.uint8)
    row[:, latent + 128:latent + 128 + 4 * (latent // 128)] = scale.contiguous().view(torch.uint8)
    return row


def _plain_decode(rows, kind, latent):
    """Float values of cache rows."""
    if kind == "bf16":
        return rows.float()
    n = rows.shape[0]
    codes = rows[:, :latent].contiguous().view(torch.float8_e4m3fn).float()
    rope = rows[:, latent:latent + 128].contiguous().view(torch.bfloat16).float()
    scale = rows[:, latent + 128:latent + 128 + 4 * (latent // 128)].contiguous().view(torch.float32)
    v = codes.reshape(n, latent // 128, 128) * scale[:, :, None]
    return torch.cat([v.reshape(n, latent), rope], 1)


def _offsets(lens):
    v = [0]
    for l in lens:
        v.append(v[-1] + l)
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new, before = _sizes(case)
    st = dict(case=case, new=new, before=before)
    op = case["op"]
    if op in ("cache", "absorbed"):
        latent, page, kind = case["latent"], case["page"], case["kind"]
        lens = [a + b for a, b in zip(new, before)] if op == "cache" else before
        table, n_pages = _pages(lens, page, gen)
        width = latent + 64 if kind == "bf16" else _row_bytes(latent)
        pool = torch.zeros((n_pages * page, width), device="cuda",
                           dtype=torch.bfloat16 if kind == "bf16" else torch.uint8)
        for b, l in enumerate(before):   # what is in the cache before the call
            if l:
                x = _latents(l, latent, gen).to(torch.bfloat16)
                pool[_slots(table, page, b, 0, l)] = _plain_encode(x, kind, latent)
        st.update(table=table, cache=pool.reshape(n_pages, page, width))
        if op == "cache":
            xt = torch.float32 if case["x"] == "f32" else torch.bfloat16
            st["x"] = _latents(sum(new), latent, gen).to(xt)
            st["slots"] = torch.cat([_slots(table, page, b, before[b], n)
                                     for b, n in enumerate(new)]).to(torch.int32)
            st["lens"], st["cu"] = lens, _offsets(lens)
        else:
            st["q"] = _scores_like((case["seqs"], case["tokens"], case["heads"], latent + 64), gen, 2,
                                   latent + 64)
            st["lengths"] = torch.tensor(before, dtype=torch.int32, device="cuda")
    else:
        H, D = case["heads"], case["head"]
        Tq, Tk = sum(new), sum(new) + sum(before)
        st["q"] = _scores_like((Tq, H, D + 64), gen, 1, D + 64)
        st["kv"] = torch.randn((Tk, H, 2 * D), generator=gen, device="cuda").to(torch.bfloat16)
        st["k_rope"] = torch.randn((Tk, 64), generator=gen, device="cuda").to(torch.bfloat16)
        st["cu_q"], st["cu_k"] = _offsets(new), _offsets([a + b for a, b in zip(new, before)])
        if op == "train":
            st["dout"] = torch.randn((Tq, H, D), generator=gen, device="cuda").to(torch.bfloat16)
    st["scale"] = _scale(case)
    if own:
        _plan(st)
    return st


def _scale(case):
    """1 / sqrt(width of an expanded head's key); the absorbed form keeps it."""
    return 1.0 / math.sqrt(case.get("head", 128) + 64)


def _plan(st):
    """What a program of the framework keeps from call to call: the configuration, output
    buffers and workspaces."""
    import deepseekmoe_routing_fp8_amd as lib
    case, dev = st["case"], "cuda"
    op, bf16 = case["op"], torch.bfloat16
    empty = lambda shape, dt: torch.empty(shape, dtype=dt, device=dev)
    if op in ("cache", "absorbed"):
        st["cfg"] = lib.make_latent_config(case.get("heads", 128), latent=case["latent"], cache=case["kind"])
    else:
        st["cfg"] = lib.make_latent_config(case["heads"], nope=case["head"], v_dim=case["head"])
    if op == "cache":
        st["out"] = empty((sum(st["lens"]), case["latent"] + 64), bf16)
    elif op == "absorbed":
        B, S, H = case["seqs"], case["tokens"], case["heads"]
        st["out"], st["lse"] = empty((B, S, H, case["latent"]), bf16), empty((B, S, H), torch.float32)
        st["ws"] = empty((lib.moe_latent_attn_absorbed_workspace_bytes(st["cfg"], B, S),), torch.uint8)
    else:
        Tq, H, D = st["q"].shape[0], case["heads"], case["head"]
        st["out"], st["lse"] = empty((Tq, H, D), bf16), empty((H, Tq), torch.float32)
        if op == "train":
            st["dq"], st["dkv"] = torch.empty_like(st["q"]), torch.empty_like(st["kv"])
            st["dk_rope"] = torch.empty_like(st["k_rope"])
            st["ws"] = empty((lib.moe_latent_attn_expanded_backward_workspace_bytes(
                st["cfg"], Tq, st["kv"].shape[0]),), torch.uint8)


# -- one pass ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import deepseekmoe_routing_fp8_amd as lib
    case, cfg = st["case"], st["cfg"]
    if case["op"] == "cache":
        lib.moe_latent_cache_write(cfg, st["x"], st["slots"], st["cache"])
        return lib.moe_latent_cache_read(cfg, st["cache"], st["table"], st["cu"], out=st["out"])
    if case["op"] == "absorbed":
        return lib.moe_latent_attn_absorbed(cfg, st["q"], st["cache"], st["table"], st["lengths"],
                                            st["scale"], out=st["out"], lse=st["lse"], ws=st["ws"])
    args = (cfg, st["q"], st["kv"], st["k_rope"], st["cu_q"], st["cu_k"], st["scale"])
    out, lse = lib.moe_latent_attn_expanded(*args, causal=case["causal"], out=st["out"], lse=st["lse"])
    if case["op"] == "expanded":
        return out, lse
    return (out,) + tuple(lib.moe_latent_attn_expanded_backward(
        *args, out, lse, st["dout"], causal=case["causal"], dq=st["dq"], dkv=st["dkv"],
        dk_rope=st["dk_rope"], ws=st["ws"]))


def _run_plain(st):
    case = st["case"]
    if case["op"] == "cache":
        pool = st["cache"].flatten(0, 1)
        pool[st["slots"].long()] = _plain_encode(st["x"], case["kind"], case["latent"])
        rows = torch.cat([_slots(st["table"], case["page"], b, 0, l) for b, l in enumerate(st["lens"])])
        return _plain_decode(pool[rows], case["kind"], case["latent"]).to(torch.bfloat16)
    if case["op"] == "absorbed":
        return _plain_absorbed(st)
    return _plain_expanded(st)


def _visible(nq, nk, causal, device):
    """[nq, nk] truth values: query i may see key j. The last query sees every key."""
    if not causal:
        return torch.ones((nq, nk), dtype=torch.bool, device=device)
    i = torch.arange(nq, device=device)[:, None]
    return torch.arange(nk, device=device)[None, :] <= i + (nk - nq)


def _softmax(s, vis):
    """Row softmax of the visible scores (a row that sees nothing is zero), and the
    logarithm of the rows' sums of exponentials."""
    s = s.masked_fill(~vis, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    return e / torch.where(l == 0, torch.ones_like(l), l), (m + torch.log(l)).squeeze(-1)


def _plain_absorbed(st):
    case, q, latent = st["case"], st["q"], st["case"]["latent"]
    B, S, H, W = q.shape
    pool = st["cache"].flatten(0, 1)
    out = torch.zeros((B, S, H, latent), dtype=torch.bfloat16, device=q.device)
    lse = torch.full((B, S, H), -math.inf, device=q.device)
    for b, l in enumerate(st["before"]):
        if l == 0:
            continue
        k = _plain_decode(pool[_slots(st["table"], case["page"], b, 0, l)], case["kind"], latent)
        s = (q[b].float().reshape(S * H, W) @ k.t()).reshape(S, H, l) * st["scale"]
        p, ls = _softmax(s, _visible(S, l, True, q.device)[:, None, :])
        out[b] = (p.reshape(S * H, l) @ k[:, :latent]).reshape(S, H, latent).to(torch.bfloat16)
        lse[b] = ls
    return out, lse


def _plain_expanded(st):
    """The expanded form, and for a training case its gradients: with P the softmax and
    D = rowsum(dO * O), dV = P^T dO, dS = P * (dO V^T - D), dQ = scale dS K,
    dK = scale dS^T Q, the rotary part of dK summed over the heads."""
    case, dev = st["case"], st["q"].device
    H, D, train = case["heads"], case["head"], case["op"] == "train"
    q, kv = st["q"], st["kv"]
    out = torch.zeros((q.shape[0], H, D), dtype=torch.bfloat16, device=dev)
    lse = torch.full((H, q.shape[0]), -math.inf, device=dev)
    if train:
        dq, dkv = torch.zeros_like(q), torch.zeros_like(kv)
        dk_rope = torch.zeros((kv.shape[0], 64), device=dev)
    tq = tk = 0
    for nq, nb in zip(st["new"], st["before"]):
        nk = nq + nb
        vis = _visible(nq, nk, case["causal"], dev)
        kr = st["k_rope"][tk:tk + nk].float()
        step = max(1, min(H, (1 << 28) // (nq * nk)))   # heads at once
        for h in range(0, H, step):
            n = min(step, H - h)
            qh = q[tq:tq + nq, h:h + n].float().transpose(0, 1).contiguous()
            kvh = kv[tk:tk + nk, h:h + n].float().transpose(0, 1).contiguous()
            kh = torch.cat([kvh[:, :, :D], kr.expand(n, nk, 64)], 2)
            vh = kvh[:, :, D:].contiguous()
            p, ls = _softmax(torch.matmul(qh, kh.transpose(1, 2).contiguous()) * st["scale"], vis)
            o = torch.matmul(p, vh)
            out[tq:tq + nq, h:h + n] = o.transpose(0, 1).to(torch.bfloat16)
            lse[h:h + n, tq:tq + nq] = ls
            if train:
                do = st["dout"][tq:tq + nq, h:h + n].float().transpose(0, 1).contiguous()
                dp = torch.matmul(do, vh.transpose(1, 2).contiguous())
                ds = p * (dp - (do * o).sum(2, keepdim=True)) * st["scale"]
                dst = ds.transpose(1, 2).contiguous()
                dk = torch.matmul(dst, qh)
                dq[tq:tq + nq, h:h + n] = torch.matmul(ds, kh).transpose(0, 1).to(torch.bfloat16)
                dkv[tk:tk + nk, h:h + n, :D] = dk[:, :, :D].transpose(0, 1).to(torch.bfloat16)
                dkv[tk:tk + nk, h:h + n, D:] = torch.matmul(
                    p.transpose(1, 2).contiguous(), do).transpose(0, 1).to(torch.bfloat16)
                dk_rope[tk:tk + nk] += dk[:, :, D:].sum(0)
        tq, tk = tq + nq, tk + nk
    return (out, dq, dkv, dk_rope.to(torch.bfloat16)) if train else (out, lse)


# -- what a pass cannot do without ---------------------------------------------------------
def work(case):
    new, before = _sizes(case)
    op = case["op"]
    if op == "cache":
        latent = case["latent"]
        row = 2 * (latent + 64) if case["kind"] == "bf16" else latent + 128 + 4 * (latent // 128)
        n, total = sum(new), sum(new) + sum(before)
        # new rows in, their cache rows out; the cached rows in (the new ones are at hand), all out as bf16
        xb = 4 if case["x"] == "f32" else 2
        return {"bytes": n * (xb * (latent + 64) + row) + (total - n) * row + total * 2 * (latent + 64),
                "flops": 2 * n * latent if case["kind"] == "fp8" else 0}
    if op == "absorbed":
        latent, H, S, B = case["latent"], case["heads"], case["tokens"], case["seqs"]
        row = 2 * (latent + 64) if case["kind"] == "bf16" else latent + 128 + 4 * (latent // 128)
        pairs = sum(max(0, l - S + 1 + s) for l in before for s in range(S))
        return {"bytes": sum(before) * row + B * S * H * (2 * (latent + 64) + 2 * latent + 4),
                "flops": 2 * pairs * H * (2 * latent + 64)}
    H, D = case["heads"], case["head"]
    pairs = 0
    for nq, nb in zip(new, before):
        pairs += nq * nb + nq * (nq + 1) // 2 if case["causal"] else nq * (nq + nb)
    Tq, Tk = sum(new), sum(new) + sum(before)
    read = 2 * (Tq * H * (D + 64) + Tk * H * 2 * D + Tk * 64)
    if op == "expanded":
        return {"bytes": read + Tq * H * (2 * D + 4), "flops": 2 * pairs * H * (2 * D + 64)}
    # forward; then the gradients from the scores and from dO V^T, each formed once
    return {"bytes": read + 2 * Tq * H * 2 * D + read,
            "flops": 2 * pairs * H * ((D + 64) * 4 + D * 3)}


# -- 64 bits ----------------------------------------------------------------------------
def exact(case, seed):
    """The outputs in 64 bits, from the definitions, pair by pair of query and key blocks of
    a head. Written over the inputs of ``prepare`` and nothing of the plain forms."""
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] in ("cache", "absorbed"):
        latent, page, lens = case["latent"], case["page"], st.get("lens", st["before"])
        host, table = st["cache"].reshape(-1, st["cache"].shape[2]), st["table"].long()
        rows = [table[b].repeat_interleave(page)[:l] * page + torch.arange(l, device="cuda") % page
                for b, l in enumerate(lens)]
    if case["op"] == "cache":
        values = torch.zeros((host.shape[0], latent + 64), dtype=f64, device="cuda")
        old = torch.cat([r[:n] for r, n in zip(rows, st["before"])])
        values[old] = _values64(host[old], case["kind"], latent)
        x = st["x"].to(f64)
        if case["kind"] == "fp8":
            for g in range(latent // 128):
                v = x[:, 128 * g:128 * (g + 1)]
                top = v.abs().amax(1, keepdim=True)
                k = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448)).clamp(min=-126)
                s = torch.exp2(k)
                x[:, 128 * g:128 * (g + 1)] = _nearest_e4m3(v / s) * s
        values[st["slots"].long()] = x
        return values[torch.cat(rows)]
    if case["op"] == "absorbed":
        B, S, H, _ = st["q"].shape
        out = torch.zeros((B, S, H, latent), dtype=f64, device="cuda")
        lse = torch.full((B, S, H), -math.inf, dtype=f64, device="cuda")
        for b, l in enumerate(lens):
            k = _values64(host[rows[b]], case["kind"], latent)
            for s in range(S):
                n = l - (S - 1 - s)   # keys that this query sees
                if n > 0:
                    z = st["q"][b, s].to(f64).mul(st["scale"]).mm(k[:n].t())
                    lse[b, s] = torch.logsumexp(z, 1)
                    out[b, s] = torch.exp(z - lse[b, s][:, None]).mm(k[:n, :latent])
        return out, lse
    return _exact_expanded(case, st)


def _values64(rows, kind, latent):
    if kind == "bf16":
        return rows.to(torch.float64)
    code = rows[:, :latent].to(torch.int64)
    mant, expo, sign = code & 7, (code >> 3) & 15, code >> 7
    # value = mantissa / 8 * 2^-6 below the normal range, else (1 + mantissa / 8) * 2^(expo - 7)
    v = torch.where(expo == 0, mant / 8.0 * 2.0 ** -6, (1 + mant / 8.0) * torch.exp2((expo - 7).to(torch.float64)))
    v = torch.where(sign == 1, -v, v)
    scale = rows[:, latent + 128:latent + 128 + 4 * (latent // 128)].contiguous().view(torch.float32)
    v = v * scale.to(torch.float64).repeat_interleave(128, dim=1)
    return torch.cat([v, rows[:, latent:latent + 128].contiguous().view(torch.bfloat16).to(torch.float64)], 1)


def _nearest_e4m3(v):
    """The E4M3 value nearest to v, halves to the even one."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_expanded(case, st):
    f64, H, D = torch.float64, case["heads"], case["head"]
    scale, train = st["scale"], case["op"] == "train"
    out = torch.zeros((st["q"].shape[0], H, D), dtype=f64, device="cuda")
    lse = torch.full((H, st["q"].shape[0]), -math.inf, dtype=f64, device="cuda")
    if train:
        gq = torch.zeros(st["q"].shape, dtype=f64, device="cuda")
        gkv = torch.zeros(st["kv"].shape, dtype=f64, device="cuda")
        gr = torch.zeros(st["k_rope"].shape, dtype=f64, device="cuda")
    cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
    for b in range(case["seqs"]):
        rq, rk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        nq, nk = rq.stop - rq.start, rk.stop - rk.start
        hidden = None
        if case["causal"]:
            hidden = torch.ones((nq, nk), dtype=torch.bool, device="cuda").triu(nk - nq + 1)
        for h in range(H):
            qh = st["q"][rq, h].to(f64)
            key = torch.cat([st["kv"][rk, h, :D], st["k_rope"][rk]], 1).to(f64)
            val = st["kv"][rk, h, D:].to(f64)
            z = qh.mm(key.t()).mul_(scale)
            if hidden is not None:
                z.masked_fill_(hidden, -math.inf)
            ls = torch.logsumexp(z, 1)
            w = torch.exp(z - torch.where(ls == -math.inf, torch.zeros_like(ls), ls)[:, None])
            out[rq, h], lse[h, rq] = w.mm(val), ls
            if train:
                g = st["dout"][rq, h].to(f64)
                gkv[rk, h, D:] = w.t().mm(g)
                gw = g.mm(val.t())
                gz = w * (gw - (w * gw).sum(1, keepdim=True)) * scale
                gq[rq, h] = gz.mm(key)
                gk = gz.t().mm(qh)
                gkv[rk, h, :D] = gk[:, :D]
                gr[rk] += gk[:, D:]
    return (out, gq, gkv, gr) if train else (out, lse)
