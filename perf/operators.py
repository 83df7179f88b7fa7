"""Plain forms, inputs and sizes of the attention operators beside BSA: cross attention to an
encoder's states of another length (serving and training), and attention of an ensemble whose
members share a long prefix of keys and add a few of their own.

Layouts are those of include/bsa.h: q, out [B][H][n_q][d]; k, v [B][H_kv][n_k][d], H a multiple of
H_kv (query head h reads key head h * H_kv / H); key_len [B] counts a batch entry's keys, those
behind it are not attended; a row without keys gives zeros and carries no gradient. A shared
prefix is [groups][H_kv][n_prefix][d]: the batch is `groups` ensembles of B / groups members each.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------- cases


def _cross(name, batch, heads, kv_heads, n_q, n_k, d, ragged):
    return dict(name=name, op="cross", batch=batch, heads=heads, kv_heads=kv_heads, n_q=n_q, n_k=n_k, d=d,
                ragged=ragged)


def _train(name, batch, heads, kv_heads, n_q, n_k, d, ragged):
    return dict(_cross(name, batch, heads, kv_heads, n_q, n_k, d, ragged), op="train")


def _prefix(name, groups, batch, heads, kv_heads, n_q, n_prefix, n_own, d, ragged):
    return dict(name=name, op="prefix", groups=groups, batch=batch, heads=heads, kv_heads=kv_heads, n_q=n_q,
                n_prefix=n_prefix, n_own=n_own, d=d, ragged=ragged)


def listed():
    return [
        # one query row against one forecast's few encoder states: a call's latency
        _cross("cross_one_row", 1, 8, 8, 1, 512, 64, False),
        # 24 ensemble members, one new row each, against their own 1.5 degree fields (121 x 240 points)
        _cross("cross_members_1p5deg", 24, 16, 4, 1, 29040, 128, False),
        # a padded batch of encoder states, odd sizes, three query heads a key head, one entry without states
        _cross("cross_ragged", 6, 12, 4, 333, 777, 128, True),
        # every HEALPix token of Nside 32 attends to every point of a 1.5 degree field
        _cross("cross_nside32_1p5deg", 1, 8, 8, 12288, 29040, 64, False),
        # a training step of the tiny resolution (Nside 8) on a handful of states
        _train("train_nside8", 1, 2, 2, 768, 200, 64, False),
        # Nside 32 tokens against a coarse trunk of Nside 8 states: few keys, many queries
        _train("train_nside32_coarse", 2, 8, 8, 12288, 768, 64, False),
        # a padded batch with shared key heads and odd lengths
        _train("train_ragged", 3, 16, 4, 1001, 2345, 128, True),
        # two Nside 32 fields attending to one another in full
        _train("train_nside32", 1, 8, 8, 12288, 12288, 64, False),
        # a small ensemble, a few rows and states each
        _prefix("prefix_small", 1, 4, 8, 8, 3, 777, 77, 64, True),
        # 24 members roll out one row at a time over a shared Nside 32 analysis and their own 40 steps
        _prefix("prefix_members", 1, 24, 16, 4, 1, 12288, 40, 128, True),
        # two ensembles of 24 over Nside 64 analyses, 16 rows a member, longer own histories
        _prefix("prefix_nside64", 2, 48, 16, 16, 16, 49152, 1024, 64, True),
        # 8 members with a whole Nside 8 field of rows each
        _prefix("prefix_fields", 1, 8, 8, 8, 768, 12288, 768, 64, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["cross", "train", "prefix"])
        d = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        heads = kv_heads * rng.choice([1, 1, 2, 3, 4])
        ragged = rng.random() < 0.5
        if op == "prefix":
            groups = rng.choice([1, 1, 2, 3])
            batch = groups * _log(rng, 1, 24)
            c = _prefix("", groups, batch, heads, kv_heads, _log(rng, 1, 512), _log(rng, 64, 49152),
                        _log(rng, 1, 1024), d, ragged)
        elif op == "cross":
            c = _cross("", _log(rng, 1, 24), heads, kv_heads, _log(rng, 1, 12288), _log(rng, 16, 29040), d, ragged)
        else:
            c = _train("", _log(rng, 1, 6), heads, kv_heads, _log(rng, 64, 12288), _log(rng, 64, 12288), d, ragged)
        del c["name"]
        w = work(c)
        keys = c["n_prefix"] + c["n_own"] if op == "prefix" else c["n_k"]
        if (w["flops"] <= (1.0e12 if op == "train" else 6e11) and w["bytes"] <= 1.4e9
                and c["batch"] * heads * c["n_q"] * keys <= 1.2e9):
            return c


# ---------------------------------------------------------------- lengths and work


def _lengths(n, count, ragged):
    """Lengths of `count` batch entries of capacity n: all full, or spread from none to full."""
    if not ragged:
        return [n] * count
    if count == 1:
        return [n - n // 3]
    return [(n * i) // (count - 1) for i in range(count)]


def work(case):
    """Every input read once, every output written once; 4 d flops a query and key forward, 10 d
    backward (its five products: scores, dP, dV, dK, dQ). Keys behind a length count for nothing
    but the zero gradients written there."""
    b, h, hk, nq, d = case["batch"], case["heads"], case["kv_heads"], case["n_q"], case["d"]
    rows = b * h * nq * d * 2
    if case["op"] == "prefix":
        own_keys = sum(_lengths(case["n_own"], b, case["ragged"]))
        pre = case["groups"] * case["n_prefix"]
        pairs = h * nq * (b * case["n_prefix"] + own_keys)
        return {"bytes": 2 * rows + 2 * hk * d * 2 * (pre + own_keys), "flops": 4 * d * pairs}
    keys = sum(_lengths(case["n_k"], b, case["ragged"]))
    pairs = h * nq * keys
    if case["op"] == "cross":
        return {"bytes": 2 * rows + 2 * hk * d * 2 * keys, "flops": 4 * d * pairs}
    # q, dout in, out, dq out; k, v in over the lengths, dk, dv out whole
    return {"bytes": 4 * rows + 2 * hk * d * 2 * (keys + b * case["n_k"]), "flops": 14 * d * pairs}


# ---------------------------------------------------------------- inputs


def _normal(gen, shape, size=1.0):
    x = torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)
    return (x * size).to(torch.bfloat16)


def _shuffled(n, count, ragged, seed, device):
    lens = _lengths(n, count, ragged)
    random.Random(seed).shuffle(lens)
    return torch.tensor(lens, dtype=torch.int32, device=device) if ragged else None


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)
    b, h, hk, nq, d = case["batch"], case["heads"], case["kv_heads"], case["n_q"], case["d"]
    # normalised tokens; queries a little larger, so that rows prefer some keys (logits of about +-2)
    st = dict(case=dict(case), q=_normal(gen, (b, h, nq, d), 2.0), layer=None)
    if case["op"] == "prefix":
        g = case["groups"]
        st["k_prefix"], st["v_prefix"] = (_normal(gen, (g, hk, case["n_prefix"], d)) for _ in range(2))
        st["k_own"], st["v_own"] = (_normal(gen, (b, hk, case["n_own"], d)) for _ in range(2))
        st["own_len"] = _shuffled(case["n_own"], b, case["ragged"], seed, dev)
    else:
        st["k"], st["v"] = (_normal(gen, (b, hk, case["n_k"], d)) for _ in range(2))
        st["key_len"] = _shuffled(case["n_k"], b, case["ragged"], seed, dev)
        if case["op"] == "train":
            st["dout"] = _normal(gen, (b, h, nq, d))
    return st


# ---------------------------------------------------------------- one pass


def run(st):
    return _run_own(st) if own else _PLAIN[st["case"]["op"]](st)


def _run_own(st):
    """The calls a user makes: a layer of fixed sizes, made once, then called."""
    from block_sparse_spherical_b200 import api
    c, layer = st["case"], st["layer"]
    sizes = (c["batch"], c["heads"], c["n_q"])
    if c["op"] == "prefix":
        if layer is None:
            layer = st["layer"] = api.PrefixAttention(*sizes, c["n_prefix"], c["n_own"], c["d"],
                                                      kv_heads=c["kv_heads"], groups=c["groups"])
        return layer(st["q"], st["k_prefix"], st["v_prefix"], st["k_own"], st["v_own"], own_len=st["own_len"])
    if c["op"] == "cross":
        if layer is None:
            layer = st["layer"] = api.CrossAttention(*sizes, c["n_k"], c["d"], kv_heads=c["kv_heads"])
        return layer(st["q"], st["k"], st["v"], key_len=st["key_len"])
    if layer is None:
        layer = st["layer"] = api.CrossAttentionTrain(*sizes, c["n_k"], c["d"], kv_heads=c["kv_heads"])
    out = layer.forward(st["q"], st["k"], st["v"], key_len=st["key_len"])
    dq, dk, dv = layer.backward(st["dout"])
    return out, dq, dk, dv


def _weights(s, allowed):
    """Softmax over the last axis of scores s, in place; `allowed` marks the keys that count, or None."""
    if allowed is not None:
        s = s.masked_fill_(~allowed, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    return p.div_(torch.where(z == 0, torch.ones_like(z), z))


def _allowed(lens, n):
    if lens is None:
        return None
    return (torch.arange(n, device=lens.device) < lens[:, None])[:, None, None, :]   # [B, 1, 1, n]


def _plain_cross(st):
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    b, h, nq, d = q.shape
    hk, n = k.shape[1], k.shape[2]
    p = _weights(q.reshape(b, hk, -1, d) @ k.transpose(-1, -2) * d ** -0.5, _allowed(st["key_len"], n))
    return (p @ v).reshape(b, h, nq, d).to(torch.bfloat16)


def _plain_train(st):
    q, k, v, do = st["q"].float(), st["k"].float(), st["v"].float(), st["dout"].float()
    b, h, nq, d = q.shape
    hk, n = k.shape[1], k.shape[2]
    c = d ** -0.5
    q, do = q.reshape(b, hk, -1, d), do.reshape(b, hk, -1, d)
    p = _weights(q @ k.transpose(-1, -2) * c, _allowed(st["key_len"], n))
    o = p @ v
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(c)
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    return tuple(x.reshape(shape).to(torch.bfloat16) for x, shape in
                 ((o, (b, h, nq, d)), (dq, (b, h, nq, d)), (dk, k.shape), (dv, v.shape)))


def _plain_prefix(st):
    q, kp, vp, ko, vo = (st[x].float() for x in ("q", "k_prefix", "v_prefix", "k_own", "v_own"))
    b, h, nq, d = q.shape
    g, hk, n = kp.shape[:3]
    c = d ** -0.5
    rows = q.reshape(g, b // g, hk, -1, d)                                   # [G, members, H_kv, rows, d]
    sp = (rows.transpose(1, 2).reshape(g, hk, -1, d) @ kp.transpose(-1, -2)) * c
    sp = sp.reshape(g, hk, b // g, -1, n).transpose(1, 2).reshape(b, hk, -1, n)
    so = (q.reshape(b, hk, -1, d) @ ko.transpose(-1, -2)) * c
    ok = _allowed(st["own_len"], ko.shape[2])
    if ok is not None:
        so = so.masked_fill_(~ok, -math.inf)
    p = _weights(torch.cat([sp, so], -1), None)
    pp = p[..., :n].reshape(g, b // g, hk, -1, n).transpose(1, 2).reshape(g, hk, -1, n)
    o = (pp @ vp).reshape(g, hk, b // g, -1, d).transpose(1, 2).reshape(b, hk, -1, d) + p[..., n:] @ vo
    return o.reshape(b, h, nq, d).to(torch.bfloat16)


_PLAIN = {"cross": _plain_cross, "train": _plain_train, "prefix": _plain_prefix}

# ---------------------------------------------------------------- in 64 bits


def _attend64(q, k, v):
    """softmax(q k^T / sqrt(d)) v of one head, in 64 bits."""
    return torch.softmax((q @ k.T) / math.sqrt(q.shape[-1]), dim=-1) @ v


def exact(case, seed):
    """Head by head in 64 bits over the keys that exist; gradients by differentiating that."""
    st = prepare(case, seed)
    b, h, hk = case["batch"], case["heads"], case["kv_heads"]
    q = st["q"].double()
    out = torch.zeros_like(q)
    if case["op"] == "prefix":
        per = b // case["groups"]
        for i in range(b):
            n = case["n_own"] if st["own_len"] is None else int(st["own_len"][i])
            for j in range(h):
                e = j * hk // h
                k = torch.cat([st["k_prefix"][i // per, e], st["k_own"][i, e, :n]]).double()
                v = torch.cat([st["v_prefix"][i // per, e], st["v_own"][i, e, :n]]).double()
                out[i, j] = _attend64(q[i, j], k, v)
        return out
    k64, v64 = st["k"].double(), st["v"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k64), torch.zeros_like(v64)
    for i in range(b):
        n = case["n_k"] if st["key_len"] is None else int(st["key_len"][i])
        if n == 0:
            continue
        for j in range(h):
            e = j * hk // h
            x = [t.clone().requires_grad_(case["op"] == "train") for t in (q[i, j], k64[i, e, :n], v64[i, e, :n])]
            o = _attend64(*x)
            out[i, j] = o.detach()
            if case["op"] == "train":
                gq, gk, gv = torch.autograd.grad(o, x, st["dout"][i, j].double())
                dq[i, j] = gq
                dk[i, e, :n] += gk
                dv[i, e, :n] += gv
    return (out, dq, dk, dv) if case["op"] == "train" else out
