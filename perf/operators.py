"""Measured cases of the cache-write, cache-read and tree-attention operators.

write: the queries, keys and values of new tokens as the projections leave
       them; per-head norms, the position rotation and the write into the K/V
       cache (bf16, f32, or 8-bit e4m3 codes with one scale a row).
read:  an 8-bit cache read back into 16-bit rows.
tree:  attention of a tree of drafted tokens (a single token is a tree of
       one) over a cache whose last rows hold the tree's own keys and values.
step:  the write of a drafted tree followed by its attention, as a
       speculative decoding step of one layer runs them.

Each case gives entries b, new tokens t, query / kv heads hq / hkv, head size
d, cached tokens s before the new ones, page size (0: dense cache), the
cache's type kv, and whether entries have lengths of their own (ragged).
"""

import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TINY = 2.0 ** -126
EPS = 1e-6
MAX_BYTES = 2.0e9       # a drawn cache's keys and values, at most
MAX_FLOPS = 1.2e11      # a drawn attention's products, at most


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # prompt of a grouped-query layer, written as it leaves the projections: bound by bandwidth
        dict(name="write-prompt-gqa", op="write", b=4, t=2048, hq=32, hkv=8, d=128, s=0, page=0, kv="bf16",
             ragged=False, rot=128, inter=False, norm=True, room=0),
        # odd-length prompt into an 8-bit paged cache
        dict(name="write-prompt-e4m3-paged", op="write", b=2, t=4093, hq=32, hkv=8, d=128, s=0, page=64, kv="e4m3",
             ragged=False, rot=128, inter=False, norm=True, room=0),
        # one token of each of 32 sequences of a multi-head layer: latency
        dict(name="write-step-e4m3", op="write", b=32, t=1, hq=32, hkv=32, d=128, s=200, page=0, kv="e4m3",
             ragged=True, rot=128, inter=False, norm=True, room=55),
        # small 32-bit heads, interleaved rotation of half the channels, no norm: latency
        dict(name="write-small-f32", op="write", b=2, t=5, hq=4, hkv=2, d=64, s=100, page=0, kv="f32",
             ragged=True, rot=32, inter=True, norm=False, room=23),
        # a long 8-bit prefix restored for the sparse decode calls: bound by bandwidth
        dict(name="read-long", op="read", b=1, t=0, hq=8, hkv=8, d=128, s=65536, page=0, kv="e4m3", ragged=False),
        # short ragged sequences read out of pages
        dict(name="read-paged", op="read", b=8, t=0, hq=8, hkv=8, d=128, s=777, page=16, kv="e4m3", ragged=False),
        # the smallest call: a few drafted tokens on a 512-token 32-bit cache
        dict(name="tree-small-f32", op="tree", b=1, t=4, hq=2, hkv=2, d=64, s=512, page=0, kv="f32", ragged=False),
        # a drafted tree of 16 on a grouped-query layer at 32K: bound by the cache's bytes
        dict(name="tree-gqa-32k", op="tree", b=4, t=16, hq=32, hkv=8, d=128, s=32768, page=0, kv="bf16",
             ragged=False),
        # multi-head layer with an 8-bit cache, 8 drafted tokens
        dict(name="tree-mha-e4m3", op="tree", b=8, t=8, hq=32, hkv=32, d=128, s=4096, page=0, kv="e4m3",
             ragged=False),
        # a wide tree over a long prompt: the tensor cores' products count as much as the bytes
        dict(name="tree-wide-128k", op="tree", b=1, t=64, hq=32, hkv=8, d=128, s=131072, page=0, kv="bf16",
             ragged=False),
        # plain single-token decode over a 256K 8-bit cache
        dict(name="token-256k-e4m3", op="tree", b=1, t=1, hq=32, hkv=32, d=128, s=262144, page=0, kv="e4m3",
             ragged=False),
        # a layer's speculative step: ragged batch in pages, norm + rotation + write, then attention
        dict(name="step-paged-ragged", op="step", b=16, t=7, hq=32, hkv=8, d=128, s=8000, page=64, kv="bf16",
             ragged=True, rot=128, inter=False, norm=True, room=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "write", "read", "tree", "tree", "tree", "step"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 16, 32])
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * hkv <= 64])
    kv = rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"])
    page = rng.choice([0, 0, 1, 16, 64, 256])
    ragged = rng.random() < 0.5
    extra = dict(rot=d // rng.choice([1, 1, 2]), inter=rng.random() < 0.4, norm=rng.random() < 0.7,
                 room=rng.randint(0, 60))
    if op == "write":
        t = _log(rng, 1, 4096)
        b = _log(rng, 1, max(1, 4096 // t))
        b = max(1, min(b, int(2.5e8 / (t * (hq + 2 * hkv) * d * 2))))
        return dict(op=op, b=b, t=t, hq=hq, hkv=hkv, d=d, s=_log(rng, 1, 200), page=page, kv=kv, ragged=ragged, **extra)
    size = {"bf16": 2, "e4m3": 1, "f32": 4}[kv]
    if op == "read":
        s = _log(rng, 1, 65536)
        b = _log(rng, 1, 16)
        b = max(1, min(b, int(2.0e8 / (hkv * s * d * 2))))
        return dict(op=op, b=b, t=0, hq=hkv, hkv=hkv, d=d, s=s, page=page, kv="e4m3", ragged=False)
    t = _log(rng, 1, 64 if kv != "f32" else 16)
    s = _log(rng, 1, 131072 if kv != "f32" else 16384)
    b = _log(rng, 1, 32)
    b = max(1, min(b, int(MAX_BYTES / (2 * hkv * (s + t) * d * size)), int(MAX_FLOPS / (4.0 * hq * t * (s + t) * d)),
                   int(4e8 / (t * hq * (s + t)))))
    if op == "step":
        s = min(s, 16384)
        b = max(1, min(b, int(4e8 / (hkv * (s + t + 60) * d * size))))
        return dict(op=op, b=b, t=t, hq=hq, hkv=hkv, d=d, s=s, page=page, kv=kv, ragged=ragged, **extra)
    return dict(op=op, b=b, t=t, hq=hq, hkv=hkv, d=d, s=s, page=page, kv=kv, ragged=ragged)


def _lengths(case):
    """Each entry's cached tokens before the new ones: s, or from about s/4 to s where ragged."""
    b, s = case["b"], case["s"]
    if not case["ragged"]:
        return [s] * b
    return [s if i == 0 else max(min(s, 1), s - (s * ((i * 2654435761) % 1000)) // 1333) for i in range(b)]


def work(case):
    b, t, hq, hkv, d = case["b"], case["t"], case["hq"], case["hkv"], case["d"]
    lens = _lengths(case)
    io = 4 if case["kv"] == "f32" else 2
    row = {"bf16": 2 * d, "f32": 4 * d, "e4m3": d + 4}[case["kv"]]
    by = fl = 0
    if case["op"] in ("write", "step"):
        by += b * t * ((2 * hq + 2 * hkv) * d * io + 2 * hkv * row) + 4 * b * t
        fl += 8 * b * t * (hq + hkv) * d
    if case["op"] == "read":
        by += sum(lens) * 2 * hkv * (row + 2 * d)
        fl += sum(lens) * 2 * hkv * d
    if case["op"] in ("tree", "step"):
        held = sum(lens) + (b * t if case["op"] == "tree" else 0)  # a step's own rows are counted at their write
        by += held * 2 * hkv * row + b * t * hq * d * 2 * io
        fl += 4 * hq * d * t * sum(n + (t + 1) / 2 for n in lens)
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ inputs

def _randn(shape, gen, dtype, scale=None):
    """N(0, 1) drawn in slices of a few hundred MB; `scale` multiplies the last axis."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1, shape[-1])
    step = max(1, (1 << 26) // shape[-1])
    for i in range(0, flat.shape[0], step):
        x = torch.randn((min(step, flat.shape[0] - i), shape[-1]), generator=gen, device=DEV)
        flat[i:i + step] = (x if scale is None else x * scale).to(dtype)
    return out


def _codes(shape, gen):
    """An 8-bit cache as a quantiser leaves it: codes whose rows reach +-448, and the rows' scales."""
    codes = torch.empty(shape, dtype=E4M3, device=DEV)
    scales = torch.empty(shape[:-1], dtype=torch.float32, device=DEV)
    flat, fs = codes.view(-1, shape[-1]), scales.view(-1)
    step = max(1, (1 << 26) // shape[-1])
    for i in range(0, flat.shape[0], step):
        x = torch.randn((min(step, flat.shape[0] - i), shape[-1]), generator=gen, device=DEV)
        sc = x.abs().amax(-1) / E4M3_MAX
        flat[i:i + step] = (x / sc[:, None]).to(E4M3)
        fs[i:i + step] = sc
    return codes, scales


def _inputs(case, seed):
    b, t, hq, hkv, d, s, page = (case[n] for n in ("b", "t", "hq", "hkv", "d", "s", "page"))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    host = torch.Generator()
    host.manual_seed(int(seed) + 1)
    io = torch.float32 if case["kv"] == "f32" else torch.bfloat16
    lens = _lengths(case)
    st = dict(case=case, io=io, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), longest=max(lens))
    room = case.get("room", 5)
    cap = s + t + room
    if page:
        per = -(-cap // page)
        blocks = b * per + 3
        table = torch.randperm(blocks, generator=host)[: b * per].view(b, per)
        st["table"] = table.to(torch.int32).to(DEV)
        shape = (blocks, hkv, page, d)
    else:
        st["table"] = None
        shape = (b, hkv, cap, d)
    st["ks"] = st["vs"] = None
    if case["op"] == "write":  # what else the cache holds does not matter: zeros
        st["k"], st["v"] = (torch.zeros(shape, dtype=E4M3 if case["kv"] == "e4m3" else io, device=DEV) for _ in "kv")
        if case["kv"] == "e4m3":
            st["ks"], st["vs"] = (torch.zeros(shape[:-1], dtype=torch.float32, device=DEV) for _ in "kv")
    elif case["kv"] == "e4m3":
        st["k"], st["ks"] = _codes(shape, gen)
        st["v"], st["vs"] = _codes(shape, gen)
    else:
        heavy = torch.ones(d, device=DEV)  # a few channels of the keys are large
        heavy[torch.randperm(d, generator=host)[:8].to(DEV)] = 4.0
        st["k"], st["v"] = _randn(shape, gen, io, heavy), _randn(shape, gen, io)
    if case["op"] in ("write", "step"):
        # one fused projection's output: queries, keys and values of a token side by side
        qkv = _randn((b, t, hq + 2 * hkv, d), gen, io)
        st["q_in"], st["k_in"], st["v_in"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        st["qw"] = st["kw"] = None
        if case["norm"]:
            st["qw"], st["kw"] = ((1.0 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(io) for _ in "qk")
        j = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
        st["inv_freq"] = torch.pow(10000.0, -2.0 * j / case["rot"]).float()
    else:
        st["q"] = _randn((b, max(t, 1), hq, d), gen, io)
    if case["op"] in ("tree", "step"):
        # every node's parent is the prefix or an earlier node; a node sees its ancestors and itself
        parent = (torch.rand((b, t), generator=host) * (torch.arange(t) + 1)).long() - 1
        sees = torch.eye(t, dtype=torch.bool).repeat(b, 1, 1)
        depth = torch.zeros((b, t), dtype=torch.int32)
        for i in range(t):
            p = parent[:, i]
            rows = torch.nonzero(p >= 0).flatten()
            sees[rows, i] |= sees[rows, p[rows]]
            depth[rows, i] = depth[rows, p[rows]] + 1
        words = -(-t // 32)
        bits = torch.zeros((b, t, words * 32), dtype=torch.int64)
        bits[:, :, :t] = sees.long()
        bits = (bits.view(b, t, words, 32) << torch.arange(32)).sum(-1)
        st["mask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).to(DEV)
        st["pos"] = st["lens"][:, None] + depth.to(DEV)
    elif case["op"] == "write":
        st["pos"] = st["lens"][:, None] + torch.arange(t, dtype=torch.int32, device=DEV)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:  # the handles that a serving loop keeps: arguments bound once, with their buffers
        import channel_token_sparse_b200 as ds
        if case["op"] in ("write", "step"):
            st["write"] = ds.PreparedWriteKV(
                st["q_in"], st["k_in"], st["v_in"], st["k"], st["v"], starts=st["lens"], positions=st["pos"],
                q_weight=st["qw"], k_weight=st["kw"], eps=EPS, inv_freq=st["inv_freq"],
                rope=ds.DS_ROPE_INTERLEAVED if case["inter"] else ds.DS_ROPE_HALF, k_scale=st["ks"], v_scale=st["vs"],
                block_table=st["table"])
        if case["op"] in ("tree", "step"):
            q = st["write"].q_out if case["op"] == "step" else st["q"]
            st["tree"] = ds.PreparedTreeDecode(
                q, st["k"], st["v"], st["longest"], mask=st["mask"], seq_lens=st["lens"] if case["ragged"] else None,
                k_scale=st["ks"], v_scale=st["vs"], block_table=st["table"], out_dtype=st["io"])
    return st


# ------------------------------------------------------------------ plain forms

def _rows(st, t):
    """Flat cache rows [b, t] (before the head) of the new tokens: row * stride and the head's stride."""
    b = st["lens"].shape[0]
    at = st["lens"].long()[:, None] + torch.arange(t, device=DEV)
    if st["table"] is None:
        return torch.arange(b, device=DEV)[:, None].expand(b, t), at
    page = st["case"]["page"]
    return st["table"].long().gather(1, at // page), at % page


def _dense(cache, table):
    """The cache as [b, hkv, tokens, ...], whatever its layout."""
    if table is None:
        return cache
    x = cache.view(torch.uint8) if cache.dtype == E4M3 else cache
    x = x[table.long()].transpose(1, 2)
    x = x.reshape(x.shape[:2] + (-1,) + x.shape[4:])
    return x.view(E4M3) if cache.dtype == E4M3 else x


def _values(cache, scale, table):
    x = _dense(cache, table).float()
    return x if scale is None else x * _dense(scale, table)[..., None]


def _normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(x, pos, inv_freq, inter):
    angle = pos.double()[:, :, None] * inv_freq.double()
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    half = inv_freq.shape[0]
    y = x.clone()
    if inter:
        a, c = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - c * sin, c * cos + a * sin
    else:
        a, c = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - c * sin, c * cos + a * sin
    return y


def _put(cache, scale, at, x):
    i, r = at
    if scale is None:
        cache[i, :, r] = x.to(cache.dtype)
        return
    sc = (x.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
    cache.view(torch.uint8)[i, :, r] = (x / sc[..., None]).to(E4M3).view(torch.uint8)
    scale[i, :, r] = sc


def _plain_write(st):
    case = st["case"]
    q, k = (_rotated(_normed(st[n], st[w]), st["pos"], st["inv_freq"], case["inter"])
            for n, w in (("q_in", "qw"), ("k_in", "kw")))
    at = _rows(st, case["t"])
    _put(st["k"], st["ks"], at, k)
    _put(st["v"], st["vs"], at, st["v_in"].float())
    return q.to(st["io"])


def _visible(st, tokens):
    """[b, t, tokens]: the prefix, and the nodes that the mask shows."""
    t = st["case"]["t"]
    at = torch.arange(tokens, device=DEV)[None, :] - st["lens"].long()[:, None]
    node = at.clamp(0, t - 1)
    bits = (st["mask"][:, :, :, None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
    bits = bits.reshape(bits.shape[0], t, -1)
    sees = bits.gather(2, node[:, None, :].expand(-1, t, -1)) != 0
    return (at < 0)[:, None, :] | (sees & ((at >= 0) & (at < t))[:, None, :])


def _plain_tree(st, q):
    b, t, hq, d = q.shape
    k, v = _values(st["k"], st["ks"], st["table"]), _values(st["v"], st["vs"], st["table"])
    hkv, g, n = k.shape[1], hq // k.shape[1], min(k.shape[2], st["longest"] + t)
    k, v = k[:, :, :n], v[:, :, :n]
    x = q.float().view(b, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * g, d)
    score = (x @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(b, hkv, t, g, n)
    score.masked_fill_(~_visible(st, n)[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hkv, t * g, n) @ v).view(b, hkv, t, g, d) / torch.where(total > 0, total, 1.0)
    return o.permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(st["io"])


def _state(st):
    """The updated cache: its values (8-bit codes as the numbers they are, beside their scales)."""
    return [st["k"], st["v"]] + ([] if st["ks"] is None else [st["ks"], st["vs"]])


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import channel_token_sparse_b200 as ds
        if op == "write":
            return {"q": st["write"](), "cache": _state(st)}
        if op == "read":
            return list(ds.read_kv(st["k"], st["v"], st["ks"], st["vs"], st["case"]["s"], block_table=st["table"],
                                   dtype=torch.bfloat16))
        if op == "tree":
            return st["tree"]()
        q = st["write"]()
        return {"q": q, "out": st["tree"](), "cache": _state(st)}
    if op == "write":
        return {"q": _plain_write(st), "cache": _state(st)}
    if op == "read":
        n = st["case"]["s"]
        return [_values(st[c], st[c + "s"], st["table"])[:, :, :n].to(torch.bfloat16) for c in "kv"]
    if op == "tree":
        return _plain_tree(st, st["q"])
    q = _plain_write(st)
    return {"q": q, "out": _plain_tree(st, q), "cache": _state(st)}


# ------------------------------------------------------------------ 64 bits

def _exact_heads(x, w, pos, inv_freq, inter):
    """Norm and rotation as complex numbers: (a + ic) e^{i angle}."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    if inv_freq is None:
        return x
    n = inv_freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[..., None] * inv_freq.double())
    head, tail = x[..., :2 * n], x[..., 2 * n:]
    pair = head.unflatten(-1, (n, 2)) if inter else head.unflatten(-1, (2, n)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, :, None, :])
    z = z if inter else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), tail], -1)


def _exact_cache(st, name, x):
    """The cache after the write, in 64 bits; 8-bit codes as they are before their rounding."""
    case = st["case"]
    cache = st[name].double()
    scale = None if st[name + "s"] is None else st[name + "s"].double()
    for b, n in enumerate(_lengths(case)):
        for i in range(case["t"]):
            r = n + i
            at = (b, slice(None), r) if st["table"] is None else (st["host_table"][b][r // case["page"]], slice(None), r % case["page"])
            if scale is None:
                cache[at] = x[b, i]
            else:
                sc = (x[b, i].abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
                scale[at] = sc
                cache[at] = x[b, i] / sc[:, None]
    return cache, scale


def exact(case, seed):
    if case["op"] in ("write", "step") and case["b"] * case["t"] > 20000:
        return None
    st = _inputs(case, seed)
    if st["table"] is not None:
        st["host_table"] = st["table"].tolist()
    result = {}
    if case["op"] in ("write", "step"):
        q = _exact_heads(st["q_in"], st["qw"], st["pos"], st["inv_freq"], case["inter"])
        k = _exact_heads(st["k_in"], st["kw"], st["pos"], st["inv_freq"], case["inter"])
        (kc, ks), (vc, vs) = _exact_cache(st, "k", k), _exact_cache(st, "v", st["v_in"].double())
        result = {"q": q, "cache": [kc, vc] + ([] if ks is None else [ks, vs])}
        if case["op"] == "write":
            return result
        if ks is None:  # the attention reads what was written: rounded to the cache's type
            kc, vc = kc.to(st["io"]).double(), vc.to(st["io"]).double()
        else:
            kc, vc = (c.float().to(E4M3).double() * sc.float().double()[..., None] for c, sc in ((kc, ks), (vc, vs)))
        q = q.to(st["io"]).double()
    elif case["op"] == "read":
        kc, vc = (st[c].double() * st[c + "s"].double()[..., None] for c in "kv")
        if st["table"] is None:
            return [kc[:, :, :case["s"]], vc[:, :, :case["s"]]]
        return [torch.stack([c[row].transpose(0, 1).flatten(1, 2)[:, :case["s"]] for row in st["table"].long()])
                for c in (kc, vc)]
    else:
        kc = vc = None
        q = st["q"].double()
    b, t, hq, d = q.shape
    hkv = case["hkv"]
    g = hq // hkv
    out = torch.zeros((b, t, hq, d), dtype=torch.float64, device=DEV)
    shifts = torch.arange(32, dtype=torch.int32, device=DEV)
    for e, n in enumerate(_lengths(case)):
        sees = ((st["mask"][e][:, :, None] >> shifts) & 1).reshape(t, -1)[:, :t].bool()
        seen = torch.cat([torch.ones((t, n), dtype=torch.bool, device=DEV), sees], 1)
        bias = torch.where(seen, 0.0, -math.inf).double().repeat_interleave(g, 0)
        for h in range(hkv):
            rows = []
            for c, done in (("k", kc), ("v", vc)):
                src = st[c] if done is None else done
                if st["table"] is None:
                    x = src[e, h, :n + t]
                    sc = None if done is not None or st[c + "s"] is None else st[c + "s"][e, h, :n + t]
                else:
                    ids = st["table"][e, : -(-(n + t) // case["page"])].long()
                    x = (src.view(torch.uint8) if src.dtype == E4M3 else src)[ids, h].flatten(0, 1)[:n + t]
                    x = x.view(E4M3) if src.dtype == E4M3 else x
                    sc = None if done is not None or st[c + "s"] is None else st[c + "s"][ids, h].flatten()[:n + t]
                rows.append(x.double() if sc is None else x.double() * sc.double()[:, None])
            w = torch.softmax(q[e, :, h * g:(h + 1) * g].reshape(t * g, d) @ rows[0].T / math.sqrt(d) + bias, -1)
            out[e, :, h * g:(h + 1) * g] = (w @ rows[1]).view(t, g, d)
    if case["op"] == "step":
        return dict(result, out=out)
    return out
