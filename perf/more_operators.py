"""What is measured of the operators that put new tokens into a dense layer's cache and check drafted ones:
csa_qk_rope, csa_kv_append and csa_tree_attn.

With `own` false `run` computes them from elementary torch operations in fp32 (angles in fp64); with `own` true
it makes the library's calls.  `exact` is each operator's definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
BASE = 10000.0


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one new token of a layer with normed queries and keys, halves of a head rotated against each other
        dict(name="rope_token", op="rope", n=1, q_heads=32, k_heads=8, dim=128, rope=128, last=False, halves=True,
             norm=True, far=65536, dtype="bf16"),
        # a decode batch's latent queries and shared row for the sparse step: the last 64 of 576 dims rotated in pairs
        dict(name="rope_latent", op="rope", n=64, q_heads=64, k_heads=1, dim=576, rope=64, last=True, halves=False,
             norm=False, far=1 << 20, dtype="bf16"),
        # fp32 heads of 80 dims of which 20 rotate, a ragged number of tokens
        dict(name="rope_odd", op="rope", n=331, q_heads=5, k_heads=3, dim=80, rope=20, last=False, halves=True,
             norm=True, far=8192, dtype="f32"),
        # a prefill chunk's queries and keys
        dict(name="rope_prefill", op="rope", n=16384, q_heads=32, k_heads=8, dim=128, rope=128, last=False, halves=True,
             norm=True, far=65536, dtype="bf16"),
        # one request, one token: its key rotated and written to its page beside its value
        dict(name="append_token", op="append", b=1, s=1, q_heads=0, kv_heads=8, dim=128, v=True, rope=128, last=False,
             halves=True, norm=False, kv="bf16", place="table", block=64, lo=1023, hi=1023, ragged=False),
        # a decode batch's drafted tokens into an 8-bit cache, their queries rotated in the same call, some padding
        dict(name="append_drafts", op="append", b=64, s=8, q_heads=32, kv_heads=4, dim=128, v=True, rope=128, last=False,
             halves=True, norm=True, kv="fp8", place="table", block=64, lo=1024, hi=65536, ragged=True),
        # indexer keys of a long prompt into the FP8 key pool, rows by slot mapping
        dict(name="append_keys", op="append", b=1, s=131072, q_heads=0, kv_heads=1, dim=128, v=False, rope=64, last=True,
             halves=False, norm=True, kv="fp8", place="slots", block=128, lo=131072, hi=131072, ragged=False),
        # prefill chunks of several requests into a paged bf16 cache, queries included
        dict(name="append_prefill", op="append", b=4, s=4096, q_heads=32, kv_heads=8, dim=128, v=True, rope=128,
             last=False, halves=True, norm=True, kv="bf16", place="table", block=64, lo=4096, hi=32768, ragged=False),
        # one request, eight drafts, a short context
        dict(name="tree_token", op="tree", b=1, s=8, heads=32, kv_heads=8, dim=128, lo=1023, hi=1023, pad=0, ragged=False,
             win=0, kv="bf16", block=64),
        # a ragged decode batch with trees of up to 16 drafts over long contexts
        dict(name="tree_ragged", op="tree", b=64, s=16, heads=32, kv_heads=4, dim=128, lo=1024, hi=65536, pad=0,
             ragged=True, win=0, kv="bf16", block=64),
        # wide trees over a cache held in 8 bits
        dict(name="tree_fp8", op="tree", b=16, s=64, heads=64, kv_heads=8, dim=128, lo=8192, hi=16384, pad=0, ragged=False,
             win=0, kv="fp8", block=128),
        # small heads, small pages, an odd number of drafts, padding requests, a sliding window
        dict(name="tree_window", op="tree", b=48, s=21, heads=16, kv_heads=8, dim=64, lo=1, hi=8192, pad=5, ragged=True,
             win=1000, kv="bf16", block=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "tree"])
    if op != "tree":
        dim = rng.choice([64, 80, 128, 128, 192, 256, 576])
        halves = rng.random() < 0.6
        rope = rng.choice([dim, 64, 32, 20, dim // 2])
        shape = dict(dim=dim, rope=min(rope, dim), last=rng.random() < 0.5, halves=halves, norm=rng.random() < 0.6)
    if op == "rope":
        q, k, dt = rng.choice([1, 5, 16, 32, 64]), rng.choice([0, 1, 3, 8]), rng.choice(["bf16", "bf16", "f32"])
        room = 16384 * 40 * 128 * 2 // ((q + k) * dim * (2 if dt == "bf16" else 4))
        return dict(op=op, n=_log(rng, 1, min(100000, max(2, room))), q_heads=q, k_heads=k, dtype=dt,
                    far=rng.choice([100, 65536, 1 << 20]), **shape)
    if op == "append":
        s, hk, q = rng.choice([1, 1, 4, 7, _log(rng, 1, 8192)]), rng.choice([1, 2, 8]), rng.choice([0, 0, 1, 3, 8])
        q, v, kv = q * hk, rng.random() < 0.75, rng.choice(["bf16", "bf16", "fp8", "f32"])
        room = 16384 * 48 * 128 * 2 // (s * (q + hk * (2 if v else 1)) * dim * (4 if kv == "f32" else 2))
        hi = _log(rng, s, 65536)
        return dict(op=op, b=_log(rng, 1, max(2, min(256, room))), s=s, q_heads=q, kv_heads=hk, v=v, kv=kv,
                    place=rng.choice(["table", "table", "slots"]), block=rng.choice([16, 48, 64, 128]),
                    lo=max(s, hi // rng.choice([1, 2, 64])), hi=hi, ragged=rng.random() < 0.4, **shape)
    kv = rng.choice(["bf16", "bf16", "fp8"])
    dim = 128 if kv == "fp8" else rng.choice([64, 128, 128, 256])
    hk, group, s = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 5, 8, 16, 33, 64, 100])
    most = (1 << 36) // (s * hk * group * dim)
    hi = _log(rng, s, min(65536, most))
    b = _log(rng, 1, max(1, min(128, (1 << 30) // (hi * hk * dim), most // hi)))
    ragged = rng.random() < 0.5
    return dict(op=op, b=b, s=s, heads=hk * group, kv_heads=hk, dim=dim, ragged=ragged,
                lo=max(1 if ragged else s, hi // rng.choice([1, 2, 64])), hi=hi, pad=rng.choice([0, 0, b // 4]),
                win=rng.choice([0, 0, 0, 128, 1000]), kv=kv, block=rng.choice([16, 48, 64, 128, 1024]))


def _lengths(case):
    """Context lengths, new tokens included; the last `pad` requests of an attention case are padding without a row."""
    r = random.Random(case["b"] * 1000003 + case["lo"] * 101 + case["hi"])
    pad = case.get("pad", 0)
    return [0 if i >= case["b"] - pad else r.randint(case["lo"], case["hi"]) for i in range(case["b"])]


def _counts(case):
    """How many of a request's S tokens are real (at most its length)."""
    r = random.Random(case["s"] * 7919 + case["b"])
    return [min(x, r.randint(1, case["s"]) if case["ragged"] else case["s"]) for x in _lengths(case)]


def _esize(dtype):
    return {"bf16": 2, "f32": 4, "fp8": 1}[dtype]


def work(case):
    if case["op"] == "rope":
        heads, e = case["n"] * (case["q_heads"] + case["k_heads"]), _esize(case["dtype"])
        return {"bytes": 2 * heads * case["dim"] * e + 4 * case["n"], "flops": heads * (4 * case["dim"] + 3 * case["rope"])}
    if case["op"] == "append":
        n, q, hk, d = sum(_counts(case)), case["q_heads"], case["kv_heads"], case["dim"]
        e, kinds = 4 if case["kv"] == "f32" else 2, 2 if case["v"] else 1
        return {"bytes": n * (2 * q * d * e + kinds * hk * (d * e + d * _esize(case["kv"]) + (4 if case["kv"] == "fp8" else 0))),
                "flops": n * ((q + hk) * (4 * d + 3 * case["rope"]) + (3 * kinds * hk * d if case["kv"] == "fp8" else 0))}
    s, h, g, d, win = case["s"], case["heads"], case["kv_heads"], case["dim"], case["win"]
    rows = pairs = 0
    for length, count in zip(_lengths(case), _counts(case)):
        prefix = length - count
        rows += min(prefix, win - 1) + count if win else length
        pairs += count * ((min(prefix, win - 1) if win else prefix) + (count + 1) / 2)
    e = 2 * d * 2 if case["kv"] == "bf16" else 2 * (d + 4)
    return {"bytes": int(rows * g * e + case["b"] * s * (h * (4 * d + 4) + 8 * -(-s // 64))), "flops": int(4 * pairs * h * d)}


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _to_e4m3(y, amax):
    """Codes and scale of y, whose last dims share the scale made of amax (kept dims)."""
    scale = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -126), torch.ones_like(amax))
    return (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = _gen(seed)
    return {"rope": _prepare_rope, "append": _prepare_append, "tree": _prepare_tree}[case["op"]](case, g, seed)


def _weight(g, case, dt):
    return (1 + 0.1 * _randn(g, case["dim"])).to(dt) if case["norm"] else None


def _prepare_rope(case, g, seed):
    n, d, dt = case["n"], case["dim"], _dtype(case["dtype"])
    st = dict(case=case, pos=torch.randint(0, case["far"], (n,), generator=g, device=DEV, dtype=torch.int32),
              q=_randn(g, n, case["q_heads"], d).to(dt), qw=_weight(g, case, dt),
              k=_randn(g, n, case["k_heads"], d).to(dt) if case["k_heads"] else None,
              kw=_weight(g, case, dt) if case["k_heads"] else None)
    if own:
        from compressed_sparse_attention_indexer_gb300 import csa
        st["op"] = csa.QkRope(st["q"], st["k"], st["pos"], q_weight=st["qw"], k_weight=st["kw"], norm=case["norm"],
                              eps=1e-6, rope_dim=case["rope"], rope_at=_at(case), halves=case["halves"], base=BASE)
    return st


def _at(case):
    """First rotated dim."""
    return case["dim"] - case["rope"] if case["last"] else 0


def _tables(lens, counts, blk, seed, whole):
    """A block table in shuffled order; not whole: of the blocks that the new tokens fall in alone."""
    stride = max(1, max(-(-x // blk) for x in lens))
    table = torch.full((len(lens), stride), -1, dtype=torch.int32)
    spans = [(0 if whole else (x - c) // blk, -(-x // blk)) for x, c in zip(lens, counts)]
    total = max(1, sum(b - a for a, b in spans))
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = 0
    for i, (a, b) in enumerate(spans):
        table[i, a:b] = perm[at:at + b - a]
        at += b - a
    return table, total


def _prepare_append(case, g, seed):
    b, s, hq, hk, d, blk = (case[x] for x in ("b", "s", "q_heads", "kv_heads", "dim", "block"))
    dt, lens, counts = _dtype(case["kv"]), _lengths(case), _counts(case)
    table, total = _tables(lens, counts, blk, seed, False)
    rows = total * blk
    st = dict(case=case, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), counts=None, table=None, slot=None,
              pos=None, k=_randn(g, b, s, hk, d).to(dt), kw=_weight(g, case, dt))
    st["v"] = _randn(g, b, s, hk, d).to(dt) if case["v"] else None
    st["q"] = _randn(g, b, s, hq, d).to(dt) if hq else None
    st["qw"] = _weight(g, case, dt) if hq else None
    st["q_out"] = torch.zeros_like(st["q"]) if hq else None
    if case["place"] == "table":
        st["table"] = table.to(DEV)
        if case["ragged"]:
            st["counts"] = torch.tensor(counts, dtype=torch.int32, device=DEV)
    else:
        # a scheduler's slot mapping and positions: the new tokens first, padding (-1) behind them
        first = torch.tensor([x - c for x, c in zip(lens, counts)])[:, None]
        r = first + torch.arange(s)
        real = torch.arange(s) < torch.tensor(counts)[:, None]
        block = table.gather(1, (r // blk).clamp_max(table.shape[1] - 1)).long()
        st["slot"] = torch.where(real, block * blk + r % blk, -1).view(-1).to(DEV)
        st["pos"] = r.to(torch.int32).view(-1).to(DEV)
    for name in ("k", "v"):
        st[name + "_pool"] = st[name + "_scale"] = None
        if name == "v" and not case["v"]:
            continue
        x = _randn(g, rows, hk, d)
        if case["kv"] == "fp8":
            codes, scale = _to_e4m3(x, x.abs().amax(2, keepdim=True))
            st[name + "_pool"], st[name + "_scale"] = codes, scale[:, :, 0].contiguous()
        else:
            st[name + "_pool"] = x.to(dt)
    if own:
        from compressed_sparse_attention_indexer_gb300 import csa
        st["op"] = csa.KvAppend(st["k"], st["v"], st["k_pool"], st["v_pool"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                ctx_len=st["lens"] if case["place"] == "table" else None, count=st["counts"],
                                table=st["table"], block=blk if case["place"] == "table" else 0, slot=st["slot"],
                                pos=st["pos"], q=st["q"], q_out=st["q_out"], q_weight=st["qw"], k_weight=st["kw"],
                                norm=case["norm"], eps=1e-6, rope_dim=case["rope"], rope_at=_at(case),
                                halves=case["halves"], base=BASE)
    return st


def _prepare_tree(case, g, seed):
    b, s, h, hk, d, blk = (case[x] for x in ("b", "s", "heads", "kv_heads", "dim", "block"))
    lens, counts = _lengths(case), _counts(case)
    table, total = _tables(lens, counts, blk, seed, True)
    # each draft's parent is an earlier draft of its request, more often a late one, or the context's last token
    gen = torch.Generator().manual_seed(seed)
    sees = torch.zeros(b, s, s, dtype=torch.bool)
    for t in range(s):
        parent = ((torch.rand(b, generator=gen).sqrt() * (t + 1)).long() - 1).clamp_max(t - 1)
        sees[:, t] = torch.where(parent[:, None] >= 0, sees[torch.arange(b), parent.clamp_min(0)], torch.tensor(False))
        sees[:, t, t] = True
    depth = sees.sum(2) - 1
    words = -(-s // 64)
    bits = torch.nn.functional.pad(sees, (0, 64 * words - s)).view(b, s, words, 64).long()
    tree = (bits << torch.arange(64)).sum(3)
    pos = torch.tensor([x - c for x, c in zip(lens, counts)])[:, None] + depth
    st = dict(case=case, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), most=max(lens), table=table.to(DEV),
              tree=tree.to(DEV), counts=torch.tensor(counts, dtype=torch.int32, device=DEV) if case["ragged"] else None,
              pos=pos.to(torch.int32).to(DEV) if case["win"] else None, q=_randn(g, b, s, h, d, dtype=torch.bfloat16),
              scale=d ** -0.5)
    for name in ("k", "v"):
        x = _randn(g, total * blk, hk, d, dtype=torch.bfloat16)
        if case["kv"] == "fp8":
            codes, scale = _to_e4m3(x, x.abs().amax(2, keepdim=True).float())
            st[name], st[name + "_scale"] = codes.view(torch.uint8), scale[:, :, 0].contiguous()
        else:
            st[name], st[name + "_scale"] = x, None
    if own:
        from compressed_sparse_attention_indexer_gb300 import csa
        st["op"] = csa.TreeAttention(st["q"], st["k"], st["v"], st["lens"], st["tree"], count=st["counts"], pos=st["pos"],
                                     table=st["table"], block=blk, k_scale=st["k_scale"], v_scale=st["v_scale"],
                                     win=case["win"], scale=st["scale"], max_len=max(1, max(lens)))
    return st


# ---------------------------------------------------------------------------
# one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return st["op"]()
    return {"rope": _plain_rope, "append": _plain_append, "tree": _plain_tree}[op](st)


def _plain_heads(case, x, weight, pos):
    """Heads [n, heads, dim], normed and rotated, in fp32."""
    y = x.float()
    if case["norm"]:
        y = y * torch.rsqrt((y * y).mean(2, keepdim=True) + 1e-6) * weight.float()
    r, at = case["rope"], _at(case)
    theta = BASE ** (-2.0 * torch.arange(r // 2, dtype=torch.float64, device=DEV) / r)
    angle = pos.double()[:, None, None] * theta
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    part = y[:, :, at:at + r]
    if case["halves"]:
        a, b = part[:, :, :r // 2], part[:, :, r // 2:]
        part = torch.cat([a * cos - b * sin, a * sin + b * cos], 2)
    else:
        a, b = part[:, :, 0::2], part[:, :, 1::2]
        part = torch.stack([a * cos - b * sin, a * sin + b * cos], 3).flatten(2)
    return torch.cat([y[:, :, :at], part, y[:, :, at + r:]], 2)


def _plain_rope(st):
    case = st["case"]
    got = {"q": _plain_heads(case, st["q"], st["qw"], st["pos"]).to(st["q"].dtype)}
    if st["k"] is not None:
        got["k"] = _plain_heads(case, st["k"], st["kw"], st["pos"]).to(st["k"].dtype)
    return got


def _plain_append(st):
    case = st["case"]
    b, s, hk, d, blk = (case[x] for x in ("b", "s", "kv_heads", "dim", "block"))
    if st["slot"] is None:
        count = (torch.full_like(st["lens"], s) if st["counts"] is None else st["counts"]).long()[:, None]
        t = torch.arange(s, device=DEV)
        pos = st["lens"].long()[:, None] - count + t
        at = (pos // blk).clamp_max(st["table"].shape[1] - 1)
        slot = torch.where(t < count, st["table"].long().gather(1, at) * blk + pos % blk, -1).view(-1)
        pos = pos.view(-1)
    else:
        slot, pos = st["slot"], st["pos"]
    real = (slot >= 0).nonzero()[:, 0]
    to, pos = slot[real], pos[real]
    got = {}
    for name in ("k", "v"):
        x = st[name]
        if x is None:
            continue
        x = x.view(b * s, hk, d)[real]
        y = _plain_heads(case, x, st["kw"], pos) if name == "k" else x.float()
        pool, scale = st[name + "_pool"], st[name + "_scale"]
        if scale is not None:
            codes, sc = _to_e4m3(y, y.abs().amax(2, keepdim=True))
            pool.view(torch.uint8)[to] = codes.view(torch.uint8)
            scale[to] = sc[:, :, 0]
            got[name + "_scale"] = scale
        else:
            pool[to] = y.to(pool.dtype)
        got[name] = pool
    if st["q"] is not None:
        q = st["q"].view(b * s, -1, d)[real]
        st["q_out"].view(b * s, -1, d)[real] = _plain_heads(case, q, st["qw"], pos).to(q.dtype)
        got["q"] = st["q_out"]
    return got


def _plain_tree(st):
    case = st["case"]
    b, s, h, hk, d, blk = (case[x] for x in ("b", "s", "heads", "kv_heads", "dim", "block"))
    length = max(1, st["most"])
    r = torch.arange(length, device=DEV)
    t = torch.arange(s, device=DEV)
    step = max(1, (1 << 29) // (h * s * length))
    outs, lses = [], []
    for i in range(0, b, step):
        of = slice(i, i + step)
        table, lens = st["table"][of].long(), st["lens"][of].long()
        nb = table.shape[0]
        count = torch.full_like(lens, s) if st["counts"] is None else st["counts"][of].long()
        prefix = (lens - count)[:, None, None]
        rows = table.clamp_min(0)[:, r // blk] * blk + r % blk                                  # [nb, length]
        bits = ((st["tree"][of][:, :, t // 64] >> (t % 64)) & 1).bool()                         # [nb, s, s]
        draft = (r - prefix).expand(nb, s, length)                                              # the row's draft
        seen = (draft < 0) | ((draft < count[:, None, None]) & bits.gather(2, draft.clamp(0, s - 1)))
        if case["win"]:
            seen = seen & ((draft >= 0) | (r > st["pos"][of].long()[:, :, None] - case["win"]))
        seen = seen & (t[:, None] < count[:, None, None])
        seen = seen[:, None, :, None, :]                                                        # [nb, 1, s, 1, length]

        def pool(name):
            x = st[name][rows]
            x = x.float() if st[name + "_scale"] is None else \
                x.view(torch.float8_e4m3fn).float() * st[name + "_scale"][rows][..., None]
            return x.permute(0, 2, 1, 3)                                                        # [nb, hk, length, d]

        q = st["q"][of].float().view(nb, s, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(nb, hk, -1, d)
        sc = (q @ pool("k").transpose(2, 3) * st["scale"]).view(nb, hk, s, h // hk, length)
        sc = torch.where(seen, sc, -math.inf)
        top = sc.amax(4, keepdim=True)
        top = torch.where(top > -math.inf, top, 0.0)
        p = torch.exp(sc - top)
        total = p.sum(4, keepdim=True)
        out = (p.view(nb, hk, -1, length) @ pool("v")).view(nb, hk, s, h // hk, d) / torch.where(total > 0, total, 1.0)
        lse = (top + torch.log(total))[..., 0]
        outs.append(out.permute(0, 2, 1, 3, 4).reshape(nb, s, h, d).to(torch.bfloat16))
        lses.append(lse.permute(0, 2, 1, 3).reshape(nb, s, h))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "append": _exact_append, "tree": _exact_tree}[case["op"]](case, st)


def _exact_heads(case, x, weight, pos):
    y = x.double()
    if case["norm"]:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6) * weight.double()
    r, at = case["rope"], _at(case)
    i = torch.arange(r // 2, device=DEV)
    first = at + (i if case["halves"] else 2 * i)
    second = first + (r // 2 if case["halves"] else 1)
    angle = pos.double()[:, None] * torch.pow(torch.tensor(BASE, dtype=torch.float64, device=DEV), -2 * i.double() / r)
    turn = torch.polar(torch.ones_like(angle), angle)
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rope(case, st):
    got = {"q": _exact_heads(case, st["q"], st["qw"], st["pos"])}
    if case["k_heads"]:
        got["k"] = _exact_heads(case, st["k"], st["kw"], st["pos"])
    return got


def _nearest_e4m3(v):
    """v (|v| <= 448) rounded to the nearest E4M3 value, ties to even, in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _exact_append(case, st):
    b, s, blk = case["b"], case["s"], case["block"]
    got = {}
    for name in ("k", "v"):
        if st[name] is not None:
            if st[name + "_scale"] is not None:
                got[name + "_scale"] = st[name + "_scale"].double()
            got[name] = st[name + "_pool"].double()
    if st["q"] is not None:
        got["q"] = st["q_out"].double()
    for i, (length, count) in enumerate(zip(_lengths(case), _counts(case))):
        if st["slot"] is not None:
            to, pos = st["slot"][i * s:i * s + count], st["pos"][i * s:i * s + count]
        else:
            pos = torch.arange(length - count, length, device=DEV)
            to = st["table"][i].long()[pos // blk] * blk + pos % blk
        for name in ("k", "v"):
            if st[name] is None:
                continue
            x = st[name][i, :count]
            y = _exact_heads(case, x, st["kw"], pos) if name == "k" else x.double()
            if st[name + "_scale"] is not None:
                most = y.abs().max(2, keepdim=True).values
                scale = torch.where(most == 0, 1.0, torch.clamp(most / E4M3_MAX, min=2.0 ** -126))
                got[name + "_scale"][to] = scale[:, :, 0]
                y = _nearest_e4m3(y / scale)
            got[name][to] = y
        if st["q"] is not None:
            got["q"][i, :count] = _exact_heads(case, st["q"][i, :count], st["qw"], pos)
    return got


def _exact_tree(case, st):
    b, s, h, hk, d, blk, win = (case[x] for x in ("b", "s", "heads", "kv_heads", "dim", "block", "win"))
    if work(case)["flops"] > 6e11:
        return None
    out = torch.zeros(b, s, h, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64, device=DEV)
    for i, (length, count) in enumerate(zip(_lengths(case), _counts(case))):
        if not count:
            continue
        pages = st["table"][i, :-(-length // blk)].long()
        rows = (pages[:, None] * blk + torch.arange(blk, device=DEV)).reshape(-1)[:length]
        k, v = st["k"][rows], st["v"][rows]
        if case["kv"] == "fp8":
            k = k.view(torch.float8_e4m3fn).double() * st["k_scale"][rows].double()[:, :, None]
            v = v.view(torch.float8_e4m3fn).double() * st["v_scale"][rows].double()[:, :, None]
        k, v = k.double(), v.double()
        prefix = length - count
        masks = st["tree"][i].tolist()
        seen = torch.zeros(count, length, dtype=torch.bool)
        for t in range(count):
            first = max(0, int(st["pos"][i, t]) - win + 1) if win else 0
            seen[t, first:prefix] = True
            for j in range(count):
                seen[t, prefix + j] = (masks[t][j // 64] >> (j % 64)) & 1 == 1
        seen = seen.to(DEV).repeat_interleave(h // hk, 0)
        for g in range(hk):
            of = slice(g * (h // hk), (g + 1) * (h // hk))
            q = st["q"][i, :count, of].double().reshape(-1, d)
            sc = (torch.mm(q, k[:, g].t()) * st["scale"]).masked_fill(~seen, -math.inf)
            total = torch.logsumexp(sc, 1)
            lse[i, :count, of] = total.view(count, -1)
            out[i, :count, of] = torch.mm(torch.exp(sc - total[:, None]), v[:, g]).view(count, -1, d)
    return {"out": out, "lse": lse}
