"""What is measured of the operators around the sparse decode step: csa_norm_rows, csa_fp8_matmul and csa_paged_attn.

With `own` false `run` computes them from elementary torch operations in fp32; with `own` true it makes the
library's calls.  `exact` is each operator's definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one new token's hidden row: the residual is added, the 8-bit row feeds the next product
        dict(name="norm_token", op="norm", n=1, width=4096, dtype="bf16", norm=True, residual=True, out=False, codes=True),
        # indexer keys of a long prompt, each 128-wide row to E4M3 with one scale (the FP8 key pool's format)
        dict(name="norm_keys", op="norm", n=131072, width=128, dtype="bf16", norm=True, residual=False, out=False,
             codes=True),
        # fp32 rows of an odd width quantised without a norm (the last block is short)
        dict(name="quantise_odd", op="norm", n=4097, width=1000, dtype="f32", norm=False, residual=False, out=False,
             codes=True),
        # a prefill chunk's hidden rows, the norm's output wanted in both forms (product and router)
        dict(name="norm_prefill", op="norm", n=16384, width=7168, dtype="bf16", norm=True, residual=True, out=True,
             codes=True),
        # one token's indexer queries: 64 heads x 128 from a 1536-wide latent
        dict(name="product_token", op="mm", m=1, n=8192, k=1536, out="bf16"),
        # a decode batch's attention queries: 64 heads x 576
        dict(name="product_batch", op="mm", m=64, n=36864, k=1536, out="bf16"),
        # odd sizes: a ragged batch, a short last block of k, an fp32 output (head weights, logits)
        dict(name="product_odd", op="mm", m=331, n=1100, k=7000, out="f32"),
        # a prefill chunk's indexer queries from the hidden rows
        dict(name="product_prefill", op="mm", m=8192, n=8192, k=7168, out="bf16"),
        # one request, one token, a short context
        dict(name="attn_token", op="attn", b=1, s=1, heads=32, kv_heads=8, dim=128, lo=1023, hi=1023, pad=0, win=0,
             kv="bf16", block=64),
        # a ragged decode batch with long contexts (the lengths of the benchmark workload)
        dict(name="attn_ragged", op="attn", b=64, s=1, heads=32, kv_heads=4, dim=128, lo=1024, hi=65536, pad=0, win=0,
             kv="bf16", block=64),
        # the cache held in 8 bits
        dict(name="attn_fp8", op="attn", b=32, s=1, heads=64, kv_heads=8, dim=128, lo=16384, hi=32768, pad=0, win=0,
             kv="fp8", block=128),
        # a few tokens per request, small heads, small pages, padding requests without a row
        dict(name="attn_multi", op="attn", b=48, s=4, heads=16, kv_heads=8, dim=64, lo=1, hi=8192, pad=5, win=0,
             kv="bf16", block=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "mm", "attn"])
    if op == "norm":
        width = rng.choice([128, 576, _log(rng, 1, 16384), 8 * _log(rng, 16, 2048)])
        n = _log(rng, 1, max(2, min(200000, 16384 * 7168 // width)))
        out, codes = rng.choice([(False, True), (True, False), (True, True)])
        return dict(op=op, n=n, width=width, dtype=rng.choice(["bf16", "bf16", "f32"]), norm=rng.random() < 0.8,
                    residual=rng.random() < 0.5, out=out, codes=codes)
    if op == "mm":
        n, k = _log(rng, 1, 36864), rng.choice([_log(rng, 1, 16384), 128 * _log(rng, 1, 128)])
        m = _log(rng, 1, max(2, min(16384, 8192 * 8192 * 7168 // (n * k))))
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(["bf16", "bf16", "f32"]))
    kv = rng.choice(["bf16", "bf16", "fp8"])
    dim = 128 if kv == "fp8" else rng.choice([64, 128, 128, 256])
    kv_heads, group, s = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 1, 1, 2, 3, 4])
    hi = _log(rng, 1, 65536)
    b = _log(rng, 1, max(2, min(128, (1 << 30) // (hi * kv_heads * dim))))
    return dict(op=op, b=b, s=s, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, lo=max(1, hi // rng.choice([1, 2, 64])),
                hi=hi, pad=rng.choice([0, 0, b // 4]), win=rng.choice([0, 0, 0, 128, 1000]), kv=kv,
                block=rng.choice([16, 48, 64, 128, 1024]))


def _lengths(case):
    """Context lengths of an attention case; the last `pad` requests are padding without a row."""
    r = random.Random(case["b"] * 1000003 + case["lo"] * 101 + case["hi"])
    return [0 if i >= case["b"] - case["pad"] else r.randint(case["lo"], case["hi"]) for i in range(case["b"])]


def work(case):
    if case["op"] == "norm":
        n, w, e = case["n"], case["width"], 2 if case["dtype"] == "bf16" else 4
        per = e + (2 * e if case["residual"] else 0) + (e if case["out"] else 0) + (1 if case["codes"] else 0)
        return {"bytes": n * w * per + (w * e if case["norm"] else 0) + (n * -(-w // 128) * 4 if case["codes"] else 0),
                "flops": 6 * n * w}
    if case["op"] == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // 128)
        return {"bytes": m * k + n * k + 4 * (m * kb + -(-n // 128) * kb) + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * n * k}
    s, h, g, d, win = case["s"], case["heads"], case["kv_heads"], case["dim"], case["win"]
    rows = pairs = 0
    for length in _lengths(case):
        rows += min(length, win + s - 1) if win else length
        for pos in range(max(0, length - s), length):
            pairs += min(pos + 1, win) if win else pos + 1
    e = 2 * d * 2 if case["kv"] == "bf16" else 2 * (d + 4)
    return {"bytes": rows * g * e + case["b"] * s * h * (4 * d + 4), "flops": 4 * pairs * h * d}


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)


def _blocks(x):
    """[n, k] -> [n, ceil(k / 128), 128], the last block filled up with zeros."""
    n, k = x.shape
    kb = -(-k // 128)
    if kb * 128 != k:
        x = torch.nn.functional.pad(x, (0, kb * 128 - k))
    return x.reshape(n, kb, 128)


def _to_e4m3(y, amax):
    """Codes and scale of y, whose last dims share the scale made of amax (kept dims)."""
    scale = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -126), torch.ones_like(amax))
    return (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _quantise_rows(x):
    """[n, k] -> codes [n, k] and scale [n, ceil(k / 128)]."""
    y = _blocks(x)
    codes, scale = _to_e4m3(y, y.abs().amax(2, keepdim=True))
    return codes.view(torch.uint8).reshape(x.shape[0], -1)[:, :x.shape[1]].contiguous(), scale[:, :, 0].contiguous()


def _padded(codes):
    """Codes whose rows start on 16-byte boundaries, as the library's pools have them."""
    k = codes.shape[1]
    if k % 16:
        codes = torch.nn.functional.pad(codes, (0, 16 - k % 16))
    return codes[:, :k]


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        return _prepare_norm(case, g)
    return _prepare_mm(case, g) if case["op"] == "mm" else _prepare_attn(case, g)


def _rows(gen, n, width, dtype):
    """Rows [n, width] that start on 16-byte boundaries."""
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    return _randn(gen, n, -(-width // unit) * unit).to(dtype)[:, :width]


def _prepare_norm(case, g):
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    n, width = case["n"], case["width"]
    st = dict(case=case, x=_rows(g, n, width, dt), residual=_rows(g, n, width, dt) if case["residual"] else None,
              weight=(1 + 0.1 * _randn(g, width)).to(dt) if case["norm"] else None, eps=1e-6)
    if own:
        from compressed_sparse_attention_indexer_gb300 import csa
        st["op"] = csa.NormRows(st["x"], weight=st["weight"], residual=st["residual"], norm=case["norm"], eps=st["eps"],
                                out=case["out"], codes=case["codes"])
    return st


def _prepare_mm(case, g):
    m, n, k = case["m"], case["n"], case["k"]
    a, sa = _quantise_rows(_randn(g, m, k))
    nb = -(-n // 128)
    w = _blocks(_randn(g, n, k) * k ** -0.5)
    kb = w.shape[1]
    w = torch.nn.functional.pad(w, (0, 0, 0, 0, 0, nb * 128 - n)).view(nb, 128, kb, 128)
    codes, sb = _to_e4m3(w, w.abs().amax((1, 3), keepdim=True))
    b = codes.view(torch.uint8).view(nb * 128, kb * 128)[:n, :k].contiguous()
    st = dict(case=case, a=_padded(a), sa=sa, b=_padded(b), sb=sb.view(nb, kb).contiguous())
    if own:
        from compressed_sparse_attention_indexer_gb300 import csa
        st["op"] = csa.Fp8Matmul(st["a"], st["sa"], st["b"], st["sb"],
                                 out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    return st


def _prepare_attn(case, g):
    b, s, h, hk, d, blk = (case[x] for x in ("b", "s", "heads", "kv_heads", "dim", "block"))
    lens = _lengths(case)
    nblk = [-(-x // blk) for x in lens]
    stride = max(1, max(nblk))
    total = max(1, sum(nblk))
    table = torch.full((b, stride), -1, dtype=torch.int32)
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(case["hi"])).to(torch.int32)
    at = 0
    for i, x in enumerate(nblk):
        table[i, :x] = perm[at:at + x]
        at += x
    st = dict(case=case, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), table=table.to(DEV),
              q=_randn(g, b, s, h, d, dtype=torch.bfloat16), scale=d ** -0.5)
    for name in ("k", "v"):
        x = _randn(g, total * blk, hk, d, dtype=torch.bfloat16)
        if case["kv"] == "fp8":
            codes, scale = _to_e4m3(x, x.abs().amax(2, keepdim=True).float())
            st[name], st[name + "_scale"] = codes.view(torch.uint8), scale[:, :, 0].contiguous()
        else:
            st[name], st[name + "_scale"] = x, None
    if own:
        from compressed_sparse_attention_indexer_gb300 import csa
        st["op"] = csa.PagedAttention(st["q"], st["k"], st["v"], st["lens"], table=st["table"], block=blk,
                                      k_scale=st["k_scale"], v_scale=st["v_scale"], win=case["win"], scale=st["scale"],
                                      max_len=max(1, max(lens)))
    return st


# ---------------------------------------------------------------------------
# one pass

def run(st):
    if own:
        return st["op"]()
    op = st["case"]["op"]
    return _plain_norm(st) if op == "norm" else _plain_mm(st) if op == "mm" else _plain_attn(st)


def _plain_norm(st):
    case, x = st["case"], st["x"]
    got = {}
    s = x.float()
    if st["residual"] is not None:
        s = s + st["residual"].float()
        got["residual"] = s.to(x.dtype)
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + st["eps"]) * st["weight"].float() if case["norm"] else s
    if case["out"]:
        got["out"] = y.to(x.dtype)
    if case["codes"]:
        codes, got["scale"] = _quantise_rows(y)
        got["codes"] = codes.view(torch.float8_e4m3fn)
    return got


def _scaled(codes, scale, rows):
    """The values that codes [n, k] stand for, with one scale per `rows` rows and 128 columns."""
    n, k = codes.shape
    s = scale if rows == 1 else scale.repeat_interleave(rows, 0)[:n]
    return codes.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 1)[:, :k]


def _plain_mm(st):
    out = _scaled(st["a"], st["sa"], 1) @ _scaled(st["b"], st["sb"], 128).t()
    return out.to(torch.bfloat16) if st["case"]["out"] == "bf16" else out


def _plain_attn(st):
    case = st["case"]
    b, s, h, hk, d, blk = (case[x] for x in ("b", "s", "heads", "kv_heads", "dim", "block"))
    table = st["table"].long()
    length = table.shape[1] * blk
    r = torch.arange(length, device=DEV)
    rows = table.clamp_min(0)[:, r // blk] * blk + r % blk                       # [b, length]
    pos = st["lens"].long()[:, None] - s + torch.arange(s, device=DEV)            # [b, s]
    seen = r <= pos[:, :, None]
    if case["win"]:
        seen = seen & (r > pos[:, :, None] - case["win"])
    seen = seen[:, None, :, None, :]                                             # [b, 1, s, 1, length]

    def pool(name):
        x = st[name][rows]
        x = x.float() if st[name + "_scale"] is None else \
            x.view(torch.float8_e4m3fn).float() * st[name + "_scale"][rows][..., None]
        return x.permute(0, 2, 1, 3)                                             # [b, hk, length, d]

    q = st["q"].float().view(b, s, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    sc = (q @ pool("k").transpose(2, 3) * st["scale"]).view(b, hk, s, h // hk, length)
    sc = torch.where(seen, sc, -math.inf)
    top = sc.amax(4, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(sc - top)
    total = p.sum(4, keepdim=True)
    out = (p.view(b, hk, -1, length) @ pool("v")).view(b, hk, s, h // hk, d) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(b, s, h, d).to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).reshape(b, s, h)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "mm": _exact_mm, "attn": _exact_attn}[case["op"]](case, st)


def _nearest_e4m3(v):
    """v (|v| <= 448) rounded to the nearest E4M3 value, ties to even, in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _exact_norm(case, st):
    y = st["x"].double()
    got = {}
    if case["residual"]:
        y = y + st["residual"].double()
        got["residual"] = y
    if case["norm"]:
        y = y / torch.sqrt(y.pow(2).sum(1, keepdim=True) / case["width"] + st["eps"]) * st["weight"].double()
    if case["out"]:
        got["out"] = y
    if case["codes"]:
        k = case["width"]
        codes, scales = torch.empty_like(y), []
        for c in range(0, k, 128):
            part = y[:, c:c + 128]
            most = part.abs().max(1, keepdim=True).values
            scale = torch.where(most == 0, 1.0, torch.clamp(most / E4M3_MAX, min=2.0 ** -126))
            codes[:, c:c + 128] = _nearest_e4m3(part / scale)
            scales.append(scale)
        got["codes"], got["scale"] = codes, torch.cat(scales, 1)
    return got


def _exact_mm(case, st):
    m, n, k = case["m"], case["n"], case["k"]
    col = torch.arange(k, device=DEV) // 128
    a = st["a"].view(torch.float8_e4m3fn).double().mul_(st["sa"].double()[:, col])
    b = st["b"].view(torch.float8_e4m3fn).double().mul_(st["sb"].double()[torch.arange(n, device=DEV) // 128][:, col])
    return torch.mm(a, b.t())


def _exact_attn(case, st):
    b, s, h, hk, d, blk = (case[x] for x in ("b", "s", "heads", "kv_heads", "dim", "block"))
    out = torch.zeros(b, s, h, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64, device=DEV)
    for i, length in enumerate(_lengths(case)):
        if not length:
            continue
        pages = st["table"][i, :-(-length // blk)].long()
        rows = (pages[:, None] * blk + torch.arange(blk, device=DEV)).reshape(-1)[:length]
        k, v = st["k"][rows], st["v"][rows]
        if case["kv"] == "fp8":
            k = k.view(torch.float8_e4m3fn).double() * st["k_scale"][rows].double()[:, :, None]
            v = v.view(torch.float8_e4m3fn).double() * st["v_scale"][rows].double()[:, :, None]
        k, v = k.double().repeat_interleave(h // hk, 1), v.double().repeat_interleave(h // hk, 1)
        for t in range(s):
            last = length - s + t
            if last < 0:
                continue
            first = max(0, last - case["win"] + 1) if case["win"] else 0
            sc = torch.einsum("hd,lhd->hl", st["q"][i, t].double(), k[first:last + 1]) * st["scale"]
            lse[i, t] = torch.logsumexp(sc, 1)
            out[i, t] = torch.einsum("hl,lhd->hd", torch.softmax(sc, 1), v[first:last + 1])
    return {"out": out, "lse": lse}
