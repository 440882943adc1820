"""The operators around the step run together as a serving layer uses them: hidden rows through the norm to
8 bits, the product to queries, keys and values, the cache update, dense attention over the paged 8-bit cache,
back to 8 bits and through the output product; and the indexer's inputs (q_idx, w, FP8 keys) made on the device
for the sparse step's own scoring and selection.

Every stage is checked against the fp64 definition on the inputs it actually got (the codes and rows the stage
before wrote), with that stage's bound: see test_norm_rows, test_fp8_matmul and test_paged_attn for them.
"""
from dataclasses import replace

import numpy as np
import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import build as csa_build
from compressed_sparse_attention_indexer_gb300 import csa

DEV = "cuda:0"


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    csa_build.build()
    torch.cuda.set_device(0)


def _weight(n, k, gen):
    """E4M3 codes [n, k] (rows on 16-byte boundaries) and their scale per 128 x 128."""
    nb, kb = -(-n // 128), -(-k // 128)
    w = torch.zeros(nb * 128, kb * 128, device=DEV)
    w[:n, :k] = torch.randn(n, k, generator=gen, device=DEV) * k ** -0.5
    t = w.view(nb, 128, kb, 128)
    scale = (t.abs().amax((1, 3)) / 448).clamp_min(1e-30)
    codes = (t / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * 128, kb * 128)
    return codes.view(torch.uint8)[:n, :-(-k // 16) * 16].contiguous()[:, :k], scale


def _values(codes, scale, rows):
    n, k = codes.shape
    s = scale.double() if rows == 1 else scale.double().repeat_interleave(rows, 0)[:n]
    return codes.contiguous().view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, 1)[:, :k]


def _check_codes(got, y, y_tol):
    """codes and scale of `got` against the fp64 values y."""
    v = got["codes"].float().double()
    for j in range(got["scale"].shape[1]):
        part, code, s = y[:, 128 * j:128 * j + 128], v[:, 128 * j:128 * j + 128], got["scale"][:, j:j + 1].double()
        z = part / s
        assert ((s[:, 0] - part.abs().amax(1) / 448).abs() <= (y_tol + 2.0 ** -23) * s[:, 0]).all()
        assert ((code - z).abs() <= torch.maximum(z.abs() * 2.0 ** -4, torch.full_like(z, 2.0 ** -10)) + 2.0 ** -17 * z.abs()).all()


def _check_product(out, a, sa, b, sb):
    pa, pb = _values(a, sa, 1), _values(b, sb, 128)
    want, size = pa @ pb.t(), pa.abs() @ pb.abs().t()
    tol = (128 + sa.shape[1] + 3) * 2.0 ** -23 * size + (2.0 ** -8 * want.abs() if out.dtype == torch.bfloat16 else 0)
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("b,s", [(1, 1), (7, 1), (5, 3), (40, 2)])
def test_a_dense_layer_over_an_8_bit_paged_cache(b, s):
    _gpu()
    hidden, heads, hk, d, block = 1000, 8, 2, 128, 64
    g = torch.Generator(device=DEV).manual_seed(b * 10 + s)
    lens = [int(x) for x in torch.randint(s, 900, (b,), generator=torch.Generator().manual_seed(b))]
    if b > 4:
        lens[2] = 0                                     # a padding request: its tokens' slots are negative
    n = b * s
    x, res = (torch.randn(n, hidden, generator=g, device=DEV).bfloat16() for _ in range(2))
    gamma = (1 + 0.1 * torch.randn(hidden, generator=g, device=DEV)).bfloat16()
    wq, sq = _weight(heads * d, hidden, g)
    wkv, skv = _weight(2 * hk * d, hidden, g)
    wo, so = _weight(hidden, heads * d, g)
    # the cache holds every row but the new ones already
    nblk = [-(-m // block) for m in lens]
    table = torch.full((b, max(nblk)), -1, dtype=torch.int32)
    perm = torch.randperm(sum(nblk), generator=torch.Generator().manual_seed(1))
    slots, at = [], 0
    for i, m in enumerate(lens):
        table[i, :nblk[i]] = perm[at:at + nblk[i]].int()
        at += nblk[i]
        for t in range(s):
            r = m - s + t
            slots.append(int(table[i, r // block]) * block + r % block if r >= 0 else -1)
    rows = sum(nblk) * block
    pool, scales = {}, {}
    for name in "kv":
        old = csa.NormRows(torch.randn(rows * hk, d, generator=g, device=DEV).bfloat16(), norm=False)()
        pool[name] = old["codes"].view(torch.uint8).view(rows, hk * d).clone()
        scales[name] = old["scale"].view(rows, hk).clone()
    slot = torch.tensor(slots, dtype=torch.int64, device=DEV)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    norm = csa.NormRows(x, gamma, res, eps=1e-6)
    mm_q = csa.Fp8Matmul(norm._out["codes"], norm._out["scale"], wq, sq, status=status)
    mm_kv = csa.Fp8Matmul(norm._out["codes"], norm._out["scale"], wkv, skv, status=status)
    to8 = csa.NormRows(mm_kv._out.view(n * 2 * hk, d), norm=False)
    codes = to8._out["codes"].view(torch.uint8).view(n, 2, hk * d)
    new_scale = to8._out["scale"].view(n, 2, hk)
    attn = csa.PagedAttention(mm_q._out.view(b, s, heads, d), pool["k"].view(rows, hk, d), pool["v"].view(rows, hk, d), ctx,
                              table=table.to(DEV), block=block, k_scale=scales["k"], v_scale=scales["v"], status=status)
    back = csa.NormRows(attn._out["out"].view(n, heads * d), norm=False)
    mm_o = csa.Fp8Matmul(back._out["codes"], back._out["scale"], wo, so, status=status)

    def layer():
        norm()
        mm_q()
        mm_kv()
        to8()
        for i, name in enumerate("kv"):
            csa.cache_writeback(codes[:, i], slot, pool[name], status)
            csa.cache_writeback(new_scale[:, i], slot, scales[name], status)
        attn()
        back()
        return mm_o()

    out = layer().clone()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    # stage by stage, on what each got
    t = x.double() + res.double()
    y = t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6) * gamma.double()
    assert ((norm._out["residual"].double() - t).abs() <= 2.0 ** -8 * t.abs() * 1.001).all()
    _check_codes(norm._out, y, 2.0 ** -18)
    for mm, w, sw in ((mm_q, wq, sq), (mm_kv, wkv, skv)):
        _check_product(mm._out, norm._out["codes"], norm._out["scale"], w, sw)
    _check_codes(to8._out, mm_kv._out.view(n * 2 * hk, d).double(), 2.0 ** -23)
    written = slot >= 0
    for i, name in enumerate("kv"):
        assert torch.equal(pool[name][slot[written]], codes[written, i])
        assert torch.equal(scales[name][slot[written]], new_scale[written, i])
    q = mm_q._out.view(b, s, heads, d).double()
    dense = {name: pool[name].view(torch.float8_e4m3fn).view(rows, hk, d).double() * scales[name].double()[..., None] for name in "kv"}
    for i, m in enumerate(lens):
        for k in range(s):
            pos = m - s + k
            if pos < 0:
                assert (attn._out["out"][i, k] == 0).all() and (attn._out["lse"][i, k] == -float("inf")).all()
                continue
            r = torch.arange(pos + 1)
            at = (table[i].long()[r // block] * block + r % block).to(DEV)
            kk, vv = (dense[name][at].repeat_interleave(heads // hk, 1) for name in "kv")
            sc = torch.einsum("hd,lhd->hl", q[i, k], kk) * d ** -0.5
            want = torch.einsum("hl,lhd->hd", torch.softmax(sc, 1), vv)
            big = vv.abs().amax((0, 2))[:, None]
            assert ((attn._out["lse"][i, k].double() - torch.logsumexp(sc, 1)).abs() <= 2e-4).all()
            assert ((attn._out["out"][i, k].double() - want).abs() <= 1.01 * 2.0 ** -8 * (big + want.abs()) + 1e-5 * big).all()
    some = attn._out["out"].view(n, -1).abs().amax(1) > 0                  # (a row of zeros has scale 1)
    _check_codes({k: back._out[k][some] for k in ("codes", "scale")}, attn._out["out"].view(n, -1).double()[some],
                 2.0 ** -23)
    _check_product(out, back._out["codes"], back._out["scale"], wo, so)
    # captured once and replayed: the same bits (the same rows are written to the same slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    mm_o._out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(mm_o._out, out) and int(status.item()) == 0


@pytest.mark.gpu
def test_the_indexers_inputs_made_on_the_device():
    # hidden rows -> q_idx (bf16) and w (fp32 product) of the new tokens; key rows -> normalised FP8 keys in the
    # pool; scores and selection of the library's own indexer on them against the oracle on the same values
    _gpu()
    import oracle
    from helpers import assert_topk_sets
    from compressed_sparse_attention_indexer_gb300.workloads import BF16_CFG, Workload, make_batch, to_device
    cfg = replace(BF16_CFG, idx_dtype="fp8")
    lens = [2600, 5001, 300]
    B, hidden = len(lens), 1536
    hb = make_batch(Workload("chain", cfg, B=B, S=1, L=1, seed=5), lens=lens)
    db = to_device(hb, DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(B, hidden, generator=g, device=DEV).bfloat16()
    wi, si = _weight(cfg.Hi * cfg.Di, hidden, g)
    ww, sw = _weight(cfg.Hi, hidden, g)
    norm = csa.NormRows(x, torch.ones(hidden, device=DEV).bfloat16())
    q_idx = csa.Fp8Matmul(norm._out["codes"], norm._out["scale"], wi, si)
    w = csa.Fp8Matmul(norm._out["codes"], norm._out["scale"], ww, sw, out_dtype=torch.float32)
    rows = int(hb["idx_k"].shape[0])
    keys = csa.NormRows(torch.randn(rows, cfg.Di, generator=g, device=DEV).bfloat16(), torch.full((cfg.Di,), 1.25, device=DEV).bfloat16())
    norm(), q_idx(), w(), keys()
    slot = torch.arange(rows, device=DEV)
    csa.cache_writeback(keys._out["codes"], slot, db["idx_k"])
    csa.cache_writeback(keys._out["scale"], slot, db["idx_scale"].view(-1, 1))
    db["q_idx"], db["w"] = q_idx._out.view(B, 1, cfg.Hi, cfg.Di), w._out.view(B, 1, cfg.Hi)
    dec = csa.Decoder(cfg, B, 1, 8192)
    idx = torch.empty(B, 1, cfg.topk, dtype=torch.int32, device=DEV)
    cnt = torch.empty(B, 1, dtype=torch.int32, device=DEV)
    dec.indexer_topk(csa.make_batch_struct(db), idx, cnt)
    assert dec.status() == csa.CSA_OK
    _check_product(w._out, norm._out["codes"], norm._out["scale"], ww, sw)
    ref = dict(hb, q_idx=q_idx._out.view(B, 1, cfg.Hi, cfg.Di).cpu(), w=w._out.view(B, 1, cfg.Hi).cpu(),
               idx_k=db["idx_k"].cpu(), idx_scale=db["idx_scale"].cpu())
    want = oracle.decode(cfg, ref)
    values = (db["idx_k"].view(torch.float8_e4m3fn).float() * db["idx_scale"][:, None]).double().cpu().numpy()

    def scores(q):
        off = int(hb["idx_off"][q])
        return oracle.index_scores(ref["q_idx"][q, 0].double().numpy(), ref["w"][q, 0].double().numpy(),
                                   values[off:off + lens[q] // 4])

    assert_topk_sets(idx.cpu().numpy().reshape(B, -1), cnt.cpu().numpy().reshape(-1), want, scores, cfg.topk, "chain")
    assert np.isfinite(values).all()
