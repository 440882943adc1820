"""The operators for new and drafted tokens run together as a serving layer uses them: a prompt's heads normed and
rotated in place and written to the pools, then steps of drafted trees: hidden rows to 8 bits, the product to queries,
keys and values, their norm and rotation and the keys and values into the cache in one call, the tree's attention over
it, back to 8 bits and through the output product.  The step is captured once and replayed for other inputs, lengths,
counts and trees.

Every stage is checked against the fp64 definition on the inputs it actually got, with that stage's bound: see
test_qk_rope, test_kv_append, test_tree_attn, test_norm_rows and test_fp8_matmul for them.
"""
import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import csa
from test_kv_append import E4M3_MAX
from test_operator_chain import _check_codes, _check_product, _weight
from test_qk_rope import U32, check, exact
from test_tree_attn import DEV, _check, _exact, _gpu, _sees, _tree

HIDDEN, D, BLOCK = 640, 128, 64


class Layer:
    """A layer's weights and pools, the operators of its step on buffers of b requests of s drafts."""

    def __init__(self, b, s, hq, hk, fp8, win, most, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.b, self.s, self.hq, self.hk, self.fp8, self.win = b, s, hq, hk, fp8, win
        rn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)
        self.wqkv, self.wo = _weight((hq + 2 * hk) * D, HIDDEN, g), _weight(HIDDEN, hq * D, g)
        self.gq, self.gk = ((1 + 0.1 * rn(D)).bfloat16() for _ in "qk")
        self.x = torch.empty(b * s, HIDDEN, dtype=torch.bfloat16, device=DEV)
        i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=DEV)
        self.n, self.count, self.pos, self.status = i32(b), i32(b), i32(b, s), i32(1)
        self.masks = torch.zeros(b, s, -(-s // 64), dtype=torch.int64, device=DEV)
        nblk = -(-most // BLOCK)
        rows = (b * nblk + 1) * BLOCK
        self.table = torch.randperm(b * nblk + 1, generator=torch.Generator().manual_seed(seed))[:-1].view(b, nblk).int().to(DEV)
        self.rows = rows
        new = lambda: torch.zeros(rows, hk, D, device=DEV).to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
        self.pool = {"k": new(), "v": new()}
        self.scale = {x: torch.ones(rows, hk, device=DEV) if fp8 else None for x in "kv"}

        self.norm = csa.NormRows(self.x, eps=1e-6)
        self.mm = csa.Fp8Matmul(self.norm._out["codes"], self.norm._out["scale"], *self.wqkv, status=self.status)
        qkv = self.mm._out.view(b, s, hq + 2 * hk, D)
        self.q, self.k, self.v = qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
        self.q_out = torch.zeros(b, s, hq, D, dtype=torch.bfloat16, device=DEV)
        where = dict(table=self.table, block=BLOCK)
        how = dict(q_weight=self.gq, k_weight=self.gk, norm=True, rope_dim=64, rope_at=64)
        self.append = csa.KvAppend(self.k, self.v, self.pool["k"], self.pool["v"], self.scale["k"], self.scale["v"], self.n,
                                   count=self.count, pos=self.pos, q=self.q, q_out=self.q_out, status=self.status, **how, **where)
        self.attn = csa.TreeAttention(self.q_out, self.pool["k"], self.pool["v"], self.n, self.masks, count=self.count, pos=self.pos,
                                      k_scale=self.scale["k"], v_scale=self.scale["v"], win=win, status=self.status, **where)
        self.back = csa.NormRows(self.attn._out["out"].view(b * s, hq * D), norm=False)
        self.mm_o = csa.Fp8Matmul(self.back._out["codes"], self.back._out["scale"], *self.wo, status=self.status)
        self.how = how

    def step(self):
        self.norm()
        self.mm()
        self.append()
        self.attn()
        self.back()
        return self.mm_o()

    def prompt(self, lens, seed):
        """The rows before the drafts: heads normed and rotated in place within a fused projection, written by slot."""
        g = torch.Generator(device=DEV).manual_seed(seed)
        n = sum(lens)
        qkv = torch.randn(n, self.hq + 2 * self.hk, D, generator=g, device=DEV).bfloat16()
        q, k, v = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hk], qkv[:, self.hq + self.hk:]
        pos = torch.cat([torch.arange(x) for x in lens]).int().to(DEV)
        req = torch.repeat_interleave(torch.arange(self.b), torch.tensor(lens)).to(DEV)
        slot = self.table[req, pos // BLOCK].long() * BLOCK + pos % BLOCK
        before = qkv.cpu()
        if self.fp8:
            csa.KvAppend(k[None], v[None], self.pool["k"], self.pool["v"], self.scale["k"], self.scale["v"], slot=slot, pos=pos,
                         k_weight=self.gk, norm=True, rope_dim=64, rope_at=64)()
        else:
            csa.QkRope(q, k, pos, q_out=q, k_out=k, **self.how)()
            for x, rows in (("k", k), ("v", v)):
                csa.cache_writeback(rows.reshape(n, self.hk * D), slot, self.pool[x].view(self.rows, self.hk * D), self.status)
            torch.cuda.synchronize()
            for got, at, w in ((q, 0, self.gq), (k, self.hq, self.gk)):
                x = before[:, at:at + got.shape[1]]
                want, size = exact(x, w.cpu(), pos.cpu(), True, 1e-6, 64, 64, False)
                check(got.cpu(), want, size, torch.bfloat16)
            assert torch.equal(self.pool["k"][slot], k) and torch.equal(self.pool["v"][slot].cpu(), before[:, self.hq + self.hk:])

    def feed(self, past, counts, seed):
        """Drafts behind `past` rows of each request."""
        self.x.copy_(torch.randn(self.x.shape, generator=torch.Generator().manual_seed(seed)).bfloat16())
        masks = _tree(self.b, self.s, seed)
        depth = _sees(masks, self.s).sum(2) - 1
        self.lens = [p + c if c else 0 for p, c in zip(past, counts)]
        self.counts = counts
        self.n.copy_(torch.tensor(self.lens))
        self.count.copy_(torch.tensor(counts))
        self.masks.copy_(masks)
        self.pos.copy_(torch.tensor(past)[:, None] + depth)

    def values(self, x):
        p = self.pool[x].float().double().cpu()
        return p * self.scale[x].double().cpu()[..., None] if self.fp8 else p

    def check_step(self, out, before):
        b, s = self.b, self.s
        assert int(self.status.item()) == 0
        t = self.x.double()
        _check_codes(self.norm._out, t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6), 2.0 ** -18)
        _check_product(self.mm._out, self.norm._out["codes"], self.norm._out["scale"], *self.wqkv)
        real = torch.arange(s)[None] < torch.tensor(self.counts)[:, None]
        first = torch.tensor(self.lens) - torch.tensor(self.counts)
        row = (first[:, None] + torch.arange(s)).clamp(0, self.table.shape[1] * BLOCK - 1)
        to = (self.table.cpu().long().gather(1, row // BLOCK) * BLOCK + row % BLOCK)[real]
        pos = self.pos.cpu()[real]
        for got, x, w in ((self.q_out, self.q, self.gq), (None, self.k, self.gk)):
            want, size = exact(x.cpu()[real], w.cpu(), pos, True, 1e-6, 64, 64, False)
            if got is not None:
                check(got.cpu()[real], want, size, torch.bfloat16)
            elif not self.fp8:
                check(self.pool["k"].cpu()[to], want, size, torch.bfloat16)
            else:
                self._check_e4m3("k", to, want, 40 * U32 * size)
        v = self.v.cpu()[real]
        if self.fp8:
            self._check_e4m3("v", to, v.double(), torch.zeros_like(v, dtype=torch.float64))
        else:
            assert torch.equal(self.pool["v"].cpu()[to], v)
        still = torch.ones(self.rows, dtype=torch.bool)
        still[to] = False
        for x in "kv":
            assert torch.equal(self.pool[x].cpu().view(torch.uint8)[still], before[x].view(torch.uint8)[still])
        want = _exact(self.q_out.cpu(), self.values("k"), self.values("v"), self.lens, self.counts, _sees(self.masks.cpu(), s),
                      self.pos.cpu(), self.table.cpu(), BLOCK, self.win, D ** -0.5)
        _check(self.attn._out, want)
        assert (self.attn._out["out"].cpu()[~real] == 0).all()
        # (a row of zeros has no maximum to scale by: codes of zero)
        rows = real.view(-1).to(DEV)
        _check_codes({x: y[rows] for x, y in self.back._out.items() if x in ("codes", "scale")},
                     self.attn._out["out"].view(b * s, -1)[rows].double(), 2.0 ** -23)
        assert (self.back._out["codes"].float()[~rows] == 0).all()
        _check_product(out, self.back._out["codes"], self.back._out["scale"], *self.wo)

    def _check_e4m3(self, x, to, want, off):
        codes, scale = self.pool[x].float().cpu()[to].double(), self.scale[x].cpu()[to].double()
        most = want.abs().amax(2)
        assert ((scale - most / E4M3_MAX).abs() <= off.amax(2) / E4M3_MAX + 2 * U32 * scale).all()
        z = want / scale[..., None]
        # half a step of the quotient, and the key's and the scale's own errors
        tol = torch.maximum(z.abs() * 2.0 ** -4, torch.full_like(z, 2.0 ** -10)) + (off + off.amax(2, keepdim=True)) / scale[..., None] + 6 * U32 * z.abs()
        assert ((codes - z).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("b,s,hq,hk,fp8,win", [(1, 5, 8, 2, False, 0), (3, 8, 8, 2, True, 0), (12, 21, 16, 2, False, 70),
                                               (8, 64, 16, 4, True, 0), (2, 1, 4, 4, False, 0)])
def test_prompt_then_captured_steps_of_drafts(b, s, hq, hk, fp8, win):
    _gpu()
    g = torch.Generator().manual_seed(b + s)
    past = [int(x) for x in torch.randint(1, 400, (b,), generator=g)]
    layer = Layer(b, s, hq, hk, fp8, win, 400 + 4 * s, seed=s)
    layer.prompt(past, seed=5)
    counts = [s] * b
    layer.feed(past, counts, 1)
    keep = lambda: {x: p.cpu().clone() for x, p in layer.pool.items()}
    before = keep()
    out = layer.step().clone()
    torch.cuda.synchronize()
    layer.check_step(out, before)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = layer.step()
    for i in range(3):
        # some drafts were accepted: the next ones lie behind them; a request has fewer, another ends
        past = [p + min(c, 1 + (i + j) % 3) for j, (p, c) in enumerate(zip(past, counts))]
        counts = [max(1, s - (i + j) % 4) for j in range(b)]
        if b > 2 and i == 1:
            counts[1] = 0
        layer.feed(past, counts, 10 + i)
        before = keep()
        graph.replay()
        torch.cuda.synchronize()
        layer.check_step(out, before)


@pytest.mark.gpu
def test_two_captured_steps_that_share_a_workspace_on_one_stream():
    """Two attention calls of one stream may share a workspace: captured in two graphs, replayed in turn."""
    _gpu()
    g = torch.Generator(device=DEV).manual_seed(3)
    s, hk, h, rows = 64, 2, 8, 64 * 40
    space = torch.empty(csa.tree_attn_workspace(D), dtype=torch.uint8, device=DEV)
    masks = _tree(2, s, 4).to(DEV)
    made = []
    for i in range(2):
        k, v = (torch.randn(rows, hk, D, generator=g, device=DEV).bfloat16() for _ in "kv")
        q = torch.randn(2, s, h, D, generator=g, device=DEV).bfloat16()
        off = torch.tensor([0, 1300], device=DEV)
        n = torch.tensor([1200 - 300 * i, 900 + 200 * i], dtype=torch.int32, device=DEV)
        op = csa.TreeAttention(q, k, v, n, masks, off=off, max_len=1 << 20, workspace=space)
        alone = {x: t.clone() for x, t in op().items()}
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            op()
        made.append((op, alone, graph))
    for _ in range(10):
        for op, _, graph in made:
            graph.replay()
    torch.cuda.synchronize()
    for op, alone, _ in made:
        assert all(torch.equal(op._out[x], alone[x]) for x in alone)
