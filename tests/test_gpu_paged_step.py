"""The serving operators together, as a decode loop uses them: norm and rotation
of the projections, quantising the new keys and values into the pages,
attention and reading back; against the plain forms (tests/_paged.py), stage
by stage on the values that the stage before it left, and against
hqmq_attention_decode over the same tokens in a contiguous cache."""
import numpy as np
import pytest
import torch

import _paged as P
from test_gpu_norm_rope import check
from test_gpu_paged_attention import plain
from test_gpu_paged_cache import cuda_ints, layout
from kv_cache_quantization_hqmq_b200 import hqmq

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

BF = torch.bfloat16
D, EPS = 128, 1e-6


class Layer:
    """A layer's cache for a batch behind a shared prefix, and its buffers; G query heads per KV head."""

    def __init__(self, seed, page, S, cap, Hk, G, prefix, lens, tables, out):
        rng = np.random.default_rng(seed)
        self.prefix, self.lens, self.Hk, self.G, self.S = prefix, list(lens), Hk, G, S
        need = -(-prefix // page)
        self.table, n = layout(rng, [m + 8 for m in lens], page, spare=need + 1)
        self.ptable = np.setdiff1d(np.arange(n), self.table)[:need].astype(np.int32)
        self.pools = [P.empty_pool(rng, n, Hk, page, S, cap) for _ in range(2)]
        if not cap:
            for p in self.pools:
                p["thr"] = None
        self.kv = [P.upload(p, P.search_tables(p["cb"]) if tables else None) for p in self.pools]
        g = torch.Generator().manual_seed(seed)
        self.g = g
        self.w = (1 + 0.1 * torch.randn(2, D, generator=g)).to(BF).cuda()
        self.w[:, 9] = 12                                      # a strong channel: outliers
        self.inv = hqmq.rope_inv_freq(D, 500000.0)
        B = len(lens)
        self.t_d, self.pt_d, self.len_d = cuda_ints(self.table, self.ptable, lens)
        self.pos_d = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
        self.o = torch.empty(B, Hk * G, D, dtype=out, device="cuda")
        self.lse = torch.empty(B, Hk * G, device="cuda")
        self.kp, self.vp = self.kv[0][0], self.kv[1][0]
        self.ws = hqmq.alloc_attention_paged_ws(B, Hk * G, self.kp, self.table.shape[1], prefix)
        self.status = hqmq.new_status()

    def projections(self, B, T):
        return torch.randn(B, T, self.G * self.Hk + 2 * self.Hk, D, generator=self.g).to(BF).cuda()

    def heads(self, qkv):
        Hq = self.G * self.Hk
        return qkv[:, :, :Hq], qkv[:, :, Hq:Hq + self.Hk], qkv[:, :, Hq + self.Hk:]

    def norm_rope(self, qkv, pos):
        q, k, _ = self.heads(qkv)
        hqmq.hqmq_qk_norm_rope(q, k, q, k, pos, self.inv, self.w[0], self.w[1], eps=EPS)

    def fill(self, table, new):
        """A prompt of new[b] tokens for each row of the table, as one packed batch."""
        cu = np.concatenate([[0], np.cumsum(new)])
        start = 0 if table is self.ptable or self.prefix == 0 else self.prefix
        pos = np.concatenate([start + np.arange(m) for m in new])[None] if cu[-1] else np.zeros((1, 0))
        qkv = self.projections(1, int(cu[-1]))
        raw = qkv.clone()
        pos_d, cu_d, pos0_d, t_d = cuda_ints(pos, cu, [0] * len(new), np.atleast_2d(table))
        if cu[-1]:
            self.norm_rope(qkv, pos_d)
            check(self.heads(qkv)[1], self.heads(raw)[1], self.w[1], pos_d, self.inv, EPS, False)
        _, k, v = self.heads(qkv)
        hqmq.hqmq_paged_write(k[0], v[0], self.kp, self.vp, t_d, cu_d, pos0_d, status=self.status)
        for pool, x in zip(self.pools, (k, v)):
            P.write(pool, x[0].float().cpu().numpy(), np.atleast_2d(table), cu, [0] * len(new))

    def decode(self, qkv, q, ones):
        """One token of every sequence; lengths live and advance on the device."""
        torch.add(self.len_d[:, None], self.prefix, out=self.pos_d)
        self.norm_rope(qkv, self.pos_d)
        hq, k, v = self.heads(qkv)
        hqmq.hqmq_paged_write(k[:, 0], v[:, 0], self.kp, self.vp, self.t_d, ones, self.len_d, status=self.status)
        self.len_d += 1
        q.copy_(hq[:, 0])
        hqmq.hqmq_attention_paged(q, self.kp, self.vp, self.t_d, self.len_d, self.o, self.ws, prefix_table=self.pt_d,
                                  prefix_len=self.prefix, lse=self.lse, status=self.status)

    def check_step(self, raw, qkv, q):
        """The plain forms of the step that ran, from what its stages left."""
        pos = torch.tensor(self.lens, dtype=torch.int32)[:, None] + self.prefix
        for x, r, w in zip(self.heads(qkv)[:2], self.heads(raw)[:2], self.w):
            check(x, r, w, pos, self.inv, EPS, False)
        assert torch.equal(self.heads(qkv)[2], self.heads(raw)[2])
        B = len(self.lens)
        for pool, x in zip(self.pools, self.heads(qkv)[1:]):
            P.write(pool, x[:, 0].float().cpu().numpy(), self.table, np.arange(B + 1), self.lens)
        self.lens = [m + 1 for m in self.lens]
        pk, pv = (P.dense(p, self.ptable, self.prefix)[0] for p in self.pools)
        for b, m in enumerate(self.lens):
            k, v = (P.bf16(np.concatenate([x, P.dense(p, self.table[b], m)[0]], 1))
                    for x, p in zip((pk, pv), self.pools))
            for h in range(self.Hk):
                rows = slice(h * self.G, (h + 1) * self.G)
                want, bound, wl, bl = plain(q[b, rows].float().cpu().numpy(), k[h], v[h],
                                            np.ones(self.prefix + m, bool), D ** -0.5, self.o.dtype)
                tol = 2 * bound + (2.0 ** -8 * np.abs(want) if self.o.dtype == BF else 0)
                assert np.all(np.abs(self.o[b, rows].double().cpu().numpy() - want) <= tol)
                assert np.all(np.abs(self.lse[b, rows].double().cpu().numpy() - wl) <= 2 * bl)

    def check_pages(self):
        for pool, (_, t) in zip(self.pools, self.kv):
            P.assert_pools_equal(t, pool)
        y = torch.zeros(len(self.lens), self.Hk, max(self.lens), D, device="cuda")
        hqmq.hqmq_paged_read(self.vp, self.t_d, self.len_d, y, status=self.status)
        for b, m in enumerate(self.lens):
            np.testing.assert_array_equal(y[b, :, :m].cpu().numpy(), P.dense(self.pools[1], self.table[b], m)[0])
        assert hqmq.read_status(self.status)["flags"] & ~hqmq.FLAG_OUTLIER_OVERFLOW == 0


@pytest.mark.parametrize("page,S,cap,Hk,G,prefix,lens,tables,out", [
    (32, 32, 96, 2, 4, 70, [0, 31, 33], True, torch.float32),
    (16, 8, 0, 1, 7, 0, [1, 15, 40, 0], False, torch.float32),
    (64, 32, 128, 1, 16, 129, [5] * 9, True, BF)])
def test_decode_loop(page, S, cap, Hk, G, prefix, lens, tables, out):
    """Prompts in packed batches, then steps: two calls and four replays of a graph."""
    layer = Layer(page + S, page, S, cap, Hk, G, prefix, lens, tables, out)
    if prefix:
        layer.fill(layer.ptable, [prefix])
    layer.fill(layer.table, lens)
    B = len(lens)
    ones = cuda_ints(np.arange(B + 1))[0]
    qkv = torch.zeros(B, 1, Hk * (G + 2), D, dtype=BF, device="cuda")
    q = torch.zeros(B, Hk * G, D, dtype=BF, device="cuda")
    graph = None
    for i in range(6):
        raw = layer.projections(B, 1)
        qkv.copy_(raw)
        if i < 2:
            layer.decode(qkv, q, ones)
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    layer.decode(qkv, q, ones)
            graph.replay()
        layer.check_step(raw, qkv, q)
    layer.check_pages()


def test_the_contiguous_cache_gives_the_same():
    """The pages' codes, gathered into a contiguous cache, through hqmq_attention_decode: its weights err by
    2^-17 (two bf16 terms), so |do| <= 2 2^-17 max|v - o| more than three terms' bound."""
    B, Hk, G, T, S, page = 3, 2, 8, 128, 32, 64
    layer = Layer(5, page, S, 0, Hk, G, 0, [T] * B, True, torch.float32)
    layer.fill(layer.table, [T] * B)
    codes, dense = [], []
    for pages, t in layer.kv:
        at = layer.t_d[:, :T // page].long()
        words, radius = (t[n][at].transpose(1, 2).reshape(B, Hk, T, -1).contiguous() for n in ("words", "radius"))
        codes.append(hqmq.kv_codes(words, radius, t["cb"]))
        dense.append(hqmq.hqmq_paged_read(pages, layer.t_d, layer.len_d,
                                          torch.empty(B, Hk, T, D, dtype=BF, device="cuda")).float().cpu().numpy())
    q = torch.randn(B, Hk * G, D, generator=layer.g).to(BF).cuda()
    o = torch.empty(B, Hk * G, D, device="cuda")
    hqmq.hqmq_attention_decode(q, *codes, S, Hk, T, o, hqmq.alloc_attention_ws(B, Hk), seq_len=layer.len_d)
    hqmq.hqmq_attention_paged(q, layer.kp, layer.vp, layer.t_d, layer.len_d, layer.o, layer.ws, lse=layer.lse)
    for b in range(B):
        for h in range(Hk):
            rows = slice(h * G, (h + 1) * G)
            k, v = (x[b, h] for x in dense)
            want, bound, _, _ = plain(q[b, rows].float().cpu().numpy(), k, v, np.ones(T, bool), D ** -0.5)
            assert np.all(np.abs(layer.o[b, rows].double().cpu().numpy() - want) <= 2 * bound)
            assert np.all(np.abs(o[b, rows].double().cpu().numpy() - want) <= 2 * (bound + 2.0 ** -16 * 2 * np.abs(v).max()))


@pytest.mark.parametrize("S,cap,out", [((8, 32), (0, 60), torch.float32), ((32, 8), (40, 0), BF), ((48, 3), (64, 9), BF),
                                       ((10, 22), (30, 30), torch.float32)])
def test_keys_and_values_of_different_codebooks(S, cap, out):
    """K and V with codebooks and outlier slots of their own, pools of different sizes; prefixes that end in
    different rows of a page; queries and outputs in one buffer."""
    rng = np.random.default_rng(S[0])
    B, Hk, G, page = 3, 2, 4, 32
    lens, prefix = [33, 0, 70], 45
    table, n = layout(rng, [m + 1 for m in lens], page, spare=3)
    ptable = np.setdiff1d(np.arange(n), table)[:2].astype(np.int32)
    pools = [P.empty_pool(rng, n + 4 * r, Hk, page, S[r], cap[r]) for r in range(2)]
    kv = [P.upload(p, P.search_tables(p["cb"])) for p in pools]
    status = hqmq.new_status()
    for tab, m in ((ptable[None], [prefix]), (table, lens), (table, [1] * B)):
        old = lens if m == [1] * B else [0] * len(m)
        cu = np.concatenate([[0], np.cumsum(m)])
        x = [torch.randn(int(cu[-1]), Hk, D, generator=torch.Generator().manual_seed(r)).to(BF) for r in range(2)]
        x[0][:, :, 7] *= 9
        hqmq.hqmq_paged_write(x[0].cuda(), x[1].cuda(), kv[0][0], kv[1][0], *cuda_ints(tab, cu, old), status=status)
        for pool, y in zip(pools, x):
            P.write(pool, y.float().numpy(), tab, cu, old)
    for pool, (_, t) in zip(pools, kv):
        P.assert_pools_equal(t, pool)
    lens = [m + 1 for m in lens]
    q = torch.randn(B, Hk * G, D, generator=torch.Generator().manual_seed(9)).to(BF)
    qo = q.cuda()
    o = qo if out == BF else torch.empty(B, Hk * G, D, device="cuda")      # (bf16: in place)
    ws = hqmq.alloc_attention_paged_ws(B, Hk * G, kv[0][0], table.shape[1], prefix)
    t_d, len_d, pt_d = cuda_ints(table, lens, ptable)
    hqmq.hqmq_attention_paged(qo, kv[0][0], kv[1][0], t_d, len_d, o, ws, prefix_table=pt_d, prefix_len=prefix,
                              status=status)
    for b, m in enumerate(lens):
        k, v = (P.bf16(np.concatenate([P.dense(p, ptable, prefix)[0], P.dense(p, table[b], m)[0]], 1)) for p in pools)
        for h in range(Hk):
            rows = slice(h * G, (h + 1) * G)
            want, bound, _, _ = plain(q[b, rows].float().numpy(), k[h], v[h], np.ones(prefix + m, bool), D ** -0.5, out)
            tol = 2 * bound + (2.0 ** -8 * np.abs(want) if out == BF else 0)
            assert np.all(np.abs(o[b, rows].double().cpu().numpy() - want) <= tol)
    assert hqmq.read_status(status)["flags"] & ~hqmq.FLAG_OUTLIER_OVERFLOW == 0


def test_two_streams_and_two_graphs():
    """Calls on two streams at once with workspaces of their own, and two graphs that share one workspace."""
    layers = [Layer(s, 32, 32, 64, 2, 4, 70, [40, 9, 64], True, BF) for s in (1, 2)]
    for layer in layers:
        layer.fill(layer.ptable, [layer.prefix])
        layer.fill(layer.table, layer.lens)
    q = torch.randn(2, 3, 8, D, generator=torch.Generator().manual_seed(3)).to(BF).cuda()

    def attend(layer, x, ws):
        hqmq.hqmq_attention_paged(x, layer.kp, layer.vp, layer.t_d, layer.len_d, layer.o, ws, prefix_table=layer.pt_d,
                                  prefix_len=layer.prefix, lse=layer.lse, status=layer.status)

    want = []
    for i, layer in enumerate(layers):
        attend(layer, q[i], layer.ws)
        want.append((layer.o.clone(), layer.lse.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for layer in layers:
        layer.o.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (layer, s) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(s):
                attend(layer, q[i], layer.ws)
    torch.cuda.synchronize()
    for layer, (o, lse) in zip(layers, want):
        assert torch.equal(layer.o, o) and torch.equal(layer.lse, lse)
        layer.o.zero_()
    graphs = []
    for i, layer in enumerate(layers):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend(layer, q[i], layers[0].ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for layer, (o, lse) in zip(layers, want):
        assert torch.equal(layer.o, o) and torch.equal(layer.lse, lse)
        assert hqmq.read_status(layer.status)["flags"] & ~hqmq.FLAG_OUTLIER_OVERFLOW == 0


def test_pages_past_32_bit_offsets():
    """The same tokens in the first pages of a small pool and in the last pages of one whose words and radii each
    pass 2^32 bytes (12 GB, only the used pages are touched): the same pages, tokens and attention, bit for bit."""
    H, page, S, cap, lens = 16, 256, 32, 512, [300, 5, 257]
    big = (1 << 32) // (H * page * 40) + 3                                # 40 bytes of words, 64 of radii
    cb = torch.from_numpy(P.make_codebook(np.random.default_rng(8), H, S)).cuda()
    thr = torch.full((H,), 4.0, device="cuda")
    table = np.array([[0, 1], [2, -1], [3, 4]], np.int32)
    cu_d, pos_d, len_d = cuda_ints(np.concatenate([[0], np.cumsum(lens)]), [0, 0, 0], lens)
    x = torch.randn(sum(lens), H, D, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    q = torch.randn(3, 2 * H, D, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    got = []
    for n, shift in ((5, 0), (big, big - 5)):
        words = torch.empty(n, H, page, 10, dtype=torch.int32, device="cuda")
        radius = torch.empty(n, H, page, 32, dtype=torch.int16, device="cuda")
        flags = torch.empty(n, H, page, dtype=torch.int32, device="cuda")
        val = torch.empty(n, H, cap, 4, dtype=torch.int16, device="cuda")
        for t in (words, radius, flags, val):
            t[shift:].zero_()
        kp = hqmq.kv_pages(words, radius, cb, flags, val, thr)
        t_d = cuda_ints(np.where(table < 0, -1, table + shift))[0]
        status = hqmq.new_status()
        hqmq.hqmq_paged_write(x, None, kp, None, t_d, cu_d, pos_d, status=status)
        y = torch.zeros(3, H, max(lens), D, dtype=BF, device="cuda")
        hqmq.hqmq_paged_read(kp, t_d, len_d, y, status=status)
        o = torch.empty(3, 2 * H, D, device="cuda")
        hqmq.hqmq_attention_paged(q, kp, kp, t_d, len_d, o, hqmq.alloc_attention_paged_ws(3, 2 * H, kp, 2, 256),
                                  prefix_table=t_d[0, :1].contiguous(), prefix_len=256, status=status)
        assert hqmq.read_status(status)["flags"] == 0
        got.append([t[shift:].clone() for t in (words, radius, flags, val)] + [y, o])
        del words, radius, flags, val, kp
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert bool(got[0][4].abs().sum() > 0) and bool(got[0][5].isfinite().all())
