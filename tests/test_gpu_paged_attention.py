"""hqmq_attention_paged against plain attention in 64 bits over the pages'
values (tests/_paged.py), and against hqmq_attention_decode.

Tolerance, per row (u = 2^-24): a score's exponent x = sl2 s errs by at most
sl2 128 2u max_t sum_d |q_d k_td| (fp32 sums of exact bf16 products) plus its
own rounding; exp2 by 2^-21; the weights by w = 2^-24 in three bf16 terms
(fp32 outputs) or 2^-9 in one (bf16 outputs); the normalised weights then by
d = 2 (ln2 |dx| + 2^-21 + w), and fp32 accumulation by (T / 16 + 64) u max|v|:
|do| <= d max|v - o| + (T / 16 + 64) u max|v|.  The test allows twice that
(once for one-term weights, whose bound is the larger part), and bf16 outputs
half a step more.  lse = ln sum exp, summed before the weights are rounded,
errs by ln2 |dx| + 2^-21 + 4 u (1 + |lse|)."""
import numpy as np
import pytest
import torch

import _paged as P
from test_gpu_paged_cache import cuda_ints, layout
from kv_cache_quantization_hqmq_b200 import hqmq

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

U = 2.0 ** -24
LN2 = np.log(2.0)


def filled_pool(rng, n_pages, H, page, S, cap, spread=1.0):
    """A pool of plausible codes: random directions, chi-distributed radii, a strong channel in the flags."""
    pool = P.empty_pool(rng, n_pages, H, page, S, cap)
    b = hqmq.hqmq_index_bits(S)
    flag = np.zeros((n_pages, H, page, 32), bool)
    if cap:
        flag = rng.random(flag.shape) < 0.03
        flag[..., 5] |= rng.random(flag.shape[:3]) < 0.6
        rank = flag.reshape(n_pages, H, -1).cumsum(-1).reshape(flag.shape)
        flag &= rank <= cap
        pool["flags"] = (flag.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
        val = rng.standard_normal((n_pages, H, cap, 4)).astype(np.float32) * 4
        pool["val"] = P.f16_bits(val)
    r = np.sqrt((rng.standard_normal((n_pages, H, page, 32, 4)) ** 2).sum(-1)).astype(np.float32) * spread
    pool["radius"] = P.f16_bits(np.where(flag, 0, r))
    idx = np.where(flag, 0, rng.integers(0, 24 * S, r.shape)).reshape(-1, 32)
    words = np.array([P.pack_words(i, b) for i in idx], dtype=np.uint64).astype(np.uint32)
    pool["words"] = words.reshape(n_pages, H, page, b)
    return pool


def plain(q, kd, vd, ok, scale, out=torch.float32):
    """(o, bound, lse, lse bound) of one sequence and KV head; q [G, 128], kd/vd [T, 128], ok [T]."""
    G = q.shape[0]
    kd, vd = kd[ok].astype(np.float64), vd[ok].astype(np.float64)
    T = kd.shape[0]
    if T == 0:
        return np.zeros((G, 128)), np.zeros((G, 1)) + 1e-30, np.full(G, -np.inf), np.zeros(G)
    q = q.astype(np.float64)
    s = scale * (q @ kd.T)
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    lse = (m + np.log(e.sum(-1, keepdims=True)))[:, 0]
    o = (e / e.sum(-1, keepdims=True)) @ vd
    sl2 = abs(scale) / LN2
    dx = sl2 * 128 * 2 * U * (np.abs(q) @ np.abs(kd).T).max(-1) + U * sl2 * np.abs(s / scale if scale else s).max(-1)
    w = 2.0 ** -24 if out == torch.float32 else 2.0 ** -9
    d = 2 * (LN2 * dx + 2.0 ** -21 + w)
    vmax = np.abs(vd).max()
    spread = np.abs(vd[None] - o[:, None]).max((1, 2))
    bound = d * spread + (T / 16 + 64) * U * vmax
    return o, (1 if out == torch.float32 else 0.5) * bound[:, None], lse, \
        LN2 * dx + 2.0 ** -21 + 4 * U * (1 + np.abs(lse))


def run(rng, B, Hk, G, page, S, cap, lens, prefix, out=torch.float32, scale=None, bad=(), spread=1.0, q_scale=1.0,
        max_extra=0):
    table, n = layout(rng, lens, page, spare=-(-prefix // page) + 1, width=max_extra)
    pools = [filled_pool(rng, n, Hk, page, S, cap, spread) for _ in range(2)]
    used = sum(-(-t // page) for t in lens)
    free = np.setdiff1d(np.arange(n), table[table >= 0])
    ptable = rng.permutation(free)[:-(-prefix // page)].astype(np.int32)
    assert used + len(ptable) <= n
    for b, col in bad:
        if b < 0:
            ptable[col] = -3
        else:
            table[b, col] = n + 5
    q = torch.from_numpy(rng.standard_normal((B, Hk * G, 128)).astype(np.float32) * np.float32(q_scale)).bfloat16()
    (kp, _), (vp, _) = (P.upload(p) for p in pools)
    t_d, len_d, pt_d = cuda_ints(table, lens, ptable)
    o = torch.full((B, Hk * G, 128), float("nan"), dtype=out, device="cuda")
    lse = torch.full((B, Hk * G), float("nan"), device="cuda")
    ws = hqmq.alloc_attention_paged_ws(B, Hk * G, kp, table.shape[1], prefix)
    ws.fill_(0xFF)                                                    # NaNs
    status = hqmq.new_status()
    hqmq.hqmq_attention_paged(q.cuda(), kp, vp, t_d, len_d, o, ws, prefix_table=pt_d, prefix_len=prefix, scale=scale,
                              lse=lse, status=status)
    torch.cuda.synchronize()
    scale = 128 ** -0.5 if scale is None else scale
    pk, pok = P.dense(pools[0], ptable, prefix)
    pv, _ = P.dense(pools[1], ptable, prefix)
    worst = 0.0
    for b in range(B):
        n_b = min(max(lens[b], 0), table.shape[1] * page)
        k, okk = P.dense(pools[0], table[b], n_b)
        v, _ = P.dense(pools[1], table[b], n_b)
        k, v = P.bf16(np.concatenate([pk, k], 1)), P.bf16(np.concatenate([pv, v], 1))
        ok = np.concatenate([pok, okk])
        for h in range(Hk):
            rows = slice(h * G, (h + 1) * G)
            want, bound, wl, bl = plain(q[b, rows].float().numpy(), k[h], v[h], ok, scale, out)
            got = o[b, rows].double().cpu().numpy()
            tol = 2 * bound + (2.0 ** -8 * np.abs(want) if out == torch.bfloat16 else 0)
            worst = max(worst, float((np.abs(got - want) / tol).max()))
            assert np.all(np.abs(got - want) <= tol), (b, h, float((np.abs(got - want) / tol).max()))
            gl = lse[b, rows].double().cpu().numpy()
            assert np.all((gl == wl) | (np.abs(gl - wl) <= 2 * bl)), (b, h, gl, wl)
    st = hqmq.read_status(status)
    assert bool(st["flags"] & hqmq.FLAG_BAD_PAGE) == bool(bad)
    print("[paged attention] largest error / tolerance %.3g" % worst)


@pytest.mark.parametrize("B,Hk,G,page,S,cap,lens,prefix,out", [
    (1, 1, 1, 16, 8, 0, [1], 0, torch.float32),                        # one token
    (2, 2, 8, 64, 32, 128, [100, 37], 0, torch.float32),
    (3, 1, 7, 16, 8, 20, [5, 0, 130], 0, torch.bfloat16),              # an empty sequence: zeros
    (2, 2, 4, 32, 32, 64, [0, 0], 77, torch.float32),                  # the prefix alone is there
    (4, 2, 8, 64, 32, 128, [70, 1, 0, 64], 129, torch.float32),
    (3, 3, 16, 16, 48, 40, [33, 16, 17], 16, torch.bfloat16),          # 16 query heads to a KV head
    (20, 1, 7, 16, 3, 25, list(range(20)), 300, torch.float32),        # 140 rows: more than one tile of them
    (5, 1, 1, 128, 11, 256, [3, 9, 1, 0, 250], 1000, torch.float32),
    (2, 1, 3, 256, 1, 500, [257, 2], 511, torch.bfloat16),
    (33, 1, 8, 32, 32, 64, [1] * 33, 400, torch.float32),              # 264 rows
    (33, 2, 8, 64, 32, 128, [1, 70, 0] * 11, 700, torch.bfloat16),     # and in bf16: two groups of 128 at once
    (20, 1, 7, 16, 8, 0, [65, 3] * 10, 3, torch.bfloat16),
    (18, 5, 16, 32, 32, 64, list(range(18)), 200, torch.bfloat16),     # 288 rows: a second pair that is mostly empty
    (40, 1, 8, 64, 20, 128, [0] * 40, 129, torch.bfloat16)])           # another index width, prefix only
def test_against_plain_attention(B, Hk, G, page, S, cap, lens, prefix, out):
    run(np.random.default_rng(B * 100 + G), B, Hk, G, page, S, cap, lens, prefix, out)


def test_lengths_are_clamped_and_bad_pages_left_out():
    rng = np.random.default_rng(20)
    run(rng, 3, 2, 4, 16, 8, 20, [40, 33, 50], 50, bad=[(0, 1), (2, 0), (-1, 2)])
    run(rng, 2, 1, 8, 16, 32, 20, [20, 16], 16, bad=[(0, 0), (0, 1), (1, 0), (-1, 0)])    # nothing is left
    run(rng, 2, 1, 2, 16, 8, 0, [-4, 30], 0, max_extra=4)
    run(rng, 2, 1, 2, 16, 8, 0, [31, 16 * 3], 40, max_extra=9)


@pytest.mark.parametrize("scale,q_scale,spread", [(0.0, 1, 1), (-0.1, 1, 1), (1.0, 3, 2), (0.3, 20, 10), (1e-6, 1, 1)])
def test_scales_from_flat_to_one_hot(scale, q_scale, spread):
    run(np.random.default_rng(21), 3, 1, 5, 32, 32, 64, [90, 3, 41], 200, scale=scale, q_scale=q_scale, spread=spread)


def test_rising_scores():
    """Scores that rise along the tokens, so that the running maximum moves in every tile."""
    rng = np.random.default_rng(22)
    n, page = 700, 16
    pools = [filled_pool(rng, 50, 1, page, 8, 0) for _ in range(2)]
    pools[0]["words"][:] = np.array(P.pack_words([7] * 32, 8), np.uint32)
    r = (np.arange(50 * page) / 60).reshape(50, 1, page, 1) + np.zeros((1, 1, 1, 32))
    pools[0]["radius"] = P.f16_bits(r)
    c = P.codewords(pools[0]["cb"], True)[0, 7]
    q = torch.from_numpy(np.tile(c.astype(np.float32), 32)[None, None]).bfloat16()
    (kp, _), (vp, _) = (P.upload(p) for p in pools)
    table = np.arange(50, dtype=np.int32)
    for prefix, own in ((n, 0), (0, n), (300, 400)):
        o, lse = torch.empty(1, 1, 128, device="cuda"), torch.empty(1, 1, device="cuda")
        first = table[:-(-prefix // page)]
        mine = table[len(first):][:max(1, -(-own // page))][None]
        ws = hqmq.alloc_attention_paged_ws(1, 1, kp, mine.shape[1], prefix)
        hqmq.hqmq_attention_paged(q.cuda(), kp, vp, *cuda_ints(mine, [own]), o, ws, prefix_len=prefix,
                                  prefix_table=cuda_ints(first)[0], lse=lse)
        k = P.bf16(np.concatenate([P.dense(pools[0], first, prefix)[0], P.dense(pools[0], mine[0], own)[0]], 1))
        v = P.bf16(np.concatenate([P.dense(pools[1], first, prefix)[0], P.dense(pools[1], mine[0], own)[0]], 1))
        want, bound, wl, bl = plain(q[0].float().numpy(), k[0], v[0], np.ones(n, bool), 128 ** -0.5)
        assert np.all(np.abs(o[0].double().cpu().numpy() - want) <= 2 * bound)
        assert np.all(np.abs(lse[0].double().cpu().numpy() - wl) <= 2 * bl)


def test_nan_values_reach_only_their_rows_and_stale_rows_reach_none():
    """A NaN radius inside one sequence's tokens makes that sequence NaN; NaN and infinity in rows behind
    the last token, in pages of others and in slots that no flag reaches change nothing."""
    rng = np.random.default_rng(23)
    B, G, page = 3, 4, 16
    table, n = layout(rng, [20, 30, 40], page, spare=3)
    pools = [filled_pool(rng, n, 1, page, 8, 30) for _ in range(2)]
    free = np.setdiff1d(np.arange(n), table[table >= 0])[:2].astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((B, G, 128)).astype(np.float32)).bfloat16().cuda()
    out = []
    for poison in (False, True):
        for p in pools:
            if poison:
                p["radius"][table[0, 1], 0, 4:] = 0x7E00
                p["radius"][table[1, 1], 0, 14:] = 0x7C00
                p["radius"][free[1], 0, 9:] = 0x7E00                 # behind the prefix's 25 tokens
                p["flags"][table[2, 2], 0, 8:] = 0xFFFFFFFF
                p["val"][table[2, 2], 0, 29] = 0x7E00
                p["radius"][table[1, 0], 0, 3, 31] = 0x7E00          # a token of sequence 1
        (kp, _), (vp, _) = (P.upload(p) for p in pools)
        o = torch.empty(B, G, 128, device="cuda")
        ws = hqmq.alloc_attention_paged_ws(B, G, kp, table.shape[1], 25)
        hqmq.hqmq_attention_paged(q, kp, vp, *cuda_ints(table, [20, 30, 40]), o, ws, prefix_len=25,
                                  prefix_table=cuda_ints(free)[0])
        out.append(o.clone())
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][2], out[1][2])
    assert bool(torch.isnan(out[1][1]).all()) and not bool(torch.isnan(out[0]).any())


def test_rows_with_nothing_but_nan_are_nan():
    """Every score NaN (all radii NaN), in the prefix or in a sequence's own tokens: NaN, not 0."""
    rng = np.random.default_rng(27)
    pools = [filled_pool(rng, 4, 1, 16, 8, 0) for _ in range(2)]
    pools[0]["radius"][1] = 0x7E00
    (kp, _), (vp, _) = (P.upload(p) for p in pools)
    for rows in (1, 5):
        q = torch.from_numpy(rng.standard_normal((rows, 8, 128)).astype(np.float32)).bfloat16().cuda()
        for prefix, ln in ((16, 0), (0, 16), (16, 16)):
            for out in (torch.float32, torch.bfloat16):
                o = torch.zeros(rows, 8, 128, dtype=out, device="cuda")
                ws = hqmq.alloc_attention_paged_ws(rows, 8, kp, 1, prefix)
                t_d, l_d, p_d = cuda_ints([[1 if prefix == 0 else 2]] * rows, [ln] * rows, [1])
                hqmq.hqmq_attention_paged(q, kp, vp, t_d, l_d, o, ws, prefix_table=p_d, prefix_len=prefix)
                assert bool(torch.isnan(o).all())


def test_same_answer_again_on_other_streams_and_in_graphs():
    """Twice the same bits; two captured graphs and an eager call with workspaces of their own, replayed
    together on two streams."""
    rng = np.random.default_rng(24)
    B, Hk, G, page = 6, 2, 8, 64
    lens = [300, 2, 190, 64, 65, 0]
    table, n = layout(rng, lens, page, spare=12)
    pools = [filled_pool(rng, n, Hk, page, 32, 128) for _ in range(2)]
    free = np.setdiff1d(np.arange(n), table[table >= 0]).astype(np.int32)
    (kp, _), (vp, _) = (P.upload(p) for p in pools)
    t_d, len_d, pt_d = cuda_ints(table, lens, free)
    q = torch.from_numpy(rng.standard_normal((B, Hk * G, 128)).astype(np.float32)).bfloat16().cuda()
    outs = [torch.zeros(B, Hk * G, 128, device="cuda") for _ in range(4)]
    wss = [hqmq.alloc_attention_paged_ws(B, Hk * G, kp, table.shape[1], 700) for _ in range(4)]

    def call(i):
        hqmq.hqmq_attention_paged(q, kp, vp, t_d, len_d, outs[i], wss[i], prefix_table=pt_d, prefix_len=700)

    call(0)
    call(3)
    torch.cuda.synchronize()
    graphs = []
    for i in (1, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    first = outs[0].clone()
    streams = [torch.cuda.Stream() for _ in graphs]
    for rep in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        call(3)
        torch.cuda.synchronize()
        for o in outs[1:]:
            assert torch.equal(o, first)
    # a captured call follows lengths and queries that change between replays
    len_d.fill_(17)
    q.mul_(-1)
    graphs[0].replay()
    call(0)
    torch.cuda.synchronize()
    assert torch.equal(outs[1], outs[0]) and not torch.equal(outs[0], first)


def test_a_shared_prefix_is_the_same_as_every_sequence_having_it():
    """Prefix pages first in every block table, or as the shared prefix; and joined by lse from halves."""
    rng = np.random.default_rng(25)
    B, Hk, G, page = 5, 2, 4, 32
    lens = [40, 1, 64, 0, 33]
    prefix = 96
    table, n = layout(rng, lens, page, spare=3)
    pools = [filled_pool(rng, n, Hk, page, 32, 64) for _ in range(2)]
    free = np.setdiff1d(np.arange(n), table[table >= 0]).astype(np.int32)
    (kp, _), (vp, _) = (P.upload(p) for p in pools)
    q = torch.from_numpy(rng.standard_normal((B, Hk * G, 128)).astype(np.float32)).bfloat16().cuda()

    def call(tab, ln, pt, plen):
        o = torch.empty(B, Hk * G, 128, device="cuda")
        lse = torch.empty(B, Hk * G, device="cuda")
        t_d, l_d = (None, None) if tab is None else cuda_ints(tab, ln)
        ws = hqmq.alloc_attention_paged_ws(B, Hk * G, kp, 0 if tab is None else tab.shape[1], plen)
        hqmq.hqmq_attention_paged(q, kp, vp, t_d, l_d, o, ws, prefix_table=cuda_ints(pt)[0], prefix_len=plen, lse=lse)
        return o.double(), lse.double()

    both = np.concatenate([np.tile(free, (B, 1)), table], 1)
    o1, l1 = call(both, [prefix + t for t in lens], free, 0)
    o2, l2 = call(table, lens, free, prefix)
    op, lp = call(None, None, free, prefix)
    os_, ls = call(table, lens, free, 0)
    m = torch.logaddexp(lp, ls)
    o3 = (lp - m).exp()[..., None] * op + (ls - m).exp()[..., None] * os_
    # scores of |q k| up to about 40 here: dx 2^-15, d about 2^-14 of values up to 16
    for o, l in ((o2, l2), (o3, m)):
        assert float((o - o1).abs().max()) <= 4 * 2.0 ** -14 * 16
        assert float((l - l1).abs().max()) <= 2.0 ** -13


def test_refusals():
    rng = np.random.default_rng(26)
    pools = [P.empty_pool(rng, 4, 2, 16, 8, 16), P.empty_pool(rng, 4, 2, 32, 8, 16)]
    kp, vp = P.upload(pools[0])[0], P.upload(P.copy_pool(pools[0]))[0]
    other = P.upload(pools[1])[0]
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(1, 8, 128, device="cuda")
    t_d, len_d, pt = cuda_ints([[0, 1]], [20], [2, 3])
    ws = hqmq.alloc_attention_paged_ws(1, 8, kp, 2, 32)
    good = dict(q=q, k=kp, v=vp, block_table=t_d, seq_len=len_d, o=o, ws=ws, prefix_table=pt, prefix_len=32)
    hqmq.hqmq_attention_paged(**good)
    for change in (dict(q=q.float()), dict(o=o[:, :4]), dict(o=o.half()), dict(prefix_len=33), dict(prefix_table=None),
                   dict(seq_len=len_d.long()), dict(block_table=t_d[0]), dict(q=q.cpu()), dict(lse=o[0]),
                   dict(q=q.transpose(0, 1))):
        with pytest.raises((ValueError, TypeError)):
            hqmq.hqmq_attention_paged(**{**good, **change})
    for change in (dict(v=other), dict(ws=ws[:256]), dict(scale=float("inf")), dict(ws=ws[1:]),
                   dict(q=q[:, :7].contiguous(), o=o[:, :7].contiguous()), dict(prefix_len=-1, prefix_table=None)):
        with pytest.raises(hqmq.HQMQError):
            hqmq.hqmq_attention_paged(**{**good, **change})
    with pytest.raises(ValueError):
        hqmq.alloc_attention_paged_ws(1, 34, kp, 2, 0)            # 17 query heads to a KV head
