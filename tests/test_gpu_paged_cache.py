"""hqmq_paged_write and hqmq_paged_read against their definitions in 64 bits
(tests/_paged.py).  Everything stored is compared bit for bit (the write's
index is the argmax of the exact scores), and so is what is read back."""
import numpy as np
import pytest
import torch

import _paged as P
from kv_cache_quantization_hqmq_b200 import hqmq

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def tokens(rng, n, H, dt, strong=30.0):
    x = rng.standard_normal((n, H, 128)).astype(np.float32)
    x[:, :, 4 * (n % 32) + 1] *= strong
    x = torch.from_numpy(x).to(dt)
    return x, x.float().numpy()


def layout(rng, lens, P_, spare=2, width=0):
    """Shuffled block table for sequences of these lengths."""
    need = [-(-n // P_) for n in lens]
    perm = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(need + [width, 1])), -1, np.int32)
    k = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[k:k + n]
        k += n
    return table, sum(need) + spare


def cuda_ints(*arrays):
    return [torch.from_numpy(np.asarray(a, np.int32)).cuda() for a in arrays]


@pytest.mark.parametrize("S,page,H,dt,cap,old,new", [
    (32, 64, 2, torch.bfloat16, 128, [0, 63, 64, 10], [1, 1, 1, 1]),          # a decode step
    (32, 32, 3, torch.bfloat16, 64, [5, 0, 31], [70, 0, 33]),                 # runs over pages, an empty one
    (8, 16, 4, torch.float32, 0, [3, 16], [40, 1]),                           # no outliers
    (8, 16, 2, torch.float32, 10, [0, 7], [35, 20]),                          # slots run out
    (1, 128, 1, torch.bfloat16, 300, [0], [150]), (48, 256, 1, torch.bfloat16, 256, [200], [90]),
    (11, 64, 2, torch.float32, 1, [1], [65]), (3, 32, 5, torch.bfloat16, 1024, [0, 0, 0], [1, 2, 3])])
@pytest.mark.parametrize("tables", [False, True])
def test_write_then_read(S, page, H, dt, cap, old, new, tables):
    rng = np.random.default_rng(S * 1000 + page)
    table, n_pages = layout(rng, [a + b for a, b in zip(old, new)], page)
    cu = np.concatenate([[0], np.cumsum(new)])
    n = int(cu[-1])
    status, expect = hqmq.new_status(), dict(n_outliers=0, overflow=0, n_saturated=0, n_nonfinite=0)
    args, pools, xs = [], [], []
    for role in range(2):
        pool = P.empty_pool(rng, n_pages, H, page, S, cap)
        if cap:                        # what lies before the new rows is a cache: few flagged chunks
            pool["flags"] &= rng.integers(0, 1 << 32, pool["flags"].shape, dtype=np.uint64).astype(np.uint32)
            pool["flags"] &= rng.integers(0, 1 << 32, pool["flags"].shape, dtype=np.uint64).astype(np.uint32)
            pool["flags"] &= np.uint32(0x01010101 if cap > 10 else 0x01000000)
        x, xf = tokens(rng, n, H, dt)
        args.append((P.upload(pool, P.search_tables(pool["cb"]) if tables else None), x.cuda()))
        pools.append(pool)
        xs.append(xf)
    t_d, cu_d, pos_d = cuda_ints(table, cu, old)
    (kp, kt), (vp, vt) = args[0][0], args[1][0]
    hqmq.hqmq_paged_write(args[0][1], args[1][1], kp, vp, t_d, cu_d, pos_d, status=status)
    for pool, xf, t in zip(pools, xs, (kt, vt)):
        tally = P.write(pool, xf, table, cu, old)
        P.assert_pools_equal(t, pool)
        for key in expect:
            expect[key] += tally[key]
    st = hqmq.read_status(status)
    assert {k: st[k] for k in ("n_outliers", "n_saturated", "n_nonfinite")} == \
        {k: v for k, v in expect.items() if k != "overflow"}
    assert bool(st["flags"] & hqmq.FLAG_OUTLIER_OVERFLOW) == (expect["overflow"] > 0)
    assert not st["flags"] & hqmq.FLAG_BAD_PAGE
    assert (cap == 10) <= (expect["overflow"] > 0)
    lens = [a + b for a, b in zip(old, new)]
    T = max(lens) + 3
    for out in (torch.float32, torch.bfloat16):
        y = torch.full((len(lens), H, T, 128), 7.0, dtype=out, device="cuda")
        hqmq.hqmq_paged_read(vp, t_d, cuda_ints(lens)[0], y, status=status)
        for b, m in enumerate(lens):
            want, _ = P.dense(pools[1], table[b], m)
            got = y[b].float().cpu().numpy()
            np.testing.assert_array_equal(got[:, :m], P.bf16(want) if out == torch.bfloat16 else want)
            assert (got[:, m:] == 7).all()


def test_calls_of_any_split_give_the_same_pages():
    """50 tokens at once, in two calls, or one by one (with a rewrite of the last ten): same bits."""
    rng = np.random.default_rng(7)
    table, n_pages = layout(rng, [53], 16)
    base = P.empty_pool(rng, n_pages, 2, 16, 32, 24)
    base["flags"][table[0, 0], :, :3] = 0
    x = tokens(rng, 50, 2, torch.bfloat16)[0].cuda()
    tab = P.search_tables(base["cb"])
    results = []
    for cuts in ([0, 50], [0, 13, 50], list(range(51)), [0, 45, (35, 50)]):
        kp, t = P.upload(base, tab)
        at = 0
        for c in cuts[1:]:
            a, e = c if isinstance(c, tuple) else (at, c)
            hqmq.hqmq_paged_write(x[a:e], None, kp, None, *cuda_ints(table, [0, e - a], [3 + a]))
            at = e
        torch.cuda.synchronize()
        results.append(t)
    want = P.copy_pool(base)
    P.write(want, x.float().cpu().numpy(), table, [0, 50], [3])
    for t in results:
        P.assert_pools_equal(t, want)


def test_special_values():
    """Zeros, NaN, infinities, norms beyond fp16 and beyond fp32, subnormals: with and without a threshold."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((6, 2, 128)).astype(np.float32)
    x[0, 0, :16] = 0
    x[0, 1, 4] = np.nan
    x[1, 0, 9] = np.inf
    x[1, 1, 8:12] = [1e5, -7e4, 3, 0]
    x[2, 0, :4] = [3e38, 3e38, 0, 0]
    x[2, 1, :4] = [1e-30, 0, 0, 0]
    x[3, 0, 4:8] = [2e-20, -3e-20, 1e-21, 0]
    x[4, 1, 12:16] = [-np.inf, np.nan, 1, 1]
    x[5, 0, :8] = [1, 0, 0, 0, 0.5, 0.5, 0.5, -0.5]
    for cap in (0, 40):
        table, n_pages = layout(rng, [6], 16)
        pool = P.empty_pool(rng, n_pages, 2, 16, 8, cap)
        for tab in (None, P.search_tables(pool["cb"])):
            status = hqmq.new_status()
            want = P.copy_pool(pool)
            kp, t = P.upload(pool, tab)
            hqmq.hqmq_paged_write(torch.from_numpy(x).cuda(), None, kp, None, *cuda_ints(table, [0, 6], [0]),
                                  status=status)
            tally = P.write(want, x, table, [0, 6], [0])
            for key in ("flags", "radius", "words"):
                P.assert_pools_equal(t, {**want, "val": None})
            if cap:                     # NaN payloads aside, the stored values too
                a, b = t["val"].cpu().numpy().view(np.float16), want["val"].view(np.float16)
                np.testing.assert_array_equal(a, b)
            st = hqmq.read_status(status)
            assert (st["n_outliers"], st["n_saturated"], st["n_nonfinite"]) == \
                (tally["n_outliers"], tally["n_saturated"], tally["n_nonfinite"])


@pytest.mark.parametrize("tables", [False, True])
def test_near_ties_go_by_the_exact_scores(tables):
    """Directions half way between two codewords of a head, in fp32 and nudged by single bits."""
    rng = np.random.default_rng(9)
    pool = P.empty_pool(rng, 20, 1, 16, 32)
    c = P.codewords(pool["cb"], False)[0]
    x = np.zeros((256, 1, 32, 4), np.float32)
    for n in range(256):
        for k in range(32):
            i = rng.integers(0, 768)
            near = np.argsort(-(c @ c[i]))[1:5]
            mid = (c[i] + c[near[rng.integers(0, 4)]]).astype(np.float32)
            x[n, 0, k] = np.nextafter(mid, np.float32(rng.integers(-1, 2) * 9), dtype=np.float32) * np.float32(2.0 ** rng.integers(-8, 8))
    x = x.reshape(256, 1, 128)
    table, _ = layout(rng, [256], 16)
    kp, t = P.upload(pool, P.search_tables(pool["cb"]) if tables else None)
    hqmq.hqmq_paged_write(torch.from_numpy(x).cuda(), None, kp, None, *cuda_ints(table, [0, 256], [0]))
    P.write(pool, x, table, [0, 256], [0])
    P.assert_pools_equal(t, pool)


def test_strided_tokens_and_bad_places():
    """x as a view of the projection; positions past the table, a negative start, page ids out of
    range: those tokens are left out and flagged, the others are written."""
    rng = np.random.default_rng(10)
    H = 2
    buf = torch.from_numpy(rng.standard_normal((40, 3 * H, 128)).astype(np.float32)).bfloat16().cuda()
    xk, xv = buf[:, H:2 * H], buf[:, 2 * H:]
    table = np.array([[3, 1, -1], [0, 99, 2], [4, 5, 6], [7, 8, 9]], np.int32)
    cu, pos0 = [0, 12, 30, 34, 40], [14, 10, -2, 45]
    pools = [P.empty_pool(rng, 10, H, 16, 8, 20) for _ in range(2)]
    for p in pools:
        p["flags"][:] = 0
    status = hqmq.new_status()
    (kp, kt), (vp, vt) = (P.upload(p) for p in pools)
    hqmq.hqmq_paged_write(xk, xv, kp, vp, *cuda_ints(table, cu, pos0), status=status)
    for x, pool, t in ((xk, pools[0], kt), (xv, pools[1], vt)):
        tally = P.write(pool, x.float().cpu().numpy(), table, cu, pos0)
        assert tally["bad"] == 12 + 4 + 3
        P.assert_pools_equal(t, pool)
    assert hqmq.read_status(status)["flags"] & hqmq.FLAG_BAD_PAGE
    # reading: the bad page's rows and the rows past the table stay as they were
    status = hqmq.new_status()
    y = torch.full((4, H, 60, 128), 7.0, device="cuda")
    hqmq.hqmq_paged_read(kp, *cuda_ints(table, [60, 40, -5, 0])[:1], cuda_ints([60, 40, -5, 0])[0], y, status=status)
    for b, m in enumerate([60, 40, 0, 0]):
        want, ok = P.dense(pools[0], table[b], m)
        got = y[b].cpu().numpy()
        np.testing.assert_array_equal(got[:, :m][:, ok], want[:, ok])
        assert (got[:, m:] == 7).all() and (got[:, :m][:, ~ok] == 7).all()
    assert hqmq.read_status(status)["flags"] & hqmq.FLAG_BAD_PAGE


def test_index_out_of_range_reads_as_zero():
    rng = np.random.default_rng(11)
    pool = P.empty_pool(rng, 2, 1, 16, 8)                # noise: b = 8, indices 192 .. 255 among it
    kp, _ = P.upload(pool)
    y = torch.empty(1, 1, 32, 128, device="cuda")
    status = hqmq.new_status()
    hqmq.hqmq_paged_read(kp, *cuda_ints([[1, 0]], [32]), y, status=status)
    want, _ = P.dense(pool, [1, 0], 32)
    np.testing.assert_array_equal(y[0].cpu().numpy(), want)
    assert hqmq.read_status(status)["flags"] & hqmq.FLAG_BAD_INDEX


def test_many_sequences_one_token_each():
    """More sequences than one warp's scan takes, empty ones among them."""
    rng = np.random.default_rng(12)
    B = 150
    new = (rng.random(B) < 0.6).astype(int) * rng.integers(1, 4, B)
    old = rng.integers(0, 20, B)
    table, n_pages = layout(rng, (old + new).tolist(), 16)
    cu = np.concatenate([[0], np.cumsum(new)])
    pool = P.empty_pool(rng, n_pages, 1, 16, 8, 64)
    pool["flags"] &= np.uint32(0x11)
    x, xf = tokens(rng, int(cu[-1]), 1, torch.bfloat16)
    kp, t = P.upload(pool)
    hqmq.hqmq_paged_write(x.cuda(), None, kp, None, *cuda_ints(table, cu, old))
    P.write(pool, xf, table, cu, old)
    P.assert_pools_equal(t, pool)


def test_write_and_read_in_a_graph():
    rng = np.random.default_rng(13)
    table, n_pages = layout(rng, [40, 40], 16)
    pool = P.empty_pool(rng, n_pages, 2, 16, 32, 40)
    pool["flags"][:] = 0
    kp, t = P.upload(pool, P.search_tables(pool["cb"]))
    x = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    t_d, cu_d, pos_d, len_d = cuda_ints(table, [0, 1, 2], [0, 0], [0, 0])
    y = torch.zeros(2, 2, 40, 128, device="cuda")

    def step():
        hqmq.hqmq_paged_write(x, None, kp, None, t_d, cu_d, pos_d)
        hqmq.hqmq_paged_read(kp, t_d, len_d, y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):
        new, xf = tokens(rng, 2, 2, torch.bfloat16)
        x.copy_(new)
        pos_d.fill_(i)
        len_d.fill_(i + 1)
        graph.replay()
        P.write(pool, xf, table, [0, 1, 2], [i, i])
    P.assert_pools_equal(t, pool)
    for b in range(2):
        want, _ = P.dense(pool, table[b], 20)
        np.testing.assert_array_equal(y[b, :, :20].cpu().numpy(), want)
    assert bool((y[:, :, 20:] == 0).all())


def test_refusals():
    rng = np.random.default_rng(14)
    pool = P.empty_pool(rng, 4, 2, 16, 8, 16)
    kp, t = P.upload(pool)
    noflags, _ = P.upload({**pool, "thr": None})
    x = torch.zeros(3, 2, 128, device="cuda")
    t_d, cu_d, pos_d = cuda_ints([[0, 1]], [0, 3], [0])
    with pytest.raises(hqmq.HQMQError):                   # flags without a threshold
        hqmq.hqmq_paged_write(x, None, noflags, None, t_d, cu_d, pos_d)
    for bad in (x[:, :1], x[:, :, :64], x.transpose(1, 2), x.half(), x.cpu()):
        with pytest.raises((ValueError, TypeError)):
            hqmq.hqmq_paged_write(bad, None, kp, None, t_d, cu_d, pos_d)
    for bad in ((t_d.long(), cu_d, pos_d), (t_d[0], cu_d, pos_d), (t_d, cu_d[:1], pos_d), (t_d, cu_d, pos_d.float()),
                (t_d.cpu(), cu_d, pos_d)):
        with pytest.raises(ValueError):
            hqmq.hqmq_paged_write(x, None, kp, None, *bad)
    odd = torch.zeros(3, 2, 130, device="cuda")[:, :, 1:129]
    with pytest.raises(hqmq.HQMQError):
        hqmq.hqmq_paged_write(odd, None, kp, None, t_d, cu_d, pos_d)
    hqmq.hqmq_paged_write(x[:0], None, kp, None, t_d, cu_d, pos_d)      # nothing to do
    for bad in (torch.zeros(1, 3, 8, 128, device="cuda"), torch.zeros(1, 2, 8, 64, device="cuda"),
                torch.zeros(1, 2, 8, 128, dtype=torch.half, device="cuda")):
        with pytest.raises((ValueError, TypeError)):
            hqmq.hqmq_paged_read(kp, t_d, pos_d, bad)
    with pytest.raises(ValueError):
        hqmq.kv_pages(t["words"], t["radius"], t["cb"][:1], t["flags"], t["val"])
    with pytest.raises(ValueError):
        hqmq.kv_pages(t["words"], t["radius"], t["cb"], t["flags"], None)
