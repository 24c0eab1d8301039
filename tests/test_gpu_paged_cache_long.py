"""hqmq_paged_read and hqmq_paged_write where a CTA takes many tokens: reads of
64, 128 and 256 tokens a CTA (the call halves 256 until there are 296 CTAs),
whose slots are scanned over several warps and pages, and writes of several
blocks of 64 tokens in one page through the search tables, whose slots carry
from block to block.  Everything is compared bit for bit (tests/_paged.py,
tests/_paged_fast.py)."""
import numpy as np
import pytest
import torch

import _paged as P
import _paged_fast as F
from test_gpu_paged_cache import cuda_ints, layout, tokens
from kv_cache_quantization_hqmq_b200 import hqmq

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def read_span(T, heads, n_seqs):
    span = 256
    while span > 32 and -(-T // span) * heads * n_seqs < 296:
        span //= 2
    return span


@pytest.mark.parametrize("span,heads,lens,T", [
    (64, 8, [1200, 611], 1203), (128, 16, [1200, 0, 129], 1200), (256, 32, [1500, 700, 1, 257], 1500)])
@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("S,full", [(32, False), (8, True)])
def test_reads_of_many_tokens_a_cta(span, heads, lens, T, page, S, full):
    """Dense flagged chunks, with slots for all of them or (full) for a part of a page's."""
    assert read_span(T, heads, len(lens)) == span
    rng = np.random.default_rng(span + page)
    table, n = layout(rng, lens, page)
    pool = P.empty_pool(rng, n, heads, page, S, 3 * page if full else 32 * page)
    pool["flags"] &= rng.integers(0, 1 << 32, pool["flags"].shape, dtype=np.uint64).astype(np.uint32)
    pool["flags"] &= rng.integers(0, 1 << 32, pool["flags"].shape, dtype=np.uint64).astype(np.uint32)
    pool["words"] = F.pack_all(rng.integers(0, 24 * S, pool["radius"].shape), pool["words"].shape[3])
    used = np.bitwise_count(pool["flags"]).sum(-1) if hasattr(np, "bitwise_count") else None
    assert used is None or bool((used > pool["cap"]).any()) == full
    kp, _ = P.upload(pool)
    t_d, len_d = cuda_ints(table, lens)
    vals = F.values(pool)
    for out in (torch.float32, torch.bfloat16):
        status = hqmq.new_status()
        y = torch.full((len(lens), heads, T, 128), 7.0, dtype=out, device="cuda")
        hqmq.hqmq_paged_read(kp, t_d, len_d, y, status=status)
        for b, m in enumerate(lens):
            want = np.ascontiguousarray(F.dense(vals, table[b], m))
            got = y[b].float().cpu().numpy()
            np.testing.assert_array_equal(got[:, :m], P.bf16(want) if out == torch.bfloat16 else want)
            assert (got[:, m:] == 7).all()
        assert hqmq.read_status(status)["flags"] == 0


def test_reads_with_bad_pages_inside_a_cta():
    """A bad page among the several of a CTA: its rows stay, and the next page's slots start anew."""
    rng = np.random.default_rng(31)
    lens, heads, page = [900, 800, 512], 40, 64
    assert read_span(900, heads, 3) == 256
    table, n = layout(rng, lens, page)
    pool = F.filled_pool(rng, n, heads, page, 32, 40)
    vals = F.values(pool)
    table[0, 1], table[0, 5], table[1, 0], table[2, 7] = -1, n, -7, 1 << 30
    kp, _ = P.upload(pool)
    status = hqmq.new_status()
    y = torch.full((3, heads, 900, 128), 7.0, device="cuda")
    hqmq.hqmq_paged_read(kp, *cuda_ints(table, lens), y, status=status)
    got = y.cpu().numpy()
    for b, m in enumerate(lens):
        ok = ((table[b] >= 0) & (table[b] < n)).repeat(page)[:m]
        want = F.dense(vals, np.where((table[b] >= 0) & (table[b] < n), table[b], 0), m)
        np.testing.assert_array_equal(got[b][:, :m][:, ok], want[:, ok])
        assert (got[b][:, :m][:, ~ok] == 7).all() and (got[b][:, m:] == 7).all()
    assert hqmq.read_status(status)["flags"] == hqmq.FLAG_BAD_PAGE


@pytest.mark.parametrize("S,page,row0,new,cap", [
    (32, 256, 0, [256], 8192), (32, 256, 37, [219], 8192), (8, 256, 0, [240], 700),      # slots run out in a later block
    (8, 128, 37, [300, 91], 60), (32, 128, 0, [128, 120], 4096), (48, 256, 5, [251, 200], 1500)])
def test_writes_of_many_tokens_to_a_page(S, page, row0, new, cap):
    rng = np.random.default_rng(S + page + row0)
    old = [row0] * len(new)
    table, n_pages = layout(rng, [a + b for a, b in zip(old, new)], page)
    cu = np.concatenate([[0], np.cumsum(new)])
    pool = P.empty_pool(rng, n_pages, 1, page, S, cap, thr=2.2)                          # about a third is above 2.2
    pool["flags"] &= np.uint32(0x00400010)
    x, xf = tokens(rng, int(cu[-1]), 1, torch.bfloat16)
    status = hqmq.new_status()
    kp, t = P.upload(pool, P.search_tables(pool["cb"]))
    hqmq.hqmq_paged_write(x.cuda(), None, kp, None, *cuda_ints(table, cu, old), status=status)
    tally = P.write(pool, xf, table, cu, old)
    P.assert_pools_equal(t, pool)
    st = hqmq.read_status(status)
    assert st["n_outliers"] == tally["n_outliers"] > 20 * len(new)
    assert bool(st["flags"] & hqmq.FLAG_OUTLIER_OVERFLOW) == (tally["overflow"] > 0) == (cap in (60, 700, 1500))


@pytest.mark.parametrize("new,tables", [(3, False), (80, True)])
def test_a_start_below_zero_leaves_the_whole_sequence_out(new, tables):
    """As the header says: also the tokens whose positions would be 0 and more; the neighbours are written."""
    rng = np.random.default_rng(41)
    table, n_pages = layout(rng, [new, new, new], 16)
    cu, pos0 = [0, new, 2 * new, 3 * new], [0, -1, 0]
    pool = P.empty_pool(rng, n_pages, 2, 16, 32, 24)
    x, xf = tokens(rng, 3 * new, 2, torch.bfloat16)
    status = hqmq.new_status()
    kp, t = P.upload(pool, P.search_tables(pool["cb"]) if tables else None)
    hqmq.hqmq_paged_write(x.cuda(), None, kp, None, *cuda_ints(table, cu, pos0), status=status)
    assert P.write(pool, xf, table, cu, pos0)["bad"] == new
    P.assert_pools_equal(t, pool)
    assert hqmq.read_status(status)["flags"] & hqmq.FLAG_BAD_PAGE


def test_special_values_through_the_tables():
    """Zeros, NaN, infinities, norms beyond fp16 and fp32 and next to their ends, among runs long enough
    for the search tables."""
    rng = np.random.default_rng(42)
    x = rng.standard_normal((70, 2, 128)).astype(np.float32)
    x[3, 0] = 0
    x[5, 1, 4] = np.nan
    x[8, 0, 9] = np.inf
    x[11, 1, 8:12] = [1e5, -7e4, 3, 0]
    x[20, 0, :4] = [3e38, 3e38, 0, 0]
    x[21, 0, :8] = [1.8e19, 0, 0, 0, 9e18, -9e18, 9e18, 9e18]          # squares next to the largest fp32
    x[22, 1, :4] = [1e-30, 0, 0, 0]
    x[23, 1, :12] = [2e-20, -3e-20, 1e-21, 0, 4e-23, 0, 0, 0, 0, 0, -3e-22, 1e-45]
    x[30, 1, 12:16] = [-np.inf, np.nan, 1, 1]
    x[40, 0, :8] = [1, 0, 0, 0, 0.5, 0.5, 0.5, -0.5]
    x[64:, 1, 64:] *= 1e4
    for S, cap in ((32, 0), (32, 40), (8, 400), (48, 100)):
        table, n_pages = layout(rng, [70], 64)
        pool = P.empty_pool(rng, n_pages, 2, 64, S, cap)
        status = hqmq.new_status()
        want = P.copy_pool(pool)
        kp, t = P.upload(pool, P.search_tables(pool["cb"]))
        hqmq.hqmq_paged_write(torch.from_numpy(x).cuda(), None, kp, None, *cuda_ints(table, [0, 70], [0]), status=status)
        tally = P.write(want, x, table, [0, 70], [0])
        P.assert_pools_equal(t, {**want, "val": None})
        if cap:                        # NaN payloads aside, the stored values too
            np.testing.assert_array_equal(t["val"].cpu().numpy().view(np.float16), want["val"].view(np.float16))
        st = hqmq.read_status(status)
        assert (st["n_outliers"], st["n_saturated"], st["n_nonfinite"]) == \
            (tally["n_outliers"], tally["n_saturated"], tally["n_nonfinite"])


@pytest.mark.parametrize("Sk,Sv,capk,capv,tk,tv", [
    (8, 32, 0, 64, True, True), (32, 8, 30, 0, True, True), (1, 48, 64, 7, True, True), (48, 11, 200, 200, True, False),
    (3, 9, 0, 40, False, False)])
@pytest.mark.parametrize("new", [[1, 0, 2], [70, 30, 0]])
def test_k_and_v_of_different_kinds(Sk, Sv, capk, capv, tk, tv, new):
    """Codebook sizes, flags, tables and pool sizes of their own; a page id that only K has."""
    rng = np.random.default_rng(Sk + Sv)
    old = [3, 5, 16]
    table, n = layout(rng, [a + b for a, b in zip(old, new)], 32)
    cu = np.concatenate([[0], np.cumsum(new)])
    last = table[0, (old[0] + new[0] - 1) // 32]
    is_last, is_top = table == last, table == n - 1
    table[is_top] = last
    table[is_last] = n - 1                                            # K's last page, which V lacks
    status, args, pools, xs = hqmq.new_status(), [], [], []
    for S, cap, tab, pages in ((Sk, capk, tk, n), (Sv, capv, tv, n - 1)):
        pool = P.empty_pool(rng, pages, 3, 32, S, cap)
        if cap:
            pool["flags"] &= np.uint32(0x01000010)
        x, xf = tokens(rng, int(cu[-1]), 3, torch.float32)
        args.append((*P.upload(pool, P.search_tables(pool["cb"]) if tab else None), x.cuda()))
        pools.append(pool)
        xs.append(xf)
    (kp, kt, xk), (vp, vt, xv) = args
    hqmq.hqmq_paged_write(xk, xv, kp, vp, *cuda_ints(table, cu, old), status=status)
    bad = [P.write(pool, xf, table, cu, old)["bad"] for pool, xf in zip(pools, xs)]
    assert bad[0] == 0 < bad[1]
    P.assert_pools_equal(kt, pools[0])
    P.assert_pools_equal(vt, pools[1])
    assert hqmq.read_status(status)["flags"] & hqmq.FLAG_BAD_PAGE


def test_as_many_heads_as_there_may_be():
    rng = np.random.default_rng(43)
    table, n = layout(rng, [20, 3], 16)
    pool = P.empty_pool(rng, n, 1024, 16, 5, 9)
    pool["flags"] &= np.uint32(0x00100001)
    x, xf = tokens(rng, 5, 1024, torch.bfloat16)
    kp, t = P.upload(pool)
    hqmq.hqmq_paged_write(x.cuda(), None, kp, None, *cuda_ints(table, [0, 3, 5], [17, 1]))
    P.write(pool, xf, table, [0, 3, 5], [17, 1])
    P.assert_pools_equal(t, pool)
    pool["words"] = F.pack_all(F.unpack_all(pool["words"], pool["words"].shape[3]) % (24 * 5), pool["words"].shape[3])
    kp, _ = P.upload(pool)
    y = torch.full((2, 1024, 20, 128), 7.0, device="cuda")
    hqmq.hqmq_paged_read(kp, *cuda_ints(table, [20, 3]), y)
    vals = F.values(pool)
    for b, m in enumerate([20, 3]):
        np.testing.assert_array_equal(y[b, :, :m].cpu().numpy(), F.dense(vals, table[b], m))
        assert bool((y[b, :, m:] == 7).all())
