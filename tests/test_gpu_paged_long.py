"""hqmq_attention_paged where a CTA takes many tiles: several times 148 tiles of
64 tokens, so that running maxima, accumulators, stages and rings carry from
tile to tile, and shares pass from segment to segment, from two groups of rows
to replicated ones and back, and from head to head.  The bounds are those of
tests/_paged_fast.py, element by element; a weight enters P V as three bf16
terms for fp32 outputs (2^-24 left) and as two for bf16 outputs (a term leaves
at most half a step of its value: 2^-8, and the second of what is left, which
is below a power of two, 2^-9 more: 2^-17)."""
import numpy as np
import pytest
import torch

import _paged as P
import _paged_fast as F

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

BF, F32 = torch.bfloat16, torch.float32
WEIGHT = {F32: 2.0 ** -24, BF: 2.0 ** -17}


def tiles(x, out):
    """Tiles of all heads, by the call's definition of its work."""
    rows = x.B * x.G
    groups = 0 if not x.prefix else -(-rows // (256 if out == BF and rows > 128 else 128))
    return x.Hk * (groups * -(-x.prefix // 64) + sum(-(-n // 64) for n in x.lens))


CASES = {
    # every head its own KV head, replicated rows over the prefix and after it
    "heads": dict(B=6, Hk=32, G=1, page=16, S=8, cap=32, lens=[400, 5, 0, 250, 64, 333], prefix=500),
    # no prefix: long and short sequences
    "own": dict(B=9, Hk=8, G=8, page=64, S=32, cap=128, lens=[3000, 1, 700, 64, 0, 1500, 130, 2048, 65], prefix=0),
    # 70 rows over the prefix, a row per thread
    "rows70": dict(B=10, Hk=4, G=7, page=32, S=16, cap=64, lens=[0, 300, 1, 64, 65, 129, 10, 200, 0, 250], prefix=9000),
    # 160 rows: two row tiles (fp32) or two groups at once (bf16), the second in part
    "rows160": dict(B=20, Hk=4, G=8, page=64, S=32, cap=128, lens=[0, 70, 1, 200] * 5, prefix=9000),
    # 320 rows: a pair of groups, and a pair whose second group is empty
    "rows320": dict(B=40, Hk=8, G=8, page=64, S=32, cap=128, lens=[1, 64, 0, 130] * 10, prefix=5000),
    # pieces longer than all rings
    "rows264": dict(B=33, Hk=8, G=8, page=64, S=32, cap=128, lens=[100] * 33, prefix=24000),
    # large pages, few own tokens
    "page256": dict(B=18, Hk=2, G=16, page=256, S=48, cap=700, lens=[300, 0, 2] * 6, prefix=20001),
    # K and V of different widths, K without flagged chunks
    "mixed": dict(B=17, Hk=6, G=8, page=128, S=8, cap=0, Sv=32, capv=200, lens=[90] * 17, prefix=5000)}


@pytest.mark.parametrize("out", [F32, BF])
@pytest.mark.parametrize("case", CASES)
def test_many_tiles_a_cta(case, out):
    x = F.Batch(len(case), **CASES[case])
    assert tiles(x, out) > 4 * 148
    o, lse = x.call(out)
    print("[paged attention, long] %s: largest error / bound %.3g" % (case, x.check(o, lse, WEIGHT[out])))


@pytest.mark.parametrize("B,Hk,G,lens,prefix", [
    (3, 2, 8, [500, 20, 0], 700), (10, 2, 8, [60] * 10, 900), (33, 2, 8, [1, 70, 0] * 11, 1000)])
def test_bf16_outputs_are_the_fp32_ones_rounded(B, Hk, G, lens, prefix):
    """Apart from the output's own rounding, a bf16 output is as good as two terms a weight: 2^-17."""
    x = F.Batch(B, B, Hk, G, 64, 32, 128, lens, prefix)
    o32, lse = x.call(F32)
    o16, lse16 = x.call(BF)
    x.check(o32, lse, WEIGHT[F32])
    x.check(o16, lse16, WEIGHT[BF])


def sawtooth(period, rise):
    """K pools whose scores rise by `rise` of radius a token over `period` tokens, then start anew; one
    codeword throughout, so that a query along it scores its norm times the radius."""
    def make(rng, n, table, ptable):
        Hk, page = make.Hk, make.page
        pools = [F.filled_pool(rng, n, Hk, page, 8, 0) for _ in range(2)]
        pools[0]["words"][:] = np.array(P.pack_words([7] * 32, 8), np.uint32)
        t = np.zeros((n, page), np.float32)
        for row in [ptable] + [r[r >= 0] for r in table]:
            t[row] = np.arange(len(row) * page).reshape(-1, page)
        r = (t % period) * rise
        pools[0]["radius"] = P.f16_bits(np.broadcast_to(r[:, None, :, None], pools[0]["radius"].shape))
        make.codeword = P.codewords(pools[0]["cb"], True)[:, 7]
        return pools
    return make


@pytest.mark.parametrize("out", [F32, BF])
@pytest.mark.parametrize("B,Hk,G,lens,prefix", [
    (1, 4, 1, [0], 40000), (2, 8, 2, [20000, 17000], 0), (8, 4, 8, [100] * 8, 30000), (25, 4, 8, [70] * 25, 30000)])
def test_rising_scores_move_the_maximum_again_and_again(B, Hk, G, lens, prefix, out):
    """Scores that rise over 1280 tokens and fall back, rows of one warp by different amounts."""
    make = sawtooth(1280, 0.03)
    make.Hk, make.page = Hk, 64
    x = F.Batch(5, B, Hk, G, 64, 8, 0, lens, prefix, pools=make)
    c = np.tile(make.codeword.astype(np.float32), 32).reshape(1, Hk, 1, 128)
    size = np.linspace(0.2, 1.0, B * G).reshape(B, 1, G, 1)
    x.q = torch.from_numpy((c * size).reshape(B, Hk * G, 128).astype(np.float32)).bfloat16().cuda()
    assert tiles(x, out) > 4 * 148
    o, lse = x.call(out)
    print("[paged attention, rising] %d rows: largest error / bound %.3g" % (B * G, x.check(o, lse, WEIGHT[out])))


def test_nan_stays_in_its_sequence_and_its_head():
    """A NaN among the own tokens of one sequence, in shares that pass through its neighbours."""
    lens = [900, 300, 0, 640, 70, 1000, 33, 64]
    x = F.Batch(6, 8, 16, 4, 32, 32, 64, lens, 700)
    o0, _ = x.call(F32)
    b, h = 3, 5
    t = next(t for t in range(333, 640) if not x.pools[1]["flags"][x.table[b, t // 32], h, t % 32] >> 9 & 1)
    x.pools[1]["radius"][x.table[b, t // 32], h, t % 32, 9] = 0x7E00
    x.vp = P.upload(x.pools[1])[0]
    o1, _ = x.call(F32)
    hit = torch.zeros_like(o0, dtype=torch.bool)
    hit[b, h * 4:(h + 1) * 4, 36:40] = True
    assert bool(torch.isnan(o1[hit]).all()) and torch.equal(o0[~hit], o1[~hit])


def test_the_same_bits_again():
    """Repeated calls, with other work between them, give the same bits."""
    x = F.Batch(7, **CASES["rows320"])
    y = F.Batch(8, **CASES["heads"])
    for out in (BF, F32):
        first = [t.clone() for t in x.call(out)]
        for _ in range(5):
            y.call(out)
            again = x.call(out)
            assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_rows_whose_scores_are_all_minus_infinity_count_as_empty():
    """An infinite query against keys of one sign: o = 0 and lse = -inf, as the header says; NaN with the
    other sign; the neighbours' rows stay."""
    def pools(rng, n, table, ptable):
        p = [F.filled_pool(rng, n, 2, 32, 8, 0) for _ in range(2)]
        p[0]["words"][:] = np.array(P.pack_words([3] * 32, 8), np.uint32)
        p[0]["radius"][:] = P.f16_bits(np.float32(1.5))
        pools.sign = np.sign(P.codewords(p[0]["cb"], True)[:, 3, 0]).astype(np.float32)
        return p
    x = F.Batch(9, 3, 2, 2, 32, 8, 0, [70, 0, 33], 100, pools=pools)
    for out in (F32, BF):
        base = x.q.clone()
        o0, lse0 = x.call(out)
        x.q[1, 0] = 0
        x.q[1, 0, 8] = -float("inf") * float(pools.sign[0])
        x.q[2, 3] = 0
        x.q[2, 3, 4] = float("inf") * float(pools.sign[1])
        o1, lse1 = x.call(out)
        assert bool((o1[1, 0] == 0).all()) and float(lse1[1, 0]) == -float("inf")
        assert bool(torch.isnan(o1[2, 3]).all())
        same = torch.ones(3, 4, dtype=torch.bool, device="cuda")
        same[1, 0] = same[2, 3] = False
        assert torch.equal(o0[same], o1[same]) and torch.equal(lse0[same], lse1[same])
        x.q = base


@pytest.mark.parametrize("out", [F32, BF])
@pytest.mark.parametrize("B,Hk,G,lens,prefix", [
    (1501, 1, 1, [0, 1, 0, 70, 2] * 300 + [0], 65), (700, 1, 1, [0] * 698 + [1, 0], 0), (2, 257, 2, [3, 130], 20),
    (1, 1024, 16, [5], 0)])
def test_many_sequences_and_many_heads(B, Hk, G, lens, prefix, out):
    """Lists of segments that are mostly empty, and shares of many heads."""
    x = F.Batch(10, B, Hk, G, 16, 3, 20, lens, prefix)
    o, lse = x.call(out)
    x.check(o, lse, WEIGHT[out])
