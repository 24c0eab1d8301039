"""The paged cache's and the rotation's entry points refuse what they do not
take before any CUDA call (no GPU needed), and the tests' plain forms agree
with the oracle."""
import ctypes

import numpy as np
import pytest

P = ctypes.c_void_p
GOOD, ODD = P(1 << 20), P((1 << 20) + 2)
F = ctypes.c_float


@pytest.fixture(scope="module")
def hq():
    from kv_cache_quantization_hqmq_b200 import build
    build.build()
    from kv_cache_quantization_hqmq_b200 import hqmq
    return hqmq


def pages(hq, **change):
    p = hq.KVPages(GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, None, 8, 4, 16, 2, 8)
    for k, v in change.items():
        setattr(p, k, v)
    return p


BAD_PAGES = [dict(idx_words=None), dict(radius=None), dict(codebook=None), dict(out_val=None), dict(S=0), dict(S=49),
             dict(n_pages=0), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(heads=0),
             dict(heads=1025), dict(out_cap=0), dict(out_cap=513)]
MISALIGNED = [dict(idx_words=ODD), dict(radius=ODD), dict(flags=ODD), dict(out_val=ODD), dict(codebook=ODD),
              dict(thr=ODD), dict(table=ODD)]


def write(hq, k, v=None, **c):
    a = dict(xk=GOOD, xv=None, dtype=0, s=(256, 128, 0, 0), n=3, seqs=1, cu=GOOD, pos0=GOOD, bt=GOOD, mp=2, st=None)
    a.update(c)
    return hq.lib().hqmq_paged_write(ctypes.byref(k), v and ctypes.byref(v), a["xk"], a["xv"], a["dtype"], *a["s"],
                                     a["n"], a["seqs"], a["cu"], a["pos0"], a["bt"], a["mp"], a["st"], None)


def read(hq, c, **ch):
    a = dict(seqs=1, ln=GOOD, bt=GOOD, mp=2, T=8, y=GOOD, dt=1, st=None)
    a.update(ch)
    return hq.lib().hqmq_paged_read(ctypes.byref(c), a["seqs"], a["ln"], a["bt"], a["mp"], a["T"], a["y"], a["dt"],
                                    a["st"], None)


def attend(hq, k, v, **ch):
    a = dict(q=GOOD, B=1, Hq=4, ln=GOOD, bt=GOOD, mp=2, pt=GOOD, pl=16, scale=0.1, o=GOOD, dt=1, lse=None, ws=GOOD,
             n=1 << 30, st=None)
    a.update(ch)
    return hq.lib().hqmq_attention_paged(a["q"], ctypes.byref(k), ctypes.byref(v), a["B"], a["Hq"], a["ln"], a["bt"],
                                         a["mp"], a["pt"], a["pl"], F(a["scale"]), a["o"], a["dt"], a["lse"], a["ws"],
                                         a["n"], a["st"], None)


def test_page_records(hq):
    for change in BAD_PAGES:
        p = pages(hq, **change)
        assert write(hq, p) == 1 and read(hq, p) == 1 and attend(hq, p, pages(hq)) == 1, change
        assert attend(hq, pages(hq), p) == 1 and write(hq, pages(hq), p, xv=GOOD) == 1, change
    for change in MISALIGNED:
        p = pages(hq, **change)
        assert write(hq, p) == 2 and read(hq, p) == 2 and attend(hq, p, pages(hq)) == 2, change


def test_write_arguments(hq):
    k = pages(hq)
    assert write(hq, pages(hq, thr=None)) == 1                            # flags without a threshold
    for c in (dict(dtype=2), dict(n=-1), dict(seqs=0), dict(seqs=65536), dict(mp=0), dict(mp=1 << 28), dict(xk=None),
              dict(cu=None), dict(pos0=None), dict(bt=None)):
        assert write(hq, k, **c) == 1, c
    for v in (pages(hq, page_size=32), pages(hq, heads=3)):
        assert write(hq, k, v, xv=GOOD) == 1
    assert write(hq, k, pages(hq), xv=None) == 1
    for c in (dict(xk=P((1 << 20) + 8)), dict(cu=ODD), dict(pos0=ODD), dict(bt=ODD), dict(st=P((1 << 20) + 4)),
              dict(s=(254, 128, 0, 0)), dict(s=(256, 2, 0, 0))):
        assert write(hq, k, **c) == 2, c
    assert write(hq, k, pages(hq), xv=GOOD, s=(256, 128, 255, 128)) == 2
    assert write(hq, k, n=0) == 0


def test_read_arguments(hq):
    c = pages(hq)
    for ch in (dict(seqs=0), dict(seqs=65536), dict(mp=0), dict(T=-1), dict(dt=3), dict(ln=None), dict(bt=None),
               dict(y=None)):
        assert read(hq, c, **ch) == 1, ch
    for ch in (dict(y=P((1 << 20) + 8)), dict(ln=ODD), dict(bt=ODD), dict(st=P((1 << 20) + 4))):
        assert read(hq, c, **ch) == 2, ch
    assert read(hq, c, T=0) == 0


def test_attention_arguments(hq):
    k, v = pages(hq), pages(hq)
    for ch in (dict(B=0), dict(B=65536), dict(Hq=0), dict(Hq=3), dict(Hq=34), dict(mp=-1), dict(mp=1 << 28),
               dict(pl=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(o=None), dict(ws=None),
               dict(ln=None), dict(bt=None), dict(pt=None), dict(dt=2)):
        assert attend(hq, k, v, **ch) == 1, ch
    for v2 in (pages(hq, page_size=32), pages(hq, heads=4)):
        assert attend(hq, k, v2) == 1
    for ch in (dict(q=P((1 << 20) + 8)), dict(o=P((1 << 20) + 8)), dict(ln=ODD), dict(bt=ODD), dict(pt=ODD),
               dict(lse=ODD), dict(ws=P((1 << 20) + 16)), dict(st=P((1 << 20) + 4))):
        assert attend(hq, k, v, **ch) == 2, ch
    need = hq.hqmq_attention_paged_workspace_size(1, 4, 2, 32, 16)
    assert need > 0 and attend(hq, k, v, n=need - 1) == 4
    assert hq.hqmq_attention_paged_workspace_size(1, 4, 3, 32, 16) == 0
    assert hq.hqmq_attention_paged_workspace_size(1, 34, 2, 32, 16) == 0
    assert hq.hqmq_attention_paged_workspace_size(1, 4, 2, -1, 16) == 0


def test_norm_rope_arguments(hq):
    def call(**ch):
        a = dict(q=hq._HeadView(GOOD, 512, 512, 128, 4), qo=hq._HeadView(GOOD, 512, 512, 128, 4), k=None, ko=None, dt=0,
                 B=1, T=2, D=128, qw=None, kw=None, wdt=0, eps=1e-6, pos=GOOD, inv=GOOD, R=128, il=0)
        a.update(ch)
        ref = [x and ctypes.byref(x) for x in (a["q"], a["qo"], a["k"], a["ko"])]
        return hq.lib().hqmq_qk_norm_rope(*ref, a["dt"], a["B"], a["T"], a["D"], a["qw"], a["kw"], a["wdt"],
                                          F(a["eps"]), a["pos"], a["inv"], a["R"], a["il"], None)

    V = hq._HeadView
    for ch in (dict(dt=2), dict(wdt=2), dict(B=-1), dict(T=-1), dict(D=0), dict(D=513), dict(R=-2), dict(R=130),
               dict(R=3), dict(inv=None), dict(eps=-1.0), dict(eps=float("inf")), dict(q=None), dict(qo=None),
               dict(q=None, qo=None), dict(qo=V(GOOD, 512, 512, 128, 3)), dict(q=V(None, 512, 512, 128, 4)),
               dict(q=V(GOOD, 512, 512, 128, 0), qo=V(GOOD, 512, 512, 128, 0)), dict(pos=None), dict(B=1 << 16, T=1 << 16)):
        assert call(**ch) == 1, ch
    for ch in (dict(q=V(P((1 << 20) + 1), 512, 512, 128, 4)), dict(pos=ODD), dict(inv=P((1 << 20) + 4)),
               dict(qw=ODD, wdt=1)):
        assert call(**ch) == 2, ch
    assert call(T=0) == 0


def test_plain_forms_agree_with_the_oracle(oracle, hq):
    """The tests' own write and read against the oracle's encode, list and decode (indices: these inputs
    have no near ties, which the oracle's scores show)."""
    import _paged as pg
    rng = np.random.default_rng(1)
    H, T, S = 3, 40, 32
    pool = pg.empty_pool(rng, 3, H, 16, S, 200)
    x = rng.standard_normal((1, H, T, 128)).astype(np.float32)
    x[..., 9] *= 30
    thr = pool["thr"]
    cb = pool["cb"]
    words, radius, best, second, _ = oracle.encode(x, cb.reshape(-1), S, thr=thr)
    idx, val, _, n_out, _ = oracle.extract(x, thr)
    tally = pg.write(pool, np.ascontiguousarray(x[0].transpose(1, 0, 2)), np.array([[2, 0, 1]]), [0, T], [0])
    assert tally["n_outliers"] == n_out > 0 and tally["overflow"] == 0
    y, _ = oracle.decode(words, radius, cb.reshape(-1), S, 1, H, T, 128, out_idx=idx, out_val=val, out_dtype=1)
    got, ok = pg.dense(pool, [2, 0, 1], T)
    clear = (best - second > 1e-5 * best) | (best <= 0)
    same = (got == y.reshape(H, T, 128)).reshape(-1, 4).all(-1)
    assert ok.all() and clear.mean() > 0.999 and same[clear.reshape(-1)].all()
