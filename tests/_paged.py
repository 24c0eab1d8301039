"""Plain CPU forms of the paged cache's operators, in 64 bits (numpy), written
from their definitions: one token, head and chunk at a time where order
matters.  A pool is a dict of numpy arrays: words uint32 [pages, H, P, b],
radius uint16 [pages, H, P, 32], flags uint32 [pages, H, P] or None, val
uint16 [pages, H, cap, 4] or None, cb float32 [H, S, 4], thr float32 [H]."""
import numpy as np
import torch

from kv_cache_quantization_hqmq_b200 import hqmq

MUL = ((0, 1, 2, 3), (1, 0, 3, 2), (2, 3, 0, 1), (3, 2, 1, 0))     # (p q)_c = sum_k sign p_k q_place
SGN = ((1, -1, -1, -1), (1, 1, 1, -1), (1, -1, 1, 1), (1, 1, -1, 1))


def two_t():
    e = np.eye(4)
    axes = [s * e[a] for a in range(4) for s in (1.0, -1.0)]
    halves = [[0.5 - ((m >> c) & 1) for c in range(4)] for m in range(16)]
    return np.array(axes + halves)


def codewords(cb, rounded):
    """[H, 24 S, 4] products q_p q_s: fp32 left-to-right sums (rounded) or fp64."""
    t, q = two_t(), cb.astype(np.float64)
    H, S, _ = cb.shape
    out = np.zeros((H, S, 24, 4))
    for c in range(4):
        acc = np.zeros((H, S, 24))
        for k in range(4):
            acc = acc + SGN[c][k] * t[None, None, :, k] * q[:, :, None, MUL[c][k]]
            if rounded:
                acc = acc.astype(np.float32).astype(np.float64)
        out[..., c] = acc
    return out.reshape(H, S * 24, 4)


def chunk_norms(x):
    """fp32 norms of [..., 4], every step rounded as the library rounds it (inputs up to 32 bits:
    a product of two is exact in 64, and so, to 2^-53, is the sum that is rounded)."""
    x = x.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        r = (x[..., 0] ** 2).astype(np.float32)
        for i in range(1, 4):
            r = (x[..., i] ** 2 + r.astype(np.float64)).astype(np.float32)
        return np.sqrt(r)


def f16_bits(v):
    """fp16 bits, round to nearest even, finite values saturating at 65504."""
    v = np.asarray(v, dtype=np.float32)
    with np.errstate(over="ignore"):
        h = v.astype(np.float16)
    big = np.isinf(h) & np.isfinite(v)
    h = np.where(big, np.copysign(np.float16(65504), v).astype(np.float16), h)
    return h.view(np.uint16)


def pack_words(idx, b):
    """32 indices -> b words, LSB first."""
    n = 0
    for k, v in enumerate(idx):
        n |= int(v) << (k * b)
    return [(n >> (32 * w)) & 0xFFFFFFFF for w in range(b)]


def unpack_words(words, b):
    n = 0
    for w, v in enumerate(words):
        n |= int(v) << (32 * w)
    return [(n >> (k * b)) & ((1 << b) - 1) for k in range(32)]


def make_codebook(rng, H, S):
    q = rng.standard_normal((H, S, 4))
    return (q / np.linalg.norm(q, axis=-1, keepdims=True)).astype(np.float32)


def empty_pool(rng, n_pages, H, P, S, cap=0, thr=None):
    """Pages of noise, as a recycled pool holds them (valid indices)."""
    b = hqmq.hqmq_index_bits(S)
    words = rng.integers(0, 1 << 32, (n_pages, H, P, b), dtype=np.uint64).astype(np.uint32)
    pool = dict(words=words, radius=rng.integers(0, 0x7C00, (n_pages, H, P, 32)).astype(np.uint16),
                flags=None, val=None, cb=make_codebook(rng, H, S), thr=None, S=S, P=P, cap=cap)
    if cap:
        pool["flags"] = rng.integers(0, 1 << 32, (n_pages, H, P), dtype=np.uint64).astype(np.uint32)
        pool["val"] = rng.integers(0, 0x7C00, (n_pages, H, cap, 4)).astype(np.uint16)
        pool["thr"] = np.full(H, 5.0 if thr is None else thr, np.float32)
    return pool


def copy_pool(p):
    return {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in p.items()}


def write(pool, x, table, cu, pos0):
    """The write's definition, token by token; x [n, H, 128] float32.  Returns
    (outliers, overflowed, saturated, nonfinite, bad pages)."""
    n_pages, H, P, b = pool["words"].shape
    exact = codewords(pool["cb"], False)
    tally = dict(n_outliers=0, overflow=0, n_saturated=0, n_nonfinite=0, bad=0)
    chunks = x.reshape(x.shape[0], H, 32, 4)
    norms = chunk_norms(chunks)
    for s in range(len(pos0)):
        for i in range(int(cu[s]), int(cu[s + 1])):
            pos = int(pos0[s]) + i - int(cu[s])
            col, row = pos // P, pos % P
            page = int(table[s, col]) if 0 <= pos and col < table.shape[1] else -1
            if pos0[s] < 0 or not 0 <= page < n_pages:
                tally["bad"] += 1
                continue
            for h in range(H):
                write_token(pool, page, h, row, chunks[i, h], norms[i, h], exact[h], tally)
    return tally


def write_token(pool, page, h, row, x, r, exact, tally):
    flag, used = 0, 0
    if pool["flags"] is not None:
        used = sum(int(f).bit_count() for f in pool["flags"][page, h, :row])
    idx, rad = [0] * 32, [0] * 32
    with np.errstate(invalid="ignore", over="ignore"):
        scores = x.astype(np.float64) @ exact.T
    for c in range(32):
        if pool["flags"] is not None and r[c] > pool["thr"][h]:
            tally["n_outliers"] += 1
            if used < pool["cap"]:
                pool["val"][page, h, used] = f16_bits(x[c])
                tally["n_saturated"] += int((np.isfinite(x[c]) & (np.abs(x[c]) >= 65520)).sum())
                flag |= 1 << c
                used += 1
                continue
            tally["overflow"] += 1
        if not np.isfinite(r[c]):
            rad[c] = 0x7E00
            tally["n_nonfinite"] += 1
            continue
        rad[c] = int(f16_bits(r[c]))
        tally["n_saturated"] += int(r[c] >= 65520)
        idx[c] = int(np.argmax(scores[c])) if r[c] > 0 else 0
    pool["words"][page, h, row] = pack_words(idx, pool["words"].shape[3])
    pool["radius"][page, h, row] = rad
    if pool["flags"] is not None:
        pool["flags"][page, h, row] = flag


def token(pool, page, h, row, words32=None):
    """The 128 fp32 values of a stored token (before the rounding to the output type)."""
    n_pages, H, P, b = pool["words"].shape
    c32 = words32 if words32 is not None else codewords(pool["cb"], True)
    idx = np.array(unpack_words(pool["words"][page, h, row], b))
    r = pool["radius"][page, h, row].view(np.float16).astype(np.float32)
    ok = idx < 24 * pool["S"]
    with np.errstate(invalid="ignore", over="ignore"):
        y = r[:, None] * c32[h, np.where(ok, idx, 0)].astype(np.float32)
    y[~ok] = 0
    if pool["flags"] is not None:
        slot = sum(int(f).bit_count() for f in pool["flags"][page, h, :row])
        for c in range(32):
            if (int(pool["flags"][page, h, row]) >> c) & 1:
                if slot < pool["cap"]:
                    y[c] = pool["val"][page, h, slot].view(np.float16).astype(np.float32)
                slot += 1
    return y.reshape(128)


def dense(pool, table_row, n):
    """[H, n, 128] fp32 of a sequence's first n tokens; bad pages give NaN rows and False."""
    n_pages, H, P, _ = pool["words"].shape
    c32 = codewords(pool["cb"], True)
    y, ok = np.zeros((H, n, 128), np.float32), np.zeros(n, bool)
    for t in range(n):
        page = int(table_row[t // P]) if t // P < len(table_row) else -1
        ok[t] = 0 <= page < n_pages
        for h in range(H):
            if ok[t]:
                y[h, t] = token(pool, page, h, t % P, c32)
    return y, ok


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16().float().numpy()


def upload(pool, table=None):
    """(KVPages, its tensors by name) of a pool, on the GPU."""
    t = {}
    for name, dt in (("words", np.int32), ("radius", np.int16), ("flags", np.int32), ("val", np.int16),
                     ("cb", np.float32), ("thr", np.float32)):
        t[name] = None if pool[name] is None else torch.from_numpy(pool[name].view(dt).copy()).cuda()
    return hqmq.kv_pages(t["words"], t["radius"], t["cb"], t["flags"], t["val"], t["thr"], table), t


def search_tables(cb):
    """The heads' search tables on the GPU."""
    d = torch.from_numpy(cb).cuda()
    H, S, _ = cb.shape
    table = torch.empty(H * hqmq.hqmq_search_table_bytes(S), dtype=torch.uint8, device="cuda")
    hqmq.hqmq_make_search_table(d, S, H, table)
    return table


def assert_pools_equal(t, pool):
    torch.cuda.synchronize()
    for name in ("flags", "val", "radius", "words"):
        if pool[name] is not None:
            got = t[name].cpu().numpy().view(pool[name].dtype)
            bad = np.argwhere(got != pool[name])
            assert bad.size == 0, (name, len(bad), bad[:4].tolist())
