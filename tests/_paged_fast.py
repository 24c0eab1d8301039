"""The paged cache's plain forms for pools of many tokens: tests/_paged.py's
definitions over whole pools at once, and attention over them in 64 bits on
the GPU, with bounds for every element."""
import numpy as np
import torch

import _paged as P
from kv_cache_quantization_hqmq_b200 import hqmq

U = 2.0 ** -24
LN2 = float(np.log(2.0))


def pack_all(idx, b):
    """[..., 32] indices -> uint32 [..., b], LSB first."""
    bits = np.stack([(idx >> k) & 1 for k in range(b)], -1).astype(np.uint8)
    return np.packbits(bits.reshape(*idx.shape[:-1], 32 * b), axis=-1, bitorder="little").view(np.uint32)


def unpack_all(words, b):
    bits = np.unpackbits(np.ascontiguousarray(words).view(np.uint8), axis=-1, bitorder="little")
    bits = bits.reshape(*words.shape[:-1], 32, b)
    idx = np.zeros(bits.shape[:-1], np.int32)
    for k in range(b):
        idx |= bits[..., k].astype(np.int32) << k
    return idx


def filled_pool(rng, n_pages, H, page, S, cap, spread=1.0):
    """A pool of plausible codes: random directions, chi-distributed radii, some flagged chunks."""
    pool = P.empty_pool(rng, n_pages, H, page, S, cap)
    shape = (n_pages, H, page, 32)
    flag = np.zeros(shape, bool)
    if cap:
        flag = rng.random(shape) < 0.03
        rank = flag.reshape(n_pages, H, -1).cumsum(-1).reshape(shape)
        flag &= rank <= cap
        pool["flags"] = (flag.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
        pool["val"] = P.f16_bits(rng.standard_normal((n_pages, H, cap, 4)).astype(np.float32) * 4)
    r = np.sqrt(rng.chisquare(4, shape)).astype(np.float32) * np.float32(spread)
    pool["radius"] = P.f16_bits(np.where(flag, 0, r))
    pool["words"] = pack_all(np.where(flag, 0, rng.integers(0, 24 * S, shape)), pool["words"].shape[3])
    return pool


def values(pool):
    """fp32 [n_pages, H, P, 128]: every token of the pool, as tests/_paged.py's token gives it."""
    n, H, page, b = pool["words"].shape
    idx = unpack_all(pool["words"], b)
    ok = idx < 24 * pool["S"]
    r = pool["radius"].view(np.float16).astype(np.float32)
    c32 = P.codewords(pool["cb"], True).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        y = r[..., None] * c32[np.arange(H)[None, :, None, None], np.where(ok, idx, 0)]
    y[~ok] = 0
    if pool["flags"] is not None:
        f = ((pool["flags"][..., None] >> np.arange(32, dtype=np.uint32)) & 1).astype(bool)
        rank = f.reshape(n, H, -1).cumsum(-1).reshape(f.shape) - 1
        f &= rank < pool["cap"]
        p, h, _, _ = np.nonzero(f)
        y[f] = pool["val"].view(np.float16)[p, h, rank[f]].astype(np.float32)
    return y.reshape(n, H, page, 128)


def dense(vals, row, n):
    """[H, n, 128] of a sequence's first n tokens (all its pages good) from values()."""
    page = vals.shape[2]
    y = vals[np.asarray(row[:-(-n // page)], np.int64)].transpose(1, 0, 2, 3)
    return y.reshape(vals.shape[1], -1, 128)[:, :n]


def attention(q, k, v, scale, weight):
    """o [G, 128], its bound, lse [G], its bound, in 64 bits on the GPU; q [G, 128], k and v [T, 128] of
    bf16 values; weight: what a softmax weight's rounding is worth.

    A score's exponent x = sl2 s errs by dx = sl2 128 2u max_t sum_d |q_d k_td| (fp32 sums of exact
    products) + 2u |x| (sl2's rounding, x's own), exp2 by 2^-21: common to numerator and sum, so they move
    o by (ln2 dx + 2^-21) sum_t p_t |v_t - o|, at most that times A + |o|, A = sum_t p_t |v_t|.  The weights'
    rounding comes after the sum is taken: weight A.  fp32 accumulation of the products over T / 16 steps,
    rescalings and the join: (T / 16 + 64) 2u A; of the sum, two accumulators a row: (T / 2 + 64) u |o|.
    1.01: products of these."""
    q, k, v = (torch.as_tensor(a).double().cuda() for a in (q, k, v))
    if k.shape[0] == 0:
        g = q.shape[0]
        z = torch.zeros(g, 128, dtype=torch.float64, device="cuda")
        return z, z + 1e-30, torch.full((g,), -np.inf, dtype=torch.float64, device="cuda"), z[:, 0]
    s = scale * (q @ k.T)
    lse = torch.logsumexp(s, -1)
    p = (s - lse[:, None]).exp()
    o, A = p @ v, p @ v.abs()
    sl2 = abs(scale) / LN2
    dx = sl2 * 128 * 2 * U * (q.abs() @ k.abs().T).amax(-1) + 2 * U / LN2 * s.abs().amax(-1)
    d = LN2 * dx + 2.0 ** -21
    T, add = k.shape[0], (k.shape[0] / 2 + 64) * U
    bound = 1.01 * (d[:, None] * (A + o.abs()) + (weight + (T / 16 + 64) * 2 * U) * A + add * o.abs()) + 1e-30
    return o, bound, lse, d + add + 4 * U * (1 + lse.abs())


class Batch:
    """K and V pools, a batch's lengths and shared prefix, and what attention over them has to give."""

    def __init__(self, seed, B, Hk, G, page, S, cap, lens, prefix, scale=None, pools=None, q=None, Sv=None, capv=None):
        from test_gpu_paged_cache import cuda_ints, layout
        rng = np.random.default_rng(seed)
        need = -(-prefix // page)
        self.table, n = layout(rng, lens, page, spare=need + 1)
        self.ptable = np.setdiff1d(np.arange(n), self.table)
        self.ptable = rng.permutation(self.ptable)[:need].astype(np.int32)
        if pools is None:
            self.pools = [filled_pool(rng, n, Hk, page, S, cap),
                          filled_pool(rng, n, Hk, page, S if Sv is None else Sv, cap if capv is None else capv)]
        else:
            self.pools = pools(rng, n, self.table, self.ptable)
        if q is None:
            q = rng.standard_normal((B, Hk * G, 128)).astype(np.float32)
        self.q = torch.from_numpy(q).bfloat16().cuda()
        self.B, self.Hk, self.G, self.lens, self.prefix = B, Hk, G, lens, prefix
        self.scale = 128 ** -0.5 if scale is None else scale
        (self.kp, _), (self.vp, _) = (P.upload(p) for p in self.pools)
        self.t_d, self.len_d, self.pt_d = cuda_ints(self.table, lens, self.ptable)
        self.ws = hqmq.alloc_attention_paged_ws(B, Hk * G, self.kp, self.table.shape[1], prefix)
        self.vals = None

    def call(self, out):
        o = torch.full((self.B, self.Hk * self.G, 128), float("nan"), dtype=out, device="cuda")
        lse = torch.full((self.B, self.Hk * self.G), float("nan"), device="cuda")
        status = hqmq.new_status()
        self.ws.fill_(0xFF)                                           # NaNs
        hqmq.hqmq_attention_paged(self.q, self.kp, self.vp, self.t_d, self.len_d, o, self.ws, prefix_table=self.pt_d,
                                  prefix_len=self.prefix, scale=self.scale, lse=lse, status=status)
        torch.cuda.synchronize()
        assert hqmq.read_status(status)["flags"] == 0
        return o, lse

    def want(self, b, h, weight):
        """attention() of sequence b's queries of KV head h."""
        if self.vals is None:
            self.vals = [P.bf16(values(p)) for p in self.pools]
            self.pre = [torch.from_numpy(np.ascontiguousarray(dense(x, self.ptable, self.prefix))).cuda() for x in self.vals]
        own = [torch.from_numpy(np.ascontiguousarray(dense(x, self.table[b], self.lens[b])[h])).cuda() for x in self.vals]
        k, v = (torch.cat([p[h], o]) for p, o in zip(self.pre, own))
        return attention(self.q[b, h * self.G:(h + 1) * self.G], k, v, self.scale, weight)

    def check(self, o, lse, weight):
        """All rows within their bounds; the worst ratio."""
        half = torch.finfo(o.dtype).eps / 2 if o.dtype == torch.bfloat16 else 0.0
        worst = 0.0
        for b in range(self.B):
            for h in range(self.Hk):
                want, bound, wl, bl = self.want(b, h, weight)
                rows = slice(h * self.G, (h + 1) * self.G)
                got, gl = o[b, rows].double(), lse[b, rows].double()
                ratio = float(((got - want).abs() / (bound * (1 + half) + half * want.abs())).max())
                assert ratio <= 1, (b, h, ratio)
                worst = max(worst, ratio)
                assert bool(((gl == wl) | ((gl - wl).abs() <= bl)).all()), (b, h, gl, wl)
        return worst
