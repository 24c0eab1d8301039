"""The serving operators around the paged HQMQ cache, as cases that can be timed.

Four operators, in the order in which a decode step uses them:

* ``norm_rope``  RMS norm of every query and key head vector and the position
  rotation, in one pass;
* ``write``      quantising new K and V tokens straight into the pages of a
  paged cache (24 S codewords, fp16 radius, flagged outliers in fp16);
* ``read``       the dense K or V of the pages' tokens;
* ``attention``  decode-phase attention read from the pages, for a batch whose
  sequences share a prefix that is processed once for all of them.

With ``own`` false everything is computed by elementary torch operations; with
``own`` true the same inputs go through the package's entry points.

Pages: words int32 [pages, H, P, b], radius fp16 [pages, H, P, 32], flags int32
[pages, H, P] (bit c: chunk c of the token is kept in fp16), values fp16
[pages, H, cap, 4] (the flagged chunks of a page and head in token and chunk
order).  A token of a head is 128 elements, 32 chunks of 4; b bits per index,
least significant bit first.
"""
import math

import torch

own = False

D = 128
CHUNKS = 32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the new token of one sequence: 64 query and 8 KV heads, a far position
        dict(name="rope_step_1", op="norm_rope", B=1, T=1, Hq=64, Hk=8, D=128, R=128,
             dtype="bf16", norm=True, interleaved=False, start=131000),
        # a prefill chunk: 8192 tokens of 32 query and 8 KV heads
        dict(name="rope_prefill_8192", op="norm_rope", B=1, T=8192, Hq=32, Hk=8, D=128, R=128,
             dtype="bf16", norm=True, interleaved=False, start=0),
        # 3 sequences of 333 tokens, 28 query and 4 KV heads of 80, 32 dimensions rotated in
        # neighbouring pairs, fp32
        dict(name="rope_partial_f32", op="norm_rope", B=3, T=333, Hq=28, Hk=4, D=80, R=32,
             dtype="f32", norm=True, interleaved=True, start=7001),
        # a decode step of 64 sequences, one token each
        dict(name="write_step_64", op="write", B=64, new=1, old=700, H=8, S=32, P=64, cap=128,
             dtype="bf16", outliers=True),
        # a prefill chunk of 4096 tokens behind 1000 that are in the cache
        dict(name="write_prefill_4096", op="write", B=1, new=4096, old=1000, H=8, S=32, P=64,
             cap=128, dtype="bf16", outliers=True),
        # 7 sequences with up to 301 new tokens, small pages, fp32, no outliers
        dict(name="write_ragged_f32", op="write", B=7, new=301, old=77, H=4, S=8, P=16, cap=0,
             dtype="f32", outliers=False),
        # 5 sequences of up to 203 tokens, small pages, fp32 out
        dict(name="read_ragged_f32", op="read", B=5, T=203, H=4, S=8, P=16, cap=32, dtype="f32",
             outliers=True),
        # one layer's K of 32768 tokens
        dict(name="read_32768", op="read", B=1, T=32768, H=8, S=32, P=64, cap=128, dtype="bf16",
             outliers=True),
        # two short sequences without a prefix
        dict(name="attn_short", op="attention", B=2, T=190, prefix=0, Hk=4, G=7, S=8, P=16, cap=32,
             dtype="f32", outliers=True),
        # 16 sequences behind a system prompt of 8191 tokens
        dict(name="attn_prefix_8k", op="attention", B=16, T=500, prefix=8191, Hk=8, G=8, S=32,
             P=64, cap=128, dtype="bf16", outliers=True),
        # every head its own KV head, 8 sequences, small pages
        dict(name="attn_mha", op="attention", B=8, T=1111, prefix=4096, Hk=32, G=1, S=8, P=16,
             cap=32, dtype="f32", outliers=True),
        # 32 sequences over one document of 131072 tokens
        dict(name="attn_prefix_128k", op="attention", B=32, T=1000, prefix=131072, Hk=8, G=8, S=32,
             P=64, cap=128, dtype="bf16", outliers=True),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "write", "read", "attention", "attention", "write"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm_rope":
        d = rng.choice([64, 80, 96, 128, 128, 256])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 4, 7, 8])
        batch = _span(rng, 1, 16)
        room = 8192 * 40 * 128 // (batch * (hq + hk) * d) // (2 if dtype == "f32" else 1)
        return dict(op=op, B=batch, T=_span(rng, 1, max(1, min(room, 9000))), Hq=hq, Hk=hk, D=d,
                    R=rng.choice([d, d, d // 2, 32]), dtype=dtype, norm=rng.random() < 0.7,
                    interleaved=rng.random() < 0.4, start=_span(rng, 1, 1000000))
    c = dict(op=op, S=rng.choice([8, 32, 32, _span(rng, 1, 48)]), P=rng.choice([16, 32, 64, 128]),
             dtype=dtype, outliers=rng.random() < 0.75)
    c["cap"] = 2 * c["P"] if c["outliers"] else 0
    if op == "write":
        batch, heads = _span(rng, 1, 64), rng.choice([1, 4, 8, 32])
        c |= dict(B=batch, H=heads, old=_span(rng, 1, 900),
                  new=_span(rng, 1, max(1, 4096 * 8 * 32 // (batch * heads * c["S"]) // 2)))
        c["new"] = min(c["new"], 4096 * 8 // (2 * batch * heads) + 1)
    elif op == "read":
        batch, heads = _span(rng, 1, 32), rng.choice([1, 4, 8, 32])
        c |= dict(B=batch, H=heads, T=_span(rng, 1, max(1, 32768 * 8 // (2 * batch * heads))))
    else:
        batch, heads = _span(rng, 1, 48), rng.choice([1, 4, 8, 32])
        g = rng.choice([1, 4, 7, 8])
        c |= dict(B=batch, Hk=heads, G=g, T=_span(rng, 1, max(1, 200000 // (batch * heads))),
                  prefix=rng.choice([0, 1, 1, 1]) * _span(rng, 1, min(131072, 20000000 // (batch * heads * g))))
    return c


def _b(S):
    return max(5, (24 * S - 1).bit_length())


def _lens(n, most):
    """n sequence lengths up to most, the first of them most: the same for a case whatever the seed."""
    return [most] + [max(1, int(most * ((0.6180339887 * i) % 1.0))) for i in range(1, n)]


def work(case):
    c = case
    if c["op"] == "norm_rope":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["B"] * c["T"] * (c["Hq"] + c["Hk"])
        return {"bytes": 2 * n * c["D"] * e + 4 * c["B"] * c["T"], "flops": n * (4 * c["D"] + 3 * c["R"])}
    code = CHUNKS * 2 + 4 * _b(c["S"]) + ((4 + 8 * 0.85) if c["outliers"] else 0)  # bytes of a token of a head
    if c["op"] == "write":
        e = 2 if c["dtype"] == "bf16" else 4
        n = 2 * sum(_lens(c["B"], c["new"])) * c["H"]
        return {"bytes": int(n * (D * e + code)), "flops": n * CHUNKS * (8 + 12 * c["S"])}
    if c["op"] == "read":
        e = 2 if c["dtype"] == "bf16" else 4
        n = sum(_lens(c["B"], c["T"])) * c["H"]
        return {"bytes": int(n * (D * e + code)), "flops": n * D}
    own_tokens = sum(_lens(c["B"], c["T"]))
    e = 2 if c["dtype"] == "bf16" else 4
    n = 2 * (own_tokens + c["prefix"]) * c["Hk"]
    rows = c["Hk"] * c["G"]
    return {"bytes": int(n * code + c["B"] * rows * D * (2 + e)),
            "flops": 4 * D * rows * (own_tokens + c["prefix"] * c["B"])}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pack(idx, b):
    """[..., 32] indices to [..., b] int32 words, least significant bit first."""
    p = torch.arange(CHUNKS, device=idx.device) * b
    at, sh = p // 32, p % 32
    w = torch.zeros(*idx.shape[:-1], b + 1, dtype=torch.int64, device=idx.device)
    v = idx.long() << sh
    w.index_add_(-1, at, v & 0xFFFFFFFF)
    w.index_add_(-1, at + 1, v >> 32)
    w = w[..., :b]
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int()


def _codebook(g, heads, S):
    q = torch.randn(heads, S, 4, generator=g, device="cuda", dtype=torch.float64)
    return (q / q.norm(dim=-1, keepdim=True)).float()


def _coded_pages(g, n_pages, heads, c):
    """Pages as a cache of normal values with one strong channel of each head fills them."""
    P, S, cap = c["P"], c["S"], c["cap"]
    idx = torch.randint(0, 24 * S, (n_pages, heads, P, CHUNKS), generator=g, device="cuda")
    x = torch.randn(n_pages, heads, P, CHUNKS, 4, generator=g, device="cuda")
    radius = x.square().sum(-1).sqrt().half()
    pages = dict(codebook=_codebook(g, heads, S), flags=None, values=None)
    if c["outliers"]:
        strong = torch.randint(0, CHUNKS, (heads,), generator=g, device="cuda")
        mask = torch.arange(CHUNKS, device="cuda") == strong[:, None, None]
        mask = mask & (torch.rand(n_pages, heads, P, 1, generator=g, device="cuda") < 0.85)
        rank = mask.flatten(2).long().cumsum(-1) - 1
        mask &= (rank < cap).view_as(mask)
        values = torch.randn(n_pages, heads, cap, 4, generator=g, device="cuda")
        values[..., 1] *= 30
        pages["flags"] = (mask.long() << torch.arange(CHUNKS, device="cuda")).sum(-1)
        pages["flags"] = torch.where(pages["flags"] >= 1 << 31, pages["flags"] - (1 << 32), pages["flags"]).int()
        pages["values"] = values.half()
        idx = idx.masked_fill(mask, 0)
        radius = radius.masked_fill(mask, 0)
    pages["words"] = _pack(idx, _b(S))
    pages["radius"] = radius
    return pages


def _tables(g, lens, P, spare):
    """Block table [B, most] of shuffled pages for these lengths, -1 where there is none, and the number of pages."""
    need = [(n + P - 1) // P for n in lens]
    perm = torch.randperm(sum(need) + spare, generator=g, device="cuda").int()
    have = torch.tensor(need, device="cuda")
    col = torch.arange(max(1, max(need)), device="cuda")
    first = have.cumsum(0) - have
    at = first[:, None] + col
    table = torch.where(col < have[:, None], perm[at.clamp(max=perm.numel() - 1)], -1)
    return table.int().contiguous(), perm


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=dict(case))
    if case["op"] == "norm_rope":
        B, T, Hq, Hk, d = (case[k] for k in ("B", "T", "Hq", "Hk", "D"))
        dt = DTYPES[case["dtype"]]
        # q and k are views of the projection's output, k leaves in the codec's [B, H, T, D] layout
        qkv = torch.randn(B, T, Hq + 2 * Hk, d, generator=g, device="cuda").to(dt)
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        s["q_out"] = torch.empty(B, T, Hq, d, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(B, Hk, T, d, dtype=dt, device="cuda").permute(0, 2, 1, 3)
        s["pos"] = (case["start"] + torch.arange(T, device="cuda") +
                    37 * torch.arange(B, device="cuda")[:, None]).int()
        s["inv_freq"] = 500000.0 ** -(torch.arange(0, case["R"], 2, device="cuda").double() / case["R"])
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
            s["kw"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        return s
    heads = case.get("H") or case["Hk"]
    B, P = case["B"], case["P"]
    if case["op"] == "write":
        new = _lens(B, case["new"])
        old = _lens(B, case["old"])
        s["table"], perm = _tables(g, [a + n for a, n in zip(old, new)], P, 3)
        s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).int()
        s["pos0"] = torch.tensor(old, device="cuda").int()
        s["n"] = sum(new)
        s["x"], s["pages"] = [], []
        for _ in range(2):
            x = torch.randn(s["n"], heads, CHUNKS, 4, generator=g, device="cuda")
            pages = _coded_pages(g, perm.numel(), heads, case)
            pages["thr"] = None
            if case["outliers"]:
                strong = torch.randint(0, CHUNKS, (heads,), generator=g, device="cuda")
                x[..., 1] *= torch.where(torch.arange(CHUNKS, device="cuda") == strong[:, None], 30.0, 1.0)
                pages["thr"] = 5.4 + 0.2 * torch.rand(heads, generator=g, device="cuda")
            s["x"].append(x.flatten(2).to(DTYPES[case["dtype"]]))
            s["pages"].append(pages)
    elif case["op"] == "read":
        lens = _lens(B, case["T"])
        s["table"], perm = _tables(g, lens, P, 3)
        s["lens"] = torch.tensor(lens, device="cuda").int()
        s["pages"] = [_coded_pages(g, perm.numel(), heads, case)]
        s["y"] = torch.zeros(B, heads, case["T"], D, dtype=DTYPES[case["dtype"]], device="cuda")
    else:
        lens = _lens(B, case["T"])
        n_prefix = (case["prefix"] + P - 1) // P
        s["table"], perm = _tables(g, lens, P, n_prefix + 3)
        s["prefix_table"] = perm[perm.numel() - n_prefix:].contiguous()
        s["lens"] = torch.tensor(lens, device="cuda").int()
        s["pages"] = [_coded_pages(g, perm.numel(), heads, case) for _ in range(2)]
        s["q"] = torch.randn(B, heads * case["G"], D, generator=g, device="cuda").bfloat16()
        s["o"] = torch.empty(B, heads * case["G"], D, dtype=DTYPES[case["dtype"]], device="cuda")
    if own:
        # what a serving program keeps: the page records, the search tables of its codebooks, the workspace
        from kv_cache_quantization_hqmq_b200 import hqmq
        s["handles"] = []
        for p in s["pages"]:
            table = None
            if case["op"] == "write" and hqmq.hqmq_search_table_bytes(case["S"]):
                table = torch.empty(heads * hqmq.hqmq_search_table_bytes(case["S"]), dtype=torch.uint8, device="cuda")
                hqmq.hqmq_make_search_table(p["codebook"], case["S"], heads, table)
            s["handles"].append(hqmq.kv_pages(p["words"], p["radius"], p["codebook"], flags=p["flags"],
                                              out_val=p["values"], thr=p.get("thr"), table=table))
        if case["op"] == "attention":
            s["ws"] = hqmq.alloc_attention_paged_ws(B, heads * case["G"], s["handles"][0],
                                                    s["table"].shape[1], case["prefix"])
    return s


# ------------------------------------------------------- the operators, plain
def run(state):
    if own:
        return _run_own(state)
    return {"norm_rope": _norm_rope, "write": _write, "read": _read, "attention": _attention}[state["case"]["op"]](state)


def _run_own(s):
    from kv_cache_quantization_hqmq_b200 import hqmq
    c = s["case"]
    if c["op"] == "norm_rope":
        hqmq.hqmq_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["pos"], s["inv_freq"], s["qw"], s["kw"],
                               eps=1e-6, interleaved=c["interleaved"])
        return s["q_out"], s["k_out"]
    if c["op"] == "write":
        hqmq.hqmq_paged_write(s["x"][0], s["x"][1], s["handles"][0], s["handles"][1], s["table"], s["cu"], s["pos0"])
        return _pool(s)
    if c["op"] == "read":
        return hqmq.hqmq_paged_read(s["handles"][0], s["table"], s["lens"], s["y"])
    return hqmq.hqmq_attention_paged(s["q"], s["handles"][0], s["handles"][1], s["table"], s["lens"], s["o"], s["ws"],
                                     prefix_table=s["prefix_table"], prefix_len=c["prefix"])


def _pool(s):
    """The updated pages, whole."""
    return {name + str(i): p[name] for i, p in enumerate(s["pages"])
            for name in ("words", "radius", "flags", "values") if p[name] is not None}


def _norm_rope(s):
    c = s["case"]
    R = c["R"]
    angle = s["pos"].double()[..., None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        a, z = (x[..., 0:R:2], x[..., 1:R:2]) if c["interleaved"] else (x[..., :R // 2], x[..., R // 2:R])
        a, z = a * cos - z * sin, z * cos + a * sin
        turned = torch.stack((a, z), -1).flatten(-2) if c["interleaved"] else torch.cat((a, z), -1)
        return torch.cat((turned, x[..., R:]), -1)

    s["q_out"].copy_(one(s["q"], s["qw"]))
    s["k_out"].copy_(one(s["k"], s["kw"]))
    return s["q_out"], s["k_out"]


def _hurwitz(device, dtype):
    """The 24 unit Hurwitz quaternions: +-1, +-i, +-j, +-k, then the half units by the bits of their signs."""
    eye = torch.eye(4, device=device, dtype=dtype)
    axes = torch.stack((eye, -eye), 1).reshape(8, 4)
    m = torch.arange(16, device=device)[:, None] >> torch.arange(4, device=device)
    return torch.cat((axes, 0.5 - (m & 1).to(dtype)))


def _codewords(cb):
    """q_p q_s of a codebook [H, S, 4], [H, 24 S, 4], the sums of the product's terms from left to right."""
    a = _hurwitz(cb.device, cb.dtype).unsqueeze(-2).unbind(-1)
    w, i, j, k = cb.unsqueeze(-3).unbind(-1)
    a0, a1, a2, a3 = (t for t in a)
    c = torch.stack((a0 * w - a1 * i - a2 * j - a3 * k, a0 * i + a1 * w + a2 * k - a3 * j,
                     a0 * j - a1 * k + a2 * w + a3 * i, a0 * k + a1 * j - a2 * i + a3 * w), -1)
    return c.transpose(-2, -3).flatten(-3, -2)


def _write(s):
    c = s["case"]
    P = c["P"]
    tok = torch.arange(s["n"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), tok, right=True)
    at = s["pos0"].long()[seq] + tok - s["cu"].long()[seq]
    page, row = s["table"].long()[seq, at // P], at % P
    for x, p in zip(s["x"], s["pages"]):
        _write_one(x.double().unflatten(-1, (CHUNKS, 4)), p, page, row, c)
    return _pool(s)


def _write_one(x, p, page, row, c):
    P, cap = c["P"], c["cap"]
    # the norm's steps round to 32 bits one by one: they decide what is an outlier
    r = (x[..., 0] * x[..., 0]).float()
    for i in range(1, 4):
        r = (x[..., i] * x[..., i] + r.double()).float()
    r = r.double().sqrt().float()
    bit = torch.arange(CHUNKS, device="cuda")
    if p["flags"] is not None:
        over = r > p["thr"][:, None]
        kept = ((p["flags"].long()[..., None] >> bit) & 1).sum(-1)  # flagged chunks of each token in the pool
        kept[page, :, row] = over.sum(-1)
        start = (kept.cumsum(-1) - kept)[page, :, row]
        slot = start[..., None] + over.long().cumsum(-1) - 1
        over &= slot < cap
        f = (over.long() << bit).sum(-1)
        p["flags"][page, :, row] = torch.where(f >= 1 << 31, f - (1 << 32), f).int()
        n, h, k = over.nonzero(as_tuple=True)
        p["values"][page[n], h, slot[n, h, k]] = x[n, h, k].clamp(-65504, 65504).half()
        x = x.masked_fill(over[..., None], 0)
        r = r.masked_fill(over, 0)
    # near ties are decided in 64 bits
    words = _codewords(p["codebook"].double())
    score = torch.bmm(x.transpose(0, 1).flatten(1, 2), words.transpose(1, 2))
    idx = score.argmax(-1).unflatten(1, (x.shape[0], CHUNKS)).transpose(0, 1)
    p["words"][page, :, row] = _pack(idx.masked_fill(r == 0, 0), _b(c["S"]))
    p["radius"][page, :, row] = r.clamp(max=65504).half()


def _dense(p, page, row, c):
    """The tokens (page, row) of a pool in 32 bits, [..., H, 128], as the codes say."""
    b = _b(c["S"])
    bits = torch.arange(CHUNKS, device="cuda") * b
    w = p["words"][page, :, row].long() & 0xFFFFFFFF
    lo, hi = w[..., bits // 32], w[..., (bits // 32 + 1).clamp(max=b - 1)]
    idx = ((lo | (hi << 32)) >> (bits % 32)) & ((1 << b) - 1)
    head = torch.arange(w.shape[-2], device="cuda")[:, None]
    y = p["radius"][page, :, row].float()[..., None] * _codewords(p["codebook"])[head, idx]
    if p["flags"] is not None:
        f = (p["flags"].long()[..., None] >> torch.arange(CHUNKS, device="cuda")) & 1
        kept = f.sum(-1)
        f, start = f[page, :, row], (kept.cumsum(-1) - kept)[page, :, row]
        slot = (start[..., None] + f.cumsum(-1) - 1).clamp(0, c["cap"] - 1)
        y = torch.where(f[..., None] == 1, p["values"][page[..., None, None], head, slot].float(), y)
    return y.flatten(-2)


def _own_tokens(s, T):
    """Page and row of every token of the batch's block table, and which of them there are."""
    P = s["case"]["P"]
    t = torch.arange(T, device="cuda")
    there = t < s["lens"][:, None]
    page = s["table"].long()[:, t // P].clamp(min=0)
    return page, (t % P).expand_as(page), there


def _read(s):
    page, row, there = _own_tokens(s, s["case"]["T"])
    y = _dense(s["pages"][0], page, row, s["case"]).transpose(1, 2)
    s["y"].copy_(torch.where(there[:, None, :, None], y, s["y"].float()))
    return s["y"]


def _attention(s):
    c = s["case"]
    Hk, G = c["Hk"], c["G"]
    page, row, there = _own_tokens(s, c["T"])
    t = torch.arange(c["prefix"], device="cuda")
    q = s["q"].float().view(c["B"], Hk, G, D)
    # the cache's values are what its codes give in bf16
    own_kv = [_dense(p, page, row, c).bfloat16().float().transpose(1, 2) for p in s["pages"]]
    pre_kv = [_dense(p, s["prefix_table"].long()[t // c["P"]], t % c["P"], c).bfloat16().float().transpose(0, 1)
              for p in s["pages"]]
    mine = (q @ own_kv[0].transpose(-1, -2)).masked_fill(~there[:, None, None, :], -math.inf)
    rows = q.transpose(0, 1).flatten(1, 2)
    pre = (rows @ pre_kv[0].transpose(-1, -2)).unflatten(1, (c["B"], G)).transpose(0, 1)
    score = torch.cat((pre, mine), -1) * D ** -0.5
    weight = torch.exp(score - score.amax(-1, keepdim=True))
    total = weight.sum(-1, keepdim=True)
    out = weight[..., c["prefix"]:] @ own_kv[1]
    out += (weight[..., :c["prefix"]].transpose(0, 1).flatten(1, 2) @ pre_kv[1]).unflatten(1, (c["B"], G)).transpose(0, 1)
    s["o"].copy_((out / total).flatten(1, 2))
    return s["o"]


# ---------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "write": _exact_write, "read": _exact_read,
            "attention": _exact_attention}[case["op"]](s, case)


def _exact_norm_rope(s, c):
    phase = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                        s["pos"].double()[:, :, None, None] * s["inv_freq"])
    R = c["R"]
    outs = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.double()
        if w is not None:
            x = x / ((x * x).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w.double()
        pairs = x[..., :R].unflatten(-1, (R // 2, 2) if c["interleaved"] else (2, R // 2))
        if not c["interleaved"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
        if not c["interleaved"]:
            z = z.transpose(-1, -2)
        outs.append(torch.cat((z.flatten(-2), x[..., R:]), -1))
    return tuple(outs)


def _token_places(case, s, lens, first):
    """Sequence by sequence, where its tokens lie: (sequence, page, row) of each."""
    places = []
    for i, n in enumerate(lens):
        t = torch.arange(n, device="cuda") + first[i]
        places.append(torch.stack((torch.full_like(t, i), s["table"][i].long()[t // case["P"]], t % case["P"])))
    return torch.cat(places, 1)


def _exact_write(s, c):
    new, old = _lens(c["B"], c["new"]), _lens(c["B"], c["old"])
    _, page, row = _token_places(c, s, new, old)
    out = {}
    for i, (x, p) in enumerate(zip(s["x"], s["pages"])):
        x = x.double().view(s["n"], c["H"], CHUNKS, 4)
        r = (x * x).sum(-1).sqrt()
        big = torch.zeros_like(r, dtype=torch.bool)
        words, radius = p["words"].clone(), p["radius"].double()
        if p["flags"] is not None:
            big = r.float() > p["thr"].view(1, -1, 1)
            powers = 2 ** torch.arange(CHUNKS, device="cuda")
            flags, values = p["flags"].long() & 0xFFFFFFFF, p["values"].double()
            # one page row after the other: how many chunks of the page are taken before it
            before = torch.zeros(flags.shape[:2], dtype=torch.long, device="cuda")
            owner = torch.full(flags.shape[::2], -1, dtype=torch.long, device="cuda")
            owner[page, row] = torch.arange(s["n"], device="cuda")
            for k in range(c["P"]):
                o = owner[:, k]
                fresh = (o >= 0).nonzero().flatten()
                if fresh.numel():
                    m = big[o[fresh]]
                    place = before[fresh][..., None] + m.long().cumsum(-1) - m.long()
                    m &= place < c["cap"]
                    big[o[fresh]] = m
                    flags[fresh, :, k] = (m.long() * powers).sum(-1)
                    a, h, ch = m.nonzero(as_tuple=True)
                    values[fresh[a], h, place[a, h, ch]] = x[o[fresh][a], h, ch].clamp(-65504, 65504)
                before += torch.stack([(flags[..., k] >> q) & 1 for q in range(CHUNKS)]).sum(0)
            out["flags%d" % i] = (flags - ((flags >> 31) << 32)).int()
            out["values%d" % i] = values
        # y = x conj(q_s) scores all 24 primaries at once: 2 max |y_i| against sum |y_i|
        w, a, b, d = p["codebook"].double().unbind(-1)
        x0, x1, x2, x3 = (t[:, :, :, None] for t in x.unbind(-1))
        w, a, b, d = (t[None, :, None, :] for t in (w, a, b, d))
        y = torch.stack((x0 * w + x1 * a + x2 * b + x3 * d, x1 * w - x0 * a - x2 * d + x3 * b,
                         x2 * w - x0 * b + x1 * d - x3 * a, x3 * w - x0 * d - x1 * b + x2 * a), -1)
        axis, half = 2 * y.abs().amax(-1), y.abs().sum(-1)
        sec = torch.maximum(axis, half).argmax(-1)
        pick = sec[..., None, None].expand(*sec.shape, 1, 4)
        y = y.gather(-2, pick).squeeze(-2)
        ax = y.abs().argmax(-1)
        neg = (y < 0).long()
        prim = torch.where(2 * y.abs().amax(-1) >= y.abs().sum(-1), 2 * ax + neg.gather(-1, ax[..., None]).squeeze(-1),
                           8 + neg[..., 0] + 2 * neg[..., 1] + 4 * neg[..., 2] + 8 * neg[..., 3])
        idx = torch.where(big | (r == 0), 0, 24 * sec + prim)
        nb = _b(c["S"])
        stream = ((idx[..., None] >> torch.arange(nb, device="cuda")) & 1).flatten(-2).unflatten(-1, (nb, 32))
        packed = (stream << torch.arange(32, device="cuda")).sum(-1)
        words[page, :, row] = (packed - ((packed >> 31) << 32)).int()
        radius[page, :, row] = torch.where(big, 0.0, r.clamp(max=65504))
        out["words%d" % i], out["radius%d" % i] = words, radius
    order = ("words", "radius", "flags", "values")
    return {n + str(i): out[n + str(i)] for i in range(2) for n in order if n + str(i) in out}


_SIGN = ((1, -1, -1, -1), (1, 1, 1, -1), (1, -1, 1, 1), (1, 1, -1, 1))
_PLACE = ((0, 1, 2, 3), (1, 0, 3, 2), (2, 3, 0, 1), (3, 2, 1, 0))


def _exact_tokens(p, page, row, c, rounded):
    """Tokens (page, row) of a pool in 64 bits, [H, n, 128]; rounded: each step to the bits that the format defines."""
    step = (lambda t: t.float().double()) if rounded else (lambda t: t)
    b = _b(c["S"])
    w = p["words"][page, :, row]
    stream = ((w[..., None] >> torch.arange(32, device="cuda")) & 1).flatten(-2).unflatten(-1, (CHUNKS, b))
    idx = (stream.long() << torch.arange(b, device="cuda")).sum(-1)
    prim = _hurwitz("cuda", torch.float64)[idx % 24]
    sec = p["codebook"].double()[torch.arange(w.shape[1], device="cuda")[None, :, None], idx // 24]
    r = p["radius"][page, :, row].double()
    comps = []
    for sign, place in zip(_SIGN, _PLACE):
        t = 0.0
        for k in range(4):
            t = step(t + sign[k] * prim[..., k] * sec[..., place[k]])
        comps.append(step(r * t))
    y = torch.stack(comps, -1)
    if p["flags"] is not None:
        f = torch.stack([(p["flags"] >> q) & 1 for q in range(CHUNKS)], -1).flatten(-2).long()
        rank = (f.cumsum(-1) - 1).unflatten(-1, (c["P"], CHUNKS))[page, :, row]
        f = f.unflatten(-1, (c["P"], CHUNKS))[page, :, row].bool()
        n, h, k = f.nonzero(as_tuple=True)
        y[n, h, k] = p["values"][page[n], h, rank[n, h, k]].double()
    y = y.flatten(-2).transpose(0, 1)
    return y.bfloat16().double() if rounded else y


def _exact_read(s, c):
    lens = _lens(c["B"], c["T"])
    seq, page, row = _token_places(c, s, lens, [0] * c["B"])
    y = s["y"].double()
    y[seq, :, torch.cat([torch.arange(n, device="cuda") for n in lens])] = \
        _exact_tokens(s["pages"][0], page, row, c, False).transpose(0, 1)
    return y


def _exact_attention(s, c):
    t = torch.arange(c["prefix"], device="cuda")
    pk, pv = (_exact_tokens(p, s["prefix_table"].long()[t // c["P"]], t % c["P"], c, True) for p in s["pages"])
    q = s["q"].double().view(c["B"], c["Hk"], c["G"], D)
    out = []
    for i, n in enumerate(_lens(c["B"], c["T"])):
        t = torch.arange(n, device="cuda")
        page, row = s["table"][i].long()[t // c["P"]], t % c["P"]
        k, v = (torch.cat((a, _exact_tokens(p, page, row, c, True)), 1)
                for a, p in zip((pk, pv), s["pages"]))
        out.append((torch.softmax(q[i] @ k.transpose(-1, -2) / D ** 0.5, -1) @ v).flatten(0, 1))
    return torch.stack(out)
