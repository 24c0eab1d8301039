"""hqmq_qk_norm_rope against the formula in 64 bits.

Tolerance (u = 2^-24): the sum of D squares has at most D roundings, the mean,
eps, root and quotient 4 more, of which the root halves those before it; the
two products with f and w and the rotation's three steps add 5: a factor
1 + (D / 2 + 10) u on each of the two terms.  cos and sin err by at most
2^-23 (two units in the last place at 1) plus the angle's rounding: its turns
are exact to 2^-52 of themselves, and their doubled fraction, at most 1, is
rounded to 2^-25 and times pi: 2^-23.4.  So |dy| <= ((D / 2 + 10) u + 2^-22)
(|y_u| + |y_v|), and the output's rounding is eps / 2 of the value."""
import numpy as np
import pytest
import torch

from kv_cache_quantization_hqmq_b200 import hqmq

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def plain(x, w, pos, inv_freq, eps, interleaved):
    """(value, |y_u| + |y_v|) in float64, on the CPU."""
    x = x.double().cpu()
    D = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double().cpu()
    y, mag = x.clone(), x.abs()
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    for i in range(R // 2):
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        # whole turns leave in long double: pos * inv_freq itself is rounded to 2^-53 on both sides
        a = pos.cpu().numpy().astype(np.longdouble) * np.longdouble(inv_freq[i].item())
        a = torch.from_numpy((a - 2 * np.pi * np.rint(a / (2 * np.pi))).astype(np.float64))
        c, s = a.cos()[..., None], a.sin()[..., None]
        y[..., u] = x[..., u] * c - x[..., v] * s
        y[..., v] = x[..., v] * c + x[..., u] * s
        mag[..., u] = mag[..., v] = x[..., u].abs() + x[..., v].abs()
    return y, mag


def check(got, x, w, pos, inv_freq, eps, interleaved):
    y, mag = plain(x, w, pos, inv_freq, eps, interleaved)
    tol = ((x.shape[-1] / 2 + 10) * U + 2.0 ** -22) * mag + torch.finfo(got.dtype).eps / 2 * y.abs() * (1 + 1e-3) + 1e-37
    err = (got.double().cpu() - y).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def inputs(B, T, Hq, Hk, D, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(B, T, Hq + 2 * Hk, D, generator=g).to(dt).cuda()
    w = (1 + 0.2 * torch.randn(2, D, generator=g)).to(dt).cuda()
    pos = torch.randint(0, 1 << 20, (B, T), generator=g).int().cuda()
    return qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], w[0], w[1], pos


@pytest.mark.parametrize("B,T,Hq,Hk,D,R,dt,inter", [
    (1, 1, 64, 8, 128, 128, BF, False), (2, 3, 28, 4, 128, 128, BF, True), (1, 257, 8, 2, 128, 64, BF, False),
    (3, 5, 4, 4, 64, 64, F32, False), (1, 7, 3, 1, 80, 32, F32, True), (2, 2, 1, 1, 256, 256, BF, False),
    (1, 2, 2, 1, 512, 512, F32, False), (1, 4, 5, 3, 33, 14, BF, False), (1, 3, 2, 2, 1, 0, F32, False),
    (2, 2, 2, 1, 2, 2, BF, True), (1, 33, 40, 8, 96, 96, F32, True), (2, 9, 16, 8, 128, 2, BF, False),
    (1, 300, 32, 8, 128, 128, F32, False), (4, 75, 7, 1, 64, 32, BF, True)])
@pytest.mark.parametrize("norm", [True, False])
def test_against_the_formula(B, T, Hq, Hk, D, R, dt, inter, norm):
    q, k, qw, kw, pos = inputs(B, T, Hq, Hk, D, dt)
    inv = hqmq.rope_inv_freq(R, 500000.0) if R else None
    qo = torch.full((B, T, Hq, D), float("nan"), dtype=dt, device="cuda")
    ko = torch.full((B, Hk, T, D), float("nan"), dtype=dt, device="cuda").permute(0, 2, 1, 3)
    hqmq.hqmq_qk_norm_rope(q, k, qo, ko, pos if R else None, inv, qw if norm else None, kw if norm else None,
                           eps=1e-5, interleaved=inter)
    for x, o, w in ((q, qo, qw), (k, ko, kw)):
        check(o, x, w if norm else None, pos, inv, 1e-5, inter)


def test_in_place_and_beside_it():
    """In place on views of the projection: v and everything else stay as they were."""
    g = torch.Generator().manual_seed(5)
    buf = torch.randn(2, 9, 14, 136, generator=g).bfloat16().cuda()      # heads of 128 in rows of 136
    before = buf.clone()
    q, k = buf[:, :, :8, 4:132], buf[:, :, 8:11, 4:132]
    pos = torch.arange(18, dtype=torch.int32, device="cuda").view(2, 9)
    inv = hqmq.rope_inv_freq(128)
    w = torch.linspace(0.5, 1.5, 128, device="cuda")                      # fp32 weights of bf16 data
    hqmq.hqmq_qk_norm_rope(q, k, q, k, pos, inv, w, w)
    check(q, before[:, :, :8, 4:132], w, pos, inv, 1e-6, False)
    check(k, before[:, :, 8:11, 4:132], w, pos, inv, 1e-6, False)
    assert torch.equal(buf[:, :, 11:], before[:, :, 11:])
    assert torch.equal(buf[..., :4], before[..., :4]) and torch.equal(buf[..., 132:], before[..., 132:])


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_unaligned_views_and_single_sided_calls(shift):
    """Vectors that start at any element, odd head strides; q alone and k alone."""
    g = torch.Generator().manual_seed(6)
    buf = torch.randn(1, 5, 6, 128 + 13, generator=g).bfloat16().cuda()
    q = buf[..., shift:shift + 128]
    out = torch.zeros(1, 5, 6, 128 + 9, dtype=BF, device="cuda")
    pos = torch.tensor([[0, 1, 131071, 2 ** 31 - 1, -7]], dtype=torch.int32, device="cuda")
    inv = hqmq.rope_inv_freq(128)
    for args in ((q, None, out[..., 3:131], None), (None, q, None, out[..., 3:131])):
        out.fill_(7)
        hqmq.hqmq_qk_norm_rope(*args, pos, inv)
        check(out[..., 3:131], q, None, pos, inv, 1e-6, False)
        assert bool((out[..., :3] == 7).all()) and bool((out[..., 131:] == 7).all())


def test_zero_vectors_huge_values_and_empty_batches():
    x = torch.zeros(1, 3, 2, 128, device="cuda")
    x[0, 1] = 3e18                                   # squares sum to about 1e39: beyond fp32
    x[0, 2] = 1e-25
    y = torch.full_like(x, float("nan"))
    w = torch.ones(128, device="cuda")
    pos = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    hqmq.hqmq_qk_norm_rope(x, None, y, None, pos, hqmq.rope_inv_freq(128), w)
    assert bool((y[0, 0] == 0).all())
    assert bool((y[0, 1] == 0).all())                # x / inf, as fp32 arithmetic has it
    check(y[0, 2][None, None], x[0, 2][None, None], w, pos[:, :1], None, 1e-6, False)
    e = x[:, :0]
    hqmq.hqmq_qk_norm_rope(e, None, e, None, pos[:, :0].contiguous(), hqmq.rope_inv_freq(128), w)


def test_captured_into_a_graph_on_another_stream():
    q, k, qw, kw, pos = inputs(1, 4, 8, 2, 128, BF)
    qo, ko = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    inv = hqmq.rope_inv_freq(128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        hqmq.hqmq_qk_norm_rope(q, k, qo, ko, pos, inv, qw, kw)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        hqmq.hqmq_qk_norm_rope(q, k, qo, ko, pos, inv, qw, kw)
    for seed in (1, 2):
        q2, k2, _, _, pos2 = inputs(1, 4, 8, 2, 128, BF, seed)
        q.copy_(q2), k.copy_(k2), pos.copy_(pos2)
        graph.replay()
        check(qo, q2, qw, pos2, inv, 1e-6, False)
        check(ko, k2, kw, pos2, inv, 1e-6, False)


def test_refusals():
    q, k, qw, kw, pos = inputs(1, 2, 4, 2, 128, BF)
    inv = hqmq.rope_inv_freq(128)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    good = dict(q=q, k=k, q_out=qo, k_out=ko, pos=pos, inv_freq=inv, q_weight=qw, k_weight=kw)
    for change in (dict(q_out=None), dict(q_out=qo[:, :, :2]), dict(k=k.float()), dict(pos=pos.long()),
                   dict(pos=pos[:, :1]), dict(inv_freq=inv.float()), dict(q_weight=qw[:64]),
                   dict(q_weight=qw.float()), dict(q=None), dict(q=q.cpu()), dict(q=q.transpose(2, 3))):
        with pytest.raises((ValueError, TypeError)):
            hqmq.hqmq_qk_norm_rope(**{**good, **change})
    for change in (dict(eps=-1.0), dict(eps=float("nan")), dict(inv_freq=hqmq.rope_inv_freq(130))):
        with pytest.raises(hqmq.HQMQError):
            hqmq.hqmq_qk_norm_rope(**{**good, **change})
