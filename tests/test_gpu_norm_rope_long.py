"""hqmq_qk_norm_rope where a CTA walks over several tokens: the call gives a CTA
the span of 1 to 16 tokens that fills its rounds best, one for few tokens.
Bounds and the formula as in tests/test_gpu_norm_rope.py."""
import pytest
import torch

from test_gpu_norm_rope import check
from kv_cache_quantization_hqmq_b200 import hqmq

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

BF, F32 = torch.bfloat16, torch.float32


def span_of(tokens, heads, D, R):
    """Tokens of a CTA, by the rule of csrc/norm_rope.cu."""
    lpv = 1
    while lpv * 16 < D:
        lpv *= 2
    most = (128 if tokens < 148 else 512) // lpv
    shares = -(-heads // most)
    threads = -(-(-(-heads // shares)) * lpv // 32) * 32
    slots, best = 148 * (1024 // threads), None
    for n in range(1, 17):
        if n * (R // 2) <= 1024:
            cost = -(-(-(-tokens // n) * shares) // slots) * (n + 2)
            if best is None or cost < best[0]:
                best = (cost, n)
    return best[1]


@pytest.mark.parametrize("B,T,Hq,Hk,D,R,dt,inter,wdt", [
    (3, 333, 28, 4, 80, 32, F32, True, F32), (5, 701, 32, 8, 128, 128, BF, False, F32), (7, 299, 8, 8, 256, 256, BF, True, BF),
    (2, 1499, 24, 8, 96, 96, F32, False, F32), (13, 401, 16, 1, 64, 32, BF, False, BF), (2500, 1, 32, 8, 128, 64, BF, False, BF),
    (2, 1111, 12, 2, 512, 512, F32, False, None), (1, 3001, 40, 8, 48, 0, BF, False, BF)])
def test_spans_of_several_tokens(B, T, Hq, Hk, D, R, dt, inter, wdt):
    """Token counts that no span divides, spans that end inside a batch row, strides that differ."""
    span = span_of(B * T, Hq + Hk, D, R)
    assert span > 1 and (B * T) % span
    g = torch.Generator().manual_seed(B)
    qkv = torch.randn(B, T, Hq + 2 * Hk, D, generator=g).to(dt).cuda()
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    w = [None if wdt is None else (1 + 0.2 * torch.randn(D, generator=g)).to(wdt).cuda() for _ in range(2)]
    pos = torch.randint(0, 1 << 20, (B, T), generator=g).int().cuda()
    inv = hqmq.rope_inv_freq(R, 500000.0) if R else None
    qo = torch.full((T, B, Hq, D), float("nan"), dtype=dt, device="cuda").transpose(0, 1)
    ko = torch.full((B, Hk, T, D), float("nan"), dtype=dt, device="cuda").permute(0, 2, 1, 3)
    hqmq.hqmq_qk_norm_rope(q, k, qo, ko, pos if R else None, inv, w[0], w[1], eps=1e-5, interleaved=inter)
    check(qo, q, w[0], pos, inv, 1e-5, inter)
    check(ko, k, w[1], pos, inv, 1e-5, inter)
    # in place, the rest of the projection untouched: the same bits
    rest = qkv[:, :, Hq + Hk:].clone()
    hqmq.hqmq_qk_norm_rope(q, k, q, k, pos if R else None, inv, w[0], w[1], eps=1e-5, interleaved=inter)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, :, Hq + Hk:], rest)
