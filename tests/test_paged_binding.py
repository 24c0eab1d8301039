"""The binding of the paged operators refuses what it would otherwise pass on
wrongly: tensors that are missing where others need them, and sizes beyond
the C ABI's 32 bits, which ctypes cuts off without a word (no GPU needed)."""
import pytest
import torch

from test_paged_abi import GOOD, hq, pages  # noqa: F401  (a fixture)


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def record(hq, **change):
    import ctypes
    p = pages(hq, **change)
    p._keep, p._ref = (ints(1),), ctypes.byref(p)
    return p


def test_tensors_that_are_missing(hq):                                   # noqa: F811
    k, v = record(hq), record(hq)
    x = torch.zeros(3, 2, 128)
    with pytest.raises(ValueError, match="xv"):
        hq.hqmq_paged_write(x, None, k, v, ints(1, 2), ints(2), ints(1))
    with pytest.raises(ValueError, match="cu_tokens"):
        hq.hqmq_paged_write(x, None, k, None, ints(1, 2), None, ints(1))
    with pytest.raises(ValueError, match="block_table"):
        hq.hqmq_paged_write(x, None, k, None, None, ints(2), ints(1))
    q, o = torch.zeros(1, 4, 128, dtype=torch.bfloat16), torch.zeros(1, 4, 128)
    with pytest.raises(ValueError, match="seq_len"):
        hq.hqmq_attention_paged(q, k, v, ints(1, 2), None, o, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="seq_len"):
        hq.hqmq_paged_read(k, ints(1, 2), None, torch.zeros(1, 2, 8, 128))
    y = torch.zeros(1, 2, 4, 128)
    with pytest.raises(ValueError, match="pos"):
        hq.hqmq_qk_norm_rope(y, None, y, None, None, torch.ones(64, dtype=torch.float64))


def test_sizes_beyond_32_bits(hq):                                       # noqa: F811
    assert hq.hqmq_attention_paged_workspace_size(1, 4, 2, 32, 16) > 0
    for size in ((1, 4, 2, (1 << 32) + 32, 16), (1, 4, 2, 32, (1 << 32) + 16), ((1 << 32) + 1, 4, 2, 32, 16),
                 (1, (1 << 32) + 4, 2, 32, 16), (1, 4, (1 << 32) + 2, 32, 16)):
        assert hq.hqmq_attention_paged_workspace_size(*size) == 0, size
    k = record(hq, page_size=256)
    with pytest.raises(ValueError):
        hq.alloc_attention_paged_ws(1, 4, k, (1 << 24) + 1, device="cpu")
    q, o = torch.zeros(1, 4, 128, dtype=torch.bfloat16), torch.zeros(1, 4, 128)
    with pytest.raises(ValueError, match="prefix_len"):
        hq.hqmq_attention_paged(q, k, k, None, None, o, torch.zeros(1 << 20, dtype=torch.uint8),
                                prefix_table=ints((1 << 24) + 1), prefix_len=(1 << 32) + 16)
    far = torch.zeros(1, 2, 128).expand((1 << 32) + 3, 2, 128)
    with pytest.raises(ValueError, match="new tokens"):
        hq.hqmq_paged_write(far, None, k, None, ints(1, 2), ints(2), ints(1))


def test_stream_handles_without_torchs_own_shortcut(hq, monkeypatch):    # noqa: F811
    """The handle of torch's current stream, also where its private shortcut does not exist."""
    class Stream:
        cuda_stream = 0x1234
    asked = []
    monkeypatch.setattr(hq, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: asked.append(dev) or Stream())
    assert hq._on(None, 5) == 0x1234 and asked == [5]
    monkeypatch.setattr(hq, "_raw_stream", lambda dev: 0x99 + dev)
    assert hq._on(None, 1) == 0x9A
