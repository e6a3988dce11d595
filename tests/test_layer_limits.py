"""Limits of the layer operators' entry points, and overlaps with the small arrays they read (CPU: nothing is launched)."""
import pytest

from test_layer_checks import L, resize_call  # noqa: F401  (L is a fixture)
import weight_only_quantized_w4a16_amd as wq


def test_resize_counts_pages_in_32_bits(L):
    """A thread's next page is up to 2^18 behind its last one, in 32 bits: no more pages than leave room for that."""
    over = dict(lens=2 << 20, want=2 << 20)  # (refused in any case, so that nothing is launched)
    assert resize_call(L, num_pages=1 << 30, free=1 << 40, **over) == 1
    assert resize_call(L, num_pages=(1 << 30) + 1, free=1 << 40, **over) == 2
    assert resize_call(L, num_pages=2 ** 31 - 1, free=1 << 40, **over) == 2
    assert wq.wq_kv_resize_workspace_bytes(2000, 8, (1 << 30) + 1, 0) == 0
    for bad in (0, (1 << 30) + 1, 2 ** 31 - 1):
        with pytest.raises(ValueError, match="num_pages"):
            wq.wq_kv_pages(bad, 16, 2, 4, device="cpu")
