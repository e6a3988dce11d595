"""Limits of the layer operators' entry points, and overlaps with the small arrays they read (CPU: nothing is launched)."""
import pytest

from test_layer_checks import L, lora_call, resize_call  # noqa: F401  (L is a fixture)
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


def test_lora_refuses_outputs_over_what_it_still_reads(L):
    """The adapters' numbers, ranks, scales and the offsets are read again by every workgroup and by the second product."""
    at = 7 << 20
    small = dict(scales=at, ranks=at + 4096, ids=at + 8192, cu=at + 12288)   # two adapters, two sequences
    size = dict(scales=8, ranks=8, ids=8, cu=12)
    two, one = dict(rows=100), dict(rows=4, ws=None, ws_bytes=0)             # 51200 and 2048 (out), 6400 (ws) bytes
    need = wq.wq_lora_workspace_bytes(100, 2, 256, 16)
    for name, p in small.items():
        for form, n_out in ((two, 100 * 512 * 2), (one, 4 * 512 * 2)):
            for out in (p // 16 * 16, p - n_out + 16):                        # its first and its last bytes
                assert lora_call(L, **small, **form, out=out) == 1, (name, out)
        for ws in (p, p - need // 16 * 16 + 16):
            assert lora_call(L, **small, rows=100, ws=ws, ws_bytes=need) == 1, (name, ws)
        for off in (1, 2):
            assert lora_call(L, **{**small, name: p + off}, rows=100) == 2, (name, off)
        # the array's last bytes over the output's first, and right in front of it (the offsets' alignment is then
        # what is refused; they are looked at last)
        out = 8 << 20
        assert lora_call(L, **{**small, name: out + 4 - size[name]}, rows=100, out=out) == 1, name
        if name != "cu":
            assert lora_call(L, **{**small, name: out - size[name], "cu": at + 12290}, rows=100, out=out) == 2, name
