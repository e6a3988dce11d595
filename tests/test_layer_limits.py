"""Limits of the layer operators' entry points, and overlaps with the small arrays they read (CPU: nothing is launched)."""
import pytest

from test_layer_checks import L, lora_call, norm_call, resize_call, rotary_call  # noqa: F401  (L is a fixture)
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


def test_rotary_refuses_outputs_over_what_it_still_reads(L):
    """The plan, positions, lengths and offsets are read by every row's threads."""
    rows, ld, at = 4, 1536, 4 << 20                           # rows of 8 (queries) and 2 heads of 128
    size = dict(turns=64 * 8, axis=64 * 4, lens=2 * 4, cu=3 * 4, pos=rows * 4)
    arrays = {name: (8 << 20) + 4096 * i for i, name in enumerate(size)}
    for name in size:
        args = dict(arrays, **({"lens": None, "cu": None} if name == "pos" else {"pos": None}))
        for out, width in (("qo", 8 * 128 * 2), ("ko", 2 * 128 * 2)):
            place = dict(qo=6 << 20, ko=7 << 20)
            place[out] = at
            for row in range(rows):
                first, end = at + row * ld * 2, at + row * ld * 2 + width
                for p in (first + 8 - size[name], first, end - 8):
                    assert rotary_call(L, **{**args, name: p}, **place) == 1, (name, out, row, p - first)
        for off in (1, 2, 3):
            assert rotary_call(L, **{**args, name: arrays[name] + off}, qo=6 << 20, ko=7 << 20) == 2, (name, off)
    # in front of an output, between its rows and behind it: it is then the positions' alignment that is refused
    args = dict(arrays, lens=None, cu=None, pos=arrays["pos"] + 2, qo=at, ko=7 << 20)
    for name in ("turns", "axis"):
        for p in (at - size[name], at + 2048, at + ld * 2 - size[name], at + 3 * ld * 2 + 2048):
            assert rotary_call(L, **{**args, name: p}) == 2, (name, p - at)
    # positions of several axes, 1 MiB apart
    args = dict(arrays, lens=None, cu=None, axes=3, ld_pos=1 << 18, qo=16 << 20, ko=17 << 20)
    for out in (16 << 20, 17 << 20):
        for ax in range(3):
            assert rotary_call(L, **{**args, "pos": out - ax * (1 << 20) + 8}) == 1
    # lengths are not read beside positions, and not looked at then
    assert rotary_call(L, **dict(arrays, lens=4 << 20, cu=None, pos=arrays["pos"] + 2, qo=4 << 20, ko=7 << 20)) == 2


def test_norm_refuses_outputs_over_its_weight(L):
    for y, w, code in ((2 << 20, (2 << 20) + 7 * 2048 + 2048 - 16, 1), (2 << 20, (2 << 20) - 256 + 16, 1),
                       (2 << 20, (2 << 20) - 256 + 8, 1), (2 << 20, (2 << 20) - 256 - 8, 2), (2 << 20, (2 << 20) + 8 * 2048 + 8, 2)):
        assert norm_call(L, y=y, w=w, rows=8) == code, (y, w)
