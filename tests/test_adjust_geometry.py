"""What loom_token_launch_config reports of the adjustment of logits (no GPU): by type and by where rows start."""
import pytest

SMS = 152


@pytest.fixture(scope="module")
def loom():
    import __graft_entry__
    __graft_entry__.build()
    import int8_dequant_dot_gb300 as m
    return m


def report(loom, rows, vocab, marks=1, dtype=0, access=2):
    L = loom.loom_token_launch_config(loom.LOOM_OP_ADJUST_LOGITS, [rows, vocab, marks, SMS, dtype, access])
    slice_ = L["units_per_cta"]
    assert L["block"][0] == 512 and L["kernel"] == loom.LOOM_KERNEL_ADJUST
    # the mask's words and one more, in whole 16 bytes; a word a token, and 16 warps' lists of 256 places of 16 bits
    assert L["smem_bytes"] == (slice_ // 32 + 4) // 4 * 16 + (4 * slice_ + 8192 if marks else 0)
    return L["grid"][0], slice_


@pytest.mark.parametrize("marks", [0, 1])
def test_slices_by_type_and_place(loom, marks):
    f32, f16, bf16 = loom.LOOM_F32, loom.LOOM_F16, loom.LOOM_BF16
    assert report(loom, 256, 131072, marks) == (256 * 8, 16384)
    # a thread takes 16 bytes at least: 2048 tokens of f32, 4096 of 16 bits
    assert report(loom, 1, 32768, marks, f32) == (16, 2048)
    for half in (f16, bf16):
        assert report(loom, 1, 32768, marks, half) == (8, 4096)
        assert report(loom, 256, 131072, marks, half) == (256 * 8, 16384)
    # rows that start off 16 bytes reach 3 (or 7) places further
    assert report(loom, 256, 131072, marks, f32, 1) == (256 * 9, 16384)
    assert report(loom, 256, 131069, marks, f32, 1) == (256 * 8, 16384) and report(loom, 256, 131069, marks, bf16, 1) == (256 * 9, 16384)
    assert report(loom, 1, 1, marks, f32, 1) == (1, 2048)
    # logits and y that start at different places: one element at a time, 16 or 4 of a thread
    assert report(loom, 256, 131072, marks, f32, 0) == (256 * 16, 8192) and report(loom, 256, 131072, marks, f16, 0) == (256 * 16, 8192)
    assert report(loom, 1, 32768, marks, f32, 0) == (16, 2048) and report(loom, 1, 32768, marks, bf16, 0) == (16, 2048)


def test_defaults_and_refusals(loom):
    cfg = loom.loom_token_launch_config
    assert cfg(loom.LOOM_OP_ADJUST_LOGITS, [256, 131072, 1, SMS]) == cfg(loom.LOOM_OP_ADJUST_LOGITS, [256, 131072, 1, SMS, loom.LOOM_F32, 2])
    for dtype, access in ((3, 2), (-1, 2), (0, 3), (0, -1), (1 << 40, 2)):
        with pytest.raises(loom.LoomError) as e:
            cfg(loom.LOOM_OP_ADJUST_LOGITS, [1, 100, 1, SMS, dtype, access])
        assert e.value.status == loom.LOOM_ERR_ARG
