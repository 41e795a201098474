"""loom_token_launch_config: what it reports of shared memory, clusters and first launches.  No GPU."""
import pytest

SMS = 152
SM_BYTES = 227 * 1024


@pytest.fixture(scope="module")
def loom():
    import __graft_entry__
    __graft_entry__.build()
    import int8_dequant_dot_gb300 as m
    return m


def _ring(rows, width, size, L, matrices):
    """Bytes of the read-ahead ring: places for whole rows and the 16-byte blocks around them, as many
    stages (up to eight) as keep 112 KiB of an SM in flight, two at least, none for a single turn."""
    per_sm = 1 if L["block"][0] >= 512 else 512 // L["block"][0]
    slot = (width * size + 30) // 16 * 16 * matrices * L["units_per_cta"]
    turns = -(-rows // (L["grid"][0] * L["units_per_cta"]))
    stages = min(max(2, min(8, 112 * 1024 // (per_sm * slot))), turns)
    if stages < 2 or per_sm * (stages * (slot + 8) + 3 * 1024) > 226 * 1024:
        return 0
    return stages * (slot + 8)


def test_shared_memory_of_the_row_kernels(loom):
    rings = 0
    for op, matrices, narrow, widest in ((loom.LOOM_OP_LAYER_NORM, 1, 512, 32768), (loom.LOOM_OP_QUANTIZE_TOKENS, 1, 512, 32768),
                                         (loom.LOOM_OP_LAYER_NORM_BACKWARD, 2, 256, 8192)):
        for rows in (1, 300, 2000, 100000):
            for width in (64, 256, 260, 512, 516, 2048, 4096, 5000, 8192, 8200, 32768, 40000):
                for dtype, size in ((loom.LOOM_F32, 4), (loom.LOOM_BF16, 2)):
                    L = loom.loom_token_launch_config(op, [rows, width, dtype, 1, SMS])
                    if width > widest:
                        want = 0
                    elif width <= narrow:       # a warp a row: the backward's warps join their columns' sums
                        want = 8 * 2 * width * 4 if matrices == 2 else 0
                    else:
                        want = _ring(rows, width, size, L, matrices)
                        rings += want > 0
                    assert L["smem_bytes"] == want and want <= SM_BYTES, (op, rows, width, dtype)
    assert rings > 50


def test_shared_memory_of_the_few_token_product(loom):
    for t, group in ((1, 1), (2, 2), (3, 4), (4, 4), (5, 8), (8, 8), (24, 8)):
        for n in (1, 5000, 1 << 20):
            L = loom.loom_token_launch_config(loom.LOOM_OP_I8_MATMUL, [t, n, 1024, 1, loom.LOOM_PATH_DIRECT, SMS])
            assert L["smem_bytes"] == L["units_per_cta"] * group * 4 <= 32 * 1024


def test_first_launch_of_the_wide_backward(loom):
    for rows, width in ((3, 8193), (5000, 9000), (100000, 20000)):
        L = loom.loom_token_launch_config(loom.LOOM_OP_LAYER_NORM_BACKWARD, [rows, width, loom.LOOM_F32, 1, SMS])
        assert L["grid"] == (rows, 1, 1) and L["block"] == (1024, 1, 1)


@pytest.mark.parametrize("vocab,few,many", [(1, 1, 1), (2048, 1, 1), (2049, 2, 1), (16384, 8, 1), (16385, 8, 2), (65536, 8, 4), (65537, 8, 8),
                                            (393216, 8, 8)])
def test_clusters_of_sampling(loom, vocab, few, many):
    # 3 rows leave SMs without work: shorter slices then; 1000 do not
    for rows, ranks in ((3, few), (1000, many)):
        L = loom.loom_token_launch_config(loom.LOOM_OP_SAMPLE_TOKENS, [rows, vocab, loom.LOOM_F32, SMS])
        assert L["cluster"] == (ranks, 1, 1) and L["grid"] == (rows * ranks, 1, 1) and L["smem_bytes"] <= SM_BYTES


def test_product_on_one_sm(loom):
    # more than 32 tokens take pairs of CTAs, which one SM cannot hold
    cfg = lambda t, path, sms: loom.loom_token_launch_config(loom.LOOM_OP_I8_MATMUL, [t, 4096, 1024, 1, path, sms])   # noqa: E731
    assert cfg(32, loom.LOOM_PATH_TENSOR, 1)["grid"] == (1, 1, 1)
    assert cfg(33, loom.LOOM_PATH_AUTO, 1)["kernel"] == loom.LOOM_KERNEL_I8_MATMUL_DP4A
    with pytest.raises(loom.LoomError) as e:
        cfg(33, loom.LOOM_PATH_TENSOR, 1)
    assert e.value.status == loom.LOOM_ERR_ARG
    for t in (33, 300):
        L = cfg(t, loom.LOOM_PATH_TENSOR, 2)
        assert L["grid"] == (2, 1, 1) and L["cluster"] == (2, 1, 1)
    for sms in range(1, 160):
        for t in (5, 40, 300):
            L = cfg(t, loom.LOOM_PATH_AUTO, sms)
            assert L["grid"][0] >= 1 and L["cluster"][0] >= 1 and L["grid"][0] % L["cluster"][0] == 0
