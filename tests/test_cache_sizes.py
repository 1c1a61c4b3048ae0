"""The scratch sizes that the header promises to callers who set it aside beforehand."""
from tests.test_cache_abi import fm  # noqa: F401  (the fixture)


def test_scratch_is_no_larger_than_documented(fm):  # noqa: F811
    # weights: two partial sums a block of at most 152, of 512 floats and their 16 bytes of metadata
    assert fm.fmha_cache_weights_workspace_size() == 2 * 152 * (512 * 4 + 16) <= 630_000
    # tree: two partials a block, of at most two 128-row blocks of O and LSE and their 20 bytes
    most = 2 * 152 * (2 * 128 * 129 * 4 + 20)
    assert most <= 40_200_000
    for B, T, H, H_k in ((1, 1, 1, 1), (64, 64, 32, 8), (1000, 200, 128, 1), (4096, 33, 64, 64)):
        for S in (1, 1000, 1 << 20, 1 << 30):
            assert 0 < fm.fmha_tree_workspace_size(B, T, H, H_k, 128, S) <= most
