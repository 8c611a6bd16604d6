"""The scratch memory that the training operators ask for. No GPU needed."""
from test_train_abi import L  # noqa: F401


def test_layer_norm_workspace_follows_the_rows(L):  # noqa: F811
    """No more partial sums than rows."""
    size = L.moe_layer_norm_workspace_size
    for K in (8, 1000, 1111, 1 << 16, 1 << 20, 1 << 24):
        assert 0 < size(1, K) <= 2 * K * 4
        assert 0 < size(5, K) <= 5 * 2 * K * 4
        assert size(0, K) <= size(1, K) <= size(100, K) <= size(1 << 20, K)
    assert size(1 << 20, 2048) == size(1 << 30, 2048)
