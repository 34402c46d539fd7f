"""Sizes that gc_orthogonalize takes, decided on the host: no GPU needed."""
import pytest


@pytest.fixture(scope="module")
def gc():
    import __graft_entry__
    __graft_entry__.build()
    from gradient_compression_ef_gb300 import gc as binding
    return binding


def test_scratch_of_the_largest_matrices(gc):
    """Four planes of X and four of A at least, or a refusal: never a wrapped number."""
    for k in range(31):
        for j in range(31):
            m, n = 1 << k, 1 << j
            got = gc.orthogonalize_scratch_bytes(m, n)
            if k + j <= 48:
                assert got >= 8 * m * n + 8 * min(m, n) ** 2, (k, j)
            else:
                assert got == -1, (k, j)
    assert gc.orthogonalize_scratch_bytes(2 ** 30, 2 ** 18 + 1) == -1
    assert gc.orthogonalize_scratch_bytes(2 ** 30 + 1, 1) == -1
    assert gc.orthogonalize_scratch_bytes(-1, 1) == -1
    assert gc.orthogonalize_scratch_bytes(0, 2 ** 30) == 0
