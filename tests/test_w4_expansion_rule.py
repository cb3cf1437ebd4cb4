"""CPU test of the rows up to which the 4-bit product needs no workspace: 128, 192 of
8192 outputs and more, 320 where the dense weight would be of more than 192 MiB."""
import pytest

from unstructured_sparse_weight_amd import w4


@pytest.mark.parametrize("M,K,rows", [
    (64, 64, 128), (4096, 4096, 128), (8176, 8192, 128), (4096, 28672, 128), (8192, 64, 192), (8192, 8192, 192),
    (16384, 4096, 192), (24576, 4096, 192), (24592, 4096, 320), (20480, 5120, 320), (28672, 8192, 320), (65536, 2048, 192),
    (49152, 2560, 192), (8192, 16384, 320)])
def test_rows_without_workspace(M, K, rows):
    assert w4._sizes(M, K, 64, rows) == (0, 0)
    need, counters = w4._sizes(M, K, 64, rows + 1)
    assert need >= 2 * M * K + (1 << 16) and (counters == 0 or counters >= 1 << 16)
