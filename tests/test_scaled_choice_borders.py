"""Small grids of the product of 8-bit operands: a tile size is taken as far as its tiles
fill the CUs evenly, 256 of them here (no GPU)."""
from test_experts_choice import T128, T128_ONCE
from test_scaled_choice import RING64, RING64x128, RING128, kernel  # noqa: F401


def test_tiles_past_an_even_share(kernel):  # noqa: F811
    def rows(r, E, H, N):
        return kernel(r * E, 1, E, H, N)
    # tiles of 64: 8 x 64 of them are two a CU, 9 x 64 and 36 x 16 more
    assert rows(50, 8, 4096, 4096) == RING64
    assert rows(50, 9, 4096, 4096) == rows(50, 9, 2048, 4096) == T128_ONCE
    assert rows(30, 36, 2048, 1024) == RING64x128
    # of 128: 8 x 32, then 9 x 32 and 36 x 8
    assert rows(100, 8, 4096, 4096) == RING128
    assert rows(100, 9, 2048, 4096) == rows(100, 36, 2048, 1024) == T128_ONCE
    assert rows(480, 5, 2048, 1664) == T128


def test_one_expert_has_the_rows_that_there_are(kernel):  # noqa: F811
    def rows(r):
        return kernel(r, 1, 1, 2048, 4096)
    assert [rows(r) for r in (512, 513, 1024, 1025)] == [RING64, RING128, RING128, T128]
