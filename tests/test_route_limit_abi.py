"""The router's row numbers stay within 32 bits: the last block's rows, and the
next row of every warp, are counted past M."""
import gemm_epilogue_fusion_gb300 as g

A, GB = 0x7F0000000000, 1 << 30
LIMIT = (1 << 31) - (1 << 24)


def at(i):
    return A + i * 64 * GB


def test_rows_near_2_to_the_31_are_refused():
    lib = g.load_library()
    for M in (LIMIT, (1 << 31) - 40, (1 << 31) - 2):
        assert lib.coda_route(at(0), 8, 1, 1, at(1), at(2), at(3), at(4), at(5), M, 8, g.CODA_BF16, None) \
            == g.CODA_ERR_INVALID_ARG
        assert b"M = " in lib.coda_last_error()
        assert lib.coda_route_backward(at(0), 8, at(1), at(2), at(3), 0, at(4), 8, M, 8, 1, g.CODA_BF16, None) \
            == g.CODA_ERR_INVALID_ARG
        assert lib.coda_route_workspace_bytes(M, 8, 1) == -1
    assert lib.coda_route_workspace_bytes(LIMIT - 1, 8, 1) > 0
    # blocks of the choice, and rows of a block, for the most rows
    rows_per_block = -(-(LIMIT - 1) // 144)
    blocks = -(-(LIMIT - 1) // rows_per_block)
    assert blocks * rows_per_block < 1 << 31
    # a warp's next row, and the gradient's blocks of 8 warps, 8 of them for each of up to 1000 SMs
    assert LIMIT - 1 + max(32, 1000 * 8 * 8) < 1 << 31
