"""The timing table's decode rows: what a call reads is not in L2 from the call before."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench_table as bt  # noqa: E402


def test_input_sets_exceed_l2():
    for B, Hq, Hkv, L, D in bt.DECODE:
        for nbytes in (bt.decode_bytes(B, Hkv, L, D), bt.prefix_bytes(B, Hkv, L, 64, D)):
            n = bt.input_sets(nbytes)
            # all other sets are read between two uses of one
            assert n >= 2 and (n - 1) * nbytes >= bt.L2_BYTES, (B, Hkv, L, D, n, nbytes)
    assert bt.decode_bytes(8, 8, 8192, 128) == 2 * 8 * 8 * 8192 * 128 * 2
    assert bt.prefix_bytes(3, 2, 100, 7, 64) == 2 * 2 * 2 * 64 * (100 + 21)
