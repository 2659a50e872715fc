"""Workspace of the attention for any batch (CPU only): sums of the pieces of rows that are
cut, whose number goes by the device and not by the batch."""
import itertools

from mamba_ssd_scan_05_amd import ssd


def test_workspace_is_bounded():
    # At most 1.6 (P + heads) pieces of cut rows with their heads, heads < P (more get none): P = 512 of 256
    # query vectors (128 of wide heads) or 4096 of 16, N sums, a maximum and a sum of 4 bytes each;
    # 16 bytes for each piece there may be (4096 + b) and for each cut row.
    most = max(1.6 * 2 * p * v * (n + 2) * 4 for p, v, n in ((512, 256, 128), (512, 128, 256), (4096, 16, 256)))
    for b, L, (Hq, Hk), N in itertools.product((1, 2, 15, 64, 65, 127, 256, 257, 511, 512, 4096, 65536), (1, 4, 17, 128, 512, 2048),
                                               ((1, 1), (8, 8), (10, 1), (32, 8), (32, 32), (64, 1)), (8, 64, 128, 256)):
        if b * L > 1 << 25:
            continue
        size = ssd.ssd_attn_workspace(b, L, Hq, Hk, N)
        assert -1 <= size <= most + 16 * (2 * 4096 + b) + 4096, (b, L, Hq, Hk, N, size)
    assert ssd.ssd_attn_workspace(127, 512, 32, 8, 128) < 127 * 512 * 32 * 128 * 2 / 4  # a quarter of the output


def test_large_batches_can_be_cut():
    # 8192 workgroups and more: one row far longer than the others is not left to a few of them
    for b, L, Hq, Hk, N in ((512, 128, 32, 8, 128), (64, 64, 32, 8, 128), (2048, 20, 16, 4, 64), (60000, 1, 8, 8, 64)):
        assert ssd.ssd_attn_workspace(b, L, Hq, Hk, N) > 0
