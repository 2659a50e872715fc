"""Arguments of the Python calls of the attention that are refused by the library, and not by an
error of Python's on the way to it (CPU only)."""
import pytest
import torch

from mamba_ssd_scan_05_amd import ssd

K = torch.zeros(5, 8, 2, 32)
TABLE, START = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)


@pytest.mark.parametrize("call,rank", [(ssd.ssd_attn_step, 3), (ssd.ssd_attn_fwd, 4)], ids=["step", "fwd"])
def test_refused_by_the_library(call, rank):
    q = torch.zeros((2, 3, 4, 32) if rank == 4 else (2, 4, 32))
    for bad, word in ((q[..., :0], "SHAPE"), (torch.zeros(()), "SHAPE"), (q[:0], "SHAPE"), (q[0], "SHAPE"),
                      (q.half(), "DTYPE"), (q[..., :12], "UNSUPPORTED")):
        with pytest.raises(ssd.SsdError, match=word):
            call(bad, K, K, TABLE, START)
    for caches in ((None, K), (K, None)):
        with pytest.raises(ssd.SsdError, match="NULL"):
            call(q, *caches, TABLE, START)
    for scale in (0.0, 1e31, float("nan")):
        with pytest.raises(ssd.SsdError, match="scale"):
            call(q, K, K, TABLE, START, scale=scale)
