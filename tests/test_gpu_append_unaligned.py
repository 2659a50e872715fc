"""The append with a q_out (and inputs) that start between 16-byte boundaries: what is
turned and what is not, and what lies on both sides of q_out."""
import pytest
import torch

from mamba_ssd_scan_05_amd import ssd
from test_gpu_append import BF, DEV, F32, check, expect, make, num

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("npair,layout", [(0, "dense"), (8, "dense"), (20, "offset"), (32, "offset")])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_q_out_at_any_element(off, npair, layout, interleaved, dtype):
    print("unaligned", off, npair, layout, interleaved, dtype, flush=True)
    t = make(2, 9, 6, 2, 64, npair, 24, dtype, layout, ctx=40)
    n = t["q"].numel()
    wide = torch.full((n + 16,), 9.0, dtype=dtype, device=DEV)
    q_out = wide[off:off + n].view(t["q"].shape)
    assert q_out.data_ptr() % 16 == off * q_out.element_size()
    kc, ek, vc, qo, eq = expect(t, [9, 4], interleaved, t["kc"], t["vc"])
    tok = torch.tensor([9, 4], dtype=torch.int32, device=DEV)
    d = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in t.items()}
    ssd.ssd_kv_append(d["k"], d["v"], d["kc"], d["vc"], d["table"], d["start"], q=d["q"], freqs=d["freqs"], tokens=tok,
                      interleaved=interleaved, q_out=q_out)
    torch.cuda.synchronize()
    check("q_out", q_out, qo, eq)
    check("k_cache", t["kc"], kc, ek)
    assert (num(t["vc"]) == vc).all()
    assert (wide[:off] == 9.0).all() and (wide[off + n:] == 9.0).all()
