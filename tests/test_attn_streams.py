"""The cache's and the attention's calls given another stream than torch's current one:
what they allocate belongs to the stream that they run on (on the CPU with tensors that
only say they are on a GPU; every call then ends in the refusal of host memory)."""
import contextlib

import pytest
import torch

from mamba_ssd_scan_05_amd import ssd
from test_streams import Claimed, tensors

BF = torch.bfloat16


def arguments(device=None):
    def n(*s, dtype=BF):
        t = torch.zeros(s, dtype=dtype, device=device)
        return t if device is not None else t.as_subclass(Claimed)

    b, L, Hq, Hk, N = 2, 3, 4, 2, 32
    cache = dict(k_cache=n(5, 16, Hk, N), v_cache=n(5, 16, Hk, N), page_table=n(b, 2, dtype=torch.int32),
                 start=n(b, dtype=torch.int32))
    return {
        "kv_append": lambda s: ssd.ssd_kv_append(n(b, L, Hk, N), n(b, L, Hk, N), **cache, q=n(b, L, Hq, N), stream=s),
        "attn_fwd": lambda s: ssd.ssd_attn_fwd(n(b, L, Hq, N), **cache, stream=s),
        "attn_step": lambda s: ssd.ssd_attn_step(n(b, Hq, N), **cache, stream=s),
    }


NAMES = list(arguments())


@pytest.mark.parametrize("name", NAMES)
def test_allocations_are_made_on_the_calls_stream(name, monkeypatch):
    call = arguments()[name]
    current, seen = [7], []

    @contextlib.contextmanager
    def under(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: current[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: h)
    monkeypatch.setattr(torch.cuda, "stream", under)
    for f in ("empty", "empty_like"):
        def logged(*a, _f=getattr(torch, f), **k):
            seen.append(current[-1])
            return _f(*a, **k)
        monkeypatch.setattr(torch, f, logged)
    for stream, where in ((99, 99), (0, 0), (7, 7), (None, 7)):
        seen.clear()
        with pytest.raises(ssd.SsdError) as e:
            call(stream)
        assert e.value.status in (4, 8) and ("device" in str(e.value) or "address" in str(e.value)), e.value
        assert seen and set(seen) == {where}, (stream, seen)
        assert current == [7]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_results_belong_to_the_calls_stream(name):
    call = arguments("cuda")[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = tensors(call(s.cuda_stream))
    torch.cuda.synchronize()
    blocks = [(g["address"], g["address"] + g["total_size"], g["stream"]) for g in torch.cuda.memory_snapshot()]
    for t in got:
        assert [st for lo, hi, st in blocks if lo <= t.data_ptr() < hi] == [s.cuda_stream]


@pytest.mark.gpu
def test_results_under_pending_work_of_the_current_stream():
    # blocks freed on the current stream with work on them still to come: the call on the
    # other stream (its outputs, its workspace) does not get them
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 8, 128, generator=g).to(BF).cuda()
    kc, vc = (torch.randn(40, 64, 2, 128, generator=g).to(BF).cuda() for _ in range(2))
    table = torch.randperm(40, generator=g).to(torch.int32).view(2, 20).cuda()
    start = torch.tensor([1200, 700], dtype=torch.int32).cuda()
    want = ssd.ssd_attn_step(q, kc, vc, table, start)
    need = ssd.ssd_attn_workspace(2, 1, 8, 2, 128)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(5_000_000)  # about 2 ms ahead of the fills
        junk = [torch.full_like(want, float("nan")), torch.full((need // 4,), float("nan"), device="cuda")]
        del junk
        out = ssd.ssd_attn_step(q, kc, vc, table, start, stream=s.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
