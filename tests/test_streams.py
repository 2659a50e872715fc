"""Calls given another stream than torch's current one: what they allocate
belongs to the stream that they run on.  On the CPU with tensors that only say
they are on a GPU (every call then ends in the refusal of host memory), on the
GPU by the allocator's own record and by results under pending work."""
import contextlib

import pytest
import torch

from mamba_ssd_scan_05_amd import ssd

BF = torch.bfloat16


class Claimed(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def arguments(device=None):
    def n(*s, dtype=torch.float32):
        t = torch.zeros(s, dtype=dtype, device=device)
        return t if device is not None else t.as_subclass(Claimed)

    b, L, H, P, N, D = 2, 80, 2, 16, 32, 24
    scan = dict(x=n(b, L, H, P, dtype=BF), dt=n(b, L, H), dt_bias=n(H), A=n(H), B=n(b, L, 1, N, dtype=BF),
                C=n(b, L, 1, N, dtype=BF))
    x = n(b, L, D)
    return {
        "scan_fwd": lambda s: ssd.ssd_scan_fwd(**scan, stream=s),
        "scan_fwd_noalloc": lambda s: ssd.ssd_scan_fwd_noalloc(**scan, stream=s),
        "scan_fwd_gated": lambda s: ssd.ssd_scan_fwd_gated(**scan, z=scan["x"], stream=s),
        "scan_fwd_rows": lambda s: ssd.ssd_scan_fwd_rows(**scan, stream=s),
        "selective_scan_fwd": lambda s: ssd.ssd_selective_scan_fwd(n(b, L, 64), n(b, L, 64), None, n(64, 16), n(b, L, 1, 16),
                                                                   n(b, L, 1, 16), stream=s),
        "scan_bwd": lambda s: ssd.ssd_scan_bwd(**scan, D=n(H), init_state=None, dout=n(b, L, H, P, dtype=BF), stream=s),
        "scan_bwd_gated": lambda s: ssd.ssd_scan_bwd_gated(**scan, z=scan["x"], D=n(H), init_state=None,
                                                           dout=n(b, L, H, P, dtype=BF), stream=s),
        "step": lambda s: ssd.ssd_step(n(b, H, P, N), n(b, H, P), n(b, H), n(H), n(b, 1, N), n(b, 1, N), stream=s),
        "glr_fwd": lambda s: ssd.ssd_glr_fwd(n(b, 300, D), n(b, 300, D), n(b, 300, D), n(D), stream=s),
        "glr_bwd": lambda s: ssd.ssd_glr_bwd(x, x, x, n(D), dout=x, stream=s),
        "glr_step": lambda s: ssd.ssd_glr_step(n(b, D), n(b, D), n(b, D), n(b, D), n(D), stream=s),
        "norm_rotate_fwd": lambda s: ssd.ssd_norm_rotate_fwd(n(b, L, H, N), n(b, L, 1, N), stream=s),
        "norm_rotate_bwd": lambda s: ssd.ssd_norm_rotate_bwd(n(b, L, H, N), n(b, L, 1, N), None, None, None, None,
                                                             n(b, L, H, N), n(b, L, 1, N), stream=s),
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


def tensors(o):
    o = o.values() if isinstance(o, dict) else o if isinstance(o, tuple) else (o,)
    return [t for t in o if t is not None]


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
    # blocks freed on the current stream with work on them still to come: the
    # call on the other stream does not get them
    g = torch.Generator().manual_seed(1)
    x, r, i = (torch.randn(2, 400, 72, generator=g).to(BF).cuda() for _ in range(3))
    A = -torch.rand(72, generator=g).cuda()
    want, wf = ssd.ssd_glr_fwd(x, r, i, A)
    wg = ssd.ssd_glr_bwd(x, r, i, A, dout=x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(5_000_000)  # about 2 ms ahead of the fills
        junk = [torch.full_like(t, float("nan")) for t in (want, wf, *wg.values())]
        del junk
        out, fin = ssd.ssd_glr_fwd(x, r, i, A, stream=s.cuda_stream)
        d = ssd.ssd_glr_bwd(x, r, i, A, dout=x, stream=s.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(fin, wf) and all(torch.equal(d[k], wg[k]) for k in wg)
