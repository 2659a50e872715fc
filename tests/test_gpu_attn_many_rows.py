"""Attention of batches whose plan is made by a kernel of its own, and of more than 8192
workgroups: results of some rows against the 64-bit reference, and that neither many rows
nor one long row among them make a call several times slower than its keys do."""
import numpy as np
import pytest
import torch

from mamba_ssd_scan_05_amd import ssd
from test_gpu_attn import BF, DEV, F32, I32, Batch, check
from test_gpu_attn_batches import some

pytestmark = pytest.mark.gpu

CASES = [
    # rows, long rows, their start, the others' up to, L, Hq, Hk, N, page, window
    (300, (7, 250), 9000, 60, 1, 16, 8, 32, 16, 0),
    (257, (256,), 6000, 40, 1, 4, 1, 200, 24, 0),
    (1100, (0, 1, 2, 1099), 3000, 30, 1, 4, 2, 64, 16, 0),
    (5000, (4999,), 5000, 20, 1, 2, 2, 16, 16, 0),
    (70, (3, 69), 6000, 100, 20, 8, 4, 64, 16, 0),       # more than 16 query vectors a key head
    (70, (3, 69), 6000, 100, 20, 8, 4, 136, 10, 2500),
    (520, (100, 519), 5000, 30, 17, 16, 8, 8, 16, 0),    # fp32: 12480 workgroups
    (1040, (1000,), 4000, 20, 17, 8, 8, 8, 16, 0),       # 8320 (fp32 16640)
    (40, (39,), 20000, 200, 100, 32, 2, 16, 64, 0),      # few rows that can be cut, many vectors
]


def batch(case, dtype):
    b, far, top, ctx, L, Hq, Hk, N, page, window = case
    starts = [top - 10 * far.index(i) if i in far else (ctx * ((37 * i) % 101)) // 100 for i in range(b)]
    counts = [L if i % 5 or i in far else (i // 5) % (L + 1) for i in range(b)] if L > 1 else [1] * b
    return Batch(starts, counts, L, Hq, Hk, N, page, dtype, seed=b + N, spare=0)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=["b%d_L%d_Hq%d_Hk%d_N%d_page%d_w%d" % (c[0], *c[4:]) for c in CASES])
def test_long_rows_among_many(case, dtype):
    print("many rows", case, dtype, flush=True)
    b, far = case[:2]
    t = batch(case, dtype)
    some(t, sorted({0, 1, 5, b // 2, b - 2, b - 1, *far}), window=case[-1], step=case[4] == 1)


def test_replayed_with_other_rows_long():
    # the plan is made again by each replay
    t = batch(CASES[0], F32)
    b = t.b
    lens = torch.tensor(t.kv, dtype=I32)
    q, table, start = t.q[:, 0].to(DEV), t.table.to(DEV), torch.tensor(t.starts, dtype=I32, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(b, 16, device=DEV)
    ssd.ssd_attn_step(q, t.kc, t.vc, table, start, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_attn_step(q, t.kc, t.vc, table, start, out=out, lse=lse)
    for k in range(5):
        new = (lens - 1 if k == 2 else (torch.rand(b, generator=t.g) * lens).to(I32))
        new[k] = -1  # before the cache: sees nothing
        start.copy_(new)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        t.starts = new.tolist()
        rows = [0, 1, 2, 3, 4, 7, 8, 250, 299]
        part = object.__new__(Batch)
        part.__dict__.update(t.__dict__, b=len(rows), starts=[t.starts[i] for i in rows], counts=[1] * len(rows),
                             k=[t.k[i] for i in rows], v=[t.v[i] for i in rows], q=t.q[rows], table=t.table[rows])
        want, wl, eo, el = part.expect(float(np.float32(32 ** -0.5)), 0)
        check("out", out[rows][:, None], want, eo)
        check("lse", lse[rows][:, None], wl, el)
        eager = ssd.ssd_attn_step(q, t.kc, t.vc, table, start)
        assert torch.equal(out, eager)


def shared(b, L, Hq, Hk, N, capacity, lens, dtype, page=64, pool=512):
    """A call over pages shared by all rows, and its time in us (the shortest of several)."""
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.randn(pool, page, Hk, N, device=DEV).to(dtype) for _ in range(2))
    table = torch.randint(0, pool, (b, -(-capacity // page)), dtype=I32, generator=g).to(DEV)
    start = torch.tensor(lens, dtype=I32, device=DEV)
    q = torch.randn(b, L, Hq, N, device=DEV).to(dtype)
    out = torch.empty_like(q)
    best = float("inf")
    for _ in range(6):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        ssd.ssd_attn_fwd(q, kc, vc, table, start, out=out, return_lse=False)
        e1.record()
        torch.cuda.synchronize()
        best = min(best, 1e3 * e0.elapsed_time(e1))
    return best


def test_many_rows_with_a_wide_table():
    # a table that allows long rows, though none is: the plan takes its share, not the time of all rows for every row
    narrow = shared(32768, 1, 1, 1, 64, 4096, [200] * 32768, BF)
    wide = shared(32768, 1, 1, 1, 64, 8192, [200] * 32768, BF)
    print("32768 rows: %.0f us, with a wide table %.0f" % (narrow, wide), flush=True)
    assert wide < 3 * narrow


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_one_long_row_of_several_tokens(dtype):
    # 8192 workgroups; as many keys in all, in one row or in all alike
    b, L = (64, 64) if dtype == F32 else (1024, 20)
    even = shared(b, L, 32, 8, 64, 66000, [300 + 65536 // b] * b, dtype)
    uneven = shared(b, L, 32, 8, 64, 66000, [300] * (b - 1) + [300 + 65536], dtype)
    print("%d rows: %.0f us, one of them long %.0f" % (b, even, uneven), flush=True)
    assert uneven < 2 * even


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b", [3, 100, 300])
def test_rows_without_any_token(b, dtype):
    # nothing is written, in the pieces' plans of any number of rows; then one row has a token
    t = Batch([5000 if i == 1 else 30 for i in range(b)], [0] * b, 20, 4, 2, 16, 16, dtype, seed=2, spare=0)
    out, lse = t.call(0.25, 0)
    assert (out == 9.0).all() and (lse == 9.0).all()
    t.counts[1], t.starts[1] = 1, t.starts[1] - 1  # its key is the last cached one
    out, lse = t.call(0.25, 0)
    keep = out[1, 0].clone(), lse[1, 0].clone()
    out[1, 0], lse[1, 0] = 9.0, 9.0
    assert (out == 9.0).all() and (lse == 9.0).all()
    out[1, 0], lse[1, 0] = keep
    part = object.__new__(Batch)
    part.__dict__.update(t.__dict__, b=1, starts=t.starts[1:2], counts=[1], k=[t.k[1]], v=[t.v[1]], q=t.q[1:2], table=t.table[1:2])
    want, wl, eo, el = part.expect(0.25, 0)
    check("out", out[1:2], want, eo)
    check("lse", lse[1:2], wl, el)
