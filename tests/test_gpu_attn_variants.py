"""Every width of heads with pages of a multiple of 16 and others, few and many query
vectors of a key head: results, the place of every value among many keys, and odd
values in keys that only some queries see."""
import numpy as np
import pytest
import torch

from test_gpu_attn import BF, DEV, F32, Batch, check

pytestmark = pytest.mark.gpu

WIDTHS = [8, 32, 40, 64, 72, 96, 104, 128, 136, 192, 200, 256]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 21])
@pytest.mark.parametrize("page", [16, 9])
@pytest.mark.parametrize("N", WIDTHS)
def test_results(N, page, L, dtype):
    print("variant", N, page, L, dtype, flush=True)
    Batch([150, 40, 0], [L, L, L], L, 6, 2, N, page, dtype, seed=N + page).check(window=0 if N % 3 else 100, step=L == 1)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 20])
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("N", WIDTHS)
def test_every_value_has_its_place(N, page, L, dtype):
    # the same weight for every key: the mean of whole numbers, exact but for one rounding, with pages of
    # infinities beside them.  The weights are 1, or 1 - 2^-8 and 2^-8 of two parts, so the products are
    # multiples of 2^-8 and their sums, up to 8 * 1300 in size, exact in fp32; the division by the count is off
    # by 2^-23 of itself (its reciprocal and the product).
    print("places", N, page, L, dtype, flush=True)
    t = Batch([1270, 31], [L, L], L, 4, 2, N, page, dtype, seed=N)
    t.q.zero_()
    used = set()
    for i in range(2):
        t.v[i].copy_(torch.randint(-8, 9, t.v[i].shape, generator=t.g))
        for e in range(-(-t.kv[i] // page)):
            m = min(page, t.kv[i] - e * page)
            used.add(int(t.table[i, e]))
            t.vc[int(t.table[i, e]), :m] = t.v[i][e * page:e * page + m].to(DEV)
    for pg in range(t.pages):
        if pg not in used:
            t.kc[pg], t.vc[pg] = float("inf"), float("-inf")
    got, lse = t.call(1.0, 0, step=L == 1)
    for i in range(2):
        for s in range(0, L, 7):
            n = t.starts[i] + s + 1
            want = t.v[i][:n].double().mean(0).repeat_interleave(2, 0)
            tol = want.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -22) + 1e-37
            assert ((got[i, s].double().cpu() - want).abs() <= tol).all(), (i, s)
            assert (lse[i, s].double().cpu() - np.log(n)).abs().max() <= 2.0 ** -20


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("page", [16, 10])
@pytest.mark.parametrize("N", [96, 128, 136, 256])
def test_odd_values_reach_only_who_sees_them(N, page, bad, dtype):
    for L, start, at, window in ((4, 70, 72, 0), (30, 10, 25, 12), (150, 0, 75, 0), (150, 5, 70, 32)):
        print("odd", N, page, bad, dtype, L, flush=True)
        t = Batch([start], [L], L, 4, 2, N, page, dtype, seed=5)
        out, lse, eo, el = t.expect(0.125, window)  # with nothing odd in it
        pg, sl = int(t.table[0, at // page]), at % page
        for cache in (t.vc, t.kc):
            keep = cache[pg, sl].clone()
            cache[pg, sl, :, 5] = bad
            got, gl = t.call(0.125, window)
            cache[pg, sl] = keep
            pos = start + np.arange(L)
            blind = (pos < at) | (window > 0) & (pos - window >= at)
            check("out", got[0, blind], out[0, blind], eo[0, blind])
            check("lse", gl[0, blind], lse[0, blind], el[0, blind])
            if cache is t.vc:
                assert not torch.isfinite(got[0, ~blind][..., 5].float()).any()
                rest = [d for d in range(N) if d != 5]
                check("out", got[..., rest], out[..., rest], eo[..., rest])
                check("lse", gl, lse, el)
            elif bad != bad:
                assert torch.isnan(got[0, ~blind]).all() and torch.isnan(gl[0, ~blind]).all()
