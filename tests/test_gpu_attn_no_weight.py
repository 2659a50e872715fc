"""Queries whose every score is -infinity: out 0 and lse -infinity, whatever the values
hold (their products with weights of 0 are NaN where a value is an infinity)."""
import pytest

from test_gpu_attn import BF, F32, Batch, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [(0, 1, 64, 16), (300, 1, 64, 16), (300, 1, 256, 24), (130, 60, 64, 16), (130, 60, 136, 10),
                                  (3000, 1, 128, 16), (1500, 40, 32, 16)],
                         ids=lambda c: "start%d_L%d_N%d_page%d" % c)
def test_only_scores_of_minus_infinity(case, dtype):
    start, L, N, page = case
    print("no weight", case, dtype, flush=True)
    t = Batch([start, 20], [L, L], L, 4, 2, N, page, dtype, seed=8)
    t.q = t.q.abs() + 0.5
    mine = [int(e) for e in t.table[0] if 0 <= int(e) < t.pages]
    t.kc[mine, ..., 3] = float("-inf")
    t.vc[mine, ..., 5] = float("inf")
    t.vc[mine, ..., 6] = float("nan")
    out, lse = t.call(0.1, 0, step=L == 1)
    assert (out[0] == 0).all() and (lse[0] == float("-inf")).all()
    want, wl, eo, el = t.expect(0.1, 0)  # the other row as ever
    check("out", out[1], want[1], eo[1])
    check("lse", lse[1], wl[1], el[1])
