"""The softmax's weights in the product with the values: up to 16 query vectors of a
row and key head take them with what bf16 leaves over.

w = h + r, where h is w's bits less a quarter of bf16's last place, cut off behind that
place: r lies between 1/4 and 5/4 of the place, at most 1.25 2^-7 w, and is exact in fp32;
as bf16 it is off by 2^-8 of itself, so the weight that the product sees by 1.25 2^-15 of
itself.  That takes the place of the 2^-8 of a weight rounded once; the rest of the
reference's bound stays.
"""
import numpy as np
import pytest
import torch

from test_gpu_attn import BF, Batch

pytestmark = pytest.mark.gpu


class Whole(Batch):
    def expect(self, scale, window):
        keep, self.dtype = self.dtype, torch.float32
        out, lse, eo, el = super().expect(scale, window)  # weights not rounded
        self.dtype = keep
        G = self.Hq // self.Hk
        for i in range(self.b):  # the weights sum to 1: at most that share of the largest value's size
            v = np.abs(self.v[i].double().numpy())
            if len(v):
                eo[i] += 1.25 * 2.0 ** -15 * v.max(0).repeat(G, 0)[None]
        return out, lse, eo, el


CASES = [
    # starts, L, Hq, Hk, N, page, window
    ([999], 1, 32, 8, 128, 16, 0),
    ([5, 700, 64], 1, 6, 2, 64, 24, 0),
    ([2000, 300], 1, 10, 1, 256, 16, 500),
    ([30000], 1, 4, 1, 32, 64, 0),
    ([300, 90], 4, 8, 2, 96, 32, 0),
    ([410], 16, 2, 2, 192, 16, 0),
]


@pytest.mark.parametrize("case", CASES, ids=["b%d_L%d_Hq%d_Hk%d_N%d_page%d_w%d" % ((len(c[0]),) + c[1:]) for c in CASES])
def test_weights_of_few_queries(case):
    starts, L, Hq, Hk, N, page, window = case
    print("weights", case, flush=True)
    Whole(starts, [L] * len(starts), L, Hq, Hk, N, page, BF, seed=11).check(window=window, step=L == 1)


@pytest.mark.parametrize("N", [64, 256])
def test_infinite_values_that_every_query_sees(N):
    # the weights' second parts have either sign, or are 0: the value stays what it is
    t = Batch([300], [2], 2, 4, 2, N, 16, BF, seed=12)
    for at, bad, scale in ((0, np.inf, 0.1), (70, -np.inf, 0.1), (299, np.inf, 0.1), (64, np.inf, 0.5)):
        t.vc[int(t.table[0, at // 16]), at % 16, :, 5] = bad
        out, gl = t.call(scale, 0)
        assert (out[..., 5].float() == bad).all()
        t.vc[int(t.table[0, at // 16]), at % 16, :, 5] = 0
