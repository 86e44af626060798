"""The tight bounds of fp32 attention, on the CPU: they hold for exact arithmetic and are broken where the
second fp16 part of the queries or of the weights is left out (in the oracle)."""

import numpy as np
import pytest

import kvq_tight as T


@pytest.mark.parametrize("d,group,bits,n,lens", T.CASES)
def test_bounds_see_a_lost_part(d, group, bits, n, lens):
    cfg, arrays, q = T.problem(d, group, bits, lens, 16, n=n)
    broken = {"q": 0.0, "w": 0.0}
    for _, qi, k, v in T.rows_of(cfg, arrays, q, lens):
        o, bound = T.row(qi, k, v, d)
        for what in broken:
            err = np.abs(T.row_in_one_part(qi, k, v, d, what) - o) / bound
            broken[what] = max(broken[what], float(err.max()))
    assert min(broken.values()) > 2, broken


def test_the_parts_are_the_oracle_s_rows():
    cfg, arrays, q = T.problem(128, 4, 4, [20, 5], 16)
    from oracle import kvq as O
    ref, _ = O.attention(cfg, arrays, q.double().numpy(), [20, 5], table=arrays["table"])
    assert T.worst(cfg, arrays, q, [20, 5], ref) < 1e-3
