"""Linear attention and the linear layer on the GPU at the edges of what their calls allow:
rows that end inside a warp, padded outputs, decays of zero, tails of the activations,
values near the largest number, many sequences, waits that give up, several threads.

Tolerances are those of test_gpu_ops.py where nothing else is said.
"""
import math

import numpy as np
import pytest

from oracle import ops
from test_gpu_ops import DT, U16, U32, _check_la, _check_linear, _f64, _la_inputs, _rand, fi  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,pad,shift", [(64, 8, 0), (64, 3, 1), (128, 8, 0), (100, 1, 0), (33, 2, 0)])
def test_prefill_sequences_that_end_inside_a_warp(fi, d, pad, shift, dtype):  # noqa: F811
    # lengths at which the lanes of one warp stand on both sides of the end, at first,
    # middle and last rows of chunks; what lies between the rows of o, before the first and
    # behind the last one stays as it was
    lens = [1, 31, 33, 70, 97, 127, 129, 255, 300]
    n, B, H = 300, len(lens), 2
    q, k, v, ld, s0 = _la_inputs(n, B, H, d, d, dtype, 17 * d + pad)
    base = torch.full((n * B * H * (d + pad) + shift + 16,), 7.0, dtype=DT[dtype], device="cuda")
    o = base[shift:shift + n * B * H * (d + pad)].view(n, B, H, d + pad)[..., :d]
    for b, m in enumerate(lens):
        for t in (q, k, v):
            t[m:, b] = math.nan
    S = torch.empty_like(s0)
    fi.linattn_prefill(q, k, v, ld, o, state_in=s0, state_out=S, scale=d ** -0.5,
                       lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    fi.op_sync()
    got = torch.zeros(n, B, H, d, dtype=DT[dtype], device="cuda")
    for b, m in enumerate(lens):
        got[:m, b] = o[:m, b]
        o[:m, b] = 7.0
        for t in (q, k, v):
            t[m:, b] = 0
    assert (base == 7.0).all()
    _check_la(got, S, q, k, v, ld, d ** -0.5, s0, lens, dtype)
