"""Attention over packed rows where one row stands out of very many: each small
weight counts to 2^-11 of itself plus 2^-26 of the largest."""
import math

import pytest
import torch

from packed_layouts import LAYOUTS
from test_gpu_packed_attend import U, Located, dhs, run  # noqa: F401

pytestmark = pytest.mark.gpu
ONE, MOST = 0x38, 0x7E  # the codes of 1 and 448


@pytest.mark.parametrize("apart", [17.6, 22.3, 25.4, 26.6])
@pytest.mark.parametrize("name", ["no_wide", "grouped", "grouped_f16", "no_wide_f16"])
def test_one_row_far_above_the_others(dhs, name, apart):  # noqa: F811
    """400000 equal rows, each 2^-apart of one row's weight.  That row is 0 in the
    first half of the value's elements, where the output is what the others share,
    and 1 in the second, where they are 0.  More queries than the GPU has SMs, so
    that most are not split: a part without that row holds the others exactly.

    Bounds: a weight is off by 2^-11 of itself and 2^-26 of the largest; its score,
    of at most 19 nats in floats, and the exponential by 2^-17; sums over n rows in
    steps of 32 by 2^-23 (n / 32 + 8); the output by its own rounding."""
    env = Located(dhs, LAYOUTS[name], B=200, seed=31)
    lay, n = env.lay, 400000
    Q = torch.cuda.get_device_properties(0).multi_processor_count + 3
    rows = env.lay.random(2, env.g)
    rows[:, :lay.off_scale] = 0
    one = torch.ones(2 * lay.kv, device="cuda").view(torch.uint8)
    rows[:, lay.off_scale:lay.off_scale + one.numel()] = one
    key, value = rows[:, :lay.off_value].view(2, lay.kv, -1), rows[:, lay.off_value:lay.off_wide].view(2, lay.kv, -1)
    key[0, :, :2] = MOST
    half = lay.value // 2
    value[1, :, :half], value[0, :, half:] = ONE, ONE
    named = env.distinct(2)
    env.write(named, rows)
    loc = named[0, 1].expand(Q, n + 1).clone()
    loc[:, 123456] = named[0, 0]
    it, (q, out, lse, _) = env.item(loc)
    # the score of the row that stands out, in two elements
    x = apart * math.log(2) / lay.scale / 448
    q.zero_()
    q[..., 0] = x
    q[..., 1] = x - q[..., 0].float()
    s = 448 * lay.scale * (q[0, 0, 0].double() + q[0, 0, 1].double()).item()
    run(dhs, env.pool, lay, [it])
    torch.cuda.synchronize()
    tail = n * math.exp(-s)
    top, rest = 1 / (1 + tail), tail / (1 + tail)
    near = 2.0 ** -11 + 2.0 ** -16 + 2.0 ** -23 * (n / 32 + 8) + U[lay.dtype]
    err = (out[..., :half].double() - rest).abs().max().item()
    assert err <= rest * near + n * 2.0 ** -26 * top + 2.0 ** -25, "off by %.3g of %.3g" % (err, rest)
    assert (out[..., half:].double() - top).abs().max().item() <= top * near
    want = s + math.log1p(tail)
    assert (lse.double() - want).abs().max().item() <= 2.0 ** -16 * want
    assert env.pool.status() == (0, 0)
