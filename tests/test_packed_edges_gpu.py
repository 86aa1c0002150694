"""The packed-batch operators where a value that must not count meets one that
could make it count: left-out keys with the largest value rows, and a bias that is
NaN.

The bounds are those stated in test_packed_gpu.py.
"""
import math

import pytest
import torch

from test_packed_gpu import attention64, gen, ints, normal, assert_within

pytestmark = pytest.mark.gpu
HUGE = 3.3e38          # finite in bf16 and fp32


@pytest.fixture(scope="module")
def wd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from flow_matching_video_b200 import build
    build.build()
    from flow_matching_video_b200 import wd as _wd
    return _wd


# ------------------------------------------------------------------ attention: keys that are left out
@pytest.mark.parametrize("low", [-math.inf, -1000.0], ids=str)
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("radius,both", [(1, False), (20, True), (200, False)])
def test_left_out_keys_have_no_weight(wd, dh, radius, both, low):
    """Keys at weight exp(low), which is zero in any precision, with value rows near the
    type's largest number: the output is that of the other keys alone."""
    g = gen(radius + dh)
    lq, lk = 64, 500
    q, k, v = normal(g, (lq, 2 * dh), torch.bfloat16), normal(g, (lk, 2 * dh), torch.bfloat16), normal(g, (lk, 2 * dh), torch.bfloat16)
    bias = normal(g, (2, 2 * radius + 1))
    if both:
        bias[:, 0] = low
    bias[:, -1] = low
    seen = lq - 1 + radius          # keys from here on lie behind the last row's window
    sign = torch.where(torch.rand((lk - seen, 2 * dh), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    v[seen:] = (HUGE * sign).bfloat16()
    out = torch.empty_like(q)
    wd.wd_attention_packed(wd.WD_BF16, 2, 2, dh, q, k, v, ints([0, lq]), ints([0, lk]), dh ** -0.5, out, bias=bias)
    wd.wd_check()
    visible = v.clone()
    visible[seen:] = 0
    want, ab = attention64(q, k, visible, [0, lq], [0, lk], 2, 2, dh, dh ** -0.5, bias)
    assert_within(out, want, 2.0 ** -8 * want.abs() + 2.0 ** -7 * ab + 1e-6)


@pytest.mark.parametrize("dh", [64, 128])
def test_far_smaller_scores_have_no_weight(wd, dh):
    """The same without a bias: scores so far below the row's largest that 2^x is zero."""
    g = gen(dh)
    q = torch.ones((70, dh), dtype=torch.bfloat16, device="cuda")
    k, v = normal(g, (200, dh), torch.bfloat16, 0.1), normal(g, (200, dh), torch.bfloat16)
    k[100:] -= 40.0
    v[100:] = HUGE
    out = torch.empty_like(q)
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, dh, q, k, v, ints([0, 70]), ints([0, 200]), 0.5, out)
    wd.wd_check()
    want, ab = attention64(q, k[:100], v[:100], [0, 70], [0, 100], 1, 1, dh, 0.5)
    assert_within(out, want, 2.0 ** -8 * want.abs() + 2.0 ** -7 * ab + 1e-6)


@pytest.mark.parametrize("dh,td", [(64, torch.bfloat16), (128, torch.float16)])
@pytest.mark.parametrize("at", [0, 3, 6, 7, 8, 16])
def test_nan_bias_gives_nan_rows(wd, dh, td, at):
    """A NaN in the table: NaN in every row that reads it, and in no other row or head."""
    g = gen(at)
    n, R = 300, 8
    q, k, v = (normal(g, (n, 2 * dh), td) for _ in range(3))
    bias = normal(g, (2, 2 * R + 1))
    clean, out = (torch.empty((n, 2 * dh), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    code, cu = wd.WD_F16 if td == torch.float16 else wd.WD_BF16, ints([0, n])
    wd.wd_attention_packed(code, 2, 2, dh, q, k, v, cu, cu, dh ** -0.5, clean, bias=bias)
    bias[1, at] = math.nan
    wd.wd_attention_packed(code, 2, 2, dh, q, k, v, cu, cu, dh ** -0.5, out, bias=bias)
    wd.wd_check()
    d = (torch.arange(n)[None] - torch.arange(n)[:, None]).clamp(-R, R) + R
    hit = (d == at).any(1).cuda()
    assert hit.any()
    assert torch.equal(out[:, :dh], clean[:, :dh]) and torch.equal(out[~hit], clean[~hit])
    assert out[hit, dh:].isnan().all()
