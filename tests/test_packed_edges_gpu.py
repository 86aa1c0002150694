"""The packed-batch operators where a value that must not count meets one that
could make it count: left-out keys with the largest value rows, a bias that is
NaN, adapters that are not finite next to requests that are, and half-precision
operands and outputs at half precision's own tolerance.

Bounds, besides those stated in test_packed_gpu.py:
- half probabilities: the reference m of a row's final exponentials is the score of
  one of its keys, whose 2^0 = 1 is in the row sum l, so l >= 1.  A probability below
  the smallest normal half is stored with an absolute error of at most 2^-25, so o
  errs by at most keys * 2^-25 * max |v| on top of the relative terms.
- two bf16 parts of the rank-wide middle: the first leaves a remainder of at most
  2^-8 of it, the second rounds that remainder by 2^-8: 2^-16.
- an element computed again by 8 fp32 sums errs by less than 2 K u sum|a b|, like
  one of the tensor cores.
"""
import math

import pytest
import torch

from test_packed_gpu import HALF, U, attention64, gen, ints, lora64, norm64, normal, offsets, rope64, assert_within

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


# ------------------------------------------------------------------ attention: half operands at half's tolerance
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("lq,lk", [([700], [700]), ([1, 300, 5], [1000, 129, 2000]), ([256, 40], [4000, 1])])
@pytest.mark.parametrize("radius", [0, 100])
def test_attention_packed_half_precision(wd, dh, lq, lk, radius):
    g = gen(sum(lk) + dh + radius)
    cu_q, cu_k = offsets(lq), offsets(lk)
    q, k, v = normal(g, (cu_q[-1], 3 * dh), torch.float16), normal(g, (cu_k[-1], 3 * dh), torch.float16), normal(g, (cu_k[-1], 3 * dh), torch.float16)
    bias = normal(g, (3, 2 * radius + 1), std=2.0) if radius else None
    out = torch.empty((cu_q[-1], 3 * dh), dtype=torch.bfloat16, device="cuda")
    wd.wd_attention_packed(wd.WD_F16, 3, 3, dh, q, k, v, ints(cu_q), ints(cu_k), dh ** -0.5, out, bias=bias)
    wd.wd_check()
    want, ab = attention64(q, k, v, cu_q, cu_k, 3, 3, dh, dh ** -0.5, bias)
    for a, b, ka, kb in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        sub = (kb - ka) * 2.0 ** -25 * float(v[ka:kb].float().abs().max())
        assert_within(out[a:b], want[a:b], 2.0 ** -8 * want[a:b].abs() + 2 * 2.0 ** -11 * ab[a:b] + sub + 1e-6)


# ------------------------------------------------------------------ row operators: widths of one or two chunks on several warps
@pytest.mark.parametrize("D", [1280, 1792, 2560, 3584, 7168])
@pytest.mark.parametrize("td", [torch.bfloat16, torch.float32], ids=str)
def test_row_operators_at_more_widths(wd, D, td):
    g = gen(D)
    n, code = 19, wd.WD_F32 if td == torch.float32 else wd.WD_BF16
    x, y = normal(g, (n, D), td), normal(g, (n, D), torch.bfloat16, 0.3)
    gain, beta = 1 + normal(g, (D,), std=0.1), normal(g, (D,), std=0.1)
    for rms in (True, False):
        S, O = torch.empty_like(x), torch.empty((n, D), device="cuda")
        wd.wd_add_norm(code, x, wd.WD_BF16, y, wd.WD_NORM_RMS if rms else wd.WD_NORM_LAYER, gain, beta, 1e-6, S, wd.WD_F32, O)
        wd.wd_check()
        s, want, bound = norm64(x, y, gain, beta, rms, 1e-6)
        assert_within(S, s, (HALF[td] + U) * s.abs())
        assert_within(O, want, bound + U * want.abs())
    dh = 128
    k = normal(g, (n, 256), td)
    gk = 1 + normal(g, (256,), std=0.1)
    pos = torch.randint(0, 1000, (n, 3), generator=g, device="cuda").int()
    xo, ko = torch.empty_like(x), torch.empty_like(k)
    wd.wd_qknorm_rope_axes(code, dh, wd.wd_rope_axes.of((44, 42, 42)), pos, x, gain, xo, k, gk, ko, 1e-6)
    wd.wd_check()
    for t, gn, out in ((x, gain, xo), (k, gk, ko)):
        want, size = rope64(t, pos, gn, dh, (44, 42, 42), 10000.0, (1, 1, 1), 1e-6)
        assert_within(out, want, 64 * U * size + HALF[td] * want.abs() + 2.0 ** -25)


# ------------------------------------------------------------------ low-rank adapters
@pytest.mark.parametrize("M,N,K,r", [(300, 64, 136, 16), (500, 256, 520, 72), (20000, 256, 264, 32)])
def test_gemm_lora_half_output_keeps_half_precision(wd, M, N, K, r):
    """Half outputs whose larger share comes from the adapter: its middle must not be
    rounded more coarsely than the output."""
    g = gen(M + r)
    seg, ids = [0, 100, 107, M], [1, -1, 0]
    A, W, bias = normal(g, (M, K), torch.bfloat16), normal(g, (N, K), torch.bfloat16, 0.002), normal(g, (N,), std=0.01)
    down, up = normal(g, (2, r, K), torch.bfloat16, K ** -0.5), normal(g, (2, N, r), torch.bfloat16, 0.3)
    out = torch.empty((M, N), dtype=torch.float16, device="cuda")
    ws = torch.empty(wd.wd_gemm_lora_bytes(M, 3, r), dtype=torch.uint8, device="cuda").fill_(255)
    wd.wd_gemm_lora(M, N, K, A, W, bias, wd.wd_lora.of(ints(seg), ints(ids), down, up), wd.EPI_STORE_F16, out, ws)
    wd.wd_check()
    want, err = lora64(A, W, bias, seg, ids, down, up, None, 3)      # its err holds 2^-24 of the middle
    for a, b, i in zip(seg, seg[1:], ids):
        if i >= 0:
            err[a:b] += 2.0 ** -16 * (A[a:b].double() @ down[i].double().t()).abs() @ up[i].double().abs().t()
    assert_within(out, want, (err + U * want.abs()) * (1 + 2.0 ** -11) + 2.0 ** -11 * want.abs() + 2.0 ** -25)


def lora_with_bad_up(wd, lens, ids, M, N, K, r, epi, bad, start=0, seed=0):
    """A run with adapter 2's `up` not finite at the places `bad` [(n, j, value)], against the
    formula: finite elements within their bounds, and not finite exactly where the formula is not."""
    g = gen(seed + M + N + K + r)
    seg = offsets(lens, start)
    A, W, bias = normal(g, (M, K), torch.bfloat16), normal(g, (N, K), torch.bfloat16, 0.05), normal(g, (N,), std=0.1)
    down, up = normal(g, (3, r, K), torch.bfloat16, K ** -0.5), normal(g, (3, N, r), torch.bfloat16, 0.3)
    scale = torch.rand(3, generator=g, device="cuda") + 0.5
    for n, j, _ in bad:
        up[2, n, j] = 0
    fp32 = epi in (wd.EPI_F32, wd.EPI_RESID)
    v, err = lora64(A, W, bias, seg, ids, down, up, scale, 3 if fp32 else 1)
    hit = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    for a, b, i in zip(seg, seg[1:], ids):
        if i == 2:
            for n, _, _ in bad:
                hit[a:b, n] = True
    for n, j, x in bad:
        up[2, n, j] = x
    ga = normal(g, (N,)) + 3 if epi == wd.EPI_RESID else None
    out = normal(g, (M, N)) if fp32 else torch.empty((M, N), dtype=torch.float16 if epi == wd.EPI_STORE_F16 else torch.bfloat16, device="cuda")
    if epi == wd.EPI_RESID:
        want = out.double() + ga.double() * v
        bound = ga.double().abs() * err + 2 * U * (out.double().abs() + (ga.double() * v).abs())
    elif epi == wd.EPI_GELU:
        want = v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
        bound = 1.13 * err + 1e-6 * (want.abs() + 1)
    else:
        want, bound = v, err + U * v.abs()
    if not fp32:
        h = HALF[out.dtype]
        bound = bound * (1 + h) + h * want.abs() + (2.0 ** -25 if out.dtype == torch.float16 else 0)
    ws = torch.empty(wd.wd_gemm_lora_bytes(M, len(ids), r), dtype=torch.uint8, device="cuda").fill_(255)
    wd.wd_gemm_lora(M, N, K, A, W, bias, wd.wd_lora.of(ints(seg), ints(ids), down, up, scale), epi, out, ws, gate_a=ga)
    wd.wd_check()
    finite = torch.isfinite(out)
    assert not finite[hit].any(), "an element of the adapter's own rows is finite where the formula is not"
    assert finite[~hit].all(), f"{int((~finite & ~hit).sum())} elements of other requests or columns are not finite"
    assert_within(out.masked_fill(hit, 0.0), want.masked_fill(hit, 0.0), bound)


BAD = [(0, 0, math.nan), (17, 3, math.inf), (63, 7, -math.inf), (40, 1, math.nan)]


@pytest.mark.parametrize("epi", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("N,K,r", [(64, 136, 8), (128, 520, 40), (256, 1104, 72)])
def test_gemm_lora_bad_up_stays_in_its_request(wd, epi, N, K, r):
    """Requests and rows of none that share 128-row tiles with an adapter that is not finite."""
    lora_with_bad_up(wd, [40, 1, 129, 0, 130, 3], [0, 2, 1, 2, 2, -1], 345, N, K, r, epi, BAD + [(N - 1, r - 1, math.inf)], start=9)


@pytest.mark.parametrize("epi", [0, 1, 2, 3, 5])
def test_gemm_lora_bad_up_stays_in_its_request_on_sm_pairs(wd, epi):
    lens = [1, 127, 128, 200, 3, 0, 56, 600, 5000, 130, 126, 1, 9000]
    lora_with_bad_up(wd, lens, [0, 1, 2, -1, 1, 0, 2, 0, 1, 2, 0, 1, 0], 20000, 256, 1104, 40, epi,
                     BAD + [(130, 2, math.nan), (255, 39, -math.inf)], start=70)


def test_gemm_lora_wholly_bad_up(wd):
    """An adapter that is NaN throughout, one row in each of many tiles; and as the last tile's
    only request, whose tile ends with the matrix."""
    bad = [(n, j, math.nan) for n in range(64) for j in (0, 5)]
    lora_with_bad_up(wd, [100, 1] * 12, [1, 2] * 12, 1300, 64, 264, 8, 0, bad)
    lora_with_bad_up(wd, [128, 72], [0, 2], 200, 64, 264, 8, 2, bad)


def test_gemm_lora_bad_offsets_stay_inside(wd):
    """Offsets outside the matrix count as its ends.  Decreasing ones have unspecified results,
    but stay inside the buffers, a broken adapter's repair too: rows behind M are left alone."""
    g = gen(30)
    M, N, K, r = 500, 128, 136, 16
    A, W = normal(g, (M, K), torch.bfloat16), normal(g, (N, K), torch.bfloat16, 0.1)
    down, up = normal(g, (2, r, K), torch.bfloat16, K ** -0.5), normal(g, (2, N, r), torch.bfloat16)
    ids = [0, 1, 0, 1, 1, 0]
    ws = torch.empty(wd.wd_gemm_lora_bytes(M, len(ids), r), dtype=torch.uint8, device="cuda").fill_(255)

    def run(seg):
        room = torch.full((M + 100, N), 7.0, dtype=torch.bfloat16, device="cuda")
        wd.wd_gemm_lora(M, N, K, A, W, None, wd.wd_lora.of(ints(seg), ints(ids), down, up), wd.EPI_STORE, room[:M], ws)
        wd.wd_check()
        assert (room[M:] == 7.0).all()
        return room[:M]

    want = run([0, 100, 230, 230, 300, 490, 500])
    assert torch.equal(run([-(1 << 30), 100, 230, 230, 300, 490, 1 << 30]), want)
    up[1, 5, 3] = math.nan
    for seg in ([400, 300, 200, 100, 50, 20, 10], [0, 500, 0, 500, 0, 500, 0], [1 << 30, -5, 300, 2, 499, 128, 127], [500] * 7):
        run(seg)
