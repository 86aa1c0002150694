"""The packed-batch operators on the GPU against plain 64-bit formulas.

Bounds (u = 2^-24, the fp32 rounding; a bf16 store rounds by 2^-8 of the value,
an IEEE half store by 2^-11 of it or 2^-25, an e4m3 store by 2^-4 of it or
2^-10 of the scale):
- attention: the output's bf16 store, 2^-8 |o|; every probability enters P V in
  the operand type, u_P = 2^-8 or 2^-11 relative (and for half 2^-25 absolute
  against a row sum of at least 2^-8 of the largest p, one per key); its 2^x
  errs by 7.5e-5 at most and the logits by fp32 rounding, which a factor of two
  on u_P covers: 2 u_P softmax(t)|v|.
- rows: a sum of squares over at most 8192 elements in chains of 64 and trees of
  7 errs by 80 u relative, its root by half of that, rsqrtf by 4 u, products by
  u each; cosine and sine by 2^-23.  64 u covers each row operator's factor.
- low-rank products: fp32 accumulation in any order and with truncating adders
  errs by 2 K u sum|a b|; the middle is rounded to bf16 (2^-8 of it), or to three
  bf16 parts (2^-24) for fp32 outputs.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}


@pytest.fixture(scope="module")
def wd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from flow_matching_video_b200 import build
    build.build()
    from flow_matching_video_b200 import wd as _wd
    return _wd


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def offsets(lens, start=0):
    out = [start]
    for n in lens:
        out.append(out[-1] + n)
    return out


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def assert_within(got, want, bound, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert over.max() <= 0, f"{what} {int((over > 0).sum())} of {over.numel()} outside the bound, by up to {float(over.max())}"


# ------------------------------------------------------------------ attention
def attention64(q, k, v, cu_q, cu_k, H, Hk, dh, scale, bias=None):
    """(o, softmax |v|) in 64 bits for the rows of the sequences; zeros elsewhere."""
    o = torch.zeros(q.shape[0], H, dh, dtype=torch.float64, device=q.device)
    ab = torch.zeros_like(o)
    for a, b, ka, kb in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        if a == b or ka == kb:
            continue
        Q = q[a:b].double().view(b - a, H, dh)
        K = k[ka:kb].double().view(kb - ka, Hk, dh).repeat_interleave(H // Hk, 1)
        V = v[ka:kb].double().view(kb - ka, Hk, dh).repeat_interleave(H // Hk, 1)
        t = torch.einsum("ihd,jhd->hij", Q, K) * scale
        if bias is not None:
            R = bias.shape[1] // 2
            d = torch.arange(kb - ka, device=q.device)[None] - torch.arange(b - a, device=q.device)[:, None]
            t = t + bias.double()[:, d.clamp(-R, R) + R]
        seen = (t > -math.inf).any(-1, keepdim=True)
        p = torch.where(seen, torch.softmax(torch.where(seen, t, 0.0), -1), 0.0)
        o[a:b] = torch.einsum("hij,jhd->ihd", p, V)
        ab[a:b] = torch.einsum("hij,jhd->ihd", p, V.abs())
    return o.view(q.shape[0], -1), ab.view(q.shape[0], -1)


def attention_bound(o, ab, td, keys, v):
    u_p = HALF[td]
    sub = keys * 2.0 ** -25 * 2.0 ** 8 * float(v.float().abs().max()) * 2 if td == torch.float16 else 0.0
    return 2.0 ** -8 * o.abs() + 2 * u_p * ab + min(sub, 2e-2) + 1e-6


def run_attention(wd, lq, lk, H, Hk, dh, td, radius=0, edges=(0.0, 0.0), seed=0, pad=3, scale=None):
    g = gen(seed + sum(lq) + dh + radius)
    cu_q, cu_k = offsets(lq, 2), offsets(lk, 1)
    nq, nk = cu_q[-1] + pad, cu_k[-1] + pad
    q, k, v = normal(g, (nq, H * dh), td), normal(g, (nk, Hk * dh), td), normal(g, (nk, Hk * dh), td)
    # rows outside every sequence hold what must not reach any output
    for t in (k, v):
        t[:1] = math.nan
        t[cu_k[-1]:] = math.nan
    q[:2] = math.inf
    bias = None
    if radius:
        bias = normal(g, (H, 2 * radius + 1), std=2.0)
        bias[:, 0] += edges[0]
        bias[:, -1] += edges[1]
    scale = scale or dh ** -0.5
    out = torch.full((nq, H * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    wd.wd_attention_packed(wd.WD_F16 if td == torch.float16 else wd.WD_BF16, H, Hk, dh, q, k, v, ints(cu_q), ints(cu_k),
                           scale, out, bias=bias)
    wd.wd_check()
    want, ab = attention64(q, k, v, cu_q, cu_k, H, Hk, dh, scale, bias)
    inside = slice(cu_q[0], cu_q[-1])
    assert_within(out[inside], want[inside], attention_bound(want[inside], ab[inside], td, max(lk), v[1:cu_k[-1]]))
    assert (out[:cu_q[0]] == 7.0).all() and (out[cu_q[-1]:] == 7.0).all()   # rows of no sequence are left alone
    return out


# lengths around the tiles' edges (128 keys, 128 and 256 rows), empty sequences among them
LENGTHS = [[1], [128], [129, 1], [256, 257, 0, 5], [63, 64, 65, 127], [700], [1, 1, 1, 300, 2], [0, 0, 40]]


@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("dh,td", [(128, torch.bfloat16), (64, torch.bfloat16), (128, torch.float16), (64, torch.float16)])
def test_attention_packed_self(wd, lens, dh, td):
    run_attention(wd, lens, lens, 2, 2, dh, td)


@pytest.mark.parametrize("lq,lk", [([5, 300, 1], [0, 9, 400]), ([260, 130], [1, 127]), ([1], [1000]), ([40, 0], [0, 40])])
@pytest.mark.parametrize("H,Hk", [(3, 3), (4, 2), (6, 1)])
def test_attention_packed_cross_and_shared_heads(wd, lq, lk, H, Hk):
    run_attention(wd, lq, lk, H, Hk, 128, torch.float16)
    run_attention(wd, lq, lk, H, Hk, 64, torch.bfloat16)


@pytest.mark.parametrize("radius", [1, 31, 128, 1024])
@pytest.mark.parametrize("lens", [[1], [300, 7], [1500], [0, 513, 255]], ids=str)
def test_attention_packed_bias_by_distance(wd, radius, lens):
    run_attention(wd, lens, lens, 3, 3, 64, torch.bfloat16, radius=radius, scale=1.0 / 8)
    run_attention(wd, lens, lens, 2, 1, 128, torch.float16, radius=radius)


@pytest.mark.parametrize("radius", [1, 2, 100, 600])
@pytest.mark.parametrize("edges", [(-math.inf, -math.inf), (0.0, -math.inf), (-math.inf, 0.0)], ids=str)
def test_attention_packed_window(wd, radius, edges):
    run_attention(wd, [900, 1, 129], [900, 1, 129], 2, 2, 128, torch.bfloat16, radius=radius, edges=edges)
    # more queries than keys: rows whose window holds no key give zeros
    run_attention(wd, [1000, 300], [200, 700], 2, 2, 64, torch.bfloat16, radius=radius, edges=edges)


def test_attention_packed_every_key_left_out(wd):
    g = gen(5)
    q, k, v = (normal(g, (300, 256), torch.bfloat16) for _ in range(3))
    out = torch.full_like(q, 7.0)
    bias = torch.full((2, 9), -math.inf, device="cuda")
    bias[1, 0] = 0.0          # head 1 sees what lies 4 or more before: rows 0 .. 3 nothing
    cu = ints([0, 300])
    wd.wd_attention_packed(wd.WD_BF16, 2, 2, 128, q, k, v, cu, cu, 0.1, out, bias=bias)
    wd.wd_check()
    assert (out[:, :128] == 0).all() and (out[:4, 128:] == 0).all()
    want, ab = attention64(q, k, v, [0, 300], [0, 300], 2, 2, 128, 0.1, bias)
    assert_within(out, want, attention_bound(want, ab, torch.bfloat16, 300, v))


def test_attention_packed_lowest_bias_is_a_number(wd):
    """A finite lowest bias absorbs every score: all keys weigh the same, and next to a
    seen key it weighs nothing."""
    g = gen(6)
    q, k, v = (normal(g, (200, 128), torch.bfloat16) for _ in range(3))
    out = torch.empty_like(q)
    low = torch.finfo(torch.float32).min
    cu = ints([0, 200])
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q, k, v, cu, cu, 0.1, out, bias=torch.full((1, 3), low, device="cuda"))
    wd.wd_check()
    mean = v.double().mean(0).expand(200, 128)
    assert_within(out, mean, 2.0 ** -8 * mean.abs() + 2.0 ** -7 * v.double().abs().mean(0) + 1e-6)
    bias = torch.tensor([[low, 0.0, low]], device="cuda")   # only the key at distance 0
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q, k, v, cu, cu, 0.1, out, bias=bias)
    wd.wd_check()
    assert_within(out, v.double(), 2.0 ** -7 * v.double().abs() + 1e-6)


def test_attention_packed_nan_and_inf_stay_in_their_rows(wd):
    g = gen(7)
    q, k, v = (normal(g, (400, 128), torch.bfloat16) for _ in range(3))
    cu = ints([0, 150, 400])
    clean = torch.empty_like(q)
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q, k, v, cu, cu, 0.1, clean)
    q2, out = q.clone(), torch.empty_like(q)
    q2[3] = math.nan          # a row of NaN scores
    q2[170, 0], k2 = math.inf, k.clone()
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q2, k2, v, cu, cu, 0.1, out)
    wd.wd_check()
    bad = torch.zeros(400, dtype=torch.bool, device="cuda")
    bad[[3, 170]] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])
    for j in (0, 6, 149):     # a NaN key (each 2^x pipe) reaches all rows of its own sequence only
        k2 = k.clone()
        k2[j, 5] = math.nan
        wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q, k2, v, cu, cu, 0.1, out)
        wd.wd_check()
        assert out[:150].isnan().all() and torch.equal(out[150:], clean[150:])


def test_attention_packed_score_jumps(wd):
    """Scores that rise by more than the reference's threshold from key block to key
    block, so that O is rescaled again and again."""
    g = gen(8)
    q, k, v = (normal(g, (700, 128), torch.bfloat16) for _ in range(3))
    k = (k.float() * (1 + torch.arange(700, device="cuda")[:, None] // 128 * 3)).bfloat16()
    out = torch.empty_like(q)
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q, k, v, ints([0, 700]), ints([0, 700]), 0.2, out)
    wd.wd_check()
    want, ab = attention64(q, k, v, [0, 700], [0, 700], 1, 1, 128, 0.2)
    assert_within(out, want, attention_bound(want, ab, torch.bfloat16, 700, v))


def test_attention_packed_many_sequences_and_fused_strides(wd):
    """More sequences than a warp scans at once, q, k, v as columns of one buffer."""
    g = gen(9)
    lens = [int(x) for x in torch.randint(0, 40, (75,), generator=torch.Generator().manual_seed(1))] + [513]
    cu = offsets(lens)
    n, H, dh = cu[-1], 3, 64
    qkv = normal(g, (n, 3 * H * dh + 8), torch.bfloat16)
    q, k, v = (qkv[:, i * H * dh:(i + 1) * H * dh] for i in range(3))
    wide = torch.zeros((n, H * dh + 16), dtype=torch.bfloat16, device="cuda")
    wd.wd_attention_packed(wd.WD_BF16, H, H, dh, q, k, v, ints(cu), ints(cu), 0.125, wide[:, :H * dh])
    wd.wd_check()
    want, ab = attention64(q, k, v, cu, cu, H, H, dh, 0.125)
    assert_within(wide[:, :H * dh], want, attention_bound(want, ab, torch.bfloat16, 513, v))
    assert (wide[:, H * dh:] == 0).all()


def test_attention_packed_bad_offsets_stay_inside(wd):
    """Offsets outside the buffers count as their ends; the rows behind stay untouched."""
    g = gen(10)
    q, k, v = (normal(g, (200, 128), torch.bfloat16) for _ in range(3))
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q, k, v, ints([-5, 100, 100000]), ints([-9, 100, 1 << 30]), 0.1, out)
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q, k, v, ints([0, 100, 200]), ints([0, 100, 200]), 0.1, want)
    wd.wd_check()
    assert torch.equal(out, want)


# ------------------------------------------------------------------ rotary positions
def rope64(x, pos, gain, dh, sec, theta, step, eps):
    x = x.double()
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()
    ang = []
    for a in range(3):
        for p in range(sec[a] // 2):
            ang.append(pos[:, a].double() * (step[a] * theta ** (-2.0 * p / sec[a])))
    ang = torch.stack(ang, 1)[:, None]
    z = x.view(x.shape[0], -1, dh // 2, 2)
    re, im, c, s = z[..., 0], z[..., 1], ang.cos(), ang.sin()
    out = torch.stack((re * c - im * s, re * s + im * c), -1).view(x.shape)
    size = (re.abs() + im.abs())[..., None].expand(z.shape).reshape(x.shape)
    return out, size


@pytest.mark.parametrize("td", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("rows,H,Hk,dh,sec", [(1, 2, 2, 128, (44, 42, 42)), (105, 2, 1, 128, (44, 42, 42)), (37, 16, 4, 128, (64, 64, 0)),
                                              (9, 4, 4, 32, (12, 10, 10)), (10, 5, 3, 40, (0, 0, 40)), (7, 40, 40, 128, (44, 42, 42)),
                                              (5, 3, 32, 256, (84, 86, 86)), (3, 1, 1, 8, (4, 2, 2)), (2500, 12, 12, 64, (24, 20, 20))])
@pytest.mark.parametrize("norm", [True, False])
def test_qknorm_rope_axes(wd, td, rows, H, Hk, dh, sec, norm):
    g = gen(rows + dh)
    q, k = normal(g, (rows, H * dh), td, 1.7), normal(g, (rows, Hk * dh), td, 1.7)
    gq = 1 + normal(g, (H * dh,), std=0.1) if norm else None
    gk = 1 + normal(g, (Hk * dh,), std=0.1)          # k normed either way: the tensors are independent
    pos = torch.randint(-3000, 1 << 20, (rows, 3), generator=g, device="cuda").int()
    pos[0] = 0
    theta, step = 10000.0, (1.0, 0.5, 2.0)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    wd.wd_qknorm_rope_axes({torch.bfloat16: wd.WD_BF16, torch.float16: wd.WD_F16, torch.float32: wd.WD_F32}[td], dh,
                           wd.wd_rope_axes.of(sec, theta, step), pos, q, gq, qo, k, gk, ko, 1e-6)
    wd.wd_check()
    for x, gain, out in ((q, gq, qo), (k, gk, ko)):
        want, size = rope64(x, pos, gain, dh, sec, theta, step, 1e-6)
        assert_within(out, want, 64 * U * size + HALF[td] * want.abs() + 2.0 ** -25)
        if gain is None:
            assert torch.equal(out[0], x[0])         # position zero turns nothing


def test_rope_far_positions_and_extremes(wd):
    """Positions over all of int32: the angle's fraction of a turn stays exact."""
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 123456789], [-1, 1, -2 ** 30]], dtype=torch.int32, device="cuda")
    q = normal(gen(1), (2, 256))
    out = torch.empty_like(q)
    wd.wd_qknorm_rope_axes(wd.WD_F32, 128, wd.wd_rope_axes.of((44, 42, 42)), pos, q, None, out)
    wd.wd_check()
    # the 64-bit reference itself loses |pos| 2^-53 of a radian: 2.4e-7 at 2^31
    want, size = rope64(q, pos, None, 128, (44, 42, 42), 10000.0, (1, 1, 1), 1e-6)
    assert_within(out, want, (64 * U + 2.0 ** -21) * size)


def test_rope_in_place_and_strided(wd):
    g = gen(2)
    qkv = normal(g, (77, 3 * 256 + 8), torch.bfloat16)
    pos = torch.randint(0, 100, (77, 3), generator=g, device="cuda").int()
    gq, gk = (1 + normal(g, (256,), std=0.1) for _ in range(2))
    ax = wd.wd_rope_axes.of((44, 42, 42))
    q, k = qkv[:, :256], qkv[:, 256:512]
    qo, ko = torch.empty((77, 256), dtype=torch.bfloat16, device="cuda"), torch.empty((77, 264), dtype=torch.bfloat16, device="cuda")
    wd.wd_qknorm_rope_axes(wd.WD_BF16, 128, ax, pos, q, gq, qo, k, gk, ko[:, :256])
    rest = qkv[:, 512:].clone()
    wd.wd_qknorm_rope_axes(wd.WD_BF16, 128, ax, pos, q, gq, q, k, gk, k)
    wd.wd_check()
    assert torch.equal(q, qo) and torch.equal(k, ko[:, :256]) and torch.equal(qkv[:, 512:], rest)


def test_rope_axes_agrees_with_the_block(wd):
    """wd_block_qkv's own QK-norm + RoPE on one grid equals this operator on the grid's positions
    (both round one bf16 value whose fp32 forms differ by a few ulp)."""
    from flow_matching_video_b200 import synth
    d = synth.SMALL_BF16.dims
    cd = wd.make_dims(d)
    g = gen(3)
    D, L = d.D, d.L
    w = {n: normal(g, s, t, 0.05) for n, s, t in (("qkv_w", (3 * D, D), torch.bfloat16), ("qkv_b", (3 * D,), torch.float32),
                                                  ("g_q", (D,), torch.float32), ("g_k", (D,), torch.float32), ("mod", (6, D), torch.float32))}
    w["g_q"] += 1
    w["g_k"] += 1
    bw = wd.wd_block_weights(**{k: v.data_ptr() for k, v in w.items()})
    X, e0 = normal(g, (1, L, D)), normal(g, (6, D), std=0.1)
    ws = torch.empty(wd.wd_workspace_bytes(cd, 1), dtype=torch.uint8, device="cuda")
    qkv = torch.empty((L, 3 * D), dtype=torch.bfloat16, device="cuda")
    wd.wd_block_qkv(cd, bw, e0, 1, 0, L, X, qkv, ws)
    s = X[0].double()
    h = (s - s.mean(-1, keepdim=True)) / torch.sqrt(s.var(-1, unbiased=False, keepdim=True) + d.eps)
    h = (h * (1 + e0[1].double() + w["mod"][1].double()) + e0[0].double() + w["mod"][0].double()).to(torch.bfloat16)
    raw = torch.empty_like(qkv)
    wd.wd_gemm(wd.WD_BF16, L, 3 * D, D, h.contiguous(), w["qkv_w"], w["qkv_b"], wd.EPI_STORE, raw)
    t = torch.arange(L, device="cuda")
    Hp, Wp = d.H // 2, d.W // 2
    pos = torch.stack((t // (Hp * Wp), t // Wp % Hp, t % Wp), 1).int()
    wd.wd_qknorm_rope_axes(wd.WD_BF16, 128, wd.wd_rope_axes.of((44, 42, 42)), pos, raw[:, :D], w["g_q"], raw[:, :D],
                           raw[:, D:2 * D], w["g_k"], raw[:, D:2 * D], d.eps)
    wd.wd_check()
    # h may round to the neighbouring bf16 on one side: 2^-8 of a few of its D elements moves q by less
    # than 2^-8 of its norm; both stores add 2^-8
    err = (raw.double() - qkv.double()).abs()
    assert (err <= 2.0 ** -7 * qkv.double().abs() + 2.0 ** -7).all()


# ------------------------------------------------------------------ residual addition + norm
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def norm64(x, y, gain, beta, rms, eps):
    s = x.double() + (0 if y is None else y.double())
    d = s if rms else s - s.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    g = torch.ones(1, device="cuda", dtype=torch.float64) if gain is None else gain.double()
    b = torch.zeros(1, device="cuda", dtype=torch.float64) if beta is None else beta.double()
    return s, d * rstd * g + b, 64 * U * (rstd * g.abs() * (s.abs() + (0 if rms else s.abs().mean(-1, keepdim=True))) + b.abs())


@pytest.mark.parametrize("rows,D", [(1, 8), (3, 128), (17, 1536), (9, 2048), (5, 2056), (6, 4096), (2, 8192), (1000, 264)])
@pytest.mark.parametrize("x,y,out", [("f32", "bf16", "e4m3"), ("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("bf16", "f32", "e4m3"),
                                     ("f32", None, "bf16"), ("bf16", None, "f32")])
@pytest.mark.parametrize("rms", [True, False])
def test_add_norm(wd, rows, D, x, y, out, rms):
    g = gen(rows + D)
    X = normal(g, (rows, D), TYPES[x]) + (0 if rms else 3)
    Y = normal(g, (rows, D), TYPES[y], 0.3) if y else None
    if rows > 2:
        X[1] = 0
        if Y is not None:
            Y[1] = 0          # a row of zeros: zeros, scale 1
    gain = 1 + normal(g, (D,), std=0.1)
    beta = None if rms else normal(g, (D,), std=0.1)
    code = {"f32": wd.WD_F32, "bf16": wd.WD_BF16, "e4m3": wd.WD_E4M3, None: wd.WD_F32}
    S = torch.empty_like(X)
    O = torch.empty((rows, D), dtype=torch.uint8 if out == "e4m3" else TYPES[out], device="cuda")
    sc = torch.empty(rows, device="cuda")
    nk = wd.WD_NORM_RMS if rms else wd.WD_NORM_LAYER
    wd.wd_add_norm(code[x], X, code[y], Y, nk, gain, beta, 1e-6, S, code[out], O, sc if out == "e4m3" else None)
    wd.wd_check()
    s, n, bound = norm64(X, Y, gain, beta, rms, 1e-6)
    assert_within(S, s, (HALF[TYPES[x]] + U) * s.abs())
    if out != "e4m3":
        assert_within(O, n, bound + HALF[TYPES[out]] * n.abs() * (1 + U))
        return
    amax = n.abs().amax(-1)
    want = torch.where(amax > 0, amax / 448, 1.0)
    assert_within(sc, want, bound.amax(-1) / 448 + 2 * U * want)
    deq = O.view(torch.float8_e4m3fn).double() * sc.double()[:, None]
    assert_within(deq, n, 1.01 * bound + (2.0 ** -4 * n.abs() + 2.0 ** -10 * sc.double()[:, None]) * (1 + 2.0 ** -10))
    # the codes and scales are wd_quant_rows_e4m3's of the same norm in fp32
    N32 = torch.empty((rows, D), device="cuda")
    wd.wd_add_norm(code[x], X, code[y], Y, nk, gain, beta, 1e-6, None, wd.WD_F32, N32)
    q2, s2 = torch.empty_like(O), torch.empty_like(sc)
    wd.wd_quant_rows_e4m3(wd.WD_F32, rows, D, N32, q2, s2)
    wd.wd_check()
    assert torch.equal(q2, O) and torch.equal(s2, sc)


def test_add_norm_in_place_and_without_gain(wd):
    g = gen(4)
    X, Y = normal(g, (50, 1536)), normal(g, (50, 1536), torch.bfloat16)
    want_s, want_n, bound = norm64(X, Y, None, None, True, 1e-6)
    O = torch.empty((50, 1536), device="cuda")
    wd.wd_add_norm(wd.WD_F32, X, wd.WD_BF16, Y, wd.WD_NORM_RMS, None, None, 1e-6, X, wd.WD_F32, O)
    wd.wd_check()
    assert_within(X, want_s, 2 * U * want_s.abs())
    assert_within(O, want_n, bound + U * want_n.abs())


def test_add_norm_nan_and_inf_stay_in_their_rows(wd):
    X = normal(gen(5), (20, 256))
    X[3, 7], X[5, 0] = math.nan, math.inf
    O, sc = torch.empty((20, 256), dtype=torch.uint8, device="cuda"), torch.empty(20, device="cuda")
    wd.wd_add_norm(wd.WD_F32, X, wd.WD_F32, None, wd.WD_NORM_RMS, None, None, 1e-6, None, wd.WD_E4M3, O, sc)
    wd.wd_check()
    v = O.view(torch.float8_e4m3fn).float()
    assert v[3].isnan().all() and v[5, 0].isnan()
    ok = [i for i in range(20) if i not in (3, 5)]
    assert torch.isfinite(v[ok]).all() and torch.isfinite(sc[ok]).all()


# ------------------------------------------------------------------ low-rank adapters
def lora64(A, W, bias, seg, ids, down, up, scale, parts):
    A, W, bias = A.double(), W.double(), bias.double()
    K, r = A.shape[1], down.shape[1]
    v = A @ W.t() + bias
    err = 2 * K * U * (A.abs() @ W.abs().t() + bias.abs())
    for a, b, i in zip(seg, seg[1:], ids):
        if 0 <= i < down.shape[0] and a < b:
            D, Up, s = down[i].double(), up[i].double(), (1.0 if scale is None else float(scale[i]))
            T = s * (A[a:b] @ D.t())
            Tb = abs(s) * (A[a:b].abs() @ D.abs().t())
            rnd = 2.0 ** -8 if parts == 1 else 2.0 ** -24
            v[a:b] += T @ Up.t()
            err[a:b] += (2 * K * U * Tb + rnd * T.abs() + 2 * (K + parts * r) * U * T.abs()) @ Up.abs().t()
    return v, err


def run_lora(wd, lens, ids, M, N, K, rank, na, epi, seed=0, start=0, scaled=True):
    g = gen(seed + M + N + K + rank)
    seg = offsets(lens, start)
    A, W, bias = normal(g, (M, K), torch.bfloat16), normal(g, (N, K), torch.bfloat16, 0.05), normal(g, (N,), std=0.1)
    down, up = normal(g, (na, rank, K), torch.bfloat16, K ** -0.5), normal(g, (na, N, rank), torch.bfloat16, 0.3)
    scale = torch.rand(na, generator=g, device="cuda") + 0.5 if scaled else None
    fp32 = epi in (wd.EPI_F32, wd.EPI_RESID)
    v, err = lora64(A, W, bias, seg, ids, down, up, scale, 3 if fp32 else 1)
    ga = normal(g, (N,)) if epi == wd.EPI_RESID else None
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
    lora = wd.wd_lora.of(ints(seg), ints(ids), down, up, scale)
    ws = torch.empty(wd.wd_gemm_lora_bytes(M, len(ids), rank), dtype=torch.uint8, device="cuda").fill_(255)   # NaN everywhere
    wd.wd_gemm_lora(M, N, K, A, W, bias, lora, epi, out, ws, gate_a=ga)
    wd.wd_check()
    assert_within(out, want, bound)
    return out


LORA_SEGS = [([1], [0], 1), ([128, 128], [1, 0], 256), ([5, 0, 120, 3, 200, 1], [0, 1, -1, 1, 0, 7], 400), ([300], [-1], 300),
             ([1] * 40, [i % 3 - 1 for i in range(40)], 77), ([130, 126, 2], [1, 1, 0], 300)]


@pytest.mark.parametrize("lens,ids,M", LORA_SEGS, ids=lambda a: str(a)[:24])
@pytest.mark.parametrize("N,K,rank", [(64, 72, 8), (192, 136, 16), (256, 1536, 64), (1536, 264, 72), (128, 64, 256)])
def test_gemm_lora_store(wd, lens, ids, M, N, K, rank):
    run_lora(wd, lens, ids, M, N, K, rank, 2, wd.EPI_STORE)


@pytest.mark.parametrize("epi", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("N", [64, 128, 256])
def test_gemm_lora_epilogues(wd, epi, N):
    run_lora(wd, [100, 57, 300], [2, 0, 1], 500, N, 520, 40, 3, epi, start=11)
    run_lora(wd, [100, 57, 300], [2, 0, 1], 500, N, 520, 128, 3, epi, scaled=False)


def test_gemm_lora_without_adapters_is_the_gemm(wd):
    g = gen(12)
    A, W = normal(g, (300, 256), torch.bfloat16), normal(g, (256, 256), torch.bfloat16, 0.1)
    out, ref = torch.empty((300, 256), device="cuda"), torch.empty((300, 256), device="cuda")
    down, up = normal(g, (1, 16, 256), torch.bfloat16), normal(g, (1, 256, 16), torch.bfloat16)
    lora = wd.wd_lora.of(ints([0, 100, 300]), ints([-1, 5]), down, up)
    ws = torch.empty(wd.wd_gemm_lora_bytes(300, 2, 16), dtype=torch.uint8, device="cuda")
    wd.wd_gemm_lora(300, 256, 256, A, W, None, lora, wd.EPI_F32, out, ws)
    wd.wd_gemm(wd.WD_BF16, 300, 256, 256, A, W, None, wd.EPI_F32, ref)
    wd.wd_check()
    # the same product; its accumulation is rounded where wd_gemm's is truncated
    exact = A.double() @ W.double().t()
    assert_within(out, exact, 2 * 256 * U * (A.double().abs() @ W.double().abs().t()))
    assert (out.double() - exact).abs().mean() <= (ref.double() - exact).abs().mean()
    half, half_ref = torch.empty((300, 256), dtype=torch.bfloat16, device="cuda"), torch.empty((300, 256), dtype=torch.bfloat16, device="cuda")
    wd.wd_gemm_lora(300, 256, 256, A, W, None, lora, wd.EPI_STORE, half, ws)
    wd.wd_gemm(wd.WD_BF16, 300, 256, 256, A, W, None, wd.EPI_STORE, half_ref)
    wd.wd_check()
    assert torch.equal(half, half_ref)


def test_gemm_lora_long_sums_are_rounded(wd):
    """fp32 outputs over a long K: 3e-6 of the result at most (measured 1e-6; the tensor cores'
    truncation alone would take 8e-6 at this K, all of one sign)."""
    g = gen(14)
    M, N, K, r = 300, 256, 8960, 16
    A, W = normal(g, (M, K), torch.bfloat16), normal(g, (N, K), torch.bfloat16, 0.02)
    down, up = normal(g, (1, r, K), torch.bfloat16, K ** -0.5), normal(g, (1, N, r), torch.bfloat16, 0.1)
    out = torch.empty((M, N), device="cuda")
    ws = torch.empty(wd.wd_gemm_lora_bytes(M, 1, r), dtype=torch.uint8, device="cuda")
    wd.wd_gemm_lora(M, N, K, A, W, None, wd.wd_lora.of(ints([0, M]), ints([0]), down, up), wd.EPI_F32, out, ws)
    wd.wd_check()
    want, _ = lora64(A, W, torch.zeros(N, device="cuda"), [0, M], [0], down, up, None, 3)
    assert float(((out.double() - want).pow(2).mean() / want.pow(2).mean()).sqrt()) <= 3e-6


@pytest.mark.parametrize("what", ["row", "down", "scale"])
def test_gemm_lora_nan_stays_in_its_request(wd, what):
    """Requests that share a 128-row tile: a NaN in one's rows, down-projection or scale does
    not reach the others' rows."""
    g = gen(13)
    M, N, K, r = 300, 128, 128, 24
    seg, ids = [0, 40, 41, 170, 300], [0, 1, 2, 0]
    A, W = normal(g, (M, K), torch.bfloat16), normal(g, (N, K), torch.bfloat16, 0.1)
    down, up = normal(g, (3, r, K), torch.bfloat16, K ** -0.5), normal(g, (3, N, r), torch.bfloat16)
    scale = torch.ones(3, device="cuda")
    ws = torch.empty(wd.wd_gemm_lora_bytes(M, 4, r), dtype=torch.uint8, device="cuda").fill_(255)
    outs = []
    for bad in (False, True):
        if bad:
            if what == "row":
                A[100, 3] = math.nan
            else:
                {"down": down, "scale": scale}[what][2] = math.nan
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        wd.wd_gemm_lora(M, N, K, A, W, None, wd.wd_lora.of(ints(seg), ints(ids), down, up, scale), wd.EPI_STORE, out, ws)
        wd.wd_check()
        outs.append(out)
    hit = torch.zeros(M, dtype=torch.bool, device="cuda")
    hit[100 if what == "row" else slice(41, 170)] = True
    assert torch.equal(outs[0][~hit], outs[1][~hit]) and not torch.isfinite(outs[1][hit]).all(1).any()


# ------------------------------------------------------------------ together, as a packed batch runs them
class Batch:
    """Half a block on a packed batch of videos with adapters of their own: the branch before
    it added and normed, q|k|v with adapters, QK-norm + rotary positions in place, attention,
    the output projection with adapters added into the residual stream, and the next norm
    in 8 bits with the FP8 GEMM on it."""

    def __init__(self, wd, lens, ids, seed, H=2, rank=16, spare=5):
        self.wd, self.lens, self.ids, self.H, self.rank = wd, lens, ids, H, rank
        g = gen(seed)
        D = self.D = H * 128
        n = self.n = sum(lens) + spare
        self.X, self.y = normal(g, (n, D)), normal(g, (n, D), torch.bfloat16)
        self.g1, self.g2 = 1 + normal(g, (D,), std=0.1), 1 + normal(g, (D,), std=0.1)
        self.Wqkv, self.bqkv = normal(g, (3 * D, D), torch.bfloat16, D ** -0.5), normal(g, (3 * D,), std=0.1)
        self.Wo, self.bo, self.gate = normal(g, (D, D), torch.bfloat16, D ** -0.5), normal(g, (D,), std=0.1), normal(g, (D,))
        self.gq, self.gk = 1 + normal(g, (D,), std=0.1), 1 + normal(g, (D,), std=0.1)
        na = 2
        self.dq, self.uq = normal(g, (na, rank, D), torch.bfloat16, D ** -0.5), normal(g, (na, 3 * D, rank), torch.bfloat16, 0.1)
        self.do, self.uo = normal(g, (na, rank, D), torch.bfloat16, D ** -0.5), normal(g, (na, D, rank), torch.bfloat16, 0.1)
        self.scale = torch.rand(na, generator=g, device="cuda") + 0.5
        self.pos = torch.randint(0, 60, (n, 3), generator=g, device="cuda").int()
        self.cu, self.adapter = ints(offsets(lens)), ints(ids)
        self.W8, self.s8 = torch.empty((256, D), dtype=torch.uint8, device="cuda"), torch.empty(256, device="cuda")
        wd.wd_quant_rows_e4m3(wd.WD_BF16, 256, D, normal(g, (256, D), torch.bfloat16), self.W8, self.s8)
        e = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
        self.h, self.qkv, self.o, self.res = e(n, D), e(n, 3 * D), e(n, D), e(n, D, t=torch.float32)
        self.h8, self.hs, self.out = e(n, D, t=torch.uint8), e(n, t=torch.float32), e(n, 256, t=torch.float32)
        self.ws = torch.empty(wd.wd_gemm_lora_bytes(n, len(ids), rank), dtype=torch.uint8, device="cuda")
        self.lq = wd.wd_lora.of(self.cu, self.adapter, self.dq, self.uq, self.scale)
        self.lo = wd.wd_lora.of(self.cu, self.adapter, self.do, self.uo, self.scale)
        self.axes = wd.wd_rope_axes.of((44, 42, 42))

    def run(self, stream=None):
        wd, n, D, H = self.wd, self.n, self.D, self.H
        wd.wd_add_norm(wd.WD_F32, self.X, wd.WD_BF16, self.y, wd.WD_NORM_RMS, self.g1, None, 1e-6, self.res, wd.WD_BF16,
                       self.h, stream=stream)
        wd.wd_gemm_lora(n, 3 * D, D, self.h, self.Wqkv, self.bqkv, self.lq, wd.EPI_STORE, self.qkv, self.ws, stream=stream)
        q, k, v = (self.qkv[:, i * D:(i + 1) * D] for i in range(3))
        wd.wd_qknorm_rope_axes(wd.WD_BF16, 128, self.axes, self.pos, q, self.gq, q, k, self.gk, k, stream=stream)
        wd.wd_attention_packed(wd.WD_BF16, H, H, 128, q, k, v, self.cu, self.cu, 128 ** -0.5, self.o, stream=stream)
        wd.wd_gemm_lora(n, D, D, self.o, self.Wo, self.bo, self.lo, wd.EPI_RESID, self.res, self.ws, gate_a=self.gate,
                        stream=stream)
        wd.wd_add_norm(wd.WD_F32, self.res, wd.WD_F32, None, wd.WD_NORM_RMS, self.g2, None, 1e-6, None, wd.WD_E4M3, self.h8,
                       self.hs, stream=stream)
        wd.wd_gemm_fp8(n, 256, D, self.h8, self.hs, self.W8, self.s8, None, wd.EPI_F32, self.out, stream=stream)
        return self.res.clone(), self.out.clone()

    def exact(self):
        """The same in 64 bits, rounded to bf16 where the operators store bf16."""
        bf = lambda t: t.float().bfloat16().double()
        cu, D = offsets(self.lens), self.D
        s, h, _ = norm64(self.X, self.y, self.g1, None, True, 1e-6)
        qkv, _ = lora64(bf(h), self.Wqkv, self.bqkv, cu, self.ids, self.dq, self.uq, self.scale, 1)
        q, k, v = (bf(qkv[:, i * D:(i + 1) * D]) for i in range(3))
        q, k = (bf(rope64(x, self.pos, gn, 128, (44, 42, 42), 10000.0, (1, 1, 1), 1e-6)[0]) for x, gn in ((q, self.gq), (k, self.gk)))
        o, _ = attention64(q, k, v, cu, cu, self.H, self.H, 128, 128 ** -0.5)
        p, _ = lora64(bf(o), self.Wo, self.bo, cu, self.ids, self.do, self.uo, self.scale, 3)
        return s + self.gate.double() * p


BATCH = ([300, 1, 0, 130, 77], [1, 0, 1, -1, 0])


def test_packed_half_block(wd):
    b = Batch(wd, *BATCH, seed=1)
    res, out = b.run()
    wd.wd_check()
    want = b.exact()
    # the bar of the bf16 path: 2e-2 of the output's RMS
    assert float((res.double() - want).abs().max() / want.pow(2).mean().sqrt()) <= 2e-2
    # the FP8 GEMM reads the norm's codes and scales
    a = b.h8.view(torch.float8_e4m3fn).double() * b.hs.double()[:, None]
    w = b.W8.view(torch.float8_e4m3fn).double() * b.s8.double()[:, None]
    assert_within(out, a @ w.t(), 2 * b.D * U * (a.abs() @ w.abs().t()) + 3 * U * (a @ w.t()).abs())
    _, n, bound = norm64(res, None, b.g2, None, True, 1e-6)
    assert_within(a, n, 1.01 * bound + (2.0 ** -4 * n.abs() + 2.0 ** -10 * b.hs.double()[:, None]) * (1 + 2.0 ** -10))
    again, out2 = b.run()
    assert torch.equal(again, res) and torch.equal(out2, out)       # no order of sums varies


def test_packed_half_block_captured_and_replayed(wd):
    """Captured into a CUDA graph, and replayed on inputs, offsets, adapters and positions
    that were rewritten in place; two graphs alive at once, each with its own workspace."""
    a, b = Batch(wd, *BATCH, seed=2), Batch(wd, [9, 200, 150, 149, 0], [0, -1, 1, 0, 0], seed=3)
    graphs = []
    for x in (a, b):
        x.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = x.run()
        graphs.append((graph, outs))
    other = Batch(wd, [150, 208, 1, 100, 49], [0, 1, 1, 0, -1], seed=4)
    assert other.n == a.n
    for name in ("X", "y", "cu", "adapter", "pos", "Wqkv", "uq"):
        getattr(a, name).copy_(getattr(other, name))
    for name in ("g1", "g2", "bqkv", "Wo", "bo", "gate", "gq", "gk", "dq", "do", "uo", "scale", "W8", "s8"):
        getattr(other, name).copy_(getattr(a, name))
    graphs[1][0].replay()
    graphs[0][0].replay()
    wd.wd_check()
    for (_, outs), eager in zip(graphs, (other, b)):
        for got, want in zip(outs, eager.run()):
            assert torch.equal(got, want)


def test_packed_half_blocks_on_two_streams(wd):
    bs = [Batch(wd, *BATCH, seed=5), Batch(wd, [508], [1], seed=6)]
    want = [b.run() for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(5):
        got = []
        for b, s in zip(bs, streams):
            with torch.cuda.stream(s):
                got.append(b.run())
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    # a stream handed over by the caller, while another one is current
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bs[0].run(stream=s)
    s.synchronize()
    assert torch.equal(bs[0].res, want[0][0])


# ------------------------------------------------------------------ far ends
def test_attention_packed_thousands_of_sequences(wd):
    """Sequences of 0 to 3 rows, more than any group of the scan, and the rows behind them."""
    g = gen(20)
    lens = torch.randint(0, 4, (3000,), generator=torch.Generator().manual_seed(2)).tolist()
    cu = offsets(lens)
    n = cu[-1]
    q, k, v = (normal(g, (n + 7, 128), torch.bfloat16) for _ in range(3))
    out = torch.full((n + 7, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    wd.wd_attention_packed(wd.WD_BF16, 2, 2, 64, q, k, v, ints(cu), ints(cu), 0.125, out)
    wd.wd_check()
    owner = torch.repeat_interleave(torch.arange(3000), torch.tensor(lens)).cuda()
    t = torch.einsum("ihd,jhd->hij", q[:n].double().view(n, 2, 64), k[:n].double().view(n, 2, 64)) * 0.125
    p = torch.softmax(t.masked_fill(owner[None, :, None] != owner[None, None, :], -math.inf), -1)
    vv = v[:n].double().view(n, 2, 64)
    want, ab = (torch.einsum("hij,jhd->ihd", p, x).reshape(n, 128) for x in (vv, vv.abs()))
    assert_within(out[:n], want, attention_bound(want, ab, torch.bfloat16, 3, v))
    assert (out[n:] == 7.0).all()


def test_attention_packed_no_rows_at_all(wd):
    q = torch.randn((300, 128), device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    zero, cu = ints([0, 0, 0]), ints([0, 100, 300])
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q, q, q, zero, cu, 0.1, out)
    wd.wd_check()
    assert (out == 7.0).all()
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 128, q, q, q, cu, zero, 0.1, out)
    wd.wd_check()
    assert (out == 0).all()


def test_many_single_row_requests(wd):
    run_lora(wd, [1] * 700, [i % 5 - 1 for i in range(700)], 705, 128, 128, 8, 4, wd.EPI_STORE)
    run_lora(wd, [0, 0, 3, 0, 0, 200, 0], [0, 1, 1, 0, 0, 1, 0], 203, 64, 64, 8, 2, wd.EPI_F32)


def test_offsets_past_32_bits(wd):
    """Buffers of more than 2^32 bytes: the rows at their far ends."""
    g = gen(21)
    rows, stride = 1_100_000, 2048                      # 2.25e9 elements
    big = torch.zeros((rows, stride), dtype=torch.bfloat16, device="cuda")
    q, k, v = (big[:, i * 256:(i + 1) * 256] for i in range(3))
    n = 300
    for t in (q, k, v):
        t[-n - 10:-10] = normal(g, (n, 256), torch.bfloat16)
    o = big[:, 1024:1280]
    cu = ints([rows - n - 10, rows - 10])
    wd.wd_attention_packed(wd.WD_BF16, 2, 2, 128, q, k, v, cu, cu, 0.1, o)
    wd.wd_check()
    want, ab = attention64(*(t[-n - 10:-10] for t in (q, k, v)), [0, n], [0, n], 2, 2, 128, 0.1)
    assert_within(o[-n - 10:-10], want, attention_bound(want, ab, torch.bfloat16, n, v[-n - 10:-10]))
    assert (o[-10:] == 0).all() and (o[:1000] == 0).all()
    pos = torch.randint(0, 100, (rows, 3), generator=g, device="cuda").int()
    r = big[:, 1280:1536]
    wd.wd_qknorm_rope_axes(wd.WD_BF16, 128, wd.wd_rope_axes.of((44, 42, 42)), pos, q, None, r)
    wd.wd_check()
    want, size = rope64(q[-n:], pos[-n:], None, 128, (44, 42, 42), 10000.0, (1, 1, 1), 1e-6)
    assert_within(r[-n:], want, 64 * U * size + 2.0 ** -8 * want.abs() + 2.0 ** -25)
    del big, q, k, v, o, r
    x = torch.zeros((540_000, 4096), dtype=torch.bfloat16, device="cuda")
    x[-5:] = normal(g, (5, 4096), torch.bfloat16)
    out = torch.empty_like(x)
    wd.wd_add_norm(wd.WD_BF16, x, wd.WD_BF16, None, wd.WD_NORM_RMS, None, None, 1e-6, None, wd.WD_BF16, out)
    wd.wd_check()
    _, want, bound = norm64(x[-5:], None, None, None, True, 1e-6)
    assert_within(out[-5:], want, bound + 2.0 ** -8 * want.abs() * (1 + U))
    del x, out
    M, N, K, r = 1_060_000, 2048, 64, 8                  # 2.17e9 outputs
    A, W = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), normal(g, (N, K), torch.bfloat16)
    A[-200:] = normal(g, (200, K), torch.bfloat16)
    down, up = normal(g, (2, r, K), torch.bfloat16, 0.1), normal(g, (2, N, r), torch.bfloat16)
    seg, ids = [0, M - 150, M - 20], [0, 1]
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(wd.wd_gemm_lora_bytes(M, 2, r), dtype=torch.uint8, device="cuda")
    wd.wd_gemm_lora(M, N, K, A, W, None, wd.wd_lora.of(ints(seg), ints(ids), down, up), wd.EPI_STORE, out, ws)
    wd.wd_check()
    v, err = lora64(A[-200:], W, torch.zeros(N, device="cuda"), [0, 50, 180], ids, down, up, None, 1)
    assert_within(out[-200:], v, err * (1 + 2.0 ** -8) + 2.0 ** -8 * v.abs())


@pytest.mark.parametrize("epi", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("M,N,K,rank", [(20000, 256, 136, 16), (19001, 512, 1536, 40), (30000, 256, 64, 136)])
def test_gemm_lora_sm_pairs(wd, epi, M, N, K, rank):
    """Shapes that run on SM pairs (256 x 256 tiles): requests that end inside either half
    of a tile, lie in one half only, or cover several tiles; rows of none at both ends."""
    lens = [1, 127, 128, 200, 3, 0, 56, 600, 5000, 130, 126, 1, 9000]
    run_lora(wd, lens, [0, 1, 2, -1, 1, 0, 2, 0, 1, 2, 0, 1, 0], M, N, K, rank, 3, epi, start=70)


def test_attention_packed_mostly_spare_rows(wd):
    """A large buffer with few rows in use: most blocks of the grid find nothing."""
    g = gen(22)
    q = torch.zeros((3_000_000, 64), dtype=torch.bfloat16, device="cuda")
    q[500:900] = normal(g, (400, 64), torch.bfloat16)
    out = torch.full_like(q, 7.0)
    cu = ints([500, 600, 600, 900])
    wd.wd_attention_packed(wd.WD_BF16, 1, 1, 64, q, q, q, cu, cu, 0.125, out)
    wd.wd_check()
    want, ab = attention64(q[500:900], q[500:900], q[500:900], [0, 100, 100, 400], [0, 100, 100, 400], 1, 1, 64, 0.125)
    assert_within(out[500:900], want, attention_bound(want, ab, torch.bfloat16, 300, q[500:900]))
    assert (out[:500] == 7.0).all() and (out[900:] == 7.0).all()


def test_gemm_lora_long_sums_with_many_rows(wd):
    """The same where the rows alone would not split K: an adapter that outweighs the rest."""
    g = gen(15)
    M, N, K, r = 20000, 256, 8960, 32
    A, W = normal(g, (M, K), torch.bfloat16), normal(g, (N, K), torch.bfloat16, 0.002)
    down, up = normal(g, (1, r, K), torch.bfloat16, K ** -0.5), normal(g, (1, N, r), torch.bfloat16)
    out = torch.empty((M, N), device="cuda")
    ws = torch.empty(wd.wd_gemm_lora_bytes(M, 1, r), dtype=torch.uint8, device="cuda")
    wd.wd_gemm_lora(M, N, K, A, W, None, wd.wd_lora.of(ints([0, M]), ints([0]), down, up), wd.EPI_F32, out, ws)
    wd.wd_check()
    want = A[:2000].double() @ (W.double() + up[0].double() @ down[0].double()).t()
    assert float(((out[:2000].double() - want).pow(2).mean() / want.pow(2).mean()).sqrt()) <= 3e-6
