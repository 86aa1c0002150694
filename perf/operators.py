"""The operators for batches of mixed requests, as cases that can be timed.

Requests of different sizes are served in one call with their rows packed one
request behind the other: the attention over such a packed buffer
(wd_attention_packed), QK-RMSNorm and the rotary positions of (frame, row,
column) per token (wd_qknorm_rope_axes), residual addition + norm with an
8-bit output (wd_add_norm), and the shared projection with each request's own
low-rank adapter (wd_gemm_lora).

`run` computes a case either in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, with `own` set, through the library.
"""
import math

import torch

own = False

# (heads, head width) of the repository's models and of its text features (c_txt = 4096)
VIDEO_HEADS, VIDEO_DH = 12, 128
WIDE_HEADS = 40
TEXT_HEADS, TEXT_DH = 64, 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # two prompts through a text encoder (heads of 64, a learned bias by distance, no 1/sqrt(d))
        dict(name="attn_prompts", op="attention", q="512,77", k="", heads=TEXT_HEADS, kv_heads=TEXT_HEADS, dh=TEXT_DH,
             type="bf16", radius=128, window=False, scale=1.0, pad=0),
        # self-attention of three videos: 17 frames at 480p, a preview, a single frame; buffer with spare rows
        dict(name="attn_videos", op="attention", q="7800,3185,405", k="", heads=VIDEO_HEADS, kv_heads=VIDEO_HEADS,
             dh=VIDEO_DH, type="bf16", radius=0, window=False, scale=128 ** -0.5, pad=130),
        # cross-attention of videos to their prompts at the prompts' own lengths (one of them empty)
        dict(name="attn_cross", op="attention", q="32760,7800,1,3185", k="512,77,9,0", heads=VIDEO_HEADS,
             kv_heads=VIDEO_HEADS, dh=VIDEO_DH, type="f16", radius=0, window=False, scale=128 ** -0.5, pad=0),
        # an 81-frame video next to a 17-frame one: the largest
        dict(name="attn_long", op="attention", q="7800,32760", k="", heads=VIDEO_HEADS, kv_heads=VIDEO_HEADS,
             dh=VIDEO_DH, type="bf16", radius=0, window=False, scale=128 ** -0.5, pad=0),
        # the tokens of one small request
        dict(name="rope_small", op="rope", rows=105, heads=2, kv_heads=2, dh=128, type="bf16", norm=True),
        # all tokens of a conditional / unconditional pair at 480p, 81 frames
        dict(name="rope_pair", op="rope", rows=65520, heads=VIDEO_HEADS, kv_heads=VIDEO_HEADS, dh=128, type="bf16",
             norm=True),
        # the wide model on an odd number of tokens
        dict(name="rope_wide", op="rope", rows=7801, heads=WIDE_HEADS, kv_heads=WIDE_HEADS, dh=128, type="bf16", norm=True),
        # a text encoder's residual stream, one prompt
        dict(name="norm_prompt", op="norm", rows=512, D=4096, x="bf16", y="bf16", norm="rms", out="bf16"),
        # the fp32 residual stream of a packed batch, output in 8 bits for the FP8 GEMMs
        dict(name="norm_videos", op="norm", rows=43745, D=1536, x="f32", y="bf16", norm="rms", out="e4m3"),
        # a few prompts with adapters of their own, one without
        dict(name="lora_prompts", op="lora", segs="512,77,1,301", ids="0,2,-1,1", M=891, N=1536, K=1536, rank=16,
             adapters=3, epilogue="store"),
        # the fused q|k|v projection of a packed batch of videos
        dict(name="lora_videos", op="lora", segs="32760,7800,3185", ids="1,0,3", M=43745, N=4608, K=1536, rank=32,
             adapters=4, epilogue="store"),
        # the feed-forward's second layer of small requests, 32-bit output (added to a residual stream by the caller)
        dict(name="lora_ffn2", op="lora", segs="1950,405,105", ids="0,1,0", M=2500, N=1536, K=8960, rank=64, adapters=2,
             epilogue="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _lengths(rng, n, lo, hi, total):
    out = []
    for _ in range(n):
        left = total - sum(out)
        if left < lo:
            break
        out.append(min(_log(rng, lo, hi), left))
    return out


def _text(a):
    return ",".join(str(x) for x in a)


def draw(rng):
    op = rng.choice(["attention", "attention", "rope", "norm", "lora"])
    if op == "attention":
        kind = rng.choice(["prompts", "videos", "cross", "window"])
        c = dict(op=op, type=rng.choice(["bf16", "f16"]), radius=0, window=False, pad=rng.choice([0, 0, 1, 200]), k="")
        if kind == "prompts":
            h = rng.choice([16, 32, TEXT_HEADS])
            c.update(q=_text(_lengths(rng, _log(rng, 1, 24), 1, 512, 6000)), heads=h, kv_heads=h, dh=TEXT_DH,
                     radius=rng.choice([32, 128, 200]), scale=rng.choice([1.0, 0.125]))
        elif kind == "cross":
            n = _log(rng, 1, 12)
            q = _lengths(rng, n, 1, 32760, 45000)
            c.update(q=_text(q), k=_text([rng.choice([0, 1, 512, rng.randint(1, 769)]) if rng.random() < 0.5
                                          else rng.randint(1, 512) for _ in q]),
                     heads=VIDEO_HEADS, kv_heads=rng.choice([VIDEO_HEADS, 4, 1]), dh=VIDEO_DH, scale=128 ** -0.5)
        else:
            h = rng.choice([2, VIDEO_HEADS, 16])
            c.update(q=_text(_lengths(rng, _log(rng, 1, 8), 1, 16000, 24000)), heads=h, kv_heads=rng.choice([h, h // 2]),
                     dh=rng.choice([VIDEO_DH, VIDEO_DH, TEXT_DH]))
            c["scale"] = c["dh"] ** -0.5
            if kind == "window":
                c.update(radius=rng.randint(1, 1024), window=True)
        return c
    if op == "rope":
        h, dh = rng.choice([(2, 128), (VIDEO_HEADS, 128), (16, 128), (WIDE_HEADS, 128), (4, 32), (24, 64), (5, 40)])
        rows = _log(rng, 1, 65520 if h * dh <= 2048 else 16000)
        return dict(op=op, rows=rows, heads=h, kv_heads=rng.choice([h, 1]), dh=dh, type=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    norm=rng.random() < 0.75)
    if op == "norm":
        D = rng.choice([128, 256, 1536, 2048, 4096, 5120, 8 * rng.randint(1, 640)])
        rows = _log(rng, 1, max(1, min(65520, 65520 * 1536 // D)))
        return dict(op=op, rows=rows, D=D, x=rng.choice(["f32", "bf16"]), y=rng.choice(["bf16", "f32"]),
                    norm=rng.choice(["rms", "rms", "layer"]), out=rng.choice(["e4m3", "e4m3", "bf16", "f32"]))
    N, K = rng.choice([(4608, 1536), (1536, 1536), (8960, 1536), (1536, 8960), (256, 256), (4096, 4096), (1536, 4096), (192, 136)])
    segs = _lengths(rng, _log(rng, 1, 32), 1, 16000, 24000)
    adapters = rng.randint(1, 8)
    return dict(op=op, segs=_text(segs), ids=_text([rng.randint(-1, adapters - 1) for _ in segs]),
                M=sum(segs) + rng.choice([0, 0, 1, 100]), N=N, K=K, rank=8 * _log(rng, 1, 16), adapters=adapters,
                epilogue=rng.choice(["store", "store", "gelu", "f32"]))


# ------------------------------------------------------------------ inputs
def _ints(s):
    return [int(x) for x in s.split(",")] if s else []


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _sections(dh):
    """The (frame, row, column) channels of a head."""
    s = 2 * (dh // 6)
    return (dh - 2 * s, s, s)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "attention":
        lq = _ints(case["q"])
        lk = _ints(case["k"]) or lq
        H, Hk, dh, td = case["heads"], case["kv_heads"], case["dh"], TYPES[case["type"]]
        st["cu_q"], st["cu_k"] = _offsets(lq), _offsets(lk)
        nq, nk = st["cu_q"][-1] + case["pad"], max(1, st["cu_k"][-1])
        # logits of unit variance, as QK-normalised heads (or an unscaled text encoder's) have
        std = (case["scale"] * dh ** 0.5) ** -0.5
        st["q"] = _normal(g, (nq, H * dh), td, std)
        st["k"] = _normal(g, (nk, Hk * dh), td, std)
        st["v"] = _normal(g, (nk, Hk * dh), td)
        st["bias"] = None
        if case["radius"]:
            R = case["radius"]
            st["bias"] = torch.randn((H, 2 * R + 1), generator=g, device="cuda")
            if case["window"]:   # keys R or more away are left out
                st["bias"][:, 0] = st["bias"][:, -1] = -math.inf
        st["out"] = torch.zeros((nq, H * dh), dtype=torch.bfloat16, device="cuda")
        st["cu_q_dev"] = torch.tensor(st["cu_q"], dtype=torch.int32, device="cuda")
        st["cu_k_dev"] = torch.tensor(st["cu_k"], dtype=torch.int32, device="cuda")
    elif case["op"] == "rope":
        n, dh, td = case["rows"], case["dh"], TYPES[case["type"]]
        # tokens of 480p grids (30 x 52), frame after frame, somewhere in a long video
        t = torch.arange(n, device="cuda") + int(torch.randint(0, 1 << 20, (), generator=g, device="cuda"))
        st["pos"] = torch.stack((t // 1560, t // 52 % 30, t % 52), 1).to(torch.int32).contiguous()
        for name, h in (("q", case["heads"]), ("k", case["kv_heads"])):
            st[name] = _normal(g, (n, h * dh), td, 1.7)
            st["g_" + name] = 1 + 0.02 * torch.randn(h * dh, generator=g, device="cuda") if case["norm"] else None
            st[name + "_out"] = torch.empty_like(st[name])
    elif case["op"] == "norm":
        n, D = case["rows"], case["D"]
        st["x"] = _normal(g, (n, D), TYPES[case["x"]])
        st["y"] = _normal(g, (n, D), TYPES[case["y"]], 0.3)
        st["gain"] = 1 + 0.02 * torch.randn(D, generator=g, device="cuda")
        st["beta"] = 0.02 * torch.randn(D, generator=g, device="cuda") if case["norm"] == "layer" else None
        st["sum"] = torch.empty_like(st["x"])
        st["out"] = torch.empty((n, D), dtype=torch.uint8 if case["out"] == "e4m3" else TYPES[case["out"]], device="cuda")
        st["row_scale"] = torch.empty(n, device="cuda")
    else:
        M, N, K, r, na = case["M"], case["N"], case["K"], case["rank"], case["adapters"]
        st["seg"], st["ids"] = _offsets(_ints(case["segs"])), _ints(case["ids"])
        st["A"] = _normal(g, (M, K), torch.bfloat16)
        st["W"] = _normal(g, (N, K), torch.bfloat16, 0.02)
        st["bias"] = 0.02 * torch.randn(N, generator=g, device="cuda")
        st["down"] = _normal(g, (na, r, K), torch.bfloat16, K ** -0.5)
        st["up"] = _normal(g, (na, N, r), torch.bfloat16, 0.1)
        st["scale"] = torch.rand(na, generator=g, device="cuda") + 0.5
        st["out"] = torch.empty((M, N), dtype=torch.float32 if case["epilogue"] == "f32" else torch.bfloat16, device="cuda")
        st["seg_dev"] = torch.tensor(st["seg"], dtype=torch.int32, device="cuda")
        st["ids_dev"] = torch.tensor(st["ids"], dtype=torch.int32, device="cuda")
        st["ws"] = None
    if own and case["op"] == "rope":
        from flow_matching_video_b200 import wd
        st["axes"] = wd.wd_rope_axes.of(_sections(case["dh"]))
    if own and case["op"] == "lora":
        from flow_matching_video_b200 import wd
        st["lora"] = wd.wd_lora.of(st["seg_dev"], st["ids_dev"], st["down"], st["up"], st["scale"])
        st["ws"] = torch.empty(wd.wd_gemm_lora_bytes(M, len(st["ids"]), r), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return {"attention": _attention, "rope": _rope, "norm": _norm, "lora": _lora}[state["case"]["op"]](state)


def _attention(st):
    c = st["case"]
    H, Hk, dh = c["heads"], c["kv_heads"], c["dh"]
    if own:
        from flow_matching_video_b200 import wd
        wd.wd_attention_packed(wd.WD_F16 if c["type"] == "f16" else wd.WD_BF16, H, Hk, dh, st["q"], st["k"], st["v"],
                               st["cu_q_dev"], st["cu_k_dev"], c["scale"], st["out"], bias=st["bias"])
        return st["out"]
    out = torch.zeros_like(st["out"])
    for a, b, ka, kb in zip(st["cu_q"], st["cu_q"][1:], st["cu_k"], st["cu_k"][1:]):
        if a == b or ka == kb:
            continue
        per = max(1, (1 << 30) // ((b - a) * (kb - ka)))     # heads at a time: 4 GB of scores at most
        for h0 in range(0, H, per):
            h1 = min(H, h0 + per)
            src = [h * Hk // H for h in range(h0, h1)]
            q = st["q"][a:b].view(b - a, H, dh)[:, h0:h1].permute(1, 0, 2).float()
            k = st["k"][ka:kb].view(kb - ka, Hk, dh)[:, src].permute(1, 2, 0).float()
            v = st["v"][ka:kb].view(kb - ka, Hk, dh)[:, src].permute(1, 0, 2).float()
            s = q @ k * c["scale"]
            if st["bias"] is not None:
                R = c["radius"]
                far = torch.arange(kb - ka, device="cuda")[None, :] - torch.arange(b - a, device="cuda")[:, None]
                s += st["bias"][h0:h1][:, far.clamp(-R, R) + R]
            m = s.amax(-1, keepdim=True)
            s = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
            l = s.sum(-1, keepdim=True)
            o = torch.where(l > 0, s @ v / l, 0.0)
            out[a:b].view(b - a, H, dh)[:, h0:h1] = o.permute(1, 0, 2).to(out.dtype)
    return out


def _rope(st):
    c = st["case"]
    if own:
        from flow_matching_video_b200 import wd
        wd.wd_qknorm_rope_axes({"bf16": wd.WD_BF16, "f16": wd.WD_F16, "f32": wd.WD_F32}[c["type"]], c["dh"], st["axes"],
                               st["pos"], st["q"], st["g_q"], st["q_out"], st["k"], st["g_k"], st["k_out"], 1e-6)
        return st["q_out"], st["k_out"]
    ang = []
    for axis, d in enumerate(_sections(c["dh"])):
        w = 10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
        ang.append(st["pos"][:, axis, None].double() * w)
    ang = torch.cat(ang, 1)
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    outs = []
    for x, gain in ((st["q"], st["g_q"]), (st["k"], st["g_k"])):
        f = x.float()
        if gain is not None:
            f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6) * gain
        f = f.view(c["rows"], -1, c["dh"] // 2, 2)
        re, im = f[..., 0], f[..., 1]
        outs.append(torch.stack((re * cos - im * sin, re * sin + im * cos), -1).view(x.shape).to(x.dtype))
    return tuple(outs)


def _norm(st):
    c = st["case"]
    if own:
        from flow_matching_video_b200 import wd
        t = {"f32": wd.WD_F32, "bf16": wd.WD_BF16, "e4m3": wd.WD_E4M3}
        wd.wd_add_norm(t[c["x"]], st["x"], t[c["y"]], st["y"], wd.WD_NORM_RMS if c["norm"] == "rms" else wd.WD_NORM_LAYER,
                       st["gain"], st["beta"], 1e-6, st["sum"], t[c["out"]], st["out"],
                       st["row_scale"] if c["out"] == "e4m3" else None)
        if c["out"] == "e4m3":
            return st["sum"], st["out"].view(torch.float8_e4m3fn), st["row_scale"]
        return st["sum"], st["out"]
    s = st["x"].float() + st["y"].float()
    n = s - s.mean(-1, keepdim=True) if c["norm"] == "layer" else s
    n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + 1e-6) * st["gain"]
    if st["beta"] is not None:
        n = n + st["beta"]
    if c["out"] != "e4m3":
        return s.to(st["x"].dtype), n.to(st["out"].dtype)
    amax = n.abs().amax(-1)
    sc = torch.where(amax > 0, amax / 448, 1.0)
    return s.to(st["x"].dtype), (n / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), sc


def _lora(st):
    c = st["case"]
    if own:
        from flow_matching_video_b200 import wd
        epi = {"store": wd.EPI_STORE, "gelu": wd.EPI_GELU, "f32": wd.EPI_F32}[c["epilogue"]]
        wd.wd_gemm_lora(c["M"], c["N"], c["K"], st["A"], st["W"], st["bias"], st["lora"], epi, st["out"], st["ws"])
        return st["out"]
    v = st["A"].float() @ st["W"].float().t() + st["bias"]
    for a, b, i in zip(st["seg"], st["seg"][1:], st["ids"]):
        if i >= 0:
            t = st["A"][a:b].float() @ st["down"][i].float().t() * st["scale"][i]
            v[a:b] += t @ st["up"][i].float().t()
    if c["epilogue"] == "gelu":
        v = 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    return v.to(st["out"].dtype)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attention":
        H, Hk, dh, R = case["heads"], case["kv_heads"], case["dh"], case["radius"]
        o = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        for n in range(len(st["cu_q"]) - 1):
            a, b, ka, kb = st["cu_q"][n], st["cu_q"][n + 1], st["cu_k"][n], st["cu_k"][n + 1]
            if kb == ka:
                continue
            for h in range(H):
                kc, oc = slice(h * Hk // H * dh, (h * Hk // H + 1) * dh), slice(h * dh, (h + 1) * dh)
                K, V = st["k"][ka:kb, kc].double(), st["v"][ka:kb, kc].double()
                j = torch.arange(kb - ka, device="cuda")
                for i0 in range(a, b, 4096):
                    i1 = min(b, i0 + 4096)
                    s = torch.einsum("id,jd->ij", st["q"][i0:i1, oc].double(), K).mul_(case["scale"])
                    if R:
                        i = torch.arange(i0 - a, i1 - a, device="cuda")
                        s += st["bias"][h].double()[(j[None] - i[:, None]).clamp_(-R, R) + R]
                    p = torch.nan_to_num(torch.exp(s - torch.logsumexp(s, -1, keepdim=True)), nan=0.0)
                    o[i0:i1, oc] = torch.einsum("ij,jd->id", p, V)
        return o
    if case["op"] == "rope":
        outs = []
        sec = _sections(case["dh"])
        for x, gain in ((st["q"], st["g_q"]), (st["k"], st["g_k"])):
            z = x.double()
            if gain is not None:
                z = z / (z.pow(2).sum(-1, keepdim=True) / z.shape[1] + 1e-6).sqrt() * gain.double()
            z = torch.view_as_complex(z.view(case["rows"], -1, case["dh"] // 2, 2).contiguous())
            j = 0
            for axis in range(3):
                for p in range(sec[axis] // 2):
                    t = st["pos"][:, axis].double() * 10000.0 ** (-2.0 * p / sec[axis])
                    z[:, :, j] *= torch.polar(torch.ones_like(t), t)[:, None]
                    j += 1
            outs.append(torch.view_as_real(z).reshape(x.shape))
        return tuple(outs)
    if case["op"] == "norm":
        s = st["x"].double() + st["y"].double()
        d = s
        if case["norm"] == "layer":
            d = s - s.sum(-1, keepdim=True) / case["D"]
        n = d / torch.sqrt(d.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6) * st["gain"].double()
        if st["beta"] is not None:
            n = n + st["beta"].double()
        if case["out"] != "e4m3":
            return s, n
        sc = n.abs().amax(-1) / 448
        return s, n / torch.where(sc > 0, sc, 1.0)[:, None], torch.where(sc > 0, sc, 1.0)
    W = st["W"].double()
    v = torch.empty((case["M"], case["N"]), dtype=torch.float64, device="cuda")
    row = torch.arange(case["M"], device="cuda")
    which = torch.full((case["M"],), -1, device="cuda")
    for n, i in enumerate(st["ids"]):
        which[(row >= st["seg"][n]) & (row < st["seg"][n + 1])] = i
    for i in range(-1, case["adapters"]):
        rows = (which == i).nonzero()[:, 0]
        Wi = W if i < 0 else W + st["scale"][i].double() * (st["up"][i].double() @ st["down"][i].double())
        v[rows] = st["A"][rows].double() @ Wi.t()
    v += st["bias"].double()
    return v * 0.5 * torch.erfc(-v / math.sqrt(2.0)) if case["epilogue"] == "gelu" else v


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "attention":
        lq = _ints(case["q"])
        lk = _ints(case["k"]) or lq
        H, Hk, dh, R = case["heads"], case["kv_heads"], case["dh"], case["radius"]
        pairs = 0
        for a, b in zip(lq, lk):
            if case["window"]:   # |j - i| < R
                pairs += sum(max(0, min(b, i + R) - max(0, i - R + 1)) for i in range(a))
            else:
                pairs += a * b
        nb = 2 * dh * (2 * H * sum(lq) + 2 * Hk * sum(lk)) + (4 * H * (2 * R + 1) if R else 0) + 8 * (len(lq) + 1)
        return {"bytes": nb, "flops": 4 * dh * H * pairs}
    if case["op"] == "rope":
        es = 4 if case["type"] == "f32" else 2
        n = case["rows"] * (case["heads"] + case["kv_heads"]) * case["dh"]
        return {"bytes": 2 * es * n + 12 * case["rows"] + (4 * n // case["rows"] if case["norm"] else 0), "flops": 7 * n}
    if case["op"] == "norm":
        es = {"f32": 4, "bf16": 2, "e4m3": 1}
        n = case["rows"] * case["D"]
        nb = n * (2 * es[case["x"]] + es[case["y"]] + es[case["out"]]) + 4 * case["D"] * (2 if case["norm"] == "layer" else 1)
        return {"bytes": nb + (4 * case["rows"] if case["out"] == "e4m3" else 0), "flops": 7 * n}
    M, N, K, r = case["M"], case["N"], case["K"], case["rank"]
    lens, ids = _ints(case["segs"]), _ints(case["ids"])
    covered = sum(n for n, i in zip(lens, ids) if i >= 0)
    used = len({i for i in ids if i >= 0})
    return {"bytes": 2 * (M * K + N * K + used * r * (K + N)) + M * N * (4 if case["epilogue"] == "f32" else 2) + 4 * N,
            "flops": 2 * M * N * K + 2 * covered * r * (N + K)}
