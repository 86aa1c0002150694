"""Refusals and sizes of the packed-batch operators: everything here returns
before any CUDA call, so no GPU is needed."""
import ctypes as C
import math

import pytest
import torch

OK, ARG, SHAPE, DTYPE, ALIGN, WORKSPACE, CUDA, TIMEOUT, UNSUPPORTED = range(9)
Q, K, V, O, CU, B = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000   # never dereferenced


@pytest.fixture(scope="module")
def wd():
    from flow_matching_video_b200 import build
    build.build()
    from flow_matching_video_b200 import wd as _wd
    return _wd


def attention(wd, **kw):
    a = dict(dtype=1, n_seq=2, heads=4, kv_heads=2, dh=128, q=Q, q_rs=512, q_rows=100, cu_q=CU, k=K, v=V, kv_rs=256,
             k_rows=100, cu_k=CU, scale=0.1, bias=None, radius=0, o=O, o_rs=512, stream=None)
    a.update(kw)
    return wd.lib().wd_attention_packed(*a.values())


@pytest.mark.parametrize("want,kw", [
    (ARG, dict(q=None)), (ARG, dict(k=None)), (ARG, dict(v=None)), (ARG, dict(o=None)), (ARG, dict(cu_q=None)), (ARG, dict(cu_k=None)),
    (ALIGN, dict(q=Q + 8)), (ALIGN, dict(o=O + 4)), (ALIGN, dict(cu_k=CU + 4)), (ALIGN, dict(bias=B + 4, radius=3)),
    (DTYPE, dict(dtype=0)), (DTYPE, dict(dtype=3)), (DTYPE, dict(dtype=9)),
    (UNSUPPORTED, dict(dh=32)), (UNSUPPORTED, dict(dh=256)), (UNSUPPORTED, dict(dh=0)),
    (SHAPE, dict(n_seq=0)), (SHAPE, dict(n_seq=65537)), (SHAPE, dict(q_rows=0)), (SHAPE, dict(k_rows=0)), (SHAPE, dict(k_rows=(1 << 30) + 1)),
    (SHAPE, dict(heads=0)), (SHAPE, dict(heads=5)), (SHAPE, dict(kv_heads=0)), (SHAPE, dict(kv_heads=3)),
    (SHAPE, dict(heads=65536, kv_heads=1)),
    (SHAPE, dict(radius=4)), (SHAPE, dict(bias=B)), (SHAPE, dict(bias=B, radius=1025)), (SHAPE, dict(bias=B, radius=-1)),
    (ARG, dict(scale=0.0)), (ARG, dict(scale=-1.0)), (ARG, dict(scale=math.nan)), (ARG, dict(scale=math.inf)), (ARG, dict(scale=3e38)),
    (SHAPE, dict(q_rs=504)), (SHAPE, dict(kv_rs=248)), (SHAPE, dict(o_rs=0)), (ALIGN, dict(q_rs=516)), (ALIGN, dict(kv_rs=257)),
], ids=str)
def test_attention_packed_refusals(wd, want, kw):
    assert attention(wd, **kw) == want
    assert wd.wd_last_error()


def rope(wd, sec=(44, 42, 42), theta=1e4, step=(1, 1, 1), **kw):
    a = dict(dtype=1, rows=10, dh=128, axes=C.byref(wd.wd_rope_axes.of(sec, theta, step)), pos=CU, q=Q, q_rs=256, heads=2, g_q=None,
             q_out=O, qo_rs=256, k=K, k_rs=128, kv_heads=1, g_k=None, k_out=V, ko_rs=128, eps=1e-6, stream=None)
    a.update(kw)
    return wd.lib().wd_qknorm_rope_axes(*a.values())


@pytest.mark.parametrize("want,kw", [
    (ARG, dict(axes=None)), (ARG, dict(pos=None)), (ARG, dict(q=None)), (ARG, dict(q_out=None)), (ARG, dict(k_out=None)),
    (ALIGN, dict(pos=CU + 4)), (ALIGN, dict(k=K + 8)), (ALIGN, dict(g_q=B + 4)),
    (DTYPE, dict(dtype=3)), (SHAPE, dict(rows=0)), (SHAPE, dict(rows=(1 << 30) + 1)), (SHAPE, dict(dh=12, sec=(4, 4, 4))),
    (SHAPE, dict(dh=264, sec=(88, 88, 88), q_rs=528)), (SHAPE, dict(sec=(43, 43, 42))), (SHAPE, dict(sec=(44, 42, 40))),
    (SHAPE, dict(sec=(130, -2, 0))), (SHAPE, dict(heads=0)), (SHAPE, dict(heads=65, q_rs=8320, qo_rs=8320)), (SHAPE, dict(kv_heads=0)),
    (ARG, dict(theta=0.0)), (ARG, dict(theta=math.nan)), (ARG, dict(step=(1, 0, 1))), (ARG, dict(step=(1, 1, math.inf))), (ARG, dict(eps=-1.0)),
    (SHAPE, dict(q_rs=128)), (SHAPE, dict(ko_rs=120)), (ALIGN, dict(q_rs=260)), (ARG, dict(q_out=Q, qo_rs=264)),
], ids=str)
def test_qknorm_rope_axes_refusals(wd, want, kw):
    assert rope(wd, **kw) == want
    assert wd.wd_last_error()


def norm(wd, **kw):
    a = dict(rows=10, D=256, x_dtype=0, x=Q, y_dtype=1, y=K, norm=1, gain=None, beta=None, eps=1e-6, sum=V, out_dtype=3, out=O, scale=B, stream=None)
    a.update(kw)
    return wd.lib().wd_add_norm(*a.values())


@pytest.mark.parametrize("want,kw", [
    (ARG, dict(x=None)), (ARG, dict(out=None)), (ARG, dict(scale=None)), (ALIGN, dict(x=Q + 8)), (ALIGN, dict(gain=B + 8)),
    (ALIGN, dict(sum=V + 4)), (DTYPE, dict(x_dtype=2)), (DTYPE, dict(y_dtype=3)), (DTYPE, dict(out_dtype=2)), (DTYPE, dict(out_dtype=7)),
    (SHAPE, dict(rows=0)), (SHAPE, dict(rows=(1 << 30) + 1)), (SHAPE, dict(D=0)), (SHAPE, dict(D=12)), (SHAPE, dict(D=8200)),
    (ARG, dict(norm=2)), (ARG, dict(eps=-1e-6)), (ARG, dict(eps=math.nan)),
], ids=str)
def test_add_norm_refusals(wd, want, kw):
    assert norm(wd, **kw) == want
    assert wd.wd_last_error()


def lora(wd, n_seg=2, n_adapters=3, rank=16, seg=CU, adapter=CU, down=K, up=V, scale=None, **kw):
    ld = wd.wd_lora(n_seg, n_adapters, rank, seg, adapter, down, up, scale)
    a = dict(M=300, N=256, K=128, A=Q, W=B, bias=None, lora=C.byref(ld), epilogue=0, out=O, gate_a=None, gate_b=None,
             ws=0x100000, ws_bytes=wd.wd_gemm_lora_bytes(300, 2, 16), stream=None)
    a.update(kw)
    return wd.lib().wd_gemm_lora(*a.values())


@pytest.mark.parametrize("want,kw", [
    (ARG, dict(A=None)), (ARG, dict(W=None)), (ARG, dict(lora=None)), (ARG, dict(ws=None)), (ARG, dict(seg=None)), (ARG, dict(adapter=None)),
    (ARG, dict(down=None)), (ARG, dict(up=None)), (ALIGN, dict(A=Q + 8)), (ALIGN, dict(up=V + 8)), (ALIGN, dict(scale=B + 4)), (ALIGN, dict(ws=0x100008)),
    (ARG, dict(epilogue=4)), (ARG, dict(epilogue=6)), (ARG, dict(epilogue=-1)),
    (SHAPE, dict(M=0)), (SHAPE, dict(N=0)), (SHAPE, dict(N=96)), (SHAPE, dict(K=0)), (SHAPE, dict(K=12)), (SHAPE, dict(M=(1 << 29) + 1)),
    (SHAPE, dict(rank=0)), (SHAPE, dict(rank=12)), (SHAPE, dict(rank=264)), (SHAPE, dict(n_seg=0)), (SHAPE, dict(n_seg=65537)),
    (SHAPE, dict(n_adapters=0)), (SHAPE, dict(n_adapters=1 << 24)), (SHAPE, dict(N=64, n_adapters=1 << 25, rank=256)), (WORKSPACE, dict(ws_bytes=1000)), (WORKSPACE, dict(M=3000)),
], ids=str)
def test_gemm_lora_refusals(wd, want, kw):
    assert lora(wd, **kw) == want
    assert wd.wd_last_error()


def test_gemm_lora_workspace_grows_with_what_it_holds(wd):
    f = wd.wd_gemm_lora_bytes
    assert f(0, 1, 8) == f(1, 0, 8) == f(1, 1, 0) == f(1, 1, 12) == f(1, 1, 264) == f((1 << 29) + 1, 1, 8) == f(1, 65537, 8) == 0
    assert f(1, 1, 8) >= 2 * 3 * 256 * 8 * 2 + 16
    for M, n, r in ((300, 2, 16), (43745, 3, 32), (1 << 29, 65535, 256)):
        assert f(M, n, r) >= ((M + 127) // 128 + n) * 3 * 128 * r * 2 + (M + 127) // 128 * 16
        assert f(M, n + 1, r) > f(M, n, r)


def test_binding_checks_tensors_against_the_sizes(wd):
    """The binding reads sizes and strides off the tensors and refuses what does not fit
    before it calls the library (here: host tensors, which it refuses last)."""
    bf, i32 = torch.bfloat16, torch.int32
    q, kv = torch.zeros((10, 512), dtype=bf), torch.zeros((12, 256), dtype=bf)
    cu = torch.zeros(3, dtype=i32)

    def attn(q=q, k=kv, v=kv, cu_q=cu, cu_k=cu, o=q, bias=None, dtype=1):
        wd.wd_attention_packed(dtype, 4, 2, 128, q, k, v, cu_q, cu_k, 0.1, o, bias=bias)

    with pytest.raises(ValueError, match="one CUDA device"):
        attn()
    for kw in (dict(q=q.float()), dict(q=q[:, :256]), dict(q=q.t()), dict(v=kv[:5]), dict(cu_k=cu[:2]), dict(cu_q=cu.long()),
               dict(o=q[:4]), dict(o=q.half()), dict(k=torch.zeros((12, 264), dtype=bf)[:, :256]), dict(dtype=9),
               dict(bias=torch.zeros(4, 6)), dict(bias=torch.zeros(3, 5)), dict(bias=torch.zeros(4, 5, dtype=bf))):
        with pytest.raises(ValueError, match="(?!.*one CUDA device)"):
            attn(**kw)
    ax = wd.wd_rope_axes.of((44, 42, 42))
    pos = torch.zeros((10, 3), dtype=i32)
    with pytest.raises(ValueError, match="one CUDA device"):
        wd.wd_qknorm_rope_axes(1, 128, ax, pos, q, None, q)
    for args in ((pos[:9], q, None, q), (pos.long(), q, None, q), (pos, q, torch.zeros(5), q), (pos, q, None, q[:9]),
                 (pos, q, None, q, q, None, None), (pos, q[:, :500], None, q[:, :500])):
        with pytest.raises(ValueError, match="(?!.*one CUDA device)"):
            wd.wd_qknorm_rope_axes(1, 128, ax, *args)
    x = torch.zeros((10, 256))
    for args in ((0, x, 1, x, 1, None, None, 1e-6, None, 0, x), (0, x, 0, x, 1, x[0, :5], None, 1e-6, None, 0, x),
                 (0, x, 0, x, 1, None, None, 1e-6, None, 3, x), (0, x, 0, x[:9], 1, None, None, 1e-6, None, 0, x)):
        with pytest.raises(ValueError, match="(?!.*one CUDA device)"):
            wd.wd_add_norm(*args)
    down, up = torch.zeros((2, 16, 128), dtype=bf), torch.zeros((2, 256, 16), dtype=bf)
    for args in ((cu, cu, down, up), (cu.long(), cu[:2], down, up), (cu, cu[:2], down, up[:1]), (cu, cu[:2], down.float(), up),
                 (cu, cu[:2], down, up, torch.zeros(3))):
        with pytest.raises(ValueError):
            wd.wd_lora.of(*args)
    ld = wd.wd_lora.of(cu, cu[:2], down, up)
    A, W, out, ws = torch.zeros((9, 128), dtype=bf), torch.zeros((256, 128), dtype=bf), torch.zeros((9, 256), dtype=bf), torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="one CUDA device"):
        wd.wd_gemm_lora(9, 256, 128, A, W, None, ld, 0, out, ws)
    with pytest.raises(ValueError, match="(?!.*one CUDA device)"):
        wd.wd_gemm_lora(9, 256, 128, A, W, None, ld, 2, out, ws)
    with pytest.raises(ValueError, match="wd_lora.of"):
        wd.wd_gemm_lora(9, 256, 128, A, W, None, wd.wd_lora(1, 1, 8, 0, 0, 0, 0, 0), 0, out, ws)
    with pytest.raises(ValueError, match="adapters of 256 x 128"):
        wd.wd_gemm_lora(9, 256, 64, A[:, :64].contiguous(), W[:, :64].contiguous(), None, ld, 0, out, ws)
