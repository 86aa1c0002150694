"""What the binding of the packed-batch operators refuses, each by its own message:
host tensors fit everything but the device, which is checked last, so a check
that is missing shows as the device's message."""
import pytest
import torch

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def wd():
    from flow_matching_video_b200 import build
    build.build()
    from flow_matching_video_b200 import wd as _wd
    return _wd


def call_attention(wd, **kw):
    q, kv, cu = torch.zeros((10, 512), dtype=BF), torch.zeros((12, 256), dtype=BF), torch.zeros(3, dtype=I32)
    a = dict(q=q, k=kv, v=kv, cu_q=cu, cu_k=cu, o=q, bias=None, dtype=1)
    a.update(kw)
    wd.wd_attention_packed(a["dtype"], 4, 2, 128, a["q"], a["k"], a["v"], a["cu_q"], a["cu_k"], 0.1, a["o"], bias=a["bias"])


def call_rope(wd, **kw):
    q = torch.zeros((10, 512), dtype=BF)
    a = dict(dtype=1, dh=128, axes=wd.wd_rope_axes.of((44, 42, 42)), pos=torch.zeros((10, 3), dtype=I32), q=q, g_q=None, q_out=q,
             k=None, g_k=None, k_out=None)
    a.update(kw)
    wd.wd_qknorm_rope_axes(*a.values())


def call_norm(wd, **kw):
    x = torch.zeros((10, 256))
    a = dict(x_dtype=0, x=x, y_dtype=0, y=x, norm=1, gain=None, beta=None, eps=1e-6, sum=None, out_dtype=0, out=x, scale=None)
    a.update(kw)
    wd.wd_add_norm(*a.values())


def adapters(wd, **kw):
    a = dict(seg=torch.zeros(3, dtype=I32), adapter=torch.zeros(2, dtype=I32), down=torch.zeros((2, 16, 128), dtype=BF),
             up=torch.zeros((2, 256, 16), dtype=BF), scale=None)
    a.update(kw)
    return wd.wd_lora.of(*a.values())


def call_lora(wd, **kw):
    a = dict(M=9, N=256, K=128, A=torch.zeros((9, 128), dtype=BF), W=torch.zeros((256, 128), dtype=BF), bias=None, lora=adapters(wd),
             epilogue=0, out=torch.zeros((9, 256), dtype=BF), ws=torch.zeros(1 << 20, dtype=torch.uint8), gate_a=None, gate_b=None)
    a.update(kw)
    wd.wd_gemm_lora(*a.values())


CALLS = dict(attention=call_attention, rope=call_rope, norm=call_norm, lora=call_lora, adapters=adapters)


@pytest.mark.parametrize("call", ["attention", "rope", "norm", "lora"])
def test_what_fits_is_refused_for_its_device_alone(wd, call):
    with pytest.raises(ValueError, match="one CUDA device is wanted"):
        CALLS[call](wd)


@pytest.mark.parametrize("call,kw,message", [
    ("attention", dict(q=torch.zeros(10, 512)), "rows of 512 dense elements are wanted, not torch.float32"),
    ("attention", dict(q=torch.zeros((10, 256), dtype=BF)), "rows of 512 dense elements are wanted"),
    ("attention", dict(q=torch.zeros((512, 10), dtype=BF).t()), "rows of 512 dense elements are wanted"),
    ("attention", dict(v=torch.zeros((5, 256), dtype=BF)), r"rows of 256 dense elements are wanted, not torch.bfloat16 \[5, 256\]"),
    ("attention", dict(k=torch.zeros((12, 264), dtype=BF)[:, :256]), "row strides 264 of k and 256 of v"),
    ("attention", dict(cu_k=torch.zeros(2, dtype=I32)), r"a dense torch.int32 tensor \[3\] is wanted"),
    ("attention", dict(cu_q=torch.zeros(3, dtype=torch.int64)), r"a dense torch.int32 tensor \[3\] is wanted"),
    ("attention", dict(cu_q=torch.zeros(6, dtype=I32)[::2]), r"a dense torch.int32 tensor \[3\] is wanted"),
    ("attention", dict(o=torch.zeros((4, 512), dtype=BF)), r"not torch.bfloat16 \[4, 512\]"),
    ("attention", dict(o=torch.zeros((10, 512), dtype=torch.float16)), "torch.bfloat16 rows of 512"),
    ("attention", dict(dtype=9), "dtype 9"),
    ("attention", dict(bias=torch.zeros(4, 6)), r"a dense torch.float32 tensor \[4, 5\] is wanted"),
    ("attention", dict(bias=torch.zeros(3, 5)), r"a dense torch.float32 tensor \[4, 5\] is wanted"),
    ("attention", dict(bias=torch.zeros((4, 5), dtype=BF)), r"a dense torch.float32 tensor \[4, 5\] is wanted"),
    ("attention", dict(bias=torch.zeros(5)), "bias: 1 dimensions, not 2"),
    ("rope", dict(pos=torch.zeros((9, 3), dtype=I32)), r"a dense torch.int32 tensor \[10, 3\] is wanted"),
    ("rope", dict(pos=torch.zeros((10, 3), dtype=torch.int64)), r"a dense torch.int32 tensor \[10, 3\] is wanted"),
    ("rope", dict(g_q=torch.zeros(5)), r"a dense torch.float32 tensor \[512\] is wanted"),
    ("rope", dict(q_out=torch.zeros((9, 512), dtype=BF)), "rows of 512 dense elements are wanted"),
    ("rope", dict(k=torch.zeros((10, 256), dtype=BF)), "k and k_out go together"),
    ("rope", dict(k_out=torch.zeros((10, 256), dtype=BF)), "k and k_out go together"),
    ("rope", dict(q=torch.zeros((10, 500), dtype=BF), q_out=torch.zeros((10, 500), dtype=BF)), "rows of 500 and 0 elements with heads of 128"),
    ("rope", dict(dh=0), "heads of 0"),
    ("norm", dict(y_dtype=1), r"a dense torch.bfloat16 tensor \[10, 256\] is wanted"),
    ("norm", dict(gain=torch.zeros(5)), r"a dense torch.float32 tensor \[256\] is wanted"),
    ("norm", dict(beta=torch.zeros(5)), r"a dense torch.float32 tensor \[256\] is wanted"),
    ("norm", dict(out_dtype=3), r"a dense torch.uint8 tensor \[10, 256\] is wanted"),
    ("norm", dict(out=torch.zeros(9, 256)), r"a dense torch.float32 tensor \[10, 256\] is wanted"),
    ("norm", dict(sum=torch.zeros((10, 512))[:, :256]), r"a dense torch.float32 tensor \[10, 256\] is wanted"),
    ("norm", dict(scale=torch.zeros(9)), r"a dense torch.float32 tensor \[10\] is wanted"),
    ("adapters", dict(seg=torch.zeros(4, dtype=I32)), r"a dense torch.int32 tensor \[3\] is wanted"),
    ("adapters", dict(seg=torch.zeros(3, dtype=torch.int64)), r"a dense torch.int32 tensor \[3\] is wanted"),
    ("adapters", dict(up=torch.zeros((1, 256, 16), dtype=BF)), r"a dense torch.bfloat16 tensor \[2, 256, 16\] is wanted"),
    ("adapters", dict(up=torch.zeros((2, 256, 8), dtype=BF)), r"a dense torch.bfloat16 tensor \[2, 256, 16\] is wanted"),
    ("adapters", dict(down=torch.zeros(2, 16, 128)), r"a dense torch.bfloat16 tensor \[2, 16, 128\] is wanted"),
    ("adapters", dict(scale=torch.zeros(3)), r"a dense torch.float32 tensor \[2\] is wanted"),
    ("lora", dict(A=torch.zeros((8, 128), dtype=BF)), r"a dense torch.bfloat16 tensor \[9, 128\] is wanted"),
    ("lora", dict(W=torch.zeros((256, 136), dtype=BF)[:, :128]), r"a dense torch.bfloat16 tensor \[256, 128\] is wanted"),
    ("lora", dict(epilogue=2), r"a dense torch.float32 tensor \[9, 256\] is wanted"),
    ("lora", dict(epilogue=5), r"a dense torch.float16 tensor \[9, 256\] is wanted"),
    ("lora", dict(bias=torch.zeros(255)), r"a dense torch.float32 tensor \[256\] is wanted"),
    ("lora", dict(gate_b=torch.zeros(255)), r"a dense torch.float32 tensor \[256\] is wanted"),
    ("lora", dict(K=64, A=torch.zeros((9, 64), dtype=BF), W=torch.zeros((256, 64), dtype=BF)), "adapters of 256 x 128 for a layer of 256 x 64"),
])
def test_what_does_not_fit_is_named(wd, call, kw, message):
    with pytest.raises(ValueError, match=message):
        CALLS[call](wd, **kw)


@pytest.mark.parametrize("call,name", [
    ("attention", "q"), ("attention", "k"), ("attention", "v"), ("attention", "o"), ("attention", "cu_q"), ("attention", "cu_k"),
    ("rope", "pos"), ("rope", "q"), ("rope", "q_out"), ("norm", "x"), ("norm", "out"),
    ("adapters", "seg"), ("adapters", "adapter"), ("adapters", "down"), ("adapters", "up"),
    ("lora", "A"), ("lora", "W"), ("lora", "out"), ("lora", "ws"),
])
def test_a_missing_tensor_is_refused(wd, call, name):
    with pytest.raises(ValueError, match="not None"):
        CALLS[call](wd, **{name: None})


def test_a_workspace_with_gaps_is_refused(wd):
    """Its bytes are counted without the gaps, which belong to someone else."""
    with pytest.raises(ValueError, match="a dense workspace is wanted, not one with strides"):
        call_lora(wd, ws=torch.zeros((1024, 2048), dtype=torch.uint8)[:, :1024])
