"""What the binding of the attention entry points refuses before the library is called, without a GPU: tensors
that stand for CUDA tensors, and a library that records its calls instead of making them."""
import types

import pytest


class FakeTensor:
    """As much of a contiguous CUDA tensor as the binding looks at."""

    def __init__(self, shape, dtype, device=0, contiguous=True):
        import torch
        self.shape, self.dtype, self._device, self._contiguous = torch.Size(shape), dtype, device, contiguous
        self.is_cuda = device >= 0
        self.device = f"cuda:{device}" if device >= 0 else "cpu"

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return self._contiguous

    def get_device(self):
        return self._device

    def data_ptr(self):
        return 4096

    def stride(self):
        out, step = [], 1
        for n in reversed(self.shape):
            out.insert(0, step)
            step *= n
        return tuple(out)


@pytest.fixture()
def J(monkeypatch):
    import torch
    from tensor_decomposition_b200 import build
    build.build()
    from tensor_decomposition_b200 import jolt
    calls = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or 0

    monkeypatch.setattr(jolt, "_lib", Recorder())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return types.SimpleNamespace(m=jolt, calls=calls, torch=torch)


def _stream(J, layers=3):
    shape = J.m.Shape(layers, 4, 300, 128, 1, J.m.JOLT_BF16)
    return J.m.Stream(None, types.SimpleNamespace(shape=shape))


def test_attention_over_a_stream_takes_its_types_and_sizes_alone(J):
    """An fp16 query would be read as bf16, an output or log-sum-exp of 16 bits would be written past its end, and
    so would tensors of fewer layers or features."""
    bf16, f16, f32, f64 = (getattr(J.torch, n) for n in ("bfloat16", "float16", "float32", "float64"))
    st = _stream(J)
    T = FakeTensor
    good = dict(Q=T((5, 8, 128), bf16), out=T((5, 8, 128), f32), lse=T((5, 8), f32))
    J.m.jolt_attention_lse(st, 1, **good, scale=0.1)
    assert J.calls == ["jolt_attention_lse"]
    half = dict(Q=T((5, 8, 64), bf16), out=T((5, 8, 64), f32))
    for bad in (dict(Q=T((5, 8, 128), f16)), dict(Q=T((5, 8, 128), f32)), dict(out=T((5, 8, 128), f16)),
                dict(out=T((5, 8, 128), bf16)), dict(out=T((5, 8, 128), f64)), dict(lse=T((5, 8), f16)), half,
                dict(Q=T((5, 8, 128), bf16, device=1)), dict(out=T((5, 8, 128), f32, device=1)),
                dict(lse=T((5, 8), f32, device=-1)), dict(out=T((5, 8, 128), f32, contiguous=False)),
                {k: T(v.shape, v.dtype, device=1) for k, v in good.items()}):
        with pytest.raises(ValueError):
            J.m.jolt_attention_lse(st, 1, **{**good, **bad}, scale=0.1)
    whole = dict(Q=T((3, 8, 5, 128), bf16), out=T((3, 8, 5, 128), f32))
    J.m.jolt_attention(st, **whole, scale=0.1)
    assert J.calls == ["jolt_attention_lse", "jolt_attention"]
    for bad in (dict(Q=T((3, 8, 5, 128), f16)), dict(out=T((3, 8, 5, 128), f16)), dict(out=T((3, 8, 5, 128), bf16)),
                dict(Q=T((3, 8, 5, 64), bf16), out=T((3, 8, 5, 64), f32)),
                dict(Q=T((2, 8, 5, 128), bf16), out=T((2, 8, 5, 128), f32)), dict(out=T((3, 8, 5, 128), f32, device=1))):
        with pytest.raises(ValueError):
            J.m.jolt_attention(st, **{**whole, **bad}, scale=0.1)
    assert len(J.calls) == 2


def test_keys_and_their_output_come_together(J):
    bf16 = J.torch.bfloat16
    Q, K = FakeTensor((5, 8, 128), bf16), FakeTensor((5, 2, 128), bf16)
    J.m.jolt_qk_norm_rope(Q, Q, K, K)
    assert J.calls == ["jolt_qk_norm_rope"]
    for kw in (dict(K=K), dict(K_out=K)):
        with pytest.raises(ValueError):
            J.m.jolt_qk_norm_rope(Q, Q, **kw)
    assert len(J.calls) == 1


def test_a_stream_of_unknown_layers_is_taken(J):
    """A stream object made around a handle from elsewhere: its layers are the caller's to know."""
    T, bf16, f32 = FakeTensor, J.torch.bfloat16, J.torch.float32
    J.m.jolt_attention(J.m.Stream(None), T((3, 8, 5, 128), bf16), T((3, 8, 5, 128), f32), 0.1)
    assert J.calls == ["jolt_attention"]
