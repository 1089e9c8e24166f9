"""The attention calls refuse memory that their launch could not reach: a workspace or a tensor of the host or
of another device.  Run on stand-ins for tensors, with a library that notes whether it was called, so nothing
reaches a GPU."""
import pytest
import torch

import nvfp4_weight_quantized_03_gb300 as q

BF, F8, I32, F32, F64 = torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float32, torch.float64


class Stand:
    """A tensor's metadata: contiguous, of one device (-1: the host)."""

    def __init__(self, shape, dtype, dev=0, contiguous=True):
        self.shape, self.dtype, self.dev, self.contiguous = torch.Size(shape), dtype, dev, contiguous
        self.is_cuda, self.device = dev >= 0, torch.device("cuda", dev) if dev >= 0 else torch.device("cpu")
        self.nbytes = self.numel() * 8

    def get_device(self):
        return self.dev

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        s = torch.empty(self.shape, device="meta").stride()
        return s if i is None else s[i]

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 0x1000


class Library:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    fake = Library()
    monkeypatch.setattr(q, "_lib", fake)
    monkeypatch.setattr(q, "_device", lambda: 0)
    monkeypatch.setattr(q, "_stream", lambda *a: 0)
    return fake


def _cache(dev=0):
    pages = lambda: Stand((5, 2, 16, 64), F8, dev)
    return q.kv_cache(pages(), pages(), Stand((3, 4), I32, dev), Stand((2,), F32, dev), Stand((2,), F32, dev))


def _calls(dev=0):
    """name -> (function, its tensors by name)."""
    rows = lambda n, h: Stand((n, h, 64), BF, dev)
    ws = lambda: Stand((1 << 20,), torch.uint8, dev)
    return {
        "append": (q.qerl_rope_append, dict(
            cache=_cache(dev), q=rows(3, 4), k=rows(3, 2), v=rows(3, 2), positions=Stand((3,), I32, dev),
            inv_freq=Stand((32,), F64, dev), q_out=rows(3, 4), k_out=rows(3, 2), workspace=ws(),
            seq_ids=Stand((3,), I32, dev))),
        "decode": (q.qerl_decode_attention, dict(
            cache=_cache(dev), q=rows(3, 4), lengths=Stand((3,), I32, dev), scale=0.1, out=rows(3, 4),
            lse=Stand((3, 4), F32, dev), workspace=ws())),
        "prompt": (q.qerl_prompt_attention, dict(
            q=rows(9, 4), k=rows(9, 2), v=rows(9, 2), cu_seqlens=Stand((3,), I32, dev), scale=0.1, out=rows(9, 4),
            lse=Stand((9, 4), F32, dev), workspace=ws())),
    }


TENSORS = [(call, name) for call, (_, kw) in _calls().items() for name, x in kw.items() if isinstance(x, Stand)]


@pytest.mark.parametrize("call", ["append", "decode", "prompt"])
def test_good_calls_go_through(lib, call):
    f, kw = _calls()[call]
    assert f(**kw) == 0 and lib.calls == 1


@pytest.mark.parametrize("dev", [-1, 1])
@pytest.mark.parametrize("call,name", TENSORS)
def test_memory_of_the_host_or_another_device(lib, call, name, dev):
    f, kw = _calls()[call]
    x = kw[name]
    with pytest.raises((TypeError, ValueError)):
        f(**{**kw, name: Stand(x.shape, x.dtype, dev)})
    assert lib.calls == 0


@pytest.mark.parametrize("call", ["append", "decode", "prompt"])
def test_everything_on_another_device_than_the_current_one(lib, call):
    f, kw = _calls(dev=1)[call]
    with pytest.raises(ValueError):
        f(**kw)
    assert lib.calls == 0


@pytest.mark.parametrize("call", ["append", "decode"])
def test_a_cache_on_another_device(lib, call):
    f, kw = _calls()[call]
    with pytest.raises(ValueError):
        f(**{**kw, "cache": _cache(1)})
    assert lib.calls == 0


@pytest.mark.parametrize("call", ["append", "decode", "prompt"])
def test_a_workspace_in_pieces(lib, call):
    f, kw = _calls()[call]
    with pytest.raises(ValueError):
        f(**{**kw, "workspace": Stand((1 << 20,), torch.uint8, 0, contiguous=False)})
    assert lib.calls == 0


@pytest.mark.parametrize("name", ["k", "v", "page_table", "k_scale", "v_scale"])
@pytest.mark.parametrize("dev", [-1, 1])
def test_a_cache_of_memory_in_two_places(name, dev):
    good = dict(k=Stand((5, 2, 16, 64), F8), v=Stand((5, 2, 16, 64), F8), page_table=Stand((3, 4), I32),
                k_scale=Stand((2,), F32), v_scale=Stand((2,), F32))
    assert q.kv_cache(**good).device == 0
    with pytest.raises((TypeError, ValueError)):
        q.kv_cache(**{**good, name: Stand(good[name].shape, good[name].dtype, dev)})
