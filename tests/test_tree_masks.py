"""A mask without words is refused by the binding: its empty tensor has no address, and none is the call's mark for
tokens in order.  Run on stand-ins for tensors, so nothing reaches a GPU."""
import pytest
import torch

from test_attention_memory_checks import Stand, lib  # noqa: F401 (lib is a fixture)
from test_cache_memory_checks import _calls


def test_a_mask_without_words(lib):
    f, kw = _calls()["tree"]
    with pytest.raises(ValueError, match="mask"):
        f(**{**kw, "mask": Stand((9, 0), torch.int64)})
    assert lib.calls == 0


def test_no_tokens_need_no_words(lib):
    f, kw = _calls()["tree"]
    none = {name: Stand((0, *kw[name].shape[1:]), kw[name].dtype) for name in ("q", "k", "v", "out", "lse")}
    assert f(**{**kw, **none, "mask": Stand((0, 0), torch.int64)}) == 0 and lib.calls == 1
