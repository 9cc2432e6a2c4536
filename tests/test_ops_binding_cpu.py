"""What the binding of the decode-step operators refuses because the C side could not see it: tensors
whose strides name more memory than they hold.  No GPU is needed: the tensors only say that they
are on one, and every call is refused before a pointer is used."""
import pytest

torch = pytest.importorskip("torch")

import sparse_moe_transformer_wave_amd as fm  # noqa: E402

BF = torch.bfloat16


class _Gpu(torch.Tensor):
    is_cuda = True


def _t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_Gpu)


def _cache(k, v):
    return fm.KVCache(k, v, 2)


@pytest.mark.parametrize("pages", [2, 40])
def test_cache_of_one_page_expanded(pages):
    """Pages that are all the same memory: the C side would read a stride of 0 as dense pages."""
    k, v = _t(1, 2, 16, 64).expand(pages, 2, 16, 64), _t(1, 2, 64, 16).expand(pages, 2, 64, 16)
    assert k.stride(0) == v.stride(0) == 0
    with pytest.raises(ValueError):
        _cache(k, v)
    overlapping = [torch.zeros(8192, dtype=BF).as_strided(s, (8, s[2] * s[3], s[3], 1)).as_subclass(_Gpu)
                   for s in ((3, 2, 16, 64), (3, 2, 64, 16))]
    with pytest.raises(ValueError):
        _cache(*overlapping)
    _cache(_t(1, 2, 16, 64), _t(1, 2, 64, 16))  # one page has no stride
    _cache(_t(5, 3, 2, 16, 64)[:, 1], _t(5, 3, 2, 64, 16)[:, 1])  # a layer's slice of a larger allocation


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 21, dtype=torch.uint8)[::2]])
def test_workspace_that_is_not_dense(ws):
    """A workspace's size counts its elements, not the memory behind them."""
    ws = ws.as_subclass(_Gpu)
    i32 = torch.int32
    c = _cache(_t(3, 2, 16, 64), _t(3, 2, 64, 16))
    with pytest.raises(ValueError):
        fm.attn_decode(c, fm.AttnDecode(1.0), _t(1, 128), _t(1, 3, dtype=i32), _t(1, dtype=i32), 0, _t(1, 128), ws, stream=0)
    f32 = torch.float32
    with pytest.raises(ValueError):
        fm.token_logprobs(_t(1, 50000, dtype=f32), None, None, _t(1, dtype=f32), None, None, ws, stream=0)
