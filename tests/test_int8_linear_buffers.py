"""Int8Linear layers that take turns share their activation buffers."""
import pytest
import torch

import precision_quantized_attention_b200 as qa


def _weight(N, K, seed):
    return (torch.randn(N, K, generator=torch.Generator().manual_seed(seed)) * K ** -0.5).to(torch.bfloat16)


def test_layers_share_memory_and_refuse_what_is_too_small(monkeypatch):
    monkeypatch.setattr(qa, "quantize_int8_rows", lambda *a, **k: None)      # no GPU here: the memory is looked at
    shared = qa.new_int8_buffers(40, 100, device="cpu")
    assert shared[0].dtype == torch.int8 and shared[0].numel() == 40 * 112 and shared[1].shape == (40,)
    a = qa.Int8Linear(_weight(8, 100, 0), max_tokens=40, buffers=shared)
    b = qa.Int8Linear(_weight(6, 33, 1), max_tokens=40, buffers=shared)
    for layer, K, ld in ((a, 100, 112), (b, 33, 48)):
        assert layer._x8.data_ptr() == shared[0].data_ptr() and layer._s_x.data_ptr() == shared[1].data_ptr()
        assert layer._x8.shape == (40, K) and layer._x8.stride() == (ld, 1) and layer._s_x.shape == (40,)
    qa.Int8Linear(_weight(6, 16, 1), max_tokens=40, buffers=shared)
    for K, tokens in ((113, 40), (100, 41), (16, 41)):
        with pytest.raises(ValueError, match="smaller"):
            qa.Int8Linear(_weight(4, K, 2), max_tokens=tokens, buffers=shared)
    own = [qa.Int8Linear(_weight(4, 64, 3), max_tokens=4) for _ in range(2)]
    assert own[0]._x8.data_ptr() != own[1]._x8.data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 17, 200])
def test_a_chain_of_layers_on_one_pair_of_buffers(tokens):
    widths = [200, 515, 96, 200]
    shared = qa.new_int8_buffers(256, max(widths))
    ws = [_weight(n, k, k).cuda() for k, n in zip(widths, widths[1:])]
    bias = torch.randn(widths[1], generator=torch.Generator().manual_seed(5)).cuda()
    make = lambda **kw: [qa.Int8Linear(w, bias if i == 0 else None, max_tokens=256, **kw) for i, w in enumerate(ws)]
    x = torch.randn(tokens, widths[0], generator=torch.Generator().manual_seed(tokens)).to(torch.bfloat16).cuda()

    def chain(layers):
        y = x
        for layer in layers:
            y = layer(y)
        return y

    alone, together = make(), make(buffers=shared)
    want = chain(alone)
    for _ in range(5):
        assert torch.equal(chain(together), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = chain(together)
    y.zero_()
    chain(together)
    graph.replay()
    assert torch.equal(y, want)
    assert qa.get_error() == 0
