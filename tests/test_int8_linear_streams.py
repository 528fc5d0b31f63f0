"""Int8Linear on a stream that is not the current one: the copy of an x that does not flatten to rows and the
memory of the result belong to the stream of the kernels, and both streams are recorded on what outlives the call.

The order is tested on the CPU (torch operations and the call recorded, no GPU); the GPU test keeps the
current stream busy, so that a copy left on it would come after the kernels that read it."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import oracle
import precision_quantized_attention_b200 as qa


def _layer(N, K, tokens):
    layer = object.__new__(qa.Int8Linear)
    layer.out_features, layer.in_features, layer.max_tokens, layer.bias = N, K, tokens, None
    layer.w8, layer.s_w = torch.zeros(N, K, dtype=torch.int8), torch.ones(N)
    layer._x8, layer._s_x = torch.zeros(tokens, K, dtype=torch.int8), torch.ones(tokens)
    return layer


class _Record(TorchDispatchMode):
    def __init__(self, where):
        super().__init__()
        self.where, self.ops = where, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.ops.append((func.overloadpacket.__name__, self.where[-1]))
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("given", [False, True])
def test_copy_result_and_kernels_share_the_given_stream(monkeypatch, given):
    where, kept, calls = ["current"], [], []

    @contextlib.contextmanager
    def on(stream):
        where.append(stream)
        yield
        where.pop()

    def linear(x, *rest):
        calls.append((where[-1], x.is_contiguous(), rest[6:] in ((), (None,))))

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: where[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t.data_ptr(), s)), raising=False)
    monkeypatch.setattr(qa, "linear_int8", linear)
    layer = _layer(16, 32, 64)
    x = torch.zeros(2, 20, 32, dtype=torch.bfloat16)[:, 3:13]        # batch rows do not flatten: a copy
    out = torch.zeros(2, 10, 16, dtype=torch.bfloat16) if given else None
    with _Record(where) as log:
        y = layer(x, out=out, stream="side")
    assert calls == [("side", True, True)]
    made = [w for name, w in log.ops if name in ("clone", "_to_copy", "copy_", "empty", "empty_strided", "contiguous")]
    assert made and set(made) == {"side"}
    assert {s for p, s in kept if p == x.data_ptr()} == {"side", "current"}
    assert {s for p, s in kept if p == y.data_ptr()} == {"side", "current"}
    kept.clear()
    calls.clear()
    layer(x)                                                         # the current stream: nothing to record
    layer(x, stream="current")
    assert [c[0] for c in calls] == ["current"] * 2 and not kept


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 20, 100])
def test_a_copied_input_on_a_side_stream(tokens):
    K, N, B = 512, 384, 2
    g = torch.Generator().manual_seed(tokens)
    whole = torch.randn(B, tokens + 3, K, generator=g).to(torch.bfloat16).cuda()
    layer = qa.Int8Linear((torch.randn(N, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda(), max_tokens=B * tokens)
    x = whole[:, 1:tokens + 1]
    want = layer(x.contiguous())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(4):
        torch.cuda._sleep(20_000_000)                                # about 10 ms of the current stream
        y = layer(x, stream=side)
        side.synchronize()
        with torch.cuda.stream(side):
            assert torch.equal(y, want)
        del y
        busy = torch.full((B, tokens, K), float(i), dtype=torch.bfloat16, device="cuda")
        assert bool((busy == i).all())
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    assert layer(x, out=out, stream=side) is out
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    xc, xs = oracle.quantize_int8_rows(x.reshape(-1, K).double().cpu().numpy())
    ref, size = oracle.gemm_int8(xc, layer.w8.cpu().numpy(), xs, layer.s_w.double().cpu().numpy())
    off = abs(want.view(-1, N).double().cpu().numpy() - ref)
    assert (off <= 2.0 ** -8 * abs(ref) + 5 * 2.0 ** -24 * size).all()
    assert qa.get_error() == 0


@pytest.mark.gpu
def test_a_copied_input_on_a_side_stream_of_a_capture():
    K, N, B, tokens = 256, 96, 3, 9
    g = torch.Generator().manual_seed(1)
    whole = torch.randn(B, tokens + 2, K, generator=g).to(torch.bfloat16).cuda()
    layer = qa.Int8Linear((torch.randn(N, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda(), max_tokens=64)
    x = whole[:, :tokens]
    want = layer(x.contiguous())
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        y = layer(x, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        z = y + 1
    for scale in (1.0, -3.0):
        whole.mul_(scale)
        graph.replay()
        want = layer(x.contiguous())
        assert torch.equal(y, want) and torch.equal(z, want + 1)
    assert qa.get_error() == 0
