"""kg_requant on a stream of its own, on the CPU: what it makes is that stream's memory, by a
model of torch's allocator that notes the stream a tensor is made on."""
from contextlib import contextmanager

import torch

import fp8_grouped_gemm_tn_amd as kg
from fp8_grouped_gemm_tn_amd import _binding


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_made_on_the_given_stream(monkeypatch):
    here, side = Stream(11), Stream(22)
    now, made, recorded = [here], [], []
    empty = torch.empty

    @contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    def new(*args, **kw):
        t = empty(*args, **kw)
        made.append((now[-1], t))
        return t

    monkeypatch.setattr(torch, "empty", new)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t, s)))
    monkeypatch.setattr(_binding, "_tensors_on_gpu", lambda *a, **kw: None)
    monkeypatch.setattr(_binding, "kg_requant_raw", lambda *a: kg.KG_OK)
    X, ks = torch.zeros(6, 128, dtype=torch.bfloat16), torch.tensor([4, 2], dtype=torch.int32)
    out = kg.kg_requant(X, None, ks, 128, kg.KG_E4M3_F32SCALE, 2, stream=side)
    assert [s for s, _ in made] == [side, side]
    assert [s for _, s in recorded] == [here, here]
    assert all(a is t and b is t for a, (_, t), (b, _) in zip(out, made, recorded))
    made.clear(), recorded.clear()
    kg.kg_requant(X, None, ks, 128, kg.KG_E4M3_F32SCALE, 2)
    assert [s for s, _ in made] == [here, here] and not recorded
