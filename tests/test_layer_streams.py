"""Memory and streams of the expert layer's calls, on the CPU: torch's allocator and streams are
replaced by a model that knows which stream a block belongs to and which streams it is
recorded on, and the library by one that notes its calls."""
import types
from contextlib import contextmanager

import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
from fp8_grouped_gemm_tn_amd import layer


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Block(torch.Tensor):
    """A CPU tensor that says it is on GPU 0."""
    @staticmethod
    def of(t, owner):
        b = t.as_subclass(Block)
        b.owner, b.recorded = owner, set()
        return b

    def get_device(self):
        return 0

    def record_stream(self, stream):
        if stream is not self.owner:
            self.recorded.add(stream)


class Machine:
    """Streams, an allocator, and a library whose calls succeed."""
    def __init__(self):
        self.main = self.current = Stream(11)
        self.capturing, self.made, self.calls = set(), [], []

    @contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        try:
            yield
        finally:
            self.current = before

    def empty(self, shape, dtype=torch.float32, device=None):
        b = Block.of(torch.zeros(shape, dtype=dtype), self.current)
        self.made.append(b)
        return b

    def new(self, *shape, dtype=torch.float32):
        return Block.of(torch.zeros(shape, dtype=dtype), self.main)

    def __getattr__(self, name):  # the library
        if not name.startswith("kg_"):
            raise AttributeError(name)
        if name.endswith("_bytes"):
            return lambda *a: 64
        return lambda *a: self.calls.append((name, a[-1])) or 0


@pytest.fixture
def machine(monkeypatch):
    m = Machine()
    cuda = types.SimpleNamespace(stream=m.stream, current_stream=lambda device=None: m.current,
                                 is_current_stream_capturing=lambda: m.current in m.capturing)
    fake = types.SimpleNamespace(empty=m.empty, cuda=cuda, uint8=torch.uint8, bool=torch.bool)
    for name, value in dict(torch=fake, _lib=m, _f32=torch.float32, _bf16=torch.bfloat16,
                            _int32=torch.int32, _current_gpu=lambda: 0,
                            _row_types={torch.bfloat16: kg.KG_ROWS_BF16, torch.float32: kg.KG_ROWS_F32},
                            _current_stream=lambda gpu: m.current.cuda_stream).items():
        monkeypatch.setattr(layer, name, value)
    return m


def calls(m):
    """Every call that makes tensors, with nothing given that it can make."""
    i32, bf16 = torch.int32, torch.bfloat16
    T, k, H = 6, 2, 32
    pos = m.new(T, k, dtype=i32)
    X, Y = m.new(T, H, dtype=bf16), m.new(T * k, H, dtype=bf16)
    return dict(
        kg_route=lambda s: kg.kg_route(m.new(T, k, dtype=i32), m.new(3, dtype=i32), stream=s),
        kg_dispatch=lambda s: kg.kg_dispatch(X, pos, stream=s),
        kg_dispatch_fp8=lambda s: kg.kg_dispatch_fp8(X, pos, stream=s),
        kg_combine=lambda s: kg.kg_combine(Y, pos, stream=s),
        kg_combine_bwd=lambda s: kg.kg_combine_bwd(X, Y, pos, stream=s))


NAMES = ("kg_route", "kg_dispatch", "kg_dispatch_fp8", "kg_combine", "kg_combine_bwd")


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_gets_memory_of_its_own(machine, name):
    """What a call on another stream makes and writes is no memory of the current stream, whose
    queued work may still use what was freed there; what is handed back is not reused before
    the current stream is done with it."""
    side = Stream(22)
    back = calls(machine)[name](side)
    assert machine.calls == [(name, side.cuda_stream)]
    assert machine.made and all(b.owner is side for b in machine.made)
    for b in back if isinstance(back, tuple) else (back,):
        assert b.recorded == {machine.main}
    assert machine.current is machine.main


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_needs_no_record(machine, name):
    side = Stream(22)
    fns = calls(machine)
    with machine.stream(side):
        fns[name](None)
        fns[name](side)
    assert [s for _, s in machine.calls] == [side.cuda_stream] * 2
    assert all(b.owner is side and not b.recorded for b in machine.made)


def adamw_table(m, packed):
    n = 300
    f32, u8, bf16 = torch.float32, torch.uint8, torch.bfloat16
    lists = [[m.new(n), m.new(7)], [m.new(n, dtype=bf16), m.new(7, dtype=bf16)]]
    lists += [[m.new(n, dtype=u8 if packed else f32), m.new(7, dtype=u8 if packed else f32)] for _ in "mv"]
    scales = [[m.new(3), m.new(1)] for _ in "mv"] if packed else [None, None]
    table = kg.AdamWTable(*lists, *scales, [m.new(n, dtype=bf16), m.new(7, dtype=bf16)])
    m.calls.clear()
    return table, [x for xs in table.tensors for x in xs if x is not None] + [table.table]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_a_table_is_kept_for_the_streams_that_step(machine, packed, given):
    """The descriptors and what the table may be the last to keep are recorded on every stream
    that a step goes to, once, whether it is given or the current one."""
    table, kept = adamw_table(machine, packed)
    kg.kg_adamw(table, 1e-3)
    assert not any(x.recorded for x in kept)
    sides = [Stream(22), Stream(33)]
    for side in sides:
        for _ in range(2):
            if given:
                kg.kg_adamw(table, 1e-3, stream=side)
            else:
                with machine.stream(side):
                    kg.kg_adamw(table, 1e-3)
    assert [s for _, s in machine.calls] == [11, 22, 22, 33, 33]
    assert all(x.recorded == set(sides) for x in kept)


def test_a_captured_step_records_nothing_and_a_later_one_does(machine):
    table, kept = adamw_table(machine, True)
    side = Stream(22)
    machine.capturing.add(side)
    kg.kg_adamw(table, 1e-3, stream=side)
    assert not any(x.recorded for x in kept)
    machine.capturing.clear()
    kg.kg_adamw(table, 1e-3, stream=side)
    assert all(x.recorded == {side} for x in kept)
