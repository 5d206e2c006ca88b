"""Memory that the binding allocates for work on a stream belongs to that stream.

torch's allocator hands a freed block out again to the stream it was allocated
on, as soon as the host has let go of it: in the order of that stream's work, and
of no other's.  So what a call writes on `stream` has to come from `stream`'s own
blocks, and what it returns is kept from reuse until the caller's stream is done
with it.  Without a GPU: torch's streams and the library are stand-ins that note
what is done on which stream."""
import contextlib

import pytest
import torch
from torch.overrides import TorchFunctionMode

CALLER = "the caller's stream"


class Library:
    """Every call succeeds; sizes are 4,096 bytes."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("_bytes") else 0


class Notes(TorchFunctionMode):
    ALLOCATE = ("empty", "empty_like", "new_empty")

    def __init__(self, world):
        super().__init__()
        self.world, self.allocated, self.filled = world, [], []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        name = getattr(func, "__name__", "")
        out = func(*args, **(kwargs or {}))
        if name in self.ALLOCATE and out.numel():
            self.allocated.append((out.untyped_storage().data_ptr(), self.world["stream"]))
        if name == "zero_":
            self.filled.append(self.world["stream"])
        return out


@pytest.fixture
def q(monkeypatch):
    from bit_kv_cache_qvg_b200 import qvg
    world = dict(stream=CALLER, kept=[])

    @contextlib.contextmanager
    def on(s):
        before, world["stream"] = world["stream"], s
        yield
        world["stream"] = before

    monkeypatch.setattr(qvg, "lib", Library)
    monkeypatch.setattr(qvg, "_on_device", lambda *t: torch.device("cpu"))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: world["stream"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: f"stream {handle}")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "stream 0")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: world["kept"].append((t.untyped_storage().data_ptr(), s)))
    qvg.world = world
    yield qvg
    del qvg.world


class Side:
    cuda_stream = 77


def calls(q):
    cfg = q.config(K=16, T=1, group_size=64)
    kp, vp = q.alloc_packed(cfg, 100, 2, device="cpu"), q.alloc_packed(cfg, 100, 2, device="cpu")
    Q, pos = torch.zeros((1, 4, 3, 128), dtype=torch.bfloat16), torch.zeros((1, 3), dtype=torch.int64)
    tables, w, X = torch.zeros(256 + 512 * 200, dtype=torch.uint8), torch.zeros((2, 100)), torch.zeros((2, 100, 128))
    return dict(
        attention_batch=lambda s: q.attention_batch(kp, vp, Q, pos, tables, stream=s),
        attention_weights=lambda s: q.attention_weights(kp, Q, pos, tables, stream=s),
        evict=lambda s: q.evict(kp, vp, w, 40, stream=s),
        quantize=lambda s: q.quantize(X, cfg, stream=s),
        quantize_static=lambda s: q.quantize_static(X, cfg, stream=s),
        dequantize=lambda s: q.dequantize(kp, stream=s),
        rope_tables=lambda s: q.rope_tables(10, device="cpu", stream=s),
        attention=lambda s: q.attention(kp, vp, Q[0], pos[0], tables, stream=s),
    )


CALLS = ["attention_batch", "attention_weights", "evict", "quantize", "quantize_static", "dequantize", "rope_tables", "attention"]


def tensors(x):
    if isinstance(x, torch.Tensor):
        return [x] if x.numel() else []
    return [t for v in vars(x).values() if isinstance(v, torch.Tensor) or hasattr(v, "codes") for t in tensors(v)]


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [Side(), 78, 0], ids=["stream", "handle", "default"])
def test_memory_belongs_to_the_stream_of_the_work(q, name, stream):
    call = calls(q)[name]
    with Notes(q.world) as n:
        out = call(stream)
    want = f"stream {stream.cuda_stream if isinstance(stream, Side) else stream}"
    assert n.allocated and all(s == want for _, s in n.allocated)
    assert all(s == want for s in n.filled)
    # what is returned is kept until the caller's stream is done with it, the rest goes back at once
    made = {at for at, _ in n.allocated}
    returned = {t.untyped_storage().data_ptr() for t in tensors(out)} & made
    assert returned and {at for at, s in q.world["kept"] if s == CALLER} == returned
    assert q.world["stream"] == CALLER


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_it_is_the_current_one_s(q, name, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)
    monkeypatch.setattr(q, "_stream", lambda s: 0)
    call = calls(q)[name]
    with Notes(q.world) as n:
        call(None)
    assert n.allocated and all(s == CALLER for _, s in n.allocated)
    assert not q.world["kept"]
