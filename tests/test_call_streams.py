"""Where the bindings allocate what they make themselves, on the CPU: a fake of
torch's allocator and streams under the real bindings, and a library that
launches nothing."""
import contextlib
import types

import pytest
import torch

from trained_kv_prefix_gb300 import cartattn as ca

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Device:
    type, index = "cuda", 0


DEVICE = Device()


class Tensor:
    """A tensor of the fake allocator: the stream whose memory it is, and the
    streams that it is kept for beside that one."""

    def __init__(self, shape, dtype, home=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, DEVICE
        self.home, self.kept_for = home, set()

    def record_stream(self, s):
        self.kept_for.add(s)

    def data_ptr(self):
        return 1 << 20

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def stride(self, i):
        return self.shape[i + 1:].numel()

    def __getitem__(self, i):
        return self


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, DEVICE


class Torch:
    """The part of torch that the bindings use, for one device."""

    bfloat16, float32, int32, uint8, Tensor = BF, F32, I32, torch.uint8, Tensor

    def __init__(self):
        self.made = []
        self.now = self.default = Stream(7)
        self.cuda = types.SimpleNamespace(
            current_device=lambda: 0, current_stream=lambda device=None: self.now,
            stream=self.on, device=lambda d: contextlib.nullcontext())

    @contextlib.contextmanager
    def on(self, s):
        was, self.now = self.now, s
        yield
        self.now = was

    def empty(self, *shape, dtype=None, device=None):
        shape = shape[0] if isinstance(shape[0], tuple) else shape
        self.made.append(Tensor(shape, dtype, self.now))
        return self.made[-1]

    zeros = empty

    def empty_like(self, t):
        return self.empty(tuple(t.shape), dtype=t.dtype)


class Library:
    """Every entry point succeeds; a size is 4096 bytes."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("_size") else 0


@pytest.fixture
def fake(monkeypatch):
    t = Torch()
    monkeypatch.setattr(ca, "torch", t)
    monkeypatch.setattr(ca, "_lib", Library())
    monkeypatch.setattr(ca, "lib", Library)
    monkeypatch.setattr(ca, "_raw_stream", lambda index: t.now.cuda_stream)
    sizes = (ca.decode_tree_workspace_size, ca.pages_workspace_size)
    for f in sizes:
        f.cache_clear()
    yield t
    for f in sizes:
        f.cache_clear()


def new(*shape, dtype=BF):
    return Tensor(shape, dtype)


def ints(*shape):
    return Tensor(shape, I32)


def pools():
    return new(2, 8, 16, 2, 64), new(2, 8, 16, 2, 64)


PAGED = {
    "tree": lambda **kw: ca.cart_attn_decode_tree(
        new(3, 4, 8, 64), new(3, 4, 2, 64), new(3, 4, 2, 64), new(5, 2, 64), new(5, 2, 64),
        new(8, 16, 2, 64), new(8, 16, 2, 64), ints(3, 2), ints(3), ints(3, 4), **kw),
    "fork": lambda **kw: ca.cart_pages_fork(ints(3, 2), ints(3), ints(8), ints(2), ints(2),
                                            page_rows=16, **kw),
    "reserve": lambda **kw: ca.cart_pages_reserve(*pools(), ints(3, 2), ints(3), ints(8), ints(3),
                                                  **kw),
    "accept": lambda **kw: ca.cart_pages_accept(*pools(), ints(3, 2), ints(3), 4, ints(3), **kw),
    "compact": lambda **kw: ca.cart_pages_compact(*pools(), ints(3, 2), ints(8), **kw),
}


def leaves():
    return new(5, 2, 64, dtype=F32), new(5, 2, 64, dtype=F32)


def seqs():
    return new(3, 4, 8, 64), new(3, 4, 2, 64), new(3, 4, 2, 64)


def packed():
    return new(12, 8, 64), new(12, 2, 64), new(12, 2, 64)


DENSE = {
    "fwd": lambda **kw: ca.cart_attn_fwd(*seqs(), *leaves(), **kw),
    "bwd": lambda **kw: ca.cart_attn_bwd(*seqs(), *leaves(), seqs()[0], new(3, 8, 4, dtype=F32),
                                         seqs()[0], accumulate=True, **kw),
    "bwd_parts": lambda **kw: ca.cart_attn_bwd(*seqs(), *leaves(), seqs()[0],
                                               new(3, 8, 4, dtype=F32), seqs()[0],
                                               frozen_rows=[2], **kw),
    "bwd_reuse": lambda **kw: ca.cart_attn_bwd(*seqs(), *leaves(), seqs()[0],
                                               new(3, 8, 4, dtype=F32), seqs()[0],
                                               fwd_workspace=new(99, dtype=torch.uint8), **kw),
    "fwd_packed": lambda **kw: ca.cart_attn_fwd_packed(*packed(), *leaves(), ints(4), 4, **kw),
    "bwd_packed": lambda **kw: ca.cart_attn_bwd_packed(*packed(), *leaves(), packed()[0],
                                                       new(8, 12, dtype=F32), packed()[0], ints(4),
                                                       4, accumulate=True, **kw),
    "decode": lambda **kw: ca.cart_attn_decode(new(3, 8, 64), new(3, 2, 64), new(3, 2, 64),
                                               new(5, 2, 64), new(5, 2, 64), new(3, 9, 2, 64),
                                               new(3, 9, 2, 64), ints(3), **kw),
    "decode_span": lambda **kw: ca.cart_attn_decode_span(*seqs(), new(5, 2, 64), new(5, 2, 64),
                                                         new(3, 9, 2, 64), new(3, 9, 2, 64),
                                                         ints(3), **kw),
}


def check(fake, call):
    """All that the call makes is memory of the stream that its kernels run on;
    what it returns, and that alone, is kept for the caller's current stream
    too, which reads it later."""
    side = Stream(9)
    out = call(stream=side)
    out = out if isinstance(out, tuple) else (out,)
    assert fake.made and all(t.home is side for t in fake.made)
    assert all(t.kept_for == ({fake.default} if t in out else set()) for t in fake.made)
    assert fake.now is fake.default
    # on the current stream, named or not, memory is that stream's
    for kw in ({}, {"stream": fake.default}):
        del fake.made[:]
        call(**kw)
        assert fake.made and all(t.home is fake.default for t in fake.made)


@pytest.mark.parametrize("name", PAGED)
def test_paged_calls_allocate_on_their_stream(fake, name):
    check(fake, PAGED[name])


@pytest.mark.parametrize("name", DENSE)
def test_dense_calls_allocate_on_their_stream(fake, name):
    check(fake, DENSE[name])


@pytest.mark.parametrize("name", PAGED)
def test_paged_calls_refuse_a_stream_of_another_device(fake, name):
    other = Stream(9)
    other.device = Device()
    with pytest.raises(ValueError):
        PAGED[name](stream=other)
    assert not fake.made and fake.now is fake.default
