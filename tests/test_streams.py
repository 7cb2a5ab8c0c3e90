"""What a call with stream= allocates comes out of that stream's memory (no GPU: the allocator and the library are
stand-ins that write down what is asked of them)."""
import contextlib
import inspect

import pytest
import torch


@pytest.fixture()
def kda(monkeypatch):
    from gated_delta_rule_155_b200 import build

    build.build()
    from gated_delta_rule_155_b200 import kda as k

    return k


class Result(torch.Tensor):
    def record_stream(self, stream):
        RECORDED.append((self.born, stream))


RECORDED = []


class Stream:
    cuda_stream = 7


class Library:
    """Entry points that answer KDA_OK and leave 1024 in a size argument."""

    def __getattr__(self, name):
        def call(*a):
            if name.endswith("workspace_size"):
                a[-1]._obj.value = 1024
            return 0
        return call


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Result)


def calls():
    """Every entry point that takes a stream, with arguments that leave all its buffers to be allocated."""
    B, T, H, d = 2, 3, 2, 64
    q, g2, s = zeros(B, T, H, d), zeros(B, T, H), zeros(B, H, d, d)
    p, pg, cu = zeros(B * T, H, d), zeros(B * T, H), zeros(B + 1, dtype=torch.int32)
    raw, conv, heads = zeros(B, T, H * d), zeros(H * d, 4), zeros(H)
    cache, refs, ids = zeros(1, 4, 8), zeros(4, dtype=torch.int32), zeros(2, dtype=torch.int32)
    taps = zeros(B, 3, H * d)
    return {
        "kda_forward_chunked": (q, q, q, q, g2),
        "kda_forward_chunked_varlen": (p, p, p, p, pg, cu),
        "kda_backward_chunked": (q, q, q, q, g2, q),
        "kda_decode_step": (s[:, :, 0], s[:, :, 0], s[:, :, 0], s[:, :, 0], s[:, :, 0, 0], s),
        "kda_layer_forward": (raw, raw, raw, conv, conv, conv, q, heads, None, g2, q),
        "kda_layer_forward_varlen": (raw[0], raw[0], raw[0], conv, conv, conv, q[0], heads, None, g2[0], q[0], cu),
        "kda_layer_decode_step": (raw[:, 0], raw[:, 0], raw[:, 0], conv, conv, conv, taps, taps, taps, q[:, 0], heads, None,
                                  g2[:, 0], q[:, 0], s),
        "kda_layer_forward_noalloc": (raw, raw, raw, conv, conv, conv, q, heads, None, g2, q),
        "kda_gdr_forward": (q, q, q, g2, g2),
        "kda_gdr_backward": (q, q, q, g2, g2, q),
        "kda_gdr_decode": (q, q, q, g2, g2, s),
        "kda_pages_fork": (cache, refs, ids),
        "kda_pages_copy": (cache, ids, ids),
        "kda_pages_free": (refs, ids),
        "kda_pages_compact": (cache, refs),
    }


def test_what_a_call_on_a_stream_allocates_is_that_streams(kda, monkeypatch):
    side, main, where = Stream(), Stream(), []

    @contextlib.contextmanager
    def on(stream):
        where.append(stream)
        yield
        where.pop()

    born = []

    def made_by(make):
        def f(*a, **kw):
            kw.pop("device", None)
            t = make(*a, **kw).as_subclass(Result)
            t.born = where[-1] if where else main
            born.append(t.born)
            return t
        return f

    for name, value in (("empty", made_by(torch.empty)), ("empty_like", made_by(torch.empty_like))):
        monkeypatch.setattr(torch, name, value)
    monkeypatch.setattr(kda, "_empty", made_by(kda._empty))
    monkeypatch.setattr(kda, "_lib", Library())
    monkeypatch.setattr(kda, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(kda, "_need_all", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: main)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw: {7: side}[raw])
    for f in (kda.kda_gdr_workspace_size, kda.kda_pages_workspace_size):
        f.cache_clear()
    try:
        entries = calls()
        named = {n for n, f in vars(kda).items() if n.startswith("kda_") and "stream" in inspect.signature(f).parameters}
        assert named - {"kda_check_device_error"} == set(entries)
        for name, args in entries.items():
            born.clear()
            RECORDED.clear()
            for t in args:
                if t is not None:
                    t.born = main
            got = getattr(kda, name)(*args, stream=side)
            assert all(b is side for b in born), name
            given = 0 if name in ("kda_pages_copy", "kda_pages_free") else 1
            assert len(born) >= given, name
            # what the caller gets is kept until the current stream, where it may be read, has passed its end
            got = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
            for t in got:
                if t is not None and t.born is side:
                    assert (side, main) in RECORDED, name
    finally:
        for f in (kda.kda_gdr_workspace_size, kda.kda_pages_workspace_size):
            f.cache_clear()
