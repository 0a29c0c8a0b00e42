"""PagedKV's calls on another stream than the current one, without a GPU: the library, the streams and the allocator's
record_stream are stand-ins, and the test looks at which memory is kept for which stream."""
import types

import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K

HERE, OTHER = 111, 222      # the current stream's handle, and another one's
CPU = torch.device("cpu")


class _Kept(torch.Tensor):
    """A tensor that notes the streams it is kept for."""

    def record_stream(self, stream):
        if not hasattr(self, "streams"):
            self.streams = []
        self.streams.append(stream.cuda_stream)


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_Kept)


def _kept(t):
    return set(getattr(t, "streams", []))


@pytest.fixture
def kv(monkeypatch):
    current = [HERE]
    stream = lambda raw: types.SimpleNamespace(cuda_stream=raw, device=CPU)  # noqa: E731
    monkeypatch.setattr(K, "_raw_stream", lambda index: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream(current[0]))
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0

    cfg = K.make_paged_config(4, 2, 1, 16, 4, 2)
    c = K.PagedKV.__new__(K.PagedKV)
    c.lib, c.cfg, c.device, c.h, c.dtype = Lib(), cfg, CPU, None, torch.float8_e4m3fn
    c.k_pool, c.v_pool = (_t(1, 4, 2, 16, 128, dtype=torch.float8_e4m3fn) for _ in range(2))
    c.k_scale, c.v_scale = (_t(1, 4, 2, dtype=torch.float32) for _ in range(2))
    c.workspace = _t(64, dtype=torch.uint8)
    c.q_row, c.kv_row = 512, 256
    if hasattr(K.PagedKV, "_remember_streams"):
        c._remember_streams()
    c.calls, c.set_current, c.stream_of = calls, lambda raw: current.__setitem__(0, raw), stream
    return c


def _batch():
    i32 = torch.int32
    return types.SimpleNamespace(device=CPU, n_tokens=2, ref=None, kv_len=_t(2, dtype=i32), page_table=_t(2, 2, dtype=i32),
                                 cu_new=_t(3, dtype=i32))


def _rope():
    return types.SimpleNamespace(device=CPU, ref=None, table=_t(8, 128, dtype=torch.float32), positions=_t(2, dtype=torch.int32))


def _memory(kv):
    return [kv.k_pool, kv.v_pool, kv.k_scale, kv.v_scale, kv.workspace]


def test_everything_a_queued_call_reads_is_kept_for_its_stream(kv):
    b, rope, k, v, q, qo = _batch(), _rope(), _t(2, 2, 128), _t(2, 2, 128), _t(2, 4, 128), _t(2, 4, 128)
    lse = _t(2, 4, dtype=torch.float32)
    s = kv.stream_of(OTHER)
    kv.append(0, b, k, v, rope=rope, q=q, q_out=qo, stream=s)
    assert kv.calls[-1][1][-1] == OTHER
    for t in (b.kv_len, b.page_table, b.cu_new, rope.table, rope.positions, k, v, q, qo, *_memory(kv)):
        assert _kept(t) == {OTHER}
    for call in (kv.decode_attn, kv.prefill_attn):
        b, q, out = _batch(), _t(2, 4, 128), _t(2, 4, 128)
        call(0, b, q, out=out, lse=lse, stream=s)
        assert kv.calls[-1][1][-1] == OTHER
        for t in (b.kv_len, b.page_table, b.cu_new, q, out, lse):
            assert _kept(t) == {OTHER}


def test_nothing_is_recorded_on_the_current_stream_and_the_cache_once_for_each_other(kv):
    b, q, out = _batch(), _t(2, 4, 128), _t(2, 4, 128)
    kv.decode_attn(0, b, q, out=out)
    kv.decode_attn(0, b, q, out=out, stream=kv.stream_of(HERE))
    assert kv.calls[-1][1][-1] == HERE
    for t in (b.kv_len, b.page_table, b.cu_new, q, out, *_memory(kv)):
        assert not _kept(t)
    # Another stream made current: its tensors are the caller's, as with torch's own calls, the cache's memory is not.
    kv.set_current(OTHER)
    for _ in range(3):
        kv.decode_attn(0, b, q, out=out)
    assert all(t.streams == [OTHER] for t in _memory(kv)) and not _kept(q) and not _kept(b.kv_len)


def test_new_outputs_belong_to_the_stream_that_writes_them(kv, monkeypatch):
    made = []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            kv.set_current(self.stream.cuda_stream)

        def __exit__(self, *a):
            kv.set_current(HERE)

    def empty(*shape, dtype, device):
        t = torch.zeros(*shape, dtype=dtype, device=device).as_subclass(_Kept)
        made.append((t, K._raw_stream(None)))
        return t

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch, "empty", empty)
    b, q, k = _batch(), _t(2, 4, 128), _t(2, 2, 128)
    for stream, raw in ((None, HERE), (kv.stream_of(HERE), HERE), (kv.stream_of(OTHER), OTHER)):
        outs = [kv.append(0, b, k, k, q=q, stream=stream), *kv.decode_attn(0, b, q, lse=True, stream=stream),
                *kv.prefill_attn(0, b, q, lse=True, stream=stream)]
        assert [t.data_ptr() for t in outs] == [t.data_ptr() for t, _ in made]
        assert all(on == raw for _, on in made)
        if raw == OTHER:
            assert all(HERE in _kept(t) for t in outs)     # and kept for the caller's stream, which will read them
        made.clear()
