"""What a PagedMass does with memory that its maker brings or that another stream had before, with stand-ins on the CPU."""
import contextlib
import types

import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from tests.test_paged_binding import CPU, HERE, OTHER, _batch, _kept, _t, kv  # noqa: F401


@pytest.mark.parametrize("given", [True, False])
def test_scratch_is_handed_out_when_the_current_stream_is_done(kv, monkeypatch, given):  # noqa: F811
    """Whatever is queued may still use the memory that the scratch is given, whoever made the mass."""
    done = []
    empty = torch.empty
    monkeypatch.setattr(K.torch, "empty", lambda *a, **k: done.append("scratch") or empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(
        cuda_stream=HERE, synchronize=lambda: done.append("waited")))
    m = K.PagedMass(kv, _t(1, 4, 2, 16, dtype=torch.float32) if given else None)
    assert done == ["scratch", "waited"]
    assert _kept(m.mass) == ({HERE} if given else set())


def test_a_given_mass_is_kept_for_every_stream_that_uses_it(kv, monkeypatch):  # noqa: F811
    stream = torch.cuda.current_stream
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(
        cuda_stream=stream().cuda_stream, synchronize=lambda: None))
    m = K.PagedMass(kv, _t(1, 4, 2, 16, dtype=torch.float32))
    b, q, out = _batch(), _t(2, 4, 128), _t(2, 4, 128)
    m.scratch = _t(64, dtype=torch.uint8)
    kv.decode_attn_mass(0, b, q, m, out=out)
    assert m.mass.streams == [HERE]
    kv.decode_attn_mass(0, b, q, m, out=out, stream=kv.stream_of(OTHER))
    assert _kept(m.mass) == {HERE, OTHER} and _kept(m.scratch) == {OTHER}
    assert m.device == CPU


def test_given_pools_are_kept_for_the_stream_they_are_given_on(monkeypatch):
    """They may have been allocated on another stream than the one that the cache is made and used on."""
    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(K, "load", Lib)
    monkeypatch.setattr(K, "paged_sizes", lambda cfg: (0, 0, 64))
    monkeypatch.setattr(K, "_raw_stream", lambda index: HERE)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=HERE))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    cfg = K.make_paged_config(4, 2, 1, 16, 4, 2)
    pools = [_t(1, 4, 2, 16, 128, dtype=torch.float8_e4m3fn) for _ in range(2)]
    scales = [_t(1, 4, 2, dtype=torch.float32) for _ in range(2)]
    c = K.PagedKV(cfg, "cpu", *pools, *scales)
    for t in (*pools, *scales):
        assert _kept(t) == {HERE}
    mine = K.PagedKV(cfg, "cpu", k_pool=pools[0])
    assert mine.k_pool is pools[0] and c.v_pool is pools[1] and not _kept(mine.v_pool)
