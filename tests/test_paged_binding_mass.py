"""Which memory the calls with mass, prefixes and eviction keep for another stream, with stand-ins on the CPU."""
import types

import torch

from compressed_kv_cache_vector_gb300 import binding as K
from tests.test_paged_binding import OTHER, CPU, _batch, _kept, _t, kv  # noqa: F401


def _mass(kv):  # noqa: F811
    return types.SimpleNamespace(mass=_t(1, 4, 2, 16, dtype=torch.float32), shape=(1, 4, 2, 16), device=CPU, scratch_bytes=64,
                                 scratch=_t(64, dtype=torch.uint8))


def test_everything_is_kept_for_the_stream(kv, monkeypatch):  # noqa: F811
    monkeypatch.setattr(K, "_dev_i32", lambda t, name, device=None: None)
    s, lse = kv.stream_of(OTHER), _t(2, 4, dtype=torch.float32)
    b, q, out, m = _batch(), _t(2, 4, 128), _t(2, 4, 128), _mass(kv)
    kv.decode_attn_mass(0, b, q, m, out=out, lse=lse, stream=s)
    assert kv.calls[-1][0] == "mk_paged_decode_attn_mass" and kv.calls[-1][1][-1] == OTHER
    for t in (b.kv_len, b.page_table, b.cu_new, q, out, lse, m.mass, m.scratch, kv.k_pool, kv.workspace):
        assert _kept(t) == {OTHER}
    b, q, lse, m = _batch(), _t(2, 4, 128), _t(2, 4, dtype=torch.float32), _mass(kv)
    kv.prefill_mass(0, b, q, lse, m, stream=s)
    assert kv.calls[-1][0] == "mk_paged_prefill_mass" and kv.calls[-1][1][-1] == OTHER
    for t in (b.kv_len, b.page_table, b.cu_new, q, lse, m.mass):
        assert _kept(t) == {OTHER}
    b, q, out = _batch(), _t(2, 4, 128), _t(2, 4, 128)
    p = types.SimpleNamespace(device=CPU, ref=None, cu_group=_t(2, dtype=torch.int32), prefix_len=_t(1, dtype=torch.int32))
    kv.prefix_attn(0, b, p, q, out=out, stream=s)
    assert kv.calls[-1][0] == "mk_paged_prefix_attn" and kv.calls[-1][1][-1] == OTHER
    for t in (b.kv_len, b.page_table, q, out, p.cu_group, p.prefix_len):
        assert _kept(t) == {OTHER}
    b, m, keep = _batch(), _mass(kv), _t(2, dtype=torch.int32)
    b.n_seqs = 2
    kept, new = _t(2, 2, 8, dtype=torch.int32), _t(2, dtype=torch.int32)
    assert kv.evict(0, b, m, keep, kept=kept, new_len=new, stream=s) == (new, kept)
    assert kv.calls[-1][0] == "mk_paged_evict" and kv.calls[-1][1][-1] == OTHER
    for t in (b.kv_len, b.page_table, m.mass, keep, kept, new):
        assert _kept(t) == {OTHER}


def test_nothing_is_recorded_on_the_current_stream(kv):  # noqa: F811
    b, q, out, m = _batch(), _t(2, 4, 128), _t(2, 4, 128), _mass(kv)
    kv.decode_attn_mass(0, b, q, m, out=out)
    for t in (b.kv_len, q, out, m.mass, m.scratch, kv.workspace):
        assert not _kept(t)


def test_the_mass_is_kept_for_a_stream_that_became_the_current_one(kv):  # noqa: F811
    b, q, out, m = _batch(), _t(2, 4, 128), _t(2, 4, 128), _mass(kv)
    kv.decode_attn_mass(0, b, q, m, out=out)
    kv.set_current(OTHER)
    kv.decode_attn_mass(0, b, q, m, out=out)
    kv.decode_attn_mass(0, b, q, m, out=out, stream=kv.stream_of(OTHER))
    assert m.mass.streams == m.scratch.streams == [OTHER] and not _kept(q)
