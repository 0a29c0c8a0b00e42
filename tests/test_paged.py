"""The paged cache on the CPU: its 64-bit oracle against torch's own e4m3 and hand cases, the configuration's sizes,
and every refusal that happens before a launch."""
import ctypes
import math

import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300 import build as B
from oracle import paged_oracle as O


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.load()


def test_oracle_e4m3_is_the_nearest_value_with_ties_to_even():
    vals = torch.tensor(O.e4m3_values(), dtype=torch.float64)
    assert float(vals[-1]) == 448.0
    assert torch.equal(O.e4m3_round(vals), vals)
    mid = (vals[1:] + vals[:-1]) / 2
    even = torch.where(torch.arange(126) % 2 == 0, vals[:-1], vals[1:])
    assert torch.equal(O.e4m3_round(mid), even)
    x = torch.randn(20000, dtype=torch.float64, generator=torch.Generator().manual_seed(1)).float() * 60
    x = x.clamp(-448, 448)
    assert torch.equal(O.e4m3_round(x.double()), x.to(torch.float8_e4m3fn).double())
    tiny = x * 2.0 ** -14
    assert torch.equal(O.e4m3_round(tiny.double()), tiny.to(torch.float8_e4m3fn).double())


def test_oracle_scale_and_page_growth_by_hand():
    assert O.scale_of(448.0) == 1.0 and O.scale_of(448.0001) == 2.0 and O.scale_of(224.0) == 0.5
    assert O.scale_of(0.0) == 2.0 ** -64
    page = torch.zeros(4, 128, dtype=torch.float64)
    a = torch.zeros(1, 128, dtype=torch.float64)
    a[0, :3] = torch.tensor([448.0, 1.0, 2.0 ** -9])
    page, s = O.append_page(page, 7.0, a, 0)          # a page written from slot 0 forgets its scale
    assert s == 1.0 and page[0, :3].tolist() == [448.0, 1.0, 2.0 ** -9]
    b = torch.full((1, 128), 900.0, dtype=torch.float64)
    page, s = O.append_page(page, s, b, 1)            # scale 4: 448 -> 112, 1 -> 0.25, 2^-9 -> a tie at 0.25 steps -> 0
    assert s == 4.0 and page[0, :3].tolist() == [112.0, 0.25, 0.0] and page[1, 0] == 224.0


def test_oracle_attention_by_hand():
    q = torch.zeros(2, 128, dtype=torch.float64)
    q[:, 0] = math.log(3.0)
    k = torch.zeros(2, 128, dtype=torch.float64)
    k[1, 0] = 1.0
    v = torch.zeros(2, 128, dtype=torch.float64)
    v[0, 0], v[1, 0] = 4.0, 8.0
    out, lse, _, _ = O.attention(q, k, v, 1.0, torch.tensor([2, 0]))
    assert abs(float(out[0, 0]) - 7.0) < 1e-12 and abs(float(lse[0]) - math.log(4.0)) < 1e-12
    assert float(out[1, 0]) == 0.0 and float(lse[1]) == -math.inf


def _cfg(**kw):
    base = dict(n_q_heads=32, n_kv_heads=8, n_layers=2, page=32, n_pages=100, max_seqs=16, kv_type=K.MK_KV_E4M3)
    base.update(kw)
    return K.make_paged_config(**base)


def test_sizes(lib):
    p, s, w = K.paged_sizes(_cfg())
    assert p == 2 * 100 * 8 * 32 * 128 and s == 2 * 100 * 8 * 4 and w > 0
    p, s, _ = K.paged_sizes(_cfg(kv_type=K.MK_KV_BF16))
    assert p == 2 * 2 * 100 * 8 * 32 * 128 and s == 0


@pytest.mark.parametrize("bad", [dict(page=8), dict(page=48), dict(n_q_heads=24), dict(n_q_heads=128), dict(n_pages=0),
                                 dict(max_seqs=0), dict(max_seqs=257), dict(kv_type=2), dict(n_layers=0),
                                 dict(n_kv_heads=0)])
def test_bad_configs_rejected(lib, bad):
    with pytest.raises(K.MosaicKVError) as e:
        K.paged_sizes(_cfg(**bad))
    assert e.value.status == 1


def test_create_refuses_before_touching_the_device(lib):
    cfg = _cfg()
    h = ctypes.c_void_p()
    good, odd, n = 1 << 20, (1 << 20) + 16, K.paged_sizes(cfg)[2]

    def create(c=cfg, k=good, v=good, ks=good, vs=good, ws=good, size=n):
        return lib.mk_paged_create(ctypes.byref(c), k, v, ks, vs, ws, size, ctypes.byref(h))

    assert create(k=0) == 1 and create(v=odd) == 1 and create(ws=odd) == 1
    assert create(ks=0) == 1 and create(vs=0) == 1 and create(ks=good + 2) == 1
    assert create(size=n - 1) == 2
    assert create(c=_cfg(kv_type=K.MK_KV_BF16)) == 1          # scales given to a bf16 cache
    assert lib.mk_paged_append(None, 0, None, None, good, 1024, good, 1024, None, 0, None, 0, None) == 1
    assert lib.mk_paged_decode_attn(None, 0, None, good, 4096, 1.0, good, 4096, None, None) == 1
    assert lib.mk_paged_prefill_attn(None, 0, None, 1, good, 4096, 1.0, good, 4096, None, None) == 1
    assert lib.mk_paged_poll_error(None, None) == 1 and lib.mk_paged_clear_error(None) == 1


def test_binding_refuses_host_tensors(lib):
    with pytest.raises(ValueError):
        K.PagedBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        K.Rope(torch.zeros(4, 128), 128)


def test_rope_table_on_the_cpu():
    t = K.rope_table(5, 64, base=100.0, device="cpu")
    assert t.shape == (5, 64) and t.dtype == torch.float32
    for i in (0, 7, 31):
        a = 3 * 100.0 ** (-2 * i / 64)
        assert abs(float(t[3, i]) - math.cos(a)) < 1e-7 and abs(float(t[3, 32 + i]) - math.sin(a)) < 1e-7


def test_mass_sizes(lib):
    m, s = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.mk_paged_mass_sizes(ctypes.byref(_cfg()), ctypes.byref(m), ctypes.byref(s)) == 0
    assert m.value == 2 * 100 * 8 * 32 * 4 and s.value == 100 * 32 * 32 * 4
    assert lib.mk_paged_mass_sizes(ctypes.byref(_cfg(page=8)), ctypes.byref(m), ctypes.byref(s)) == 1


def test_oracle_mass_and_evicted_tokens_by_hand():
    q = torch.zeros(2, 128, dtype=torch.float64)
    q[:, 0] = math.log(3.0)
    k = torch.zeros(3, 128, dtype=torch.float64)
    k[1, 0] = 1.0
    w, _ = O.mass(q, k, 1.0, torch.tensor([2, 3]))
    assert torch.allclose(w, torch.tensor([1 / 4 + 1 / 5, 3 / 4 + 3 / 5, 1 / 5], dtype=torch.float64))
    w, _ = O.mass(q, k, 1.0, torch.tensor([3, 3]), torch.tensor([-math.inf, 0.0], dtype=torch.float64))
    assert torch.allclose(w, torch.tensor([1.0, 3.0, 1.0], dtype=torch.float64))
    assert O.evict_tokens([9, 1, 1, 5, 1, 0, 7], 4, 1, 1) == [0, 1, 3, 6]
    assert O.evict_tokens([9, 1, math.nan, -5, 1, 0, 7], 6, 1, 1) == [0, 1, 3, 4, 5, 6]
    assert O.evict_tokens([1, 2], 2, 0, 0) == [0, 1] and O.evict_tokens([1, 2], 0, 0, 0) == []


def test_new_calls_refuse_a_null_handle(lib):
    good = 1 << 20
    assert lib.mk_paged_prefix_attn(None, 0, None, None, good, 4096, 1.0, good, 4096, None, None) == 1
    assert lib.mk_paged_decode_attn_mass(None, 0, None, good, 4096, 1.0, good, 4096, None, good, 0, good, 1 << 30, None) == 1
    assert lib.mk_paged_prefill_mass(None, 0, None, 1, good, 4096, 1.0, good, good, 0, 1, None) == 1
    assert lib.mk_paged_evict(None, 0, None, good, good, 0, 0, good, 8, good, None) == 1
