"""Eviction from the paged cache where it is easily wrong, on the GPU through the C ABI, against the definition."""
import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from tests.test_gpu_paged import Made, _gen, _i32
from tests.test_gpu_paged_mass import _evict_check, _evict_run

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.mark.parametrize("cut", [True, False])
def test_longest_sequence_that_a_table_can_name(cut):
    """2^31 - 256 tokens behind a prefix that is one page over and over: the last page's one free choice is cut, or
    nothing is."""
    P, columns = 64, (2 ** 31 - 256) // 64
    T = columns * P
    c = K.PagedKV(K.make_paged_config(1, 1, 1, P, 3, 1, K.MK_KV_E4M3), DEV)
    c.k_pool.view(torch.uint8).copy_(torch.randint(0, 120, c.k_pool.shape, dtype=torch.uint8, device=DEV))
    c.v_pool.view(torch.uint8).copy_(torch.randint(0, 120, c.v_pool.shape, dtype=torch.uint8, device=DEV))
    c.k_scale.fill_(2.0 ** 20)                                                          # so that a page's scale is formed anew
    c.v_scale.fill_(2.0 ** 20)
    table = torch.zeros(1, columns, dtype=torch.int32, device=DEV)
    table[0, -1] = 2
    m = K.PagedMass(c)
    before = [t.clone() for t in (c.k_pool.float(), c.v_pool.float())]
    keep = T - 1 if cut else T
    new_len, kept = c.evict(0, K.PagedBatch(torch.tensor([T], dtype=torch.int32, device=DEV), table), m,
                            torch.tensor([keep], dtype=torch.int32, device=DEV), first=T - 2, recent=1, max_keep=keep)
    assert c.poll_error() == (0, 0) and new_len.tolist() == [keep]
    step = 1 << 28
    for a in range(0, keep - cut, step):
        e = min(keep - cut, a + step)
        assert torch.equal(kept[0, 0, a:e], torch.arange(a, e, dtype=torch.int32, device=DEV))
    for t, was, scale in ((c.k_pool, before[0], c.k_scale), (c.v_pool, before[1], c.v_scale)):
        now = t.float() * scale[..., None, None]
        assert torch.equal(now[0, :2], was[0, :2] * 2.0 ** 20)                           # the pages of the prefix, and one of nobody
        assert torch.equal(now[0, 2, 0, :62], was[0, 2, 0, :62] * 2.0 ** 20)
        assert torch.equal(now[0, 2, 0, 62], was[0, 2, 0, 63 if cut else 62] * 2.0 ** 20)
    if cut:
        assert int(kept[0, 0, -1]) == T - 1


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_call_behind_an_error_changes_nothing(kv):
    """Neither selection nor move works until the error is cleared; then the same call does."""
    made = Made(kv, 16, 2, 2, [300, 500], 5)
    c, m = made.c, K.PagedMass(made.c)
    m.mass.uniform_(generator=_gen(1))
    b, keeps = K.PagedBatch(made.kv_len, made.table), [100, 222]
    keep, kept, new_len = _i32(keeps), torch.full((2, 2, 222), -1, dtype=torch.int32, device=DEV), _i32([-3, -3])
    c.evict(0, b, m, _i32([5, 5]), first=4, recent=4)                                   # below what always stays: an error
    state = [c.k_pool.view(torch.uint8), c.v_pool.view(torch.uint8), m.mass, kept, new_len]
    state += [c.k_scale, c.v_scale] if kv == "e4m3" else []
    was = [t.clone() for t in state]
    for _ in range(2):
        c.evict(0, b, m, keep, first=4, recent=4, kept=kept, new_len=new_len)
        assert c.poll_error() == (5, 16)
        for t, w in zip(state, was):
            assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
    c.clear_error()
    c.evict(0, b, m, keep, first=4, recent=4, kept=kept, new_len=new_len)
    assert c.poll_error() == (0, 0)
    before = {"k": was[0], "v": was[1]}
    if kv == "e4m3":
        before.update(ks=was[5], vs=was[6])
    _evict_check(made, before, was[2], m.mass, keeps, 4, 4, kept, new_len)


# The CTAs of a (sequence, kv head) are 8, 4, 2 or 1 as two CTAs on every SM allow; a slice beyond 22 528 tokens does not
# fit shared memory.
@pytest.mark.parametrize("kv,many,longest,ctas", [("bf16", 0, 200000, 8), ("e4m3", 40, 100000, 4), ("bf16", 80, 60000, 2),
                                                  ("e4m3", 80, 60000, 2), ("bf16", 170, 50000, 1), ("e4m3", 170, 25000, 1)])
def test_slices_beyond_shared_memory(kv, many, longest, ctas):
    """Alone and among many short sequences, with many equal masses, so that the border lies among equals of every slice."""
    lens = [70 + i % 50 for i in range(many)]
    lens[len(lens) // 2:len(lens) // 2] = [longest]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert next(x for x in (8, 4, 2, 1) if len(lens) * x <= 2 * sms or x == 1) == ctas and longest > ctas * 22528
    made = Made(kv, 64, 1, 1, lens, 7, spread=3)

    def tweak(w):
        w.copy_(torch.round(w))

    _evict_run(made, [t // 3 if t == longest else t - 8 for t in lens], 4, 30, 9, tweak)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n_kv,n", [(8, 10), (8, 20)])
def test_many_units_of_middle_lengths(kv, n_kv, n):
    """77 to 152 (sequence, kv head) units, and more, past 2048 tokens: two CTAs a unit, and one."""
    lens = [2100 + 97 * i for i in range(n)]
    made = Made(kv, 64, n_kv, 1, lens, 9)
    _evict_run(made, [t // 2 for t in lens], 4, 16, 3)
