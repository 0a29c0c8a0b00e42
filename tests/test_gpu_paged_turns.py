"""Calls of one handle one behind the other, which use the same workspace, on the GPU through the C ABI."""
import pytest
import torch

from compressed_kv_cache_vector_gb300 import binding as K
from compressed_kv_cache_vector_gb300.build import build
from tests.test_gpu_paged import Made, _gen, _i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_every_call_behind_every_other(kv):
    """Shared prefixes, a step with mass, a prompt's mass and eviction in every order of two, without a wait and replayed
    from a graph: each leaves what it leaves when the device is idle before and after it."""
    lens, n = [4100 + 50 * i for i in range(12)], 12
    made = Made(kv, 32, 4, 4, lens, 3, extra_cols=(160 << 20) // (12 * 32 * 4 * 256))
    for row in made.rows[1:]:
        row[:124] = made.rows[0][:124]                                                  # 3968 tokens
    made.table.copy_(_i32(made.rows))
    c, mass = made.c, K.PagedMass(made.c)
    q = torch.randn(n, 16, 128, generator=_gen(2), device=DEV).to(torch.bfloat16)
    step, prefix = K.PagedBatch(made.kv_len, made.table), K.PagedPrefix(_i32([0, n]), _i32([3968]))
    chunk = K.PagedBatch(made.kv_len, made.table, _i32([40 * i for i in range(n + 1)]), 40, 40 * n)
    qc = torch.randn(40 * n, 16, 128, generator=_gen(3), device=DEV).to(torch.bfloat16)
    lse_c = c.prefill_attn(0, chunk, qc, lse=True)[1]
    out, lse = torch.zeros_like(q), torch.zeros(n, 16, device=DEV)
    out2, lse2 = torch.zeros_like(q), torch.zeros(n, 16, device=DEV)
    keep, kept, new_len = _i32([t - 60 for t in lens]), torch.zeros(n, 4, max(lens), dtype=torch.int32, device=DEV), _i32([0] * n)
    state = [c.k_pool.view(torch.uint8), c.v_pool.view(torch.uint8), mass.mass, out, lse, out2, lse2, kept, new_len]
    state += [c.k_scale, c.v_scale] if kv == "e4m3" else []
    mass.mass.copy_(torch.rand(mass.mass.shape, generator=_gen(5), device=DEV))
    start = [t.clone() for t in state]
    calls = [lambda: c.prefix_attn(0, step, prefix, q, out=out, lse=lse),
             lambda: c.decode_attn_mass(0, step, q, mass, first=3968, out=out2, lse=lse2),
             lambda: c.prefill_mass(0, chunk, qc, lse_c, mass, first=3968),
             lambda: c.evict(0, step, mass, keep, first=3968, recent=5, kept=kept, new_len=new_len)]

    def after(run):
        for t, s in zip(state, start):
            t.copy_(s)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert c.poll_error() == (0, 0)
        return [t.clone() for t in state]

    for a in calls:
        for b in calls:
            def apart():
                for f in (a, b, a):
                    f()
                    torch.cuda.synchronize()

            def together():
                for f in (a, b, a):
                    f()

            graph = torch.cuda.CUDAGraph()
            want = after(apart)
            with torch.cuda.graph(graph):
                together()
            for run in (together, graph.replay):
                for x, y in zip(after(run), want):
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
