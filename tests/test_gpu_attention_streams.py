"""Plans whose own memory (workspace, outputs) was made on one stream and is used on another: the zeros are there before
the first call reads them, and the memory is not handed on while a call uses it."""
import numpy as np
import pytest
import torch

from tests import _attention as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
BUSY = 100_000_000                                            # cycles that a stream is kept busy: about 50 ms
LENS = [9000, 3, 700]                                         # runs that are cut between CTAs, and joined through the workspace


def case(seed):
    E = H.pkg()
    cache, table = H.filled(LENS, 16, 2, 128, "bf16", seed)
    q = torch.randn((3, 8, 128), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).bfloat16()
    return E, cache, table, q, torch.from_numpy(table).to(DEV), torch.tensor(LENS, dtype=torch.int32, device=DEV)


def junk():
    """Leaves freed blocks of every size a plan takes, full of ones."""
    made = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in (1 << 12, 1 << 14, 1 << 16, 1 << 20, 3 << 20, 5 << 20)]
    torch.cuda.synchronize()
    return made


def test_a_plan_made_behind_a_busy_stream_runs_on_another():
    E, cache, table, q, bt, sl = case(1)
    side = torch.cuda.Stream()
    made = junk()
    del made
    torch.cuda._sleep(BUSY)                                   # the zeros are written behind this
    plan = E.PagedAttentionPlan(cache, q, bt, sl, lse=True)
    plan.run(side)
    with torch.cuda.stream(side):
        plan.run()
    side.synchronize()
    H.check_attention(cache, table, LENS, q, plan.out, plan.lse, 128 ** -0.5)
    assert not plan.workspace[:16384].any()


def test_a_plan_dropped_while_another_stream_uses_its_workspace():
    E, cache, table, q, bt, sl = case(2)
    side = torch.cuda.Stream()
    out, lse = torch.empty((3, 8, 128), dtype=torch.bfloat16, device=DEV), torch.empty((3, 8), device=DEV)
    plan = E.PagedAttentionPlan(cache, q, bt, sl, out=out, lse=lse)
    size = plan.workspace.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        plan.run()
    del plan
    over = [torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    H.check_attention(cache, table, LENS, q, out, lse, 128 ** -0.5)
    assert all(bool((x == 0xFF).all()) for x in over)


def test_a_capture_on_a_stream_that_has_not_run_the_plan():
    E, cache, table, q, bt, sl = case(3)
    plan = E.PagedAttentionPlan(cache, q, bt, sl, lse=True)
    plan.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                             # a stream of its own
        plan.run()
    plan.out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    H.check_attention(cache, table, LENS, q, plan.out, plan.lse, 128 ** -0.5)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_the_function_forms_on_a_side_stream(fmt):
    E = H.pkg()
    rng = np.random.default_rng(4)
    lens, page, side = [300, 2], 16, torch.cuda.Stream()
    table, pages = H.tables(lens, page, rng)
    cache = H.empty_cache(pages, page, 2, 64, fmt)
    g = torch.Generator(device=DEV).manual_seed(4)
    slots = torch.from_numpy(np.concatenate([H.slots_of(table, b, 0, n, page) for b, n in enumerate(lens)])).to(DEV)
    k, v = (torch.randn((len(slots), 2, 64), generator=g, device=DEV) for _ in range(2))
    q = torch.randn((2, 4, 64), generator=g, device=DEV)
    bt, sl = torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    nr = E.NormRope(None, None, 0.0, None)
    side.wait_stream(torch.cuda.current_stream())
    E.engram_kv_write(cache, k, v, slots, stream=side)
    turned, _ = E.engram_qk_norm_rope(nr, q, None, None, stream=side)
    out, lse = E.engram_paged_attention(cache, turned, bt, sl, lse=True, stream=side)
    side.synchronize()
    assert torch.equal(turned, q.bfloat16())
    H.check_attention(cache, table, lens, turned, out, lse, 0.125)


def test_weights_and_angles_written_by_the_kernel_before():
    # a call may start while the kernel that writes its weights and angles still runs: every call takes the new ones
    E = H.pkg()
    T, D = 600, 128
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k = torch.randn((T, 8, D), generator=g, device=DEV), torch.randn((T, 2, D), generator=g, device=DEV)
    angles = [6.28 * torch.rand((64, D // 2), generator=g, device=DEV) for _ in range(3)]
    tables = [torch.cat([a.cos(), a.sin()], 1) for a in angles]
    weights = [(1 + 0.1 * torch.randn((2, D), generator=g, device=DEV)).bfloat16() for _ in range(3)]
    pos = torch.randint(0, 64, (T,), generator=g, device=DEV, dtype=torch.int32)
    want = []
    for t, w in zip(tables, weights):
        want.append(E.engram_qk_norm_rope(E.NormRope(w[0].clone(), w[1].clone(), 1e-6, t), q, k, pos))
    table, weight = torch.empty_like(tables[0]), torch.empty_like(weights[0])
    nr = E.NormRope(weight[0], weight[1], 1e-6, table)
    outs = [tuple(torch.empty((T, h, D), dtype=torch.bfloat16, device=DEV) for h in (8, 2)) for _ in range(90)]
    plans = [E.QKNormRopePlan(nr, q, k, pos, *o) for o in outs]
    torch.cuda.synchronize()
    for i, plan in enumerate(plans):
        weight.copy_(weights[i % 3])
        table.copy_(tables[i % 3])
        plan.run()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(outs):
        assert torch.equal(a, want[i % 3][0]) and torch.equal(b, want[i % 3][1]), f"call {i}"
