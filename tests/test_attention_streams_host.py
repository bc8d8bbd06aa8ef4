"""Which stream a plan's own memory belongs to, without a GPU: the calls and streams are recorded by stand-ins, and the
order of what they were asked is checked."""
import contextlib

import pytest
import torch


class Stream:
    def __init__(self, handle, log):
        self.cuda_stream, self.log, self.capturing = handle, log, False

    def wait_stream(self, other):
        self.log.append(("wait", self.cuda_stream, other.cuda_stream))




@pytest.fixture
def world(monkeypatch):
    from engram_gram_hash_02_gb300 import attention as M, binding, build
    build.build()
    log, real = [], binding.lib()
    home, side = Stream(1, log), Stream(2, log)

    class Lib:
        engram_attention_workspace_bytes = real.engram_attention_workspace_bytes

        def __getattr__(self, name):
            def call(*args):
                log.append(("call", args[-1]))
                return 0
            return call

    current = [home]
    monkeypatch.setattr(M, "lib", lambda: Lib())
    monkeypatch.setattr(M, "_on", lambda device, **tensors: None)
    monkeypatch.setattr(M, "_current_raw_stream", lambda index: current[0].cuda_stream)
    monkeypatch.setattr(M, "_current_device", lambda: None)               # (a CPU device has no index)
    monkeypatch.setattr(M, "_capturing", lambda stream: stream.capturing, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[0])
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("record", s.cuda_stream)))
    return M, log, home, side, current


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def plans(M):
    """Every plan that makes something, and how many tensors it makes."""
    cache = M.KVCache.allocate(4, 8, 2, 64, device="cpu")
    nr = M.NormRope(None, None, 0.0, None)
    q, k, table, lens, slots = z(3, 4, 64), z(3, 2, 64), z(3, 2, dtype=torch.int32), z(3, dtype=torch.int32), z(3, dtype=torch.int64)
    ws, out = M.attention_workspace(cache, 4, 3), z(3, 4, 64)
    return {
        "norm": (lambda **s: M.QKNormRopePlan(nr, q, k, None, **s), 2),
        "norm, keys": (lambda **s: M.QKNormRopePlan(nr, q, k, None, q_out=q, **s), 1),
        "read": (lambda **s: M.KVReadPlan(cache, slots, **s), 2),
        "attention": (lambda **s: M.PagedAttentionPlan(cache, q, table, lens, lse=True, **s), 3),
        "attention, workspace": (lambda **s: M.PagedAttentionPlan(cache, q, table, lens, out=out, **s), 1),
        "attention, out": (lambda **s: M.PagedAttentionPlan(cache, q, table, lens, workspace=ws, **s), 1),
        "step": (lambda **s: M.AttentionStepPlan(nr, cache, q, k, k, None, slots, table, lens, **s), 2),
    }


NAMES = ["norm", "norm, keys", "read", "attention", "attention, workspace", "attention, out", "step"]


@pytest.mark.parametrize("name", NAMES)
def test_the_first_run_on_another_stream_waits_for_the_making(world, name):
    M, log, home, side, current = world
    make, n = plans(M)[name]
    plan = make()
    plan.run()
    plan.run(home)
    assert log == [("call", 1), ("call", 1)]
    del log[:]
    plan.run(side)
    assert log == [("wait", 2, 1)] + [("record", 2)] * n + [("call", 2)]
    del log[:]
    plan.run(side)
    current[0] = side
    plan.run()
    plan.run(home)
    assert log == [("call", 2), ("call", 2), ("call", 1)]


@pytest.mark.parametrize("name", NAMES)
def test_a_plan_made_for_a_stream_is_at_home_there(world, name):
    M, log, home, side, current = world
    make, n = plans(M)[name]
    plan = make(stream=side)
    plan.run(side)
    assert log == [("call", 2)]
    del log[:]
    plan.run()
    assert log == [("wait", 1, 2)] + [("record", 1)] * n + [("call", 1)]


def test_a_capture_is_left_alone(world):
    M, log, home, side, current = world
    plan = plans(M)["step"][0]()
    side.capturing = True
    plan.run(side)
    assert log == [("call", 2)]
    side.capturing = False
    plan.run(side)
    assert ("wait", 2, 1) in log
    other = Stream(3, log)
    home.capturing = True
    del log[:]
    plan.run(other)
    assert log == [("call", 3)]


def test_a_plan_on_the_callers_tensors_waits_for_nothing(world):
    M, log, home, side, current = world
    cache = M.KVCache.allocate(4, 8, 2, 64, device="cpu")
    k = z(3, 2, 64)
    plan = M.KVWritePlan(cache, k, k, z(3, dtype=torch.int64))
    plan.run(side)
    ws = M.attention_workspace(cache, 4, 3)
    M.PagedAttentionPlan(cache, z(3, 4, 64), z(3, 2, dtype=torch.int32), z(3, dtype=torch.int32), out=z(3, 4, 64), workspace=ws).run(side)
    assert log == [("call", 2), ("call", 2)]
