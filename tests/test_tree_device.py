"""StepPlan and TreeDecodeStep work on their own device whichever is current (no GPU: the calls are recorded)."""
import contextlib

import pytest

from latent_attention_decode_absorbed_b200 import StepPlan, TreeDecodeStep
from latent_attention_decode_absorbed_b200 import tree as tree_module

torch = pytest.importorskip("torch")


def test_calls_run_on_the_plan_s_device(monkeypatch):
    now, calls = [0], []
    for name in ("mla_step_plan", "mla_cache_append_slots", "mla_absorb_q", "mla_decode_tree", "mla_out_uv",
                 "mla_cache_commit"):
        monkeypatch.setattr(tree_module, name, lambda *a, _n=name, **k: calls.append((_n, now[0])))

    @contextlib.contextmanager
    def device(index):
        old, now[0] = now[0], index
        yield
        now[0] = old

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    plan = StepPlan(batch=2, num_pages=4, max_pages=2, max_rows=8, device="cpu")
    step = TreeDecodeStep(plan, n_heads=2)
    plan.index = 3                                        # as if its buffers were on cuda:3
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    counts, nodes = torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    plan.plan(counts, nodes)
    step.run(bf(8, 576), bf(8, 2, 128), bf(8, 2, 64), bf(2, 128, 512), bf(2, 128, 512))
    plan.commit([step], counts, nodes)
    plan.keep_all()
    assert len(calls) == 6 and all(d == 3 for _, d in calls)
    assert now == [0]
    now[0] = 3
    calls.clear()
    plan.plan(counts)
    assert calls == [("mla_step_plan", 3)] and now == [3]


def test_a_plan_knows_its_device():
    plan = StepPlan(batch=1, num_pages=1, max_pages=1, max_rows=1, device="cpu")
    assert plan.index is None


@pytest.mark.gpu
def test_a_plan_on_the_current_gpu():
    plan = StepPlan(batch=1, num_pages=1, max_pages=1, max_rows=1)
    assert plan.index == torch.cuda.current_device()
    plan.plan(torch.ones(1, dtype=torch.int32, device="cuda"))
    plan.check()
    assert plan.slots.tolist() == [0]
