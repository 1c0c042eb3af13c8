"""StepPlan's stream arguments (no GPU): every form that the calls accept."""
import contextlib

import pytest

from latent_attention_decode_absorbed_b200 import StepPlan

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("stream", [None, 7, "object"])
def test_keep_all_takes_the_streams_that_the_calls_take(monkeypatch, stream):
    """None (the current stream), an integer handle, a stream object."""
    plan = StepPlan(batch=2, num_pages=4, max_pages=2, max_rows=8, device="cpu")
    plan.kv_lens.copy_(torch.tensor([3, 70], dtype=torch.int32))
    used = []

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle

    @contextlib.contextmanager
    def on(s):
        used.append(s.cuda_stream)
        yield

    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    plan.keep_all(Stream(9) if stream == "object" else stream)
    assert plan.seq_lens.tolist() == [3, 70]
    assert used == {None: [], 7: [7], "object": [9]}[stream]


@pytest.mark.gpu
def test_keep_all_on_a_raw_handle():
    plan = StepPlan(batch=3, num_pages=4, max_pages=2, max_rows=8)
    plan.kv_lens.copy_(torch.tensor([3, 70, 0], dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.keep_all(side.cuda_stream)
    side.synchronize()
    assert plan.seq_lens.tolist() == [3, 70, 0]
    plan.kv_lens.add_(1)
    torch.cuda.synchronize()
    plan.keep_all(0)                      # the default stream's handle
    torch.cuda.synchronize()
    assert plan.seq_lens.tolist() == [4, 71, 1]
