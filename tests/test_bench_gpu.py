"""What the benchmark times is the call that its line names, and nothing beside it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_shared_prefix_and_its_baselines_time_one_call_each():
    """Every callable of the shared-prefix workload allocates its call's outputs only: preparing the
    lengths of the copied caches inside it would add an allocation and a launch to the baseline alone."""
    import bench
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    dev = torch.device("cuda")
    calls, keys = bench.shared_prefix_calls(3, 300, 64, 16, 4, 128, dev, True)
    assert keys == 32 + 48 + 64
    outputs = {"prefix_us": 2, "copied_prefix_us": 1, "copied_prefix_varlen_us": 1}  # o and lse; o; o
    assert set(calls) == set(outputs)
    results = {}
    for name, call in calls.items():
        call()
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        results[name] = call()[0]
        assert torch.cuda.memory_stats()["allocation.all.allocated"] - before == outputs[name], name
    # The same step: either side rounds its probabilities and its result to bf16 (2^-8 of |v| < 6 each).
    for name, o in results.items():
        assert (o.float() - results["prefix_us"].float()).abs().max() <= 4 * 2.0 ** -8 * 6, name
