"""The benchmark's side measurement from hidden states to logits runs for every workload with draft logits, in its type."""

import math

import pytest
import torch

from workloads import CONFIGS, make_workload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("config", [k for k in CONFIGS if k != "greedy"])
def test_head_leg(config):
    import bench
    import draft_verification_04_amd as sv
    sv.load_library()
    w = make_workload(config, torch.device("cuda:0"), B=3, V=1000)
    r = bench.head_leg(sv, torch, w, torch.cuda.current_stream(), d=256, reps=1)
    assert set(r["ms"]) == {"norm_to_8_bits", "logits", "adjust_in_place", "verify"}
    assert all(math.isfinite(v) and v > 0 for v in r["ms"].values()) and r["rows"] == w.B * (w.gamma + 1)
