"""The layer's calls captured into a CUDA graph and replayed on new inputs."""
import pytest
import torch

import synth
import top_routing_expert_gemm_b200 as moe
from tests import moe_harness as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("cfg", [
    synth.LayerConfig("capture_decode", 4, 512, 8, 2, 512, "bf16", synth.SOFTMAX_TOPK, seed=41),
    synth.LayerConfig("capture_batch", 700, 512, 8, 2, 512, "bf16", synth.SOFTMAX_TOPK, n_shared=1, d_ff_shared=256,
                      seed=42),
    synth.LayerConfig("capture_f32", 33, 256, 8, 2, 256, "f32", synth.SOFTMAX_ALL_RENORM, seed=43),
], ids=lambda c: c.name)
def test_captured_forward_replays_as_the_eager_call(cfg):
    inp = H.make_inputs(cfg)
    want = H.run_forward(inp)
    c = H.moe_cfg(cfg)
    dev = inp.dev
    x = dev["x"].clone()
    y = torch.zeros_like(want["y"])
    ids, w, counts = (torch.zeros_like(want[n]) for n in ("ids", "w", "counts"))
    ws = torch.zeros_like(want["ws"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward(c, x, dev["w_router"], dev["bias"], dev["w_gate_up"], dev["w_down"], dev.get("ws_gate_up"),
                        dev.get("ws_down"), y, ids, w, counts, ws)
    for shift in (0, 1, 0):
        x.copy_(dev["x"].roll(shift, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert moe.moe_device_status(ws) == 0
        assert torch.equal(ids, want["ids"].roll(shift, 0)) and torch.equal(counts, want["counts"])
        if shift == 0:
            assert torch.equal(y, want["y"]) and torch.equal(w, want["w"])
