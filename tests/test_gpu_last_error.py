"""The error call of the hybrid and KV-cache layers, and the streams it answers for."""
import pytest
import torch

from hybrid_linear_attention_arl2_b200 import arl2, build
from hybrid_linear_attention_arl2_b200 import workloads as W
from tests.gpu_util import dev, make_layer

pytestmark = pytest.mark.gpu
ERR_TIMEOUT = 5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    arl2.load_library()


def test_last_error_waits_for_a_replay_on_another_stream():
    """A frame's query captured with a wait limit of a microsecond, replayed behind a delay on a stream that the handle
    never saw: its timeout is there when last_error returns, and cleared for the query after it."""
    cfg = W.CONFIGS[1]
    wl = W.Workload(cfg)
    layer, _ = make_layer(cfg, wl)
    q, k, v = (dev(x, "bf16") for x in wl.qkv(0, 0, 0))
    ref = layer.query(q, k, v)
    assert layer.last_error() == 0
    out = torch.empty_like(ref)
    arl2.arl2_state_set_wait_limit(layer.handle, 1000)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.query(q, k, v, o=out, stream=torch.cuda.current_stream().cuda_stream)
    arl2.arl2_state_set_wait_limit(layer.handle, 0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
            g.replay()
        assert layer.last_error() == ERR_TIMEOUT and layer.last_error() == 0
        with torch.cuda.stream(side):
            o = layer.query(q, k, v, stream=side.cuda_stream)
            assert torch.equal(o, ref)
        assert layer.last_error() == 0
    layer.close()
