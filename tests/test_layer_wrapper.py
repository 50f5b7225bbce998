"""The torch-tensor wrapper of the layer without a GPU: on which stream a call
with stream= allocates its outputs. Tensors, streams and library are
stand-ins."""
import types

import pytest

torch = pytest.importorskip("torch")

from test_attention_wrapper import Streams, Tensor
from w4a16_routed_expert_gb300 import capi, layer


def test_outputs_belong_to_the_stream_that_writes_them(monkeypatch):
    own = types.SimpleNamespace(cuda_stream=9)
    x = Tensor(3, 64)
    for stream, number in ((None, 7), (own, 9)):
        at, calls = Streams(monkeypatch), []

        def entry(*args):
            calls.append(args[-1])
            return capi.MOE_OK

        monkeypatch.setattr(capi, "moe_layer_forward", entry, raising=False)
        monkeypatch.setattr(capi, "moe_layer_routing", entry, raising=False)
        monkeypatch.setattr(capi, "lib", lambda: types.SimpleNamespace(moe_stack_forward=entry))
        ml, st = layer.MoELayer.__new__(layer.MoELayer), layer.MoEStack.__new__(layer.MoEStack)
        ml.handle = st.handle = None
        ml.num_experts, ml.top_k = 8, 2
        outs = [ml.forward(x, stream=stream), st.forward(x, stream=stream)]
        ml.routing(3, stream=stream)
        assert all(o.shape == x.shape and o.dtype == x.dtype for o in outs)
        assert calls == [number] * 3
        assert len(at.allocated) == 6 and all(s.cuda_stream == number for s in at.allocated)
        assert at.recorded == ([] if stream is None else [at.current] * 6)
        monkeypatch.undo()
