"""Which stream owns the memory that dit_paged_attention allocates for itself:
the one it runs on, or its blocks could be reused while the call still runs."""
import pytest
import torch

import dit_token_b200 as dit
from dit_token_b200 import paged


def test_the_default_stream_is_not_taken_from_a_pool(monkeypatch):
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: ("external", raw, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    assert paged._allocating_stream(1, 0, 0) == ("default", 1)
    assert paged._allocating_stream(1, 1, 1) == ("default", 1)  # cudaStreamLegacy
    assert paged._allocating_stream(1, 0x5000, 0x5000) == ("external", 0x5000, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 200])
def test_allocations_belong_to_the_calls_stream(monkeypatch, n):
    from _paged import Batch, check_attention
    x = Batch([n, 1], [3000, 700], 8, 2, 128, seed=n).fill()
    lens, seen, empty = x.kv_lens(), [], torch.empty
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def counted(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)
    for stream, raw in ((None, 0), (0, 0), (torch.cuda.default_stream(), 0), (torch.cuda.current_stream(), 0),
                        (side, side.cuda_stream), (side.cuda_stream, side.cuda_stream)):
        with monkeypatch.context() as m:
            m.setattr(torch, "empty", counted)
            out = dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, lens, x.cs, x.cp, stream=stream,
                                          **x.sizes())
        assert seen == [raw, raw]  # the output and the workspace
        seen.clear()
        home = [s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= out.data_ptr() < s["address"] + s["total_size"]]
        assert home == [raw]
        side.synchronize()
        check_attention(x, out, None, True, 0)
