"""The Python binding of the scoring operators: refusals that need no GPU."""
import pytest
import torch

import precision_label_chunk_b200 as elmo


@pytest.mark.parametrize("grid,own,other", [("e4m3", torch.float8_e4m3fn, torch.float8_e5m2),
                                            ("fp8_ge5m2", torch.float8_e4m3fn, torch.float8_e5m2),
                                            ("e5m2", torch.float8_e5m2, torch.float8_e4m3fn)])
def test_pack_reads_8_bit_weights_on_their_own_grid(grid, own, other):
    codes, scales = torch.zeros(10, 32, dtype=torch.uint8), torch.zeros(10, 2, dtype=torch.bfloat16)
    W = torch.zeros(10, 64)
    with pytest.raises(ValueError, match=str(own)):
        elmo.elmo_q4_pack(W.to(other), grid, 32, codes, scales)
    for good in (W.to(own), W.to(torch.uint8)):                 # bytes are what the format says
        with pytest.raises(ValueError, match="CUDA device"):
            elmo.elmo_q4_pack(good, grid, 32, codes, scales)


def test_the_stream_needs_public_functions_alone(monkeypatch):
    """torch's accessor of the raw handle is used where there is one, and nothing depends on it."""
    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: Stream() if d == 3 else None)
    monkeypatch.setattr(elmo, "_raw_stream", lambda d: 5678 if d == 3 else None)
    assert elmo._stream(None).value == 5678
    monkeypatch.setattr(elmo, "_raw_stream", None)
    assert elmo._stream(None).value == 1234


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [True, False])
def test_the_current_stream_is_the_one_that_torch_names(raw, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not raw:
        monkeypatch.setattr(elmo, "_raw_stream", None)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert elmo._stream(None).value == side.cuda_stream
    assert (elmo._stream(None).value or 0) == torch.cuda.current_stream().cuda_stream


def test_arguments_of_the_scoring_calls_lie_on_the_current_device(monkeypatch):
    class Fake(torch.Tensor):                                   # a tensor that says it lies on cuda:1
        is_cuda = True

        def get_device(self):
            return 1

    t = torch.zeros(4).as_subclass(Fake)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        elmo._arg("lse", t, (4,), (torch.float32,))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert elmo._arg("lse", t, (4,), (torch.float32,)) == t.data_ptr()
    for other in (torch.zeros(4), torch.zeros(4).as_subclass(type("On2", (Fake,), {"get_device": lambda s: 2}))):
        with pytest.raises(ValueError, match="device"):
            elmo._arg("entropy", other, (4,), (torch.float32,), 1)
    assert elmo._arg("entropy", t, (4,), (torch.float32,), 1) == t.data_ptr()
