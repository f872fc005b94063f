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
