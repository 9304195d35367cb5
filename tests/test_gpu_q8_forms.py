"""The forms that the 8-bit store's calls take by size: each is run here, against decode rows bit
for bit, against the 64-bit form, or against the same rows alone."""
import pytest
import torch

import invariant_deterministic_04_b200 as bi
import synth
from gpu_util import dev, same_bits
from test_gpu_q8 import fill

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3"]


@pytest.mark.parametrize("Hq,Hkv,period", [(16, 2, 2), (8, 2, 4), (8, 2, 2), (4, 4, 16), (16, 1, 1)])
def test_rows_of_sequences_in_turn_are_few_row_tiles(Hq, Hkv, period):
    """Runs of one row: none of them may take a wide tile. The first two numbers of the workspace are the
    counts of wide and of few-row tiles. A run of one row more than a few-row tile holds is wide."""
    D, few = 64, 16 // (Hq // Hkv)
    lens = [40 + i for i in range(period + 1)]
    S, _ = fill("int8", lens, Hkv, D, 8, seed=500)
    T = 20 * (period + 1)
    seq = torch.arange(T, dtype=torch.int32, device=dev()) % (period if period > 1 else 2)
    seq[T - few - 1:] = period  # one run of few + 1 rows
    pos = torch.arange(T, dtype=torch.int32, device=dev()) % 40
    q = synth.normal_bf16((T, Hq, D), 501).to(dev())
    ws = torch.zeros(bi.attention_prefill_q8_workspace_size(T), dtype=torch.uint8, device=dev())
    pre = bi.attention_prefill_q8(q, seq, pos, *S.args, workspace=ws)
    dec = bi.attention_decode_q8(q, *S.args[:4], S.pt[seq.long()].contiguous(), pos + 1)
    assert same_bits(pre, dec) and bi.get_device_error() == 0
    assert ws[:8].view(torch.int32).tolist() == [1, T - few - 1]
