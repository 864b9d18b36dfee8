"""Chunks that turn their keys, as long as there are places for blocks and one token
either side of it: up to four tokens for each SM a block takes one of them, beyond that
runs of four, the last of which may be shorter."""
import pytest
import torch

import test_gpu_append_rope as TA
from decode_attention_pruned_gb300 import binding as lkb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", TA.FORMATS, ids=TA.NAMES)
@pytest.mark.parametrize("batch", [1, 3])
def test_lengths_around_the_change(cuda, fmt, batch):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = 4 * sms // batch
    w, masks = TA._workload(batch, sink=4, local=64)
    TA._run(w, masks, fmt, TA._rope("plain" if batch == 1 else "axes"), [n - 1, n, n + 1, n + 2, n + 3],
            own_positions=batch == 1)


@pytest.mark.parametrize("paged", [False, True], ids=["flat", "paged"])
def test_ragged_lengths_around_the_change(cuda, paged):
    """Sequences that end inside a run."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = 2 * sms + 1
    w, masks = TA._workload(2, sink=2, local=20)
    for fmt in (lkb.KV_BF16, lkb.KV_FP8_BLOCK):
        TA._run(w, masks, fmt, TA._rope("half-part"), [n, n, 2 * n], paged=paged, ragged=True, fused=True)
