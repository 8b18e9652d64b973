"""Rotations on the GPU: positions with more axes than the pairs use."""
import numpy as np
import pytest
import torch

import trainable_sparse_attention_decode_gb300 as nosa
from test_quant4_gpu import Cache, Turn
from test_quant_gpu import config, dev, query

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("axes,more", [([0] * 20 + [1] * 12, 3), ([0, 2] * 16, 4), (None, 3)])
def test_positions_of_more_axes_than_the_pairs_use(axes, more):
    """A map that uses the first axes takes positions of all of them, as the C calls do."""
    rng = np.random.default_rng(more)
    turn = Turn(64, 500, axes)
    pos = rng.integers(0, 500, size=(more, 2, 5)).astype(np.int32)
    pos[turn.n_axes:] = -1  # (not read)
    few, many = dev(pos[:turn.n_axes]), dev(pos)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cfg, q = config(2, 4, 2, 64, "bf16"), query(rng, 2, 5, 4, 64, "bf16")
    a, b = torch.empty_like(q), torch.empty_like(q)
    nosa.nosa_rotate(cfg, turn.rope, few, q, q_out=a)
    nosa.nosa_rotate(cfg, turn.rope, many, q, q_out=b, status=status)
    assert torch.equal(a, b) and not torch.equal(a, q)
    c = Cache(rng, "bf16", 2, 4, 2, 64, [70, 64, 9, 130]).upload()
    x, y = c.run(q, rope=turn.rope, positions=few), c.run(q, rope=turn.rope, positions=many)
    assert torch.equal(x[0], y[0]) and y[2] == 0
    k = query(rng, 2, 5, 2, 64, "bf16")
    tails = []
    for p in (few, many):
        tail, lens = torch.zeros_like(c.tail), torch.zeros(4, dtype=torch.int32, device="cuda")
        nosa.nosa_quant4_append(cfg, k, k, None, c.units, c.t_tab, tail, lens, rope=turn.rope, positions=p, status=status)
        tails.append(tail)
    assert torch.equal(*tails) and status.item() == 0
    five = torch.zeros(5, 2, 5, dtype=torch.int32, device="cuda")
    for bad in (five, many[:turn.n_axes - 1], many[:, :, :4], many.long(), many[:, :1].expand(more, 2, 5)):
        with pytest.raises((ValueError, nosa.NosaError)):
            nosa.nosa_rotate(cfg, turn.rope, bad, q)
