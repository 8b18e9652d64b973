"""Rotations on the GPU: every variant that the launch chooses between, unaligned tables and values, and positions with
more axes than the pairs use."""
import numpy as np
import pytest
import torch

import trainable_sparse_attention_decode_gb300 as nosa
from test_quant4_gpu import Cache, Turn, some_axes
from test_quant_gpu import DT, config, dev, f64, query

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


HEADS = [  # dtype, hq, hkv, d, rot, kind, interleaved: every number of heads a thread, with heads left over and without
    ("bf16", 32, 8, 128, 128, "one", False), ("bf16", 8, 2, 128, 96, "mixed", True), ("bf16", 6, 3, 128, 128, "sections", False),
    ("bf16", 12, 6, 128, 64, "one", True), ("bf16", 6, 1, 128, 112, "uneven", False), ("bf16", 24, 8, 128, 128, "one", True),
    ("bf16", 27, 9, 64, 64, "four", False), ("bf16", 18, 6, 64, 48, "one", True), ("bf16", 6, 1, 64, 32, "one", False),
    ("bf16", 36, 9, 64, 64, "sections", True), ("f32", 6, 3, 128, 128, "one", False), ("f32", 6, 1, 64, 32, "mixed", True),
    ("f32", 2, 1, 128, 96, "sections", False), ("f32", 8, 2, 64, 64, "one", True)]


@pytest.mark.parametrize("dtype,hq,hkv,d,rot,kind,interleaved", HEADS)
def test_rotate_several_heads_a_thread(dtype, hq, hkv, d, rot, kind, interleaved):
    """More than 77 824 chunks of sixteen elements: bit for bit the oracle's, forward, backward and in place, one of the two alone."""
    rng = np.random.default_rng(hq + d)
    batch, n = 3, 80000 // ((hq + hkv) * (d // 16) * 3) + 2
    turn = Turn(rot, 900, some_axes(kind, rot // 2), interleaved)
    cfg, pos = config(batch, hq, hkv, d, dtype), turn.positions(rng, batch, n)
    q, k = query(rng, batch, n, hq, d, dtype, 3.0), query(rng, batch, n, hkv, d, dtype, 3.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for backward in (False, True):
        qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        nosa.nosa_rotate(cfg, turn.rope, dev(pos), q, k, q_out=qo, k_out=ko, backward=backward, status=status)
        assert np.array_equal(f64(qo), turn.oracle(f64(q), pos, dtype, backward)), backward
        assert np.array_equal(f64(ko), turn.oracle(f64(k), pos, dtype, backward)), backward
    wide = torch.randn(batch, n, hq + hkv + 1, d, device="cuda").to(DT[dtype])
    ref = wide.clone()
    nosa.nosa_rotate(cfg, turn.rope, dev(pos), wide[:, :, 1:hq + 1], wide[:, :, hq + 1:], status=status)
    assert np.array_equal(f64(wide[:, :, 1:]), turn.oracle(f64(ref[:, :, 1:]), pos, dtype)) and torch.equal(wide[:, :, 0], ref[:, :, 0])
    assert status.item() == 0


@pytest.mark.parametrize("dtype,hq,hkv,d,interleaved", [("bf16", 32, 8, 128, False), ("bf16", 8, 1, 64, True), ("f32", 24, 8, 128, False), ("f32", 6, 1, 64, True)])
def test_rotate_prompts_as_their_pieces(dtype, hq, hkv, d, interleaved):
    """More than 2^22 chunks: the same bits as in pieces of a few tokens."""
    rng = np.random.default_rng(hq)
    n = (1 << 22) // ((hq + hkv) * (d // 16)) + 301
    turn = Turn(d, 5000, None, interleaved)
    cfg, pos = config(1, hq, hkv, d, dtype), dev(turn.positions(rng, 1, n))
    q, k = (torch.randn(1, n, h, d, device="cuda").to(DT[dtype]) for h in (hq, hkv))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    nosa.nosa_rotate(cfg, turn.rope, pos, q, k, q_out=qo, k_out=ko)
    step = 77824 // ((hq + hkv) * (d // 16))
    for i in range(0, n, step):
        nosa.nosa_rotate(cfg, turn.rope, pos[:, :, i:i + step].contiguous(), q[:, i:i + step], k[:, i:i + step])
    assert torch.equal(qo, q) and torch.equal(ko, k)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_tables_and_values_on_16_byte_boundaries(dtype, d):
    """A table, or values, that lie 16 bytes off a 32-byte boundary: the same bits, where 32 bytes are loaded at once otherwise."""
    rng = np.random.default_rng(d)
    batch, hq, hkv, n = 2, 8, 2, 200
    cfg, turn = config(batch, hq, hkv, d, dtype), Turn(d, 700)
    table = torch.empty(700 * d + 4, device="cuda")[4:].view(700, d // 2, 2).copy_(dev(turn.table))
    assert table.data_ptr() % 32 == 16
    rope, pos = nosa.nosa_rope(table), dev(turn.positions(rng, batch, n))
    q, k, v = (query(rng, batch, n, h, d, dtype) for h in (hq, hkv, hkv))
    a, b = torch.empty_like(q), torch.empty_like(q)
    nosa.nosa_rotate(cfg, turn.rope, pos, q, q_out=a)
    nosa.nosa_rotate(cfg, rope, pos, q, q_out=b)
    assert torch.equal(a, b)
    few = pos[:, :, :3].contiguous()
    c = Cache(rng, dtype, batch, hq, hkv, d, [300, 300, 64, 64]).upload()
    x, y = (c.run(q[:, :3].contiguous(), rope=r, positions=few) for r in (turn.rope, rope))
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    elt = 16 // q.element_size()  # elements of 16 bytes
    base = torch.empty(v.numel() + elt, dtype=v.dtype, device="cuda")[elt:].view(v.shape).copy_(v)
    apart = torch.empty(batch, n, hkv, d + elt, dtype=v.dtype, device="cuda")[..., :d].copy_(v)
    assert base.data_ptr() % 32 == 16 and apart.stride(2) * apart.element_size() % 32 == 16
    got = []
    for r, vv in ((turn.rope, v), (rope, v), (turn.rope, base), (turn.rope, apart)):
        for m in (n, 64, 7):
            units = torch.zeros(batch * hkv * 4, nosa.nosa_quant4_unit_bytes(cfg), dtype=torch.uint8, device="cuda")
            tail = torch.zeros(batch * hkv * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
            lens = torch.zeros(batch * hkv, dtype=torch.int32, device="cuda")
            tab = torch.arange(batch * hkv * 4, dtype=torch.int32, device="cuda").view(batch * hkv, 4)
            nosa.nosa_quant4_append(cfg, k[:, :m], vv[:, :m], None, units, tab, tail, lens, rope=r, positions=pos[:, :, :m].contiguous())
            got.append((m, units, tail))
    for m, units, tail in got:
        ref = next(g for g in got if g[0] == m)
        assert torch.equal(units, ref[1]) and torch.equal(tail, ref[2])
        assert units.any() == (m >= 64) and tail.any() == (m != 64)
