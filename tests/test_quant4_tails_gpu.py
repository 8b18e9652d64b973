"""Tails of every length under the 4-bit block cache's attention, for every number of rows."""
import numpy as np
import pytest

from test_quant4_gpu import Cache
from test_quant_gpu import dev, f64, query

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,G,T", [
    *[("bf16", d, G, 1) for d in (64, 128) for G in (1, 2, 3, 4, 6, 8)], ("bf16", 128, 3, 3), ("bf16", 64, 6, 5), ("f32", 64, 3, 1), ("f32", 128, 8, 1)])
@pytest.mark.parametrize("full", [0, 1])
def test_tails_of_every_length(dtype, d, G, T, full):
    """1 to 63 tokens behind a full block and without one; some of them masked, with NaN and infinities there."""
    rng = np.random.default_rng(d + 8 * G + T)
    c = Cache(rng, dtype, 64, G, 1, d, [64 * full + t for t in range(64)], masked=0.1)
    gone = np.isneginf(c.te)
    c.tk[gone], c.tv[gone] = np.nan, np.inf
    c.upload()
    q = query(rng, 64, T, G, d, dtype)
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass = dev(m0)
    out, lse, status = c.run(q, mass=mass, decay=0.5)
    assert status == 0
    c.tk[gone] = c.tv[gone] = 0.0  # (not looked at)
    c.check(q, out, lse, mass0=m0, mass=f64(mass), decay=0.5)
