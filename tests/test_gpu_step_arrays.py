"""decode_step on batch buffers: queries and outputs with more rows than the block table."""
import math

import pytest
import torch

import chunk_reference as R
import tree_reference as T
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (100, 17)])
@pytest.mark.parametrize("kv", [api.F16, api.BF16, api.F32, api.Q8_0])
def test_the_first_rows_of_longer_arrays(kv, window, sinks):
    """The rows of the table are computed; those behind them are neither read nor written."""
    rows = [(1, L) for L in (1, 40, 700)]
    c = R.Chunk(kv, 2, 4, rows, seed=3)
    c.pool.set_window(0, window)
    c.pool.set_sinks(0, sinks)
    q, k, v = c.normal(5, c.n_q, 128), c.normal(3, 2, 128), c.normal(3, 2, 128)
    q[3:] = math.nan
    out = torch.full_like(q, 7.0)
    ws = api.Workspace(c.pool, c.n_q, 3)
    assert api.decode_step(c.pool, 0, q, k, v, c.bt, c.lens, SCALE, out=out, workspace=ws) is out
    T.check(c, q[:3], out[:3], None, SCALE, window=window, sinks=sinks)
    assert (out[3:] == 7).all()
    made = api.decode_step(c.pool, 0, q, k, v, c.bt, c.lens, SCALE)  # the same tokens into the same slots
    assert made.shape == q.shape
    T.check(c, q[:3], made[:3], None, SCALE, window=window, sinks=sinks)


def test_arrays_that_do_not_fit():
    """Fewer rows of queries than the table has, an output unlike the queries, and new tokens of other rows; and
    paged_decode_attention takes the table's rows alone."""
    c = R.Chunk(api.F16, 2, 4, [(1, 40), (1, 20)], seed=1)
    q, k = c.normal(2, c.n_q, 128), c.normal(2, 2, 128)
    for args, kw in (((q[:1], k, k), {}), ((q[0], k, k), {}), ((q[:, :, :64].contiguous(), k, k), {}),
                     ((q, k[:1], k), {}), ((q, k, torch.cat([k, k])), {}), ((q, k, k), dict(out=torch.empty_like(q[:1])))):
        with pytest.raises(ValueError):
            api.decode_step(c.pool, 0, *args, c.bt, c.lens, SCALE, **kw)
    with pytest.raises(ValueError):
        api.paged_decode_attention(c.pool, 0, torch.cat([q, q]), c.bt, c.lens, SCALE)
    assert c.pool.read_status() == 0
