"""Values at the ends of the stored formats, and values that must not reach a result, in paged_chunk_attention and
paged_attention_mass."""
import math

import pytest
import torch

import chunk_reference as R
from paged_kv_decode_09_gb300 import api

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


def test_rows_computed_again_do_not_stop_the_rest():
    """A value that is not finite in the last token of a long row: the 252 (query, head) rows of the tile that do
    not attend to it are computed again, two KV heads by one CTA.  That takes longer than a wait's limit (a second):
    no wait may stand behind it."""
    n, L = 64, 200_000
    c = R.Chunk(api.F16, 2, 4, [(n, L)], seed=31)
    c.pool.v_data[0, c.bt[0, (L - 1) // 16].long(), :, (L - 1) % 16, 5] = math.inf
    q = c.normal(n, c.n_q, 128, dtype=torch.float16)
    lse = torch.empty(n, c.n_q, device=c.device)
    out = api.paged_chunk_attention(c.pool, 0, q, c.cu, c.bt, c.lens, SCALE, lse=lse,
                                    workspace=api.WorkspaceChunk(c.pool, c.n_q, 1))
    torch.cuda.synchronize()
    assert c.pool.read_status() == 0
    assert torch.isinf(out[-1, :, 5]).all()
    assert torch.isfinite(out[:-1]).all() and torch.isfinite(out[-1, :, 6:]).all()
    c.pool.v_data[0, c.bt[0, (L - 1) // 16].long(), :, (L - 1) % 16, 5] = 0
    want, tol, wl, lt = R.attention(c, q, SCALE)
    assert ((out.double() - want).abs() <= tol)[:-1].all() and ((lse.double() - wl).abs() <= lt).all()
