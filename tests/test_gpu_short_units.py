"""Verification over units of two or three tiles, many to a CTA: the query
buffer passes from unit to unit faster than the ring of tiles goes round, for
sparse and dense verification at both head dimensions."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU too
    pytest.skip("needs a GPU", allow_module_level=True)

import sparse_kv_verify_gb300 as dk  # noqa: E402
from synth import WORKLOADS  # noqa: E402

from _cases import Case, assert_attention  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("d,k,L", [(64, 64, 60), (64, 128, 120), (128, 64, 60)])
def test_verify_many_short_units_per_cta(d, k, L):
    wl = WORKLOADS["tiny"].with_(B=300, Hq=8, Hkv=8, d=d, L=L, k=k, gamma=1, sinks=2, window=8, m=8, n_planted=2,
                                 slack=4)
    c = Case(wl)
    x = c.x
    grid, tiles = dk.verify_split(c.p, 8, 8, d, 1, False)
    assert tiles <= 3 and wl.B * wl.Hkv * tiles >= 10 * grid
    rng = np.random.default_rng(k + d)
    I_ref = np.full((wl.B, k), -1, np.int64)
    for b in range(wl.B):
        n = int(rng.integers(1, min(k, L) + 1))
        I_ref[b, :n] = np.sort(rng.choice(L, n, replace=False))
    I = torch.as_tensor(I_ref.astype(np.int32), device="cuda")
    ws = dk.workspace(c.p, verify=(8, 8, d, 1))
    for _ in range(3):
        o = dk.dustin_verify_attn(c.p, x.Q[0], x.K[0], x.V[0], x.Kb[0], x.Vb[0], I, c.seq, ws=ws)
        assert dk.check(ws) == 0
        assert_attention(o, c.oracle_verify(I_ref))
        o = dk.dense_verify_attn(c.p, x.Q[0], x.K[0], x.V[0], x.Kb[0], x.Vb[0], c.seq, ws=ws)
        assert dk.check(ws) == 0
        assert_attention(o, c.oracle_dense())
