"""Stores of different shapes in one process, taking turns: what one store's calls set up must not undo another's."""
import pytest
import torch

from chunk_helpers import random_rows
from test_gpu_chunk import make_cfg, pkv, queries  # noqa: F401

pytestmark = pytest.mark.gpu

RANKS = [(40, 32), (8, 8), (24, 24), (30, 38), (32, 30), (1, 2)]  # record sizes above and below a dense page's


@pytest.mark.parametrize("kw", [dict(head_dim=64), dict(head_dim=64, rope_theta=1e4), dict(page_size=32),
                                dict(head_dim=64, factor_int4=True)])
def test_stores_of_different_ranks_take_turns(pkv, kw):
    most = kw.get("page_size", 64) // (2 if "factor_int4" in kw else 1)
    stores, first = [], {}
    for i, (rk, rv) in enumerate(RANKS):
        cfg = make_cfg(pkv, num_layers=1, max_batch=1, rank_k=min(rk, most), rank_v=min(rv, most), **kw)
        store = pkv.Store(cfg)
        K, V = (x.cuda() for x in random_rows(cfg, 700, i, 1))
        store.load_prefill(0, K, V)
        stores.append((cfg, store))
    for i in [0, 1, 2, 3, 4, 5, 0, 1, 2, 3, 4, 5, 3, 0]:
        cfg, store = stores[i]
        k, v = (x.cuda() for x in random_rows(cfg, 140, 9))
        q = queries(cfg, 140, 8).cuda()
        dec = torch.empty(1, cfg.num_q_heads, cfg.head_dim, device="cuda")
        got = [store.decode_attention(0, q[:1], dec, [0]), store.chunk_attention(0, q, k, v, [0], [140]),
               store.chunk_attention(0, q[:3], k[:3], v[:3], [0], [3]), *store.read_tokens(0, [0], [0], [700])]
        for x, y in zip(got, first.setdefault(i, got)):
            assert torch.equal(x, y) and torch.isfinite(x.float()).all()
        assert store.check_device_status() == 0
