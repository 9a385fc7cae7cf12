"""Buffers of one chunk call that share memory: the output in the queries' place, and the overlaps that are refused."""
import ctypes

import pytest
import torch

from chunk_helpers import random_rows
from test_gpu_chunk import STORES, filled, make_cfg, pkv, queries  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["llama", "g1-p16", "g3-d64", "int4", "prerope", "fp32"])
@pytest.mark.parametrize("lens,counts", [([0, 700, 63, 1], [3, 2, 1, 5]), ([1500, 0, 130, 64], [300, 140, 2, 31])])
def test_output_in_the_queries_place(pkv, name, lens, counts):
    cfg = make_cfg(pkv, num_layers=1, **STORES[name])
    store, _ = filled(pkv, cfg, lens)
    k, v = (x.cuda() for x in random_rows(cfg, sum(counts), 1))
    q = queries(cfg, sum(counts), 2).cuda()
    want = store.chunk_attention(0, q, k, v, [0, 1, 2, 3], counts)
    for _ in range(3):
        x = q.clone()
        assert store.chunk_attention(0, x, k, v, [0, 1, 2, 3], counts, out=x) is x
        assert torch.equal(x, want)


def test_overlaps_are_refused(pkv):
    cfg = make_cfg(pkv, num_layers=1, num_kv_heads=2, num_q_heads=2)
    store, _ = filled(pkv, cfg, [700, 0, 0, 0])
    n, row = 40, 2 * 128
    buf = torch.zeros((n + 1) * row, dtype=cfg.kv_dtype, device="cuda")
    a, b = buf[:n * row].view(n, 2, 128), buf[row:].view(n, 2, 128)  # the same rows, one further
    k, v = (x.cuda() for x in random_rows(cfg, n, 1))
    q = queries(cfg, n, 2).cuda()
    need = store.chunk_workspace(0, [0], [n])["attention"]
    work = torch.empty(need + 4 * n * row, dtype=torch.uint8, device="cuda")
    inside = work[need - 256:need - 256 + 2 * n * row].view(cfg.kv_dtype).view(n, 2, 128)  # begins inside the workspace
    for kw in (dict(out=k), dict(out=v), dict(q=a, out=b), dict(k=a, out=b), dict(v=a, out=b), dict(q=inside), dict(k=inside),
               dict(v=inside), dict(out=inside)):
        x = dict(q=q, k=k, v=v, out=torch.empty_like(q), **{}) | kw
        with pytest.raises(pkv.PuzzleKVError, match="overlap"):
            store.chunk_attention(0, x["q"], x["k"], x["v"], [0], [n], out=x["out"], workspace=work)
    last = work[need + (-need) % 256:][:2 * n * row].view(cfg.kv_dtype).view(n, 2, 128)  # just behind it
    want = store.chunk_attention(0, q, k, v, [0], [n])
    assert torch.equal(store.chunk_attention(0, q, k, v, [0], [n], out=last, workspace=work[:need]), want)
    L, one, zero = pkv.lib(), (ctypes.c_int32 * 1)(n), (ctypes.c_int32 * 1)(0)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.puzzlekv_read_tokens(store.handle, 0, zero, zero, one, 1, p(a), p(b), stream) != 0
    assert "overlap" in pkv.last_error()
    grow = 600  # longer than the ring: the pages leave through the workspace
    k, v = (x.cuda() for x in random_rows(cfg, grow, 3))
    need = store.chunk_workspace(0, [0], [grow])["append"]
    assert need > 0
    work = torch.empty(need + 2 * grow * row, dtype=torch.uint8, device="cuda")
    inside = work[need - 256:need - 256 + 2 * grow * row].view(cfg.kv_dtype)
    for x in ((inside, v), (k, inside)):
        assert L.puzzlekv_append_chunk(store.handle, 0, p(x[0]), p(x[1]), zero, (ctypes.c_int32 * 1)(grow), 1, p(work),
                                       need, stream) != 0
        assert "overlap" in pkv.last_error()
    assert store.stats(0, 0)["length"] == 700


def test_misaligned_buffers_are_refused(pkv):
    """Every device pointer of the chunk calls off by one element or byte: refused before anything is launched."""
    cfg = make_cfg(pkv, num_layers=1)
    store, _ = filled(pkv, cfg, [700, 0, 0, 0])
    L, B = pkv.lib(), (ctypes.c_int32 * 1)(0)
    n = (ctypes.c_int32 * 1)(3)
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    work = torch.zeros(store.chunk_workspace(0, [0], [3])["attention"], dtype=torch.uint8, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    at = lambda i, off: ctypes.c_void_p(buf.data_ptr() + (i << 17) + off)
    before = store.factor_pool.clone()

    def attend(p):
        return L.puzzlekv_chunk_attention(store.handle, 0, *p, B, n, 1, ctypes.c_void_p(work.data_ptr()), work.numel(), stream)

    def append(p):
        return L.puzzlekv_append_chunk(store.handle, 0, *p, B, n, 1, None, 0, stream)

    def read(p):
        return L.puzzlekv_read_tokens(store.handle, 0, B, B, n, 1, *p, stream)

    def load(p):
        return L.puzzlekv_load_factors(store.handle, 0, 0, 2, 1, *p, stream)

    for call, count in ((attend, 4), (append, 2), (read, 2), (load, 4)):
        for i in range(count):
            for off in (1, 2, 8):
                assert call([at(j, off if j == i else 0) for j in range(count)]) == pkv._lib.ERR_INVALID_ARG
                assert "aligned" in pkv.last_error()
    assert torch.equal(before, store.factor_pool) and store.stats(0, 0)["length"] == 700
    assert load([at(j, 0) for j in range(4)]) == 0 and attend([at(j, 0) for j in range(4)]) == 0
