"""Failure detection of the chunk, read and copy kernels, exercised without a GPU fault: one barrier of the first CTA
expects 16 bytes that no copy delivers, and that launch's waits run out after 2 ms.  The launch ends by itself, the host
learns of it from the status, and the next call answers as before."""
import pytest
import torch

from chunk_helpers import random_rows
from test_gpu_chunk import STORES, filled, live_state, make_cfg, pkv, queries, same_state  # noqa: F401

pytestmark = pytest.mark.gpu
FEW, STAGE, TILED, READ, COPY = 1, 2, 3, 4, 5


def ran_out(pkv, store):
    return store.check_device_status() == pkv._lib.ERR_DEVICE_TIMEOUT


@pytest.mark.parametrize("name,where,n", [("llama", FEW, 4), ("g1-p16", FEW, 60), ("llama", STAGE, 150), ("int4", STAGE, 4),
                                          ("prerope", STAGE, 40), ("llama", TILED, 150), ("g3-d64", TILED, 400),
                                          ("int4", TILED, 3)])
def test_attention(pkv, name, where, n):
    cfg = make_cfg(pkv, num_layers=1, **STORES[name])
    store, _ = filled(pkv, cfg, [1500, 300, 0, 0])
    k, v = (x.cuda() for x in random_rows(cfg, 2 * n, 1))
    q = queries(cfg, 2 * n, 2).cuda()
    attend = lambda: store.chunk_attention(0, q, k, v, [0, 1], [n, n])
    want = attend()
    assert store.check_device_status() == 0
    store.debug_fail_next_chunk_wait(where)
    got = attend()
    assert ran_out(pkv, store)
    if where == FEW:  # the first CTA works for the first KV head alone
        G = cfg.num_q_heads // cfg.num_kv_heads
        assert torch.equal(got[:, G:], want[:, G:])
    for _ in range(2):
        assert torch.equal(attend(), want)
    assert store.check_device_status() == 0, pkv.last_error()


@pytest.mark.parametrize("name", ["llama", "int4", "prerope", "g1-p16"])
def test_reads(pkv, name):
    cfg = make_cfg(pkv, num_layers=1, **STORES[name])
    store, _ = filled(pkv, cfg, [1500, 0, 0, 0])
    want = store.read_tokens(0, [0], [0], [1500])
    store.debug_fail_next_chunk_wait(READ)
    store.read_tokens(0, [0], [0], [1500])
    assert ran_out(pkv, store)
    for x, y in zip(store.read_tokens(0, [0], [0], [1500]), want):
        assert torch.equal(x, y)
    assert store.check_device_status() == 0


@pytest.mark.parametrize("name", ["llama", "fp32"])
def test_copies(pkv, name):
    cfg = make_cfg(pkv, **STORES[name])
    store, _ = filled(pkv, cfg, [1500, 0, 700, 0])
    want = [live_state(store, cfg, 0, l) for l in range(cfg.num_layers)]
    store.debug_fail_next_chunk_wait(COPY)
    store.copy_sequences([0, 0], [1, 2])
    assert ran_out(pkv, store)
    store.copy_sequences([0, 0], [1, 2])
    assert store.check_device_status() == 0
    for b in range(3):
        for l in range(cfg.num_layers):
            same_state(want[l], live_state(store, cfg, b, l))


def test_requests(pkv):
    """A request waits for its kernel, can be cleared, and is refused outside its range."""
    cfg = make_cfg(pkv, num_layers=1)
    store, _ = filled(pkv, cfg, [700, 0, 0, 0])
    k, v = (x.cuda() for x in random_rows(cfg, 3, 1))
    q = queries(cfg, 3, 2).cuda()
    want = store.chunk_attention(0, q, k, v, [0], [3])
    store.debug_fail_next_chunk_wait(READ)
    assert torch.equal(store.chunk_attention(0, q, k, v, [0], [3]), want)  # another kernel's
    store.debug_fail_next_chunk_wait(0)
    store.read_tokens(0, [0], [0], [700])
    assert store.check_device_status() == 0
    for bad in ((6, 50_000), (-1, 50_000), (1, 10), (1, 2_000_000_000)):
        with pytest.raises(pkv.PuzzleKVError):
            store.debug_fail_next_chunk_wait(*bad)
    fp32 = pkv.Store(make_cfg(pkv, num_layers=1, **STORES["fp32"]))
    with pytest.raises(pkv.PuzzleKVError, match="fp32"):
        fp32.debug_fail_next_chunk_wait(FEW)
