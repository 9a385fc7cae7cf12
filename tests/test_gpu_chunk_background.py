"""Background factorization beside calls on several streams: every stream that reaches a batch's pages waits for the
batch, whichever stream did so first, and a capture is let through only after it.  The internal stream is held up by
a timed kernel, so that the batch has certainly not finished when the calls are queued."""
import pytest
import torch

from chunk_helpers import random_rows
from test_gpu_chunk import STORES, make_cfg, pkv, queries  # noqa: F401

pytestmark = pytest.mark.gpu


def hold_background(store):
    """Keep the store's internal stream busy for about half a second; returns the event behind which it is free."""
    done = torch.cuda.Event()
    with torch.cuda.stream(store.background_stream()):
        torch.cuda._sleep(1000)  # whatever a first use loads
        torch.cuda.synchronize()
        torch.cuda._sleep(1_000_000_000)
        done.record()
    return done


def check_held(held):
    """`held`: was the internal stream still busy when all calls were queued?  A host too slow for that shows nothing."""
    if not held:
        pytest.skip("the calls were queued too late: right, but nothing was pending any more")


@pytest.mark.parametrize("name", ["llama", "int4", "prerope", "fp32"])
def test_every_stream_waits_for_a_background_prefill(pkv, name):
    T, cfg = 1000, make_cfg(pkv, num_layers=1, **STORES[name])
    K, V = (x.cuda() for x in random_rows(cfg, T, 3, 1))
    k, v = (x.cuda() for x in random_rows(cfg, 150, 4))
    q = queries(cfg, 150, 5).cuda()
    want, got = pkv.Store(cfg), pkv.Store(cfg)
    want.load_prefill(1, K, V)
    rows = want.read_tokens(0, [1], [0], [T])
    long = want.chunk_attention(0, q, k, v, [1], [150])
    few = want.chunk_attention(0, q[:4], k[:4], v[:4], [1], [4])
    dec = torch.empty(1, cfg.num_q_heads, cfg.head_dim, device="cuda")
    want.decode_attention(0, q[:1], dec, [1])
    got.factor_pool.zero_()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(5)]
    hold = hold_background(got)
    got.factorize_layer(1, 0, K[0], V[0], background=True)
    ready = torch.cuda.Event()
    ready.record()  # the dense pages and the page table are the caller's to order
    for x in s:
        x.wait_event(ready)
    dec2 = torch.empty_like(dec)
    a = got.read_tokens(0, [1], [0], [T], stream=s[0])
    b = got.read_tokens(0, [1], [0], [T], stream=s[1])
    c = got.chunk_attention(0, q, k, v, [1], [150], stream=s[2])
    d = got.chunk_attention(0, q[:4], k[:4], v[:4], [1], [4], stream=s[3])
    got.decode_attention(0, q[:1], dec2, [1], stream=s[4])
    held = not hold.query()
    torch.cuda.synchronize()
    for x in (a, b):
        assert torch.equal(x[0], rows[0]) and torch.equal(x[1], rows[1])
    assert torch.equal(c, long) and torch.equal(d, few) and torch.equal(dec2, dec)
    check_held(held)


def test_conversions_beside_two_streams(pkv):
    """Two sequences whose pages are converted by one batch, grown past it on two streams."""
    cfg = make_cfg(pkv, num_layers=1)
    want, got = pkv.Store(cfg), pkv.Store(cfg)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in (want, got):
        for b in range(2):
            K, V = (x.cuda() for x in random_rows(cfg, 640, 20 + b, 1))
            s.load_prefill(b, K, V)
    lens = [640, 640]
    for step in range(6):
        grow = [[x.cuda() for x in random_rows(cfg, 64, 30 + 2 * step + b)] for b in range(2)]
        for b in range(2):
            want.append_chunk(0, *grow[b], [b], [64])
        rows = [want.read_tokens(0, [b], [0], [lens[b] + 64]) for b in range(2)]
        torch.cuda.synchronize()
        got.convert_ready_pages()
        read = []
        for b, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            got.append_chunk(0, *grow[b], [b], [64], stream=s)
            lens[b] += 64
            read.append(got.read_tokens(0, [b], [0], [lens[b]], stream=s))
        torch.cuda.synchronize()
        for x, y in zip(read, rows):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("name", ["llama", "nosink-nowindow"])
def test_tokens_alone_after_a_conversion(pkv, name):
    """Appends that never attend, past the ring's round: the batch's pages keep the rows it reads."""
    cfg = make_cfg(pkv, **STORES[name])
    want, got = pkv.Store(cfg), pkv.Store(cfg)
    K, V = (x.cuda() for x in random_rows(cfg, 640, 20, cfg.num_layers))
    n = 450
    k, v = (x.cuda() for x in random_rows(cfg, n, 21))
    for s in (want, got):
        s.load_prefill(0, K, V)
    for layer in range(cfg.num_layers):
        want.append_chunk(layer, k, v, [0], [n])
    for t in range(n):
        for layer in range(cfg.num_layers):
            got.append_token(layer, k[t:t + 1], v[t:t + 1], [0])
        got.convert_ready_pages()
    for layer in range(cfg.num_layers):
        for x, y in zip(want.read_tokens(layer, [0], [0], [640 + n]), got.read_tokens(layer, [0], [0], [640 + n])):
            assert torch.equal(x, y)


def test_more_batches_than_events(pkv):
    """More layers in the background than the store keeps events for."""
    T, L = 400, 13
    cfg = make_cfg(pkv, num_layers=L)
    K, V = (x.cuda() for x in random_rows(cfg, T, 3, L))
    want, got = pkv.Store(cfg), pkv.Store(cfg)
    want.load_prefill(0, K, V)
    rows = [want.read_tokens(l, [0], [0], [T]) for l in range(L)]
    torch.cuda.synchronize()
    hold = hold_background(got)
    for l in range(L):
        got.factorize_layer(0, l, K[l], V[l], background=True)
    ready = torch.cuda.Event()
    ready.record()
    streams = [torch.cuda.Stream() for _ in range(2)]
    read = []
    for s in streams:
        s.wait_event(ready)
        read.append([got.read_tokens(l, [0], [0], [T], stream=s) for l in range(L)])
    held = not hold.query()
    torch.cuda.synchronize()
    for r in read:
        for x, y in zip(r, rows):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert got.check_device_status() == 0
    check_held(held)


@pytest.mark.parametrize("here", [True, False])
def test_capture_beside_a_running_batch(pkv, here):
    """Let through where the captured stream itself has waited for the batch, refused where another one has."""
    cfg = make_cfg(pkv, num_layers=1)
    store = pkv.Store(cfg)
    K, V = (x.cuda() for x in random_rows(cfg, 640, 20, 1))
    store.load_prefill(0, K, V)
    k, v = (x.cuda() for x in random_rows(cfg, 3, 1))
    q = queries(cfg, 3, 2).cuda()
    want = store.chunk_attention(0, q, k, v, [0], [3])
    out, count = torch.zeros_like(q), torch.zeros(1, device="cuda")
    work = torch.empty(store.chunk_workspace(0, [0], [3])["attention"], dtype=torch.uint8, device="cuda")
    s, dense, g, refused = torch.cuda.Stream(), torch.cuda.Event(), torch.cuda.CUDAGraph(), False
    torch.cuda.synchronize()
    hold = hold_background(store)
    store.factorize_layer(0, 0, K[0], V[0], background=True)
    dense.record()
    s.wait_event(dense)
    store.wait_background(stream=s if here else None)
    with torch.cuda.stream(s):
        held = not hold.query()
        g.capture_begin()
        count.add_(1)
        try:
            store.chunk_attention(0, q, k, v, [0], [3], out=out, workspace=work)
        except pkv.PuzzleKVError as e:
            refused = "pending" in str(e)
        g.capture_end()
        g.replay()
    torch.cuda.synchronize()
    assert count.item() == 1
    if here:
        assert not refused and torch.equal(out, want)
    else:
        assert refused or not held
    check_held(held)
