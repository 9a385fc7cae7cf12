"""Copies and cuts of whole sequences: forks, permutations and cycles, roll-back
of drafted tokens, and the run of chunk calls a server makes with them."""
import numpy as np
import pytest
import torch

import oracle
from chunk_helpers import cache_rows, chunk_reference, excess, random_rows
from gpu_helpers import HostCache, check_page_table
from test_gpu_chunk import STORES, append_host, check_attention, filled, live_state, make_cfg, pkv, queries, same_state  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["llama", "g1-p16", "int4", "prerope", "fp32", "nosink-nowindow"])
@pytest.mark.parametrize("src,dst", [
    ([0], [3]),                      # one copy into an empty slot
    ([0, 0, 0], [1, 2, 3]),          # a fork over filled slots
    ([1, 0], [0, 1]),                # a swap
    ([1, 2, 0, 2], [0, 1, 2, 3]),    # a cycle with a fork
    ([2, 1, 2], [0, 1, 1 + 2]),      # a sequence onto itself beside others
])
def test_copies_are_simultaneous(pkv, name, src, dst):
    cfg = make_cfg(pkv, **STORES[name])
    lens = [900, 131, 470, 0]
    store, host = filled(pkv, cfg, lens)
    want = {(b, l): live_state(store, cfg, b, l) for b in range(4) for l in range(cfg.num_layers)}
    store.copy_sequences(src, dst)
    came = {d: s for s, d in zip(src, dst)}
    for b in range(4):
        for l in range(cfg.num_layers):
            same_state(want[(came.get(b, b), l)], live_state(store, cfg, b, l))
            assert store.stats(b, l)["length"] == lens[came.get(b, b)]
    assert store.check_device_status() == 0


def test_many_sources(pkv):
    """64 pairs: the narrowest staging tile, a full rotation."""
    cfg = make_cfg(pkv, num_layers=1, num_kv_heads=1, num_q_heads=2, max_batch=64, max_tokens_per_seq=600)
    lens = [1 + 9 * b for b in range(64)]
    store, _ = filled(pkv, cfg, lens)
    want = [live_state(store, cfg, b, 0) for b in range(64)]
    store.copy_sequences([(b + 1) % 64 for b in range(64)], list(range(64)))
    for b in range(64):
        same_state(want[(b + 1) % 64], live_state(store, cfg, b, 0))


def test_copies_go_their_own_way(pkv):
    """After a fork both sequences grow with different tokens, window pages converted ahead included."""
    cfg = make_cfg(pkv, num_layers=1)
    store, host = filled(pkv, cfg, [500, 0, 0, 0])
    store.factorize_pages()  # also the complete pages still in the window
    store.copy_sequences([0, 0], [1, 2])
    for h in range(cfg.num_kv_heads):
        for b in (1, 2):
            host.k[(b, 0, h)], host.v[(b, 0, h)] = list(host.k[(0, 0, h)]), list(host.v[(0, 0, h)])
    lens = [500] * 3
    for step in range(4):
        counts = [70, 3, 129]
        k, v = random_rows(cfg, sum(counts), 40 + step)
        q = queries(cfg, sum(counts), 60 + step)
        out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), [2, 0, 1], counts)
        assert check_attention(store, cfg, host, 0, [2, 0, 1], [lens[2], lens[0], lens[1]], counts, q, k, v, out) <= 1.0
        store.append_chunk(0, k.cuda(), v.cuda(), [2, 0, 1], counts)
        append_host(host, 0, [2, 0, 1], counts, k, v)
        lens = [lens[0] + 3, lens[1] + 129, lens[2] + 70]
        for b in range(3):
            check_page_table(store, cfg, b, 0, lens[b])


@pytest.mark.parametrize("name", ["llama", "p32", "g1-p16", "nosink-nowindow", "fp32", "int4"])
def test_rejected_tokens_leave_no_trace(pkv, name):
    """Append drafts, cut back, append others: the same bytes as a store that never saw the drafts, at every
    position relative to the pages and with conversions running ahead."""
    cfg = make_cfg(pkv, **STORES[name])
    P = cfg.page_size
    a, _ = filled(pkv, cfg, [P + 5, 0, 3 * P, 0])
    b, _ = filled(pkv, cfg, [P + 5, 0, 3 * P, 0])
    lens = {0: P + 5, 2: 3 * P}
    rng = np.random.RandomState(1)
    for step in range(14):
        for layer in range(cfg.num_layers):
            good = {i: random_rows(cfg, 1 + (7 * step + i) % P, 1000 * step + i + layer) for i in lens}
            # the layers take different numbers of drafts
            drop = {i: random_rows(cfg, int(rng.randint(1, P - 1)), 5000 + 1000 * step + i) for i in lens}
            ids = list(lens)
            cat = lambda rows, j: torch.cat([rows[i][j] for i in ids]).cuda()
            a.append_chunk(layer, cat(good, 0), cat(good, 1), ids, [good[i][0].shape[0] for i in ids])
            b.append_chunk(layer, cat(drop, 0), cat(drop, 1), ids, [drop[i][0].shape[0] for i in ids])
        b.convert_ready_pages()  # pages completed by drafts are factorized ahead; the cut voids them
        b.truncate_sequences(ids, [lens[i] for i in ids])
        for layer in range(cfg.num_layers):
            good = {i: random_rows(cfg, 1 + (7 * step + i) % P, 1000 * step + i + layer) for i in lens}
            b.append_chunk(layer, cat(good, 0), cat(good, 1), ids, [good[i][0].shape[0] for i in ids])
        for i in ids:
            lens[i] += 1 + (7 * step + i) % P
            for layer in range(cfg.num_layers):
                same_state(live_state(a, cfg, i, layer), live_state(b, cfg, i, layer))
    assert b.check_device_status() == 0


def test_cut_to_nothing_and_reuse(pkv):
    cfg = make_cfg(pkv)
    a, _ = filled(pkv, cfg, [700, 0, 0, 0])
    a.factorize_pages()
    a.truncate_sequences([0, 1], [0, 0])
    assert a.stats(0, 0)["length"] == 0 and a.stats(0, 0)["dense_pages"] == 0
    with pytest.raises(pkv.PuzzleKVError, match="no tokens"):
        a.decode_attention(0, torch.zeros(1, 8, 128, dtype=torch.bfloat16, device="cuda"),
                           torch.zeros(1, 8, 128, device="cuda"), [0])
    b, _ = filled(pkv, cfg, [0, 0, 0, 0])
    k, v = (x.cuda() for x in random_rows(cfg, 333, 6))
    for s in (a, b):
        for layer in range(cfg.num_layers):
            s.append_chunk(layer, k, v, [0], [333])
    for layer in range(cfg.num_layers):
        same_state(live_state(a, cfg, 0, layer), live_state(b, cfg, 0, layer))


def test_cut_too_far_is_refused(pkv):
    """A page that would be dense again has left the ring, or came factorized with the prompt: nothing changes."""
    cfg = make_cfg(pkv)
    store, _ = filled(pkv, cfg, [700, 700, 0, 0])
    k, v = (x.cuda() for x in random_rows(cfg, 300, 6))
    for layer in range(cfg.num_layers):
        store.append_chunk(layer, k, v, [0], [300])
    before = [live_state(store, cfg, b, l) for b in range(2) for l in range(cfg.num_layers)]
    for b, T in ((0, 700), (1, 500), (1, 639)):
        with pytest.raises(pkv.PuzzleKVError, match="cannot go back"):
            store.truncate_sequences([b], [T])
    for x, (b, l) in zip(before, [(b, l) for b in range(2) for l in range(cfg.num_layers)]):
        same_state(x, live_state(store, cfg, b, l))
    # within the guarantee, and as far as the ring goes
    store.truncate_sequences([0, 1], [1000 - 64, 700 - 60])
    for l in range(cfg.num_layers):
        check_page_table(store, cfg, 0, l, 936)
        check_page_table(store, cfg, 1, l, 640)
    store.truncate_sequences([0], [63])  # only the sink page is left: always there
    check_page_table(store, cfg, 0, 0, 63)


@pytest.mark.parametrize("name,T", [("llama", 40), ("llama", 64), ("p32", 9), ("nosink-nowindow", 320), ("fp32", 16)])
def test_grown_again_after_a_long_cut(pkv, name, T):
    """A cut that leaves no dense page past the sink (the ring has moved on): pages filled afterwards are in the ring,
    so they are copied and can be cut into like any others."""
    cfg = make_cfg(pkv, **STORES[name])
    P = cfg.page_size
    store, _ = filled(pkv, cfg, [900, 0, 0, 0])
    fresh, _ = filled(pkv, cfg, [900, 0, 0, 0])
    n = 2 * P + 3
    for layer in range(cfg.num_layers):
        k, v = (x.cuda() for x in random_rows(cfg, 300, 6 + layer))
        store.append_chunk(layer, k, v, [0], [300])
    for s in (store, fresh):  # `fresh` is cut without having grown
        s.truncate_sequences([0], [T])
        for layer in range(cfg.num_layers):
            k, v = (x.cuda() for x in random_rows(cfg, n, 60 + layer))
            s.append_chunk(layer, k, v, [0], [n])
        s.copy_sequences([0, 0], [1, 2])
        s.truncate_sequences([0, 2], [T + n - 2, T + n - 2])
    for layer in range(cfg.num_layers):
        cut = live_state(store, cfg, 0, layer)
        same_state(cut, live_state(store, cfg, 2, layer))
        same_state(cut, live_state(fresh, cfg, 0, layer))
        same_state(live_state(store, cfg, 1, layer), live_state(fresh, cfg, 1, layer))
        k1, v1 = store.read_tokens(layer, [1], [0], [T + n - 2])
        k0, v0 = store.read_tokens(layer, [0], [0], [T + n - 2])
        lo = max(0, T + n - 2 - P)  # the rows of the last pages are dense at both lengths
        assert torch.equal(k1[lo:], k0[lo:]) and torch.equal(v1[lo:], v0[lo:])


def test_offsets_past_32_bits(pkv):
    """Long sequences whose records and operand images lie more than 4 GiB into their buffers: the same rows as a
    store of one sequence, and the same attention.  The two calls share their operands but cut the keys in other
    places, so weights and states round differently (2^-11 of sum w |v| each, at most max |v| = 2^-11 * 8 here) and both
    outputs round once (2^-8 of the value each)."""
    T, n, last = 131000, 70, 17
    base = dict(num_layers=1, num_kv_heads=8, num_q_heads=32, max_tokens_per_seq=131072)
    big, one = pkv.Store(make_cfg(pkv, max_batch=last + 1, **base)), pkv.Store(make_cfg(pkv, max_batch=1, **base))
    assert big.factor_pool.numel() > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *shape: (0.6 * torch.randn(shape, generator=g, device="cuda")).clamp(-4, 4).bfloat16()
    K, V = rnd(1, 8, T, 128), rnd(1, 8, T, 128)
    big.load_prefill(0, K, V)
    big.copy_sequences([0] * (last - 1), list(range(1, last)))
    V += 2  # the last sequence's outputs are near 2, the others' near 0
    big.load_prefill(last, K, V)
    one.load_prefill(0, K, V)
    for start in (0, T - 500):
        for x, y in zip(big.read_tokens(0, [last], [start], [500]), one.read_tokens(0, [0], [start], [500])):
            assert torch.equal(x, y)
    for x, y in zip(big.read_tokens(0, [last - 1], [64], [500]), big.read_tokens(0, [0], [64], [500])):
        assert torch.equal(x, y)
    q, k, v = rnd(n, 32, 128), rnd(n, 8, 128), rnd(n, 8, 128) + 2
    ids = list(range(8, last + 1))
    assert big.chunk_workspace(0, ids, [n] * len(ids))["attention"] > 1 << 32
    got = big.chunk_attention(0, *(x.repeat(len(ids), 1, 1) for x in (q, k, v)), ids, [n] * len(ids))[-n:]
    want = one.chunk_attention(0, q, k, v, [0], [n])
    few = [s.chunk_attention(0, q[:4], k[:4], v[:4], [b], [4]) for s, b in ((big, last), (one, 0))]  # over the pages
    for a, b in ((got, want), few):
        assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2 * 2.0 ** -11 * 8).all()
    assert want.float().mean() > 1.5
    big.append_chunk(0, k, v, [last], [n])
    one.append_chunk(0, k, v, [0], [n])
    for x, y in zip(big.read_tokens(0, [last], [T - 300], [300 + n]), one.read_tokens(0, [0], [T - 300], [300 + n])):
        assert torch.equal(x, y)
    assert big.check_device_status() == 0


def test_serving_run(pkv):
    """A prompt in chunks, forked, drafts verified, some rejected, beams reordered, single tokens decoded: every answer
    against 64 bits."""
    cfg = make_cfg(pkv, num_layers=1)
    store, host = filled(pkv, cfg, [0, 0, 0, 0])
    T = 0
    for step, n in enumerate((300, 257, 1, 90)):
        k, v = random_rows(cfg, n, step)
        q = queries(cfg, n, 50 + step)
        out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), [0], [n])
        assert check_attention(store, cfg, host, 0, [0], [T], [n], q, k, v, out) <= 1.0
        store.append_chunk(0, k.cuda(), v.cuda(), [0], [n])
        append_host(host, 0, [0], [n], k, v)
        T += n
    store.copy_sequences([0, 0, 0], [1, 2, 3])
    for h in range(cfg.num_kv_heads):
        for b in (1, 2, 3):
            host.k[(b, 0, h)], host.v[(b, 0, h)] = list(host.k[(0, 0, h)]), list(host.v[(0, 0, h)])
    lens, ids = [T] * 4, [0, 1, 2, 3]
    for step in range(25):
        counts = [(step * 3 + 2 * b) % 7 + 1 for b in range(4)]
        k, v = random_rows(cfg, sum(counts), 700 + step)
        q = queries(cfg, sum(counts), 800 + step)
        out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), ids, counts)
        assert check_attention(store, cfg, host, 0, ids, lens, counts, q, k, v, out) <= 1.0
        store.append_chunk(0, k.cuda(), v.cuda(), ids, counts)
        accepted = [max(1, c - (step + b) % 3) for b, c in enumerate(counts)]
        at = 0
        for b in range(4):
            append_host(host, 0, [b], [accepted[b]], k[at:], v[at:])
            at += counts[b]
        lens = [a + n for a, n in zip(lens, accepted)]
        store.truncate_sequences(ids, lens)
        store.convert_ready_pages()
        if step % 5 == 4:
            store.copy_sequences([1, 3, 0, 3], ids)
            lens = [lens[1], lens[3], lens[0], lens[3]]
            old = {key: list(x) for key, x in host.k.items()}, {key: list(x) for key, x in host.v.items()}
            for h in range(cfg.num_kv_heads):
                for d, s in enumerate((1, 3, 0, 3)):
                    host.k[(d, 0, h)], host.v[(d, 0, h)] = list(old[0][(s, 0, h)]), list(old[1][(s, 0, h)])
        for b in range(4):
            check_page_table(store, cfg, b, 0, lens[b])
    k, v = random_rows(cfg, 4, 1)
    q = queries(cfg, 4, 2)
    dec = torch.empty(4, cfg.num_q_heads, cfg.head_dim, device="cuda")
    store.append_token(0, k.cuda(), v.cuda(), ids)
    append_host(host, 0, ids, [1] * 4, k, v)
    store.decode_attention(0, q.cuda(), dec, ids)
    for b in range(4):  # the decode output at its own length: a chunk reference whose last cached row is the new token
        K, V, Ka, Va = cache_rows(store, cfg, host, b, 0, lens[b] + 1)
        rows = K[:, :-1], V[:, :-1], Ka[:, :-1], Va[:, :-1]
        ref, bound = chunk_reference(cfg, rows, k[b:b + 1], v[b:b + 1], q[b:b + 1], lens[b])
        assert excess(dec[b:b + 1], ref, bound) <= 1.0
    assert store.check_device_status() == 0
