"""Chunk attention, chunk append, row reads and factor loads against 64-bit
references built from the factors the store holds, at the sizes and page kinds
where they can go wrong, and the refusals of each call."""
import itertools

import numpy as np
import pytest
import torch

import oracle
from chunk_helpers import U, U32, cache_rows, chunk_reference, excess, pair_abs, random_rows, turned
from gpu_helpers import HostCache, check_page_table
from store_layout import Layout, descriptors, factor_pool_slice, lengths, read_factors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from page_wise_rank_gb300 import build
    build.build()
    import page_wise_rank_gb300 as m
    return m


def make_cfg(pkv, **kw):
    base = dict(num_layers=2, num_kv_heads=2, num_q_heads=8, head_dim=128, page_size=64, rank_k=16, rank_v=24,
                sink_tokens=4, recent_tokens=128, max_batch=4, max_tokens_per_seq=2048, kv_dtype=torch.bfloat16)
    base.update(kw)
    return pkv.StoreConfig(**base)


# head counts, page sizes, ranks (odd and padded), windows of 0 and of odd sizes, types
STORES = {
    "llama": dict(),
    "g8": dict(num_q_heads=16, rank_k=24),
    "p32": dict(page_size=32, rank_v=14, recent_tokens=64),
    "g3-d64": dict(num_q_heads=6, head_dim=64, page_size=32, rank_k=8, rank_v=9, recent_tokens=33),
    "g1-p16": dict(num_kv_heads=3, num_q_heads=3, head_dim=64, page_size=16, rank_k=5, rank_v=7, sink_tokens=20,
                   recent_tokens=40),
    "nosink-nowindow": dict(sink_tokens=0, recent_tokens=0),
    "fullrank": dict(page_size=32, rank_k=32, rank_v=32, recent_tokens=32),
    "int4": dict(factor_int4=True),
    "int4-p32": dict(factor_int4=True, page_size=32, rank_v=14, recent_tokens=64),
    "prerope": dict(rope_theta=5e5),
    "prerope-d64": dict(head_dim=64, page_size=32, rank_k=8, rank_v=16, rope_theta=1e4, recent_tokens=50),
    "p16-d128": dict(page_size=16, rank_k=6, rank_v=16, recent_tokens=30),
    "p64-d64": dict(head_dim=64, rank_k=20, rank_v=12, num_q_heads=10),
    "int4-p16": dict(factor_int4=True, page_size=16, rank_k=8, rank_v=5, recent_tokens=30),
    "int4-p64-d64": dict(factor_int4=True, head_dim=64, rank_k=32, rank_v=9),
    "prerope-p64-d64": dict(head_dim=64, rank_k=8, rank_v=8, rope_theta=1e6, num_q_heads=6),
    "prerope-p32": dict(page_size=32, rank_k=12, rank_v=20, rope_theta=1e4),
    "fp32-d128": dict(kv_dtype=torch.float32, rank_k=20, rank_v=7, num_q_heads=4),
    "fp32": dict(kv_dtype=torch.float32, head_dim=64, page_size=32, rank_k=8, rank_v=8, recent_tokens=64),
    "fp32-g5": dict(kv_dtype=torch.float32, num_q_heads=10, page_size=16, rank_k=3, rank_v=11, recent_tokens=17),
}


def filled(pkv, cfg, lens, seed=0):
    """A store whose slot b holds lens[b] tokens (0 = empty) in every layer, and the rows it was fed."""
    store, host = pkv.Store(cfg), HostCache()
    for b, T in enumerate(lens):
        if T == 0:
            for l in range(cfg.num_layers):
                for h in range(cfg.num_kv_heads):
                    z = torch.zeros(0, cfg.head_dim, dtype=cfg.kv_dtype)
                    host.k[(b, l, h)], host.v[(b, l, h)] = [z], [z]
            continue
        K, V = random_rows(cfg, T, seed + 17 * b + 1, cfg.num_layers)
        store.load_prefill(b, K.cuda(), V.cuda())
        host.set_prefill(b, K, V)
    return store, host


def queries(cfg, N, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.3 * torch.randn(N, cfg.num_q_heads, cfg.head_dim, generator=g)).to(cfg.kv_dtype)


def append_host(host, layer, ids, counts, k, v):
    at = 0
    for b, n in zip(ids, counts):
        for j in range(n):
            host.append(b, layer, k[at + j], v[at + j])
        at += n


def check_attention(store, cfg, host, layer, ids, lens, counts, q, k, v, out, u_in=None):
    at, worst = 0, 0.0
    for b, T, n in zip(ids, lens, counts):
        s = slice(at, at + n)
        if n:
            ref, bound = chunk_reference(cfg, cache_rows(store, cfg, host, b, layer, T), k[s], v[s], q[s], T, u_in)
            worst = max(worst, excess(out[s], ref, bound))
        at += n
    return worst


@pytest.mark.parametrize("name", list(STORES))
@pytest.mark.parametrize("lens,counts", [
    ([0, 1, 63, 700], [3, 1, 2, 5]),          # empty slot, single tokens, short lists
    ([64, 65, 0, 1000], [1, 0, 1, 17]),       # a page's end, a sequence with nothing new
    ([131, 0, 500, 1], [140, 200, 1, 70]),    # long chunks beside single tokens
])
def test_attention_matches_64_bit(pkv, name, lens, counts):
    cfg = make_cfg(pkv, **STORES[name])
    store, host = filled(pkv, cfg, lens)
    ids = [2, 0, 3, 1]  # list order is not slot order
    lens_i, N = [lens[b] for b in ids], sum(counts)
    k, v = random_rows(cfg, N, 99)
    q = queries(cfg, N, 98)
    before = store.page_table.clone()
    for layer in range(cfg.num_layers):
        out = store.chunk_attention(layer, q.cuda(), k.cuda(), v.cuda(), ids, counts)
        assert out.dtype == cfg.kv_dtype and out.shape == q.shape
        assert check_attention(store, cfg, host, layer, ids, lens_i, counts, q, k, v, out) <= 1.0
        again = store.chunk_attention(layer, q.cuda(), k.cuda(), v.cuda(), ids, counts)
        assert torch.equal(out, again)  # sums are in a fixed order
    assert torch.equal(before, store.page_table)
    assert store.check_device_status() == 0


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 257])
@pytest.mark.parametrize("T", [0, 300, 1537])
def test_every_chunk_size(pkv, n, T):
    cfg = make_cfg(pkv, num_layers=1, max_batch=1, sink_tokens=4)
    store, host = filled(pkv, cfg, [T], seed=n)
    k, v = random_rows(cfg, n, n)
    q = queries(cfg, n, n + 1)
    out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), [0], [n])
    assert check_attention(store, cfg, host, 0, [0], [T], [n], q, k, v, out) <= 1.0


def test_sharp_and_flat_scores(pkv):
    """Scores of hundreds (one key takes all weight) and all equal (zero queries)."""
    cfg = make_cfg(pkv, num_layers=1, max_batch=1)
    store, host = filled(pkv, cfg, [900])
    for n in (5, 150):
        k, v = random_rows(cfg, n, 3)
        q = queries(cfg, n, 4)
        q[0::3] *= 60.0
        q[1::3] = 0.0
        out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), [0], [n])
        got = out.double().cpu().numpy()
        ref, bound = chunk_reference(cfg, cache_rows(store, cfg, host, 0, 0, 900), k, v, q, 900)
        keep = np.ones(n, bool)
        keep[0::3] = False  # there the bound's e^(2 ds) is no bound any more: only finite
        assert np.isfinite(got).all()
        assert excess(got[keep], ref[keep], bound[keep]) <= 1.0


@pytest.mark.parametrize("name", ["llama", "g3-d64", "g1-p16", "int4", "prerope", "fp32", "p64-d64"])
@pytest.mark.parametrize("T,n", [(0, 2), (5, 9), (1537, 6), (1537, 200), (130, 300)])
def test_nonfinite_tokens_reach_no_earlier_token(pkv, name, T, n):
    """Infinities and NaN in a value row turn their columns of the outputs that see them (weights are positive), and
    NaN in a key row the outputs of its own token; every other element is as if they were not there."""
    cfg = make_cfg(pkv, **STORES[name])
    store, host = filled(pkv, cfg, [T, 77, 0, 0])
    k, v = random_rows(cfg, n + 3, 31)
    q = queries(cfg, n + 3, 32)
    at, inf = n // 2, float("inf")
    poison = {0: inf, 9: float("nan"), cfg.head_dim - 1: -inf}
    bad_k, bad_v = k.clone(), v.clone()
    for c, x in poison.items():
        bad_v[at, 0, c], v[at, 0, c] = x, 0.0
    bad_k[n - 1, :, 5] = float("nan")
    out = store.chunk_attention(0, q.cuda(), bad_k.cuda(), bad_v.cuda(), [0, 1], [n, 3]).double().cpu().numpy()
    last, out[n - 1] = out[n - 1].copy(), 0.0
    assert np.isnan(last).all()
    G = cfg.num_q_heads // cfg.num_kv_heads
    for c, x in poison.items():
        got = out[at:n - 1, :G, c]
        assert np.isnan(got).all() if np.isnan(x) else (got == x).all()
        out[at:n - 1, :G, c] = 0.0
    ref, bound = chunk_reference(cfg, cache_rows(store, cfg, host, 0, 0, T), k[:n], v[:n], q[:n], T)
    ref[n - 1] = 0.0
    ref[at:n - 1, :G, list(poison)] = 0.0
    assert excess(out[:n], ref, bound) <= 1.0
    ref, bound = chunk_reference(cfg, cache_rows(store, cfg, host, 1, 0, 77), k[n:], v[n:], q[n:], 77)
    assert excess(out[n:], ref, bound) <= 1.0
    assert store.check_device_status() == 0


@pytest.mark.parametrize("n", [20, 1500])
def test_all_values_nonfinite(pkv, n):
    """Every value of a long chunk NaN: the answers are NaN, and the call ends as soon as any other."""
    cfg = make_cfg(pkv, num_layers=1, max_tokens_per_seq=4096)
    store, _ = filled(pkv, cfg, [400, 0, 0, 0])
    k, v = random_rows(cfg, n, 31)
    out = store.chunk_attention(0, queries(cfg, n, 2).cuda(), k.cuda(), torch.full_like(v, float("nan")).cuda(), [0], [n])
    assert out.isnan().all()
    assert store.check_device_status() == 0


def test_rows_beyond_the_lists_are_left_alone(pkv):
    """Padding after the last sequence (NaN inputs, a marked output) is neither read nor written."""
    cfg = make_cfg(pkv)
    store, host = filled(pkv, cfg, [200, 333, 0, 64])
    for counts in ([3, 2], [40, 90]):
        N, pad = sum(counts), 37
        k, v = random_rows(cfg, N, 5)
        q = queries(cfg, N, 6)
        big = [torch.cat([x, torch.full((pad, *x.shape[1:]), float("nan"), dtype=x.dtype)]).cuda() for x in (q, k, v)]
        out = torch.full_like(big[0], 7.0)
        store.chunk_attention(1, big[0][:N], big[1][:N], big[2][:N], [1, 0], counts, out=out[:N])
        assert check_attention(store, cfg, host, 1, [1, 0], [333, 200], counts, q, k, v, out[:N]) <= 1.0
        assert (out[N:] == 7.0).all()


def test_single_token_equals_decode(pkv):
    """A chunk of one token per sequence answers as the decode step does (no page leaves the window here)."""
    cfg = make_cfg(pkv, num_layers=1)
    lens = [200, 333, 90, 1001]
    store, host = filled(pkv, cfg, lens)
    k, v = random_rows(cfg, 4, 21)
    q = queries(cfg, 4, 22)
    out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), [0, 1, 2, 3], [1] * 4)
    dec = torch.empty(4, cfg.num_q_heads, cfg.head_dim, device="cuda")
    store.decode_step(0, q.cuda(), k.cuda(), v.cuda(), dec, [0, 1, 2, 3])
    at = 0
    for b, T in enumerate(lens):
        host_rows = cache_rows(store, cfg, host, b, 0, T)
        ref, bound = chunk_reference(cfg, host_rows, k[b:b + 1], v[b:b + 1], q[b:b + 1], T)
        assert excess(out[b:b + 1], ref, bound) <= 1.0 and excess(dec[b:b + 1], ref, bound) <= 1.0


def test_workspace_given_and_too_small(pkv):
    cfg = make_cfg(pkv)
    store, host = filled(pkv, cfg, [700, 0, 0, 0])
    k, v = (x.cuda() for x in random_rows(cfg, 9, 1))
    q = queries(cfg, 9, 2).cuda()
    need = store.chunk_workspace(0, [0], [9])
    assert need["attention"] > 0 and need["append"] == 0
    out = store.chunk_attention(0, q, k, v, [0], [9])
    work = torch.full((need["attention"],), 255, dtype=torch.uint8, device="cuda")  # NaN bit patterns
    assert torch.equal(out, store.chunk_attention(0, q, k, v, [0], [9], workspace=work))
    with pytest.raises(pkv.PuzzleKVError, match="workspace"):
        store.chunk_attention(0, q, k, v, [0], [9], workspace=work[:need["attention"] - 256])
    with pytest.raises(pkv.PuzzleKVError, match="workspace"):
        store.chunk_attention(0, q, k, v, [0], [9], workspace=torch.empty(need["attention"] + 64, dtype=torch.uint8,
                                                                         device="cuda")[64:])
    with pytest.raises(ValueError, match="workspace"):
        store.chunk_attention(0, q, k, v, [0], [9], workspace=work.cpu())


def test_capture_and_replay(pkv):
    """Attention replays from a graph; two graphs own two workspaces; calls that change the store are refused in a capture."""
    cfg = make_cfg(pkv)
    store, host = filled(pkv, cfg, [700, 130, 0, 0])
    store.wait_background()
    cases = [([0, 1], [4, 1]), ([1, 0], [150, 90])]
    graphs = []
    for ids, counts in cases:
        N = sum(counts)
        k, v = (x.cuda() for x in random_rows(cfg, N, N))
        q = queries(cfg, N, N).cuda()
        eager = store.chunk_attention(0, q, k, v, ids, counts)
        out = torch.zeros_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            store.chunk_attention(0, q, k, v, ids, counts, out=out)
        graphs.append((g, q, k, v, ids, counts, out, eager))
    for g, *_, out, eager in graphs + graphs:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    g, q, k, v, ids, counts, out, eager = graphs[0]
    q2 = queries(cfg, q.shape[0], 5).cuda()
    q.copy_(q2)
    g.replay()  # new queries through the same graph
    assert torch.equal(out, store.chunk_attention(0, q2, k, v, ids, counts))
    before = [dict(store.stats(b, 0)) for b in range(2)]
    s = torch.cuda.Stream()
    refused = []
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        torch.zeros(1, device="cuda")
        for call in (lambda: store.append_chunk(0, k, v, ids, counts), lambda: store.copy_sequences([0], [2]),
                     lambda: store.truncate_sequences([0], [690])):
            try:
                call()
            except pkv.PuzzleKVError as e:
                refused.append("captured" in str(e))
    assert refused == [True] * 3
    assert before == [dict(store.stats(b, 0)) for b in range(2)]


def test_side_stream(pkv):
    cfg = make_cfg(pkv)
    store, host = filled(pkv, cfg, [700, 130, 0, 0])
    k, v = (x.cuda() for x in random_rows(cfg, 150, 1))
    q = queries(cfg, 150, 2).cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = store.chunk_attention(0, q, k, v, [0], [150], stream=s)
    store.append_chunk(0, k, v, [0], [150], stream=s)
    kr, vr = store.read_tokens(0, [0], [700], [150], stream=s)
    s.synchronize()
    kc, vc = kr[-100:].clone(), vr[-100:].clone()  # the window's rows are exact
    assert torch.equal(kc, k[-100:]) and torch.equal(vc, v[-100:])
    assert check_attention(store, cfg, host, 0, [0], [700], [150], q.cpu(), k.cpu(), v.cpu(), out) <= 1.0


def test_values_of_every_size(pkv):
    """Value and key magnitudes from 1e-9 to 1e9, page by page and inside the chunk: the operand images' scales."""
    cfg = make_cfg(pkv, num_layers=1, max_batch=1)
    T = 1000
    for n in (6, 150):
        g = torch.Generator().manual_seed(n)
        K, V = random_rows(cfg, T, 70, 1)
        page = torch.arange(T) // 64
        V = (V.float() * (10.0 ** torch.randint(-9, 10, (17,), generator=g).float())[page][None, None, :, None]).to(cfg.kv_dtype)
        K = (K.float() * (10.0 ** torch.randint(-9, 1, (17,), generator=g).float())[page][None, None, :, None]).to(cfg.kv_dtype)
        store, host = pkv.Store(cfg), HostCache()
        store.load_prefill(0, K.cuda(), V.cuda())
        host.set_prefill(0, K, V)
        k, v = random_rows(cfg, n, 71)
        v = (v.float() * (10.0 ** torch.randint(-6, 7, (n, 1, 1), generator=g).float())).to(cfg.kv_dtype)
        q = queries(cfg, n, 72)
        out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), [0], [n])
        # beside values 2^60 times larger, a block's weights keep fewer bits
        assert check_attention(store, cfg, host, 0, [0], [T], [n], q, k, v, out, U[cfg.kv_dtype]) <= 1.0


@pytest.mark.parametrize("kw", [dict(rank_k=48, rank_v=24), dict(rank_k=1, rank_v=64), dict(rank_k=64, rank_v=8),
                                dict(num_kv_heads=1, num_q_heads=7), dict(recent_tokens=1000), dict(sink_tokens=300)])
def test_wide_ranks_heads_and_windows(pkv, kw):
    cfg = make_cfg(pkv, num_layers=1, **kw)
    lens, counts = [1500, 1, 640, 129], [5, 17, 1, 90]
    store, host = filled(pkv, cfg, lens)
    k, v = random_rows(cfg, sum(counts), 31)
    q = queries(cfg, sum(counts), 32)
    out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), [0, 1, 2, 3], counts)
    assert check_attention(store, cfg, host, 0, [0, 1, 2, 3], lens, counts, q, k, v, out) <= 1.0
    kr, vr = store.read_tokens(0, [0], [0], [1500])
    K, V, Ka, Va = cache_rows(store, cfg, host, 0, 0, 1500)
    for got, X, Xa in ((kr, K, Ka), (vr, V, Va)):
        bound = U[cfg.kv_dtype] * np.abs(X) + 84 * U32 * Xa
        assert excess(got, X.transpose(1, 0, 2), bound.transpose(1, 0, 2) * 1.01) <= 1.0


@pytest.mark.parametrize("name", ["llama", "g1-p16", "int4", "fp32"])
def test_sixty_four_sequences(pkv, name):
    """The longest list, lengths from empty to several pages, one to a few tokens and two longer chunks."""
    cfg = make_cfg(pkv, num_layers=1, max_batch=64, max_tokens_per_seq=700, **STORES[name])
    rng = np.random.RandomState(2)
    lens = [int(x) for x in rng.randint(0, 500, 64)]
    counts = [int(x) for x in rng.randint(0, 7, 64)]
    counts[5], counts[40] = 130, 77
    ids = [int(x) for x in rng.permutation(64)]
    store, host = filled(pkv, cfg, lens)
    N = sum(counts)
    k, v = random_rows(cfg, N, 41)
    q = queries(cfg, N, 42)
    out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), ids, counts)
    assert check_attention(store, cfg, host, 0, ids, [lens[b] for b in ids], counts, q, k, v, out) <= 1.0
    store.append_chunk(0, k.cuda(), v.cuda(), ids, counts)
    for b, n in zip(ids, counts):
        if lens[b] + n:
            check_page_table(store, cfg, b, 0, lens[b] + n)
    assert store.check_device_status() == 0


@pytest.mark.parametrize("n", [3, 40])
def test_long_context(pkv, n):
    cfg = make_cfg(pkv, num_layers=1, num_kv_heads=1, num_q_heads=4, max_batch=1, max_tokens_per_seq=70000)
    T = 65537
    store, host = filled(pkv, cfg, [T])
    k, v = random_rows(cfg, n, 1)
    q = queries(cfg, n, 2)
    out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), [0], [n])
    assert check_attention(store, cfg, host, 0, [0], [T], [n], q, k, v, out) <= 1.0


def test_two_streams_at_once(pkv):
    cfg = make_cfg(pkv)
    store, _ = filled(pkv, cfg, [900, 500, 0, 0])
    jobs = []
    for i, (ids, counts) in enumerate([([0], [4]), ([1], [200]), ([0, 1], [120, 3]), ([0], [90])]):
        N = sum(counts)
        k, v = (x.cuda() for x in random_rows(cfg, N, i))
        q = queries(cfg, N, i).cuda()
        jobs.append((ids, counts, q, k, v, store.chunk_attention(0, q, k, v, ids, counts)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = [store.chunk_attention(0, q, k, v, ids, counts, stream=s)
               for s, (ids, counts, q, k, v, _) in zip(streams, jobs)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b[-1]) for a, b in zip(got, jobs))


def test_pending_conversions_refuse_a_capture(pkv):
    cfg = make_cfg(pkv)
    store, _ = filled(pkv, cfg, [640, 0, 0, 0])
    k, v = (x.cuda() for x in random_rows(cfg, 3, 1))
    q = queries(cfg, 3, 2).cuda()
    want = store.chunk_attention(0, q, k, v, [0], [3])
    out = torch.zeros_like(q)
    store.convert_ready_pages()  # a batch on the internal stream
    g = torch.cuda.CUDAGraph()
    refused = False
    with torch.cuda.graph(g):
        torch.zeros(1, device="cuda")
        try:
            store.chunk_attention(0, q, k, v, [0], [3], out=out)
        except pkv.PuzzleKVError as e:
            refused = "pending" in str(e)
    assert refused
    store.wait_background()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        store.chunk_attention(0, q, k, v, [0], [3], out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---------------------------------------------------------------- rows


@pytest.mark.parametrize("name", list(STORES))
def test_read_tokens_matches_64_bit(pkv, name):
    cfg = make_cfg(pkv, **STORES[name])
    lens = [1000, 1, 0, 333]
    store, host = filled(pkv, cfg, lens)
    P = cfg.page_size
    pieces = [([0, 3], [0, 0], [1000, 333]), ([3, 1, 0, 2], [P - 1, 0, 5 * P + 3, 0], [2 * P + 3, 1, 1, 0]),
              ([0], [999], [1])]
    u, rank = U[cfg.kv_dtype], max(cfg.rank_k, cfg.rank_v)
    for ids, starts, counts in pieces:
        for layer in range(cfg.num_layers):
            k, v = store.read_tokens(layer, ids, starts, counts)
            at = 0
            for b, lo, n in zip(ids, starts, counts):
                K, V, Ka, Va = cache_rows(store, cfg, host, b, layer, lens[b])
                Ka = pair_abs(Ka, cfg.rope_theta)
                K = turned(K, 0, cfg.rope_theta) if lens[b] else K
                for got, X, Xa in ((k, K, Ka), (v, V, Va)):
                    ref = X[:, lo:lo + n].transpose(1, 0, 2)
                    # one rounding to kv_dtype; fp32 products of `rank` terms, scales and angles
                    bound = u * np.abs(ref) + (rank + 20) * U32 * Xa[:, lo:lo + n].transpose(1, 0, 2)
                    assert excess(got[at:at + n], ref, bound * 1.01 + 1e-30) <= 1.0
                at += n


def live_state(store, cfg, seq, layer):
    """Length, page table, live dense rows and factor records of one (sequence, layer), as stored."""
    lay = Layout(cfg)
    T = int(lengths(store, lay)[seq, layer])
    n = (T + cfg.page_size - 1) // cfg.page_size
    kinds, slots = descriptors(store, lay, seq, layer, lay.n_pg_max)
    assert (kinds[n:] == 0).all() and (slots[n:] == 0).all()
    k, v = store.read_tokens(layer, [seq], [0], [T]) if T else (None, None)
    records = []
    for h in range(cfg.num_kv_heads):
        pool = factor_pool_slice(store, lay, layer, seq, h)
        for p in np.nonzero(kinds[:n] == oracle.FACTORED)[0]:
            o = lay.record_offset(layer, seq, h, int(p))
            records.append(pool[o:o + lay.rec_bytes].copy())
    return T, kinds, slots, k, v, records


def same_state(a, b):
    T, kinds, slots, k, v, rec = a
    T2, kinds2, slots2, k2, v2, rec2 = b
    assert T == T2 and np.array_equal(kinds, kinds2) and np.array_equal(slots, slots2)
    assert (k is None and k2 is None) or (torch.equal(k, k2) and torch.equal(v, v2))
    assert len(rec) == len(rec2) and all(np.array_equal(x, y) for x, y in zip(rec, rec2))


@pytest.mark.parametrize("name", ["llama", "p32", "g1-p16", "nosink-nowindow", "int4", "prerope", "fp32"])
def test_append_chunk_equals_token_by_token(pkv, name):
    """Any cutting of the same tokens into chunks leaves the same bytes: lengths, page table, rows, records."""
    cfg = make_cfg(pkv, **STORES[name])
    lens = [0, 1, 130, 320]
    a, _ = filled(pkv, cfg, [1, 1, 130, 320])
    b, _ = filled(pkv, cfg, lens)
    grow = [700, 5, 200, 64]
    rows = [random_rows(cfg, n, 50 + i) for i, n in enumerate(grow)]
    first = random_rows(cfg, 1, 1, cfg.num_layers)  # slot 0 of `a` was given this prompt; b gets it as a token
    one = [x[:, :, 0].cuda() for x in first]
    rng = np.random.RandomState(3)
    for layer in range(cfg.num_layers):
        for t in range(max(grow)):
            ids = [i for i in range(4) if t < grow[i]]
            k = torch.stack([rows[i][0][t] for i in ids]).cuda()
            v = torch.stack([rows[i][1][t] for i in ids]).cuda()
            a.append_token(layer, k, v, ids)
        b.append_chunk(layer, one[0][layer][None].contiguous(), one[1][layer][None].contiguous(), [0], [1])
        at = [0] * 4
        while any(at[i] < grow[i] for i in range(4)):
            ids = list(rng.permutation(4))
            counts = [min(grow[i] - at[i], int(rng.choice([0, 1, 3, 64, 65, 400]))) for i in ids]
            k = torch.cat([rows[i][0][at[i]:at[i] + n] for i, n in zip(ids, counts)]).cuda()
            v = torch.cat([rows[i][1][at[i]:at[i] + n] for i, n in zip(ids, counts)]).cuda()
            b.append_chunk(layer, k, v, ids, counts)
            for i, n in zip(ids, counts):
                at[i] += n
    for layer in range(cfg.num_layers):
        for i in range(4):
            same_state(live_state(a, cfg, i, layer), live_state(b, cfg, i, layer))
            check_page_table(b, cfg, i, layer, [1, 1, 130, 320][i] + grow[i])
    assert b.check_device_status() == 0


def test_whole_prompt_as_one_chunk_equals_prefill(pkv):
    cfg = make_cfg(pkv, max_tokens_per_seq=4096)
    T = 3001
    K, V = random_rows(cfg, T, 8, cfg.num_layers)
    a, b = pkv.Store(cfg), pkv.Store(cfg)
    a.load_prefill(1, K.cuda(), V.cuda())
    for layer in range(cfg.num_layers):
        b.append_chunk(layer, K[layer].transpose(0, 1).contiguous().cuda(), V[layer].transpose(0, 1).contiguous().cuda(), [1], [T])
        same_state(live_state(a, cfg, 1, layer), live_state(b, cfg, 1, layer))


def test_chunked_prefill_with_background_conversion(pkv):
    """Chunks, decode steps and background conversions interleaved: the page kinds and the answers stay right."""
    cfg = make_cfg(pkv, num_layers=1, max_batch=2)
    store, host = filled(pkv, cfg, [0, 150])
    lens, rng = [0, 150], np.random.RandomState(5)
    for step in range(12):
        counts = [int(rng.choice([0, 1, 5, 60, 64, 190])) for _ in range(2)]
        if sum(counts) == 0:
            continue
        k, v = random_rows(cfg, sum(counts), 100 + step)
        q = queries(cfg, sum(counts), 200 + step)
        out = store.chunk_attention(0, q.cuda(), k.cuda(), v.cuda(), [0, 1], counts)
        assert check_attention(store, cfg, host, 0, [0, 1], lens, counts, q, k, v, out) <= 1.0
        store.append_chunk(0, k.cuda(), v.cuda(), [0, 1], counts)
        append_host(host, 0, [0, 1], counts, k, v)
        lens = [a + n for a, n in zip(lens, counts)]
        store.convert_ready_pages()
        if lens[0]:
            k1, v1 = random_rows(cfg, 2, 300 + step)
            q1 = queries(cfg, 2, 400 + step)
            dec = torch.empty(2, cfg.num_q_heads, cfg.head_dim, device="cuda")
            store.decode_step(0, q1.cuda(), k1.cuda(), v1.cuda(), dec, [0, 1])
            append_host(host, 0, [0, 1], [1, 1], k1, v1)
            lens = [a + 1 for a in lens]
    for b in range(2):
        check_page_table(store, cfg, b, 0, lens[b])
    assert store.check_device_status() == 0


@pytest.mark.parametrize("name", ["llama", "p32", "g1-p16", "fp32"])
def test_load_factors_roundtrip(pkv, name):
    cfg = make_cfg(pkv, **STORES[name])
    store, _ = filled(pkv, cfg, [0, 0, 1000, 0])
    P, H, d = cfg.page_size, cfg.num_kv_heads, cfg.head_dim
    g = torch.Generator().manual_seed(4)
    p0, n = 3, 5
    f = [torch.randn(H, n, *s, generator=g).to(cfg.kv_dtype) for s in
         ((P, cfg.rank_k), (cfg.rank_k, d), (P, cfg.rank_v), (cfg.rank_v, d))]
    before = live_state(store, cfg, 2, 0)
    store.load_factors(1, 2, p0, *(x.cuda() for x in f))
    lay = Layout(cfg)
    for h in range(H):
        pool = factor_pool_slice(store, lay, 1, 2, h)
        for i in range(n):
            for got, x in zip(read_factors(pool, lay, 1, 2, h, p0 + i), f):
                assert np.array_equal(got, x[h, i].double().numpy())
    same_state(before, live_state(store, cfg, 2, 0))  # the other layer is untouched


# ---------------------------------------------------------------- refusals


def test_refusals(pkv):
    cfg = make_cfg(pkv, max_tokens_per_seq=300)
    store, _ = filled(pkv, cfg, [200, 0, 64, 0])
    k, v = (x.cuda() for x in random_rows(cfg, 101, 1))
    q = queries(cfg, 101, 2).cuda()
    before = store.page_table.clone()

    def bad(fn, *a, match=None, **kw):
        with pytest.raises((pkv.PuzzleKVError, ValueError), match=match):
            fn(*a, **kw)

    bad(store.chunk_attention, 0, q, k, v, [0], [101], match="exceed")      # past the capacity
    bad(store.append_chunk, 0, k, v, [0], [101], match="exceed")
    bad(store.chunk_attention, 2, q, k, v, [0], [101], match="layer")
    bad(store.chunk_attention, 0, q, k, v, [4], [101], match="out of range")
    bad(store.chunk_attention, 0, q, k, v, [0, 0], [50, 51], match="twice")
    bad(store.chunk_attention, 0, q, k, v, [0, 2], [-1, 102], match="negative")
    bad(store.chunk_attention, 0, q, k, v, [], [])
    bad(store.chunk_attention, 0, q, k, v, [0], [101, 0], match="counts")
    bad(store.chunk_attention, 0, q[:50], k, v, [2], [101])
    bad(store.chunk_attention, 0, q.float(), k, v, [2], [101])
    bad(store.chunk_attention, 0, q.transpose(0, 1), k, v, [2], [101])
    bad(store.chunk_attention, 0, q, k, v, [2], [101], out=torch.empty_like(q, dtype=torch.float32))
    bad(store.chunk_attention, 0, q.cpu(), k, v, [2], [101])
    bad(store.read_tokens, 0, [0], [0], [201], match="rows")
    bad(store.read_tokens, 0, [0], [-1], [1])
    bad(store.read_tokens, 0, [1], [0], [1])
    bad(store.read_tokens, 0, [0], [2 ** 31 - 1], [2 ** 31 - 1])
    bad(store.truncate_sequences, [0], [201], match="fewer")
    bad(store.truncate_sequences, [0], [-1], match="negative")
    bad(store.truncate_sequences, [0, 0], [10, 10], match="twice")
    bad(store.copy_sequences, [1], [0], match="no tokens")
    bad(store.copy_sequences, [0, 2], [1, 1], match="twice")
    bad(store.copy_sequences, [0], [4], match="out of range")
    bad(store.copy_sequences, [-1], [1], match="out of range")
    z = [torch.zeros(2, 1, *s, dtype=cfg.kv_dtype, device="cuda") for s in ((64, 16), (16, 128), (64, 24), (24, 128))]
    bad(store.load_factors, 0, 0, 0, *z, match="pages")   # a sink page
    bad(store.load_factors, 0, 0, 3, *z, match="pages")   # an incomplete page
    bad(store.load_factors, 0, 1, 1, *z, match="pages")   # an empty slot
    assert torch.equal(before, store.page_table)
    # nothing to do is no error
    e = [x[:0] for x in (q, k, v)]
    assert store.chunk_attention(0, *e, [0, 1], [0, 0]).shape[0] == 0
    store.append_chunk(0, e[1], e[2], [0, 1], [0, 0])
    assert store.read_tokens(0, [1], [0], [0])[0].shape[0] == 0
    store.chunk_attention(0, q[:100], k[:100], v[:100], [0], [100])  # exactly to the capacity
    store.append_chunk(0, k[:100], v[:100], [0], [100])
    assert store.stats(0, 0)["length"] == 300
    bad(store.copy_sequences, [0], [1], match="different lengths")  # layer 1 is behind
    q4 = filled(pkv, make_cfg(pkv, factor_int4=True), [200, 0, 0, 0])[0]
    bad(q4.load_factors, 0, 0, 1, *z, match="INT4")
