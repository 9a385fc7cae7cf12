"""Chunk attention over values of unlike sizes: the tensor-core path holds values and weights in fp16 with powers of
two, and each answer is held to a bound set by the row's own weighted sum, not by the largest value in the store."""
import math

import numpy as np
import pytest
import torch

from chunk_helpers import U, U32, U_IN, cache_rows, pair_abs, turned
from gpu_helpers import HostCache
from test_gpu_chunk import make_cfg, pkv, queries  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = {
    "bf16": dict(),
    "int4": dict(factor_int4=True),
    "prerope": dict(rope_theta=5e5),
    "d64-p16": dict(head_dim=64, page_size=16, rank_k=6, rank_v=7, recent_tokens=40),
}
SINK, LOW = 6.0, -11.0  # what the first tokens' and the low blocks' scores are raised by (before RoPE)


def excess_of_tokens(cfg, rows, k, v, q, T, tokens, out, weight_floor=2.0 ** -21):
    """Largest error over its bound among the outputs of chunk tokens `tokens`.

    With ui = 2^-11, the half step of fp16 operands: a score is off by ds = (2 ui + (d + rank + 20) 2^-24) max |q||k|
    / sqrt(d), a weight by the factor e^(2 ds), by ui of itself and, under fp16's normal range, by `weight_floor` of the
    row's largest weight (half a step there is 2^-25; a block's values may be a step of 2^4 short of the others'
    power); a value by ui of itself and, under the range, by 2^-36 of the largest value of its head (a block's image
    reaches 2^11).  Sums are fp32; the output is rounded once."""
    K, V, Ka, Va = rows
    H, G, d = cfg.num_kv_heads, cfg.num_q_heads // cfg.num_kv_heads, cfg.head_dim
    kn, vn = (x.double().cpu().numpy().transpose(1, 0, 2) for x in (k, v))
    K = np.concatenate([turned(K, 0, cfg.rope_theta), turned(kn, T, cfg.rope_theta)], 1)
    Ka = pair_abs(np.concatenate([Ka, np.abs(kn)], 1), cfg.rope_theta)
    V, Va = np.concatenate([V, vn], 1), np.concatenate([Va, np.abs(vn)], 1)
    qn, got = q.double().cpu().numpy(), out.double().cpu().numpy()
    assert np.isfinite(got).all()
    u, ui, rank, worst = U[cfg.kv_dtype], U_IN[cfg.kv_dtype], max(cfg.rank_k, cfg.rank_v), 0.0
    for j in tokens:
        see = T + j + 1
        for h in range(H):
            qr = qn[j, h * G:(h + 1) * G]
            s = qr @ K[h, :see].T / math.sqrt(d)
            A = (np.abs(qr) @ Ka[h, :see].T / math.sqrt(d)).max(1, keepdims=True)
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            o, B = w @ V[h, :see], w @ Va[h, :see]
            ds = (2 * ui + (d + rank + 20) * U32) * A
            inner = ((np.expm1(2 * ds) + 2.05 * ui + (see + rank + 40) * U32) * B +
                     weight_floor * w.max(1, keepdims=True) * np.abs(V[h, :see]).sum(0, keepdims=True) +
                     2.0 ** -36 * np.abs(V[h]).max())
            bound = inner + u * (np.abs(o) + inner)
            worst = max(worst, float((np.abs(got[j, h * G:(h + 1) * G] - o) / np.maximum(bound, 1e-300)).max()))
    return worst


def sized_values(name, n, d, g):
    """Values of n positions, [n, d] factors and offsets applied to normal numbers: (scale, mean) per position and column."""
    scale, mean = torch.ones(n, d), torch.zeros(n, d)
    blk = torch.arange(n) // 128
    if name == "around-2^-8":          # blocks' maxima on both sides of 1/256
        scale *= 0.00085
        mean += 0.000425
    elif name == "one-step":           # a larger block before smaller ones
        scale *= torch.where(blk == 0, 0.0012, 0.0007)[:, None]
    elif name == "one-ordinary":       # one ordinary block among small ones
        scale *= torch.where(blk == 4, 0.6, 1e-4 + 4e-4 * torch.rand(n, generator=g))[:, None]
    elif name == "zero-first":         # no size at all in the first blocks, nor in one in between
        scale *= torch.where((blk < 2) | (blk == 6), 0.0, 0.002)[:, None]
    elif name == "alternating":        # neighbours 2^-17 and 2^17 apart, both ways
        scale *= torch.where(blk % 2 == 1, 1.0, 1e-5)[:, None]
        mean += torch.where(blk % 2 == 1, 0.0, 2e-5)[:, None]
    elif name == "columns":            # columns of unlike sizes side by side
        scale *= 10.0 ** -(torch.arange(d) % 9).float()[None]
        mean += 0.5 * scale
    elif name == "falling":            # every block a quarter of the one before
        scale *= (4.0 ** -(blk % 12).float())[:, None]
    return scale, mean


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("name", ["around-2^-8", "one-step", "one-ordinary", "zero-first", "alternating", "columns", "falling"])
def test_values_of_unlike_sizes(pkv, kind, name):
    """1,024 tokens over 1,500: long enough that a CTA's piece holds many blocks.  The first tokens are sinks that draw
    weight, and the large blocks of "one-ordinary" and "alternating" draw little."""
    cfg = make_cfg(pkv, num_layers=1, num_kv_heads=8, num_q_heads=32, max_batch=1, max_tokens_per_seq=4096, **KINDS[kind])
    T, n, H, d = 1500, 1024, cfg.num_kv_heads, cfg.head_dim
    g = torch.Generator().manual_seed(len(name) + 7)
    scale, mean = sized_values(name, T + n, d, g)
    axis = torch.zeros(d)
    axis[d - 1] = axis[d // 2 - 1] = 0.5 ** 0.5  # the slowest pair under RoPE
    k = 0.6 * torch.randn(H, T + n, d, generator=g)
    v = torch.randn(H, T + n, d, generator=g) * scale + mean
    lift = torch.zeros(T + n)
    lift[:4] = SINK
    low = torch.arange(T + n) // 128
    if name == "one-ordinary":
        lift[low == 4] = LOW
    if name == "alternating":
        lift[low % 2 == 1] = LOW
    k += axis * (lift * math.sqrt(d) / 8)[None, :, None]
    q = queries(cfg, n, 3).float() * 0.6 + 8 * axis
    k, v, q = k.to(cfg.kv_dtype), v.to(cfg.kv_dtype), q.to(cfg.kv_dtype)
    store, host = pkv.Store(cfg), HostCache()
    store.load_prefill(0, k[None, :, :T].contiguous().cuda(), v[None, :, :T].contiguous().cuda())
    host.set_prefill(0, k[None, :, :T], v[None, :, :T])
    kn, vn = (x[:, T:].transpose(0, 1).contiguous() for x in (k, v))
    out = store.chunk_attention(0, q.cuda(), kn.cuda(), vn.cuda(), [0], [n])
    rows = cache_rows(store, cfg, host, 0, 0, T)
    tokens = [0, 1, 35, 36, 163, 164, 400, 675, 676, 1000, n - 1]  # ends of blocks among them
    assert excess_of_tokens(cfg, rows, kn, vn, q, T, tokens, out) <= 1.0
    few = store.chunk_attention(0, q[:5].cuda(), kn[:5].cuda(), vn[:5].cuda(), [0], [5])
    assert excess_of_tokens(cfg, rows, kn, vn, q, T, range(5), few) <= 1.0
    assert store.check_device_status() == 0


@pytest.mark.parametrize("bits", [20.5, 25.5, 28.0])
def test_long_tails_count(pkv, bits):
    """One key draws nearly all weight and its value is zero: the answer is what thousands of keys of 2^-bits of its
    weight add up to.  All blocks share a power here, and weights are held to 2^-32 of the largest."""
    T, n = 3600, 1024
    cfg = make_cfg(pkv, num_layers=1, num_kv_heads=8, num_q_heads=32, max_batch=1, max_tokens_per_seq=T + n,
                   recent_tokens=T)
    H, d = cfg.num_kv_heads, cfg.head_dim
    g = torch.Generator().manual_seed(5)
    axis = torch.zeros(d)
    axis[3] = 1.0
    k = 0.05 * torch.randn(H, T + n, d, generator=g)
    k[:, 0] = axis * (bits * math.log(2) * math.sqrt(d) / 8)
    v = 1 + 0.1 * torch.randn(H, T + n, d, generator=g)
    v[:, 0] = 0.0
    q = (8 * axis).expand(n, cfg.num_q_heads, d)
    k, v, q = k.to(cfg.kv_dtype), v.to(cfg.kv_dtype), q.to(cfg.kv_dtype).contiguous()
    store, host = pkv.Store(cfg), HostCache()
    store.load_prefill(0, k[None, :, :T].contiguous().cuda(), v[None, :, :T].contiguous().cuda())
    host.set_prefill(0, k[None, :, :T], v[None, :, :T])
    kn, vn = (x[:, T:].transpose(0, 1).contiguous() for x in (k, v))
    out = store.chunk_attention(0, q.cuda(), kn.cuda(), vn.cuda(), [0], [n])
    rows = cache_rows(store, cfg, host, 0, 0, T)
    assert excess_of_tokens(cfg, rows, kn, vn, q, T, range(0, n, 100), out, 2.0 ** -32) <= 1.0
    few = store.chunk_attention(0, q[:5].cuda(), kn[:5].cuda(), vn[:5].cuda(), [0], [5])
    assert excess_of_tokens(cfg, rows, kn, vn, q, T, range(5), few, 2.0 ** -32) <= 1.0


@pytest.mark.parametrize("kind", ["bf16", "int4", "prerope", "d64-p16"])
@pytest.mark.parametrize("power", [-66, -60, -120, 120])
def test_products_outside_fp32(pkv, kind, power):
    """Queries and keys of 2^power: products at fp32's lower end or under it and, at 2^120, zeros beside factors whose
    product overflows.  All scores are zero, or as good as: every answer is the mean of the seen values."""
    cfg = make_cfg(pkv, num_layers=1, max_batch=2, **{**KINDS[kind], "recent_tokens": 128})  # nothing is factorized
    T, n, H, d = 100, 150, cfg.num_kv_heads, cfg.head_dim
    g = torch.Generator().manual_seed(power + 200)
    size = 2.0 ** power
    k, v = (torch.randn(H, T + n, d, generator=g) for _ in range(2))
    q = torch.randn(n, cfg.num_q_heads, d, generator=g)
    if power > 0:  # orthogonal supports (pairs that RoPE turns stay inside one of them)
        odd = (torch.arange(d) % (d // 2)) % 2 == 1
        k, q = torch.where(odd, k.sign(), 0.0), torch.where(odd, 0.0, q.sign())
    k, q, v = (k * size).to(cfg.kv_dtype), (q * size).to(cfg.kv_dtype), v.to(cfg.kv_dtype)
    store = pkv.Store(cfg)
    store.append_chunk(0, *(x[:, :T].transpose(0, 1).contiguous().cuda() for x in (k, v)), [0], [T])
    kn, vn = (x[:, T:].transpose(0, 1).contiguous() for x in (k, v))
    V = v.double().numpy()
    G = cfg.num_q_heads // H
    for m in (n, 5):
        out = store.chunk_attention(0, q[:m].cuda(), kn[:m].cuda(), vn[:m].cuda(), [0], [m]).double().cpu().numpy()
        assert np.isfinite(out).all()
        for j in range(m):
            for h in range(H):
                seen = V[h, :T + j + 1]
                # weights and values are off by 2^-11 each and by 2^-36 of the largest value;
                # scores are below 2^-80
                inner = 2.05 * 2.0 ** -11 * np.abs(seen).mean(0) + 2.0 ** -30 * np.abs(V).max()
                bound = inner + 2.0 ** -8 * (np.abs(seen.mean(0)) + inner)
                assert (np.abs(out[j, h * G:(h + 1) * G] - seen.mean(0)) <= bound).all()
    assert store.check_device_status() == 0
