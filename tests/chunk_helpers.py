"""64-bit answers for the chunk calls: the rows a store holds as attention
sees them (factors copied back and multiplied in fp64, dense rows as fed), and
the error bounds the chunk calls are held to."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle
from gpu_helpers import HostCache
from store_layout import Layout, factor_pool_slice, read_factors

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative: outputs and rows
U_IN = {torch.bfloat16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # of rebuilt operands and weights (fp16 for bf16 stores)
U32 = 2.0 ** -24


def random_rows(cfg, n, seed, layers=None):
    """(k, v) of n tokens, [L, H, n, d] (or [n, H, d] without `layers`): outlier channels, modest scores."""
    g = torch.Generator().manual_seed(seed)
    shape = (cfg.num_kv_heads, n, cfg.head_dim) if layers is None else (layers, cfg.num_kv_heads, n, cfg.head_dim)
    out = []
    for _ in range(2):
        x = 0.6 * torch.randn(shape, generator=g)
        x[..., ::37] *= 4.0
        x = x.to(cfg.kv_dtype)
        out.append(x.transpose(0, 1).contiguous() if layers is None else x)
    return out


def cache_rows(store, cfg, host: HostCache, seq, layer, T):
    """(K, V, Ka, Va) per head, [H, T, d] fp64: the rows, and the same with |L| |R| in place of L R
    (what the rounding of the products is relative to).  Keys unturned."""
    lay, P, H, d = Layout(cfg), cfg.page_size, cfg.num_kv_heads, cfg.head_dim
    kinds = oracle.page_kinds(T, P, cfg.sink_tokens, cfg.recent_tokens)
    K, V = np.zeros((H, T, d)), np.zeros((H, T, d))
    Ka, Va = np.zeros((H, T, d)), np.zeros((H, T, d))
    for h in range(H):
        if T == 0:
            continue
        Kd, Vd = host.rows(seq, layer, h)
        K[h], V[h] = Kd[:T], Vd[:T]
        Ka[h], Va[h] = np.abs(K[h]), np.abs(V[h])
        pages = np.nonzero(kinds == oracle.FACTORED)[0]
        if len(pages) == 0:
            continue
        pool = factor_pool_slice(store, lay, layer, seq, h)
        for p in pages:
            LK, RK, LV, RV = read_factors(pool, lay, layer, seq, h, int(p))
            s = slice(p * P, (p + 1) * P)
            K[h, s], V[h, s] = LK @ RK, LV @ RV
            Ka[h, s], Va[h, s] = np.abs(LK) @ np.abs(RK), np.abs(LV) @ np.abs(RV)
    return K, V, Ka, Va


def turned(X, first, theta):
    return np.stack([oracle.rope(x, np.arange(first, first + x.shape[0]), theta) for x in X]) if theta > 0 else X


def pair_abs(Xa, theta):
    """Bound on |turned row| from |row|: a turned element is at most the sum of its pair."""
    if theta <= 0:
        return Xa
    h = Xa.shape[-1] // 2
    s = Xa[..., :h] + Xa[..., h:]
    return np.concatenate([s, s], -1)


def chunk_reference(cfg, rows, k, v, q, T, u_in=None):
    """64-bit attention of one sequence's chunk and its error bound.

    rows: cache_rows at length T; k, v [n, H, d], q [n, Hq, d] torch tensors.
    The bound: with ui the half step of the operands (fp16 in bf16 stores, which
    the few-token path's split operands keep as well) and u that of the output, a
    key is off by ui |k| (one rounding of the rebuilt row), the query by ui |q|,
    plus (rank + 20) U32 |L||R| (fp32 products and angles), so a score is off by
    at most ds = (2 ui + (d + rank + 20) U32) A, A = max over seen keys of sum
    |q||k| / sqrt(d); a weight, normalised, by the factor e^(2 ds); the weight's
    own rounding and the value's (ui each, and its fp32 products) enter linearly,
    sums of T weights as T U32, and the output is rounded once (u |o|).  U32
    terms also cover exp2 (2^-22).  Below fp16's normal range a weight or a value
    is off by 2^-25 absolute."""
    K, V, Ka, Va = rows
    H, G, d, n = cfg.num_kv_heads, cfg.num_q_heads // cfg.num_kv_heads, cfg.head_dim, q.shape[0]
    theta = float(cfg.rope_theta)
    kn = k.double().cpu().numpy().transpose(1, 0, 2)
    vn = v.double().cpu().numpy().transpose(1, 0, 2)
    K = np.concatenate([K, kn], 1)
    V = np.concatenate([V, vn], 1)
    Ka = pair_abs(np.concatenate([Ka, np.abs(kn)], 1), theta)
    Va = np.concatenate([Va, np.abs(vn)], 1)
    K = turned(K, 0, theta)
    qn = q.double().cpu().numpy()
    u = U[cfg.kv_dtype]
    ui = U_IN[cfg.kv_dtype] if u_in is None else u_in
    tiny = 2.0 ** -25 if cfg.kv_dtype == torch.bfloat16 else 0.0
    rank = max(cfg.rank_k, cfg.rank_v)
    out, bound = np.zeros((n, H * G, d)), np.zeros((n, H * G, d))
    for j in range(n):
        see = T + j + 1
        for h in range(H):
            qr = qn[j, h * G:(h + 1) * G]
            s = qr @ K[h, :see].T / math.sqrt(d)
            A = (np.abs(qr) @ Ka[h, :see].T / math.sqrt(d)).max(1, keepdims=True)
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            o = w @ V[h, :see]
            B = w @ Va[h, :see]
            ds = (2 * ui + (d + rank + 20) * U32) * A
            out[j, h * G:(h + 1) * G] = o
            inner = ((np.expm1(2 * ds) + 2.05 * ui + (see + rank + 40) * U32) * B +
                     tiny * (1 + see * np.abs(V[h, :see]).max(0, keepdims=True)))
            bound[j, h * G:(h + 1) * G] = inner + u * (np.abs(o) + inner)
    return out, bound


def excess(got, ref, bound):
    """Largest error over its bound."""
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all()
    return float((np.abs(got - ref) / np.maximum(bound, 1e-300)).max()) if got.size else 0.0
