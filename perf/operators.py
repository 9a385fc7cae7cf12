"""Workloads of the store's chunk operators, their plain forms and their 64-bit answers.

Four operators of a paged low-rank cache ("PuzzleKV: Page-Wise Low-Rank Decomposition for KV Cache
Compression", section 3.3):

  attend  attention of a chunk of new tokens per sequence over the mixed dense / factorized cache and,
          causally, over the chunk itself: a continued prompt, or drafted tokens being verified
  read    rows of the cache as attention sees them: factorized pages as L R, dense pages as stored
  append  a ragged chunk appended to every sequence, read back, and taken off again
  copy    sequences of a store copied over others (forked, or reordered beams), pages and page table

Each case names its store (KV heads H, query heads Hq, head dimension d, page size P, ranks rk and rv, dense
sink and recent window W) and the sequences' lengths.  With ``own`` false, ``run`` computes a case with
elementary torch operations in 32 bits; with ``own`` true it makes the package's calls.
"""
import math

import torch

own = False

LLAMA = dict(H=8, Hq=32, d=128, P=64, rk=16, rv=24, sink=4, W=128, dtype="bf16", theta=0.0)
QWEN = dict(LLAMA, Hq=64, rk=24)
PAGES32 = dict(LLAMA, P=32, rv=14, W=64)
TINY = dict(H=2, Hq=8, d=64, P=32, rk=8, rv=8, sink=4, W=64, dtype="f32", theta=0.0)


_LISTS = ("T", "n", "start", "src", "dst")


def _text(case):
    """Lists of a case as texts, so that a case holds plain values."""
    return {k: " ".join(map(str, v)) if k in _LISTS else v for k, v in case.items()}


def _lists(case):
    return {k: [int(x) for x in v.split()] if k in _LISTS else v for k, v in case.items()}


def listed():
    return [_text(c) for c in _listed()]


def _listed():
    return [
        # drafted tokens of one request verified against a 32K context: the smallest call, where latency counts
        dict(LLAMA, name="attend-verify", op="attend", T=[32741], n=[6]),
        # a serving batch between prompts: 16 requests of 8K to 32K tokens, one to eight drafted tokens each
        dict(LLAMA, name="attend-verify-batch", op="attend",
             T=[8192, 31011, 12345, 20480, 9001, 27777, 16383, 24576, 32768, 14002, 10101, 18888, 22222, 29999, 11264, 25601],
             n=[5, 1, 8, 3, 4, 2, 7, 8, 1, 6, 5, 3, 8, 2, 4, 1]),
        # one chunk of a chunked prefill in a 32K context
        dict(LLAMA, name="attend-chunk", op="attend", T=[30720], n=[2048]),
        # a mixed batch with small pages: a first chunk into an empty slot, a continued prompt and single tokens
        dict(PAGES32, name="attend-mixed", op="attend", T=[0, 5003, 12001, 777], n=[511, 300, 1, 1]),
        # the last chunk of a 128K prompt, eight query heads per KV head: the largest call
        dict(QWEN, name="attend-long", op="attend", T=[130048], n=[1024]),
        # the small fp32 store, an odd chunk
        dict(TINY, name="attend-f32", op="attend", T=[1024], n=[37]),
        # a request's whole layer handed to an engine that attends densely
        dict(LLAMA, name="read-layer", op="read", T=[32768], start=[0], n=[32768]),
        # pieces of several requests, starting and ending inside pages
        dict(PAGES32, name="read-pieces", op="read", T=[4096, 1000, 9000], start=[17, 0, 8000], n=[2001, 1000, 999]),
        # eight requests of 4K tokens take their verified tokens
        dict(LLAMA, name="append-drafts", op="append", T=[4096, 4099, 4127, 4150, 4160, 4161, 4200, 4210],
             n=[4, 1, 8, 2, 5, 8, 3, 7]),
        # short prompts admitted into empty slots
        dict(LLAMA, name="append-prompts", op="append", T=[0] * 16,
             n=[96, 17, 128, 64, 33, 101, 5, 77, 128, 59, 1, 110, 88, 42, 127, 65]),
        # one prompt forked into three more samples
        dict(LLAMA, name="copy-fork", op="copy", L=32, T=[1000, 0, 0, 0], src=[0, 0, 0], dst=[1, 2, 3]),
        # eight beams after a step: three of them are replaced by copies of better ones
        dict(LLAMA, name="copy-beams", op="copy", L=8, T=[4096] * 8, src=[0, 2, 2, 5], dst=[1, 3, 4, 7]),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    return _text(_draw(rng))


def _draw(rng):
    store = rng.choice([LLAMA, QWEN, PAGES32, TINY,
                        dict(TINY, dtype="bf16", Hq=6),
                        dict(LLAMA, H=4, Hq=4, d=64, P=16, rk=5, rv=7, sink=20, W=40),
                        dict(LLAMA, theta=5e5)])
    op = rng.choice(["attend", "attend", "attend", "read", "append", "copy"])
    B = _log(rng, 1, 8)
    if op == "attend":
        big, most = (4096, 256) if store["dtype"] == "f32" else (40000, 1024)
        T = [0 if rng.random() < 0.1 else _log(rng, 1, big) for _ in range(B)]
        n = [_log(rng, 1, most if rng.random() < 0.5 else 12) for _ in range(B)]
        while sum(m * (t + m) for t, m in zip(T, n)) * store["Hq"] * store["d"] > 1e12:
            T, n = T[1:], n[1:]
        return dict(store, op=op, T=T, n=n)
    if op == "read":
        T = [_log(rng, 1, 24000) for _ in range(B)]
        start = [rng.randrange(t) for t in T]
        return dict(store, op=op, T=T, start=start, n=[rng.randint(1, t - s) for t, s in zip(T, start)])
    if op == "append":
        # pages of the window only: no page is factorized inside the call
        T = [0 if rng.random() < 0.2 else _log(rng, 1, 8000) for _ in range(B)]
        n = [_log(rng, 1, store["W"] if t == 0 else store["P"]) for t in T]
        if any(_kinds(t, store).count(0) != _kinds(t + m, store).count(0) for t, m in zip(T, n)):
            T, n = [0] * B, [_log(rng, 1, store["W"]) for _ in range(B)]
        return dict(store, op=op, T=T, n=n)
    B = rng.randint(2, 8)
    keep = rng.sample(range(B), rng.randint(1, B - 1))
    dst = [b for b in range(B) if b not in keep]
    t = _log(rng, 1, 4096)
    T = [t if rng.random() < 0.5 else _log(rng, 1, 4096) for _ in range(B)]
    return dict(store, op="copy", L=rng.choice([1, 3, 8]), T=T, src=[rng.choice(keep) for _ in dst], dst=dst)


def _sink_pages(c):
    return -(-c["sink"] // c["P"])


def _kinds(T, c):
    """1 = dense, 0 = factorized, per page of a T-token sequence (sink pages, the window and an incomplete page are dense)."""
    P = c["P"]
    return [int(p < _sink_pages(c) or (p + 1) * P > T or (p + 1) * P > T - c["W"]) for p in range(-(-T // P))]


def _split(T, c):
    """First factorized page and the page after the last one."""
    kinds = _kinds(T, c)
    return (kinds.index(0), len(kinds) - kinds[::-1].index(0)) if 0 in kinds else (min(_sink_pages(c), len(kinds)),) * 2


def _dt(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _bytes(c):
    return 2 if c["dtype"] == "bf16" else 4


# ---------------------------------------------------------------- inputs


def _rows(g, c, H, n, scale):
    x = torch.randn(H, n, c["d"], generator=g, device="cuda") * 0.5
    return (x * scale[:, None, :]).to(_dt(c))


def _factors(g, c, H, n, r, scale):
    """Orthonormal left factors and right factors with decaying singular values, head dimensions scaled as ``scale``."""
    P, d = c["P"], c["d"]
    basis = torch.linalg.qr(torch.randn(64, P, P, generator=g, device="cuda"))[0]
    pick = torch.randint(64, (H, n), generator=g, device="cuda")
    L = basis[pick][..., :r].to(_dt(c)).contiguous()
    decay = torch.linspace(1.0, 0.2, r, device="cuda") * math.sqrt(P) * 0.35
    R = torch.randn(H, n, r, d, generator=g, device="cuda") * decay[:, None] * scale[:, None, None, :]
    return L, R.to(_dt(c)).contiguous()


def _sequences(g, c):
    """Per sequence: its factorized pages' factors and its dense rows, sink first, then window."""
    H, P = c["H"], c["P"]
    out = []
    for T in c["T"]:
        fs, fw = _split(T, c)
        s = dict(T=T, fs=fs, fw=fw)
        for kind, r in (("k", c["rk"]), ("v", c["rv"])):
            scale = torch.ones(H, c["d"], device="cuda")
            scale[:, torch.randperm(c["d"], generator=g, device="cuda")[:4]] = 4.0  # outlier channels
            if T:
                s["L" + kind], s["R" + kind] = _factors(g, c, H, fw - fs, r, scale)
            s["sink_" + kind] = _rows(g, c, H, min(T, fs * P), scale)
            s["tail_" + kind] = _rows(g, c, H, max(0, T - fw * P) if fw > 0 else 0, scale)
            s["scale_" + kind] = scale
        out.append(s)
    return out


def _own_store(c, seqs, layers=1, capacity=None):
    import page_wise_rank_gb300 as pkv
    cfg = pkv.StoreConfig(num_layers=layers, num_kv_heads=c["H"], num_q_heads=c["Hq"], head_dim=c["d"], page_size=c["P"],
                          rank_k=c["rk"], rank_v=c["rv"], sink_tokens=c["sink"], recent_tokens=c["W"],
                          max_batch=len(c["T"]), max_tokens_per_seq=capacity, kv_dtype=_dt(c), rope_theta=c["theta"])
    store = pkv.Store(cfg)
    for b, s in enumerate(seqs):
        if not s["T"]:
            continue
        kv = []
        for kind in "kv":
            x = torch.zeros(layers, c["H"], s["T"], c["d"], dtype=_dt(c), device="cuda")
            x[:, :, :s["sink_" + kind].shape[1]] = s["sink_" + kind]
            if s["tail_" + kind].shape[1]:
                x[:, :, -s["tail_" + kind].shape[1]:] = s["tail_" + kind]
            kv.append(x)
        store.load_prefill(b, *kv)
        if s["fw"] > s["fs"]:
            store.load_factors(0, b, s["fs"], s["Lk"], s["Rk"], s["Lv"], s["Rv"])
    return store


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = _lists(case)
    state = dict(case=c)
    if c["op"] == "copy":
        return _prepare_copy(c, g, state)
    H, Hq, d, N = c["H"], c["Hq"], c["d"], sum(c["n"])
    seqs = _sequences(g, c)
    state["ids"], state["n"] = list(range(len(c["T"]))), list(c["n"])
    if c["op"] in ("attend", "append"):
        for kind in "kv":
            x = torch.randn(N, H, d, generator=g, device="cuda") * 0.5
            scale = torch.cat([s["scale_" + kind].expand(n, H, d) for s, n in zip(seqs, c["n"])])
            state[kind] = (x * scale).to(_dt(c))
        # scores of about unit spread
        state["q"] = (torch.randn(N, Hq, d, generator=g, device="cuda") * 1.5).to(_dt(c))
    if own:
        grow = c["n"] if c["op"] in ("attend", "append") else [0] * len(c["T"])
        state["store"] = _own_store(c, seqs, capacity=max(t + m for t, m in zip(c["T"], grow)))
    elif c["op"] == "append":
        cap = max(t + m for t, m in zip(c["T"], c["n"]))
        state["cache"] = {kind: torch.zeros(len(seqs), H, cap, d, dtype=_dt(c), device="cuda") for kind in "kv"}
        state["len"] = torch.tensor(c["T"], device="cuda")
    else:
        state["seqs"] = seqs
    return state


def _prepare_copy(c, g, state):
    """The pools hold arbitrary bytes: copying does not look inside a page."""
    L, B, H, P, d, e = c["L"], len(c["T"]), c["H"], c["P"], c["d"], _bytes(c)
    pages = -(-max(c["T"]) // P)
    rec = (-(-c["rk"] // 8) * 8 + -(-c["rv"] // 8) * 8) * (P + d) * e
    slots = _sink_pages(c) + -(-c["W"] // P) + 2
    shapes = dict(factors=(L, B, H, pages, rec), dense=(L, B, slots, H, 2, P * d * e))
    if own:
        store = state["store"] = _own_store(c, [dict(s, fw=s["fs"]) for s in _empty_rows(c)], L, max(c["T"]))
        pools = dict(factors=store.factor_pool, dense=store.dense_pool)
        table = store.page_table.view(torch.int32)
        at = (B * L * 4 + 255) // 256 * 64
        state["len"], state["desc"] = table[:B * L].view(B, L), table[at:at + B * L * pages].view(B, L, pages)
    else:
        pools = {k: torch.empty(math.prod(s), dtype=torch.uint8, device="cuda") for k, s in shapes.items()}
        state["len"] = torch.zeros(B, L, dtype=torch.int32, device="cuda")
        state["desc"] = torch.zeros(B, L, pages, dtype=torch.int32, device="cuda")
        for b, T in enumerate(c["T"]):
            state["len"][b] = T
            for p, dense in enumerate(_kinds(T, c)):
                state["desc"][b, :, p] = (1 << 30 | _slot(p, c, slots)) if dense else p
    for k, s in shapes.items():
        pools[k].view(torch.int64).random_(generator=g)
        state[k] = pools[k].view(s)
    state["src"], state["dst"], state["slots"] = list(c["src"]), list(c["dst"]), slots
    return state


def _empty_rows(c):
    H, d = c["H"], c["d"]
    none = torch.zeros(H, 0, d, dtype=_dt(c), device="cuda")
    return [dict(T=T, fs=0, fw=0, sink_k=none, sink_v=none, tail_k=none, tail_v=none) for T in c["T"]]


def _slot(p, c, slots):
    s = _sink_pages(c)
    return p if p < s else s + p % (slots - s)


def _live(T, c, slots):
    """Factorized page range and the dense slots in use of a T-token sequence."""
    fs, fw = _split(T, c)
    return fs, fw, sorted(_slot(p, c, slots) for p, dense in enumerate(_kinds(T, c)) if dense)


# ---------------------------------------------------------------- one pass


def run(state):
    c = state["case"]
    if c["op"] == "attend":
        if own:
            return state["store"].chunk_attention(0, state["q"], state["k"], state["v"], state["ids"], state["n"])
        return _plain_attend(state, c)
    if c["op"] == "read":
        if own:
            return state["store"].read_tokens(0, state["ids"], c["start"], state["n"])
        return _plain_read(state, c)
    if c["op"] == "append":
        return _own_append(state, c) if own else _plain_append(state, c)
    if own:
        state["store"].copy_sequences(state["src"], state["dst"])
    else:
        _plain_copy(state, c)
    return _copied(state, c)


def _turn(x, first, theta):
    """Rotate-half position embedding of rows first, first + 1, ... (angles in 64 bits)."""
    d = x.shape[-1]
    inv = theta ** (-torch.arange(d // 2, dtype=torch.float64, device=x.device) * 2.0 / d)
    a = torch.arange(first, first + x.shape[-2], dtype=torch.float64, device=x.device)[:, None] * inv
    cos, sin = a.cos().to(x.dtype), a.sin().to(x.dtype)
    x1, x2 = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1)


def _rebuilt(s, kind, h, lo, hi):
    """Rows [lo, hi) of one head's cache in 32 bits, factorized pages as L R."""
    P, fs, fw = s["P"], s["fs"], s["fw"]
    a, b = max(lo // P, fs), min(-(-hi // P), fw)
    parts = [s["sink_" + kind][h].float()[lo:hi]]
    if b > a:
        x = (s["L" + kind][h, a - fs:b - fs].float() @ s["R" + kind][h, a - fs:b - fs].float()).reshape((b - a) * P, -1)
        parts.append(x[max(0, lo - a * P):hi - a * P])
    t = max(fs, fw) * P
    parts.append(s["tail_" + kind][h].float()[max(0, lo - t):max(0, hi - t)])
    return torch.cat(parts)


def _plain_attend(state, c):
    H, Hq, d = c["H"], c["Hq"], c["d"]
    G, at = Hq // H, 0
    out = torch.empty(sum(c["n"]), Hq, d, dtype=_dt(c), device="cuda")
    for s, n in zip(state["seqs"], c["n"]):
        s, T = dict(s, P=c["P"]), s["T"]
        for h in range(H):
            K = torch.cat([_rebuilt(s, "k", h, 0, T), state["k"][at:at + n, h].float()])
            V = torch.cat([_rebuilt(s, "v", h, 0, T), state["v"][at:at + n, h].float()])
            if c["theta"]:
                K = _turn(K, 0, c["theta"])
            step = max(1, (1 << 28) // (G * (T + n)))
            for i in range(0, n, step):
                j = min(n, i + step)
                q = state["q"][at + i:at + j, h * G:(h + 1) * G].float().reshape(-1, d)
                w = (q @ K.T / math.sqrt(d)).view(j - i, G, T + n)
                seen = torch.arange(T + n, device="cuda")[None] <= T + torch.arange(i, j, device="cuda")[:, None]
                w = w.masked_fill(~seen[:, None], -math.inf)
                w = torch.exp(w - w.amax(-1, keepdim=True))
                o = (w / w.sum(-1, keepdim=True)).view(-1, T + n) @ V
                out[at + i:at + j, h * G:(h + 1) * G] = o.view(j - i, G, d).to(_dt(c))
        at += n
    return out


def _plain_read(state, c):
    both = []
    for kind in "kv":
        parts = []
        for s, lo, n in zip(state["seqs"], c["start"], c["n"]):
            s = dict(s, P=c["P"])
            x = torch.stack([_rebuilt(s, kind, h, lo, lo + n) for h in range(c["H"])])
            if kind == "k" and c["theta"]:
                x = _turn(x, lo, c["theta"])
            parts.append(x.transpose(0, 1).to(_dt(c)))
        both.append(torch.cat(parts).contiguous())
    return tuple(both)


def _plain_append(state, c):
    at, got = 0, {"k": [], "v": []}
    for b, (T, n) in enumerate(zip(c["T"], c["n"])):
        for kind in "kv":
            state["cache"][kind][b, :, T:T + n] = state[kind][at:at + n].transpose(0, 1)
        state["len"][b] += n
        at += n
    for b, (T, n) in enumerate(zip(c["T"], c["n"])):
        for kind in "kv":
            x = state["cache"][kind][b, :, T:T + n].transpose(0, 1)
            got[kind].append(_turn(x.transpose(0, 1).float(), T, c["theta"]).transpose(0, 1).to(_dt(c))
                             if kind == "k" and c["theta"] else x)
        state["len"][b] -= n
    return torch.cat(got["k"]), torch.cat(got["v"])


def _own_append(state, c):
    store, ids = state["store"], state["ids"]
    store.append_chunk(0, state["k"], state["v"], ids, state["n"])
    got = store.read_tokens(0, ids, c["T"], state["n"])
    store.truncate_sequences(ids, c["T"])
    return got


def _plain_copy(state, c):
    for a, b in zip(state["src"], state["dst"]):
        fs, fw, slots = _live(c["T"][a], c, state["slots"])
        if fw > fs:
            state["factors"][:, b, :, fs:fw] = state["factors"][:, a, :, fs:fw]
        for s in slots:
            state["dense"][:, b, s] = state["dense"][:, a, s]
        state["len"][b] = state["len"][a]
        state["desc"][b] = state["desc"][a]


def _copied(state, c):
    out = []
    for a, b in zip(state["src"], state["dst"]):
        fs, fw, slots = _live(c["T"][a], c, state["slots"])
        pages = -(-c["T"][a] // c["P"])
        out.append(dict(factors=state["factors"][:, b, :, fs:fw], dense=[state["dense"][:, b, s] for s in slots],
                        length=state["len"][b], pages=state["desc"][b, :, :pages]))
    return out


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c, e = _lists(case), _bytes(case)
    H, Hq, d, P, rk, rv = c["H"], c["Hq"], c["d"], c["P"], c["rk"], c["rv"]
    record, row = H * (rk + rv) * (P + d) * e, H * 2 * d * e
    b = f = 0
    if c["op"] == "copy":
        slots = _sink_pages(c) + -(-c["W"] // P) + 2
        def size(T):
            fs, fw, live = _live(T, c, slots)
            rec = (-(-rk // 8) * 8 + -(-rv // 8) * 8) * (P + d) * e
            return c["L"] * (H * (fw - fs) * rec + len(live) * H * 2 * P * d * e)
        b = sum(size(c["T"][a]) for a in set(c["src"])) + sum(size(c["T"][a]) for a in c["src"])
        return dict(bytes=b, flops=0)
    if c["op"] == "append":
        return dict(bytes=4 * row * sum(c["n"]), flops=0)  # in, into the cache, out of it, back
    for i, (T, n) in enumerate(zip(c["T"], c["n"])):
        fs, fw = _split(T, c)
        if c["op"] == "attend":
            pages, dense = fw - fs, T - (fw - fs) * P
            b += pages * record + dense * row + n * row + 2 * n * Hq * d * e
            f += n * Hq * (2 * pages * (d + P) * (rk + rv) + 4 * d * dense) + 2 * d * Hq * n * (n + 1)
        else:
            lo, hi = c["start"][i], c["start"][i] + n
            a, z = max(lo // P, fs), max(max(lo // P, fs), min(-(-hi // P), fw))
            rebuilt = max(0, min(hi, fw * P) - max(lo, fs * P))
            b += (z - a) * record + (n - rebuilt) * row + n * row
            f += rebuilt * H * 2 * d * (rk + rv)
    return dict(bytes=b, flops=f)


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    """attend by eq. (4) page by page: (q R_K^T) L_K^T and (p L_V) R_V, no page rebuilt, one softmax over all; read by
    the product; append gives its rows back; copies have no computed values."""
    global own
    c = _lists(case)
    if c["op"] == "copy":
        return None
    if c["op"] == "attend" and sum(n * (T + n) for n, T in zip(c["n"], c["T"])) * c["Hq"] * c["d"] * 4 > 7e12:
        return None
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    return {"attend": _exact_attend, "read": _exact_read, "append": _exact_append}[c["op"]](state, c)


def _spin(x, pos, theta):
    """Rows of x turned by their positions as complex numbers, in 64 bits."""
    h = x.shape[-1] // 2
    ang = pos.double()[:, None] * torch.exp(-math.log(theta) * torch.arange(h, device=x.device).double() / h)
    z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(torch.ones_like(ang), ang)
    return torch.cat([z.real, z.imag], -1)


def _exact_attend(state, c):
    H, Hq, d, P, theta = c["H"], c["Hq"], c["d"], c["P"], c["theta"]
    G, at = Hq // H, 0
    out = torch.empty(sum(c["n"]), Hq, d, dtype=torch.float64, device="cuda")
    for s, n in zip(state["seqs"], c["n"]):
        T, fs, fw = s["T"], s["fs"], s["fw"]
        pages = max(0, fw - fs) if T else 0
        sink = s["sink_k"].shape[1]
        # dense keys with their positions: sink, tail, chunk
        pos = torch.cat([torch.arange(sink), torch.arange(T - s["tail_k"].shape[1], T), torch.arange(T, T + n)]).cuda()
        for h in range(H):
            Kd = torch.cat([s["sink_k"][h], s["tail_k"][h], state["k"][at:at + n, h]]).double()
            Vd = torch.cat([s["sink_v"][h], s["tail_v"][h], state["v"][at:at + n, h]]).double()
            if theta:
                Kd = _spin(Kd, pos, theta)
            if pages:
                Lk, Rk, Lv, Rv = (s[x][h].double() for x in ("Lk", "Rk", "Lv", "Rv"))
            step = max(1, (1 << 26) // (G * (T + n)))
            for i in range(0, n, step):
                j = min(n, i + step)
                q = state["q"][at + i:at + j, h * G:(h + 1) * G].double().reshape(-1, d) * d ** -0.5
                own_pos = T + torch.arange(i, j, device="cuda").repeat_interleave(G)
                sd = torch.where(pos[None] <= own_pos[:, None], q @ Kd.T, -math.inf)
                m = sd.amax(1, keepdim=True)
                if pages:
                    if theta:  # turned keys are no product of the factors: rebuild them
                        Kf = _spin((Lk @ Rk).reshape(pages * P, d), torch.arange(fs * P, fw * P, device="cuda"), theta)
                        sf = (q @ Kf.T).view(-1, pages, P)
                    else:
                        sf = torch.einsum("xpr,ptr->xpt", torch.einsum("xd,prd->xpr", q, Rk), Lk)
                    m = torch.maximum(m, sf.flatten(1).amax(1, keepdim=True))
                wd = torch.exp(sd - m)
                num, den = wd @ Vd, wd.sum(1, keepdim=True)
                if pages:
                    wf = torch.exp(sf - m[..., None])
                    num = num + torch.einsum("xpr,prd->xd", torch.einsum("xpt,ptr->xpr", wf, Lv), Rv)
                    den = den + wf.flatten(1).sum(1, keepdim=True)
                out[at + i:at + j, h * G:(h + 1) * G] = (num / den).view(j - i, G, d)
        at += n
    return out


def _exact_append(state, c):
    k = state["k"].double()
    if c["theta"]:
        pos = torch.cat([torch.arange(T, T + n) for T, n in zip(c["T"], c["n"])]).cuda()
        k = _spin(k.transpose(0, 1), pos, c["theta"]).transpose(0, 1)
    return k, state["v"].double()


def _exact_read(state, c):
    P, both = c["P"], []
    for kind in "kv":
        parts = []
        for s, lo, n in zip(state["seqs"], c["start"], c["n"]):
            x = torch.zeros(c["H"], s["T"], c["d"], dtype=torch.float64, device="cuda")
            x[:, :s["sink_" + kind].shape[1]] = s["sink_" + kind]
            x[:, s["T"] - s["tail_" + kind].shape[1]:] = s["tail_" + kind]
            if s["fw"] > s["fs"]:
                pages = torch.einsum("hptr,hprd->hptd", s["L" + kind].double(), s["R" + kind].double())
                x[:, s["fs"] * P:s["fw"] * P] = pages.flatten(1, 2)
            if kind == "k" and c["theta"]:
                x = _spin(x, torch.arange(s["T"], device="cuda"), c["theta"])
            parts.append(x[:, lo:lo + n].transpose(0, 1))
        both.append(torch.cat(parts))
    return tuple(both)
