"""Numbers that do not fit in 32 bits are refused; their low 32 bits may well be a valid argument."""
import ctypes
import dataclasses

import pytest
import torch

WIDE = [2 ** 31, 2 ** 32, 2 ** 32 + 3, -2 ** 31 - 1, -2 ** 32, 10 ** 30]


@pytest.fixture(scope="module")
def pkv():
    from page_wise_rank_gb300 import build
    build.build()
    import page_wise_rank_gb300 as m
    return m


def make_cfg(pkv, **kw):
    base = dict(num_layers=2, num_kv_heads=1, num_q_heads=1, head_dim=64, page_size=32, rank_k=8, rank_v=8,
                sink_tokens=4, recent_tokens=40, max_batch=2, max_tokens_per_seq=300, kv_dtype=torch.float32)
    return pkv.StoreConfig(**{**base, **kw})


@pytest.mark.parametrize("wide", WIDE)
def test_lists(pkv, wide):
    for call in (lambda: pkv._ints([1, wide], 2, "lengths"), lambda: pkv._seq_ids([0, wide])):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    assert list(pkv._ints([2 ** 31 - 1, -2 ** 31], 2, "counts")) == [2 ** 31 - 1, -2 ** 31]


@pytest.mark.parametrize("wide", WIDE)
def test_numbers(pkv, wide):
    edge = 2 ** 31 - 1 if wide > 0 else -2 ** 31
    assert pkv._lib.Int32.from_param(wide).value == edge
    assert pkv._lib.Int32.from_param(ctypes.c_int32(5)).value == 5
    n = ctypes.c_int64()
    assert pkv.lib().puzzlekv_int4_record_bytes(32, 64, 8 + wide if wide > 0 else wide, 8, ctypes.byref(n)) != 0


@pytest.mark.parametrize("field", ["num_layers", "num_kv_heads", "max_batch", "max_tokens_per_seq", "rank_k", "sink_tokens"])
def test_configuration(pkv, field):
    with pytest.raises(pkv.PuzzleKVError):
        pkv.query_sizes(dataclasses.replace(make_cfg(pkv), **{field: 2 ** 32 + getattr(make_cfg(pkv), field)}))


@pytest.mark.gpu
@pytest.mark.parametrize("wide", WIDE)
def test_calls_change_nothing(pkv, wide):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    cfg = make_cfg(pkv)
    store = pkv.Store(cfg)
    k, v = (torch.randn(100, 1, 64, device="cuda") for _ in range(2))
    for layer in range(2):
        store.append_chunk(layer, k, v, [0], [100])
    before = [store.stats(b, l) for b in range(2) for l in range(2)]
    f = [torch.zeros(1, 1, *s, device="cuda") for s in ((32, 8), (8, 64), (32, 8), (8, 64))]
    calls = [lambda: store.truncate_sequences([0], [wide]), lambda: store.truncate_sequences([wide], [10]),
             lambda: store.copy_sequences([wide], [1]), lambda: store.copy_sequences([0], [1 + wide]),
             lambda: store.read_tokens(0, [0], [wide], [1]), lambda: store.read_tokens(wide, [0], [0], [1]),
             lambda: store.chunk_attention(wide, k[:1], k[:1], v[:1], [0], [1]),
             lambda: store.append_chunk(wide, k[:1], v[:1], [1], [1]),
             lambda: store.append_chunk(0, k[:1], v[:1], [1], [1 + wide]),
             lambda: store.load_factors(0, 0, wide + 1, *f), lambda: store.load_factors(0, wide, 1, *f),
             lambda: store.load_factors(wide, 0, 1, *f), lambda: store.load_prefill(wide, k[None, None, :, 0].repeat(2, 1, 1, 1),
                                                                                  v[None, None, :, 0].repeat(2, 1, 1, 1)),
             lambda: store.factorize_pages([(0, wide + 1)]), lambda: store.append_token(0, k[:1], v[:1], [wide])]
    for call in calls:
        with pytest.raises((pkv.PuzzleKVError, ValueError)):
            call()
    assert before == [store.stats(b, l) for b in range(2) for l in range(2)]
