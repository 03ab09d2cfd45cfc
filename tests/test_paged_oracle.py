"""Pins of the paged cache's oracle, and the library's and the binding's refusals (no GPU)."""
import ctypes as C
import itertools

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_lsa_b200 as lsa
from lookahead_sparse_kv_lsa_b200 import _lib
from oracle import paged_oracle as po


# ---------------------------------------------------------------------- oracle pins
def _pool(rng, pages, Hkv, d):
    return rng.standard_normal((pages, 2, Hkv, 64, d))


def test_attend_is_softmax_attention():
    rng = np.random.default_rng(0)
    pool, q = _pool(rng, 4, 2, 8), rng.standard_normal((6, 8))
    out, mass, _, _ = po.attend(q, pool, [2, 0, 3], [0, 1, 2], 3, 17, 0.3)
    for h in range(6):
        K = np.concatenate([pool[2, 0, h // 3], pool[0, 0, h // 3], pool[3, 0, h // 3][:17]])
        V = np.concatenate([pool[2, 1, h // 3], pool[0, 1, h // 3], pool[3, 1, h // 3][:17]])
        ref = torch.nn.functional.scaled_dot_product_attention(
            *(torch.from_numpy(x)[None] for x in (q[h:h + 1], K, V)), scale=0.3)
        assert np.allclose(out[h], ref[0, 0].numpy(), atol=1e-12)
    assert np.isclose(mass.sum(), 6)


@pytest.mark.parametrize("prefix,doc,window", list(itertools.product((0, 1, 70, 500), (0, 65, 10 ** 6), (0, 1, 64, 130))))
def test_masks_against_a_loop(prefix, doc, window):
    pos, n, tail = [0, 1, 5, 6], 4, 9
    x_b = 64 * 6 + 8
    seen, got_x = po.seen_positions(pos, n, tail, prefix, doc, window)
    assert got_x == x_b
    want = []
    for j, p in enumerate(pos):
        for t in range(64 if j < 3 else 9):
            x = 64 * p + t
            in_window = window == 0 or x > x_b - window
            if x < prefix or (x >= doc and in_window):
                want.append((j, t, x))
    assert seen == want


def test_cap_and_bias_closed_form():
    # two tokens, q.k = a and b: weights sigma of the difference of capped, biased scores
    pool = np.zeros((1, 2, 1, 64, 1))
    pool[0, 0, 0, 0, 0], pool[0, 0, 0, 1, 0] = 3.0, -1.0
    pool[0, 1, 0, 0, 0] = 1.0
    out, mass, _, _ = po.attend(np.array([[2.0]]), pool, [0], [0], 1, 2, 0.5, cap=4.0, slopes=[0.25])
    z0, z1 = 4 * np.tanh(3 / 4) - 0.25, 4 * np.tanh(-1 / 4)
    assert np.isclose(out[0, 0], 1 / (1 + np.exp(z1 - z0)), atol=1e-14)
    assert np.isclose(mass[0], 1)


def test_evict_against_exhaustive_choice():
    rng = np.random.default_rng(1)
    for _ in range(200):
        n = int(rng.integers(1, 9))
        sink, recent = int(rng.integers(0, 3)), int(rng.integers(1, 3))
        budget = sink + recent + int(rng.integers(0, 4))
        score = rng.integers(0, 3, n).astype(float)
        kept, gone = po.evict(score, n, budget, sink, recent)
        assert sorted(kept + gone) == list(range(n))
        if n <= budget:
            assert not gone
            continue
        assert len(kept) == budget and set(range(sink)) <= set(kept) and set(range(n - recent, n)) <= set(kept)
        mid = range(sink, n - recent)
        # best by total score, then the lexicographically first set among those equal in score multiset
        sets = [s for s in itertools.combinations(mid, budget - sink - recent)]
        top = max(sets, key=lambda s: (sorted((score[j] for j in s), reverse=True), [-j for j in s]))
        assert [j for j in kept if j in mid] == list(top)


def test_append_against_token_loop():
    n, tail, free, dest, opened = po.append(2, 63, [9, 8, 7], 66, [4, 5], [0, 3], 8)
    assert (n, tail, free) == (4, 1, [9]) and opened == {2: (7, 4), 3: (8, 5)}
    assert dest[0] == (5, 63) and dest[1] == (7, 0) and dest[64] == (7, 63) and dest[65] == (8, 0)
    assert po.append(0, 0, [], 1, [], [], 8) is None
    assert po.append(8, 64, [1], 1, list(range(8)), list(range(8)), 8) is None


# ---------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from lookahead_sparse_kv_lsa_b200 import build
    build.build()
    return _lib.lib()


def _cache(**kw):
    s = _lib.LsaPagedCacheC()
    s.B, s.H, s.Hkv, s.d, s.dtype, s.bt_stride, s.free_stride, s.window = 2, 8, 2, 128, 0, 10, 4, 0
    s.scale, s.cap, s.decay = 0.1, 0.0, 1.0
    s.pool, s.n_pages, s.ws, s.ws_bytes, s.err = 256, 100, 256, 1 << 40, 256
    for f in ("block_table", "block_pos", "score", "n_entries", "tail_len", "free_list", "free_cnt"):
        setattr(s.t, f, 256)
    for k, v in kw.items():
        setattr(s.t if hasattr(s.t, k) else s, k, v)
    return s


BAD = [dict(B=0), dict(B=65537), dict(H=0), dict(H=7), dict(Hkv=0), dict(H=130), dict(H=2048, Hkv=64),
       dict(d=64), dict(d=96), dict(d=640), dict(dtype=2), dict(dtype=-1), dict(bt_stride=0),
       dict(free_stride=-1), dict(B=65536, bt_stride=1 << 14), dict(bt_stride=(1 << 25) + 1), dict(window=-1), dict(scale=0.0), dict(scale=float("nan")),
       dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")),
       dict(decay=-0.1), dict(decay=1.5), dict(decay=float("nan")), dict(pool=None), dict(pool=8),
       dict(n_pages=0), dict(n_pages=(1 << 22) + 1), dict(block_table=None), dict(n_entries=None),
       dict(tail_len=None), dict(free_list=None), dict(free_cnt=None), dict(err=None)]


def test_struct_sizes(lib):
    assert lib.lsa_paged_cache_size() == C.sizeof(_lib.LsaPagedCacheC)


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_cache_refusals(lib, bad):
    assert lib.lsa_paged_check(C.byref(_cache())) == _lib.LSA_OK
    s = _cache(**bad)
    inv = _lib.LSA_ERR_INVALID_ARG
    assert lib.lsa_paged_check(C.byref(s)) == inv
    assert lib.lsa_paged_attn(C.byref(s), 256, 256, None) == inv
    assert lib.lsa_paged_append(C.byref(s), 256, 256, 2, None, None, None) == inv
    assert lib.lsa_paged_evict(C.byref(s), 5, 1, 1, None, None) == inv


def test_call_refusals(lib):
    s, inv = _cache(), _lib.LSA_ERR_INVALID_ARG
    r = C.byref(s)
    assert lib.lsa_paged_check(None) == inv
    for q, out in ((None, 256), (256, None), (264, 256), (256, 264)):
        assert lib.lsa_paged_attn(r, q, out, None) == inv
    for ws in (None, 8):
        assert lib.lsa_paged_attn(C.byref(_cache(ws=ws)), 256, 256, None) == inv
    for k, v, n in ((None, 256, 2), (256, None, 2), (264, 256, 2), (256, 256, 3), (256, 256, -1)):
        assert lib.lsa_paged_append(r, k, v, n, None, None, None) == inv
    assert lib.lsa_paged_append(r, 256, 256, 1 << 31, 256, None, None) == inv
    for budget, sink, recent in ((0, 0, 1), (5, -1, 1), (5, 1, 0), (5, 3, 3), (1 << 30, (1 << 31) - 1, 1)):
        assert lib.lsa_paged_evict(r, budget, sink, recent, None, None) == inv
    assert lib.lsa_paged_evict(C.byref(_cache(score=None)), 5, 1, 1, None, None) == inv
    assert lib.lsa_paged_evict(C.byref(_cache(free_stride=0)), 5, 1, 1, None, None) == inv
    for opt in (dict(window=5), dict(slopes=256), dict(prefix_len=256), dict(doc_start=256)):
        assert lib.lsa_paged_evict(C.byref(_cache(block_pos=None, **opt)), 5, 1, 1, None, None) == inv
    # a dst with arrays missing, or kept where the cache keeps none
    for bad in (dict(block_table=None), dict(n_entries=None), dict(tail_len=None), dict(block_pos=None),
                dict(score=None), dict(free_list=None), dict(free_cnt=None)):
        d = _cache(**bad).t
        assert lib.lsa_paged_evict(r, 5, 1, 1, C.byref(d), None) == inv
        assert lib.lsa_paged_append(r, 256, 256, 2, None, C.byref(d), None) == inv
    assert lib.lsa_paged_append(C.byref(_cache(score=None)), 256, 256, 2, None, C.byref(_cache().t), None) == inv


def test_workspace_size(lib):
    f = lib.lsa_paged_attn_workspace_size
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    for B, H, Hkv, d, E in ((1, 64, 1, 512, 16385), (64, 64, 8, 128, 64), (3, 21, 7, 256, 1)):
        slots, G = 2 * 148 + B * Hkv, H // Hkv
        base = up(B * 16) + up(B * Hkv * 8) + up(slots * G * 8) + up(slots * G * d * 4)
        assert f(B, H, Hkv, d, E, 0, 148) == base
        assert f(B, H, Hkv, d, E, 1, 148) == base + up(B * E * 2 * H * 8)
    for bad in ((0, 8, 1, 128, 4), (1, 9, 2, 128, 4), (1, 65, 1, 128, 4), (1, 8, 1, 100, 4), (1, 8, 1, 128, 0)):
        assert f(*bad, 1, 148) == 0
    assert f(1, 8, 1, 128, 4, 1, 0) == 0


def test_binding_refuses_host_tensors():
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        lsa.LsaPagedTables(torch.zeros((2, 4), dtype=torch.int32), i32, i32)
    with pytest.raises(ValueError):
        lsa.LsaPagedCache(torch.zeros((3, 2, 1, 64, 128)), None, 8)
