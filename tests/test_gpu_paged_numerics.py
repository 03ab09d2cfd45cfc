"""Paged attention where its numbers are hardest: long caches in fp16, weights far below their row's
largest, biases of either sign over long distances, and scores that are not numbers.

The reference is the definition in float64. Tolerance, with u = eps / 2 of the inputs' type, one
rounding:
  scores    a d-term sum of exact products, 16 terms at a time, and the roundings behind it: dz <=
            big ((d/16 + 5) 2^-23) + 2^-22, big the largest scale * sum |q k|; a cap adds cap 2^-22.
            A bias is relative to the end of the seen positions that it favours, so it only lowers
            scores: a token b log2 units down has at most the weight 2^(r - b), r <= 3 big the range of
            the other scores, and b 2^-23 of it is below (3 big + 1) 2^-23. A weight is off by 2 dz.
  weights   rounded to the inputs' type for the product with V: u each; in fp16, where they are
            scaled by 2^7 and subnormal below 2^-14, also 2^-25 2^-7 of the row's largest weight,
            which is 1 / sum(exp(z - max))
  sums      the product adds 16 tokens a step, each step off by at most 2^-23 of the partial sum;
            the fp32 sums of the weights add a step per 128 tokens and some dozens of the parts:
            s = (T/16 + T/128 + 64) 2^-23 for T seen tokens
  output    rounded once: u |ref|, in fp16 at least 2^-25
  |out - ref| <= 1.01 ((u + 2 dz + s) sum w|V| + u |ref| + fp16: 2^-32 sum|V| / sum(exp(z - max)) + 2^-25)
(1.01 for products of these terms). A page's weight: 2 dz + s of it, and a rounding.
"""
import numpy as np
import pytest
import torch

import lookahead_sparse_kv_lsa_b200 as lsa
from lookahead_sparse_kv_lsa_b200 import _lib
from oracle import paged_oracle as po
from test_gpu_paged import DEV, TYPES, Case, i32

pytestmark = pytest.mark.gpu


def seen_rows(c, b):
    """Page, slot, entry and position (tensors) of the positions that sequence b's newest token sees."""
    n = int(c.n[b])
    if n == 0:
        return None, None
    at, x_b = po.seen_positions(c.pos[b], n, int(c.tail[b]), int(c.prefix[b]), int(c.docs[b]), c.window)
    at = np.array([p for p in at if 0 <= c.table[b, p[0]] < c.pages], dtype=np.int64).reshape(-1, 3)
    return at, x_b


def reference(c, b):
    """Sequence b from the definition: out [H][d], mass [n], and for the tolerance the sums w|V| and
    |V| [H][d], sum(exp(z - max)) [H], big [H] and the number of seen tokens."""
    H, G, d, n = c.H, c.H // c.Hkv, c.d, int(c.n[b])
    f64 = dict(dtype=torch.float64, device=DEV)
    out, absv, sumv = (torch.zeros(H, d, **f64) for _ in range(3))
    denom, big, mass = torch.ones(H, **f64), torch.zeros(H, **f64), torch.zeros(n, **f64)
    at, x_b = seen_rows(c, b)
    T = 0 if at is None else len(at)
    for g in range(c.Hkv if T else 0):
        page = torch.from_numpy(c.table[b, at[:, 0]].astype(np.int64)).to(DEV)
        slot, ent = (torch.from_numpy(at[:, k].copy()).to(DEV) for k in (1, 0))
        K, V = (c.cache.pool[page, k, g, slot].double() for k in (0, 1))
        h = slice(g * G, (g + 1) * G)
        q = c.q[b, h].to(DEV).double()
        z = K @ q.T * c.scale                                               # [T][G]
        big[h] = (K.abs() @ q.abs().T * c.scale).amax(0)
        if c.cap > 0:
            z = c.cap * torch.tanh(z / c.cap)
        if c.slopes is not None:
            far = torch.from_numpy((x_b - at[:, 2]).astype(np.float64)).to(DEV)
            z = z - far[:, None] * torch.from_numpy(c.slopes[h].astype(np.float64)).to(DEV)
        e = torch.exp(z - z.amax(0))
        denom[h] = e.sum(0)
        w = e / denom[h]
        out[h], absv[h], sumv[h] = w.T @ V, w.T @ V.abs(), V.abs().sum(0).expand(G, d)
        mass.index_add_(0, ent, w.sum(1))
    return [x.cpu().numpy() for x in (out, mass, absv, sumv, denom, big)] + [T]


def check(c, seqs=None, err=0, norm=False):
    """The tolerance above; with `norm` also the relative 2-norm of each head's error, for values
    that do not depend on the weights: there a weight's error e_w adds a term of random sign, and
    the norm grows by max |e_w| of itself (1.3 for the spread of d such sums), where the
    elementwise bound has to allow for sum w|V|, many times the result in a long row."""
    assert c.cache.read_err() == err
    u, fp16 = torch.finfo(c.t).eps / 2, c.dtype == "fp16"
    for b in range(c.B) if seqs is None else seqs:
        ref, mass, absv, sumv, denom, big, T = reference(c, b)
        got = c.out[b].double().cpu().numpy()
        dz = big * ((c.d / 16 + 5) * 2.0 ** -23) + 2.0 ** -22 + c.cap * 2.0 ** -22
        if c.slopes is not None:
            dz = dz + (3 * big + 1) * 2.0 ** -23
        s = (T / 16 + T / 128 + 64) * 2.0 ** -23
        low = 2.0 ** -32 / denom[:, None] if fp16 else 0.0
        tol = 1.01 * ((u + 2 * dz[:, None] + s) * absv + u * np.abs(ref) + low * sumv + (2.0 ** -25 if fp16 else 0.0))
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])
        if norm:
            size = np.linalg.norm(ref, axis=1)
            rel = np.linalg.norm(got - ref, axis=1) / size
            v = np.sqrt((sumv / max(T, 1)) ** 2 * np.pi / 2).mean(1)            # rms of normal values
            lim = 1.3 * (2 * u + 2 * dz) + 4 * s + (1.3 * low[:, 0] * np.sqrt(T * c.d) * v / size if fp16 else 0.0)
            assert (rel <= lim).all(), (b, rel, lim)
        if c.score0 is not None:
            n = int(c.n[b])
            sc, s0 = c.tables.score[b].double().cpu().numpy(), c.score0[b].double().numpy()
            want = s0.copy()
            want[:n] = c.decay * s0[:n] + mass
            lim = np.abs(want) * 2.0 ** -22 + 1e-30
            lim[:n] += mass * (2 * dz.max() + s)
            off = ~(np.abs(sc - want) <= lim)
            assert not off.any(), (b, np.argwhere(off)[:5], sc[off][:5], want[off][:5], lim[off][:5])


# ------------------------------------------------------------------- scores that are not numbers
NAN_CASES = [
    # lens, H, Hkv, d, options: pairs held whole, split pairs joined by a warp and by a block
    ([40, 100], 8, 2, 128, {}),
    ([9000, 40, 0, 3000], 8, 2, 128, {}),
    ([9000], 8, 1, 128, {}),
    ([5000], 64, 1, 512, dict(cap=30.0)),
    ([4000, 77], 24, 1, 256, dict(window=3000, prefix=[100, 10])),
    ([1500 + 64 * i for i in range(20)], 16, 8, 128, dict(docs=[50 * i for i in range(20)])),
]


def twin(c):
    """The same case's results before something in it turns into NaN."""
    c.run()
    out, score = c.out.clone(), c.tables.score.clone()
    c.tables.score.copy_(c.score0)
    c.out.fill_(7.0)
    return out, score


@pytest.mark.parametrize("lens,H,Hkv,d,kw", NAN_CASES, ids=lambda x: str(x)[:20].replace(" ", ""))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_nan_query_gives_nan_however_its_pair_is_split(cuda_ok, lens, H, Hkv, d, kw, dtype):
    c = Case(lens, H, Hkv, d, dtype, seed=21, **kw)
    out, score = twin(c)
    hit = [(0, 1), (len(lens) - 1, H - 1)]
    for b, h in hit:
        c.q[b, h, 5] = float("nan")
    c.run()
    assert c.cache.read_err() == 0
    nan = torch.zeros((c.B, H), dtype=torch.bool, device=DEV)
    for b, h in hit:
        nan[b, h] = True
    assert torch.isnan(c.out[nan]).all()
    assert torch.equal(c.out[~nan], out[~nan])
    # every page with a position that is seen gets its weight from that head too
    for b in range(c.B):
        at, _ = seen_rows(c, b)
        touched = torch.zeros(c.E, dtype=torch.bool)
        if b in [x for x, _ in hit] and at is not None:
            touched[np.unique(at[:, 0])] = True
        sc = c.tables.score[b].cpu()
        assert torch.isnan(sc[touched]).all()
        assert torch.equal(sc[~touched], score[b].cpu()[~touched])


@pytest.mark.parametrize("H,Hkv,d,lens", [(8, 2, 128, [9000, 40]), (64, 1, 512, [5000]), (24, 1, 256, [6000, 900])])
@pytest.mark.parametrize("slopes", [False, True])
def test_nan_keys_of_far_pages_reach_every_head(cuda_ok, H, Hkv, d, lens, slopes):
    """NaN keys in a run of pages that other CTAs than the newest token's hold, with a bias under
    which these pages' other weights are zero."""
    c = Case(lens, H, Hkv, d, seed=22, slopes=np.full(H, 1.0) if slopes else None)
    out, score = twin(c)
    n = int(c.n[0])
    pages = torch.from_numpy(c.table[0, n // 4:n // 2].astype(np.int64)).to(DEV)
    c.cache.pool[pages, 0, 0] = float("nan")
    c.run()
    assert c.cache.read_err() == 0
    G = H // Hkv
    assert torch.isnan(c.out[0, :G]).all()
    assert torch.equal(c.out[0, G:], out[0, G:]) and torch.equal(c.out[1:], out[1:])
    assert torch.isnan(c.tables.score[0, :n]).all()
    assert torch.equal(c.tables.score[1:], score[1:])


@pytest.mark.parametrize("H,d,lens", [(8, 128, [9000]), (64, 512, [5000, 100]), (4, 128, [100])])
def test_a_nan_value_counts_where_its_weight_is_zero_in_fp32(cuda_ok, H, d, lens):
    """0 * NaN is NaN, in one dimension, whichever CTA holds the token."""
    c = Case(lens, H, 1, d, seed=23, slopes=np.full(H, 2.0))
    out, score = twin(c)
    c.cache.pool[int(c.table[0, 0]), 1, 0, 3, 77] = float("nan")
    c.run()
    assert c.cache.read_err() == 0
    assert torch.isnan(c.out[0, :, 77]).all()
    rest = torch.arange(d, device=DEV) != 77
    assert torch.equal(c.out[0][:, rest], out[0][:, rest]) and torch.equal(c.out[1:], out[1:])
    assert torch.equal(c.tables.score, score)


@pytest.mark.parametrize("lens", [[100], [9000]])
def test_scores_of_minus_infinity_only_give_zeros(cuda_ok, lens):
    c = Case(lens, 8, 2, 128, seed=24)
    c.q.abs_()
    c.cache.pool[torch.from_numpy(c.table[0, :int(c.n[0])].astype(np.int64)).to(DEV), 0] = float("-inf")
    c.run()
    assert c.cache.read_err() == 0
    assert torch.count_nonzero(c.out) == 0
    want = c.score0.clone()
    want[0, :int(c.n[0])] *= c.decay
    assert torch.equal(c.tables.score.cpu(), want)


# ------------------------------------------------------------- weights far below the largest one
def peaked(c, b, nats):
    """Sequence b's newest token outweighs every other by `nats` in every head; it has the value 0, so
    that the output is what the others' small weights make of it."""
    n, t = int(c.n[b]), int(c.tail[b])
    page = int(c.table[b, n - 1])
    c.cache.pool[page, 0, :, t - 1] = 0
    c.cache.pool[page, 0, :, t - 1, 0] = 16.0
    c.cache.pool[page, 1, :, t - 1] = 0
    c.q[b, :, 0] = nats / (16.0 * c.scale)


FLAT = [
    # lens, H, Hkv, d, nats: all but the newest token of the same key, weights at and below 2^-24
    ([128], 4, 1, 128, 17.4), ([100, 7], 16, 2, 128, 17.0), ([64], 64, 1, 512, 18.0), ([128], 24, 1, 256, 16.0),
    ([9000, 2000], 8, 2, 128, 17.4), ([4097], 64, 1, 512, 17.4),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens,H,Hkv,d,nats", FLAT, ids=lambda x: str(x).replace(" ", ""))
def test_small_weights_count(cuda_ok, lens, H, Hkv, d, nats, dtype):
    c = Case(lens, H, Hkv, d, dtype, seed=31, junk=False)
    for b in range(c.B):
        own = torch.from_numpy(c.table[b, :int(c.n[b])].astype(np.int64)).to(DEV)
        c.cache.pool[own, 0] = 0
        c.cache.pool[own, 1] = c.cache.pool[own, 1].abs() * 256 + 256       # outputs in fp16's normal range
        peaked(c, b, nats)
    check(c.run())


@pytest.mark.parametrize("nats", [12.0, 14.0, 16.0])
def test_small_weights_of_whole_pairs_count(cuda_ok, nats):
    """592 pairs over 296 CTAs: a row of 8,192 tokens, scores N(0, 1) but for the newest token's, in
    one segment. The tables name the same pages many times."""
    B, Hkv, d, E = 74, 8, 128, 128
    c = Case([64 * E] + [64] * 199, Hkv, Hkv, d, "fp16", seed=32, junk=False, score=False)
    g = np.random.default_rng(5)
    table = g.choice(c.table[0, :E], (B, E)).astype(np.int32)
    table[:, -1] = c.table[1:B + 1, 0]
    c.B, c.E, c.table, c.pos = B, E, table, np.tile(np.arange(E), (B, 1))
    c.lens, c.n, c.tail = np.full(B, 64 * E), np.full(B, E), np.full(B, 64)
    c.prefix = c.docs = np.zeros(B, np.int64)
    c.q = c.q[:B].clone()
    c.cache.pool[:, 1] = c.cache.pool[:, 1] * 0.5 + 1
    c.cache.pool[:, 0, :, :, 0] = 0
    old = c.cache
    c.tables = lsa.LsaPagedTables(i32(table), i32(c.n), i32(c.tail), i32(c.pos))
    c.cache = lsa.LsaPagedCache(old.pool, c.tables, c.H)
    c.out = torch.empty((B, c.H, d), dtype=c.t, device=DEV)
    for b in range(B):
        peaked(c, b, nats)
    check(c.run(), seqs=[0, 1, 36, 73])
    # and with values of mean 1 under the newest token too
    c.cache.pool[torch.from_numpy(table[:, -1].astype(np.int64)).to(DEV), 1, :, -1] = 1
    check(c.run(), seqs=[0, 40, 73])


def test_scores_too_large_for_the_weights_scale(cuda_ok):
    """Score differences of 2^20 and more, where neighbouring fp32 numbers are further apart than the
    room above the running max: one token takes all the weight, and none overflows."""
    c = Case([1000, 70], 8, 2, 128, "fp16", seed=33, q_scale=1.0, junk=False)
    for k in (4096.0, 32768.0):                  # powers of two: equal sums stay equal in fp32
        c.q = (torch.sign(c.q.float()) * k).to(c.t)
        c.cache.pool[:, 0] = torch.sign(c.cache.pool[:, 0]) * k
        big = (c.q.float().abs().max() * c.cache.pool[:, 0].float().abs().max()).item()
        assert big > 2 ** 23
        c.tables.score.copy_(c.score0)
        c.run()
        assert c.cache.read_err() == 0 and torch.isfinite(c.out.float()).all()
        for b in range(c.B):
            # the weights are 1 / m for the m largest scores: sums of +-1, equal ones exactly so
            ref = reference(c, b)[0]
            got = c.out[b].double().cpu().numpy()
            assert (np.abs(got - ref) <= 2.0 ** -9 * np.abs(c.pool.float().abs().max().item())).all()


# ---------------------------------------------------------------------------- long rows
LONG = [
    ([1000 + 37 * i for i in range(16)], 32, 8, 128, dict(cap=30.0, window=700, prefix=[100 + i for i in range(16)])),
    ([20017], 64, 1, 512, dict(window=15001, prefix=[700], gap=2)),
    ([8003, 16001], 32, 2, 384, dict(prefix=[1000, 33], docs=[4001, 9000])),
    ([50021], 64, 2, 128, dict(prefix=[5000], window=40000)),
    ([30011], 20, 1, 512, dict(window=20000)),
    ([100003], 4, 1, 128, {}),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens,H,Hkv,d,kw", LONG, ids=[str(c[0][0]) for c in LONG])
def test_long_rows_by_their_norm(cuda_ok, lens, H, Hkv, d, kw, dtype):
    check(Case(lens, H, Hkv, d, dtype, seed=H, **kw).run(), seqs=range(0, len(lens), 5), norm=True)


# --------------------------------------------------------------------- biases of either sign
@pytest.mark.parametrize("lens,H,Hkv,d,kw", [
    ([100003], 4, 1, 128, {}),
    ([30000], 8, 2, 128, dict(gap=40)),                         # over 1.2M positions
    ([30000, 2000], 8, 2, 128, dict(gap=40, prefix=[300, 0], window=200000)),
    ([9000, 500], 8, 2, 128, dict(gap=40, docs=[100000, 999], cap=20.0)),
    ([9000], 40, 1, 256, dict(gap=100)),
    ([5000, 30, 0], 64, 1, 512, dict(gap=200)),
    ([50, 64, 65, 1], 8, 8, 128, {}),
], ids=lambda x: str(x)[:24].replace(" ", ""))
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_biases_of_either_sign_over_long_distances(cuda_ok, lens, H, Hkv, d, kw, dtype):
    slopes = np.resize([-0.5, 0.5, -2.0, 0.0, -0.01, 1.0, -1e-4, 1e-6], H)
    check(Case(lens, H, Hkv, d, dtype, seed=41, slopes=slopes, **kw).run())


# ------------------------------------------------------------------------- blocks nobody sees
@pytest.mark.parametrize("prefix", [None, [100, 0, 64, 576]])
@pytest.mark.parametrize("gap", [1, 3])
def test_a_document_that_starts_behind_the_newest_token(cuda_ok, prefix, gap):
    """doc_start in the tail block's unfilled slots: no slot of that block is seen, and it is not
    looked at. Its table entry lies outside the pool."""
    c = Case([600, 577, 10, 639], 8, 2, 128, seed=51, gap=gap, docs=[0] * 4, prefix=prefix)
    n = c.n - 1
    c.docs = 64 * c.pos[np.arange(4), n] + c.tail + np.array([0, 5, 3, 0])
    c.cache.doc_start.copy_(i32(c.docs))
    if prefix is not None:                       # up to the tail block, not into it
        c.prefix = np.minimum(c.prefix, 64 * c.pos[np.arange(4), n])
        c.cache.prefix_len.copy_(i32(c.prefix))
    c.table[np.arange(4), n] = [-1, 1 << 20, -7, c.pages]
    c.tables.block_table.copy_(i32(c.table))
    check(c.run())


def test_a_prefix_that_reaches_into_an_unseen_tail_block(cuda_ok):
    c = Case([600, 577, 10, 640], 8, 2, 128, seed=52, docs=[610, 578, 11, 10 ** 6], prefix=[590, 577, 64, 600],
             junk=True)
    check(c.run())
    c.table[0, -1] = -1                          # the prefix reaches this one
    c.tables.block_table.copy_(i32(c.table))
    c.tables.score.copy_(c.score0)
    check(c.run(), err=_lib.DEVERR_BAD_PAGE)


# ------------------------------------------------------------------ tables of the LSA step driver
def test_options_on_a_gathered_table(cuda_ok):
    """lsa_gather writes no positions. Formed as the header says, from the ids of the kept blocks and
    of the window's, they give window, document, prefix and bias their meaning on its table."""
    from types import SimpleNamespace

    import lsa_inputs as LI
    wl = LI.Workload(LI.tiny(), pin=True)
    cfg, dev = wl.cfg, torch.device("cuda")
    nc = max(1, max((int(x) - cfg.W) // 64 for x in wl.ctx0))
    dec = lsa.LsaDecoder(wl.w_q.to(dev), wl.k_idx.to(dev), wl.blk_off[:cfg.B], torch.from_numpy(wl.bias).to(dev),
                         wl.host_pool, wl.blk_off, wl.nb0, W=cfg.W, H=cfg.H, cap=nc, max_cand=nc, scale=cfg.scale)
    dec.load_window(0)
    k, v = wl.kv_new(0, 0)
    a = torch.empty((cfg.B, cfg.H, cfg.d), dtype=torch.bfloat16, device=dev)
    dec.step(0, wl.h(0).to(dev), wl.q(0, 0).to(dev), k.to(dev), v.to(dev), a)
    torch.cuda.synchronize()
    assert dec.read_err() == 0
    E = dec.block_table.shape[1]
    j = torch.arange(E, dtype=torch.int32, device=dev)[None]
    kept = dec.sel_cnt[:, None]
    ids = torch.cat([dec.sel_ids, torch.zeros((cfg.B, E - dec.sel_ids.shape[1]), dtype=torch.int32, device=dev)], 1)
    pos = torch.where(j < kept, ids, dec.n_cand[:, None] + j - kept)
    n = dec.n_entries.cpu().numpy()
    assert any((np.diff(pos[b, :n[b]].cpu().numpy()) > 1).any() for b in range(cfg.B))      # blocks were left out
    assert [int(pos[b, n[b] - 1]) for b in range(cfg.B)] == [int(x) for x in wl.nb0]
    W = int(cfg.W)
    for kw in (dict(slopes=True), dict(window=2 * W + 700), dict(docs=True), dict(window=W // 2, prefix=True, cap=5.0, slopes=True)):
        c = SimpleNamespace(B=cfg.B, H=cfg.H, Hkv=1, d=cfg.d, E=E, t=torch.bfloat16, dtype="bf16", cap=kw.get("cap", 0.0),
                            window=kw.get("window", 0), decay=0.5, scale=float(np.float32(cfg.scale)), n=n,
                            tail=dec.tail_len.cpu().numpy(), table=dec.block_table.cpu().numpy(), pos=pos.cpu().numpy(),
                            q=wl.q(0, 0), pages=dec.n_pages, score0=torch.rand((cfg.B, E)), slopes=None)
        last = 64 * np.asarray(wl.nb0)
        c.prefix = np.full(cfg.B, 1000 if "prefix" in kw else 0)
        c.docs = last // 3 + 17 if "docs" in kw else np.zeros(cfg.B, np.int64)
        if "slopes" in kw:
            c.slopes = (2.0 ** -np.arange(6, 6 + cfg.H)).astype(np.float32)
        c.tables = lsa.LsaPagedTables(dec.block_table, dec.n_entries, dec.tail_len, pos.contiguous(), c.score0.to(dev))
        c.cache = lsa.LsaPagedCache(dec.hbm_pool.unsqueeze(2), c.tables, cfg.H, scale=cfg.scale, cap=c.cap, window=c.window,
                                    decay=0.5, slopes=None if c.slopes is None else torch.from_numpy(c.slopes).to(dev),
                                    prefix_len=i32(c.prefix) if "prefix" in kw else None,
                                    doc_start=i32(c.docs) if "docs" in kw else None)
        c.out = torch.empty_like(a)
        c.cache.attend(c.q.to(dev), c.out)
        torch.cuda.synchronize()
        check(c)
