"""The paged grouped-query cache on the GPU: attention with score options, append and eviction
against plain float64 implementations, and a run of all three together.

Attention tolerance, per output. With z off by at most dz, a weight is off by a factor of at most
1 +- 2 dz (its own score and the normaliser's). Scores: products of 16-bit values are exact in
fp32; a d-term sum formed 16 terms at a time, each step off by at most 2^-23 of the largest
partial sum, is off by (d/16 + 1) 2^-23 of sum |q k|; scaling, cap, bias and the exponent's
argument add a few fp32 roundings of |z| and of the bias (at most 4 of 2^-23 together, of terms no
larger than the score range used here), and 2^x 2^-22. Each weight is then rounded to the inputs'
type (eps / 2), the fp32 sums add (parts + tokens/32) 2^-24, covered by the 2^-19 below, and the
output is rounded once (eps / 2 of itself):
    |out - ref| <= (eps/2 + 2 dz + 2^-19) sum w|V| + (eps/2) |ref|  (+ fp16: T 2^-25 max|V|,
weights below fp16's normal range). A page's weight: (2 dz + 2^-19) of it, no rounding to 16 bits.
"""
import math

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_lsa_b200 as lsa
from lookahead_sparse_kv_lsa_b200 import _lib
from oracle import paged_oracle as po

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).to(DEV)


class Case:
    """A cache with scattered pages; everything that must not matter holds NaN or infinity."""

    def __init__(self, lens, H, Hkv, d, dtype="bf16", seed=0, gap=1, score=True, cap=0.0, window=0,
                 slopes=None, prefix=None, docs=None, q_scale=1.0, spare=2, dense_pos=False, junk=True,
                 extra=0, decay=0.75):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        t = TYPES[dtype]
        B = len(lens)
        lens = np.asarray(lens)
        n = (lens + 63) // 64
        tail = np.where(n > 0, lens - (n - 1) * 64, 0)
        E = max(1, int(n.max())) + extra
        self.pages = int(n.sum()) + spare
        pool = torch.randn((self.pages, 2, Hkv, 64, d), generator=g).to(t)
        perm = rng.permutation(self.pages)
        table = np.full((B, E), -1, np.int32)
        pos = np.cumsum(rng.integers(1, 2 * gap, (B, E)), 1) - 1 if gap > 1 else np.tile(np.arange(E), (B, 1))
        k = 0
        for b in range(B):
            table[b, :n[b]] = perm[k:k + n[b]]
            k += n[b]
        if junk:
            for p in perm[k:]:
                pool[p] = float("nan")
            for b in range(B):
                if n[b]:
                    pool[table[b, n[b] - 1], 0, :, tail[b]:] = float("inf")
                    pool[table[b, n[b] - 1], 1, :, tail[b]:] = float("nan")
        self.lens, self.n, self.tail, self.B, self.E = lens, n, tail, B, E
        self.H, self.Hkv, self.d, self.t, self.dtype = H, Hkv, d, t, dtype
        self.table, self.pos = table, pos
        self.prefix = np.zeros(B, np.int64) if prefix is None else np.asarray(prefix)
        self.docs = np.zeros(B, np.int64) if docs is None else np.asarray(docs)
        self.cap, self.window, self.decay, self.scale = cap, window, decay, float(np.float32(d ** -0.5))
        self.slopes = None if slopes is None else np.asarray(slopes, np.float32)
        self.q = (torch.randn((B, H, d), generator=g) * q_scale).to(t)
        self.score0 = torch.rand((B, E), generator=g) if score else None
        if junk and (self.prefix.any() or self.docs.any() or window):
            for b in range(B):     # positions behind the masks
                if n[b] == 0:
                    continue
                seen, _ = po.seen_positions(pos[b], n[b], tail[b], self.prefix[b], self.docs[b], window)
                hide = np.ones((n[b], 64), bool)
                for j, s, _ in seen:
                    hide[j, s] = False
                hide = torch.from_numpy(hide)
                for j in range(n[b]):
                    pool[table[b, j], 0, :, hide[j]] = float("nan")
                    pool[table[b, j], 1, :, hide[j]] = float("-inf")
        self.pool = pool
        self.tables = lsa.LsaPagedTables(i32(table), i32(n), i32(tail), None if dense_pos else i32(pos),
                                         self.score0.to(DEV) if score else None)
        self.cache = lsa.LsaPagedCache(
            pool.to(DEV), self.tables, H, cap=cap, window=window, decay=decay,
            slopes=None if slopes is None else torch.from_numpy(self.slopes).to(DEV),
            prefix_len=None if prefix is None else i32(self.prefix),
            doc_start=None if docs is None else i32(self.docs))
        self.out = torch.full((B, H, d), 7.0, dtype=t, device=DEV)

    def run(self):
        self.cache.attend(self.q.to(DEV), self.out)
        torch.cuda.synchronize()
        return self

    def check(self, err=0, seqs=None):
        assert self.cache.read_err() == err
        got = self.out.double().cpu().numpy()
        eps = torch.finfo(self.t).eps
        for b in (range(self.B) if seqs is None else seqs):
            own = np.unique(self.table[b, :self.n[b]])
            own = own[(own >= 0) & (own < self.pages)]
            pool = dict(zip(own.tolist(), self.pool[own].double().numpy()))
            look = np.stack([pool[p] for p in own]) if len(own) else np.zeros((0, 2, self.Hkv, 64, self.d))
            back = np.full(self.E, -1)
            for j in range(self.n[b]):
                hit = np.flatnonzero(own == self.table[b, j])
                back[j] = hit[0] if len(hit) else -1
            ref, mass, absv, big = po.attend(
                self.q[b].double().numpy(), look, back, self.pos[b], int(self.n[b]), int(self.tail[b]),
                self.scale, self.cap, None if self.slopes is None else self.slopes.astype(np.float64),
                int(self.prefix[b]), int(self.docs[b]), self.window)
            far = 0.0
            if self.slopes is not None and self.n[b] > 0:
                # the bias, relative to the last seen position, is rounded twice in log2 units. Where it
                # lowers scores, the weights fall with it (b 2^-b < 1); where it raises them, its
                # largest value counts
                span = float(self.pos[b, self.n[b] - 1] - self.pos[b, 0] + 1) * 64
                far = max(2.0, 2 * span * float(max(0.0, -self.slopes.min())) * 1.5)
            dz = big * ((self.d / 16 + 1 + 4) * 2.0 ** -23) + far * 2.0 ** -23 + self.cap * 2.0 ** -22 + 2.0 ** -22
            tol = (eps / 2 + 2 * dz[:, None] + 2.0 ** -19) * absv + eps / 2 * np.abs(ref)
            if self.dtype == "fp16":
                tol = tol + self.lens[b] * 2.0 ** -25 * 8.0 + 2.0 ** -25     # and subnormal outputs
            bad = ~(np.abs(got[b] - ref) <= tol)
            assert not bad.any(), (b, np.argwhere(bad)[:5], got[b][bad][:5], ref[bad][:5], tol[bad][:5])
            if self.score0 is not None:
                sc = self.tables.score[b].double().cpu().numpy()
                s0 = self.score0[b].double().numpy()
                want = s0.copy()
                want[:self.n[b]] = self.decay * s0[:self.n[b]] + mass
                lim = np.abs(want) * 2.0 ** -22
                lim[:self.n[b]] += mass * (2 * dz.max() + 2.0 ** -19)
                assert np.array_equal(sc[self.n[b]:], s0[self.n[b]:])
                off = ~(np.abs(sc - want) <= lim + 1e-30)
                assert not off.any(), (b, np.argwhere(off)[:5], sc[off][:5], want[off][:5])
        return self


SHAPES = [
    # lens, H, Hkv, d, dtype
    ([1], 8, 1, 128, "bf16"),
    ([17], 8, 1, 128, "fp16"),
    ([31, 32, 33, 63, 64, 65], 4, 2, 128, "bf16"),
    ([127, 128, 129, 0, 1, 191], 64, 1, 512, "bf16"),
    ([0], 8, 8, 128, "bf16"),
    ([0, 0, 5], 3, 1, 256, "fp16"),
    ([700, 1, 0, 350, 64], 32, 8, 128, "fp16"),
    ([1000], 1, 1, 128, "bf16"),
    ([513, 20], 21, 7, 256, "bf16"),
    ([2049], 17, 1, 384, "bf16"),
    ([1531, 77], 32, 1, 512, "fp16"),
    ([900, 33], 33, 1, 128, "bf16"),
    ([400, 130], 64, 1, 256, "fp16"),
    ([350], 64, 1, 384, "fp16"),
    ([260, 70], 40, 2, 384, "bf16"),
    ([300, 31], 60, 3, 512, "bf16"),
    ([5000], 16, 4, 128, "bf16"),
    ([100, 200], 256, 4, 128, "bf16"),
    ([90], 512, 8, 128, "fp16"),
    ([33], 1024, 16, 128, "bf16"),
]


@pytest.mark.parametrize("lens,H,Hkv,d,dtype", SHAPES, ids=lambda x: str(x)[:24].replace(" ", ""))
def test_attend_shapes(cuda_ok, lens, H, Hkv, d, dtype):
    Case(lens, H, Hkv, d, dtype, seed=H + d).run().check()


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("B", [193, 400])
def test_many_short_sequences(cuda_ok, B, score):
    # more sequences than a block has threads, and more per CTA than are planned at a time
    lens = [(i * 37) % 70 for i in range(B)]
    lens[B // 2] = 9000
    Case(lens, 2, 1, 128, seed=B, score=score, extra=3).run().check(seqs=list(range(0, B, 7)) + [B // 2, B - 1])


def test_many_records_per_cta(cuda_ok):
    # one long sequence sets the share of a CTA, which then holds dozens of one-token sequences
    lens = [40000] + [1] * 300
    Case(lens, 1, 1, 128, seed=5).run().check(seqs=[0, 1, 2, 16, 17, 33, 150, 299, 300])


LONG = [
    # lens, H, Hkv, d, dtype, options: many tiles per segment, segments that end anywhere
    ([1000 + 37 * i for i in range(16)], 32, 8, 128, "fp16", dict(cap=30.0, window=700, prefix=[100 + i for i in range(16)])),
    ([2500 - 91 * i for i in range(12)], 64, 8, 128, "bf16", dict(docs=[150 * i for i in range(12)], gap=2)),
    ([9001, 30, 12345, 640], 64, 1, 512, "bf16", dict(cap=50.0)),
    ([20017], 64, 1, 512, "fp16", dict(window=15001, prefix=[700], gap=2)),
    ([30011], 20, 1, 512, "bf16", dict(window=20000)),
    ([8003, 16001], 32, 2, 384, "fp16", dict(prefix=[1000, 33], docs=[4001, 9000])),
    ([60001, 5], 16, 1, 256, "bf16", dict(window=50001)),
    ([31000, 200], 33, 1, 256, "bf16", dict(docs=[17, 100])),
    ([50021], 64, 2, 128, "fp16", dict(prefix=[5000], window=40000)),
    ([100003], 4, 1, 128, "bf16", dict(slopes=[1.0, 0.1, 0.001, 0.0])),
    ([60001], 8, 1, 128, "bf16", dict(q_scale=6.0)),
]


@pytest.mark.parametrize("lens,H,Hkv,d,dtype,kw", LONG, ids=[str(c[0][0]) for c in LONG])
def test_many_tiles_per_cta(cuda_ok, lens, H, Hkv, d, dtype, kw):
    c = Case(lens, H, Hkv, d, dtype, seed=H, **kw)
    c.run().check(seqs=range(0, len(lens), 1 if len(lens) < 5 else 5))
    first = c.out.clone()
    for _ in range(3):
        c.run()
        assert torch.equal(c.out, first)
    assert c.cache.read_err() == 0


@pytest.mark.parametrize("H,d", [(8, 128), (64, 512), (24, 256)])
def test_a_bad_page_hides_a_whole_tile(cuda_ok, H, d):
    # the newest units of a segment show nothing, the older ones set its running max
    c = Case([70000], H, 1, d, seed=14)
    c.table[0, ::3] = -1
    c.table[0, 1::3] = 1 << 24
    c.tables.block_table.copy_(i32(c.table))
    c.run().check(err=_lib.DEVERR_BAD_PAGE)


MASKS = [
    dict(window=1), dict(window=64), dict(window=65), dict(window=200), dict(window=10 ** 6),
    dict(prefix=[1, 63, 64, 65]), dict(prefix=[1, 63, 64, 65], window=1),
    dict(prefix=[100, 200, 300, 600], window=130), dict(docs=[0, 1, 64, 500]),
    dict(docs=[10 ** 6] * 4), dict(docs=[10 ** 6] * 4, prefix=[0, 1, 70, 500]),
    dict(docs=[599, 598, 560, 575], prefix=[0, 577, 577, 5]), dict(docs=[300, 10, 130, 64], window=256),
    dict(prefix=[-5, 0, 10 ** 6, 2], docs=[-7, 3, 4, 5], window=3),
    # both bounds in one page: slots are missing in its middle
    dict(docs=[100, 90, 127, 40], prefix=[70, 65, 66, 10]), dict(docs=[599, 590, 576, 63], prefix=[598, 577, 570, 3]),
    dict(window=30), dict(docs=[590, 580, 570, 20], prefix=[500, 576, 540, 0]),
]


@pytest.mark.parametrize("gap", [1, 5])
@pytest.mark.parametrize("kw", MASKS, ids=str)
def test_masks(cuda_ok, kw, gap):
    Case([600, 599, 577, 64], 8, 2, 128, seed=3, gap=gap, **kw).run().check()


@pytest.mark.parametrize("H,d,dtype", [(8, 128, "bf16"), (32, 256, "fp16"), (64, 512, "bf16")])
def test_masks_of_other_tiles(cuda_ok, H, d, dtype):
    Case([1500, 700], H, 1, d, dtype, seed=9, gap=3, prefix=[77, 100], docs=[2000, 900], window=5000).run().check()


@pytest.mark.parametrize("kw", [dict(cap=0.5), dict(cap=30.0), dict(cap=1e4), dict(cap=30.0, q_scale=20.0),
                                dict(q_scale=20.0), dict(slopes="alibi"), dict(slopes="alibi", gap=7),
                                dict(slopes="rising"), dict(slopes="alibi", cap=20.0, window=300, prefix=[40, 9])],
                         ids=str)
@pytest.mark.parametrize("H,Hkv,d", [(16, 2, 128), (64, 1, 512)])
def test_score_options(cuda_ok, H, Hkv, d, kw):
    kw = dict(kw)
    if kw.get("slopes") == "alibi":
        kw["slopes"] = 2.0 ** (-8.0 * np.arange(1, H + 1) / H)
    elif kw.get("slopes") == "rising":          # far tokens gain: the running max rises tile by tile
        kw["slopes"] = np.where(np.arange(H) % 2, -0.05, 0.05)
    Case([3001, 150], H, Hkv, d, seed=11, **kw).run().check()


def test_no_positions_means_consecutive(cuda_ok):
    a = Case([600, 130], 8, 2, 128, seed=4, window=100, dense_pos=True).run().check()
    b = Case([600, 130], 8, 2, 128, seed=4, window=100).run()
    assert torch.equal(a.out, b.out) and torch.equal(a.tables.score, b.tables.score)


def test_first_token_returns_its_value(cuda_ok):
    c = Case([1, 1], 8, 2, 128, seed=2).run()
    for b in range(2):
        v = c.pool[c.table[b, 0], 1, :, 0]
        assert torch.equal(c.out[b].cpu(), v.repeat_interleave(4, 0))


def test_bad_pages_and_sizes(cuda_ok):
    c = Case([300, 300, 300, 300], 8, 2, 128, seed=6)
    c.table[0, 1], c.table[1, 4] = 1 << 30, -1
    c.tables.block_table.copy_(i32(c.table))
    c.run().check(err=_lib.DEVERR_BAD_PAGE)
    c = Case([300, 300, 300, 300, 300], 8, 2, 128, seed=7)
    n, tail = c.n.copy(), c.tail.copy()
    n[0], n[1], tail[2], tail[3] = -1, c.E + 1, 0, 65
    c.tables.n_entries.copy_(i32(n))
    c.tables.tail_len.copy_(i32(tail))
    c.run().check(err=_lib.DEVERR_BAD_SIZE, seqs=[4])
    assert torch.count_nonzero(c.out[:4]) == 0
    assert torch.equal(c.tables.score[:4].cpu(), c.score0[:4])


def test_same_bits_again_and_on_a_stream_and_in_a_graph(cuda_ok):
    c = Case([3000, 41, 700], 16, 4, 128, seed=8, cap=30.0)
    c.run()
    first, s1 = c.out.clone(), c.tables.score.clone()
    q = c.q.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.tables.score.copy_(c.score0)
    c.out.zero_()
    torch.cuda.synchronize()
    c.cache.attend(q, c.out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(c.out, first) and torch.equal(c.tables.score, s1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.cache.attend(q, c.out)
        c.cache.attend(q, c.out)
    for _ in range(2):
        c.tables.score.copy_(c.score0)
        c.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first)
    c.tables.score.copy_(c.score0)
    c.cache.attend(q, c.out)
    c.cache.attend(q, c.out)
    twice = c.tables.score.clone()
    c.tables.score.copy_(c.score0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.tables.score, twice)


def test_workspace_carries_no_state(cuda_ok):
    c = Case([2000, 300], 8, 1, 256, seed=12)
    c.run()
    first = c.out.clone()
    c.cache.ws.fill_(255)
    c.tables.score.copy_(c.score0)
    c.run().check()
    assert torch.equal(c.out, first)


def test_positions_out_of_order_stay_in_bounds(cuda_ok):
    """What such a table attends to is not specified; nothing outside it is read, and its neighbours
    are right."""
    rng = np.random.default_rng(0)
    for kw in (dict(window=300), dict(prefix=[500] * 4, docs=[900] * 4), dict(slopes=[0.1] * 8, window=700, prefix=[70] * 4)):
        c = Case([1500, 900, 1200, 640], 8, 2, 128, seed=15, junk=False, **kw)
        pos = c.pos.copy()
        pos[0] = rng.permutation(c.E)
        pos[1] = rng.integers(-5, 1 << 25, c.E)
        pos[3] = 7
        c.tables.block_pos.copy_(i32(pos))
        c.run()
        assert c.cache.read_err() == 0
        c.check(seqs=[2])


def test_far_offsets(cuda_ok):
    # a pool past 2^32 bytes: pages near its end
    H, d = 8, 128
    pages = (1 << 32) // (2 * 64 * d * 2) + 300
    pool = torch.zeros((pages, 2, 1, 64, d), dtype=torch.bfloat16, device=DEV)
    c = Case([500], H, 1, d, seed=13, junk=False)
    at = torch.arange(pages - 8, pages)
    pool[at] = c.pool[c.table[0, :8]].to(DEV)
    t = lsa.LsaPagedTables(i32(at[None]), i32(c.n), i32(c.tail), i32(c.pos[:, :8]), c.tables.score)
    cache = lsa.LsaPagedCache(pool, t, H, decay=c.decay)
    cache.attend(c.q.to(DEV), c.out)
    torch.cuda.synchronize()
    c.check()


def test_agrees_with_lsa_decode_attn_on_a_gathered_table(cuda_ok):
    """The pool and the block table of the LSA step driver, attended with one key head."""
    import lsa_inputs as LI
    wl = LI.Workload(LI.tiny(), pin=True)
    cfg, dev = wl.cfg, torch.device("cuda")
    nc = (int(wl.ctx0[0]) - cfg.W) // 64
    dec = lsa.LsaDecoder(wl.w_q.to(dev), wl.k_idx.to(dev), wl.blk_off[:1], torch.from_numpy(wl.bias).to(dev),
                         wl.host_pool, wl.blk_off, wl.nb0, W=cfg.W, H=cfg.H, cap=nc, max_cand=nc, scale=cfg.scale)
    dec.load_window(0)
    a = torch.empty((1, cfg.H, cfg.d), dtype=torch.bfloat16, device=dev)
    b = torch.empty_like(a)
    k, v = wl.kv_new(0, 0)
    q = wl.q(0, 0).to(dev)
    dec.step(0, wl.h(0).to(dev), q, k.to(dev), v.to(dev), a)
    t = lsa.LsaPagedTables(dec.block_table, dec.n_entries, dec.tail_len)
    lsa.LsaPagedCache(dec.hbm_pool.unsqueeze(2), t, cfg.H, scale=cfg.scale).attend(q, b)
    torch.cuda.synchronize()
    assert dec.read_err() == 0
    # each rounds its weights and its output to bf16: twice 2 * eps/2 of sum w|V| <= max|V| < 6
    assert (a.float() - b.float()).abs().max().item() <= 2 * torch.finfo(torch.bfloat16).eps * 6


# ------------------------------------------------------------------------------ append
def check_append(B, Hkv, d, held, new, dtype="bf16", ragged=True, spare=3, in_place=True, pos=True, seed=0,
                 bt_extra=40, bad=None):
    rng = np.random.default_rng(seed)
    t = TYPES[dtype]
    held, new = np.asarray(held), np.asarray(new)
    n = (held + 63) // 64
    tail = np.where(n > 0, held - (n - 1) * 64, 0)
    E = int(n.max()) + bt_extra
    F = int(((held + new + 63) // 64 - n).max()) + spare
    pages = B * (E + F)
    perm = rng.permutation(pages).astype(np.int32).reshape(B, E + F)
    table, free = perm[:, :E].copy(), perm[:, E:].copy()
    cnt = rng.integers(0, F + 1, B) if spare == 0 else np.full(B, F)
    bpos = np.cumsum(rng.integers(1, 4, (B, E)), 1).astype(np.int32) if pos else np.tile(np.arange(E, dtype=np.int32), (B, 1))
    pool = torch.randn((pages, 2, Hkv, 64, d)).to(t)
    total = int(new.sum())
    k, v = torch.randn((total + 2 * ragged, Hkv, d)).to(t), torch.randn((total + 2 * ragged, Hkv, d)).to(t)
    off = np.concatenate([[0], np.cumsum(new)])
    score = rng.random((B, E)).astype(np.float32)
    src = lsa.LsaPagedTables(i32(table), i32(n), i32(tail), i32(bpos) if pos else None, torch.from_numpy(score).to(DEV),
                             i32(free), i32(cnt))
    dst = None
    if not in_place:
        dst = lsa.LsaPagedTables(i32(np.full_like(table, -3)), i32(n * 0 - 1), i32(n * 0 - 1),
                                 i32(np.full_like(table, -3)) if pos else None, torch.full((B, E), -3.0, device=DEV),
                                 i32(free * 0), i32(n * 0 - 1))
    c = lsa.LsaPagedCache(pool.to(DEV), src, Hkv)
    c.append(k.to(DEV), v.to(DEV), i32(off) if ragged else None, dst=dst)
    torch.cuda.synchronize()
    out = dst or src
    want_pool, err = pool.clone(), 0
    w_table = table.copy() if in_place else np.full_like(table, -3)
    w_pos = bpos.copy() if in_place else np.full_like(table, -3)
    w_score = score.copy() if in_place else np.full_like(score, -3.0)
    w_n, w_tail, w_cnt = n.copy(), tail.copy(), cnt.copy()
    for b in range(B):
        got = po.append(int(n[b]), int(tail[b]), free[b, :cnt[b]], int(new[b]), table[b, :n[b]].tolist(),
                        bpos[b, :n[b]].tolist(), E)
        if got is None:
            err |= _lib.DEVERR_POOL_CAPACITY
            continue
        w_n[b], left, w_cnt[b] = got[0], got[2], len(got[2])
        w_tail[b] = got[1] if got[0] else tail[b]
        for j, (p, x) in got[4].items():
            w_table[b, j], w_pos[b, j], w_score[b, j] = p, x, 0.0
        for i, (p, s) in enumerate(got[3]):
            want_pool[p, 0, :, s], want_pool[p, 1, :, s] = k[off[b] + i], v[off[b] + i]
    assert c.read_err() == err
    assert np.array_equal(out.n_entries.cpu().numpy(), w_n)
    assert np.array_equal(out.tail_len.cpu().numpy(), w_tail)
    assert np.array_equal(out.free_cnt.cpu().numpy(), w_cnt)
    assert np.array_equal(out.block_table.cpu().numpy(), w_table)
    if pos:
        assert np.array_equal(out.block_pos.cpu().numpy(), w_pos)
    assert np.array_equal(out.score.cpu().numpy(), w_score)
    assert torch.equal(c.pool.cpu().view(torch.int16), want_pool.view(torch.int16))
    return err


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,Hkv,d,dtype", [(1, 1, 128, "bf16"), (5, 3, 384, "fp16"), (70, 8, 128, "bf16"), (2, 8, 512, "fp16")])
def test_append_one_token(cuda_ok, B, Hkv, d, dtype, in_place):
    held = [(64 * i + (0, 1, 63, 64, 0, 127)[i % 6]) % 300 for i in range(B)]
    check_append(B, Hkv, d, held, [1] * B, dtype, ragged=False, in_place=in_place, seed=B)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("held,new", [([0], [1]), ([0], [0]), ([63], [2]), ([0, 64, 5, 200, 0], [130, 0, 59, 300, 64]),
                                      ([1] * 40, [(i * 13) % 90 for i in range(40)])], ids=str)
def test_append_ragged(cuda_ok, held, new, in_place):
    check_append(len(held), 2, 128, held, new, "fp16", in_place=in_place, seed=len(held), pos=len(held) != 5)


def test_append_out_of_pages(cuda_ok):
    assert check_append(8, 2, 128, [0, 64, 30, 128, 64, 0, 64, 60], [200, 1, 30, 500, 64, 1, 65, 9], spare=0, seed=21)
    # the table's width runs out before the pages do
    assert check_append(3, 1, 128, [64, 128, 100], [70, 1, 20], bt_extra=0, spare=4, seed=22)
    assert check_append(3, 1, 128, [64, 128, 100], [1, 1, 1], ragged=False, bt_extra=0, spare=4, seed=23)


def test_append_bad_sizes_and_pages(cuda_ok):
    B, E, F = 7, 4, 3
    pool = torch.zeros((64, 2, 1, 64, 128), dtype=torch.bfloat16, device=DEV)
    n, tail, cnt = np.array([1, -1, 5, 1, 1, 1, 1]), np.array([5, 5, 5, 0, 65, 64, 5]), np.array([1, 1, 1, 1, 1, 4, 1])
    table = np.arange(B * E).reshape(B, E)
    table[0, 0] = 64                     # outside the pool
    free = 32 + np.arange(B * F).reshape(B, F)
    for off in (None, [0, 1, 2, 3, 4, 5, 6, 5], [0, 1, 2, 3, 4, 5, 6, 99], [3, 1, 2, 3, 4, 5, 6, 7]):
        t = lsa.LsaPagedTables(i32(table), i32(n), i32(tail), None, None, i32(free), i32(cnt))
        c = lsa.LsaPagedCache(pool.zero_(), t, 1)
        k = torch.ones((B, 1, 128), dtype=torch.bfloat16, device=DEV)
        c.append(k, k, None if off is None else i32(off))
        torch.cuda.synchronize()
        err = c.read_err()
        assert err & _lib.DEVERR_BAD_SIZE
        assert (err & _lib.DEVERR_BAD_PAGE) != 0 or (off is not None and off[0] == 3)
        new_n, new_tail = t.n_entries.cpu().numpy(), t.tail_len.cpu().numpy()
        assert np.array_equal(new_n, n) and np.array_equal(new_tail[1:6], tail[1:6])
        assert np.array_equal(t.free_cnt.cpu().numpy(), cnt)
        good = off is None or off[-1] == 7          # the last sequence's token is well formed
        assert torch.count_nonzero(pool).item() == (2 * 128 if good else 0)


# ------------------------------------------------------------------------------ eviction
def check_evict(n, budget, sink, recent, score=None, in_place=True, pos=True, seed=0, E=None, cnt=None, F=None):
    rng = np.random.default_rng(seed)
    n = np.asarray(n)
    B, E = len(n), E or max(1, int(n.max()))
    F = F or E + 5
    table = rng.integers(0, 1 << 20, (B, E)).astype(np.int32)
    bpos = np.cumsum(rng.integers(1, 5, (B, E)), 1).astype(np.int32)
    score = np.exp(2 * rng.standard_normal((B, E))).astype(np.float32) if score is None else score
    free = rng.integers(0, 1 << 20, (B, F)).astype(np.int32)
    cnt = rng.integers(0, 6, B) if cnt is None else np.asarray(cnt)
    tail = rng.integers(1, 65, B)
    src = lsa.LsaPagedTables(i32(table), i32(n), i32(tail), i32(bpos) if pos else None, torch.from_numpy(score).to(DEV),
                             i32(free), i32(cnt))
    dst = None
    if not in_place:
        dst = lsa.LsaPagedTables(i32(table * 0 - 3), i32(n * 0), i32(n * 0), i32(table * 0 - 3) if pos else None,
                                 torch.full((B, E), -3.0, device=DEV), i32(free * 0 - 3), i32(n * 0))
    c = lsa.LsaPagedCache(torch.zeros((1, 2, 1, 64, 128), dtype=torch.bfloat16, device=DEV), src, 1)
    c.evict(budget, sink, recent, dst=dst)
    torch.cuda.synchronize()
    out = dst or src
    w = [x.copy() if in_place else np.full_like(x, -3) for x in (table, bpos, score, free)]
    w_n, w_cnt, err = n.copy(), cnt.copy(), 0
    for b in range(B):
        if n[b] < 0 or n[b] > E or cnt[b] < 0 or cnt[b] > F:
            err |= _lib.DEVERR_BAD_SIZE
            continue
        kept, gone = po.evict(score[b], int(n[b]), budget, sink, recent)
        if cnt[b] + len(gone) > F:
            err |= _lib.DEVERR_POOL_CAPACITY
            kept, gone = list(range(n[b])), []
        w_n[b], w_cnt[b] = len(kept), cnt[b] + len(gone)
        for x, y in zip(w[:3], (table, bpos, score)):
            x[b, :len(kept)] = y[b, kept]
        w[3][b, cnt[b]:cnt[b] + len(gone)] = table[b, gone]
    assert c.read_err() == err
    assert np.array_equal(out.n_entries.cpu().numpy(), w_n)
    assert np.array_equal(out.free_cnt.cpu().numpy(), w_cnt)
    assert np.array_equal(out.tail_len.cpu().numpy(), tail)
    assert np.array_equal(out.block_table.cpu().numpy(), w[0])
    if pos:
        assert np.array_equal(out.block_pos.cpu().numpy(), w[1])
    assert np.array_equal(out.score.cpu().numpy().view(np.int32), w[2].view(np.int32))
    assert np.array_equal(out.free_list.cpu().numpy(), w[3])
    return err


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("n,budget,sink,recent", [
    ([1], 1, 0, 1), ([2], 1, 0, 1), ([5, 0, 3, 4], 3, 1, 1), ([65] * 8, 64, 1, 16), ([65, 64, 63, 200], 64, 30, 34),
    ([1000, 3, 999, 512], 100, 0, 1), ([4097, 4096, 1], 512, 4, 64), ([16385], 1351, 1, 129), ([20000, 17000], 5000, 2, 3),
    ([33] * 70, 20, 5, 5), ([256, 255, 250], 250, 3, 3), ([257, 300], 100, 0, 2), ([4096, 100], 99, 1, 1), ([4097], 4096, 1, 1),
    ([18432, 18431], 18431, 1, 1), ([4097, 5, 0, 4100, 33], 20, 4, 9), ([32768, 40, 7], 9000, 100, 100),
    ([32769, 5], 9000, 100, 100)], ids=str)
def test_evict(cuda_ok, n, budget, sink, recent, in_place):
    check_evict(n, budget, sink, recent, in_place=in_place, seed=len(n), pos=budget != 100)


@pytest.mark.parametrize("kind", ["zeros", "few", "negative", "signed_zero", "inf", "nan", "all_nan", "near"])
def test_evict_ties_and_odd_scores(cuda_ok, kind):
    rng = np.random.default_rng(3)
    n = [700, 300, 64, 1500]
    s = rng.standard_normal((4, 1500)).astype(np.float32)
    if kind == "zeros":
        s[:] = 0
    elif kind == "few":
        s = rng.integers(0, 3, s.shape).astype(np.float32)
    elif kind == "negative":
        s = -np.abs(s)
    elif kind == "signed_zero":
        s = np.where(rng.random(s.shape) < 0.5, -0.0, 0.0).astype(np.float32)
    elif kind == "inf":
        s = rng.choice(np.array([np.inf, -np.inf, 1.0, np.finfo(np.float32).min], np.float32), s.shape)
    elif kind == "nan":
        s[rng.random(s.shape) < 0.6] = np.nan
    elif kind == "all_nan":
        s[:] = np.nan
    else:
        s = (1 + rng.integers(0, 9, s.shape) * 2.0 ** -23).astype(np.float32)
    check_evict(n, 200, 3, 10, score=s, seed=4)
    check_evict(n, 13, 3, 10, score=s, seed=5, in_place=False)
    wide = np.tile(s, (1, 4))                      # rows of more scores a thread
    check_evict([5900, 4200, 64, 6000], 2001, 3, 10, score=wide, seed=6)
    long = np.tile(s, (1, 22))                     # rows that are read again
    check_evict([33000, 300, 64, 32900], 2001, 3, 10, score=long, seed=7)


def test_evict_full_stack_and_bad_sizes(cuda_ok):
    assert check_evict([50, 50, 50, 10], 20, 1, 1, F=32, cnt=[2, 3, 32, 32], seed=6) == _lib.DEVERR_POOL_CAPACITY
    assert check_evict([50, 50, 50, 10], 20, 1, 1, F=32, cnt=[2, 3, 32, 32], seed=6, in_place=False)
    assert check_evict([50, -1, 61, 60, 50, 10], 20, 1, 1, E=60, cnt=[0, 0, 0, -1, 99, 0], seed=7) == _lib.DEVERR_BAD_SIZE


def test_evict_long_rows(cuda_ok):
    """Rows whose keys do not fit the registers of a cluster."""
    check_evict([50000, 40], 3001, 7, 9, seed=8)


# ------------------------------------------------------------------------------ together
def test_a_bounded_cache_decodes(cuda_ok):
    """Prompts in, then decode with the budget held by eviction, against a token-by-token model of
    the same rules in float64: contents, tables, scores and outputs stay together."""
    B, H, Hkv, d, budget, sink, recent = 3, 8, 2, 128, 6, 1, 2
    g = torch.Generator().manual_seed(0)
    t = lsa.LsaPagedTables.allocate(B, 12, 14, DEV)
    pool = torch.full((B * 14, 2, Hkv, 64, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(H)], device=DEV)
    c = lsa.LsaPagedCache(pool, t, H, cap=30.0, decay=0.9, slopes=slopes)
    prompt = [500, 0, 130]
    model = [dict(ent=[]) for _ in range(B)]      # entries: [pos, score, [k..], [v..]]

    def add(b, k, v):
        ent = model[b]["ent"]
        if not ent or len(ent[-1][2]) == 64:
            ent.append([ent[-1][0] + 1 if ent else 0, 0.0, [], []])
        ent[-1][2].append(k)
        ent[-1][3].append(v)

    def new(n):
        return (torch.randn((n, Hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))

    k, v = new(sum(prompt))
    c.append(k.to(DEV), v.to(DEV), i32(np.concatenate([[0], np.cumsum(prompt)])))
    at = 0
    for b in range(B):
        for i in range(prompt[b]):
            add(b, k[at].double().numpy(), v[at].double().numpy())
            at += 1
    out = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV)
    for step in range(150):
        k, v = new(B)
        q = torch.randn((B, H, d), generator=g).to(torch.bfloat16)
        c.append(k.to(DEV), v.to(DEV))
        c.attend(q.to(DEV), out)
        check = step % 37 == 0 or step == 149
        before = t.score.cpu().numpy() if check else None
        c.evict(budget, sink, recent)
        for b in range(B):
            add(b, k[b].double().numpy(), v[b].double().numpy())
            ent = model[b]["ent"]
            n, tail = len(ent), len(ent[-1][2])
            P = np.zeros((n, 2, Hkv, 64, d))
            for j, e in enumerate(ent):
                P[j, 0, :, :len(e[2])] = np.stack(e[2], 1)
                P[j, 1, :, :len(e[3])] = np.stack(e[3], 1)
            pos = [e[0] for e in ent]
            ref, mass, absv, _ = po.attend(q[b].double().numpy(), P, range(n), pos, n, tail, d ** -0.5, cap=30.0,
                                           slopes=slopes.double().cpu().numpy())
            for e, m in zip(ent, mass):
                e[1] = 0.9 * e[1] + m
            if check:
                got = out[b].double().cpu().numpy()
                assert (np.abs(got - ref) <= 2.0 ** -8 * (absv + np.abs(ref)) + 1e-4).all(), (step, b)
                assert np.allclose(before[b, :n], [e[1] for e in ent], rtol=1e-4, atol=1e-6), (step, b)
            kept, _ = po.evict(np.array([e[1] for e in ent]), n, budget, sink, recent)
            model[b]["ent"] = [ent[j] for j in kept]
    torch.cuda.synchronize()
    assert c.read_err() == 0
    for b in range(B):
        ent = model[b]["ent"]
        n = int(t.n_entries[b])
        assert n == len(ent) and int(t.tail_len[b]) == len(ent[-1][2])
        assert t.block_pos[b, :n].tolist() == [e[0] for e in ent]
        held = t.block_table[b, :n].tolist()
        free = t.free_list[b, :int(t.free_cnt[b])].tolist()
        assert sorted(held + free) == list(range(b * 14, (b + 1) * 14))


def test_two_caches_on_two_streams(cuda_ok):
    """Caches of their own, at the same time: each gets what it gets alone."""
    cs = [Case([30000, 41, 700], 16, 4, 128, seed=8, cap=30.0), Case([9000, 400], 64, 1, 512, "fp16", seed=9)]
    alone = [c.run().out.clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    qs = [c.q.to(DEV) for c in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, st in zip(cs, qs, streams):
            c.out.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for c, q, st in zip(cs, qs, streams):
                c.cache.attend(q, c.out, stream=st)
        torch.cuda.synchronize()
        for c, o in zip(cs, alone):
            assert torch.equal(c.out, o) and c.cache.read_err() == 0


def test_a_captured_step_decodes(cuda_ok):
    """append, attend and evict of one step in a graph: replays advance the cache as calls do."""
    B, H, Hkv, d, budget = 5, 16, 4, 128, 5
    g = torch.Generator().manual_seed(1)
    prompt = [300, 0, 1, 64, 447]
    off = i32(np.concatenate([[0], np.cumsum(prompt)]))
    kp, vp = (torch.randn((sum(prompt), Hkv, d), generator=g).to(torch.float16).to(DEV) for _ in range(2))
    steps = [[torch.randn(s, generator=g).to(torch.float16).to(DEV) for s in ((B, Hkv, d), (B, Hkv, d), (B, H, d))]
             for _ in range(140)]
    got = []
    for captured in (False, True):
        t = lsa.LsaPagedTables.allocate(B, 10, 12, DEV)
        pool = torch.full((B * 12, 2, Hkv, 64, d), float("nan"), dtype=torch.float16, device=DEV)
        c = lsa.LsaPagedCache(pool, t, H, cap=20.0, window=200, prefix_len=i32([10, 0, 64, 1, 70]), decay=0.9)
        c.append(kp, vp, off)
        k, v, q = (x.clone() for x in steps[0])
        out = torch.empty((B, H, d), dtype=torch.float16, device=DEV)

        def step():
            c.append(k, v)
            c.attend(q, out)
            c.evict(budget, 1, 2)

        graph = None
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        outs = []
        for s in steps:
            for x, y in zip((k, v, q), s):
                x.copy_(y)
            graph.replay() if captured else step()
            outs.append(out.clone())
        torch.cuda.synchronize()
        assert c.read_err() == 0
        got.append((torch.stack(outs), t))
    assert torch.equal(got[0][0], got[1][0])
    for name in ("block_table", "block_pos", "score", "n_entries", "tail_len", "free_list", "free_cnt"):
        assert torch.equal(getattr(got[0][1], name), getattr(got[1][1], name)), name
    assert torch.isfinite(got[0][0].float()).all()


def test_binding_refusals(cuda_ok):
    c = Case([100, 10], 8, 2, 128, seed=1)
    q = c.q.to(DEV)
    for bad in (c.q, q[:1], q.float(), q.to(torch.float16), q.transpose(0, 1), q[:, :, :64],
                torch.empty((2, 8, 256), dtype=torch.bfloat16, device=DEV)[:, :, ::2]):
        with pytest.raises(ValueError):
            c.cache.attend(bad, c.out)
        with pytest.raises(ValueError):
            c.cache.attend(q, bad)
    kv = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device=DEV)
    for bad in (kv[:, :1], kv.cpu(), kv.float(), kv[0]):
        with pytest.raises((ValueError, lsa.LsaError)):
            c.cache.append(bad, kv)
        with pytest.raises((ValueError, lsa.LsaError)):
            c.cache.append(kv, bad)
    with pytest.raises(ValueError):
        c.cache.append(kv, kv, i32([0, 1]))
    with pytest.raises(lsa.LsaError):
        c.cache.append(torch.cat([kv, kv]), torch.cat([kv, kv]))       # four tokens, no offsets
    with pytest.raises(lsa.LsaError):
        c.cache.evict(5)                                               # no free stack
    other = Case([100, 10], 8, 2, 128, seed=1, extra=1)
    with pytest.raises(ValueError):
        c.cache.append(kv, kv, dst=other.tables)
    with pytest.raises(lsa.LsaError):
        lsa.LsaPagedCache(c.cache.pool, c.tables, 7)
    with pytest.raises(ValueError):
        lsa.LsaPagedCache(c.cache.pool[:, :, :, :32], c.tables, 8)
    mis = torch.empty(2 * 8 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, 8, 128)
    with pytest.raises(lsa.LsaError):
        c.cache.attend(mis, c.out)
