"""The quantized cache: lines as they are written into pages and read back.

Everything bit for bit: a line's codes, scales and amax are those of the
framework's quantizers (the oracle's for NVFP4), the values read back are two or
three rounded FP32 steps that the host takes alike. Every byte of the cache that
no token names keeps what it held.
"""
import numpy as np
import pytest
import torch

import oracle
import precision_quantization_row_amd as p
from parity_utils import say
from product_utils import DEV, E4M3, unpack

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
FORMATS = ("nvfp4", "e4m3", "int8")
QTYPE = {"nvfp4": torch.uint8, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    p.load_library()


class Cache:
    """Pages of one kind of lines, filled with a pattern, and the same on the host as bytes."""

    def __init__(self, fmt, pages, size, H, D, seed=0):
        r = np.random.RandomState(seed)
        self.fmt, self.pages, self.size, self.H, self.D = fmt, pages, size, H, D
        n = (pages, size, H)
        width = (D + 1) // 2 if fmt == "nvfp4" else D
        self.hq = r.randint(0, 256, n + (width,)).astype(np.uint8)
        if fmt == "e4m3":
            self.hq &= 0xF7   # no NaN
        self.hs = r.randint(0, 127, n + ((D + 15) // 16,)).astype(np.uint8) if fmt == "nvfp4" else None
        self.ha = np.exp(r.standard_normal(n)).astype(np.float32)
        self.q = torch.from_numpy(self.hq).to(DEV).view(QTYPE[fmt])
        self.s = None if self.hs is None else torch.from_numpy(self.hs).to(DEV)
        self.amax = torch.from_numpy(self.ha).to(DEV)

    def args(self):
        return self.q, self.s, self.amax

    def put(self, slot, x, bound):
        """Lines x [n, H, D] (float32, host) at rows `slot` of the host's copy."""
        n = len(slot)
        if n == 0:
            return
        lines = np.ascontiguousarray(x.reshape(n * self.H, self.D))
        a = np.abs(lines).max(1)
        with np.errstate(all="ignore"):
            enc = lambda top: np.where(a == 0, np.float32(1), np.minimum(np.float32(top) / a, np.finfo(np.float32).max)).astype(np.float32)[:, None]
            if self.fmt == "nvfp4":
                q, s = oracle.quantize_rowwise(lines, oracle.MODE_LINE, a, bound)
                self.hs.reshape(-1, self.H, self.hs.shape[-1])[slot] = np.asarray(s).reshape(n, self.H, -1)
            elif self.fmt == "e4m3":
                q = torch.from_numpy(np.clip(lines * enc(448), -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            else:
                q = np.clip(np.rint(lines * enc(127)), -127, 127).astype(np.int8).view(np.uint8)
        self.hq.reshape(-1, self.H, self.hq.shape[-1])[slot] = np.asarray(q).reshape(n, self.H, -1)
        self.ha.reshape(-1, self.H)[slot] = a.reshape(n, self.H)

    def values(self, slot, bound):
        """FP32 values of rows `slot`, [n, H, D]."""
        f = np.float32
        q, a = self.hq.reshape(-1, self.H, self.hq.shape[-1])[slot], self.ha.reshape(-1, self.H)[slot][..., None]
        if self.fmt == "nvfp4":
            sc = E4M3[self.hs.reshape(-1, self.H, self.hs.shape[-1])[slot]].astype(f)
            d = np.repeat((sc * a) * (f(1) / (f(bound) * f(6))), 16, -1)[..., :self.D]
            return unpack(q.reshape(-1, q.shape[-1]), self.D).astype(f).reshape(len(slot), self.H, self.D) * d
        if self.fmt == "e4m3":
            return E4M3[q].astype(f) * (a * (f(1) / f(448)))
        return q.view(np.int8).astype(f) * (a * (f(1) / f(127)))

    def check(self):
        assert np.array_equal(self.q.view(torch.uint8).cpu().numpy(), self.hq)
        assert self.hs is None or np.array_equal(self.s.cpu().numpy(), self.hs)
        assert np.array_equal(self.amax.cpu().numpy().view(np.uint32), self.ha.view(np.uint32))


class Plan:
    """Sequences of new (or read) tokens: lengths, positions, a table of shuffled pages."""

    def __init__(self, lengths, first, size, seed=0, spare=3, lead=0, behind=0):
        r = np.random.RandomState(seed)
        self.lengths, self.first = np.array(lengths), np.array(first)
        need = -(-(self.first + self.lengths) // size)
        self.pages = int(need.sum()) + spare
        order, at = r.permutation(self.pages), np.concatenate(([0], np.cumsum(need)))
        self.table = np.full((len(lengths), max(1, int(need.max())) + 1), -1, np.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = order[at[b]:at[b + 1]]
        self.starts = (lead + np.concatenate(([0], np.cumsum(lengths)))).astype(np.int32)
        self.T, self.size = int(self.starts[-1]) + behind, size
        row, slot = [], []
        for b, n in enumerate(lengths):
            pos = self.first[b] + np.arange(n)
            row.append(self.starts[b] + np.arange(n))
            slot.append(self.table[b, pos // size].astype(np.int64) * size + pos % size)
        self.row, self.slot = np.concatenate(row).astype(np.int64), np.concatenate(slot).astype(np.int64)

    def dev(self, first=True):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)
        return (t(self.table), t(self.starts)), dict(first=t(self.first) if first else None)


def rows(g, T, H, D, dtype, wide=False):
    """[T, H, D]; wide: a slice of longer rows."""
    if not wide:
        return torch.randn(T, H, D, generator=g).to(dtype).to(DEV)
    x = torch.randn(T, (2 * H + 1) * D + 3, generator=g).to(dtype).to(DEV)
    return x[:, D + 1:(H + 1) * D + 1].unflatten(1, (H, D))


# lengths, positions, page size
PLANS = [([1], [0], 16), ([1, 1, 1, 1], [0, 5, 15, 16], 16), ([7, 0, 0, 33, 1], [0, 3, 0, 60, 2], 16), ([100], [13], 1),
         ([5, 64, 3], [62, 0, 1], 64), ([200, 31], [3, 0], 7), ([40, 40], [0, 1000], 256)]
# H, D: every number of lanes a line takes, odd sizes, a latent line
HEADS = [(1, 1), (2, 7), (3, 16), (8, 64), (4, 80), (5, 100), (8, 128), (2, 129), (1, 192), (3, 256), (1, 257), (2, 512), (1, 576), (1, 1023),
         (2, 1024), (70, 24)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,D", HEADS)
def test_write_and_read(H, D, dtype, fmt):
    say(f"[gpu] cache {H}x{D} {dtype} {fmt}")
    g = torch.Generator().manual_seed(H * 100 + D)
    for i, (lengths, first, size) in enumerate(PLANS):
        pl = Plan(lengths, first, size, seed=i, lead=i % 3, behind=(0, 5)[i % 2])
        bound = (448.0, 256.0)[i % 2]
        kc, vc = Cache(fmt, pl.pages, size, H, D, 1), Cache(fmt, pl.pages, size, H, D, 2)
        k, v = rows(g, pl.T, H, D, dtype, wide=i % 2 == 0), rows(g, pl.T, H, D, dtype, wide=i % 3 == 0)
        seq, kw = pl.dev()
        p.nvfp4_cache_write(k, v, *kc.args(), *vc.args(), *seq, **kw, bound=bound)
        torch.cuda.synchronize()
        for c, x in ((kc, k), (vc, v)):
            c.put(pl.slot, x.float().cpu().numpy()[pl.row], bound)
            c.check()
        for out in (BF, FP):
            ko, vo = torch.full((pl.T, H, D), 7.0, dtype=out, device=DEV), rows(g, pl.T, H, D, out, wide=True)
            v0 = vo.clone()
            p.nvfp4_cache_read(ko, vo, *kc.args(), *vc.args(), *seq, **kw, bound=bound)
            torch.cuda.synchronize()
            for c, x, before in ((kc, ko, torch.full_like(ko, 7.0)), (vc, vo, v0)):
                before[torch.from_numpy(pl.row).to(DEV)] = torch.from_numpy(c.values(pl.slot, bound)).to(out).to(DEV)
                assert torch.equal(x, before)   # rows of no sequence as they were
        kc.check()
        vc.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_keys_alone(fmt):
    g = torch.Generator().manual_seed(3)
    pl = Plan([9, 30], [0, 7], 16)
    c, k = Cache(fmt, pl.pages, 16, 1, 576), rows(g, pl.T, 1, 576, BF)
    seq, kw = pl.dev()
    p.nvfp4_cache_write(k, None, *c.args(), None, None, None, *seq, **kw)
    c.put(pl.slot, k.float().cpu().numpy()[pl.row], 448.0)
    c.check()
    out = torch.empty(pl.T, 1, 576, device=DEV)
    p.nvfp4_cache_read(out, None, *c.args(), None, None, None, *seq, **kw)
    assert np.array_equal(out.cpu().numpy()[pl.row], c.values(pl.slot, 448.0))


@pytest.mark.parametrize("B", [1, 63, 64, 65, 127, 128, 300, 4095, 4096, 5000, 300000])
def test_many_sequences(B):
    """The search over the sequences' starts, empty ones among them, one to three levels deep."""
    say(f"[gpu] cache, {B} sequences")
    r = np.random.RandomState(B)
    lengths = r.randint(0, 3, B) if B < 300000 else (r.rand(B) < 0.05).astype(np.int64)
    lengths[B // 2] = 5
    pl = Plan(lengths, r.randint(0, 4, B), 8, behind=2)
    g = torch.Generator().manual_seed(B)
    c, k = Cache("int8", pl.pages, 8, 2, 16), rows(g, pl.T, 2, 16, FP)
    seq, kw = pl.dev()
    p.nvfp4_cache_write(k, None, *c.args(), None, None, None, *seq, **kw)
    c.put(pl.slot, k.cpu().numpy()[pl.row], 448.0)
    c.check()


@pytest.mark.parametrize("T", [1, 3, 1000, 1030, 5000, 40000])
@pytest.mark.parametrize("H,D", [(8, 128), (1, 64)])
def test_many_tokens(T, H, D):
    """Every number of tokens a workgroup takes."""
    say(f"[gpu] cache, {T} tokens {H}x{D}")
    g = torch.Generator().manual_seed(T)
    lengths = [T // 3, T - T // 3 - T // 5, T // 5]
    pl = Plan(lengths, [0, 21, 3], 16, behind=1)
    for fmt in FORMATS:
        c, k = Cache(fmt, pl.pages, 16, H, D), rows(g, pl.T, H, D, BF, wide=True)
        seq, kw = pl.dev()
        p.nvfp4_cache_write(k, None, *c.args(), None, None, None, *seq, **kw)
        c.put(pl.slot, k.float().cpu().numpy()[pl.row], 448.0)
        c.check()
        out = torch.empty(pl.T, H, D, device=DEV)
        p.nvfp4_cache_read(out, None, *c.args(), None, None, None, *seq, **kw)
        assert np.array_equal(out.cpu().numpy()[pl.row], c.values(pl.slot, 448.0))


@pytest.mark.parametrize("fmt", FORMATS)
def test_tokens_without_a_page(fmt):
    """Positions and pages that do not exist: skipped by the write, zeros from the read, whatever the arrays hold."""
    g = torch.Generator().manual_seed(4)
    H, D, size = 3, 40, 8
    pl = Plan([10, 12, 6, 9], [0, 3, 0, 2], size)
    table, first, starts = pl.table.copy(), pl.first.copy(), pl.starts.copy()
    ok = np.ones(len(pl.row), bool)
    seq_of, pos = np.repeat(np.arange(4), pl.lengths), np.concatenate([f + np.arange(n) for f, n in zip(first, pl.lengths)])
    table[0, 1] = -5                       # page before the first
    ok[(seq_of == 0) & (pos // size == 1)] = False
    table[1, 0] = pl.pages                 # one past the last
    ok[(seq_of == 1) & (pos // size == 0)] = False
    first[2] = -2                          # two negative positions; the others move
    first[3] = size * table.shape[1] - 4   # past the table's row after 4 tokens
    slot = pl.slot.copy()
    for b in (2, 3):
        for j in np.flatnonzero(seq_of == b):
            q = first[b] + j - np.flatnonzero(seq_of == b)[0]
            page = table[b, q // size] if 0 <= q < size * table.shape[1] else -1
            ok[j] = 0 <= page < pl.pages
            slot[j] = page * size + q % size
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)
    args = (dev(table), dev(starts))
    c, k = Cache(fmt, pl.pages, size, H, D), rows(g, pl.T, H, D, FP)
    p.nvfp4_cache_write(k, None, *c.args(), None, None, None, *args, first=dev(first))
    c.put(slot[ok], k.cpu().numpy()[pl.row[ok]], 448.0)
    c.check()
    out = torch.full((pl.T, H, D), 7.0, device=DEV)
    p.nvfp4_cache_read(out, None, *c.args(), None, None, None, *args, first=dev(first))
    want = np.zeros((pl.T, H, D), np.float32)
    want[pl.row[ok]] = c.values(slot[ok], 448.0)
    assert np.array_equal(out.cpu().numpy(), want)
    # arrays of garbage: nothing outside the cache is touched, nothing but lines of the cache is written
    r = np.random.RandomState(0)
    for _ in range(4):
        bad = (dev(r.randint(-2 ** 31, 2 ** 31, table.shape)), dev(r.randint(-50, 50, starts.shape)))
        p.nvfp4_cache_write(k, None, *c.args(), None, None, None, *bad, first=dev(r.randint(-2 ** 31, 2 ** 31 - 1, 4)))
        p.nvfp4_cache_read(out, None, *c.args(), None, None, None, *bad, first=dev(r.randint(-2 ** 31, 2 ** 31 - 1, 4)))
    torch.cuda.synchronize()
    c.check()   # (no page of these exists)


def test_without_first_and_at_any_address():
    g = torch.Generator().manual_seed(6)
    pl = Plan([20, 13], [0, 0], 16)
    for fmt in FORMATS:
        for D in (24, 37, 128):
            c = Cache(fmt, pl.pages, 16, 2, D)
            for shift in (0, 1, 3):
                buf = torch.randn(pl.T * 2 * D + 8, generator=g).to(BF).to(DEV)
                k = buf[shift:shift + pl.T * 2 * D].view(pl.T, 2, D)
                qb = torch.empty(c.q.numel() + 8, dtype=torch.uint8, device=DEV)[shift:shift + c.q.numel()]
                qb.copy_(c.q.view(torch.uint8).view(-1))
                c.q = qb.view(c.hq.shape).view(QTYPE[fmt])
                seq, _ = pl.dev()
                p.nvfp4_cache_write(k, None, *c.args(), None, None, None, *seq)
                c.put(pl.slot, k.float().cpu().numpy()[pl.row], 448.0)
                c.check()
                ob = torch.full((pl.T * 2 * D + 8,), 5.0, device=DEV)
                out = ob[shift:shift + pl.T * 2 * D].view(pl.T, 2, D)
                p.nvfp4_cache_read(out, None, *c.args(), None, None, None, *seq)
                assert np.array_equal(out.cpu().numpy()[pl.row], c.values(pl.slot, 448.0))
                assert bool((ob[:shift] == 5).all()) and bool((ob[shift + pl.T * 2 * D:] == 5).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_zeros_infinities_and_nan(fmt):
    """Lines of zeros; a line that holds a NaN reads back as NaN, its neighbours keep their bits."""
    g = torch.Generator().manual_seed(9)
    pl = Plan([6], [0], 8)
    k = rows(g, 6, 4, 64, FP)
    k[0, 1] = 0.0
    k[1, 2] = -0.0
    c = Cache(fmt, pl.pages, 8, 4, 64)
    seq, kw = pl.dev()
    p.nvfp4_cache_write(k, None, *c.args(), None, None, None, *seq, **kw)
    c.put(pl.slot, k.cpu().numpy(), 448.0)
    c.check()
    before = torch.empty_like(k)
    p.nvfp4_cache_read(before, None, *c.args(), None, None, None, *seq, **kw)
    k[2, 3, 5] = float("nan")
    k[3, 0, 63] = float("inf")
    p.nvfp4_cache_write(k, None, *c.args(), None, None, None, *seq, **kw)
    out = torch.empty_like(k)
    p.nvfp4_cache_read(out, None, *c.args(), None, None, None, *seq, **kw)
    assert bool(torch.isnan(out[2, 3]).all()) and not bool(torch.isfinite(out[3, 0]).any())
    keep = torch.ones(6, 4, dtype=torch.bool, device=DEV)
    keep[2, 3] = keep[3, 0] = False
    assert torch.equal(out[keep], before[keep])


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: lines in its last pages."""
    say("[gpu] cache past 2^32 bytes")
    H, D, size = 8, 128, 64
    pages = (1 << 32) // (size * H * D) + 40
    q = torch.zeros(pages, size, H, D, dtype=torch.int8, device=DEV)
    amax = torch.zeros(pages, size, H, device=DEV)
    assert q.numel() > 1 << 32
    g = torch.Generator().manual_seed(1)
    k = rows(g, 200, H, D, BF)
    table = torch.tensor([[pages - 1, 3, pages - 39, pages - 2]], dtype=torch.int32, device=DEV)
    starts, first = torch.tensor([0, 200], dtype=torch.int32, device=DEV), torch.tensor([10], dtype=torch.int32, device=DEV)
    p.nvfp4_cache_write(k, None, q, None, amax, None, None, None, table, starts, first=first)
    wq, wa = torch.empty(200 * H, D, dtype=torch.int8, device=DEV), torch.empty(200 * H, device=DEV)
    p.nvfp4_int8_quantize(k.view(-1, D), wa, wq)
    pos = torch.arange(10, 210, device=DEV)
    page = table[0].long()[pos // size]
    assert torch.equal(q[page, pos % size], wq.view(200, H, D)) and torch.equal(amax[page, pos % size], wa.view(200, H))
    assert int((amax != 0).sum()) == 200 * H
    out = torch.empty(200, H, D, device=DEV)
    p.nvfp4_cache_read(out, None, q, None, amax, None, None, None, table, starts, first=first)
    assert torch.equal(out, wq.view(200, H, D).float() * (wa * float(np.float32(1) / np.float32(127))).view(200, H, 1))


def test_noop_stream_and_replay():
    """Decode steps replayed from one graph: lengths and table change on the device."""
    g = torch.Generator().manual_seed(5)
    H, D, size, B = 8, 128, 16, 5
    pl = Plan([1] * B, [30, 0, 15, 16, 47], size)
    for fmt in FORMATS:
        kc, vc = Cache(fmt, pl.pages, size, H, D, 1), Cache(fmt, pl.pages, size, H, D, 2)
        k, v = rows(g, B, H, D, BF), rows(g, B, H, D, BF)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        seq, kw = pl.dev()

        def call(noop=None, stream=None):
            p.nvfp4_cache_write(k, v, *kc.args(), *vc.args(), *seq, **kw, noop=noop, stream=stream)
            p.nvfp4_cache_read(ko, vo, *kc.args(), *vc.args(), *seq, **kw, noop=noop, stream=stream)
        ko.fill_(3)
        call(noop=torch.ones(1, device=DEV))
        torch.cuda.synchronize()
        kc.check()
        assert bool((ko == 3).all())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(noop=torch.zeros(1, device=DEV), stream=side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        first = pl.first.copy()
        for c, x in ((kc, k), (vc, v)):
            c.put(pl.slot, x.float().cpu().numpy(), 448.0)
        for step in range(4):
            k.copy_(torch.randn(B, H, D, generator=g))
            v.copy_(torch.randn(B, H, D, generator=g))
            first = (first + 7) % (size * (pl.table.shape[1] - 1))
            kw["first"].copy_(torch.from_numpy(first.astype(np.int32)))
            graph.replay()
            torch.cuda.synchronize()
            pages = pl.table[np.arange(B), first // size].astype(np.int64)
            ok = pages >= 0
            slot = pages * size + first % size
            for c, x, o in ((kc, k, ko), (vc, v, vo)):
                c.put(slot[ok], x.float().cpu().numpy()[ok], 448.0)
                c.check()
                want = torch.zeros(B, H, D)
                want[torch.from_numpy(ok)] = torch.from_numpy(c.values(slot[ok], 448.0))
                assert torch.equal(o.cpu(), want.to(BF))


def test_refusals():
    H, D = 2, 32
    c, v = Cache("int8", 4, 16, H, D), Cache("int8", 4, 16, H, D)
    n = Cache("nvfp4", 4, 16, H, D)
    k = torch.zeros(3, H, D, device=DEV)
    t, s, f = (torch.zeros(*x, dtype=torch.int32, device=DEV) for x in ((1, 4), (2,), (1,)))
    none = (None, None, None)
    for call in (p.nvfp4_cache_write, p.nvfp4_cache_read):
        ok = lambda k=k, vx=None, kc=c.args(), vc=none, t=t, s=s, **kw: call(k, vx, *kc, *vc, t, s, **kw)
        ok(first=f)
        ok(vx=k.clone(), vc=v.args())
        for kw in (dict(k=k.cpu()), dict(k=k[0]), dict(k=k[:, :1]), dict(k=torch.zeros(3, D, H, device=DEV).transpose(1, 2)), dict(vx=k),
                   dict(vc=v.args()), dict(vx=k[:2], vc=v.args()), dict(kc=(c.q, n.s, c.amax)), dict(kc=(c.q[:3], None, c.amax)),
                   dict(kc=(c.q, None, c.amax.view(-1))), dict(kc=(n.q, None, n.amax)), dict(t=t[0]), dict(t=t.cpu()), dict(s=s[:1]),
                   dict(first=torch.zeros(2, dtype=torch.int32, device=DEV)), dict(vx=k, vc=(v.q, None, None))):
            with pytest.raises(ValueError):
                ok(**kw)
        for kw in (dict(k=k.half()), dict(kc=(c.q.short(), None, c.amax)), dict(t=t.long()), dict(s=s.long()), dict(k=None),
                   dict(kc=(c.q, None, c.amax.double())), dict(vx=k.bfloat16(), vc=v.args()), dict(vx=k, vc=n.args())):
            with pytest.raises((TypeError, ValueError)):
                ok(**kw)
        with pytest.raises(p.Nvfp4Error):
            ok(kc=n.args(), bound=0.0)
    with pytest.raises(p.Nvfp4Error):   # rows that overlap would be written twice
        p.nvfp4_cache_read(torch.zeros(1, H, D, device=DEV).expand(3, H, D), None, *c.args(), *none, t, s)
    p.nvfp4_cache_write(torch.zeros(1, H, D, device=DEV).expand(3, H, D), None, *c.args(), *none, t, s)
