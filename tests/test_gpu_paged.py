"""The paged cache on the GPU against the float64 oracle: writing and reading
back (bit for bit), attention of chunks and of single tokens.

Attention tolerances, from the arithmetic (eps of a rounding = half a step):
  dz = scale * max_t sum_d |q_d k_d| * 32 * 2^-23: a score's 128 products in
       16-long tensor-core steps, each adding at most a few units of the last
       place of the partial sum, and the scaling and exp2 conversions;
  a weight is off by a factor of at most exp(2 dz), and is represented to
  2^-16 (fp32 outputs) or 2^-8 (bf16 outputs); the sum over N tokens adds N / 16
  + 64 steps of 2^-23 each; outputs are sums of weights times values, so
  err(out) <= max |v| * (2 dz + w + (N / 16 + 64) * 2^-23) + r * |out|
       with w = 2^-16, r = 2^-24 (fp32) or w = 2^-8, r = 2^-8 (bf16);
  err(lse) <= 2 dz + 2^-16 + (N / 16 + 64) * 2^-23 + 2^-23 |lse|.
"""
import math

import numpy as np
import pytest
import torch

import oracle.paged_oracle as PO

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def sa():
    import block_sparse_kv_page_b200
    return block_sparse_kv_page_b200


class Case:
    """A paged cache with random contents, its host copies and the calls'
    arguments.  lens: tokens per sequence; rows: new rows per sequence."""

    def __init__(self, sa, dev, *, lens, rows, hq, hkv, page, cache="bf16", order="head", out="fp32", seed=0, spare=3,
                 gaps=0, extra_pages=0, stale=None, q_pad=0):
        self.sa, self.lens, self.rows, self.hq, self.hkv, self.page = sa, lens, rows, hq, hkv, page
        self.e4m3 = cache == "e4m3"
        g = torch.Generator(device="cpu").manual_seed(seed)
        B = len(lens)
        per = [-(-n // page) for n in lens]
        self.max_pages = max(1, max(per)) + extra_pages
        n_pages = sum(per) + spare
        perm = torch.randperm(n_pages, generator=g).tolist()
        table = torch.full((B, self.max_pages), -7, dtype=torch.int32)  # entries past the sequence: never looked at
        at = 0
        for b in range(B):
            table[b, :per[b]] = torch.tensor(perm[at: at + per[b]], dtype=torch.int32)
            at += per[b]
        self.table = table

        def pool(scale):
            x = (torch.randn((n_pages, hkv, page, D), generator=g) * scale).to(torch.bfloat16)
            return x
        k, v = pool(torch.exp(torch.empty(1, hkv, 1, D).uniform_(-0.7, 1.4, generator=g))), pool(1.0)
        self.ks = self.vs = None
        if self.e4m3:
            self.ks = torch.randint(118, 128, (n_pages, hkv, page), generator=g, dtype=torch.uint8)
            self.vs = torch.randint(118, 128, (n_pages, hkv, page), generator=g, dtype=torch.uint8)
            k, v = ((x * 40).float().clamp(-448, 448).to(torch.float8_e4m3fn) for x in (k, v))
        if stale is not None:  # every slot past a sequence's end, and every spare page, holds NaN
            live = torch.zeros((n_pages, page), dtype=torch.bool)
            for b in range(B):
                for t in range(lens[b]):
                    live[table[b, t // page], t % page] = True
            for x in (k, v):
                bits = x.view(torch.int16 if not self.e4m3 else torch.uint8)
                bits[~live[:, None, :].expand(-1, hkv, -1)] = 0x7f if self.e4m3 else stale
        self.k, self.v = k, v
        dv = {"head": lambda x: x.to(dev),
              "token": lambda x: x.transpose(1, 2).contiguous().to(dev).transpose(1, 2),
              "part": lambda x: torch.stack([x.view(torch.uint8)] * 3, 3).to(dev).view(x.dtype)[:, :, :, 1]}[order]
        self.dk, self.dv = dv(k), dv(v)
        self.dks, self.dvs = (None, None) if not self.e4m3 else (self.ks.to(dev), self.vs.to(dev))
        off, r = [], gaps
        for m in rows:
            off.append(r)
            r += m
        off.append(r)
        self.off, self.n_rows = off, r + gaps
        self.row_off = torch.tensor(off, dtype=torch.int32, device=dev)
        self.cache = sa.PagedCache(self.dk, self.dv, table.to(dev),
                                   torch.tensor(lens, dtype=torch.int32, device=dev),
                                   k_scale=self.dks, v_scale=self.dvs)
        self.ws = sa.make_paged_workspace(self.cache, hq)
        self.q = torch.randn((self.n_rows, hq + q_pad, D), generator=g).to(torch.bfloat16)
        self.dq = self.q.to(dev)[:, :hq]
        self.q = self.q[:, :hq]
        self.out_dtype = torch.bfloat16 if out == "bf16" else torch.float32
        self.dev = dev

    def held(self, b, h):
        """fp64 K, V [N][D] of sequence b, head h, and which tokens' pages are good."""
        N = self.lens[b]
        t = np.arange(N)
        pages = self.table[b].numpy()[t // self.page] if N else np.zeros(0, np.int64)
        ok = (pages >= 0) & (pages < self.k.shape[0])
        pg, sl = np.where(ok, pages, 0), t % self.page
        out = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            rows = x[pg, h, sl].float().numpy().astype(np.float64)
            if self.e4m3:
                rows = rows * 2.0 ** (s[pg, h, sl].numpy().astype(np.float64) - 127)[:, None]
            out.append(rows)
        return out[0], out[1], ok

    def run(self, window=0, sinks=0, scale=1 / math.sqrt(D), decode=False, lse=True, stream=None):
        out = torch.full((self.n_rows, self.hq, D), 7.0, dtype=self.out_dtype, device=self.dev)
        ls = torch.full((self.n_rows, self.hq), 7.0, dtype=torch.float32, device=self.dev) if lse else None
        if decode:
            self.sa.sparse_attn_paged_decode(self.cache, self.dq, scale, window, sinks, out, ls, self.ws, stream)
        else:
            self.sa.sparse_attn_chunk(self.cache, self.dq, self.row_off, scale, window, sinks, out, ls, self.ws, stream)
        torch.cuda.synchronize()
        return out, ls

    def check(self, got, window=0, sinks=0, scale=1 / math.sqrt(D)):
        out, ls = got
        o = out.float().cpu().numpy().astype(np.float64)
        bf = self.out_dtype == torch.bfloat16
        l = ls.cpu().numpy().astype(np.float64) if ls is not None else None
        owned = np.zeros(self.n_rows, bool)
        G = self.hq // self.hkv
        for b, (N, m) in enumerate(zip(self.lens, self.rows)):
            if not m:
                continue
            r0 = self.off[b]
            owned[r0:r0 + m] = True
            for h in range(self.hkv):
                k, v, ok = self.held(b, h)
                q = self.q[r0:r0 + m, h * G:(h + 1) * G].float().numpy().astype(np.float64)
                want, wl = PO.attend_rows(q, k, v, np.arange(N - m, N), ok, window, sinks, scale)
                vmax = np.abs(v[ok]).max() if ok.any() else 0.0
                dz = abs(scale) * (np.abs(q) @ np.abs(k[ok]).T).max() * 32 * 2.0 ** -23 if ok.any() else 0.0
                steps = (N / 16 + 64) * 2.0 ** -23
                tol = vmax * (2 * dz + (2.0 ** -8 if bf else 2.0 ** -16) + steps) \
                    + (2.0 ** -8 if bf else 2.0 ** -24) * np.abs(want)
                err = np.abs(o[r0:r0 + m, h * G:(h + 1) * G] - want)
                assert (err <= tol).all(), (b, h, float((err - tol).max()), np.argwhere(err > tol)[:3].tolist())
                if l is not None:
                    gl = l[r0:r0 + m, h * G:(h + 1) * G]
                    none = np.isinf(wl)
                    assert np.array_equal(np.isneginf(gl), none), (b, h)
                    wf = np.where(none, 0, wl)
                    assert (np.abs(np.where(none, 0, gl) - wf) <= 2 * dz + 2.0 ** -16 + steps
                            + 2.0 ** -23 * np.abs(wf)).all(), (b, h)
                seen_none = np.isinf(wl)
                assert (o[r0:r0 + m, h * G:(h + 1) * G][seen_none] == 0).all()
        assert (o[~owned] == 7.0).all(), "rows of no sequence were written"
        if l is not None:
            assert (l[~owned] == 7.0).all()

    def status(self):
        return self.sa.sparse_attn_get_device_status(self.ws)


# ---------------------------------------------------------------- write and read back
@pytest.mark.parametrize("order", ["head", "token", "part"])
@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_write_then_read_back(cuda_dev, sa, cache, page, order):
    lens, rows = [300, 1, 17, 0, 64, 256], [300, 1, 5, 0, 0, 255]
    c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=4, hkv=2, page=page, cache=cache, order=order, seed=11, gaps=2)
    g = torch.Generator().manual_seed(12)
    x = torch.randn((c.n_rows, 7, D), generator=g)
    x *= 10.0 ** torch.randint(-30, 30, (c.n_rows, 7, 1), generator=g)
    x[3, 2] = 0
    x[4, 2, 5:] = 0
    x[5, 3] = 2.0 ** -133
    x[6, 4] = torch.tensor(3.0e38)
    x[7, 2, :] = 448.0
    x[8, 2, :] = 450.0
    x = x.to(torch.bfloat16)
    dx = x.to(cuda_dev)
    sa.sparse_attn_cache_write(c.cache, dx[:, 2:4], dx[:, 4:6], c.row_off, c.ws)
    torch.cuda.synchronize()
    assert c.status() == sa.SA_OK
    for name, part, dt, ds in (("k", 2, c.dk, c.dks), ("v", 4, c.dv, c.dvs)):
        want = getattr(c, name).clone()
        wbits = want.view(torch.uint8 if c.e4m3 else torch.int16)
        wscale = None if not c.e4m3 else getattr(c, name + "s").clone()
        for b, (N, m) in enumerate(zip(lens, rows)):
            for i in range(m):
                t = N - m + i
                pg, sl = int(c.table[b, t // page]), t % page
                for h in range(2):
                    row = x[c.off[b] + i, part + h]
                    if c.e4m3:
                        code, e = PO.quantise_row(row.double().numpy())
                        wbits[pg, h, sl] = torch.from_numpy(code)
                        wscale[pg, h, sl] = e
                    else:
                        want[pg, h, sl] = row
        got = dt.cpu()
        assert torch.equal(got.view(torch.uint8 if c.e4m3 else torch.int16), wbits), name
        if c.e4m3:
            assert torch.equal(ds.cpu(), wscale), name
        setattr(c, name, want)
        if c.e4m3:
            setattr(c, name + "s", wscale)
    # read back into a contiguous cache: everything, and the last tokens only
    for first in (0, 40, -3, 1 << 20):
        for cap in (c.max_pages * page, c.max_pages * page + 24, 310):
            ko = torch.full((len(lens), 2, cap, D), 5.0, dtype=torch.bfloat16, device=cuda_dev)
            vo = torch.full_like(ko, 6.0)
            sa.sparse_attn_cache_read(c.cache, first, ko, vo, c.ws)
            torch.cuda.synchronize()
            assert c.status() == sa.SA_OK
            for out, fill, which in ((ko, 5.0, 0), (vo, 6.0, 1)):
                want = torch.full(out.shape, fill, dtype=torch.bfloat16)
                for b, N in enumerate(lens):
                    t0 = first if first >= 0 else max(0, N + first)
                    for h in range(2):
                        rows_ = torch.from_numpy(c.held(b, h)[which]).to(torch.bfloat16)
                        want[b, h, min(t0, N):N] = rows_[min(t0, N):]
                assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16)), (first, cap)


def test_every_bf16_row_quantises_as_defined(cuda_dev, sa):
    """Rows that hold every finite bf16 value once."""
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x.float())]
    x = torch.cat([x, x[torch.randperm(x.numel(), generator=torch.Generator().manual_seed(1))]])
    x = x[: x.numel() // 256 * 256].reshape(-1, 2, D)
    n = x.shape[0]
    c = Case(sa, cuda_dev, lens=[n], rows=[n], hq=2, hkv=2, page=16, cache="e4m3", seed=3)
    dx = x.to(cuda_dev)
    sa.sparse_attn_cache_write(c.cache, dx, dx, c.row_off, None)
    torch.cuda.synchronize()
    held = [(c.dk.cpu().view(torch.uint8), c.dks.cpu()), (c.dv.cpu().view(torch.uint8), c.dvs.cpu())]
    for t in range(n):
        pg, sl = int(c.table[0, t // 16]), t % 16
        for h in range(2):
            code, e = PO.quantise_row(x[t, h].double().numpy())
            for got, sc in held:
                assert np.array_equal(got[pg, h, sl].numpy(), code) and int(sc[pg, h, sl]) == e, (t, h)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_write_and_read_skip_what_is_bad(cuda_dev, sa, cache):
    """A page out of range, a length the table cannot hold, more rows than
    tokens, a row range past the arrays: flagged and skipped, the rest done."""
    def fresh(**kw):
        c = Case(sa, cuda_dev, lens=[40, 33, 20], rows=[8, 4, 20], hq=2, hkv=2, page=16, cache=cache, seed=21, spare=4)
        return c
    x = torch.randn(32, 2, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(cuda_dev)
    ref = fresh()
    sa.sparse_attn_cache_write(ref.cache, x, x, ref.row_off, ref.ws)
    bits = lambda t: t.cpu().view(torch.uint8)  # noqa: E731

    def pages_of(c, b):
        return [int(p) for p in c.table[b] if p >= 0]
    for bad in ("page", "length", "rows", "range"):
        c = fresh()
        before = bits(c.dk).clone()
        off = c.row_off.clone()
        if bad == "page":
            c.cache.page_table[0, 2] = c.k.shape[0]
        elif bad == "length":
            c.cache.seq_len[0] = c.max_pages * 16 + 1
        elif bad == "rows":
            c.cache.seq_len[0] = 5
        else:
            off[3] = 33
        sa.sparse_attn_cache_write(c.cache, x, x, off, c.ws)
        torch.cuda.synchronize()
        assert c.status() == sa.SA_ERR_DEVICE_CHECK, bad
        got, want = bits(c.dk), bits(ref.dk)
        lost = 2 if bad == "range" else 0
        for b in range(3):
            for p in pages_of(c, b):
                if b == lost and bad == "rows" and p == pages_of(c, 0)[0]:
                    continue  # its last five rows land on tokens 0 .. 4
                assert torch.equal(got[p], before[p] if b == lost else want[p]), (bad, b, p)
        if bad == "rows":  # rows 3 .. 7 are tokens 0 .. 4; the first three have no place
            p = pages_of(c, 0)[0]
            assert torch.equal(got[p][:, 5:], before[p][:, 5:])
            assert not torch.equal(got[p][:, :5], before[p][:, :5])
        ko = torch.full((3, 2, 48, D), 9.0, dtype=torch.bfloat16, device=cuda_dev)
        vo = ko.clone()
        sa.sparse_attn_cache_read(c.cache, 0, ko, vo, c.ws)
        torch.cuda.synchronize()
        assert c.status() == (sa.SA_ERR_DEVICE_CHECK if bad in ("page", "length") else sa.SA_OK), bad
        if bad == "page":
            assert (ko[0, :, 32:] == 9.0).all() and (ko[0, :, :32] != 9.0).any()
        if bad == "length":
            assert (ko[0] == 9.0).all()
    c = fresh()  # a contiguous cache shorter than the sequences
    ko = torch.full((3, 2, 24, D), 9.0, dtype=torch.bfloat16, device=cuda_dev)
    sa.sparse_attn_cache_read(c.cache, 0, ko, ko.clone(), c.ws)
    torch.cuda.synchronize()
    assert c.status() == sa.SA_ERR_DEVICE_CHECK
    assert torch.equal(ko[2, 0, :20].double().cpu(), torch.from_numpy(c.held(2, 0)[0]))
    assert torch.equal(ko[0, 0].double().cpu(), torch.from_numpy(c.held(0, 0)[0][:24]))


# ---------------------------------------------------------------- attention
HEADS = [(8, 1), (14, 2), (4, 4), (6, 2)]
MASKS = [(0, 0), (1, 0), (16, 4), (100, 17), (130, 500), (5000, 3)]


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", MASKS)
def test_chunk_masks(cuda_dev, sa, cache, out, window, sinks):
    c = Case(sa, cuda_dev, lens=[700, 1, 16, 129, 0, 400], rows=[70, 1, 16, 2, 0, 400], hq=8, hkv=2, page=16,
             cache=cache, out=out, seed=31, gaps=3, stale=0x7fc0)
    got = c.run(window, sinks)
    assert c.status() == sa.SA_OK
    c.check(got, window, sinks)


@pytest.mark.parametrize("order", ["head", "token", "part"])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 256, 80])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_chunk_pages(cuda_dev, sa, cache, page, order):
    c = Case(sa, cuda_dev, lens=[517, 33, 256], rows=[40, 33, 100], hq=6, hkv=2, page=page, cache=cache, out="bf16",
             order=order, seed=41, stale=0x7f80, q_pad=4, extra_pages=2)
    c.check(c.run(0, 0), 0, 0)
    c.check(c.run(150, 20), 150, 20)
    assert c.status() == sa.SA_OK


@pytest.mark.parametrize("hq,hkv", HEADS + [(5, 1), (21, 3)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_chunk_heads_and_row_counts(cuda_dev, sa, hq, hkv, out):
    """Row counts around a tile of query vectors, contexts around a block."""
    c = Case(sa, cuda_dev, lens=[255, 256, 257, 1100, 64, 65], rows=[31, 32, 33, 257, 64, 1], hq=hq, hkv=hkv, page=16,
             cache="e4m3", out=out, seed=51)
    c.check(c.run(), 0, 0)
    c.check(c.run(33, 2), 33, 2)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", MASKS)
def test_decode_masks(cuda_dev, sa, cache, out, window, sinks):
    lens = [700, 1, 16, 129, 0, 2000, 15, 17, 128]
    c = Case(sa, cuda_dev, lens=lens, rows=[1] * len(lens), hq=8, hkv=2, page=16, cache=cache, out=out, seed=61,
             stale=0x7fc0)
    got = c.run(window, sinks, decode=True)
    assert c.status() == sa.SA_OK
    c.check(got, window, sinks)


@pytest.mark.parametrize("order", ["head", "token", "part"])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 256, 80])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_decode_pages(cuda_dev, sa, cache, page, order):
    c = Case(sa, cuda_dev, lens=[517, 33, 256], rows=[1] * 3, hq=6, hkv=2, page=page, cache=cache, order=order, seed=71,
             stale=0x7f80, q_pad=3, extra_pages=1)
    c.check(c.run(0, 0, decode=True), 0, 0)
    c.check(c.run(150, 20, decode=True), 150, 20)
    assert c.status() == sa.SA_OK


@pytest.mark.parametrize("hq,hkv", HEADS + [(5, 1), (21, 3)])
def test_decode_heads(cuda_dev, sa, hq, hkv):
    c = Case(sa, cuda_dev, lens=[300, 3000], rows=[1, 1], hq=hq, hkv=hkv, page=32, cache="e4m3", out="bf16", seed=81)
    c.check(c.run(decode=True))
    c.check(c.run(decode=True, lse=False))


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
@pytest.mark.parametrize("decode", [False, True])
def test_scales(cuda_dev, sa, scale, decode):
    rows = [1, 1] if decode else [20, 3]
    c = Case(sa, cuda_dev, lens=[150, 37], rows=rows, hq=4, hkv=2, page=16, cache="bf16", seed=91)
    c.check(c.run(decode=decode, scale=scale), scale=scale)
    c.check(c.run(20, 3, decode=decode, scale=scale), 20, 3, scale=scale)


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_bad_pages_and_lengths_are_skipped(cuda_dev, sa, cache, decode):
    rows = [1, 1, 1, 1] if decode else [50, 7, 3, 4]
    c = Case(sa, cuda_dev, lens=[300, 40, 20, 64], rows=rows, hq=4, hkv=2, page=16, cache=cache, seed=101, spare=6)
    for b, p, bad in ((0, 2, -1), (0, 5, c.k.shape[0]), (0, 6, 2 ** 31 - 1), (1, 0, -2 ** 31), (2, 0, -5), (2, 1, -5)):
        c.table[b, p] = bad
        c.cache.page_table[b, p] = bad
    c.cache.seq_len[3] = c.max_pages * 16 + 1  # no such length: counts as empty
    c.lens[3] = 0
    got = c.run(decode=decode)
    assert c.status() == sa.SA_ERR_DEVICE_CHECK
    # sequence 3 sees nothing; check() places its rows before token 0
    c.check(got)
    # pages that a window has passed are not looked at
    c2 = Case(sa, cuda_dev, lens=[400], rows=[1] if decode else [20], hq=4, hkv=2, page=16, cache=cache, seed=102)
    c2.table[0, 1:18] = -1
    c2.cache.page_table[0, 1:18] = -1
    got = c2.run(64, 5, decode=decode)
    assert c2.status() == sa.SA_OK
    c2.check(got, 64, 5)


def test_more_rows_than_tokens(cuda_dev, sa):
    c = Case(sa, cuda_dev, lens=[5, 30], rows=[9, 30], hq=4, hkv=2, page=16, seed=111)
    got = c.run()
    assert c.status() == sa.SA_ERR_DEVICE_CHECK
    c.check(got)


def test_row_range_outside_the_arrays(cuda_dev, sa):
    c = Case(sa, cuda_dev, lens=[50, 30], rows=[9, 30], hq=4, hkv=2, page=16, seed=112)
    c.row_off[2] = 40
    got = c.run()
    assert c.status() == sa.SA_ERR_DEVICE_CHECK
    c.rows = [9, 0]
    c.check(got)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_large_scores_and_one_hot_rows(cuda_dev, sa, cache, out):
    """Scores of several hundred: the softmax is one token, in the first, a
    middle and the last block; running maxima that rise block after block."""
    c = Case(sa, cuda_dev, lens=[900, 900], rows=[24, 1], hq=4, hkv=1, page=16, cache=cache, out=out, seed=121)
    c.check(c.run(scale=2.0), scale=2.0)
    c.check(c.run(scale=20.0), scale=20.0)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("falling", [False, True])
def test_scores_that_rise_or_fall_along_the_context(cuda_dev, sa, cache, out, falling):
    """Keys that are a query times a factor growing (or shrinking) from token to
    token: the running reference has to follow, for some heads and not others."""
    for decode in (False, True):
        c = Case(sa, cuda_dev, lens=[800], rows=[1] if decode else [40], hq=8, hkv=2, page=16, cache=cache, out=out,
                 seed=125)
        q = c.q[0, ::4].float()                                    # one query head per KV head
        for t in range(800):
            f = (800 - t if falling else t) / 800.0 * 12.0
            for h in range(2):
                pg, sl = int(c.table[0, t // 16]), t % 16
                row = (q[h] * f).to(torch.bfloat16)
                if c.e4m3:
                    code, e = PO.quantise_row(row.double().numpy())
                    c.k.view(torch.uint8)[pg, h, sl] = torch.from_numpy(code)
                    c.ks[pg, h, sl] = e
                else:
                    c.k[pg, h, sl] = row
        c.dk.view(torch.uint8).copy_(c.k.view(torch.uint8))
        if c.e4m3:
            c.dks.copy_(c.ks)
        for scale in (0.09, 1.0, -0.5):
            c.check(c.run(decode=decode, scale=scale), scale=scale)
            c.check(c.run(300, 20, decode=decode, scale=scale), 300, 20, scale=scale)
        assert c.status() == sa.SA_OK


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("decode", [False, True])
def test_row_scales_far_apart(cuda_dev, sa, out, decode):
    """V rows of a cache in e4m3 whose scales differ by up to 2^60, K rows by 2^8."""
    c = Case(sa, cuda_dev, lens=[900, 70, 33], rows=[1, 1, 1] if decode else [30, 7, 33], hq=8, hkv=2, page=16,
             cache="e4m3", out=out, seed=126)
    g = torch.Generator().manual_seed(9)
    c.vs.copy_(torch.randint(90, 151, c.vs.shape, generator=g, dtype=torch.uint8))
    c.dvs.copy_(c.vs)
    c.check(c.run(decode=decode))
    c.check(c.run(50, 3, decode=decode), 50, 3)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("longest", [40, 9000])
def test_nan_queries_give_nan_and_leave_others_alone(cuda_dev, sa, cache, decode, longest):
    """A NaN in q makes its own row and head NaN, output and lse, whether the
    row lies in one part or in many; every other row is as it was."""
    lens = [longest, 33, longest // 2]
    rows = [1] * 3 if decode else [20, 3, 7]
    c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=8, hkv=2, page=16, cache=cache, seed=93)
    c.dq[1, 3, 5] = float("nan")
    c.dq[2, 7] = float("nan")
    out, lse = c.run(decode=decode)
    for r, h in ((1, 3), (2, 7)):
        assert torch.isnan(out[r, h]).all() and torch.isnan(lse[r, h])
    c.dq.copy_(c.q)
    want = c.run(decode=decode)
    for r, h in ((1, 3), (2, 7)):
        out[r, h], lse[r, h] = want[0][r, h], want[1][r, h]
    c.check(want)
    c.check((out, lse))


def test_nan_in_a_row_of_the_cache_reaches_the_rows_that_see_it(cuda_dev, sa):
    """bf16 cache: a NaN key makes the heads that share it NaN in the decode of
    its sequence, and leaves the other sequences and heads alone."""
    c = Case(sa, cuda_dev, lens=[5000, 70], rows=[1, 1], hq=8, hkv=2, page=16, cache="bf16", seed=94)
    want = c.run(decode=True)
    page, slot = int(c.table[0, 1234 // 16]), 1234 % 16
    c.dk[page, 1, slot, 9] = float("nan")
    out, lse = c.run(decode=True)
    assert torch.isnan(out[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.equal(out[0, :4], want[0][0, :4]) and torch.equal(out[1], want[0][1])
    assert torch.equal(lse[0, :4], want[1][0, :4]) and torch.equal(lse[1], want[1][1])


@pytest.mark.parametrize("power", [-112, -90, 90, 110])
@pytest.mark.parametrize("decode", [False, True])
def test_key_scales_near_the_ends_of_the_range(cuda_dev, sa, decode, power):
    """Ordinary scores from tiny queries and huge keys, and the other way round."""
    c = Case(sa, cuda_dev, lens=[700, 40], rows=[1, 1] if decode else [9, 2], hq=8, hkv=2, page=16, cache="e4m3",
             seed=97)
    # queries times 2^power (exact in bf16: normal powers), keys times 2^-power
    c.q = (c.q.float() * 2.0 ** power).to(torch.bfloat16)
    c.dq.copy_(c.q)
    c.ks = (c.ks.int() - power).to(torch.uint8)
    c.dks.copy_(c.ks)
    c.check(c.run(decode=decode))


def test_offsets_past_32_bits(cuda_dev, sa):
    """Pages 1.5 GiB apart: element and byte offsets pass 2^32."""
    far, n_pages = 3 << 29, 6
    buf = torch.zeros(far * (n_pages - 1) + 2 * 16 * D, dtype=torch.uint8, device=cuda_dev)
    x = buf.as_strided((n_pages, 2, 16, D), (far, 16 * D, D, 1)).view(torch.float8_e4m3fn)
    c = Case(sa, cuda_dev, lens=[90], rows=[30], hq=4, hkv=2, page=16, cache="e4m3", seed=131, spare=0)
    kk = x  # K and V share the far pool in turn
    kk.view(torch.uint8).copy_(c.k.view(torch.uint8))
    cache = sa.PagedCache(kk, kk, c.cache.page_table, c.cache.seq_len, k_scale=c.dks, v_scale=c.dks)
    c.cache, c.v, c.vs = cache, c.k, c.ks
    c.check(c.run())
    c.n_rows, c.rows, c.off = 1, [1], [0, 1]
    c.q, c.dq = c.q[:1], c.dq[:1]
    c.check(c.run(decode=True))
    ko = torch.zeros((1, 2, 96, D), dtype=torch.bfloat16, device=cuda_dev)
    vo = torch.zeros_like(ko)
    sa.sparse_attn_cache_read(cache, 0, ko, vo)
    new = torch.randn(30, 2, D).to(torch.bfloat16).to(cuda_dev)
    ref = Case(sa, cuda_dev, lens=[90], rows=[30], hq=4, hkv=2, page=16, cache="e4m3", seed=131, spare=0)
    sa.sparse_attn_cache_write(ref.cache, new, new, ref.row_off)
    sa.sparse_attn_cache_write(cache, new, new, ref.row_off)
    torch.cuda.synchronize()
    assert torch.equal(ko[0, 1, :90].cpu().double(), torch.from_numpy(c.held(0, 1)[0]))
    assert torch.equal(kk.cpu().view(torch.uint8), ref.dk.cpu().view(torch.uint8))


@pytest.mark.parametrize("decode", [False, True])
def test_captured_call_replays_with_other_lengths_on_another_stream(cuda_dev, sa, decode):
    rows = [1, 1, 1] if decode else [20, 5, 40]
    c = Case(sa, cuda_dev, lens=[600, 90, 333], rows=rows, hq=8, hkv=2, page=16, cache="e4m3", out="bf16", seed=141)
    out = torch.zeros((c.n_rows, 8, D), dtype=torch.bfloat16, device=cuda_dev)
    lse = torch.zeros((c.n_rows, 8), dtype=torch.float32, device=cuda_dev)

    def call():
        if decode:
            sa.sparse_attn_paged_decode(c.cache, c.dq, 0.1, 40, 3, out, lse, c.ws)
        else:
            sa.sparse_attn_chunk(c.cache, c.dq, c.row_off, 0.1, 40, 3, out, lse, c.ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, r in (([600, 90, 333], rows), ([41, 17, 40], rows), ([333, 0, 1], [1, 1, 1] if decode else [4, 0, 1])):
        c.lens, c.rows, off = lens, r, [0]
        for m in r:
            off.append(off[-1] + m)
        c.off = off
        # lengths above the first ones would need table entries that are not there
        c.cache.seq_len.copy_(torch.tensor([min(a, b) for a, b in zip(lens, [600, 90, 333])], dtype=torch.int32))
        c.row_off.copy_(torch.tensor(off, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert c.status() == sa.SA_OK
        c.check((out, lse), 40, 3, scale=0.1)


def test_two_streams_with_a_workspace_each(cuda_dev, sa):
    a = Case(sa, cuda_dev, lens=[3000, 900], rows=[60, 9], hq=8, hkv=2, page=16, cache="bf16", seed=151)
    b = Case(sa, cuda_dev, lens=[2000], rows=[1], hq=8, hkv=2, page=64, cache="e4m3", seed=152)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for c, s, dec in ((a, s1, False), (b, s2, True)):
            with torch.cuda.stream(s):
                o = torch.zeros((c.n_rows, 8, D), dtype=torch.float32, device=cuda_dev)
                l = torch.zeros((c.n_rows, 8), dtype=torch.float32, device=cuda_dev)
                if dec:
                    sa.sparse_attn_paged_decode(c.cache, c.dq, 0.1, 0, 0, o, l, c.ws)
                else:
                    sa.sparse_attn_chunk(c.cache, c.dq, c.row_off, 0.1, 0, 0, o, l, c.ws)
                outs.append((c, o, l))
    torch.cuda.synchronize()
    firsts = {}
    for c, o, l in outs:
        f = firsts.setdefault(id(c), (o, l))
        assert torch.equal(o, f[0]) and torch.equal(l, f[1])
        if f[0] is o:
            c.check((o, l), scale=0.1)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_long_context_repeats_bit_for_bit(cuda_dev, sa, cache):
    """A context long enough to be split many ways, for a chunk and a token."""
    c = Case(sa, cuda_dev, lens=[20000], rows=[5], hq=8, hkv=2, page=64, cache=cache, seed=161)
    first = c.run()
    c.check(first)
    for _ in range(3):
        again = c.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    d = Case(sa, cuda_dev, lens=[20000, 3], rows=[1, 1], hq=8, hkv=2, page=64, cache=cache, seed=162)
    first = d.run(decode=True)
    d.check(first)
    for _ in range(3):
        again = d.run(decode=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_many_sequences(cuda_dev, sa):
    rng = np.random.default_rng(7)
    lens = [int(x) for x in rng.integers(0, 60, 700)]
    c = Case(sa, cuda_dev, lens=lens, rows=[1] * 700, hq=2, hkv=1, page=16, cache="e4m3", seed=171)
    c.check(c.run(decode=True))
    rows = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 9, 700))]
    c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=2, hkv=1, page=16, cache="bf16", out="bf16", seed=172)
    c.check(c.run())


@pytest.mark.parametrize("B", [31, 32, 33, 127, 128, 129, 640, 641, 897])
def test_sequence_counts_around_a_warp_and_a_block(cuda_dev, sa, B):
    """Where the plan of the work changes hands: a warp, a block, several rounds."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 40, B)]
    lens[B // 2], lens[B - 1] = 900, 33
    c = Case(sa, cuda_dev, lens=lens, rows=[1] * B, hq=2, hkv=1, page=16, cache="bf16", seed=B)
    c.check(c.run(decode=True))
    rows = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 5, B))]
    for cache in ("bf16", "e4m3") if B < 600 or B == 897 else ("bf16",):
        c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=2, hkv=1, page=16, cache=cache, seed=B)
        c.check(c.run())


def test_long_chunks_of_many_tiles(cuda_dev, sa):
    """More pairs of tiles than a warp has lanes, in the first and the last sequence."""
    c = Case(sa, cuda_dev, lens=[1150, 40, 1300], rows=[1150, 0, 1090], hq=8, hkv=1, page=32, out="bf16", seed=181)
    c.check(c.run(100, 3), 100, 3)


# ---------------------------------------------------------------- as a run
@pytest.mark.parametrize("window,sinks", [(0, 0), (96, 4)])
def test_prompt_then_tokens_as_they_are_served(cuda_dev, sa, window, sinks):
    """A prompt in two chunks, then tokens one by one: each step writes its
    rows, attends, and the whole agrees with the oracle on the values held;
    the cache read back serves the framework's own decode over all pages."""
    hq, hkv, page, total = 8, 2, 16, 230
    steps = [100, 121, 1, 1, 1, 1, 1, 1, 1, 1, 1]
    assert sum(steps) == total
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(total, hq + 2 * hkv, D, generator=g).to(torch.bfloat16)
    n_pages = -(-total // page)
    dev = cuda_dev
    table = torch.randperm(n_pages, generator=g).to(torch.int32)[None].to(dev)
    k = torch.zeros((n_pages, hkv, page, D), device=dev).to(torch.float8_e4m3fn)
    v = torch.zeros_like(k)
    ks = torch.zeros((n_pages, hkv, page), dtype=torch.uint8, device=dev)
    vs = torch.zeros_like(ks)
    seq = torch.zeros(1, dtype=torch.int32, device=dev)
    cache = sa.PagedCache(k, v, table, seq, k_scale=ks, v_scale=vs)
    ws = sa.make_paged_workspace(cache, hq)
    scale = 1 / math.sqrt(D)
    deq = np.zeros((2, hkv, total, D))
    for t in range(total):
        for h in range(hkv):
            for i in range(2):
                deq[i, h, t] = PO.dequantise_row(*PO.quantise_row(qkv[t, hq + i * hkv + h].double().numpy()))
    done = 0
    for m in steps:
        x = qkv[done:done + m].to(dev)
        off = torch.tensor([0, m], dtype=torch.int32, device=dev)
        done += m
        seq.fill_(done)
        sa.sparse_attn_cache_write(cache, x[:, hq:hq + hkv], x[:, hq + hkv:], off, ws)
        out = torch.empty((m, hq, D), dtype=torch.float32, device=dev)
        if m == 1:
            sa.sparse_attn_paged_decode(cache, x[:, :hq], scale, window, sinks, out, None, ws)
        else:
            sa.sparse_attn_chunk(cache, x[:, :hq], off, scale, window, sinks, out, None, ws)
        for h in range(hkv):
            G = hq // hkv
            q = x[:, h * G:(h + 1) * G].float().cpu().numpy().astype(np.float64)
            want, _ = PO.attend_rows(q, deq[0, h, :done], deq[1, h, :done], np.arange(done - m, done),
                                     np.ones(done, bool), window, sinks, scale)
            dz = scale * (np.abs(q) @ np.abs(deq[0, h, :done]).T).max() * 32 * 2.0 ** -23
            tol = np.abs(deq[1, h, :done]).max() * (2 * dz + 2.0 ** -16 + (done / 16 + 64) * 2.0 ** -23)
            assert np.abs(out[:, h * G:(h + 1) * G].cpu().numpy() - want).max() <= tol
    assert sa.sparse_attn_get_device_status(ws) == sa.SA_OK
    if window:
        return
    cap = n_pages * page
    ko = torch.zeros((1, hkv, cap, D), dtype=torch.bfloat16, device=dev)
    vo = torch.zeros_like(ko)
    sa.sparse_attn_cache_read(cache, 0, ko, vo, ws)
    kv = sa.KvCache(ko, vo, seq, page_size=page, max_pages=n_pages)
    meta = kv.meta_buffer()
    ws2 = sa.make_workspace(kv, hq, 1, n_pages)
    sel = torch.empty((1, hkv, n_pages), dtype=torch.int32, device=dev)
    cnt = torch.empty((1, hkv), dtype=torch.int32, device=dev)
    dense = torch.empty((1, hq, D), dtype=torch.float32, device=dev)
    q = qkv[-1:, :hq].contiguous().to(dev)
    sa.sparse_attn_build_meta(kv, "envelope", 0, meta)
    sa.sparse_attn_select(kv, meta, "envelope", q, sa.budget_topk(n_pages), n_pages, sel, cnt, None, ws2)
    sa.sparse_attn_decode(kv, q, 1, 0, 1, scale, sel, cnt, n_pages, dense, None, ws2)
    torch.cuda.synchronize()
    # the same tokens through the framework's page list: both within the tolerance of the oracle's value
    assert float((dense[0] - out[0]).abs().max()) <= 2 * float(tol)
