"""The paged cache where numbers go to their limits: weights far below the
largest one, against the float64 oracle and relative to the row's own size.

Tolerances, from the arithmetic.  An output is sum p_t v_t, so a relative error
w of every weight moves it by at most w * sum p_t |v_t|:
  w: a weight's representation - one f16 or bf16 term for bf16 outputs (2^-11,
     2^-8), two f16 terms that hold 2^-19 or three bf16 terms for fp32 outputs;
  dz: the exponent z * log2(e) takes four roundings (log2(e), its product with
     scale, the score, the difference to the maximum), each 2^-24 of |z| log2(e),
     once for a weight and once for the sum; exp2 itself 2^-22;
  steps: (N / 16 + 64) partial sums of 2^-23 each, as the products add up;
  floor: weights are held relative to a reference that is at most the row's
      maximum, and a weight there, or the factor exp2(old - new reference) that
      later takes it to a higher one, is zero under 2^-126, fp32's smallest normal
      number.  A chunk keeps its reference while a half block's weights sum to at
      most 2^20, so what such a factor drops lies below 2^20 * 2^-126 = 2^-106 of
      the row's largest weight.  The sum that weights are divided by is at least
      1, so N of them move the output by at most N * 2^-106 * max |v|;
and the output is rounded once: 2^-8 of it (bf16) or 2^-24 (fp32).
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.paged_oracle as PO
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu

D = 128
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sa():
    import block_sparse_kv_page_b200
    return block_sparse_kv_page_b200


def upload(c):
    """The host copies of a case to its cache and queries."""
    for host, held in ((c.k, c.dk), (c.v, c.dv)):
        held.view(torch.uint8).copy_(host.view(torch.uint8))
    if c.e4m3:
        c.dks.copy_(c.ks)
        c.dvs.copy_(c.vs)
    c.dq.copy_(c.q)


def check_rows(c, got, scale, zmax, decode, window=0, sinks=0):
    """Against the oracle, relative to sum p |v|; zmax: the largest |z| in log2
    units, of scores that are one product each; None: of scores of 128 products,
    dz = scale * max sum |q_d k_d| * 32 * 2^-23 for their sums and exponents."""
    out, ls = got
    bf = c.out_dtype == torch.bfloat16
    G = c.hq // c.hkv
    for b, (N, m) in enumerate(zip(c.lens, c.rows)):
        if not m:
            continue
        r0 = c.off[b]
        for h in range(c.hkv):
            k, v, ok = c.held(b, h)
            q = c.q[r0:r0 + m, h * G:(h + 1) * G].double().numpy()
            pos = np.arange(N - m, N)
            want, wl = PO.attend_rows(q, k, v, pos, ok, window, sinks, scale)
            size, _ = PO.attend_rows(q, k, np.abs(v), pos, ok, window, sinks, scale)
            w = (2.0 ** -11 if decode and c.e4m3 else 2.0 ** -8) if bf else 2.0 ** -19
            if zmax is None:
                dz = abs(scale) * (np.abs(q) @ np.abs(k).T).max() * 32 * 2.0 ** -23 + 2.0 ** -22 if N else 0.0
            else:
                dz = 4 * zmax * 2.0 ** -24 + 2.0 ** -22
            steps = (N / 16 + 64) * 2.0 ** -23
            tol = (w + 2 * dz + steps) * size + (2.0 ** -8 if bf else 2.0 ** -24) * np.abs(want)
            tol += N * 2.0 ** -106 * (np.abs(v).max() if N else 0.0)
            o = out[r0:r0 + m, h * G:(h + 1) * G].double().cpu().numpy()
            err = np.abs(o - want)
            assert (err <= tol).all(), (b, h, float((err / np.maximum(size, 1e-300)).max()),
                                        np.argwhere(~(err <= tol))[:3].tolist())
            gl = ls[r0:r0 + m, h * G:(h + 1) * G].double().cpu().numpy()
            none = np.isinf(wl)
            assert np.array_equal(np.isneginf(gl), none)
            el, wl = np.abs(np.where(none, 0, gl) - np.where(none, 0, wl)), np.where(none, 0, wl)
            assert (el <= 2 * dz + steps + 2.0 ** -23 * np.abs(wl)).all(), (b, h, float(el.max()))


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("cache,spread", [("bf16", 0), ("e4m3", 0), ("e4m3", 8)])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("N,at", [(40, 5), (300, 299), (32768, 20000)])
def test_one_dominant_token_without_a_value(cuda_dev, sa, cache, out, decode, spread, N, at):
    """One token has all but 2^-gap of the weight and a value of zero, as
    attention sinks have: the output is what the others give, each of them gap
    bits below the largest weight.  spread: every other V row is held with a
    scale that many places smaller."""
    c = Case(sa, cuda_dev, lens=[N], rows=[1], hq=8, hkv=2, page=16, cache=cache, out=out, seed=201)
    c.q.zero_()
    c.q[:, :, 3] = 1
    page, slot = int(c.table[0, at // 16]), at % 16
    k, v = torch.zeros_like(c.k.float()), c.v.float().abs().clamp(min=2.0 ** -5)
    k[page, :, slot, 3] = 1
    v[page, :, slot] = 0
    c.k, c.v = k.to(c.k.dtype), v.to(c.v.dtype)
    if c.e4m3:
        c.ks.fill_(127)
        c.vs.fill_(127)
        c.vs[:, :, 1::2] -= spread
    upload(c)
    for gap in (12, 20, 24.5, 28, 33.25, 60):
        scale = float(np.float32(gap * math.log(2)))
        check_rows(c, c.run(decode=decode, scale=scale), scale, gap, decode)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("louder", [10, 16, 40])
def test_a_loud_value_that_is_hardly_seen(cuda_dev, sa, out, decode, louder):
    """One V row whose scale is 2^louder times the others' and whose weight is
    2^-60 of theirs."""
    c = Case(sa, cuda_dev, lens=[700], rows=[1], hq=8, hkv=2, page=16, cache="e4m3", out=out, seed=202)
    c.q.zero_()
    c.q[:, :, 3] = 1
    k, v = torch.zeros_like(c.k.float()), c.v.float().abs().clamp(min=2.0 ** -5)
    page, slot = int(c.table[0, 2]), 7
    k[page, :, slot, 3] = -1
    c.k, c.v = k.to(c.k.dtype), v.to(c.v.dtype)
    c.ks.fill_(127)
    c.vs.fill_(120)
    c.vs[page, :, slot] += louder
    upload(c)
    scale = float(np.float32(60 * math.log(2)))
    check_rows(c, c.run(decode=decode, scale=scale), scale, 60, decode)


# Powers of two of the queries, of the keys and of the scale; the scores are
# those of (0, 0, 0): huge queries and tiny keys, the other way round, a huge
# and a tiny scale.  (Sums of query times key stay within fp32 in all of them.)
POWERS = [(112, -124, 12), (122, -124, 2), (-100, 110, -10), (-124, 117, 7), (0, -124, 124), (-20, -100, 120),
          (60, 50, -110), (0, 112, -112), (0, 0, 0)]


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("q_power,k_power,s_power", POWERS)
def test_ordinary_scores_from_factors_far_apart(cuda_dev, sa, out, decode, q_power, k_power, s_power):
    """Query, key scale and scale of the scores at the ends of their range,
    where partial products in another order pass what fp32 holds; scores to
    about 40."""
    c = Case(sa, cuda_dev, lens=[700, 40], rows=[1, 1] if decode else [9, 2], hq=8, hkv=2, page=16, cache="e4m3",
             out=out, seed=203)
    g = torch.Generator().manual_seed(1)
    c.q = (c.q.float().abs().clamp(0.25, 1.75) * 2.0 ** q_power).to(torch.bfloat16)
    sign = torch.where(torch.rand((*c.k.shape[:3], 1), generator=g) < 0.5, -1.0, 1.0)
    c.k = (c.k.float().abs() * sign).to(c.k.dtype)   # (a token's products have one sign)
    c.ks.copy_(torch.randint(127, 130, c.ks.shape, generator=g) + k_power)
    upload(c)
    scale = 0.003 * 2.0 ** s_power
    scale = float(np.float32(scale))
    c.check(c.run(decode=decode, scale=scale), scale=scale)
    c.check(c.run(30, 3, decode=decode, scale=scale), 30, 3, scale=scale)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("power", [20, 31, 45, 127, -100])
def test_one_query_dim_far_above_the_others(cuda_dev, sa, out, decode, power):
    """One dim of some heads' queries is 2^power (or all others 2^power), where
    the keys are zero: the other dims make the scores."""
    c = Case(sa, cuda_dev, lens=[700, 40], rows=[1, 1] if decode else [9, 2], hq=8, hkv=2, page=16, cache="e4m3",
             out=out, seed=204)
    scale = 1 / math.sqrt(D)
    c.q[:, ::3, 77] = 2.0 ** max(power, 0)
    if power < 0:
        c.q = torch.where(torch.arange(D) == 77, c.q.float(), c.q.float() * 2.0 ** power).to(torch.bfloat16)
        scale *= 2.0 ** -power
    k = c.k.float()
    k[..., 77] = 0
    c.k = k.to(c.k.dtype)
    upload(c)
    c.check(c.run(decode=decode, scale=scale), scale=scale)
    c.check(c.run(30, 3, decode=decode, scale=scale), 30, 3, scale=scale)


def sees(p, t, window, sinks):
    return t <= p and (window == 0 or t > p - window or t < sinks)


# sequences, new rows of each, window, first tokens: pairs cut between blocks
# of threads and whole ones, pairs with rows for one tile only, several pairs
# one after another in a block of threads
ODD = [([300], [40], 0, 0), ([300, 77], [40, 77], 60, 4), ([9000], [20], 0, 0), ([9000, 300], [70, 1], 500, 17),
       ([700] * 20, [300] * 20, 0, 0), ([700] * 20, [300] * 20, 150, 5), ([257] * 60, [1, 33, 64] * 20, 0, 0)]


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,rows,window,sinks", ODD)
@pytest.mark.parametrize("value", ["nan", "-inf"])
def test_a_value_that_is_no_number_reaches_the_rows_that_see_it_only(cuda_dev, sa, out, lens, rows, window, sinks, value):
    """bf16 cache: rows that see a token lose the dims in which its value is no
    number; rows that do not - before it, or with a window past it - and all
    other dims are what they are with a zero in its place."""
    hq, hkv = 8, 2
    c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=hq, hkv=hkv, page=16, cache="bf16", out=out, seed=205, gaps=2)
    lost = torch.zeros((c.n_rows, hq, D), dtype=torch.bool, device=cuda_dev)
    rng = np.random.default_rng(3)
    marked = []
    for b, (N, m) in enumerate(zip(lens, rows)):
        if b % 3 == 2:
            continue  # every third sequence stays whole
        first = max(0, N - m - window) if window else N - m
        for t in {N - 1, N - m, N - m // 2, max(0, N - m - 1), 2} | {int(t) for t in rng.integers(first, N, 3)}:
            h, d = int(rng.integers(hkv)), int(rng.integers(D))
            marked.append((int(c.table[b, t // 16]), h, t % 16, d))
            for i in range(m):
                if sees(N - m + i, t, window, sinks):
                    lost[c.off[b] + i, h * 4:(h + 1) * 4, d] = True
    for at in marked:
        c.v[at] = 0
    upload(c)
    want = c.run(window, sinks)
    for at in marked:
        c.dv[at] = float(value)
    got = c.run(window, sinks)
    assert c.status() == sa.SA_OK
    assert not torch.isfinite(got[0][lost]).any()
    got[0][lost] = want[0][lost]
    c.check(got, window, sinks)
    again = c.run(window, sinks)
    again[0][lost] = want[0][lost]
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    # one call's values leave nothing for the next
    upload(c)
    again = c.run(window, sinks)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,rows,window,sinks", ODD)
def test_a_nan_key_reaches_the_rows_that_see_it_only(cuda_dev, sa, out, lens, rows, window, sinks):
    hq, hkv = 8, 2
    c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=hq, hkv=hkv, page=16, cache="bf16", out=out, seed=206, gaps=2)
    want = c.run(window, sinks)
    lost = torch.zeros_like(want[1], dtype=torch.bool)
    for b, (N, m) in enumerate(zip(lens, rows)):
        t, h = N - 1 - m // 3, b % hkv
        c.dk[int(c.table[b, t // 16]), h, t % 16, 77] = float("nan")
        for i in range(m):
            if sees(N - m + i, t, window, sinks):
                lost[c.off[b] + i, h * 4:(h + 1) * 4] = True
    got = c.run(window, sinks)
    assert c.status() == sa.SA_OK
    assert torch.isnan(got[0][lost]).all() and torch.isnan(got[1][lost]).all()
    assert torch.equal(got[0][~lost], want[0][~lost]) and torch.equal(got[1][~lost], want[1][~lost])


def test_first_calls_from_several_threads(cuda_dev):
    """In a process of its own: the first launches of kernels that ask for
    different amounts of shared memory, from threads at once."""
    code = """
import threading, torch
import block_sparse_kv_page_b200 as sa
dev, D = torch.device("cuda:0"), 128
made = []
for i in range(12):
    g = torch.Generator().manual_seed(i % 3)
    dt = torch.float8_e4m3fn if i & 1 else torch.bfloat16
    k, v = (torch.randn(40, 2, 16, D, generator=g).to(dt).to(dev) for _ in range(2))
    sc = torch.full((40, 2, 16), 127, dtype=torch.uint8, device=dev) if i & 1 else None
    table = torch.randperm(40, generator=g).to(torch.int32)[None].to(dev)
    kv = sa.PagedCache(k, v, table, torch.tensor([600], dtype=torch.int32, device=dev), k_scale=sc, v_scale=sc)
    decode = i % 3 == 0
    rows = 1 if decode else 50
    q = torch.randn(rows, 8, D, generator=g).to(torch.bfloat16).to(dev)
    out = torch.zeros(rows, 8, D, device=dev, dtype=torch.float32 if i & 2 else torch.bfloat16)
    off = torch.tensor([0, rows], dtype=torch.int32, device=dev)
    made.append((kv, decode, q, out, off, sa.make_paged_workspace(kv, 8), torch.cuda.Stream()))
def call(m, out):
    kv, decode, q, _, off, ws, s = m
    if decode:
        sa.sparse_attn_paged_decode(kv, q, 0.1, 0, 0, out, None, ws, s)
    else:
        sa.sparse_attn_chunk(kv, q, off, 0.1, 0, 0, out, None, ws, s)
torch.cuda.synchronize()
start, failed = threading.Barrier(len(made)), []
def work(m):
    start.wait()
    try:
        for _ in range(5):
            call(m, m[3])
    except Exception as e:
        failed.append(e)
threads = [threading.Thread(target=work, args=(m,)) for m in made]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
for m in made:
    again = torch.zeros_like(m[3])
    call(m, again)
    torch.cuda.synchronize()
    assert torch.equal(again, m[3])
    assert sa.sparse_attn_get_device_status(m[5]) == sa.SA_OK
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=150)
    assert run.returncode == 0, run.stderr[-2000:]


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("decode", [True, False])
def test_every_value_row_counts_once(cuda_dev, sa, out, cache, page, decode):
    """The value of token t is one-hot in dim t mod 128, so a dim is the sum of a
    few tokens' weights and one lost or added row changes it by a tenth or more:
    tolerances are relative to that sum.  Lengths, rows, windows and first tokens
    around blocks of 64, pages and tiles."""
    lens = [517, 33, 256, 700, 65, 1]
    rows = [1] * 6 if decode else [40, 33, 100, 300, 2, 1]
    c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=6, hkv=2, page=page, cache=cache, out=out, seed=207, gaps=1 - decode)
    v = torch.zeros_like(c.v.float())
    for b, N in enumerate(lens):
        for t in range(N):
            v[int(c.table[b, t // page]), :, t % page, t % D] = (1 + (t // D) / 8) * (-1 if t % 3 else 1)
    c.v = v.to(c.v.dtype)
    if c.e4m3:
        c.vs.fill_(127)
    upload(c)
    q = c.q.clone()
    for zero in (True, False):
        c.q = torch.zeros_like(q) if zero else q
        upload(c)
        for window, sinks in ((0, 0), (1, 0), (63, 1), (64, 16), (65, 4), (150, 20), (300, 130)):
            got = c.run(window, sinks, decode=decode)
            check_rows(c, got, 1 / math.sqrt(D), None, decode, window, sinks)
    assert c.status() == sa.SA_OK


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("scale_byte", [0, 255])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_scale_bytes_of_hidden_tokens_may_be_anything(cuda_dev, sa, out, decode, scale_byte, window, sinks):
    """Slots past a sequence's end, spare pages and tokens that a window has
    passed: bit for bit as with ordinary scale bytes there."""
    lens = [517, 33, 256, 70]
    rows = [1] * 4 if decode else [40, 33, 1, 65]
    c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=8, hkv=2, page=64, cache="e4m3", out=out, seed=208, stale=0x7f)
    want = c.run(window, sinks, decode=decode)
    c.check(want, window, sinks)
    live = torch.zeros(c.ks.shape[0], 64, dtype=torch.bool)
    for b, (N, m) in enumerate(zip(lens, rows)):
        for t in range(N):
            if window == 0 or t >= max(0, N - m - window + 1) or t < sinks:
                live[int(c.table[b, t // 64]), t % 64] = True
    for held in (c.ks, c.vs):
        held[~live[:, None, :].expand(-1, 2, -1)] = scale_byte
    upload(c)
    got = c.run(window, sinks, decode=decode)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert c.status() == sa.SA_OK


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("longest", [40, 9000])
def test_nan_queries_with_bf16_outputs(cuda_dev, sa, cache, decode, longest):
    """Also the first vector of a tile, which is looked at for values that are no numbers."""
    lens = [longest, 33, longest // 2]
    rows = [1] * 3 if decode else [20, 3, 7]
    c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=8, hkv=2, page=16, cache=cache, out="bf16", seed=209)
    want = c.run(decode=decode)
    c.check(want)
    lost = ((0, 0), (1, 3), (2, 7))
    for r, h in lost:
        c.dq[r, h, 5] = float("nan")
    out, lse = c.run(decode=decode)
    for r, h in lost:
        assert torch.isnan(out[r, h]).all() and torch.isnan(lse[r, h])
        out[r, h], lse[r, h] = want[0][r, h], want[1][r, h]
    # (not bit for bit: the rows of two warps raise their references together, so
    # one row's scores may choose the one that another's weights are rounded against)
    c.check((out, lse))


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_a_nan_value_in_the_single_token_form(cuda_dev, sa, out, window, sinks):
    """Its dim of the heads that share it, if the window or the first tokens
    show it; nothing where they do not."""
    c = Case(sa, cuda_dev, lens=[5000, 70], rows=[1, 1], hq=8, hkv=2, page=16, cache="bf16", out=out, seed=210)
    want = c.run(window, sinks, decode=True)
    for t, d in ((1234, 9), (4990, 100), (3, 50)):
        c.dv[int(c.table[0, t // 16]), 1, t % 16, d] = float("nan")
    got = c.run(window, sinks, decode=True)
    lost = torch.zeros_like(got[0], dtype=torch.bool)
    lost[0, 4:, [100, 50] + ([] if window else [9])] = True
    assert torch.isnan(got[0][lost]).all()
    assert torch.equal(got[0][~lost], want[0][~lost]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,rows,window,sinks", ODD[:4])
@pytest.mark.parametrize("which", ["last", "all"])
def test_whole_value_rows_of_no_numbers(cuda_dev, sa, out, lens, rows, window, sinks, which):
    """All dims of the newest token's value: the newest row alone loses its
    output; of all new tokens' values: every row does.  lse is as it was."""
    c = Case(sa, cuda_dev, lens=lens, rows=rows, hq=8, hkv=2, page=16, cache="bf16", out=out, seed=211, gaps=2)
    want = c.run(window, sinks)
    lost = torch.zeros(c.n_rows, dtype=torch.bool)
    for b, (N, m) in enumerate(zip(lens, rows)):
        for t in range(N - 1 if which == "last" else N - m, N):
            c.dv[int(c.table[b, t // 16]), :, t % 16] = float("nan")
            lost[c.off[b] + t - (N - m)] = True
    got = c.run(window, sinks)
    assert c.status() == sa.SA_OK
    assert torch.isnan(got[0][lost]).all()
    got[0][lost] = want[0][lost]
    c.check(got, window, sinks)
    assert torch.equal(got[1], want[1])
