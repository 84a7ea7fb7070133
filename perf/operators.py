"""Workloads of the paged-cache operators, with the operators in plain torch.

The operators serve a cache of keys and values held in pages that a page table
maps, in bf16 or in e4m3 with a power-of-two scale per row: `write` stores new
tokens (quantising them), `read` copies the cache back into one contiguous
bf16 cache, `decode` attends with one query row per sequence and `chunk` with
a run of new rows per sequence, causally, over the whole cache or over a
sliding window and a few first tokens that stay visible.

`run` computes them with elementary torch operations in 32 bits where `own` is
false, and with block_sparse_kv_page_b200's calls where it is true.
"""
import math
import random

import numpy as np
import torch

own = False
if torch.backends.cuda.matmul.allow_tf32:  # the plain form is a 32-bit one
    torch.backends.cuda.matmul.allow_tf32 = False

D = 128
SCALE = 1.0 / math.sqrt(D)


# ---------------------------------------------------------------- the cases
def _case(op, *, hq, hkv, page, batch, longest, rows, cache="e4m3", ragged=0, window=0, sinks=0,
          out="bf16", order="head", fused=False):
    """hq, hkv: query and KV heads.  longest: tokens of the longest sequence,
    its new ones included; rows: most new tokens of a sequence.  ragged: 0 for
    sequences of one length, else the seed of their lengths.  order: pages
    held head by head or token by token.  fused: q, k and v are parts of the
    rows of one projection."""
    return dict(op=op, hq=hq, hkv=hkv, page=page, batch=batch, longest=longest, rows=rows, cache=cache,
                ragged=ragged, window=window, sinks=sinks, out=out, order=order, fused=fused)


def listed():
    return [
        # the newest token of each of 8 sequences: what every decode step does first
        dict(_case("write", hq=64, hkv=8, page=16, batch=8, longest=32768, rows=1, ragged=1, fused=True),
             name="write-step-b8"),
        # one prefill chunk, token-major pages
        dict(_case("write", hq=28, hkv=4, page=64, batch=1, longest=32768, rows=2048, order="token", fused=True),
             name="write-chunk-2048"),
        # eight whole prompts of unequal length
        dict(_case("write", hq=64, hkv=8, page=16, batch=8, longest=32768, rows=32768, ragged=2),
             name="write-prompts-b8"),
        # one web-agent context handed to the operators of the contiguous cache
        dict(_case("read", hq=32, hkv=4, page=16, batch=1, longest=29504, rows=1), name="read-29.5k"),
        # a whole batch read back, unequal lengths, token-major pages
        dict(_case("read", hq=64, hkv=8, page=64, batch=8, longest=32768, rows=1, ragged=3, order="token"),
             name="read-32k-b8"),
        # one agent's next token over its whole bf16 context
        dict(_case("decode", hq=32, hkv=4, page=16, batch=1, longest=29504, rows=1, cache="bf16", out="fp32"),
             name="decode-29.5k-b1-bf16"),
        # a batch's next tokens, a window of 4096 and 4 first tokens
        dict(_case("decode", hq=64, hkv=8, page=16, batch=8, longest=32768, rows=1, window=4096, sinks=4, fused=True),
             name="decode-window-b8"),
        # a larger batch of unequal lengths over all of its context
        dict(_case("decode", hq=64, hkv=8, page=64, batch=32, longest=32768, rows=1, ragged=4, order="token"),
             name="decode-32k-b32"),
        # 16 drafted tokens checked at once, fp32 outputs as the framework's decode gives them
        dict(_case("chunk", hq=32, hkv=4, page=16, batch=1, longest=29504, rows=16, cache="bf16", out="fp32"),
             name="chunk-16-of-29.5k-bf16"),
        # a chunk of 2048 prompt tokens late in its context
        dict(_case("chunk", hq=28, hkv=4, page=64, batch=1, longest=32768, rows=2048, cache="bf16", fused=True),
             name="chunk-2048-of-32k-bf16"),
        # four short prompts of unequal length in one call
        dict(_case("chunk", hq=32, hkv=4, page=16, batch=4, longest=2048, rows=2048, ragged=5),
             name="chunk-prompts-b4"),
        # a chunk late in its context that sees a window of 4096 and 4 first tokens
        dict(_case("chunk", hq=64, hkv=8, page=64, batch=1, longest=29504, rows=1024, window=4096, sinks=4,
                   order="token"), name="chunk-1024-window"),
    ]


def lengths(case):
    """([tokens of each sequence], [new tokens of each sequence])"""
    B, longest, rows = case["batch"], case["longest"], case["rows"]
    n, m = [longest] * B, [min(rows, longest)] * B
    if case["ragged"]:
        r = random.Random(case["ragged"])
        for b in range(1, B):
            n[b] = r.randint(max(1, longest // 8), longest)
            m[b] = min(n[b], r.randint(max(1, rows // 8), rows))
    return n, m


def _between(rng, lo, hi):
    """A whole number, even over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    top = [work(c) for c in listed()]
    while True:
        op = rng.choice(("write", "read", "decode", "decode", "chunk", "chunk"))
        hq, hkv = rng.choice(((32, 4), (64, 8), (28, 4), (16, 2), (8, 1), (4, 4), (10, 5)))
        longest = _between(rng, 16, 65536)
        window = rng.choice((0, 0, _between(rng, 1, 8192)))
        c = _case(op, hq=hq, hkv=hkv, page=rng.choice((16, 16, 32, 48, 64, 128, 256)), batch=_between(rng, 1, 48),
                  longest=longest, rows=1 if op in ("decode", "read") else _between(rng, 1, min(longest, 8192)),
                  cache=rng.choice(("bf16", "e4m3")), ragged=rng.randint(0, 1 << 20) * rng.randint(0, 1),
                  window=window, sinks=rng.choice((0, 4, 17)) if window else 0,
                  out=rng.choice(("bf16", "bf16", "fp32")), order=rng.choice(("head", "token")),
                  fused=rng.random() < 0.5)
        n, m = lengths(c)
        w = work(c)
        scores = c["batch"] * hq * max(m) * longest if op in ("decode", "chunk") else 0
        rows = c["batch"] * hkv * longest
        if w["bytes"] <= max(t["bytes"] for t in top) and w["flops"] <= max(t["flops"] for t in top) \
                and scores <= 2.0e9 and rows <= 8.5e6 and sum(m) * hq <= 1.0e7:
            return c


def work(case):
    n, m = lengths(case)
    hq, hkv, win, sinks = case["hq"], case["hkv"], case["window"], case["sinks"]
    row = 2 * (D + 1) if case["cache"] == "e4m3" else 4 * D  # a token's K and V of one head, as held
    if case["op"] == "write":
        return {"bytes": sum(m) * hkv * (4 * D + row), "flops": 0}
    if case["op"] == "read":
        return {"bytes": sum(n) * hkv * (4 * D + row), "flops": 0}
    held, pairs = 0, 0
    for N, M in zip(n, m):
        first = max(0, N - M - win + 1) if win else 0
        held += N - first + min(sinks, first)
        see = np.arange(N - M + 1, N + 1, dtype=np.int64)
        if win:
            see = np.where(see > win, win + np.minimum(sinks, see - win), see)
        pairs += int(see.sum())
    return {"bytes": held * hkv * row + sum(m) * hq * (2 * D + D * (2 if case["out"] == "bf16" else 4) + 4),
            "flops": pairs * hq * 4 * D}


# ---------------------------------------------------------------- the inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    n, m = lengths(case)
    B, hq, hkv, page = case["batch"], case["hq"], case["hkv"], case["page"]
    per = [-(-x // page) for x in n]
    max_pages, n_pages = max(per), sum(per) + 5

    # the pages of the sequences, in no order
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.zeros((B, max_pages), dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, : per[b]] = perm[at: at + per[b]]
        at += per[b]

    def pool():
        shape = (n_pages, hkv, page, D) if case["order"] == "head" else (n_pages, page, hkv, D)
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        x.normal_(generator=g)
        return x if case["order"] == "head" else x.transpose(1, 2)

    # keys with a scale of its own for every channel, as outlier channels have
    channel = torch.exp(torch.empty((hkv, 1, D), device=dev).uniform_(math.log(0.5), math.log(4.0), generator=g))
    k, v = pool().mul_(channel.to(torch.bfloat16)), pool()
    s = {"case": case, "page_table": table.to(dev), "seq_len": torch.tensor(n, dtype=torch.int32, device=dev),
         "k_scale": None, "v_scale": None}
    if case["cache"] == "e4m3":
        (k, s["k_scale"]), (v, s["v_scale"]) = _held(k), _held(v)
    s["k"], s["v"] = k, v

    off = np.concatenate([[0], np.cumsum(m)])
    s["row_off"] = torch.tensor(off, dtype=torch.int32, device=dev)
    rows = int(off[-1])
    if case["op"] != "read":
        heads = hq + 2 * hkv
        if case["fused"]:
            x = torch.empty((rows, heads, D), dtype=torch.bfloat16, device=dev).normal_(generator=g)
            s["q"], s["k_new"], s["v_new"] = x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:]
        elif case["op"] == "write":
            s["k_new"] = torch.empty((rows, hkv, D), dtype=torch.bfloat16, device=dev).normal_(generator=g)
            s["v_new"] = torch.empty((rows, hkv, D), dtype=torch.bfloat16, device=dev).normal_(generator=g)
        else:
            s["q"] = torch.empty((rows, hq, D), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    if case["op"] == "read":
        cap = max_pages * page
        s["k_out"] = torch.zeros((B, hkv, cap, D), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros((B, hkv, cap, D), dtype=torch.bfloat16, device=dev)
    if case["op"] in ("decode", "chunk"):
        s["out"] = torch.empty((rows, hq, D), dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32,
                               device=dev)
        s["lse"] = torch.empty((rows, hq), dtype=torch.float32, device=dev)
    if own:  # the handle and workspace that a serving program keeps
        import block_sparse_kv_page_b200 as sa
        s["cache"] = sa.PagedCache(s["k"], s["v"], s["page_table"], s["seq_len"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"])
        s["ws"] = sa.make_paged_workspace(s["cache"], hq)
    return s


# ---------------------------------------------------------------- the plain forms
def _two_to(k):
    """2^k in fp32, exactly, for int32 k in [-126, 127]"""
    return ((k + 127) << 23).view(torch.float32)


def _quantise(x):
    """fp32 rows -> e4m3 codes and the biased exponents of the rows' scales:
    the smallest power of two that leaves the row within 448."""
    frac, e = torch.frexp(x.abs().amax(-1))          # amax = frac * 2^e, 0.5 <= frac < 1; 448 = 0.875 * 2^9
    k = torch.where(frac <= 0.875, e - 9, e - 8)
    k = torch.where(frac == 0, torch.full_like(k, -124), k).clamp(-124, 119)
    y = x * _two_to(-k)[..., None]
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), (k + 127).to(torch.uint8)


def _value(code, scale):
    """e4m3 codes and biased exponents -> fp32 rows"""
    return code.float() * _two_to(scale.to(torch.int32) - 127)[..., None]


def _held(x):
    """A bf16 pool as it is held in e4m3, in the same order in memory."""
    code, scale = _quantise(x.float())
    held = torch.empty_strided(x.shape, x.stride(), dtype=torch.float8_e4m3fn, device=x.device)
    held.copy_(code)
    return held, scale.contiguous()


def _gather(s, name):
    """The cache through its page table: fp32 [B][Hkv][max_pages * page][128]"""
    table = s["page_table"].long()
    x = s[name].view(torch.uint8)[table].view(torch.float8_e4m3fn) if s["case"]["cache"] == "e4m3" else s[name][table]
    x = _value(x, s[name + "_scale"][table]) if s["case"]["cache"] == "e4m3" else x.float()
    B, pages, hkv, page, _ = x.shape
    return x.transpose(1, 2).reshape(B, hkv, pages * page, D)


def _row_places(s):
    """For every new row: its sequence, and its place among that sequence's new rows."""
    off = s["row_off"].long()
    rows = torch.arange(s["q" if "q" in s else "k_new"].shape[0], device=off.device)
    b = torch.searchsorted(off, rows, right=True) - 1
    return b, rows - off[b]


def _plain_write(s):
    b, i = _row_places(s)
    off, page = s["row_off"].long(), s["case"]["page"]
    t = s["seq_len"].long()[b] - (off[b + 1] - off[b]) + i
    at, slot = s["page_table"].long()[b, t // page], t % page
    if s["case"]["cache"] == "e4m3":
        kc, ks = _quantise(s["k_new"].float())
        vc, vs = _quantise(s["v_new"].float())
        s["k"].view(torch.uint8)[at, :, slot] = kc.view(torch.uint8)
        s["v"].view(torch.uint8)[at, :, slot] = vc.view(torch.uint8)
        s["k_scale"][at, :, slot] = ks
        s["v_scale"][at, :, slot] = vs
    else:
        s["k"][at, :, slot] = s["k_new"]
        s["v"][at, :, slot] = s["v_new"]


def _plain_read(s):
    t = torch.arange(s["k_out"].shape[2], device=s["seq_len"].device)
    held = (t < s["seq_len"].long()[:, None])[:, None, :, None]
    s["k_out"].copy_(torch.where(held, _gather(s, "k").to(torch.bfloat16), s["k_out"]))
    s["v_out"].copy_(torch.where(held, _gather(s, "v").to(torch.bfloat16), s["v_out"]))


def _plain_attend(s):
    c = s["case"]
    b, i = _row_places(s)
    off, n = s["row_off"].long(), s["seq_len"].long()
    m = off[1:] - off[:-1]
    B, hkv, G, M = c["batch"], c["hkv"], c["hq"] // c["hkv"], min(c["rows"], c["longest"])
    k, v = _gather(s, "k"), _gather(s, "v")
    N = k.shape[2]
    q = torch.zeros((B, M, hkv, G, D), dtype=torch.float32, device=k.device)
    q[b, i] = s["q"].float().reshape(-1, hkv, G, D)
    z = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, hkv, G * M, D), k.transpose(2, 3)).mul_(SCALE)
    t = torch.arange(N, device=k.device)
    p = (n - m)[:, None] + torch.arange(M, device=k.device)          # positions [B][M]
    see = t <= p[:, :, None]
    if c["window"]:
        see &= (t > p[:, :, None] - c["window"]) | (t < c["sinks"])
    z.view(B, hkv, G, M, N).masked_fill_(~see[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).view(B, hkv, G, M).permute(0, 3, 1, 2)[b, i].reshape(-1, c["hq"])
    o = o.view(B, hkv, G, M, D).permute(0, 3, 1, 2, 4)[b, i].reshape(-1, c["hq"], D)
    return {"out": o.to(s["out"].dtype), "lse": lse}


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import block_sparse_kv_page_b200 as sa
        if op == "write":
            sa.sparse_attn_cache_write(s["cache"], s["k_new"], s["v_new"], s["row_off"], s["ws"])
        elif op == "read":
            sa.sparse_attn_cache_read(s["cache"], 0, s["k_out"], s["v_out"], s["ws"])
        elif op == "decode":
            sa.sparse_attn_paged_decode(s["cache"], s["q"], SCALE, c["window"], c["sinks"], s["out"], s["lse"],
                                        s["ws"])
        else:
            sa.sparse_attn_chunk(s["cache"], s["q"], s["row_off"], SCALE, c["window"], c["sinks"], s["out"],
                                 s["lse"], s["ws"])
        if op in ("decode", "chunk"):
            return {"out": s["out"], "lse": s["lse"]}
    elif op == "write":
        _plain_write(s)
    elif op == "read":
        _plain_read(s)
    else:
        return _plain_attend(s)
    if op == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    held = {"k": s["k"], "v": s["v"]}
    if c["cache"] == "e4m3":
        held.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return held


# ---------------------------------------------------------------- the definition, in 64 bits
_POWERS = 2.0 ** np.arange(-200, 201)


def _power64(k):
    """2^k in 64 bits for whole k, from a table"""
    return torch.from_numpy(_POWERS).to(k.device)[k.long() + 200]


def _code64(x):
    """Rows of values -> their e4m3 codes, by the definition of its grid."""
    x = x.double()
    a = x.abs().amax(-1)
    k = torch.full_like(a, -124.0)
    big = a > 0
    k[big] = torch.ceil(torch.log2(a[big] / 448.0))
    k = torch.where(a > 448.0 * _power64(k), k + 1, k)
    k = torch.where((a <= 448.0 * _power64(k - 1)) & big, k - 1, k).clamp(-124, 119)
    y = x * _power64(-k)[..., None]
    grid = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    grid = torch.where(y.abs() < _power64(grid), grid - 1, grid)
    step = _power64(grid.clamp_min(-6.0) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    n, m = lengths(case)
    page, hkv, hq = case["page"], case["hkv"], case["hq"]
    G = hq // hkv
    off = np.concatenate([[0], np.cumsum(m)])
    e4m3 = case["cache"] == "e4m3"
    table = s["page_table"].long()
    if case["op"] == "write":
        out = {"k": s["k"].double(), "v": s["v"].double()}
        for b in range(case["batch"]):
            t = torch.arange(n[b] - m[b], n[b], device=table.device)
            for name in ("k", "v"):
                x = s[name + "_new"][off[b]: off[b + 1]]
                out[name][table[b][t // page], :, t % page] = _code64(x) if e4m3 else x.double()
        if e4m3:
            out.update(k_scale=None, v_scale=None)
        return out

    def tokens(b, name, h):
        x = s[name][:, h].view(torch.uint8)[table[b]].view(torch.float8_e4m3fn) if e4m3 else s[name][:, h][table[b]]
        x = x.double().reshape(-1, D)[: n[b]]
        if e4m3:
            x = x * _power64(s[name + "_scale"][:, h][table[b]].reshape(-1)[: n[b]].long() - 127)[:, None]
        return x

    if case["op"] == "read":
        if sum(n) * hkv > 2.0e6:
            return None
        out = {"k": s["k_out"].double(), "v": s["v_out"].double()}
        for b in range(case["batch"]):
            for h in range(hkv):
                for name in ("k", "v"):
                    out[name][b, h, : n[b]] = tokens(b, name, h)
        return out

    if work(case)["flops"] > 4e12 or case["batch"] * hq > 4096:
        return None
    out = torch.zeros((int(off[-1]), hq, D), dtype=torch.float64, device=table.device)
    lse = torch.zeros((int(off[-1]), hq), dtype=torch.float64, device=table.device)
    for b in range(case["batch"]):
        p = torch.arange(n[b] - m[b], n[b], device=table.device)[:, None]
        t = torch.arange(n[b], device=table.device)[None]
        hidden = t > p
        if case["window"]:
            hidden = hidden | ((p - t >= case["window"]) & (t >= case["sinks"]))
        for h in range(hkv):
            k, v = tokens(b, "k", h), tokens(b, "v", h)
            for j in range(h * G, h * G + G):
                z = (s["q"][off[b]: off[b + 1], j].double() @ k.T) * SCALE
                z[hidden] = -math.inf
                l = torch.logsumexp(z, -1)
                lse[off[b]: off[b + 1], j] = l
                out[off[b]: off[b + 1], j] = torch.exp(z - l[:, None]) @ v
    return {"out": out, "lse": lse}
