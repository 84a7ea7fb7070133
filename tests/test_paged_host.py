"""The paged-cache calls refuse bad arguments on the host, before any launch
(CPU only: the pointers below are never dereferenced)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def abi():
    from block_sparse_kv_page_b200 import _abi
    return _abi


@pytest.fixture(scope="module")
def lib(abi):
    return abi.load()


def _desc(abi, **kw):
    d = dict(batch=2, n_kv_heads=4, head_dim=128, page_size=16, n_pages=64, dtype=abi.SA_KV_BF16, max_pages=8,
             k=0x10000, v=0x20000, page_stride=16 * 4 * 128, head_stride=16 * 128, token_stride=128,
             k_scale=None, v_scale=None, page_table=0x30000, seq_len=0x40000)
    d.update(kw)
    return abi.sa_paged_desc(**d)


def _e4m3(abi, **kw):
    return _desc(abi, **{**dict(dtype=abi.SA_KV_E4M3, k_scale=0x50000, v_scale=0x60000), **kw})


BAD = [
    (dict(batch=0), "INVALID"), (dict(n_kv_heads=0), "INVALID"), (dict(max_pages=0), "INVALID"),
    (dict(n_pages=0), "INVALID"), (dict(dtype=2), "INVALID"), (dict(dtype=-1), "INVALID"),
    (dict(head_dim=64), "UNSUPPORTED"), (dict(page_size=8), "UNSUPPORTED"), (dict(page_size=24), "UNSUPPORTED"),
    (dict(page_size=272), "UNSUPPORTED"), (dict(page_size=0), "UNSUPPORTED"), (dict(n_pages=1 << 31), "UNSUPPORTED"),
    (dict(max_pages=1 << 27), "UNSUPPORTED"), (dict(k=None), "INVALID"), (dict(v=None), "INVALID"),
    (dict(k=0x10008), "INVALID"), (dict(v=0x20002), "INVALID"), (dict(token_stride=64), "INVALID"),
    (dict(token_stride=129), "INVALID"), (dict(head_stride=0), "INVALID"), (dict(head_stride=-2048), "INVALID"),
    (dict(page_stride=8196), "INVALID"), (dict(page_stride=1 << 39), "UNSUPPORTED"),
    (dict(k_scale=0x50000), "INVALID"), (dict(page_table=None), "INVALID"), (dict(page_table=0x30002), "INVALID"),
    (dict(seq_len=None), "INVALID"),
]
BAD_E4M3 = [(dict(k_scale=None), "INVALID"), (dict(v_scale=None), "INVALID"), (dict(k_scale=0x50008), "INVALID"),
            (dict(token_stride=136), "INVALID")]


def _calls(lib, abi, desc, **kw):
    a = dict(x=0x100000, y=0x200000, stride=64 * 128, hq=32, off=0x300000, rows=10, window=0, sinks=0, scale=0.088,
             out=0x400000, dtype=abi.SA_OUT_F32, lse=0x500000, ws=0x600000, ws_bytes=1 << 32, cap=128)
    a.update(kw)
    p = C.byref(desc) if desc is not None else None
    return {
        "write": lib.sparse_attn_cache_write(p, a["x"], a["y"], a["stride"], a["off"], a["rows"], a["ws"],
                                             a["ws_bytes"], None),
        "read": lib.sparse_attn_cache_read(p, 0, a["x"], a["y"], a["cap"], a["ws"], a["ws_bytes"], None),
        "chunk": lib.sparse_attn_chunk(p, a["x"], a["stride"], a["hq"], a["off"], a["rows"], a["window"], a["sinks"],
                                       a["scale"], a["out"], a["dtype"], a["lse"], a["ws"], a["ws_bytes"], None),
        "decode": lib.sparse_attn_paged_decode(p, a["x"], a["stride"], a["hq"], a["window"], a["sinks"], a["scale"],
                                               a["out"], a["dtype"], a["lse"], a["ws"], a["ws_bytes"], None),
    }


@pytest.mark.parametrize("kw,why", BAD)
def test_bad_cache(lib, abi, kw, why):
    want = getattr(abi, "SA_ERR_" + why)
    assert set(_calls(lib, abi, _desc(abi, **kw)).values()) == {want}
    assert lib.sparse_attn_paged_workspace_size(C.byref(_desc(abi, **kw)), 32) == 0


@pytest.mark.parametrize("kw,why", BAD_E4M3)
def test_bad_e4m3_cache(lib, abi, kw, why):
    assert set(_calls(lib, abi, _e4m3(abi, **kw)).values()) == {getattr(abi, "SA_ERR_" + why)}


def test_null_cache(lib, abi):
    assert set(_calls(lib, abi, None).values()) == {abi.SA_ERR_INVALID}
    assert lib.sparse_attn_paged_workspace_size(None, 32) == 0


@pytest.mark.parametrize("kw,calls,why", [
    (dict(x=None), ("write", "read", "chunk", "decode"), "INVALID"),
    (dict(x=0x100008), ("write", "read", "chunk", "decode"), "INVALID"),
    (dict(y=None), ("write", "read"), "INVALID"),
    (dict(stride=128), ("write", "chunk", "decode"), "INVALID"),
    (dict(stride=64 * 128 + 4), ("write", "chunk", "decode"), "INVALID"),
    (dict(off=None), ("write", "chunk"), "INVALID"),
    (dict(off=0x300002), ("write", "chunk"), "INVALID"),
    (dict(rows=-1), ("write", "chunk"), "INVALID"),
    (dict(cap=0), ("read",), "INVALID"),
    (dict(hq=30), ("chunk", "decode"), "INVALID"),
    (dict(hq=0), ("chunk", "decode"), "INVALID"),
    (dict(hq=36), ("chunk", "decode"), "UNSUPPORTED"),
    (dict(window=-1), ("chunk", "decode"), "INVALID"),
    (dict(sinks=-1), ("chunk", "decode"), "INVALID"),
    (dict(scale=float("nan")), ("chunk", "decode"), "INVALID"),
    (dict(scale=float("inf")), ("chunk", "decode"), "INVALID"),
    (dict(scale=3e38), ("chunk", "decode"), "INVALID"),   # times log2(e) it is not finite
    (dict(out=None), ("chunk", "decode"), "INVALID"),
    (dict(out=0x400004), ("chunk", "decode"), "INVALID"),
    (dict(dtype=2), ("chunk", "decode"), "INVALID"),
    (dict(lse=0x500002), ("chunk", "decode"), "INVALID"),
    (dict(ws=None), ("chunk", "decode"), "WORKSPACE"),
    (dict(ws=0x600010), ("write", "read", "chunk", "decode"), "WORKSPACE"),
    (dict(ws_bytes=128), ("write", "read", "chunk", "decode"), "WORKSPACE"),
])
def test_bad_arguments(lib, abi, kw, calls, why):
    for make in (_desc, _e4m3):
        # one bad argument only ever reaches calls that refuse it: the others would launch
        d = make(abi)
        a = dict(x=0x100000, y=0x200000, stride=64 * 128, hq=32, off=0x300000, rows=10, window=0, sinks=0,
                 scale=0.088, out=0x400000, dtype=abi.SA_OUT_F32, lse=0x500000, ws=0x600000, ws_bytes=1 << 32, cap=128)
        a.update(kw)
        p = C.byref(d)
        for c in calls:
            if c == "write":
                r = lib.sparse_attn_cache_write(p, a["x"], a["y"], a["stride"], a["off"], a["rows"], a["ws"],
                                                a["ws_bytes"], None)
            elif c == "read":
                r = lib.sparse_attn_cache_read(p, 0, a["x"], a["y"], a["cap"], a["ws"], a["ws_bytes"], None)
            elif c == "chunk":
                r = lib.sparse_attn_chunk(p, a["x"], a["stride"], a["hq"], a["off"], a["rows"], a["window"],
                                          a["sinks"], a["scale"], a["out"], a["dtype"], a["lse"], a["ws"],
                                          a["ws_bytes"], None)
            else:
                r = lib.sparse_attn_paged_decode(p, a["x"], a["stride"], a["hq"], a["window"], a["sinks"], a["scale"],
                                                 a["out"], a["dtype"], a["lse"], a["ws"], a["ws_bytes"], None)
            assert r == getattr(abi, "SA_ERR_" + why), c


def test_workspace_one_byte_short(lib, abi):
    d = _e4m3(abi)
    need = lib.sparse_attn_paged_workspace_size(C.byref(d), 32)
    assert need > 0
    p = C.byref(d)
    assert lib.sparse_attn_chunk(p, 0x100000, 64 * 128, 32, 0x300000, 10, 0, 0, 0.1, 0x400000, 0, None, 0x600000,
                                 need - 1, None) == abi.SA_ERR_WORKSPACE
    assert lib.sparse_attn_paged_decode(p, 0x100000, 64 * 128, 32, 0, 0, 0.1, 0x400000, 0, None, 0x600000, need - 1,
                                        None) == abi.SA_ERR_WORKSPACE


def test_no_rows_is_no_work(lib, abi):
    p = C.byref(_desc(abi))
    assert lib.sparse_attn_cache_write(p, 0x100000, 0x200000, 64 * 128, 0x300000, 0, None, 0, None) == abi.SA_OK
    assert lib.sparse_attn_chunk(p, 0x100000, 64 * 128, 32, 0x300000, 0, 0, 0, 0.1, 0x400000, 0, None, 0x600000,
                                 1 << 32, None) == abi.SA_OK


def _cache(**kw):
    import block_sparse_kv_page_b200 as sa
    a = dict(k=torch.zeros(5, 2, 16, 128, dtype=torch.bfloat16), v=torch.zeros(5, 2, 16, 128, dtype=torch.bfloat16),
             page_table=torch.zeros(3, 2, dtype=torch.int32), seq_len=torch.zeros(3, dtype=torch.int32))
    a.update(kw)
    return sa.PagedCache(a.pop("k"), a.pop("v"), a.pop("page_table"), a.pop("seq_len"), **a)


def test_binding_takes_token_major_pages_and_parts():
    big = torch.zeros(7, 16, 2, 3, 128, dtype=torch.bfloat16)
    c = _cache(k=big[:5, :, :, 0].transpose(1, 2), v=big[:5, :, :, 2].transpose(1, 2))
    assert (c.desc.page_stride, c.desc.head_stride, c.desc.token_stride) == (16 * 6 * 128, 3 * 128, 6 * 128)
    one = torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16)
    c = _cache(k=one.as_strided((1, 1, 16, 128), (1, 1, 128, 1)), v=one)
    assert c.desc.page_stride == 2048 and c.desc.head_stride == 2048


@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros(5, 2, 16, 128)), dict(v=torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)),
    dict(k=torch.zeros(5, 16, 2, 128, dtype=torch.bfloat16).transpose(1, 2)),
    dict(k=torch.zeros(5, 2, 128, 16, dtype=torch.bfloat16).transpose(2, 3)),
    dict(page_table=torch.zeros(3, 2, dtype=torch.int64)), dict(page_table=torch.zeros(2, 3, dtype=torch.int32).T),
    dict(seq_len=torch.zeros(2, dtype=torch.int32)), dict(seq_len=torch.zeros(3)),
    dict(k_scale=torch.zeros(5, 2, 16, dtype=torch.uint8)),
    dict(k=torch.zeros(5, 2, 16, 128).to(torch.float8_e4m3fn), v=torch.zeros(5, 2, 16, 128).to(torch.float8_e4m3fn)),
])
def test_binding_refuses_bad_caches(kw):
    with pytest.raises(ValueError):
        _cache(**kw)


def test_binding_refuses_bad_rows():
    import block_sparse_kv_page_b200 as sa
    c = _cache()
    off = torch.zeros(4, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    for k, v, o in ((bf(4, 3, 128), bf(4, 3, 128), off), (torch.zeros(4, 2, 128), bf(4, 2, 128), off),
                    (bf(4, 2, 128), bf(5, 2, 128), off), (bf(4, 2, 128), bf(4, 2, 128), off[:3]),
                    (bf(4, 2, 128), bf(4, 2, 128), off.long()), (bf(4, 2, 128), bf(4, 4, 128)[:, :2], off),
                    (bf(4, 2, 256)[:, :, ::2], bf(4, 2, 128), off)):
        with pytest.raises(ValueError):
            sa.sparse_attn_cache_write(c, k, v, o)
    for q, out, lse in ((bf(3, 4, 128), bf(3, 4, 64), None), (bf(3, 4, 128), torch.zeros(3, 4, 128).half(), None),
                        (bf(3, 4, 128), bf(3, 4, 128), torch.zeros(3, 2)), (bf(2, 4, 128), bf(2, 4, 128), None),
                        (bf(3, 4, 64), bf(3, 4, 64), None)):
        with pytest.raises(ValueError):
            sa.sparse_attn_paged_decode(c, q, 0.1, 0, 0, out, lse, None)
    with pytest.raises(ValueError):
        sa.sparse_attn_cache_read(c, 0, bf(3, 2, 32, 128), bf(3, 2, 33, 128))


def test_workspace_size_through_the_binding():
    import block_sparse_kv_page_b200 as sa
    c = _cache()
    n = sa.sparse_attn_paged_workspace_size(c, 8)
    assert n > 256 and n % 256 == 0
    assert sa.sparse_attn_paged_workspace_size(c, 7) == 0


def test_longest_sequence(abi, lib):
    """Lengths are held, and blocks of 64 tokens ended, in 32 bits."""
    for pages, page in (((1 << 27) - 1, 16), ((1 << 23) - 1, 256), ((1 << 25) - 1, 64)):
        ok = pages * page <= 2 ** 31 - 256
        kv = _desc(abi, max_pages=pages, page_size=page)
        assert (lib.sparse_attn_paged_workspace_size(C.byref(kv), 32) > 0) == ok
        if not ok:
            assert set(_calls(lib, abi, kv).values()) == {abi.SA_ERR_UNSUPPORTED}


class _Stub:
    """A library that only notes which of its calls were reached."""

    def __init__(self, real):
        self.real, self.reached = real, []

    def __getattr__(self, name):
        if name.endswith("_size") or name.endswith("_string"):
            return getattr(self.real, name)
        return lambda *a: self.reached.append(name) or 0


def test_binding_refuses_tensors_in_host_memory(monkeypatch):
    """A forgotten .to("cuda") is an error here, not an illegal access there."""
    import block_sparse_kv_page_b200 as sa
    from block_sparse_kv_page_b200 import ops
    stub = _Stub(ops.lib)
    monkeypatch.setattr(ops, "lib", stub)
    c = _cache()
    off = torch.zeros(4, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: sa.sparse_attn_cache_write(c, bf(4, 2, 128), bf(4, 2, 128), off, stream=0),
                 lambda: sa.sparse_attn_cache_write(c, bf(0, 2, 128), bf(0, 2, 128), off, ws, stream=0),
                 lambda: sa.sparse_attn_cache_read(c, 0, bf(3, 2, 32, 128), bf(3, 2, 32, 128), stream=0),
                 lambda: sa.sparse_attn_chunk(c, bf(4, 4, 128), off, 0.1, 0, 0, bf(4, 4, 128), None, ws, stream=0),
                 lambda: sa.sparse_attn_paged_decode(c, bf(3, 4, 128), 0.1, 0, 0, bf(3, 4, 128), None, ws, stream=0),
                 lambda: sa.make_paged_workspace(c, 4, stream=0)):
        with pytest.raises(ValueError):
            call()
    assert not stub.reached


@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 16, -(1 << 31) - 1, 10 ** 12])
def test_binding_refuses_numbers_past_32_bits(value):
    """ctypes would keep their low 32 bits: a window of 2^32 + 16 would be 16."""
    import block_sparse_kv_page_b200 as sa
    c = _cache()
    off = torch.zeros(4, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    for call in (lambda: sa.sparse_attn_cache_read(c, value, bf(3, 2, 32, 128), bf(3, 2, 32, 128)),
                 lambda: sa.sparse_attn_chunk(c, bf(4, 4, 128), off, 0.1, value, 0, bf(4, 4, 128), None, None),
                 lambda: sa.sparse_attn_chunk(c, bf(4, 4, 128), off, 0.1, 5, value, bf(4, 4, 128), None, None),
                 lambda: sa.sparse_attn_paged_decode(c, bf(3, 4, 128), 0.1, value, 0, bf(3, 4, 128), None, None),
                 lambda: sa.sparse_attn_paged_decode(c, bf(3, 4, 128), 0.1, 5, value, bf(3, 4, 128), None, None)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_workspace_calls_run_on_the_workspace_s_device(monkeypatch):
    """Status and initialisation of a workspace on a device that is not the
    current one: on that device's current stream, behind its calls."""
    import block_sparse_kv_page_b200 as sa
    from block_sparse_kv_page_b200 import ops
    seen, now = [], [0]

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, now[0], a[-1])) or 0

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.was, now[0] = now[0], self.index

        def __exit__(self, *e):
            now[0] = self.was

    class Workspace:
        def __init__(self, index):
            self.index = index

        def get_device(self):
            return self.index

        def data_ptr(self):
            return 0x100

        def numel(self):
            return 512

        def element_size(self):
            return 1

    monkeypatch.setattr(ops, "lib", Lib())
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("S", (), {"cuda_stream": 700 + now[0]}))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 700 + i, raising=False)
    for index in (0, 1):
        sa.sparse_attn_workspace_init(Workspace(index))
        assert sa.sparse_attn_get_device_status(Workspace(index)) == 0
        assert sa.sparse_attn_get_device_status(Workspace(index), 5) == 0
    assert [(d, s) for _, d, s in seen] == [(0, 700), (0, 700), (0, 5), (1, 701), (1, 701), (1, 5)]
