"""Host-side refusals of the paged KV cache and the attention over it, before any device call (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

OK = 1 << 20  # 16-byte aligned, never dereferenced: the checks come first


@pytest.fixture(scope="module")
def fak():
    from q4_weight_quantized_block_gb300 import build
    build.build()
    import q4_weight_quantized_block_gb300 as m
    return m


def structs():
    from q4_weight_quantized_block_gb300 import _lib as L
    cache = L.KvCacheDesc(1, 4, 256, 64, 100, OK, OK, OK, OK)
    batch = L.KvBatchDesc(2, 8, OK, OK, OK)
    rows = L.KvRows(0, 24, 64, 1e-6, 10, OK, OK, OK, 512 * 24, 512, 1024, 256, 1024, 256, OK, OK, OK, OK)
    args = L.AttnArgs(24, 0, 0, 4, 512, 0.0625, 10, OK, 6144, 256, OK, 12288, 512, OK, 6144, 256, OK, 1 << 40)
    return cache, batch, rows, args


def ref(x):
    return None if x is None else ctypes.addressof(x)


BAD_CACHE = [("kind", 3, 1), ("kind", -1, 1), ("k", None, 1), ("v", None, 1), ("k_scale", None, 1), ("v_scale", None, 1),
             ("dh", 96, 2), ("dh", 512, 2), ("page", 8, 2), ("page", 48, 2), ("page", 512, 2), ("n_kv", 0, 2),
             ("n_pages", 0, 2), ("n_pages", 1 << 31, 2), ("n_pages", 1 << 23, 2), ("k", OK + 8, 3), ("v", OK + 4, 3),
             ("v_scale", OK + 2, 3)]
BAD_BATCH = [("n_seqs", -1, 2), ("max_pages", 0, 2), ("page_table", None, 1), ("row_start", None, 1), ("kv_len", None, 1),
             ("kv_len", OK + 2, 3)]
BAD_ROWS = [("type", 2, 1), ("nq", -1, 2), ("rows", -1, 2), ("rows", 1 << 31, 2), ("rot", 24, 2), ("rot", 272, 2),
            ("rot", -16, 2), ("k", None, 1), ("v", None, 1), ("q", None, 1), ("q_out", None, 1), ("rope", None, 1),
            ("eps", -1.0, 1), ("eps", math.nan, 1), ("q_head", 510, 3), ("k_row", 1026, 3), ("v_head", 2, 3),
            ("q", OK + 4, 3), ("q_out", OK + 8, 3), ("k_norm_w", OK + 4, 3), ("rope", OK + 4, 3)]
BAD_ARGS = [("nq", 0, 2), ("nq", 22, 2), ("nq", 4 * 129, 2), ("window", -1, 1), ("sinks", -1, 1), ("scale", 0.0, 1),
            ("scale", -1.0, 1), ("scale", math.inf, 1), ("scale", math.nan, 1), ("rows", -1, 2), ("rows", 1 << 31, 2),
            ("max_q", -1, 2), ("max_kv", -1, 2), ("max_kv", (1 << 30) + 1, 2), ("q", None, 1), ("out", None, 1),
            ("q", OK + 8, 3), ("out", OK + 2, 3), ("gate", OK + 4, 3), ("q_row", 6145, 3), ("out_head", 252, 3),
            ("gate_head", 513, 3), ("workspace", OK + 16, 3)]


def calls(fak):
    lib = fak.lib
    return {"append": lambda c, b, r, a: lib.fak_kv_append(ref(c), ref(b), ref(r), None),
            "read": lambda c, b, r, a: lib.fak_kv_read(ref(c), ref(b), 10, 0, OK, OK, None),
            "attn": lambda c, b, r, a: lib.fak_paged_attn(ref(c), ref(b), ref(a), None)}


@pytest.mark.parametrize("which", ["append", "read", "attn"])
def test_bad_caches_and_batches(fak, which):
    call = calls(fak)[which]
    for i, table in ((0, BAD_CACHE), (1, BAD_BATCH)):
        for field, value, status in table:
            s = structs()
            setattr(s[i], field, value)
            assert call(*s) == status, (which, field, value)
    c, b, r, a = structs()
    assert call(None, b, r, a) == 1 and call(c, None, r, a) == 1


def test_bad_rows(fak):
    for field, value, status in BAD_ROWS:
        s = structs()
        setattr(s[2], field, value)
        assert calls(fak)["append"](*s) == status, (field, value)
    c, b, r, a = structs()
    assert calls(fak)["append"](c, b, None, a) == 1


def test_bad_attention_arguments(fak):
    for field, value, status in BAD_ARGS:
        s = structs()
        setattr(s[3], field, value)
        assert calls(fak)["attn"](*s) == status, (field, value)
    c, b, r, a = structs()
    assert calls(fak)["attn"](c, b, r, None) == 1


def test_bad_reads(fak):
    c, b, _, _ = structs()
    read = fak.lib.fak_kv_read
    assert read(ref(c), ref(b), 10, 2, OK, OK, None) == 1
    assert read(ref(c), ref(b), 10, 0, None, None, None) == 1
    assert read(ref(c), ref(b), -1, 0, OK, OK, None) == 2
    assert read(ref(c), ref(b), 1 << 31, 0, OK, OK, None) == 2
    assert read(ref(c), ref(b), 10, 0, OK + 4, OK, None) == 3


def test_nothing_to_do_is_fine(fak):
    c, b, r, a = structs()
    r.rows = a.rows = 0
    assert calls(fak)["append"](c, b, r, a) == 0 and calls(fak)["attn"](c, b, r, a) == 0
    assert fak.lib.fak_kv_read(ref(c), ref(b), 0, 0, OK, None, None) == 0
    c, b, r, a = structs()
    b.n_seqs = 0
    assert all(call(c, b, r, a) == 0 for call in calls(fak).values())


def test_workspace_size_and_its_check(fak):
    c, b, _, a = structs()
    size = fak.lib.fak_paged_attn_workspace_bytes
    for nulls in ((None, b, a), (c, None, a), (c, b, None)):
        assert size(*(ref(x) for x in nulls)) == 0
    a.nq = 23
    assert size(ref(c), ref(b), ref(a)) == 0
    for new, past in ((1, 100000), (64, 30000)):
        c, b, _, a = structs()
        b.n_seqs, a.max_q, a.max_kv, a.rows = 1, new, past, new
        n = size(ref(c), ref(b), ref(a))
        if n:  # too small a workspace, or none, is refused
            a.workspace_bytes = n - 1
            assert calls(fak)["attn"](c, b, None, a) == 2
            a.workspace, a.workspace_bytes = None, n
            assert calls(fak)["attn"](c, b, None, a) == 1


def test_rope_table(fak):
    t = fak.fak_rope_table(64, 1e7).astype(np.uint64).astype(np.float64) / 2.0**64
    want = 1e7 ** (-2.0 * np.arange(32) / 64) / (2 * math.pi)
    assert np.all(np.abs(t - want) <= want * 2.0**-51 + 2.0**-63)
    for rot, theta, status in ((0, 1e4, 2), (3, 1e4, 2), (258, 1e4, 2), (64, 0.5, 1), (64, math.inf, 1), (64, math.nan, 1)):
        with pytest.raises(fak.FakError) as e:
            fak.fak_rope_table(rot, theta)
        assert e.value.status == status
    assert fak.lib.fak_rope_table(64, 1e4, None) == 1


def test_binding_refuses_wrong_tensors(fak):
    torch = pytest.importorskip("torch")
    u8 = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    sc = torch.zeros(4, 2, 16)
    cache = fak.KVCache(fak.FAK_KV_E4M3, u8, u8, sc, sc)
    for bad in ((fak.FAK_KV_BF16, u8, u8), (fak.FAK_KV_I8, u8, u8[..., :32], sc, sc), (fak.FAK_KV_I8, u8, u8, sc, sc[:2]),
                (fak.FAK_KV_E4M3, u8.transpose(0, 1), u8.transpose(0, 1), None, None)):
        with pytest.raises(fak.FakError):
            fak.KVCache(*bad)
    i32 = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    batch = fak.KVBatch(*i32)
    for bad in ((i32[0], i32[1][:2], i32[2]), (i32[0], i32[1], i32[2].long()), (i32[0].T, i32[1], i32[2])):
        with pytest.raises(fak.FakError):
            fak.KVBatch(*bad)
    x = torch.zeros(5, 2, 64)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    for k, v in ((x[:, :1], x), (x, x[:4]), (x.to(torch.float64), x), (x[..., ::2], x), (x, x.to(torch.bfloat16))):
        with pytest.raises(fak.FakError):
            fak.fak_kv_append(cache, batch, k, v, stream=0)
    with pytest.raises(fak.FakError):
        fak.fak_kv_append(cache, batch, x, x, q=torch.zeros(5, 4, 64), stream=0)
    for a, o in ((q, q[:4]), (q.float(), q.float()), (q[..., ::2], q[..., ::2]), (q, q.float())):
        with pytest.raises(fak.FakError):
            fak.fak_paged_attn(cache, batch, a, o, 1, 1, stream=0)
    with pytest.raises(fak.FakError):
        fak.fak_paged_attn(cache, batch, q, q, 1, 1, gate=q, stream=0)
    for a, o in ((None, None), (x, x[:4]), (x, x.to(torch.bfloat16)), (x.transpose(0, 1), None)):
        with pytest.raises(fak.FakError):
            fak.fak_kv_read(cache, batch, a, o, stream=0)


@pytest.mark.parametrize("field,value", [("q_row", 0), ("q_row", -6144), ("q_head", 0), ("q_head", -256),
                                         ("q_row", (1 << 38) + 8), ("q_head", 1 << 40)])
def test_query_strides_are_positive(fak, field, value):
    c, b, r, a = structs()
    setattr(a, field, value)
    assert calls(fak)["attn"](c, b, r, a) == 2


def test_strides_that_are_never_taken(fak):
    c, b, r, a = structs()
    b.n_seqs = 0  # (nothing to do: no device call)
    r.rows = a.rows = 1
    for x, names in ((r, ("q_row", "k_row", "v_row")), (a, ("q_row", "gate_row", "out_row"))):
        for name in names:
            setattr(x, name, -3)
    assert calls(fak)["append"](c, b, r, a) == 0 and calls(fak)["attn"](c, b, r, a) == 0
    r.rows = a.rows = 2
    assert calls(fak)["append"](c, b, r, a) == 3 and calls(fak)["attn"](c, b, r, a) == 2


def test_more_queries_than_memory_holds(fak):
    c, b, r, a = structs()
    a.nq, a.rows = 65532, (1 << 31) - 1
    c.n_kv = 65532
    assert calls(fak)["attn"](c, b, r, a) == 2
    assert fak.lib.fak_paged_attn_workspace_bytes(ref(c), ref(b), ref(a)) == 0


def test_binding_refuses_other_float_types(fak):
    torch = pytest.importorskip("torch")
    u8, sc = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16)
    cache = fak.KVCache(fak.FAK_KV_I8, u8, u8, sc, sc)
    batch = fak.KVBatch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                        torch.zeros(2, dtype=torch.int32))
    x, q = torch.zeros(5, 2, 64), torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: fak.fak_kv_append(cache, batch, x.half(), x.half(), stream=0),
                 lambda: fak.fak_kv_append(cache, batch, x, x, q=torch.zeros(5, 4, 64), q_out=q.half(), stream=0),
                 lambda: fak.fak_kv_append(cache, batch, x.int(), x.int(), stream=0),
                 lambda: fak.fak_paged_attn(cache, batch, q.half(), q, 1, 1, stream=0),
                 lambda: fak.fak_paged_attn(cache, batch, q, q.half(), 1, 1, stream=0),
                 lambda: fak.fak_paged_attn(cache, batch, q, q, 1, 1, gate=torch.zeros(5, 4, 64, dtype=torch.int32), stream=0),
                 lambda: fak.fak_kv_read(cache, batch, x.half(), None, stream=0)):
        with pytest.raises(fak.FakError) as e:
            call()
        assert e.value.status == 1


def status_of(fak, call):
    try:
        call()
    except fak.FakError as e:
        return e.status
    return 0


def test_binding_looks_at_the_types_of_caches_and_batches(fak):
    torch = pytest.importorskip("torch")
    shape = (4, 2, 16, 64)
    z = lambda dtype, *s: torch.zeros(*(s or shape), dtype=dtype)
    sc = z(torch.float32, *shape[:3])
    u8, i8, f8 = z(torch.uint8), z(torch.int8), z(torch.uint8).view(torch.float8_e4m3fn)
    bf, half, e5 = z(torch.bfloat16), z(torch.float16), z(torch.uint8).view(torch.float8_e5m2)
    bf16, e4m3, int8 = fak.FAK_KV_BF16, fak.FAK_KV_E4M3, fak.FAK_KV_I8
    for good in ((bf16, bf, bf), (e4m3, u8, u8, sc, sc), (e4m3, f8, f8, sc, sc), (int8, i8, i8, sc, sc), (int8, u8, u8, sc, sc)):
        fak.KVCache(*good)
    for bad in ((bf16, half, half), (bf16, bf, half), (bf16, z(torch.int16), z(torch.int16)), (e4m3, e5, e5, sc, sc),
                (e4m3, z(torch.bool), u8, sc, sc), (int8, f8, f8, sc, sc), (int8, i8, i8, sc.int(), sc), (int8, i8, i8, sc, sc.int()),
                (3, u8, u8, sc, sc)):
        assert status_of(fak, lambda: fak.KVCache(*bad)) == 1, bad[0]
    t, s, n = z(torch.int32, 2, 3), z(torch.int32, 3), z(torch.int32, 2)
    fak.KVBatch(t, s, n)
    for bad in ((t.float(), s, n), (t, s.float(), n), (t, s, n.float()), (t, s.view(torch.uint32), n)):
        assert status_of(fak, lambda: fak.KVBatch(*bad)) == 1


def test_binding_looks_at_gains_tables_and_workspaces(fak):
    torch = pytest.importorskip("torch")
    u8, sc = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16)
    cache = fak.KVCache(fak.FAK_KV_I8, u8, u8, sc, sc)
    batch = fak.KVBatch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                        torch.zeros(2, dtype=torch.int32))
    batch.desc.n_seqs = 0  # (nothing to do, whatever is let through)
    x, q = torch.zeros(5, 2, 64), torch.zeros(5, 4, 64)
    out, w = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.ones(64)
    append = lambda **kw: status_of(fak, lambda: fak.fak_kv_append(cache, batch, x, x, q=q, q_out=out, stream=0, **kw))
    for gain, status in ((w.to(torch.bfloat16), 1), (w.double(), 1), (torch.ones(128)[::2], 1), (w[:3], 2), (torch.ones(256), 2),
                         (w[:0], 2), (w[:1].expand(64), 1)):
        assert append(q_norm_w=gain) == status and append(k_norm_w=gain) == status
    rope = torch.zeros(32, dtype=torch.int64)
    for table, status in ((rope[:1], 2), (rope[:31], 2), (rope.double(), 1), (torch.zeros(64, dtype=torch.int32), 1), (rope[:1].expand(32), 1),
                          (torch.zeros(64, dtype=torch.int64)[::2], 1)):
        assert append(rope=table, rot=64) == status
    ws = torch.zeros(1, dtype=torch.uint8).expand(1 << 20)
    assert status_of(fak, lambda: fak.fak_paged_attn(cache, batch, out, out, 1, 1, workspace=ws, stream=0)) == 1


def test_binding_refuses_tensors_of_the_host(fak):
    """The kernels read what they are given on the device: a host tensor (a batch's lengths, say) must not get that far."""
    torch = pytest.importorskip("torch")
    u8, sc = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16)
    cache = fak.KVCache(fak.FAK_KV_I8, u8, u8, sc, sc)
    batch = fak.KVBatch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                        torch.zeros(2, dtype=torch.int32))
    batch.desc.n_seqs = 0  # (nothing to do, whatever is let through)
    x, q = torch.zeros(5, 2, 64), torch.zeros(5, 4, 64)
    out = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    calls = [lambda: fak.fak_kv_append(cache, batch, x, x, q=q, q_out=out, stream=0), lambda: fak.fak_kv_read(cache, batch, x, x, stream=0),
             lambda: fak.fak_paged_attn(cache, batch, out, out, 1, 1, stream=0)]
    for call in calls:
        assert status_of(fak, call) == 8
    # a cache and lengths of device 0, as far as the binding sees, and rows of the host
    cache.device = batch.device = 0
    for call in calls:
        assert status_of(fak, call) == 8
    with pytest.raises(fak.FakError) as e:
        fak.KVBatch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                    torch.zeros(2, dtype=torch.int32, device="meta"))
    assert e.value.status == 8


def test_wait_hooks(fak):
    hook = fak.lib.fak_paged_attn_debug_wait
    assert hook(-1, 0) == 1 and hook(0, 2) == 1 and hook(0, -1) == 1
    assert hook(10**9, 0) == 0 and hook(0, 0) == 0


def test_empty_tensors_have_no_address(fak):
    """A step without rows, or without sequences: torch gives empty tensors the address 0."""
    c, b, r, a = structs()
    r.rows = a.rows = 0
    r.k = r.v = r.q = r.q_out = a.q = a.out = a.gate = None
    assert calls(fak)["append"](c, b, r, a) == 0 and calls(fak)["attn"](c, b, r, a) == 0
    assert fak.lib.fak_kv_read(ref(c), ref(b), 0, 1, None, None, None) == 0
    c, b, r, a = structs()
    b.n_seqs = 0
    b.page_table = b.kv_len = None
    b.max_pages = 0
    assert all(call(c, b, r, a) == 0 for call in calls(fak).values())
    b.n_seqs = 1  # (only then)
    assert all(call(c, b, r, a) == 1 for call in calls(fak).values())
