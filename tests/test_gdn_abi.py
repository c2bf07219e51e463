"""Host-side refusals of the Gated DeltaNet operators and the norm around a block, before any device call (no GPU needed)."""
import ctypes
import math

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
    batch = L.GdnBatchDesc(3, OK, OK, OK)
    rows = L.GdnRows(0, 16, 48, 9, 1e-6, 10, OK, OK, OK, 16480, 16480, 16480, OK, OK, OK, OK, OK, OK, OK, OK, OK)
    args = L.GdnArgs(16, 48, 4, 1, 9, 0.1, 1e-6, 10, OK, OK, OK, 2048, 128, 2048, 128, 6144, 128, OK, OK, OK, OK, OK, 6144, 128, OK,
                     6144, 128)
    norm = L.NormArgs(0, 0, 1, 5120, 1, 0, 1.0, 1e-6, 0.0, 10, OK, OK, OK, 5120, 5120, 5120, OK, OK, OK, 5120, 1)
    return batch, rows, args, norm


def ref(x):
    return None if x is None else ctypes.addressof(x)


BAD_BATCH = [("n_seqs", -1, 2), ("row_start", None, 1), ("kv_len", None, 1), ("slot", None, 1), ("slot", OK + 2, 3),
             ("row_start", OK + 1, 3)]
BAD_ROWS = [("type", 2, 1), ("type", -1, 1), ("nk", 0, 2), ("nv", 0, 2), ("nv", -3, 2), ("n_slots", 0, 2), ("rows", -1, 2), ("rows", 1 << 31, 2),
            ("eps", -1.0, 1), ("eps", math.nan, 1)]
BAD_ROWS += [(f, None, 1) for f in ("x", "b", "a", "conv_w", "a_log", "dt_bias", "conv_state", "q", "k", "v", "g", "beta")]
BAD_ROWS += [(f, OK + 8, 3) for f in ("conv_w", "conv_state", "q", "k", "v")]
BAD_ROWS += [(f, OK + 2, 3) for f in ("x", "b", "a", "a_log", "dt_bias", "g", "beta")]
BAD_ARGS = [("nk", 0, 2), ("nv", 0, 2), ("nv", 40, 2), ("max_q", -1, 2), ("out_type", 2, 1), ("n_slots", 0, 2), ("scale", 0.0, 1),
            ("scale", -1.0, 1), ("scale", math.inf, 1), ("scale", math.nan, 1), ("eps", -1.0, 1), ("rows", -1, 2), ("rows", 1 << 31, 2)]
BAD_ARGS += [(f, None, 1) for f in ("q", "k", "v", "g", "beta", "state", "out")]
BAD_ARGS += [(f, OK + 8, 3) for f in ("q", "k", "v", "state", "norm_w", "out")] + [(f, OK + 2, 3) for f in ("g", "beta", "z")]
BAD_ARGS += [(f, 2052, 3) for f in ("q_row", "k_row", "v_row", "out_row", "q_head", "k_head", "v_head", "out_head")]
BAD_NORM = [("h_type", 2, 1), ("y_type", -1, 1), ("n_type", 3, 1), ("d", 0, 2), ("d", 32769, 2), ("gate_kind", 2, 1), ("scale", math.inf, 1),
            ("scale", math.nan, 1), ("eps", -1.0, 1), ("gain_offset", math.nan, 1), ("rows", -1, 2), ("rows", 1 << 31, 2), ("h", None, 1),
            ("h", OK + 2, 3), ("y", OK + 2, 3), ("n", OK + 1, 3), ("w", OK + 2, 3), ("y_w", OK + 1, 3), ("gate", OK + 2, 3),
            ("gate_col", 2, 1)]


@pytest.mark.parametrize("which,table", [("batch", BAD_BATCH), ("rows", BAD_ROWS), ("args", BAD_ARGS), ("norm", BAD_NORM)])
def test_bad_arguments(fak, which, table):
    conv = lambda b, r, a, n: fak.lib.fak_gdn_conv(ref(b), ref(r), None)  # noqa: E731
    attn = lambda b, r, a, n: fak.lib.fak_gdn_attn(ref(b), ref(a), None)  # noqa: E731
    norm = lambda b, r, a, n: fak.lib.fak_residual_norm(ref(n), None)  # noqa: E731
    i, calls = {"batch": (0, (conv, attn)), "rows": (1, (conv,)), "args": (2, (attn,)), "norm": (3, (norm,))}[which]
    for field, value, status in table:
        for call in calls:
            s = structs()
            setattr(s[i], field, value)
            assert call(*s) == status, (field, value)
    for call in calls:
        s = list(structs())
        s[i] = None
        assert call(*s) == 1


def test_too_many_heads(fak):
    b, r, a, n = structs()
    b.n_seqs = 1 << 27
    assert fak.lib.fak_gdn_attn(ref(b), ref(a), None) == 2


def test_nothing_to_do_is_fine(fak):
    b, r, a, n = structs()
    r.rows = a.rows = n.rows = 0
    r.x = r.q = a.q = a.out = n.h = None
    assert fak.lib.fak_gdn_conv(ref(b), ref(r), None) == 0 and fak.lib.fak_gdn_attn(ref(b), ref(a), None) == 0
    assert fak.lib.fak_residual_norm(ref(n), None) == 0
    b, r, a, n = structs()
    b.n_seqs, b.row_start, b.kv_len, b.slot = 0, None, None, None
    assert fak.lib.fak_gdn_conv(ref(b), ref(r), None) == 0 and fak.lib.fak_gdn_attn(ref(b), ref(a), None) == 0
    n.y = n.n = None
    assert fak.lib.fak_residual_norm(ref(n), None) == 0


def test_strides_of_single_rows_and_heads_are_not_looked_at(fak):
    """(They would be refused for their alignment before the device is looked at.)"""
    b, r, a, n = structs()
    a.rows = a.nk = a.nv = r.rows = 1
    for f in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head", "z_row", "z_head", "out_row", "out_head"):
        setattr(a, f, 3)
    r.x_row = 3
    b.n_seqs = 0  # no launch
    assert fak.lib.fak_gdn_attn(ref(b), ref(a), None) == 0 and fak.lib.fak_gdn_conv(ref(b), ref(r), None) == 0


def test_debug_wait_refuses(fak):
    for args in ((-1, 0), (0, 2), (1000, -1)):
        assert fak.lib.fak_gdn_debug_wait(*args) == 1
    assert fak.lib.fak_gdn_debug_wait(0, 0) == 0


def test_binding_refuses_wrong_tensors(fak):
    torch = pytest.importorskip("torch")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    for bad in ((i32(3), i32(2), i32(3)), (i32(3), i32(1), i32(2)), (i32(3).long(), i32(2), i32(2)), (i32(6)[::2], i32(2), i32(2))):
        with pytest.raises(fak.FakError):
            fak.GDNBatch(*bad)
    batch = fak.GDNBatch(i32(3), i32(2), i32(2))
    f16, bf16 = torch.float16, torch.bfloat16
    good = dict(q=torch.zeros(5, 2, 128, dtype=f16), k=torch.zeros(5, 2, 128, dtype=f16), v=torch.zeros(5, 4, 128, dtype=bf16),
                g=torch.zeros(5, 4), beta=torch.zeros(5, 4), state=torch.zeros(3, 4, 128, 128), out=torch.zeros(5, 4, 128))
    opt = dict(z=torch.zeros(5, 4, 128), norm_w=torch.zeros(128))
    bad = [("q", good["q"].float()), ("q", good["q"][:4]), ("k", good["k"][..., :64]), ("k", good["k"].to(bf16)), ("v", good["v"].half()),
           ("v", good["v"][..., ::2]), ("g", good["g"][:, :3]), ("g", good["g"].half()), ("beta", good["beta"].T), ("state", good["state"][:, :2]),
           ("state", good["state"].half()), ("state", good["state"].transpose(2, 3)), ("out", good["out"].half()), ("out", good["out"][:, :3]),
           ("z", opt["z"].to(bf16)), ("z", opt["z"][:3]), ("norm_w", torch.zeros(64)), ("norm_w", torch.zeros(128).half())]
    def attn(batch, q, k, v, g, beta, state, out, **more):
        fak.fak_gdn_attn(batch, q, k, v, g, beta, state, out, 2, stream=0, **more)
    for name, t in bad:
        with pytest.raises(fak.FakError) as e:
            attn(batch, **{**good, **opt, name: t})
        assert e.value.status in (1, 2), name
    with pytest.raises(fak.FakError) as e:  # tensors of the host
        attn(batch, **good, **opt)
    assert e.value.status == 8
    good = dict(x=torch.zeros(5, 1024), b=torch.zeros(5, 4), a=torch.zeros(5, 4), conv_w=torch.zeros(1024, 4), a_log=torch.zeros(4),
                dt_bias=torch.zeros(4), conv_state=torch.zeros(3, 3, 1024), q=torch.zeros(5, 2, 128, dtype=f16),
                k=torch.zeros(5, 2, 128, dtype=f16), v=torch.zeros(5, 4, 128, dtype=bf16), g=torch.zeros(5, 4), beta=torch.zeros(5, 4))
    bad = [("x", good["x"].half()), ("x", good["x"][:, :1000]), ("b", good["b"].to(bf16)), ("a", good["a"][:4]), ("conv_w", torch.zeros(4, 1024).T),
           ("a_log", torch.zeros(3)), ("dt_bias", torch.zeros(4).double()), ("conv_state", torch.zeros(3, 4, 1024)), ("q", good["q"].float()),
           ("k", good["k"][:, :1]), ("v", good["v"].half()), ("g", good["g"].T), ("beta", good["beta"][:, :2])]
    for name, t in bad:
        with pytest.raises(fak.FakError) as e:
            fak.fak_gdn_conv(batch, **{**good, name: t}, stream=0)
        assert e.value.status in (1, 2), name
    with pytest.raises(fak.FakError) as e:
        fak.fak_gdn_conv(batch, **good, stream=0)
    assert e.value.status == 8
    h = torch.zeros(5, 64)
    for over in (dict(y=h[:4]), dict(y=h.half()), dict(y=torch.zeros(5, 128)[:, ::2]), dict(n=h.double()), dict(w=torch.zeros(63)),
                 dict(w=torch.zeros(64).half()), dict(gate=h.to(bf16)), dict(gate=torch.zeros(5, 128)[:, ::2]), dict(gate=h[:, :1])):
        with pytest.raises(fak.FakError) as e:
            fak.fak_residual_norm(h, **{**dict(y=h, n=h), **over}, stream=0)
        assert e.value.status in (1, 2), over
    with pytest.raises(fak.FakError) as e:
        fak.fak_residual_norm(h, h, h, stream=0)
    assert e.value.status == 8
