"""GPU parity of the paged KV cache's writes and reads (fak_kv_append, fak_kv_read): RMSNorm, RoPE, quantisation and
paging against the same steps in 64 bits.

Bars.  A vector after norm and RoPE in f32 is off by at most 2^-20 of its largest magnitudes (a few roundings, the
rotary pair mixes two elements): a bf16 code by 2^-8 of itself more, an e4m3 code by half its step (2^-4 of itself, or
2^-10 scales below the normal range), an int8 code by half a scale.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import _kv

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "i8"]


@pytest.fixture(scope="module")
def fak():
    from q4_weight_quantized_block_gb300 import build
    build.build()
    import q4_weight_quantized_block_gb300 as m
    assert torch.cuda.is_available()
    return m


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def transformed(x, w, pos, rot, theta, eps):
    """RMSNorm with gain w (None: none), then RoPE, in 64 bits.  x [n, heads, dh], pos [n]."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if rot:
        h = rot // 2
        ang = pos.double()[:, None] * theta ** (-2.0 * torch.arange(h, device=x.device, dtype=torch.float64) / rot)
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        a, b = x[..., :h], x[..., h:rot]
        x = torch.cat([a * c - b * s, b * c + a * s, x[..., rot:]], -1)
    return x


def append_case(fak, kind, nq, n_kv, dh, page, lengths, rot, norm, dtype, seed, theta=1e7, pad_rows=0):
    table, start, kv_len, rows, n_pages = _kv.batch_tensors(lengths, page, seed=seed, pad_rows=pad_rows)
    cache, mem = _kv.empty_cache(fak, kind, n_pages, n_kv, page, dh)
    batch = fak.KVBatch(table, start, kv_len)
    t = randn(seed, rows, (2 * nq + 2 * n_kv) * dh).to(dtype)
    q = t[:, :2 * nq * dh].view(rows, nq, 2 * dh)[..., :dh] if nq else None
    k = t[:, 2 * nq * dh:(2 * nq + n_kv) * dh].view(rows, n_kv, dh)
    v = t[:, (2 * nq + n_kv) * dh:].view(rows, n_kv, dh)
    qw, kw = (1 + 0.1 * randn(seed + 1, dh), 1 + 0.1 * randn(seed + 2, dh)) if norm else (None, None)
    rope = torch.from_numpy(fak.fak_rope_table(rot, theta)).cuda() if rot else None
    q_out = torch.full((rows, nq, dh), 7.0, dtype=torch.bfloat16, device="cuda") if nq else None
    fak.fak_kv_append(cache, batch, k, v, q=q, q_out=q_out, q_norm_w=qw, k_norm_w=kw, eps=1e-6, rope=rope, rot=rot)
    before = [None if m is None else m.clone() for m in mem]
    assert fak.fak_device_status() == 0
    touched = torch.zeros(n_pages, page, dtype=torch.bool)
    written = torch.zeros(rows, dtype=torch.bool)
    for (r, pg, sl), (n, total) in zip(_kv.places(table, start, kv_len, page), lengths):
        touched[pg, sl] = True
        written[r] = True
        r = r.cuda()
        pos = torch.arange(total - len(r), total, device="cuda")
        wk, wv = transformed(k[r], kw, pos, rot, theta, 1e-6), transformed(v[r], None, pos, 0, theta, 1e-6)
        gk, gv = _kv.held(mem, kind, pg, sl)
        for got, want, what in ((gk, wk, "k"), (gv, wv, "v")):
            big = want.abs().amax(-1, keepdim=True)
            tol = 2.0**-20 * big
            if kind == "bf16":
                tol = tol + 2.0**-8 * want.abs()
            elif kind == "e4m3":
                tol = tol + torch.maximum(2.0**-4 * want.abs(), 2.0**-10 * big / 448)
            else:
                tol = tol + big / 127 / 2
            _kv.check(got, want, tol, what)
        if nq:
            want = transformed(q[r], qw, pos, rot, theta, 1e-6)
            _kv.check(q_out[r], want, 2.0**-20 * want.abs().amax(-1, keepdim=True) + 2.0**-8 * want.abs(), "q")
    # every other place of the cache and row of q_out is as it was
    fresh = _kv.empty_cache(fak, kind, n_pages, n_kv, page, dh)[1]
    keep = (~touched).cuda()
    for m, f in zip(before, fresh):
        if m is not None:
            a, b = m.transpose(1, 2)[keep], f.transpose(1, 2)[keep]
            assert torch.equal(a.nan_to_num(-5) if a.is_floating_point() else a, b.nan_to_num(-5) if b.is_floating_point() else b)
    if nq and not written.all():
        assert bool((q_out[(~written).cuda()] == 7.0).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dh,nq,n_kv,rot", [(256, 24, 4, 64), (128, 8, 2, 128), (64, 3, 1, 16), (256, 5, 5, 256)])
def test_append_norm_rope(fak, kind, dh, nq, n_kv, rot):
    append_case(fak, kind, nq, n_kv, dh, 16, [(1, 1), (5, 40), (0, 9), (17, 17)], rot, True, torch.float32, 10 + dh)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dh", [64, 128, 256])
def test_append_plain_keys_and_values(fak, kind, dtype, dh):
    append_case(fak, kind, 0, 3, dh, 32, [(33, 70), (1, 64)], 0, False, dtype, 20 + dh)


def test_append_many_rows_and_sequences(fak):
    # more rows than SMs (four vectors to a warp), more sequences than one round of the search
    lengths = [(1 + 7 * (i % 3), 20 + i) for i in range(70)]
    append_case(fak, "e4m3", 24, 4, 256, 64, lengths, 64, True, torch.float32, 30)
    append_case(fak, "bf16", 2, 1, 128, 16, lengths, 32, True, torch.bfloat16, 31)


def test_append_padding_rows_are_left_alone(fak):
    # the second sequence has three more rows than positions; five rows belong to no sequence
    append_case(fak, "i8", 4, 2, 128, 16, [(2, 30), (8, 5), (1, 1)], 32, True, torch.float32, 32, pad_rows=5)


def test_rope_at_far_positions(fak):
    # position 10^6 with theta 10^4: a million radians in f32 would be off by 0.03
    append_case(fak, "bf16", 2, 1, 64, 256, [(3, 1000003)], 64, False, torch.float32, 33, theta=1e4)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_append_extreme_vectors(fak, kind):
    dh, page = 128, 16
    table, start, kv_len, rows, n_pages = _kv.batch_tensors([(7, 7)], page)
    cache, mem = _kv.empty_cache(fak, kind, n_pages, 1, page, dh)
    x = randn(40, 7, 1, dh)
    x[0] = 0
    x[1] *= 1e-33  # below 2^-100
    x[2] *= 1e30
    x[3, 0, 5] = float("nan")
    x[4, 0, 6] = -float("inf")
    x[5] *= 1e-25
    fak.fak_kv_append(cache, fak.KVBatch(table, start, kv_len), x, x.clone())
    k_out, v_out = (torch.full((7, 1, dh), 3.0, device="cuda") for _ in range(2))
    fak.fak_kv_read(cache, fak.KVBatch(table, start, kv_len), k_out, v_out)
    assert fak.fak_device_status() == 0
    for got in (k_out, v_out):
        assert bool((got[:2] == 0).all())
        assert bool(torch.isnan(got[3:5]).all())
        for r in (2, 5, 6):
            big = x[r].double().abs().amax()
            tol = torch.maximum(2.0**-4 * x[r].double().abs(), 2.0**-10 * big / 448) if kind == "e4m3" else big / 254
            _kv.check(got[r], x[r].double(), tol + 2.0**-20 * big, "row %d" % r)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dh,n_kv,page", [(256, 4, 64), (128, 1, 16), (64, 5, 256)])
def test_read(fak, kind, dtype, dh, n_kv, page):
    lengths = [(40, 40), (0, 12), (3, 700), (1, 1), (6, 4)]  # the last with two padding rows
    table, start, kv_len, rows, n_pages = _kv.batch_tensors(lengths, page, seed=3, pad_rows=2)
    cache, mem = _kv.empty_cache(fak, kind, n_pages, n_kv, page, dh)
    K = [randn(50 + i, t, n_kv, dh) for i, (_, t) in enumerate(lengths)]
    V = [randn(60 + i, t, n_kv, dh) for i, (_, t) in enumerate(lengths)]
    _kv.fill(mem, kind, table, kv_len, page, K, V)
    k_out, v_out = (torch.full((rows, n_kv, dh), 9.0, dtype=dtype, device="cuda") for _ in range(2))
    fak.fak_kv_read(cache, fak.KVBatch(table, start, kv_len), k_out, v_out)
    assert fak.fak_device_status() == 0
    for r, pg, sl in _kv.places(table, start, kv_len, page):
        for got, want in zip((k_out, v_out), _kv.held(mem, kind, pg, sl)):
            _kv.check(got[r.cuda()], want, (2.0**-24 if dtype == torch.float32 else 2.0**-8 + 2.0**-23) * want.abs(), "read")
    first = int(start[4])
    for got in (k_out, v_out):
        assert bool((got[first:first + 2] == 0).all())  # negative positions
        assert bool((got[int(start[-1]):] == 9.0).all())
    only = torch.empty_like(k_out)
    fak.fak_kv_read(cache, fak.KVBatch(table, start, kv_len), None, only)
    assert torch.equal(only[:int(start[-1])], v_out[:int(start[-1])])


def test_bad_numbers_are_recorded_and_left_out(fak):
    dh, page, n_kv = 64, 16, 2
    lengths = [(4, 20), (4, 20), (4, 20)]
    table, start, kv_len, rows, n_pages = _kv.batch_tensors(lengths, page)
    K = [randn(70 + i, 20, n_kv, dh) for i in range(3)]
    cache, mem = _kv.empty_cache(fak, "bf16", n_pages, n_kv, page, dh)
    _kv.fill(mem, "bf16", table, kv_len, page, K, K)
    new = randn(73, rows, n_kv, dh)
    good = torch.full((rows, n_kv, dh), 9.0, device="cuda")
    fak.fak_kv_read(cache, fak.KVBatch(table, start, kv_len), good, None)
    for change in ("len", "negative", "start", "page"):
        t, st, ln = table.clone(), start.clone(), kv_len.clone()
        if change == "len":
            ln[1] = 33  # two pages a sequence
        elif change == "negative":
            ln[1] = -1
        elif change == "start":
            st[3] = rows + 1
        else:
            t[1, 1] = -1
        b = fak.KVBatch(t, st, ln)
        out = torch.full((rows, n_kv, dh), 9.0, device="cuda")
        fak.fak_kv_read(cache, b, out, None)
        assert fak.fak_device_status() == 7, change
        left = slice(8, 12) if change == "start" else slice(4, 8)
        ok = [r for r in range(12) if not left.start <= r < left.stop]
        assert torch.equal(out[ok], good[ok]), change
        assert bool((out[left] == 9.0).all()) or change == "page"
        was = [None if m is None else m.clone() for m in mem]
        fak.fak_kv_append(cache, b, new, new)
        assert fak.fak_device_status() == 7, change
        after = torch.empty_like(good)
        fak.fak_kv_read(cache, fak.KVBatch(table, start, kv_len), after, None)
        assert torch.equal(after[left], good[left]), change
        assert torch.equal(after[ok], new[ok].to(torch.bfloat16).float()), change
        mem[0].copy_(was[0])
        mem[1].copy_(was[1])
    assert fak.fak_device_status() == 0


def test_offsets_past_32_bits(fak):
    # 10.2M vectors of 256 in bf16: 5.2 GB of keys; the sequence's pages stand at both ends
    dh, page, n_pages = 256, 256, 40000
    k = torch.empty(n_pages, 1, page, dh, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    cache = fak.KVCache(fak.FAK_KV_BF16, k, v)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2]], dtype=torch.int32, device="cuda")
    b = fak.KVBatch(table, torch.tensor([0, 600], dtype=torch.int32, device="cuda"), torch.tensor([600], dtype=torch.int32, device="cuda"))
    x, y = randn(80, 600, 1, dh).to(torch.bfloat16), randn(81, 600, 1, dh).to(torch.bfloat16)
    fak.fak_kv_append(cache, b, x, y)
    assert torch.equal(k[n_pages - 1, 0], x[:256, 0]) and torch.equal(v[n_pages - 2, 0, :88], y[512:, 0])
    a, c = torch.empty_like(x), torch.empty_like(y)
    fak.fak_kv_read(cache, b, a, c)
    assert fak.fak_device_status() == 0
    assert torch.equal(a, x) and torch.equal(c, y)
    q = randn(82, 600, 2, dh).to(torch.bfloat16)
    out = torch.empty_like(q)
    n = fak.fak_paged_attn_workspace_bytes(cache, b, 2, 600, 600, 600)
    fak.fak_paged_attn(cache, b, q, out, 600, 600, workspace=torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"))
    assert fak.fak_device_status() == 0
    want, tol = _kv.attention(q, x.double(), y.double(), 0, dh**-0.5)
    _kv.check(out, want, tol, "attention over far pages")
    assert math.isfinite(float(out.float().sum()))


def test_int8_codes_bit_for_bit(fak):
    """No norm, no RoPE: rint(x * (127 * (1 / a))) in f32, to the last code."""
    lengths = [(700, 700), (300, 333)]
    table, start, kv_len, rows, n_pages = _kv.batch_tensors(lengths, 64, seed=4)
    cache, mem = _kv.empty_cache(fak, "i8", n_pages, 4, 64, 256)
    k, v = randn(41, rows, 4, 256), randn(42, rows, 4, 256) * 1e-3
    fak.fak_kv_append(cache, fak.KVBatch(table, start, kv_len), k, v)
    assert fak.fak_device_status() == 0
    t, row = table.cpu(), 0
    for s, (n, total) in enumerate(lengths):
        pos = torch.arange(total - n, total)
        pages, slots = t[s, pos // 64].long().cuda(), (pos % 64).cuda()
        for codes, x in ((mem[0], k), (mem[1], v)):
            x = x[row:row + n]
            inv = torch.ones_like(x[..., 0]).div(x.abs().amax(-1)).mul(127.0)
            assert torch.equal(codes[pages, :, slots], (x * inv[..., None]).round().to(torch.int8))
        row += n



@pytest.mark.parametrize("bad", [1000, -5])
@pytest.mark.parametrize("n,new", [(4, 3), (31, 1), (32, 1), (70, 3)])
def test_a_bad_start_leaves_out_its_own_sequences_only(fak, n, new, bad):
    dh, page, n_kv, total = 64, 16, 2, 20
    table, start, kv_len, rows, n_pages = _kv.batch_tensors([(new, total)] * n, page, pad_rows=2)
    cache, mem = _kv.empty_cache(fak, "bf16", n_pages, n_kv, page, dh)
    good = fak.KVBatch(table, start, kv_len)
    old, x, q = randn(90, rows, n_kv, dh), randn(91, rows, n_kv, dh), randn(92, rows, n_kv, dh)
    fak.fak_kv_append(cache, good, old, old)
    i = n // 2 // 2 * 2
    st = start.clone()
    st[i] = bad if bad < 0 else rows + bad  # sequences i - 1 and i
    broken = fak.KVBatch(table, st, kv_len)
    ok = [r for r in range(n * new) if not (i - 1) * new <= r < (i + 1) * new]
    left = [r for r in range(n * new) if r not in ok]
    assert fak.fak_device_status() == 0
    got = torch.full((rows, n_kv, dh), 9.0, device="cuda")
    fak.fak_kv_read(cache, broken, got, None)
    assert fak.fak_device_status() == 7
    assert torch.equal(got[ok], old[ok].to(torch.bfloat16).float())
    assert bool((got[left] == 9.0).all()) and bool((got[n * new:] == 9.0).all())
    q_out = torch.full((rows, n_kv, dh), 9.0, dtype=torch.bfloat16, device="cuda")
    fak.fak_kv_append(cache, broken, x, x, q=q, q_out=q_out)
    assert fak.fak_device_status() == 7
    fak.fak_kv_read(cache, good, got, None)
    assert fak.fak_device_status() == 0
    assert torch.equal(got[ok], x[ok].to(torch.bfloat16).float()) and torch.equal(got[left], old[left].to(torch.bfloat16).float())
    assert torch.equal(q_out[ok], q[ok].to(torch.bfloat16))
    assert bool((q_out[left] == 9.0).all()) and bool((q_out[n * new:] == 9.0).all())


def test_rope_near_whole_quarters_of_a_turn(fak):
    """The rotation of (1, 0) is (cos, sin): next to a multiple of a quarter turn one of them is small, and as good as it
    would be next to zero.  An angle less the quarters is off by 2^-24 of itself, a sine or cosine by 2 units in the last
    place, 2^-22 of itself; the result is rounded to bf16, 2^-8 of itself."""
    dh, n_kv, rows = 64, 1, 9
    g = torch.Generator().manual_seed(5)
    # fractions of a turn: quarters plus up to 2^-10 .. 2^-30 of a turn, as 64-bit integers that wrap
    off = (torch.rand(32, generator=g, dtype=torch.float64) - 0.5) * 2.0 ** (54 - torch.arange(32, dtype=torch.float64) % 21)
    turn = off.round().to(torch.int64) + ((torch.arange(32, dtype=torch.int64) % 4) << 62)
    table, start, kv_len, _, n_pages = _kv.batch_tensors([(rows, rows)], 16)
    cache, mem = _kv.empty_cache(fak, "bf16", n_pages, n_kv, 16, dh)
    k = torch.zeros(rows, n_kv, dh, device="cuda")
    k[..., :32] = 1.0
    fak.fak_kv_append(cache, fak.KVBatch(table, start, kv_len), k, k.clone(), rope=turn.cuda(), rot=64)
    assert fak.fak_device_status() == 0
    (r, pg, sl), = _kv.places(table, start, kv_len, 16)
    got, _ = _kv.held(mem, "bf16", pg, sl)
    angle = turn * torch.arange(rows)[:, None]  # wraps at whole turns
    quarter = (angle + (1 << 61)) >> 62
    rest = (angle - (quarter << 62)).double() * (2.0 * math.pi / 2.0**64)
    c, s = torch.cos(rest), torch.sin(rest)
    q = quarter % 4
    cos = torch.where(q == 0, c, torch.where(q == 1, -s, torch.where(q == 2, -c, s)))
    sin = torch.where(q == 0, s, torch.where(q == 1, c, torch.where(q == 2, -s, -c)))
    want = torch.cat([cos, sin], -1)[:, None].cuda()
    _kv.check(got, want, (2.0**-8 + 2.0**-22) * want.abs(), "cosines and sines")
