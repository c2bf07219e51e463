"""fak_gdn_conv and fak_gdn_attn against the rule row by row in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import _gdn as G

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def fak():
    from q4_weight_quantized_block_gb300 import build
    build.build()
    import q4_weight_quantized_block_gb300 as m
    assert torch.cuda.is_available()
    return m


# (new rows, positions in all): single tokens, none, chunks around the sizes that kernels cut at, padding, beginnings
BATCHES = {
    "token": [(1, 9)],
    "first token": [(1, 1)],
    "tokens": [(1, 5), (1, 1), (0, 4), (1, 300), (1, 2)],
    "none": [(0, 3), (0, 0)],
    "drafts": [(4, 10), (4, 4), (2, 100), (5, 5), (7, 9)],
    "padded": [(5, 3), (4, 0), (1, 0), (3, 1), (70, 66), (68, 4)],
    "one chunk": [(64, 64), (64, 100), (63, 63), (17, 18)],
    "chunks": [(65, 65), (128, 130), (129, 129), (200, 1000), (1, 7), (0, 2), (31, 31)],
    "prompt": [(700, 700)],
    "mixed": [(1, 800), (333, 333), (1, 1), (9, 20), (190, 191), (16, 16), (33, 40)],
}


def attn_case(fak, lengths, nk, nv, seed=1, out=torch.bfloat16, z=True, norm=True, wild=False, pad_rows=3, scale=None, views=False,
              max_q=None):
    start, kv_len, slot, rows, slots = G.batch_tensors(lengths, seed, pad_rows)
    q, k, v, g, beta, zz, w = G.inputs(nk, nv, rows, seed, wild=wild)
    state = torch.randn(slots, nv, 128, 128, device="cuda") * 0.3
    for (n, t), s in zip(lengths, slot.tolist()):
        if t <= n:
            state[s] = NAN  # not read
    keep = state.clone()
    o = torch.full((rows, nv, 128), 7.0, dtype=out, device="cuda")
    if views:  # rows and heads of larger tensors
        def view(t, by):
            big = torch.full((t.shape[0], t.shape[1] + 1, 128 + by), NAN, dtype=t.dtype, device="cuda")
            big[:, :t.shape[1], :128] = t
            return big[:, :t.shape[1], :128]
        q, k, v, zz, o = view(q, 8), view(k, 16), view(v, 8), view(zz, 4), view(o, 8)
    batch = fak.GDNBatch(start, kv_len, slot)
    most = max([n for n, _ in lengths]) if max_q is None else max_q
    fak.fak_gdn_attn(batch, q, k, v, g, beta, state, o, most, scale=scale, z=zz if z else None, norm_w=w if norm else None, eps=G.EPS)
    assert fak.fak_device_status() == 0
    sc = 128 ** -0.5 if scale is None else scale
    at = 0
    for (n, t), (first, end, fresh), s in zip(lengths, G.real_rows(lengths), slot.tolist()):
        assert bool((o[at:first] == 0).all())  # padding
        at += n
        if first == end:
            assert torch.equal(state[s].nan_to_num(1e9), keep[s].nan_to_num(1e9))
            continue
        r = slice(first, end)
        S0 = torch.zeros_like(keep[s]) if fresh else keep[s]
        want, S, most = G.gdn_ref(q[r], k[r], v[r], g[r], beta[r], S0, sc)
        # a product of the state is off by 2^-24 of itself in f32, or 2^-22 where it is split over two f16; the rule only
        # shrinks what is there, so the errors of its sums of 128, of either sign, add up over the rows like their root
        tol = 2.0 ** -20 * (end - first) ** 0.5 * max(most, 1e-30)
        err = float((state[s].double() - S).abs().max())
        assert err <= tol, ("state", (n, t), err / tol)
        tol_o = torch.full_like(want, tol * sc)
        if norm:
            tol_o = tol_o / torch.sqrt((want * want).mean(-1, keepdim=True) + G.EPS) * 2 * w.double().abs()
        if z:
            zd = zz[r].double()
            tol_o = tol_o * (zd / (1 + torch.exp(-zd))).abs()
        want = G.gated(want, w if norm else None, zz[r] if z else None)
        tol_o = tol_o + want.abs() * (2.0 ** -18 + torch.finfo(out).eps / 2) + 1e-30
        diff = (o[r].double() - want).abs()
        assert bool((diff <= tol_o).all()), ("out", (n, t), float((diff / tol_o).max()))
    assert bool((o[rows - pad_rows:] == 7).all())  # rows of no sequence
    rest = [i for i in range(slots) if i not in slot.tolist()]
    assert torch.equal(state[rest], keep[rest])


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("nk,nv", [(2, 6), (3, 3)])
def test_attn_lengths(fak, name, nk, nv):
    attn_case(fak, BATCHES[name], nk, nv)


@pytest.mark.parametrize("name", ["tokens", "drafts", "chunks"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("z,norm", [(False, False), (True, False), (False, True)])
def test_attn_outputs(fak, name, out, z, norm):
    attn_case(fak, BATCHES[name], 1, 2, out=out, z=z, norm=norm, scale=0.3, seed=4)


@pytest.mark.parametrize("name", ["tokens", "drafts", "mixed"])
def test_attn_strides(fak, name):
    attn_case(fak, BATCHES[name], 2, 4, views=True, seed=5)


@pytest.mark.parametrize("name", ["drafts", "padded", "chunks", "prompt"])
def test_attn_resets_and_repeated_keys(fak, name):
    """Decays of 0 and -inf, strengths of 0 and 1, the same key twice, values 10^4 times the others."""
    attn_case(fak, BATCHES[name], 2, 2, wild=True, out=torch.float32, seed=6)


def test_attn_many_heads(fak):
    attn_case(fak, [(1, 3)] * 9 + [(2, 2), (130, 131)], 16, 48, seed=7)


def test_attn_large_bound(fak):
    """max_q is a bound: one far above the rows changes nothing that matters."""
    attn_case(fak, BATCHES["drafts"], 1, 3, max_q=100000, seed=8)


def test_attn_split_prompt_goes_on(fak):
    """A prompt in one call, and in pieces with the state between them."""
    n, nk, nv = 300, 2, 4
    q, k, v, g, beta, z, w = G.inputs(nk, nv, n, 11)
    ident = torch.tensor([0], dtype=torch.int32, device="cuda")
    results = []
    for cuts in ([0, n], [0, 1, 64, 65, 70, 200, 201, n]):
        state = torch.full((1, nv, 128, 128), NAN, device="cuda")
        o = torch.empty(n, nv, 128, device="cuda")
        for a, b in zip(cuts, cuts[1:]):
            batch = fak.GDNBatch(torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                                 torch.tensor([b], dtype=torch.int32, device="cuda"), ident)
            fak.fak_gdn_attn(batch, *(t[a:b] for t in (q, k, v, g, beta)), state, o[a:b], b - a, z=z[a:b], norm_w=w)
        results.append((o, state))
    (o1, s1), (o2, s2) = results
    assert fak.fak_device_status() == 0
    tol = 2 * 2.0 ** -20 * n ** 0.5 * float(s1.norm(dim=2).max())
    assert float((s1 - s2).abs().max()) <= tol
    assert float((o1 - o2).norm() / o1.norm()) < 1e-4


def many(n, seed, most=200):
    """Lengths of n sequences: tokens, short and long ones, some with no rows, some that go on, one padded."""
    gen = torch.Generator().manual_seed(seed)
    pick = lambda hi: int(torch.randint(hi, (1,), generator=gen))  # noqa: E731
    out = []
    for _ in range(n):
        rows = (0, 1, 1 + pick(20), 1 + pick(most))[pick(4)]
        out.append((rows, rows + (0 if pick(2) else pick(500))))
    return out[:-1] + [(90, 70)]


@pytest.mark.parametrize("n,nk,nv", [(40, 1, 4), (70, 2, 2), (150, 1, 1)])
def test_attn_many_sequences(fak, n, nk, nv):
    """More sequences than a warp looks over at a time, and more heads of them than go at once."""
    attn_case(fak, many(n, n), nk, nv, seed=n)


@pytest.mark.parametrize("wild", [False, True])
def test_attn_from_rows_to_chunks(fak, wild):
    """On both sides of the length from which a sequence goes over chunks; alone, the rows of the call decide."""
    attn_case(fak, [(28, 28), (29, 29), (27, 400), (30, 100), (1, 1)], 2, 4, wild=wild)
    for n in (28, 29):
        attn_case(fak, [(n, n + 5)], 1, 2, wild=wild, pad_rows=0, max_q=5000)


@pytest.mark.parametrize("nv", [5, 8, 11])
def test_attn_many_heads_to_a_key_head(fak, nv):
    attn_case(fak, [(130, 200), (70, 70), (3, 9)], 1, nv)


@pytest.mark.parametrize("bad", [-5, 10 ** 6, 0])
def test_attn_bad_starts_among_many(fak, bad):
    """A start that is out of range takes its two sequences with it, wherever it stands; so does one that falls."""
    lengths = [(n + 9, n + 9) for n, _ in many(39, 3)] + [(300, 300)]
    start, kv_len, slot, rows, slots = G.batch_tensors(lengths, 3)
    q, k, v, g, beta, z, w = G.inputs(1, 2, rows, 3)
    state = torch.full((slots, 2, 128, 128), NAN, device="cuda")
    old = start.tolist()
    start[20] = bad
    o = torch.full((rows, 2, 128), 7.0, device="cuda")
    fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot), q, k, v, g, beta, state, o, 300, z=z, norm_w=w)
    assert fak.fak_device_status() == 7
    for s in range(40):
        r = slice(old[s], old[s + 1])
        if s == 19:  # ends before it begins, or behind the last row
            assert bool((o[r] == 7).all()) and bool(state[slot[s]].isnan().all())
        elif s != 20:
            want, S, m = G.gdn_ref(*(t[r] for t in (q, k, v, g, beta)), torch.zeros_like(state[slot[s]]), 128 ** -0.5)
            assert float((state[slot[s]].double() - S).abs().max()) <= 2.0 ** -20 * (r.stop - r.start) ** 0.5 * m
    assert fak.fak_device_status() == 0


@pytest.mark.parametrize("name", ["few sequences", "many sequences"])
def test_attn_more_chunks_than_a_launch_takes(fak, name):
    """Records of 33,536 bytes a chunk and head: where all of them pass 1 GiB, a call goes over them in parts, of every
    sequence, or, where these would be short, of the batch."""
    lengths = [(19000, 19000), (2, 2), (13003, 20000)]
    if name == "many sequences":
        lengths = [(600 + 37 * i % 301, (i % 3) * 1000 + 901) for i in range(38)] + [(1, 50), (30, 30), (4000, 4000)]
    nk, nv = 4, 64
    start, kv_len, slot, rows, slots = G.batch_tensors(lengths, 4)
    assert (rows // 64 + 3) * nv * 33536 > 1 << 30
    q, k, v, g, beta, z, w = G.inputs(nk, nv, rows, 4)
    s0 = torch.randn(slots, nv, 128, 128, device="cuda") * 0.3
    a, oa = s0.clone(), torch.zeros(rows, nv, 128, device="cuda")
    fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot), q, k, v, g, beta, a, oa, 19000)
    b, ob = s0.clone(), torch.zeros_like(oa)
    for i, (n, t) in enumerate(lengths):  # one sequence at a time
        r = slice(int(start[i]), int(start[i + 1]))
        one = fak.GDNBatch(torch.tensor([0, n], dtype=torch.int32, device="cuda"), kv_len[i:i + 1], slot[i:i + 1])
        fak.fak_gdn_attn(one, q[r], k[r], v[r], g[r], beta[r], b, ob[r], n)
    assert fak.fak_device_status() == 0
    # each is off by the tests' tolerance at most; a column's length is at least what it is at the end, values are 9 at most
    for i, (n, _) in enumerate(lengths):
        r = slice(int(start[i]), int(start[i + 1]))
        tol = 2 * 2.0 ** -20 * n ** 0.5 * max(float(b[slot[i]].norm(dim=1).max()), float(v[r].abs().max()))
        assert float((a[slot[i]] - b[slot[i]]).abs().max()) <= tol
        assert float((oa[r] - ob[r]).abs().max()) <= tol * 128 ** -0.5 + 2.0 ** -23 * float(ob[r].abs().max())
    rest = [i for i in range(slots) if i not in slot.tolist()]
    assert torch.equal(a[rest], s0[rest])


def test_attn_bad_values_stay_in_their_sequence(fak):
    """Infinities and NaN in one sequence's rows and in the rows of no sequence reach no other sequence."""
    lengths = [(70, 70), (70, 75), (1, 4), (70, 70), (1, 2)]
    start, kv_len, slot, rows, slots = G.batch_tensors(lengths, 3, 5)
    got = []
    for bad in (False, True):
        q, k, v, g, beta, z, w = G.inputs(1, 2, rows, 12)
        state = torch.randn(slots, 2, 128, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
        if bad:
            for r in (slice(70, 140), slice(140, 141), slice(rows - 5, rows)):
                q[r], k[r], v[r], g[r], beta[r], z[r] = NAN, float("inf"), NAN, NAN, float("inf"), NAN
            state[[i for i in range(slots) if i not in slot.tolist()]] = NAN
        o = torch.zeros(rows, 2, 128, device="cuda")
        fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot), q, k, v, g, beta, state, o, 70, z=z, norm_w=w)
        got.append((o, state))
    for s in (0, 3, 4):
        r = slice(int(start[s]), int(start[s + 1]))
        assert torch.equal(got[0][0][r], got[1][0][r]) and torch.equal(got[0][1][slot[s]], got[1][1][slot[s]])
    assert fak.fak_device_status() == 0


@pytest.mark.parametrize("most", [1, 300])
def test_bad_batches_are_left_out(fak, most):
    """Numbers out of range: the sequence is left out and recorded, the others come out."""
    good = [(1, 4), (most, most), (1, 9), (1, 1)]
    for what in ("len", "slot low", "slot high", "max_q", "start"):
        start, kv_len, slot, rows, slots = G.batch_tensors(good, 2)
        q, k, v, g, beta, z, w = G.inputs(1, 2, rows, 13)
        state = torch.randn(slots, 2, 128, 128, device="cuda")
        keep = state.clone()
        old, max_q = slot.clone(), most
        if what == "len":
            kv_len[2] = -1
        elif what == "slot low":
            slot[2] = -1
        elif what == "slot high":
            slot[2] = slots
        elif what == "start":
            start[3] = rows + 9  # the last two sequences' bounds
        else:
            if most == 1:
                continue
            max_q = most - 1
        o = torch.full((rows, 2, 128), 7.0, device="cuda")
        fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot), q, k, v, g, beta, state, o, max_q, z=z, norm_w=w)
        assert fak.fak_device_status() == 7, what
        out = {"max_q": [1], "start": [2, 3]}.get(what, [2])
        for s, (first, end, fresh) in enumerate(G.real_rows(good)):
            if s in out:
                assert bool((o[first:end] == 7).all()) and torch.equal(state[old[s]], keep[old[s]]), what
                continue
            want, S, m = G.gdn_ref(*(t[first:end] for t in (q, k, v, g, beta)),
                                   keep[old[s]] * 0 if fresh else keep[old[s]], 128 ** -0.5)
            assert float((state[old[s]].double() - S).abs().max()) <= 2.0 ** -20 * (end - first) ** 0.5 * m
        assert fak.fak_device_status() == 0


def test_attn_same_bits_again_captured_and_on_another_stream(fak):
    lengths = BATCHES["mixed"]
    start, kv_len, slot, rows, slots = G.batch_tensors(lengths, 9)
    q, k, v, g, beta, z, w = G.inputs(2, 4, rows, 14)
    s0 = torch.randn(slots, 4, 128, 128, device="cuda")
    batch = fak.GDNBatch(start, kv_len, slot)

    def call(state, o):
        fak.fak_gdn_attn(batch, q, k, v, g, beta, state, o, 333, z=z, norm_w=w)

    a, oa = s0.clone(), torch.zeros(rows, 4, 128, device="cuda")
    call(a, oa)
    b, ob = s0.clone(), torch.zeros_like(oa)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(b, ob)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b) and torch.equal(oa, ob)
    c, oc = s0.clone(), torch.zeros_like(oa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, oc)
    assert torch.equal(c, s0)
    graph.replay()
    assert torch.equal(a, c) and torch.equal(oa, oc)
    # the numbers are read when the graph runs
    c.copy_(s0)
    oc.zero_()
    kv_len[0], kv_len[1] = 1, 900
    slot.copy_(slot.flip(0))
    graph.replay()
    d, od = s0.clone(), torch.zeros_like(oa)
    call(d, od)
    assert torch.equal(c, d) and torch.equal(oc, od) and not torch.equal(oa, oc)
    assert fak.fak_device_status() == 0


def test_attn_two_calls_at_once(fak):
    """On two streams, each with its own scratch."""
    lengths = [(700, 700), (1, 9), (130, 400), (64, 64)]
    calls = []
    for seed in (21, 22):
        start, kv_len, slot, rows, slots = G.batch_tensors(lengths, seed)
        q, k, v, g, beta, z, w = G.inputs(2, 16, rows, seed)
        calls.append((fak.GDNBatch(start, kv_len, slot), q, k, v, g, beta, torch.randn(slots, 16, 128, 128, device="cuda"), z, w, rows))
    outs = []
    for at_once in (False, True):
        streams = [torch.cuda.Stream() if at_once else torch.cuda.current_stream() for _ in calls]
        here = []
        for s, (batch, q, k, v, g, beta, s0, z, w, rows) in zip(streams, calls):
            here.append((s0.clone(), torch.zeros(rows, 16, 128, device="cuda")))
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            for s, (state, o), (batch, q, k, v, g, beta, s0, z, w, rows) in zip(streams, here, calls):
                with torch.cuda.stream(s):
                    fak.fak_gdn_attn(batch, q, k, v, g, beta, state, o, 700, z=z, norm_w=w)
        torch.cuda.synchronize()
        outs += here
    assert fak.fak_device_status() == 0
    for i in range(2):
        assert torch.equal(outs[i][0], outs[2 + i][0]) and torch.equal(outs[i][1], outs[2 + i][1])


def test_offsets_that_pass_32_bits(fak):
    """Rows, and slots of the pools, more than 2^31 elements behind the first."""
    far, rows = 1 << 20, 2200
    lengths = [(2150, 2150), (1, 5), (49, 49)]
    start, kv_len, _, _, _ = G.batch_tensors(lengths, 0)
    slots = 1500
    slot = torch.tensor([slots - 1, slots - 3, slots - 2], dtype=torch.int32, device="cuda")
    nk, nv = 2, 96
    state = torch.empty(slots, nv, 128, 128, device="cuda")
    assert state.numel() > 1 << 31 and far * (rows - 100) > 1 << 31
    state[-3:] = 0.3 * torch.randn(3, nv, 128, 128, device="cuda")
    keep = state[-3:].clone()
    q, k, v, g, beta, z, w = G.inputs(nk, nv, rows, 31)

    def view(t):
        big = torch.empty(rows * far, dtype=t.dtype, device="cuda").view(rows, far)
        big = big[:, :t.shape[1] * 128].unflatten(1, (t.shape[1], 128))
        return big.copy_(t)

    o = view(torch.zeros(rows, nv, 128, device="cuda", dtype=torch.bfloat16))
    fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot), view(q), view(k), view(v), g, beta, state, o, 2150, z=view(z), norm_w=w)
    assert fak.fak_device_status() == 0
    near = torch.empty(3, nv, 128, 128, device="cuda").copy_(keep)
    on = torch.zeros(rows, nv, 128, device="cuda", dtype=torch.bfloat16)
    fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot - (slots - 3)), q, k, v, g, beta, near, on, 2150, z=z, norm_w=w)
    assert torch.equal(o, on) and torch.equal(state[-3:], near)
    del state, o
    chans = (2 * nk + 4) * 128
    x, b, a = torch.randn(rows, chans, device="cuda"), torch.randn(rows, 4, device="cuda"), torch.randn(rows, 4, device="cuda")
    big = torch.empty(rows * far, device="cuda").view(rows, far)[:, :chans].copy_(x)
    conv_w, a_log, dt = torch.randn(chans, 4, device="cuda"), torch.rand(4, device="cuda"), torch.rand(4, device="cuda")
    got = []
    for t, n in ((x, 3), (big, 1 << 20)):
        st = torch.zeros(n, 3, chans, device="cuda")
        assert n == 3 or st.numel() > 1 << 31
        out = [torch.zeros(rows, nk, 128, dtype=torch.float16, device="cuda") for _ in range(2)]
        out += [torch.zeros(rows, 4, 128, dtype=torch.bfloat16, device="cuda"), *(torch.zeros(rows, 4, device="cuda") for _ in range(2))]
        fak.fak_gdn_conv(fak.GDNBatch(start, kv_len, slot - (slots - n)), t, b, a, conv_w, a_log, dt, st, *out, eps=G.EPS)
        got.append(out + [st[-3:].clone()])
    assert fak.fak_device_status() == 0
    assert all(torch.equal(i, j) for i, j in zip(*got)) and bool(got[0][0].any())


# ------------------------------------------------------------------ the convolution
def conv_case(fak, lengths, nk, nv, kind=torch.float32, seed=1, pad_rows=2, views=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    start, kv_len, slot, rows, slots = G.batch_tensors(lengths, seed, pad_rows)
    chans = (2 * nk + nv) * 128
    t = rand(rows, chans + 2 * nv + 8).to(kind)
    x, b, a = t[:, :chans], t[:, chans:chans + nv], t[:, chans + nv:chans + 2 * nv]
    if not views:
        x, b, a = (u.contiguous() for u in (x, b, a))
    if rows > 9:
        b[5], a[6], a[7] = 60.0, -90.0, 90.0
    w, a_log, dt = 0.5 * rand(chans, 4), torch.log(1 + 15 * torch.rand(nv, device="cuda")), rand(nv)
    state = rand(slots, 3, chans)
    for (n, ln), s in zip(lengths, slot.tolist()):
        if ln <= n:
            state[s] = NAN
    keep = state.clone()
    q, k = (torch.full((rows, nk, 128), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    v = torch.full((rows, nv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    g, beta = (torch.full((rows, nv), 7.0, device="cuda") for _ in range(2))
    fak.fak_gdn_conv(fak.GDNBatch(start, kv_len, slot), x, b, a, w, a_log, dt, state, q, k, v, g, beta, eps=G.EPS)
    assert fak.fak_device_status() == 0
    seen = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for (first, end, fresh), s in zip(G.real_rows(lengths), slot.tolist()):
        if first == end:
            assert torch.equal(state[s].nan_to_num(1e9), keep[s].nan_to_num(1e9))
            continue
        r = slice(first, end)
        seen[r] = True
        c, after = G.conv_ref(x[r], w, torch.zeros_like(keep[s]) if fresh else keep[s])
        assert torch.equal(state[s], after.float())  # inputs, kept as they are
        c = c.view(end - first, -1, 128)
        # four products of f32 (sums off by 4 * 2^-24 of the terms' magnitudes, here below 16), silu by fast functions (2^-20)
        near = 16 * 2.0 ** -22 + c.abs() * 2.0 ** -20
        for got, want in ((q[r], c[:, :nk]), (k[r], c[:, nk:2 * nk])):
            size = torch.sqrt((want * want).sum(-1, keepdim=True) + G.EPS)
            tol = want.abs() / size * (2.0 ** -11 + 2.0 ** -18) + 2.0 ** -25 + 4 * 16 * 2.0 ** -22 / size
            assert bool(((got.double() - want / size).abs() <= tol).all())
        want = c[:, 2 * nk:]
        assert bool(((v[r].double() - want).abs() <= want.abs() * 2.0 ** -8 + near[:, 2 * nk:]).all())
        u = a[r].double() + dt.double()
        want = -torch.exp(a_log.double()) * torch.nn.functional.softplus(u, threshold=1000.0)
        # u is off by 2^-24 of its terms, and so softplus by as much of its own slope; a few roundings of f32 behind it
        off = torch.exp(a_log.double()) * torch.sigmoid(u) * (a[r].double().abs() + dt.abs()) * 2.0 ** -23
        assert bool(((g[r].double() - want).abs() <= want.abs() * 2.0 ** -20 + off).all())
        want = torch.sigmoid(b[r].double())
        assert bool(((beta[r].double() - want).abs() <= want * 2.0 ** -21).all())
    for t in (q, k, v, g, beta):
        assert bool((t[~seen] == 7).all())
    rest = [i for i in range(slots) if i not in slot.tolist()]
    assert torch.equal(state[rest], keep[rest])


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_conv_lengths(fak, name, kind):
    conv_case(fak, BATCHES[name], 2, 3, kind)


@pytest.mark.parametrize("seed", range(4))
def test_conv_many_short_sequences(fak, seed):
    """Over 608 rows, so that a block has several: sequences of 0 to 12 rows begin and end anywhere in a block's range."""
    rng = np.random.default_rng(seed)
    lengths = [(int(n), int(n + rng.integers(-1, 3)) if n else 3) for n in rng.integers(0, 13, 160)]
    lengths = [(n, max(t, 0)) for n, t in lengths] + [(40, 40), (3, 3), (2, 2)]
    conv_case(fak, lengths, 1, 2, seed=20 + seed, views=seed % 2 == 0)


def test_conv_large(fak):
    conv_case(fak, [(2000, 2000), (1, 5), (700, 701)], 16, 48, seed=30)


def test_conv_bad_batches_are_left_out(fak):
    for rows_each in (2, 200):
        good = [(rows_each, rows_each + 3)] * 4
        for what in ("len", "slot low", "slot high", "start"):
            start, kv_len, slot, rows, slots = G.batch_tensors(good, 2)
            chans = 3 * 128
            x, ba = torch.randn(rows, chans, device="cuda"), torch.randn(rows, 1, device="cuda")
            state = torch.randn(slots, 3, chans, device="cuda")
            keep, old = state.clone(), slot.tolist()
            out = [2]
            if what == "len":
                kv_len[2] = -1
            elif what == "slot low":
                slot[2] = -2
            elif what == "slot high":
                slot[2] = slots
            else:
                start[3], out = rows + 1, [2, 3]
            q, k = (torch.full((rows, 1, 128), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
            v = torch.full((rows, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
            g, beta = (torch.full((rows, 1), 7.0, device="cuda") for _ in range(2))
            w = torch.randn(chans, 4, device="cuda")
            zero = torch.zeros(1, device="cuda")
            fak.fak_gdn_conv(fak.GDNBatch(start, kv_len, slot), x, ba, ba, w, zero, zero, state, q, k, v, g, beta)
            assert fak.fak_device_status() == 7, what
            for s in range(4):
                r = slice(s * rows_each, (s + 1) * rows_each)
                if s in out:
                    assert bool((v[r] == 7).all()) and bool((g[r] == 7).all()) and torch.equal(state[old[s]], keep[old[s]])
                else:
                    c, after = G.conv_ref(x[r], w, keep[old[s]])
                    assert torch.equal(state[old[s]], after.float())
                    assert float((v[r].double() - c.view(-1, 3, 128)[:, 2:]).abs().max()) <= 2.0 ** -8 * float(c.abs().max()) + 1e-4
            assert fak.fak_device_status() == 0


def test_calls_without_rows_or_sequences(fak):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    state = torch.randn(1, 2, 128, 128, device="cuda")
    for start, ln, slot, rows in ((i32(0), i32(), i32(), 3), (i32(0, 0), i32(4), i32(0), 0)):
        batch = fak.GDNBatch(start, ln, slot)
        keep = state.clone()
        o = torch.full((rows, 2, 128), 7.0, device="cuda")
        h = e(rows, 1, 128, dtype=torch.float16)
        fak.fak_gdn_attn(batch, h, h, e(rows, 2, 128, dtype=torch.bfloat16), e(rows, 2), e(rows, 2), state, o, 5)
        fak.fak_gdn_conv(batch, e(rows, 512), e(rows, 2), e(rows, 2), e(512, 4), e(2), e(2), e(1, 3, 512), h, h,
                         e(rows, 2, 128, dtype=torch.bfloat16), e(rows, 2), e(rows, 2))
        assert fak.fak_device_status() == 0 and torch.equal(state, keep) and bool((o == 7).all())


@pytest.mark.parametrize("lengths", [[(130, 130)], [(70, 75), (1, 3), (300, 300)]])
def test_a_wait_that_runs_out_is_recorded_and_ends(fak, lengths):
    start, kv_len, slot, rows, slots = G.batch_tensors(lengths, 1)
    q, k, v, g, beta, z, w = G.inputs(1, 2, rows, 15)
    s0 = torch.randn(slots, 2, 128, 128, device="cuda")
    batch = fak.GDNBatch(start, kv_len, slot)
    fak.fak_gdn_debug_wait(1000000, 1)
    try:
        fak.fak_gdn_attn(batch, q, k, v, g, beta, s0.clone(), torch.empty(rows, 2, 128, device="cuda"), 300, z=z, norm_w=w)
        assert fak.fak_device_status() == 5
    finally:
        fak.fak_gdn_debug_wait()
    outs = []
    for _ in range(2):
        s, o = s0.clone(), torch.zeros(rows, 2, 128, device="cuda")
        fak.fak_gdn_attn(batch, q, k, v, g, beta, s, o, 300, z=z, norm_w=w)
        outs.append((s, o))
    assert fak.fak_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and bool(torch.isfinite(outs[0][1]).all())
