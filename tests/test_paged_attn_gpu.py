"""GPU parity of the attention over the paged KV cache (fak_paged_attn) against plain attention in 64 bits on what the
cache holds, with the bar that tests/_kv.py derives: single tokens, chunks and prompts, mixed in ragged batches, every
head dim, cache type and page, windows and sinks, gates, and what a row must not see."""
import pytest

torch = pytest.importorskip("torch")
import _kv

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "i8"]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def fak():
    from q4_weight_quantized_block_gb300 import build
    build.build()
    import q4_weight_quantized_block_gb300 as m
    assert torch.cuda.is_available()
    return m


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


class Setup:
    def __init__(self, fak, kind, nq, n_kv, dh, page, lengths, seed=0, gate=False, pad_rows=0, sharp=1.0, window=0, sinks=0,
                 edit=None):
        self.fak, self.kind, self.nq, self.dh, self.page, self.lengths = fak, kind, nq, dh, page, lengths
        self.window, self.sinks = window, sinks
        self.table, self.start, self.kv_len, self.rows, n_pages = _kv.batch_tensors(lengths, page, seed=seed, pad_rows=pad_rows)
        self.cache, self.mem = _kv.empty_cache(fak, kind, n_pages, n_kv, page, dh)
        K = [randn(seed + 100 + i, t, n_kv, dh) for i, (_, t) in enumerate(lengths)]
        V = [randn(seed + 200 + i, t, n_kv, dh) + 0.25 for i, (_, t) in enumerate(lengths)]
        if edit:
            edit(K, V)
        _kv.fill(self.mem, kind, self.table, self.kv_len, page, K, V)
        self.batch = fak.KVBatch(self.table, self.start, self.kv_len)
        # queries, gates and results as slices of wider rows
        self.q = (sharp * randn(seed + 1, self.rows, nq, 2 * dh)).to(torch.bfloat16)[..., dh:]
        self.gate = randn(seed + 2, self.rows, 2 * nq, dh)[:, 1::2] if gate else None
        self.out = torch.full((self.rows, nq + 1, dh), 9.0, dtype=torch.bfloat16, device="cuda")[:, :nq]
        self.max_q, self.max_kv = max(n for n, _ in lengths), max(t for _, t in lengths)
        self.scale = dh**-0.5

    def workspace(self, max_q=None, max_kv=None):
        n = self.fak.fak_paged_attn_workspace_bytes(self.cache, self.batch, self.nq, self.rows, max_q or self.max_q,
                                                    max_kv or self.max_kv, window=self.window, sinks=self.sinks)
        return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten

    def run(self, out=None, workspace=None, max_q=None, max_kv=None, stream=None):
        ws = self.workspace(max_q, max_kv) if workspace is None else workspace
        self.fak.fak_paged_attn(self.cache, self.batch, self.q, self.out if out is None else out, max_q or self.max_q,
                                max_kv or self.max_kv, scale=self.scale, window=self.window, sinks=self.sinks, gate=self.gate,
                                workspace=ws, stream=stream)
        return ws

    def want(self, lengths=None):
        """Per sequence: rows, values, tolerance."""
        t, row = self.table.cpu(), 0
        for s, (n, total) in enumerate(lengths or self.lengths):
            pos = torch.arange(total)
            k, v = _kv.held(self.mem, self.kind, t[s, pos // self.page].long(), pos % self.page)
            r = slice(row, row + n)
            o, tol = _kv.attention(self.q[r], k, v, total - n, self.scale, self.window, self.sinks,
                                   None if self.gate is None else self.gate[r])
            yield r, o, tol
            row += n

    def check(self, lengths=None):
        torch.cuda.synchronize()
        assert self.fak.fak_device_status() == 0
        for s, (r, o, tol) in enumerate(self.want(lengths)):
            _kv.check(self.out[r], o, tol, "sequence %d" % s)
        assert bool((self.out[int(self.start[-1]):] == 9.0).all())
        assert bool((self.out.as_strided((self.rows, self.dh), (self.out.stride(0), 1), self.nq * self.dh) == 9.0).all())


def case(fak, *a, **kw):
    s = Setup(fak, *a, **kw)
    s.run()
    s.check()
    return s


HEADS = [(24, 4, 256), (6, 6, 256), (16, 1, 256), (32, 8, 128), (3, 1, 128), (40, 1, 128), (8, 2, 64), (5, 5, 64)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq,n_kv,dh", HEADS)
def test_single_tokens(fak, kind, nq, n_kv, dh):
    case(fak, kind, nq, n_kv, dh, 16, [(1, 1), (1, 2), (1, 17), (1, 128), (1, 129), (1, 500)], seed=nq, gate=dh == 256)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nq,n_kv,dh", HEADS)
def test_chunks(fak, kind, nq, n_kv, dh):
    case(fak, kind, nq, n_kv, dh, 32, [(33, 33), (50, 300), (2, 131), (0, 40), (129, 129)], seed=nq + 1, gate=dh != 128)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(fak, kind, page):
    case(fak, kind, 6, 1, 256, page, [(1, 257), (40, 255), (7, 640), (1, page), (1, page + 1)], seed=page)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,total", [(1, 5000), (3, 4097), (20, 3333), (64, 2048), (300, 2500)])
def test_few_rows_over_a_long_past(fak, kind, new, total):
    # the keys are split over several blocks and joined
    case(fak, kind, 12, 2, 256, 64, [(new, total)], seed=new, gate=True)
    case(fak, kind, 8, 1, 128, 64, [(new, total)], seed=new + 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (100, 0), (128, 130), (500, 3), (5000, 4)])
def test_window_and_sinks(fak, kind, window, sinks):
    lengths = [(1, 1), (1, 700), (90, 700), (200, 200), (5, 70)]
    case(fak, kind, 8, 2, 128, 16, lengths, seed=window, window=window, sinks=sinks, gate=True)
    case(fak, kind, 6, 1, 256, 64, lengths, seed=window + 1, window=window, sinks=sinks)


def test_sinks_without_a_window_change_nothing(fak):
    a = case(fak, "bf16", 4, 1, 128, 16, [(20, 90)])
    b = Setup(fak, "bf16", 4, 1, 128, 16, [(20, 90)], sinks=9)
    b.run()
    assert torch.equal(a.out, b.out)


def test_a_prompt_of_many_tiles(fak):
    case(fak, "bf16", 6, 1, 256, 64, [(1500, 1500)], seed=5)
    case(fak, "e4m3", 4, 1, 128, 16, [(1100, 2000), (900, 900)], seed=6)


@pytest.mark.parametrize("kind", KINDS)
def test_many_blocks_to_an_sm(fak, kind):
    # each SM works on several blocks one after the other: short ones (a window), cut ones, ragged ones, one tile only,
    # and blocks that see nothing between others
    case(fak, kind, 32, 8, 128, 32, [(2048, 5000)], seed=30, window=1024, sinks=4)
    case(fak, kind, 24, 4, 256, 64, [(700, 3000)], seed=31, gate=True)
    case(fak, kind, 16, 16, 64, 16, [(900, 1300), (1, 2000), (0, 70), (640, 640)], seed=32)
    case(fak, kind, 24, 4, 256, 16, [(200 + 37 * i, 200 + 37 * i) for i in range(9)], seed=33, window=100, sinks=1)
    case(fak, kind, 32, 8, 128, 16, [(40 + i, 100 * (i % 3) + 3) for i in range(40)], seed=34)


def test_a_full_batch_of_single_tokens(fak):
    lengths = [(1, 1 + (37 * i) % 900) for i in range(64)]
    case(fak, "e4m3", 24, 4, 256, 64, lengths, seed=7, gate=True)
    case(fak, "bf16", 8, 1, 64, 16, lengths + [(3, 90)] * 3, seed=8)


@pytest.mark.parametrize("kind", KINDS)
def test_sharp_scores(fak, kind):
    # scores of +-100 and more: one key takes all the weight, maxima jump along the row
    case(fak, kind, 6, 1, 256, 64, [(70, 600), (1, 999)], seed=9, sharp=30.0)


def test_padding_rows_get_zeros_and_others_nothing(fak):
    # more rows than positions: the first rows see nothing
    case(fak, "bf16", 4, 2, 128, 16, [(1, 30), (8, 5), (200, 140), (3, 0), (1, 0)], seed=10, pad_rows=6, gate=True)
    case(fak, "i8", 4, 2, 256, 16, [(1, 30), (1, 0), (2, 1)], seed=11, pad_rows=1)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("new,total,at", [(100, 100, 60), (100, 300, 290), (1, 200, 3), (3, 140, 138)])
def test_odd_values_reach_only_the_rows_that_see_them(fak, bad, new, total, at):
    def edit(K, V):
        V[0][at, 0, 5] = bad

    case(fak, "bf16", 6, 1, 256, 16, [(new, total)], seed=12, edit=edit)
    case(fak, "bf16", 4, 2, 128, 16, [(new, total)], seed=13, edit=edit, window=50, sinks=2)


@pytest.mark.parametrize("kind", KINDS)
def test_nan_keys_and_values_behind_a_row_are_not_seen(fak, kind):
    def edit(K, V):
        K[0][70:75] = NAN
        V[0][70:75] = NAN

    s = Setup(fak, kind, 6, 1, 256, 16, [(100, 100)], seed=14, edit=edit)
    s.run()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(s.out[:70]).all()) and bool(torch.isnan(s.out[70:]).all())
    for r, o, tol in s.want():
        _kv.check(s.out[:70], o[:70], tol[:70], "rows before")
    w = Setup(fak, kind, 6, 1, 256, 16, [(3, 500)], seed=15, edit=edit, window=100, sinks=8)
    w.run()
    w.check()


def test_equal_scores_of_the_lowest_value(fak):
    # keys of zero: all weights equal, whatever the mask
    def edit(K, V):
        K[0].zero_()

    case(fak, "bf16", 4, 1, 128, 16, [(40, 333)], seed=16, edit=edit, window=37, sinks=3)


def test_bounds_above_the_lengths(fak):
    s = Setup(fak, "bf16", 12, 2, 256, 64, [(1, 300), (4, 90)], seed=17)
    s.run(max_q=64, max_kv=100000)
    s.check()
    s.out.fill_(9.0)
    s.run(max_q=2000, max_kv=301)
    s.check()


def test_sequences_out_of_bounds_are_left_out(fak):
    s = Setup(fak, "bf16", 4, 1, 128, 16, [(2, 60), (5, 40), (1, 90)], seed=18)
    s.run(max_q=4, max_kv=90)
    assert fak.fak_device_status() == 7
    want = list(s.want())
    for i in (0, 2):
        _kv.check(s.out[want[i][0]], want[i][1], want[i][2], "sequence %d" % i)
    assert bool((s.out[want[1][0]] == 9.0).all())
    s.out.fill_(9.0)
    s.run(max_q=5, max_kv=80)
    assert fak.fak_device_status() == 7
    for i in (0, 1):
        _kv.check(s.out[want[i][0]], want[i][1], want[i][2], "sequence %d" % i)
    assert bool((s.out[want[2][0]] == 9.0).all())


def test_a_bad_page_is_recorded(fak):
    for lengths in ([(1, 60), (1, 40)], [(30, 60), (40, 40)]):
        s = Setup(fak, "i8", 4, 1, 128, 16, lengths, seed=19)
        s.table[1, 1] = 1 << 30
        s.run()
        assert fak.fak_device_status() == 7
        r, o, tol = next(iter(s.want()))
        _kv.check(s.out[r], o, tol, "the other sequence")


def test_same_bits_every_time_and_on_another_stream(fak):
    for lengths in ([(1, 3000)], [(77, 900), (1, 40)]):
        s = Setup(fak, "e4m3", 24, 4, 256, 64, lengths, seed=20, gate=True)
        s.run()
        torch.cuda.synchronize()
        first = s.out.clone()
        side = torch.cuda.Stream()
        for _ in range(3):
            s.out.fill_(9.0)
            side.wait_stream(torch.cuda.current_stream())
            s.run(stream=side)
            side.synchronize()
            assert torch.equal(first.view(torch.int16), s.out.view(torch.int16))


def test_two_calls_at_once_with_their_own_workspaces(fak):
    a = Setup(fak, "bf16", 24, 4, 256, 64, [(1, 4000)], seed=21)
    b = Setup(fak, "bf16", 24, 4, 256, 64, [(60, 2000)], seed=22)
    wa, wb = a.workspace(), b.workspace()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a.run(workspace=wa, stream=s)
        b.run(workspace=wb, stream=t)
    a.check()
    b.check()


def test_captured_once_replayed_with_other_lengths(fak):
    full = [(1, 2000), (1, 700), (1, 64)]
    s = Setup(fak, "i8", 12, 2, 256, 64, full, seed=23, gate=True)
    ws = s.workspace()
    s.run(workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run(workspace=ws)
    for lengths in (full, [(1, 1999), (1, 1), (1, 33)], [(1, 130), (1, 699), (1, 64)]):
        s.kv_len.copy_(torch.tensor([t for _, t in lengths], dtype=torch.int32))
        s.out.fill_(9.0)
        g.replay()
        s.check(lengths)
    # and with rows divided otherwise: the second sequence has them all
    s2 = Setup(fak, "bf16", 12, 2, 256, 64, [(10, 100), (10, 900)], seed=24)
    ws2 = s2.workspace(max_q=20)
    g2 = torch.cuda.CUDAGraph()
    s2.run(workspace=ws2, max_q=20)
    torch.cuda.synchronize()
    with torch.cuda.graph(g2):
        s2.run(workspace=ws2, max_q=20)
    for lengths in ([(10, 100), (10, 900)], [(0, 100), (20, 900)], [(1, 100), (3, 500)]):
        s2.start.copy_(torch.tensor([0, lengths[0][0], lengths[0][0] + lengths[1][0]], dtype=torch.int32))
        s2.kv_len.copy_(torch.tensor([t for _, t in lengths], dtype=torch.int32))
        s2.out.fill_(9.0)
        g2.replay()
        s2.check(lengths)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dh,new", [(64, 1), (128, 1), (256, 1), (256, 2), (128, 70)])
def test_values_of_any_size(fak, kind, dh, new):
    """Zeros first, which count in the sum alone; all tiny; sizes from 1e-18 to 1e18 beside each other."""
    def edit(K, V):
        V[0][:600] = 0.0
        V[1].mul_(1e-25)
        size = torch.rand(V[2].shape[0], 1, 1, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
        V[2].mul_(10.0 ** (36.0 * size - 18.0))

    case(fak, kind, 8, 2, dh, 32, [(new, 900), (new, 700), (new, 800)], seed=dh + new, edit=edit)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sharp", [1e-38, 1e-20, 12.0])
def test_queries_of_any_size(fak, kind, sharp):
    case(fak, kind, 24, 4, 256, 64, [(1, 300), (2, 77)], seed=5, sharp=sharp)


@pytest.mark.parametrize("kind", KINDS)
def test_many_pieces_of_many_rows(fak, kind):
    case(fak, kind, 24, 4, 256, 64, [(64, 8255)], seed=6, gate=True)


@pytest.mark.parametrize("kind,max_q", [("bf16", 1), ("i8", 40)])
def test_strides_that_are_never_taken(fak, kind, max_q):
    s = Setup(fak, kind, 4, 4, 128, 16, [(1, 90)], seed=8)
    s.max_q = max_q
    s.q, s.out = s.q.as_strided((1, 4, 128), (1, s.q.stride(1), 1)), s.out.as_strided((1, 4, 128), (3, 128, 1))
    s.run()
    torch.cuda.synchronize()
    assert fak.fak_device_status() == 0
    for r, o, tol in s.want():
        _kv.check(s.out[r], o, tol, "one row")



@pytest.mark.parametrize("code", [0x7F, 0xFF])
@pytest.mark.parametrize("nq,n_kv,dh", [(6, 1, 256), (4, 2, 256), (6, 3, 128), (8, 1, 128), (4, 1, 64), (8, 1, 64)])
@pytest.mark.parametrize("new,total,at,window,blind", [
    (2, 100, 99, 0, [0]),  # the last token's own key
    (2, 200, 149, 50, [1]),  # the first token's window still holds it, the second's does not
    (2, 2000, 1999, 0, [0]),  # in the last piece of many
    (2, 128, 5, 30, [0, 1]),  # in nobody's window
])
def test_nan_codes_reach_only_the_rows_that_see_them(fak, code, nq, n_kv, dh, new, total, at, window, blind):
    s = Setup(fak, "e4m3", nq, n_kv, dh, 16, [(new, total)], seed=at, window=window)
    page, slot = int(s.table[0, at // 16]), at % 16
    for d in (5, dh - 2):
        s.mem[1][page, 0, slot, d] = code
    s.run()
    torch.cuda.synchronize()
    assert fak.fak_device_status() == 0
    (_, o, tol), = s.want()
    others = [d for d in range(dh) if d not in (5, dh - 2)]
    _kv.check(s.out[blind], o[blind], tol[blind], "rows that do not see it")
    _kv.check(s.out[..., others], o[..., others], tol[..., others], "the other elements")



@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1e17, 1e30])
@pytest.mark.parametrize("where", ["later keys", "earlier keys", "every second step", "one warp's keys", "one key"])
@pytest.mark.parametrize("new,total", [(1, 300), (2, 300), (1, 6000), (40, 300)])
def test_zeros_beside_large_values(fak, kind, size, where, new, total):
    """Equal scores: a value's share is one part in as many as a row sees, whatever its size."""
    def edit(K, V):
        K[0].zero_()
        j = torch.arange(total, device="cuda")
        large = {"later keys": j >= total // 2, "earlier keys": j < total // 2, "every second step": (j // 128) % 2 == 1,
                 "one warp's keys": (j // 16) % 8 == 5, "one key": j == 17}[where]
        V[0].mul_(torch.where(large, size, 0.0)[:, None, None])

    case(fak, kind, 4, 2, 128, 16, [(new, total)], seed=3, edit=edit)
    case(fak, kind, 6, 1, 256, 16, [(new, total)], seed=4, edit=edit)



@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,total", [(1, 300), (2, 300), (1, 6000), (40, 300)])
@pytest.mark.parametrize("zeros", [False, True])
def test_smallest_values(fak, kind, new, total, zeros):
    """Values just above the size that the 8-bit kinds hold as zeros, the same at each key, with zeros between or without."""
    def edit(K, V):
        sign = torch.where(V[0][:1] < 0, -1.0, 1.0)
        V[0].copy_(sign.expand_as(V[0]) * 1e-30)
        if zeros:
            V[0][:total // 2] = 0

    for nq, n_kv, dh in ((4, 2, 128), (6, 1, 256)):
        s = Setup(fak, kind, nq, n_kv, dh, 16, [(new, total)], seed=5, edit=edit)
        s.run()
        torch.cuda.synchronize()
        assert fak.fak_device_status() == 0
        for r, o, tol in s.want():
            _kv.check(s.out[r], o, tol - 1e-30, "1e-30")  # (the bar without its absolute part)


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("new,total", [(1, 300), (2, 300), (1, 6000)])
def test_largest_values_of_few_rows(fak, kind, new, total):
    """Values whose sum over the keys is beyond f32, and their mean is not; sharp scores beside equal ones."""
    def edit(K, V):
        V[0].mul_(1e37)

    case(fak, kind, 4, 2, 128, 16, [(new, total)], seed=6, edit=edit)
    case(fak, kind, 6, 1, 256, 16, [(new, total)], seed=7, edit=edit, sharp=8.0)



@pytest.mark.parametrize("bad", [1000, -5])
@pytest.mark.parametrize("kind,new,total,n", [("bf16", 1, 60, 4), ("e4m3", 1, 3000, 4), ("bf16", 40, 90, 4), ("i8", 200, 3000, 4),
                                              ("e4m3", 1, 3000, 40), ("bf16", 40, 90, 40), ("i8", 3, 70, 70)])
def test_a_bad_start_leaves_out_its_own_sequences_only(fak, kind, new, total, n, bad):
    s = Setup(fak, kind, 4, 1, 128, 16, [(new, total)] * n, seed=21)
    i = n // 2 // 2 * 2
    s.start[i] = bad if bad < 0 else s.rows + bad  # sequences i - 1 and i
    s.run()
    torch.cuda.synchronize()
    assert fak.fak_device_status() == 7
    for q, (r, o, tol) in enumerate(s.want()):
        if q in (i - 1, i):
            assert bool((s.out[r] == 9.0).all()), q
        else:
            _kv.check(s.out[r], o, tol, "sequence %d" % q)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,total", [(1, 16), (2, 60), (1, 90), (1, 3000), (20, 90), (40, 90), (100, 300)])
def test_a_wait_that_runs_out_is_recorded_and_ends(fak, kind, new, total):
    s = Setup(fak, kind, 4, 1, 128, 16, [(new, total)], seed=25)
    ws = s.workspace()
    fak.fak_paged_attn_debug_wait(5_000_000, 1)
    try:
        s.run(workspace=ws)
        torch.cuda.synchronize()
        assert fak.fak_device_status() == 5
    finally:
        fak.fak_paged_attn_debug_wait()
    assert ws.numel() > 16 or bool((s.out == 9.0).all())  # (where keys are cut, pieces that never came were joined)
    s.out.fill_(9.0)
    s.run(workspace=ws)
    s.check()


@pytest.mark.parametrize("n_seqs", [0, 2])
def test_a_step_without_rows(fak, n_seqs):
    cache, mem = _kv.empty_cache(fak, "i8", 4, 2, 16, 64)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    batch = fak.KVBatch(i32(n_seqs, 3), i32(n_seqs + 1), i32(n_seqs))
    x, q = torch.empty(0, 2, 64, device="cuda"), torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    fak.fak_kv_append(cache, batch, x, x, q=torch.empty(0, 4, 64, device="cuda"), q_out=q)
    fak.fak_kv_read(cache, batch, x, x)
    n = fak.fak_paged_attn_workspace_bytes(cache, batch, 4, 0, 0, 0)
    fak.fak_paged_attn(cache, batch, q, torch.empty_like(q), 0, 0, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert fak.fak_device_status() == 0


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("new,total", [(1, 90), (2, 3000), (1, 60000)])
def test_values_at_the_top_of_f32(fak, kind, new, total):
    """Every value 3e38 in size: their mean is too, whatever number of keys, warps and pieces is added up."""
    def edit(K, V):
        sign = torch.where(V[0][:1] < 0, -1.0, 1.0)
        V[0].copy_((sign * 3e38).expand_as(V[0]))

    case(fak, kind, 4, 2, 128, 16, [(new, total)], seed=26, edit=edit)
    case(fak, kind, 6, 1, 256, 16, [(new, total)], seed=27, edit=edit)
