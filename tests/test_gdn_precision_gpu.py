"""fak_gdn_attn where magnitudes differ from row to row: every output and state against the rule in 64 bits, by what the rows up
to it have brought to its own value column, less what has decayed since."""
import pytest

torch = pytest.importorskip("torch")
import _gdn as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fak():
    from q4_weight_quantized_block_gb300 import build
    build.build()
    import q4_weight_quantized_block_gb300 as m
    assert torch.cuda.is_available()
    return m


def rule(q, k, v, g, beta, S, scale):
    """o [rows, nv, 128], S behind, and M [rows, nv, 128], in 64 bits.  M of a column: its state's length before the first row;
    from row to row it decays with the state, and is at least the row's value and the length that the column then has."""
    nv = v.shape[1]
    q, k = (t.double().repeat_interleave(nv // t.shape[1], 1) for t in (q, k))
    v, g, beta, S = v.double(), g.double(), beta.double(), S.double()
    out, most, m = torch.empty_like(v), torch.empty_like(v), S.norm(dim=1)
    for t in range(v.shape[0]):
        e = torch.exp(g[t])[:, None]
        S = e[:, :, None] * S
        u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
        S = S + k[t][:, :, None] * u[:, None, :]
        m = torch.maximum(torch.maximum(e * m, v[t].abs()), S.norm(dim=1))
        out[t], most[t] = scale * torch.einsum("hkv,hk->hv", S, q[t]), m
    return out, S, most


LENGTHS = [(200, 200), (150, 400), (29, 29), (64, 64), (20, 33), (70, 75)]


def check(fak, change, out=torch.float32, lengths=LENGTHS, seed=1, nk=1, nv=3, gate=False, max_q=None):
    start, kv_len, slot, rows, slots = G.batch_tensors(lengths, seed)
    q, k, v, g, beta, z, w = G.inputs(nk, nv, rows, seed)
    state = torch.randn(slots, nv, 128, 128, device="cuda") * 0.3
    parts = [slice(first, end) for first, end, _ in G.real_rows(lengths)]
    for r in parts:
        change(q[r], k[r], v[r], g[r], beta[r])
    for (n, t), s in zip(lengths, slot.tolist()):
        if t <= n:
            state[s] = 0
    keep = state.clone()
    o = torch.empty(rows, nv, 128, dtype=out, device="cuda")
    fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot), q, k, v, g, beta, state, o, max_q or max(n for n, _ in lengths),
                     z=z if gate else None, norm_w=w if gate else None, eps=G.EPS)
    assert fak.fak_device_status() == 0
    scale = 128 ** -0.5
    for r, s in zip(parts, slot.tolist()):
        want, S, most = rule(q[r], k[r], v[r], g[r], beta[r], keep[s], scale)
        # A row's u goes through three products (the state by its key, T's row, u by the key), whose operands keep 22 bits at least:
        # each is off by 2^-21.4 at most of what it multiplies, keys are no longer than 1: 2^-20 of M.  Errors of earlier rows
        # have either sign and decay with what they belong to, so that they add up like the root of the rows.
        # Decays over rows of a chunk that are below f32's smallest normal number count as none left: each of the t rows before, and
        # the state, is off by 2^-126 of what it brought, at most twice (the strength) what its column then had.
        t = torch.arange(1, want.shape[0] + 1, device="cuda")[:, None, None]
        tol = 2.0 ** -20 * t.sqrt() * most + 2.0 ** -125 * t * most.cummax(0).values
        err = (state[s].double() - S).abs() / (tol[-1][:, None, :] + 1e-37)
        assert float(err.max()) <= 1, ("state", r, float(err.max()))
        length = q[r].double().norm(dim=-1).repeat_interleave(nv // nk, 1)[:, :, None]
        off = tol * scale * length
        if gate:
            # the root of the mean square is off by no more than the row's errors' own; the norm's sums, the gate and their products
            # by 2^-18
            rms = torch.sqrt((want * want).mean(-1, keepdim=True) + G.EPS)
            off = off / rms + want.abs() / rms * torch.sqrt((off * off).mean(-1, keepdim=True)) / rms
            zd = z[r].double()
            off = off * w.double().abs() * (zd / (1 + torch.exp(-zd))).abs()
            want = G.gated(want, w, z[r])
            off = 2 * off + want.abs() * 2.0 ** -18
        err = (o[r].double() - want).abs() / (off + want.abs() * torch.finfo(out).eps / 2 + 1e-37)
        assert float(err.max()) <= 1, ("out", r, float(err.max()))


def nothing(q, k, v, g, beta):
    pass


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_ordinary_rows(fak, out):
    check(fak, nothing, out)
    check(fak, nothing, out, [(1, 1), (5, 9), (28, 28), (65, 65), (129, 200), (700, 700)], 2, 2, 4)


@pytest.mark.parametrize("size", [1e4, 1e6, 1e7, 1e20, 1e-20])
@pytest.mark.parametrize("at", [slice(50, 52), slice(-1, None), slice(0, 3), slice(100, 101)])
def test_rows_of_other_size(fak, size, at):
    """A few rows larger or smaller by far: the rows before them, and those that they have decayed for, keep their digits."""
    def change(q, k, v, g, beta):
        v[at] *= size
    check(fak, change)


@pytest.mark.parametrize("size", [1e4, 1e8, 1e-8])
@pytest.mark.parametrize("rows", [1, 20, 70])
def test_a_reset_behind_rows_of_other_size(fak, size, rows):
    """Rows of another size, a decay that leaves nothing of them, ordinary rows."""
    def change(q, k, v, g, beta):
        v[:rows] *= size
        g[rows:rows + 1] = -float("inf")
    check(fak, change)


@pytest.mark.parametrize("rate", [0.5, 3.0, 20.0])
def test_fast_decays(fak, rate):
    """Every 17th row a million times the others, decays by which it is gone after some of them."""
    def change(q, k, v, g, beta):
        g.fill_(-rate)
        v[3::17] *= 1e6
    check(fak, change)


def test_columns_of_other_size(fak):
    def change(q, k, v, g, beta):
        v[:, :, ::3] *= 1e-9
        v[:, :, 1::3] *= 1e9
    check(fak, change)


def test_values_of_zero_until_late(fak):
    """An empty state stays empty, whatever the rows behind hold."""
    def change(q, k, v, g, beta):
        v[:40] = 0
        v[40:] *= 1e5
    check(fak, change)


def test_the_same_key_and_full_strength(fak):
    """Each row replaces what the one before wrote."""
    def change(q, k, v, g, beta):
        k[:] = k[:1].clone()
        beta.fill_(1.0)
        v[::9] *= 1e5
    check(fak, change)


def test_a_large_state_that_goes(fak):
    """States 10^6 times the rows' values, resets in the first and in the second chunk."""
    def change(q, k, v, g, beta):
        v *= 1e-6
        g[10:11] = -float("inf")
        g[100:101] = -100.0
    check(fak, change)


@pytest.mark.parametrize("size", [1e-2, 1e-5, 1e3, 2e5])
def test_queries_of_any_length(fak, size):
    """Short ones down to f16's smallest steps, and long ones up to its end."""
    def change(q, k, v, g, beta):
        q.copy_((q.double() * size).clamp(-65504, 65504))
    check(fak, change)


def test_queries_of_different_lengths(fak):
    def change(q, k, v, g, beta):
        q[::3] *= 1e-3
        q[1::3] *= 1e3
        q[4::8] = 0
    check(fak, change)


@pytest.mark.parametrize("bits", [8, 12, 14, 16, 18, 20, 22, 24, 28])
def test_around_what_two_f16_hold(fak, bits):
    """Rows of columns that differ by 2^bits, in one head up, in one down, at places that differ by column; one head as it is."""
    def change(q, k, v, g, beta):
        n = v.shape[0]
        at = torch.arange(n, device="cuda")[:, None] % 37 == torch.arange(128, device="cuda")[None] % 37
        v[:, 0] *= torch.where(at, 2.0 ** bits, 1.0)
        v[:, 1] *= torch.where(at, 2.0 ** -bits, 1.0)
    check(fak, change, seed=bits)


def test_values_without_a_pattern(fak):
    """Magnitudes from 2^-40 to 2^40, zeros, decays from none to all."""
    def change(q, k, v, g, beta):
        gen = torch.Generator(device="cuda").manual_seed(v.shape[0])
        v *= torch.exp2(80 * torch.rand(v.shape, generator=gen, device="cuda") - 40)
        v[torch.rand(v.shape, generator=gen, device="cuda") < 0.05] = 0
        g.copy_(-torch.exp(12 * torch.rand(g.shape, generator=gen, device="cuda") - 7))
    check(fak, change)
    check(fak, change, torch.bfloat16, seed=2, nk=2, nv=4)


def test_small_and_large_values_altogether(fak):
    for size in (1e-25, 1e-32, 1e25, 1e33):
        def change(q, k, v, g, beta):
            v *= size
        check(fak, change, lengths=[(100, 100), (64, 64), (20, 20)])


@pytest.mark.parametrize("size", [1e4, 1e7, 1e15])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_norm_and_gate_of_rows_of_other_size(fak, size, out):
    def change(q, k, v, g, beta):
        v[37::50] *= size
    check(fak, change, out, gate=True)
    check(fak, change, out, [(66, 66), (1, 3), (640, 640), (100, 70)], 3, 2, 2, gate=True)


def test_one_sequence_of_rows_of_other_size(fak):
    """Alone, with a bound on the rows far above them: a few rows go over chunks too."""
    def change(q, k, v, g, beta):
        v[1::5] *= 1e12
        v[3::7] = 0
    for n in (1, 5, 29, 64, 65, 150):
        check(fak, change, lengths=[(n, n + n % 2)], max_q=5000, nk=1, nv=2)


def test_infinite_values_leave_the_rows_before_them(fak):
    """(Where a value is an infinity; of NaN up to 63 rows before are given up.)"""
    start, kv_len, slot, rows, slots = G.batch_tensors([(150, 150)], 1, 0)
    q, k, v, g, beta, _, _ = G.inputs(1, 2, rows, 4)
    got = []
    for last in (1.0, float("inf")):
        v[100] = last
        state, o = torch.zeros(slots, 2, 128, 128, device="cuda"), torch.empty(rows, 2, 128, device="cuda")
        fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot), q, k, v, g, beta, state, o, 150)
        got.append(o)
    assert fak.fak_device_status() == 0
    want, _, most = rule(q[:100], k[:100], v[:100], g[:100], beta[:100], torch.zeros(2, 128, 128, device="cuda"), 128 ** -0.5)
    tol = 2.0 ** -20 * torch.arange(1, 101, device="cuda")[:, None, None].sqrt() * most * 128 ** -0.5 * 1.001 + want.abs() * 2.0 ** -24 + 1e-37
    for o in got:
        assert bool(((o[:100].double() - want).abs() <= tol).all())
    assert not bool(torch.isfinite(got[1][100]).any())
