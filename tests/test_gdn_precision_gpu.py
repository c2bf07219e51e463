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


def check(fak, change, out=torch.float32, lengths=LENGTHS, seed=1, nk=1, nv=3):
    start, kv_len, slot, rows, slots = G.batch_tensors(lengths, seed)
    q, k, v, g, beta, _, _ = G.inputs(nk, nv, rows, seed)
    state = torch.randn(slots, nv, 128, 128, device="cuda") * 0.3
    parts = [slice(first, end) for first, end, _ in G.real_rows(lengths)]
    for r in parts:
        change(q[r], k[r], v[r], g[r], beta[r])
    for (n, t), s in zip(lengths, slot.tolist()):
        if t <= n:
            state[s] = 0
    keep = state.clone()
    o = torch.empty(rows, nv, 128, dtype=out, device="cuda")
    fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot), q, k, v, g, beta, state, o, max(n for n, _ in lengths))
    assert fak.fak_device_status() == 0
    scale = 128 ** -0.5
    for r, s in zip(parts, slot.tolist()):
        want, S, most = rule(q[r], k[r], v[r], g[r], beta[r], keep[s], scale)
        # A row's u goes through three products (the state by its key, T's row, u by the key), whose operands keep 22 bits at least:
        # each is off by 2^-21.4 at most of what it multiplies, keys are no longer than 1: 2^-20 of M.  Errors of earlier rows
        # have either sign and decay with what they belong to, so that they add up like the root of the rows.
        tol = 2.0 ** -20 * torch.arange(1, want.shape[0] + 1, device="cuda")[:, None, None].sqrt() * most
        err = (state[s].double() - S).abs() / (tol[-1][:, None, :] + 1e-37)
        assert float(err.max()) <= 1, ("state", r, float(err.max()))
        length = q[r].double().norm(dim=-1).repeat_interleave(nv // nk, 1)[:, :, None]
        err = (o[r].double() - want).abs() / (tol * scale * length + want.abs() * torch.finfo(out).eps / 2 + 1e-37)
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
