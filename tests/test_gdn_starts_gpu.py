"""The Gated DeltaNet operators and the norm around a block where numbers are out of range: a sequence comes out right or not at
all, a call's arguments are refused as others are."""
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


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# starts, and the sequences that are left out besides those whose own bounds fall: sequence s has its records from place
# start / 64 + s on, one for 64 rows (where there are many sequences, from start / 28 on: disjoint rows never share one)
FALLING = {
    # both at 3
    "one place": ([192, 256, 64, 128], [0, 2]),
    # 5 to 7, 3 to 5, 7
    "one place, longer": ([320, 500, 100, 256, 300], [0, 2, 3]),
    "no place in common": ([300, 400, 0, 100], []),
    "few rows": ([192, 212, 64, 128], []),
}


@pytest.mark.parametrize("name", list(FALLING))
@pytest.mark.parametrize("spare", [0, 40])
def test_starts_that_fall(fak, name, spare):
    """Sequences of disjoint rows; with spare, sequences without rows behind them."""
    starts, out = FALLING[name]
    out = [] if spare else out
    rows, n = 512, len(starts) - 1
    lengths = [b - a for a, b in zip(starts, starts[1:])]
    start = i32(*(starts + [starts[-1]] * spare))
    kv_len = i32(*([max(m, 0) for m in lengths] + [0] * spare))
    slot = torch.randperm(n + spare + 2, generator=torch.Generator().manual_seed(3))[:n + spare].to(torch.int32).cuda()
    q, k, v, g, beta, _, _ = G.inputs(1, 2, rows, 8)
    state = torch.full((n + spare + 2, 2, 128, 128), NAN, device="cuda")
    o = torch.full((rows, 2, 128), 7.0, device="cuda")
    fak.fak_gdn_attn(fak.GDNBatch(start, kv_len, slot), q, k, v, g, beta, state, o, 256)
    assert fak.fak_device_status() == 7
    seen = torch.zeros(rows, dtype=torch.bool)
    for s, m in enumerate(lengths):
        if m < 0 or s in out:
            assert bool(state[slot[s]].isnan().all())
            continue
        r = slice(starts[s], starts[s + 1])
        seen[r] = True
        want, S, most = G.gdn_ref(*(t[r] for t in (q, k, v, g, beta)), torch.zeros_like(state[slot[s]]), 128 ** -0.5)
        tol = 2.0 ** -20 * m ** 0.5 * most  # (as the operator's other tests have it)
        assert float((state[slot[s]].double() - S).abs().max()) <= tol
        assert float((o[r].double() - want).abs().max()) <= tol * 128 ** -0.5 + 2.0 ** -23 * float(want.abs().max())
    assert bool((o[~seen.cuda()] == 7).all())
    assert fak.fak_device_status() == 0


BAD = {
    "slot of a sequence without rows": ([0, 5, 5, 9], [5, 3, 4], [0, 99, 1]),
    "negative slot, the last": ([0, 5, 9, 9], [5, 4, 0], [0, 1, -1]),
    "length of a sequence without rows": ([0, 0, 5, 9], [-1, 5, 4], [2, 0, 1]),
    "a start that falls, its rows another's": ([0, 9, 4, 9], [9, 4, 5], [0, 1, 2]),
}


@pytest.mark.parametrize("name", list(BAD))
@pytest.mark.parametrize("rows", [9, 900])
@pytest.mark.parametrize("spare", [0, 70])
def test_sequences_that_no_row_leads_to_are_recorded(fak, name, rows, spare):
    """By both operators, with few rows and many, and among more sequences than a warp looks at together."""
    starts, lens, slots = BAD[name]
    if spare:
        starts, lens, slots = starts + [starts[-1]] * spare, lens + [0] * spare, slots + [3] * spare
    batch = fak.GDNBatch(i32(*starts), i32(*lens), i32(*slots))
    x, ba = torch.randn(rows, 512, device="cuda"), torch.randn(rows, 2, device="cuda")
    q, k = (torch.empty(rows, 1, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    v = torch.empty(rows, 2, 128, dtype=torch.bfloat16, device="cuda")
    g, beta = torch.empty(rows, 2, device="cuda"), torch.empty(rows, 2, device="cuda")
    conv_state, zero = torch.zeros(4, 3, 512, device="cuda"), torch.zeros(2, device="cuda")
    fak.fak_gdn_conv(batch, x, ba, ba, torch.randn(512, 4, device="cuda"), zero, zero, conv_state, q, k, v, g, beta)
    assert fak.fak_device_status() == 7
    q, k, v, g, beta, _, _ = G.inputs(1, 2, rows, 8)
    fak.fak_gdn_attn(batch, q, k, v, g, beta, torch.zeros(4, 2, 128, 128, device="cuda"), torch.empty(rows, 2, 128, device="cuda"), 9)
    assert fak.fak_device_status() == 7
    good = fak.GDNBatch(i32(0, 5, 9), i32(5, 4), i32(0, 1))
    fak.fak_gdn_conv(good, x, ba, ba, torch.randn(512, 4, device="cuda"), zero, zero, conv_state, q, k, v, g, beta)
    assert fak.fak_device_status() == 0


@pytest.mark.parametrize("over", [dict(max_q=1 << 31), dict(max_q=2.5), dict(scale=1e39), dict(scale="1"), dict(eps=1e300), dict(eps=None)])
def test_numbers_that_the_call_cannot_hold_are_refused(fak, over):
    """By the binding, with its own error."""
    batch = fak.GDNBatch(i32(0, 3), i32(3), i32(0))
    q, k, v, g, beta, _, _ = G.inputs(1, 2, 3, 8)
    state, o, h = torch.zeros(1, 2, 128, 128, device="cuda"), torch.empty(3, 2, 128, device="cuda"), torch.ones(3, 64, device="cuda")
    with pytest.raises(fak.FakError) as e:
        fak.fak_gdn_attn(batch, q, k, v, g, beta, state, o, **{**dict(max_q=3), **over})
    assert e.value.status == 1
    if "max_q" in over:
        return
    with pytest.raises(fak.FakError) as e:
        fak.fak_residual_norm(h, h.clone(), h.clone(), **over)
    assert e.value.status == 1
    if "eps" in over:
        x, ba, n = torch.randn(3, 512, device="cuda"), torch.randn(3, 2, device="cuda"), torch.zeros(2, device="cuda")
        with pytest.raises(fak.FakError) as e:
            fak.fak_gdn_conv(batch, x, ba, ba, torch.randn(512, 4, device="cuda"), n, n, torch.zeros(1, 3, 512, device="cuda"), q, k, v, g,
                             beta, **over)
        assert e.value.status == 1
