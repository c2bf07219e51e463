"""fak_residual_norm against its formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
EPS = 1e-6
T = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def fak():
    from q4_weight_quantized_block_gb300 import build
    build.build()
    import q4_weight_quantized_block_gb300 as m
    assert torch.cuda.is_available()
    return m


def case(fak, rows, d, ht="f32", yt="f32", nt="bf16", post=True, y_w=True, w=True, gate="rows", sigmoid=False, scale=0.7, off=0.0,
         views=False, with_y=True, with_n=True, seed=0, size=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731

    def tensor(dtype, by):
        if not views:
            return (size * rand(rows, d)).to(T[dtype])
        return (size * rand(rows, d + by)).to(T[dtype])[:, by // 2:by // 2 + d]

    h, y, n = tensor(ht, 6), tensor(yt, 10), tensor(nt, 2)
    wt, ywt = 1 - off + 0.1 * rand(d), 1 - off + 0.1 * rand(d)
    gt = {"none": None, "rows": rand(rows, d), "row": rand(1, d).expand(rows, d), "column": rand(rows, 1).expand(rows, d),
          "one": rand(1, 1).expand(rows, d), "slice": rand(rows, d + 3)[:, 3:]}[gate]
    h0 = h.double().clone()
    y0 = y.clone()
    fak.fak_residual_norm(h, y if with_y else None, n if with_n else None, w=wt if w else None, post_norm=post,
                          y_w=ywt if y_w else None, gate=gt, gate_sigmoid=sigmoid, scale=scale, eps=EPS, gain_offset=off)
    want_h = h0
    # f32: the sum of d squares is off by at most 40 * 2^-24 of itself (a thread's 32 terms, then a tree); half of it in the
    # root; a handful of roundings in the products; sigmoid's exponential and division by 2^-20
    rel = 2.0 ** -18
    if with_y:
        yy = y.double()
        if post:
            yy = yy / torch.sqrt((yy * yy).mean(-1, keepdim=True) + EPS)
            if y_w:
                yy = yy * (off + ywt.double())
        if gt is not None:
            yy = yy * (torch.sigmoid(gt.double()) if sigmoid else gt.double())
        want_h = h0 + scale * yy
        tol = rel * (scale * yy).abs() + (2.0 ** -23 + torch.finfo(T[ht]).eps / 2) * want_h.abs() + rel * 2.0 ** -20
        assert bool(((h.double() - want_h).abs() <= tol).all())
    else:
        assert torch.equal(h.double(), h0)
    if with_n:
        r = 1 / torch.sqrt((want_h * want_h).mean(-1, keepdim=True) + EPS)
        want = want_h * r * ((off + wt.double()) if w else 1.0)
        slack = rel * (scale * yy).abs() * r * 2 if with_y else 0.0
        assert bool(((n.double() - want).abs() <= want.abs() * (rel + torch.finfo(T[nt]).eps / 2) + slack + 2.0 ** -60).all())
    assert torch.equal(y, y0)
    assert fak.fak_device_status() == 0


@pytest.mark.parametrize("d", [1, 2, 3, 4, 31, 128, 255, 256, 1023, 1024, 1028, 4096, 4100, 5119, 5120, 8192, 8196, 16384, 17408, 32768, 32767])
def test_widths(fak, d):
    case(fak, 5, d, seed=d)


@pytest.mark.parametrize("d", [6, 30, 1022, 2050, 4094, 8190, 8194, 16382, 20002, 32766])
def test_widths_by_twos(fak, d):
    case(fak, 5, d, seed=d)
    case(fak, 3, d, "bf16", "bf16", "f32", gate="one", seed=d + 1)
    case(fak, 3, d, "bf16", "f32", "bf16", gate="none", views=True, seed=d + 2)


@pytest.mark.parametrize("d", [1001, 1026, 1500, 5122, 9999, 10004, 16390])
def test_many_rows_of_odd_widths(fak, d):
    case(fak, 700, d, "bf16", seed=d)
    case(fak, 700, d, "f32", "bf16", "f32", gate="slice", views=True, seed=d + 1)


@pytest.mark.parametrize("ht", list(T))
@pytest.mark.parametrize("yt", list(T))
@pytest.mark.parametrize("nt", list(T))
def test_types(fak, ht, yt, nt):
    case(fak, 7, 640, ht, yt, nt, seed=1)
    case(fak, 7, 641, ht, yt, nt, seed=2, views=True)


@pytest.mark.parametrize("gate", ["none", "rows", "row", "column", "one", "slice"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("post", [False, True])
def test_gates(fak, gate, sigmoid, post):
    case(fak, 9, 512, gate=gate, sigmoid=sigmoid, post=post, seed=3)
    case(fak, 4, 77, gate=gate, sigmoid=sigmoid, post=post, seed=4)


@pytest.mark.parametrize("over", [dict(y_w=False), dict(w=False), dict(off=1.0), dict(off=1.0, w=False, y_w=False), dict(with_y=False),
                                  dict(with_n=False), dict(scale=0.0), dict(scale=-2.0), dict(size=1e-4), dict(size=1e6),
                                  dict(views=True)])
def test_parts(fak, over):
    case(fak, 6, 1280, seed=5, **over)
    case(fak, 6, 321, seed=6, **over)


def test_rows(fak):
    for rows in (1, 64, 3000):
        case(fak, rows, 5120, seed=rows)


def test_zeros_and_bad_values_stay_in_their_row(fak):
    h, y = torch.zeros(4, 384, device="cuda"), torch.zeros(4, 384, device="cuda")
    y[1], h[2, 5], y[3, 7] = 1.0, float("nan"), float("inf")
    n = torch.empty(4, 384, device="cuda")
    fak.fak_residual_norm(h, y, n, post_norm=True)
    assert bool((n[0] == 0).all()) and bool((h[0] == 0).all())
    assert float((n[1] - 1).abs().max()) < 1e-5
    assert bool(n[2].isnan().all()) and bool(n[3].isnan().any())


def test_nothing_to_do(fak):
    h = torch.randn(3, 64, device="cuda")
    keep = h.clone()
    fak.fak_residual_norm(h)
    fak.fak_residual_norm(h[:0], h[:0], h[:0])
    assert torch.equal(h, keep) and fak.fak_device_status() == 0


def test_captured_and_on_another_stream(fak):
    h0, y = torch.randn(33, 1024, device="cuda"), torch.randn(33, 1024, device="cuda")
    a, na = h0.clone(), torch.empty_like(h0)
    fak.fak_residual_norm(a, y, na, post_norm=True)
    b, nb = h0.clone(), torch.empty_like(h0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fak.fak_residual_norm(b, y, nb, post_norm=True)
    torch.cuda.current_stream().wait_stream(side)
    c, nc = h0.clone(), torch.empty_like(h0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fak.fak_residual_norm(c, y, nc, post_norm=True)
    graph.replay()
    assert torch.equal(a, b) and torch.equal(na, nb) and torch.equal(a, c) and torch.equal(na, nc)
