"""A Gated DeltaNet layer run from the operators as a serving program runs them: fak_residual_norm, the Q4_K input
projection, fak_gdn_conv, fak_gdn_attn with the gated norm, the output projection, and the norm around the next block; a
prompt in chunks, then drafted and single tokens, two sequences in one batch.  The body against the oracle's step in 64
bits on the projection's own rows, the norms against their formula."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import oracle
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fak():
    from q4_weight_quantized_block_gb300 import build
    build.build()
    import q4_weight_quantized_block_gb300 as m
    assert torch.cuda.is_available()
    return m


def rms(x):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)


@pytest.mark.parametrize("nk,nv", [(2, 6), (1, 2)])
def test_layer_in_chunks_and_single_tokens(fak, nk, nv):
    D = 512
    d = oracle.MixerDims(nk=nk, nv=nv)
    width, mix, chans = d.gdn_in, nv * 128, (2 * nk + nv) * 128
    W = torch.from_numpy(oracle.q4k_pack(synth.normal(6, 1, (width, D), 0.05))).cuda()
    Wo = torch.from_numpy(oracle.q4k_pack(synth.normal(6, 2, (D, mix), 0.02))).cuda()
    prm = oracle.MixerParams(conv_w=0.5 * synth.normal(6, 3, (chans, 4)), a_log=np.log(1 + 15 * synth.uniforms(6, 4, nv)),
                             dt_bias=synth.normal(6, 5, (nv,)) - 3, norm_w=1 + 0.1 * synth.normal(6, 6, (128,)))
    dev = {n: torch.from_numpy(np.ascontiguousarray(prm.arrays[n], np.float32)).cuda()
           for n in ("conv_w", "a_log", "dt_bias", "norm_w")}
    conv_state = torch.full((5, 3, chans), float("nan"), device="cuda")
    S = torch.full((5, nv, 128, 128), float("nan"), device="cuda")
    slot = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    oc, os_ = [np.zeros((chans, 3)) for _ in range(2)], [np.zeros((nv, 128, 128)) for _ in range(2)]
    ln, step = [0, 0], 0
    for new in ((70, 133), (150, 1), (1, 1), (4, 3), (1, 1), (0, 3)):
        rows = sum(new)
        h = torch.from_numpy(synth.normal(6, 50 + step, (rows, D), 1.0)).cuda()
        y = torch.from_numpy(synth.normal(6, 90 + step, (rows, D), 1.0)).cuda()
        step += 1
        ln = [a + b for a, b in zip(ln, new)]
        few = rows <= 64  # a batch of tokens: f32 rows for the matrix-vector products
        n = torch.empty(rows, D, dtype=torch.float32 if few else torch.bfloat16, device="cuda")
        want_h = h.double() + rms(y.double())
        fak.fak_residual_norm(h, y, n, post_norm=True)
        assert float((h.double() - want_h).abs().max()) <= 1e-5
        assert float((n.double() - rms(want_h)).abs().max()) <= float(rms(want_h).abs().max()) * (2.0 ** -8 if not few else 2.0 ** -18)
        T = torch.empty(rows, width, device="cuda")
        out = torch.empty(rows, nv, 128, dtype=n.dtype, device="cuda")
        Y = torch.empty(rows, D, device="cuda")
        if few:
            fak.fak_q4k_gemv_batch(W, width, D, n, rows, T)
        else:
            fak.fak_q4k_gemm(W, width, D, n, rows, T)
        batch = fak.GDNBatch(torch.tensor([0, new[0], rows], dtype=torch.int32, device="cuda"),
                             torch.tensor(ln, dtype=torch.int32, device="cuda"), slot)
        q, k = (torch.empty(rows, nk, 128, dtype=torch.float16, device="cuda") for _ in range(2))
        v = torch.empty(rows, nv, 128, dtype=torch.bfloat16, device="cuda")
        g, beta = torch.empty(rows, nv, device="cuda"), torch.empty(rows, nv, device="cuda")
        z = T[:, chans:chans + mix].view(rows, nv, 128)
        fak.fak_gdn_conv(batch, T[:, :chans], T[:, chans + mix:chans + mix + nv], T[:, chans + mix + nv:], dev["conv_w"],
                         dev["a_log"], dev["dt_bias"], conv_state, q, k, v, g, beta)
        fak.fak_gdn_attn(batch, q, k, v, g, beta, S, out, max(new), z=z, norm_w=dev["norm_w"])
        if few:
            fak.fak_q4k_gemv_batch(Wo, D, mix, out, rows, Y)
        else:
            fak.fak_q4k_gemm(Wo, D, mix, out, rows, Y)
        want_h = h.double() + Y.double()
        fak.fak_residual_norm(h, Y, n)
        assert float((h.double() - want_h).abs().max()) <= 1e-5
        assert fak.fak_device_status() == 0 and bool(torch.isfinite(n).all())
        Th, Oh, r = T.cpu().numpy().astype(np.float64), out.float().cpu().numpy().reshape(rows, -1), 0
        for s in range(2):
            for i in range(new[s]):
                want, _ = oracle.gdn_step(d, prm, Th[r], oc[s], os_[s])
                got = Oh[r].astype(np.float64)
                # v to bf16 (2^-8 of itself at most), q and k to f16 (2^-11), results to bf16: a hundredth or so of a row's norm
                assert np.linalg.norm(got - want) <= 0.02 * np.linalg.norm(want), (step, s, i)
                r += 1
        for s in range(2):
            got = S[slot[s]].double().cpu().numpy()
            assert np.linalg.norm(got - os_[s]) <= 0.01 * np.linalg.norm(os_[s])
