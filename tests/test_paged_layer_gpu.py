"""A full-attention layer run from the operators as a serving program runs them: the Q4_K input projections, fak_kv_append,
fak_paged_attn with the output gate, the output projection; a prompt in chunks, then single tokens, two sequences in one
batch.  Against the oracle's gated attention step in 64 bits on the projections' own rows."""
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


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_layer_in_chunks_and_single_tokens(fak, kind):
    D, nq, n_kv, dh, page, rot, theta = 512, 6, 2, 256, 16, 64, 1e7
    width = (2 * nq + 2 * n_kv) * dh
    W = torch.from_numpy(oracle.q4k_pack(synth.normal(5, 1, (width, D), 0.05))).cuda()
    Wo = torch.from_numpy(oracle.q4k_pack(synth.normal(5, 2, (D, nq * dh), 0.02))).cuda()
    prm = oracle.MixerParams(q_norm_w=1 + 0.1 * synth.normal(5, 3, (dh,)), k_norm_w=1 + 0.1 * synth.normal(5, 4, (dh,)))
    qw, kw = (torch.from_numpy(np.asarray(x, np.float32)).cuda() for x in (prm.arrays["q_norm_w"], prm.arrays["k_norm_w"]))
    rope = torch.from_numpy(fak.fak_rope_table(rot, theta)).cuda()
    shape = (24, n_kv, page, dh)
    if kind == "bf16":
        cache = fak.KVCache(fak.FAK_KV_BF16, *(torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    else:
        cache = fak.KVCache(fak.FAK_KV_I8, *(torch.empty(shape, dtype=torch.int8, device="cuda") for _ in range(2)),
                            *(torch.empty(shape[:3], device="cuda") for _ in range(2)))
    table = torch.from_numpy(np.random.default_rng(0).permutation(24).astype(np.int32).reshape(2, 12)).cuda()
    d = oracle.MixerDims(nq=nq, nkv=n_kv, rot=rot, theta=theta)
    kc, vc = ([np.zeros((n_kv, 192, dh)) for _ in range(2)] for _ in range(2))
    ln, step = [0, 0], 0
    for new in ((70, 33), (50, 1), (1, 1), (1, 1), (0, 3)):
        rows = sum(new)
        X = torch.from_numpy(synth.normal(5, 50 + step, (rows, D), 1.0)).cuda().to(torch.bfloat16)
        step += 1
        T = torch.empty(rows, width, device="cuda")
        fak.fak_q4k_gemm(W, width, D, X, rows, T)
        qg = T[:, :2 * nq * dh].view(rows, nq, 2 * dh)
        k, v = T[:, 2 * nq * dh:].view(rows, 2, n_kv, dh).unbind(1)
        ln = [a + b for a, b in zip(ln, new)]
        batch = fak.KVBatch(table, torch.tensor([0, new[0], rows], dtype=torch.int32, device="cuda"),
                            torch.tensor(ln, dtype=torch.int32, device="cuda"))
        q = torch.empty(rows, nq, dh, dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(q)
        fak.fak_kv_append(cache, batch, k, v, q=qg[..., :dh], q_out=q, q_norm_w=qw, k_norm_w=kw, rope=rope, rot=rot)
        n = fak.fak_paged_attn_workspace_bytes(cache, batch, nq, rows, max(new), max(ln))
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        fak.fak_paged_attn(cache, batch, q, out, max(new), max(ln), gate=qg[..., dh:], workspace=ws)
        Y = torch.empty(rows, D, device="cuda")
        fak.fak_q4k_gemm(Wo, D, nq * dh, out, rows, Y)
        assert fak.fak_device_status() == 0 and bool(torch.isfinite(Y).all())
        Th, Oh, r = T.cpu().numpy().astype(np.float64), out.float().cpu().numpy().reshape(rows, -1), 0
        for s in range(2):
            for i in range(new[s]):
                t = Th[r]
                want = oracle.attn_step(d, prm, t[:2 * nq * dh], t[2 * nq * dh:(2 * nq + n_kv) * dh],
                                        t[(2 * nq + n_kv) * dh:], ln[s] - new[s] + i, kc[s], vc[s])
                got = Oh[r].astype(np.float64)
                # the cache's own rounding (bf16 2^-8, int8 1/254 of the largest of 256: scores of order one move by
                # hundredths at most) and bf16 weights and results: a few hundredths of the row's norm at most
                assert np.linalg.norm(got - want) <= 0.03 * np.linalg.norm(want), (step, s, i)
                r += 1
