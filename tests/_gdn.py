"""Ragged batches, and plain 64-bit forms of the Gated DeltaNet operators and the norms around a block, for their tests."""
import torch

EPS = 1e-6


def batch_tensors(lengths, seed=0, pad_rows=0, spare=2):
    """lengths: (new rows, positions in all) per sequence.  Returns row_start, kv_len, slot (CUDA int32), rows, slots."""
    start = torch.tensor([0] + [n for n, _ in lengths]).cumsum(0).to(torch.int32)
    kv_len = torch.tensor([t for _, t in lengths], dtype=torch.int32)
    slots = len(lengths) + spare
    slot = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:len(lengths)].to(torch.int32)
    return start.cuda(), kv_len.cuda(), slot.cuda(), int(start[-1]) + pad_rows, slots


def real_rows(lengths):
    """Per sequence: first row of the call that is no padding, behind its last row, whether it begins with an empty state."""
    out, at = [], 0
    for n, t in lengths:
        out.append((at + n - min(n, t), at + n, t <= n))
        at += n
    return out


def conv_ref(x, w, before):
    """c [rows, channels], state behind: causal convolution of 4 taps and silu in 64 bits."""
    x = torch.cat([before.double(), x.double()])
    n = x.shape[0] - 3
    c = sum(x[j:j + n] * w[:, j].double() for j in range(4))
    return c / (1 + torch.exp(-c)), x[-3:]


def gdn_ref(q, k, v, g, beta, S, scale):
    """o [rows, nv, 128], S behind [nv, 128, 128], and the largest length that a column of S or a value had, in 64 bits."""
    nv = v.shape[1]
    q, k = (t.double().repeat_interleave(nv // t.shape[1], 1) for t in (q, k))
    v, g, beta, S = v.double(), g.double(), beta.double(), S.double()
    most = torch.maximum(S.norm(dim=1).amax(), v.abs().amax() if v.numel() else S.new_zeros(()))
    out = torch.empty_like(v)
    for t in range(v.shape[0]):
        S = torch.exp(g[t])[:, None, None] * S
        u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
        S = S + k[t][:, :, None] * u[:, None, :]
        out[t] = scale * torch.einsum("hkv,hk->hv", S, q[t])
        most = torch.maximum(most, S.norm(dim=1).amax())
    return out, S, float(most)


def gated(o, w, z):
    if w is not None:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * w.double()
    if z is not None:
        z = z.double()
        o = o * z / (1 + torch.exp(-z))
    return o


def inputs(nk, nv, rows, seed, out=torch.bfloat16, wild=False):
    """q, k, v, g, beta, z, norm_w of a call: unit queries and keys with a common part, decays of slow and of fast heads."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k = ((lambda x: (x / x.norm(dim=-1, keepdim=True)).half())(rand(rows, nk, 128) + 0.5) for _ in range(2))
    v = (1.5 * rand(rows, nv, 128)).bfloat16()
    rate = torch.exp(3 * rand(nv) - 3)
    g = -rate * torch.rand(rows, nv, generator=gen, device="cuda")
    beta = torch.sigmoid(2 * rand(rows, nv))
    if wild and rows:
        g = torch.where(torch.rand(rows, nv, generator=gen, device="cuda") < 0.1, torch.full_like(g, -1e4), g)
        g[::7] = 0.0
        g[3::11] = -float("inf")
        beta[::5] = 0.0
        beta[1::9] = 1.0
        k[2::6] = k[1::6][:k[2::6].shape[0]]  # the same key twice
        v[4::8] *= 1e4
    return q, k, v, g, beta, rand(rows, nv, 128), 1 + 0.1 * rand(128)
