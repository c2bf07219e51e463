"""Paged caches, ragged batches and plain 64-bit forms for the tests of the paged KV cache."""
import math

import torch

TOP = {"e4m3": 448.0, "i8": 127.0}
NAN = float("nan")


def batch_tensors(lengths, page, n_pages=None, seed=0, pad_rows=0):
    """lengths: (new rows, positions in all) per sequence.  Pages are handed out in a shuffled order; the table's
    unused places hold a page that is not there.  Returns table, row_start, kv_len (CUDA int32), rows, n_pages."""
    per = [max(0, -(-t // page)) for _, t in lengths]
    n_pages = n_pages or sum(per) + 2
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((len(lengths), max(1, max(per))), n_pages + 7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    start = torch.tensor([0] + [n for n, _ in lengths]).cumsum(0).to(torch.int32)
    kv_len = torch.tensor([t for _, t in lengths], dtype=torch.int32)
    return table.cuda(), start.cuda(), kv_len.cuda(), int(start[-1]) + pad_rows, n_pages


def empty_cache(fak, kind, n_pages, n_kv, page, dh):
    """A cache whose memory holds NaN wherever its type can."""
    shape = (n_pages, n_kv, page, dh)
    if kind == "bf16":
        k, v = (torch.full(shape, NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return fak.KVCache(fak.FAK_KV_BF16, k, v), (k, v, None, None)
    if kind == "e4m3":
        k, v = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    else:
        k, v = (torch.full(shape, 111, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full(shape[:3], NAN, device="cuda") for _ in range(2))
    return fak.KVCache(fak.FAK_KV_E4M3 if kind == "e4m3" else fak.FAK_KV_I8, k, v, ks, vs), (k, v, ks, vs)


def places(table, start, kv_len, page):
    """Per sequence: (rows of the call, pages, slots) of its new rows at positions >= 0."""
    out = []
    t, st, ln = table.cpu(), start.cpu().tolist(), kv_len.cpu().tolist()
    for s in range(len(ln)):
        n = st[s + 1] - st[s]
        pos = torch.arange(ln[s] - n, ln[s])
        keep = pos >= 0
        pos = pos[keep]
        out.append((torch.arange(st[s], st[s + 1])[keep], t[s, pos // page].long(), pos % page))
    return out


def fill(mem, kind, table, kv_len, page, K, V):
    """Puts K, V (per sequence [positions, n_kv, dh] f64 or f32) into the cache's memory by plain torch."""
    k, v, ks, vs = mem
    t = table.cpu()
    for s, (a, b) in enumerate(zip(K, V)):
        pos = torch.arange(a.shape[0])
        pg, sl = t[s, pos // page].long().cuda(), (pos % page).cuda()
        for codes, scales, x in ((k, ks, a), (v, vs, b)):
            x = x.cuda().float()
            if kind == "bf16":
                codes[pg, :, sl] = x.to(torch.bfloat16)
                continue
            most = x.abs().amax(-1)
            y = x * torch.where(most > 0, TOP[kind] / most, 0.0)[..., None]  # (zeros are held as zeros)
            codes[pg, :, sl] = y.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "e4m3" else y.round().to(torch.int8)
            scales[pg, :, sl] = most / TOP[kind]


def held(mem, kind, pages, slots):
    """The cache's vectors at these places in 64 bits: (k, v) [n, n_kv, dh]."""
    out = []
    for codes, scales in ((mem[0], mem[2]), (mem[1], mem[3])):
        x = codes[pages.cuda(), :, slots.cuda()]
        x = (x.view(torch.float8_e4m3fn) if kind == "e4m3" else x).to(torch.float64)
        out.append(x if scales is None else x * scales[pages.cuda(), :, slots.cuda()].double()[..., None])
    return out


def attention(q, k, v, first, scale, window=0, sinks=0, gate=None):
    """Plain attention in 64 bits of rows q [n, nq, dh] at positions first, first + 1, ... over k, v [t, n_kv, dh], and
    what a bf16 result of 32-bit sums over bf16 weights may be off by, element by element.

    With A = sum_j w_j |v_j| / sum_j w_j: a weight is off by 2^-8 of itself (rounded to bf16), by what its score is off
    (a sum of dh products, each addition off by at most 2^-23 of the magnitudes' sum, eight more roundings of the score
    on the way) and by 2^-20 (the exponential); the sum of n weights by n 2^-23; the result is rounded once, 2^-8."""
    n, nq, dh = q.shape
    t, n_kv = k.shape[:2]
    grp = nq // n_kv
    pos = first + torch.arange(n, device=q.device)[:, None]
    j = torch.arange(t, device=q.device)[None]
    sees = j <= pos
    if window:
        sees = sees & ((j > pos - window) | (j < sinks))
    out = torch.zeros(n, nq, dh, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    if t == 0:
        return out, tol
    for h in range(nq):
        kk, vv = k[:, h // grp], v[:, h // grp]
        qq = q[:, h].double()
        s = (qq @ kk.T * scale).masked_fill(~sees, -math.inf)
        mag = (qq.abs() @ kk.nan_to_num(0, 0, 0).abs().T * scale).masked_fill(~sees, 0)
        w = torch.softmax(s, -1)
        w = torch.where(sees, w, torch.zeros_like(w))
        live = sees.any(-1)
        # only what a row sees is multiplied: NaN elsewhere stays out of it
        o = w @ vv.nan_to_num(0, 0, 0)
        odd = ~torch.isfinite(vv)
        if odd.any():
            o = o + torch.stack([torch.where(sees[i][:, None] & odd, vv, torch.zeros_like(vv)).sum(0) for i in range(n)])
        a = w @ vv.nan_to_num(0, 0, 0).abs()
        off = 2.0**-8 + 2 * (dh + 8) * 2.0**-23 * mag.amax(-1) + t * 2.0**-23 + 2.0**-20
        tol[:, h] = torch.where(live[:, None], a * off[:, None] + 2.0**-8 * o.abs().nan_to_num(0, 0, 0) * (1 + off[:, None]), torch.zeros_like(a))
        out[:, h] = torch.where(live[:, None], o, torch.zeros_like(o))
    if gate is not None:
        g = torch.sigmoid(gate.double())
        out, tol = out * g, tol * g + 2.0**-20 * out.abs().nan_to_num(0, 0, 0)
    return out, tol + 1e-30


def check(got, want, tol, what):
    got = got.double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    bad = ~(err <= tol) & ~same
    if bad.any():
        i = int(torch.where(torch.isnan(err), torch.full_like(err, math.inf), err / tol).flatten().argmax())
        assert False, "%s: %d of %d off; worst at %d: %g for %g, allowed %g" % (
            what, int(bad.sum()), bad.numel(), i, float(got.flatten()[i]), float(want.flatten()[i]), float(tol.flatten()[i]))
