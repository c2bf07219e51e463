"""What is measured of the Gated DeltaNet layers' operators on ragged batches, and of the norms around a block.

Three operators, each as a serving program calls it between the Q4_K projections of a layer:
  norm   fak_residual_norm: a block's output normed, gated, scaled and added to the residual stream, and the
         norm before the next block
  conv   fak_gdn_conv: the short causal convolution over the input projection's rows, with its state; the l2 norms
         of queries and keys, the heads' decays and write strengths
  gdn    fak_gdn_attn: the gated delta rule (linear attention with a decay for each head) over single tokens,
         chunks and whole prompts, with its state and the gated norm of its output

A case of norm holds the rows, the width, the types and what is fused; a case of conv or gdn the head layout, the
number of sequences and the most new rows a sequence has; with "ragged" the sequences differ, and with "fresh" some
of them begin at position 0 and so from an empty state.
"""
import math

import torch

own = False

EPS = 1e-6
DH = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _norm(name, rows, d, h="f32", y="f32", n="bf16", post=False, gate="none", scale=1.0, offset=0.0):
    return dict(name=name, op="norm", rows=rows, d=d, h=h, y=y, n=n, post=post, gate=gate, scale=scale, offset=offset)


def _conv(name, nk, nv, seqs, new, kind="f32", ragged=False, fresh=False):
    return dict(name=name, op="conv", nk=nk, nv=nv, seqs=seqs, new=new, kind=kind, ragged=ragged, fresh=fresh)


def _gdn(name, nk, nv, seqs, new, out="bf16", gate=True, ragged=False, fresh=False):
    return dict(name=name, op="gdn", nk=nk, nv=nv, seqs=seqs, new=new, out=out, gate=gate, ragged=ragged, fresh=fresh)


def listed():
    return [
        # a decoded token of one sequence, on its way to the next matrix-vector product
        _norm("norm 1x5120", 1, 5120, n="f32"),
        # a batch of decoded tokens with norms on both sides of the block and a gain of 1 + w
        _norm("norm 64x5120 both sides", 64, 5120, post=True, scale=0.5, offset=1.0),
        # the tokens of a long prompt, each with a gate of its own channels
        _norm("norm 16384x5120 gated", 16384, 5120, post=True, gate="rows"),
        # one decoded token: 16 key and 48 value heads of 128
        _conv("conv 1 token", 16, 48, 1, 1),
        # a full batch of decoded tokens, bf16 projections
        _conv("conv 64 tokens bf16", 16, 48, 64, 1, kind="bf16"),
        # chunks of prompts of all lengths
        _conv("conv 8 chunks", 16, 48, 8, 2048, ragged=True, fresh=True),
        # a decode step of one sequence, f32 for the matrix-vector product that follows
        _gdn("gdn 1 token", 16, 48, 1, 1, out="f32"),
        # a decode step of a full batch
        _gdn("gdn 64 tokens", 16, 48, 64, 1),
        # drafted tokens of sixteen sequences
        _gdn("gdn 16x4 tokens", 16, 48, 16, 4, out="f32"),
        # a prompt's first chunk beside others, of all lengths down to a single token
        _gdn("gdn 8 chunks", 16, 48, 8, 1000, ragged=True, fresh=True),
        # a whole prompt at once
        _gdn("gdn prompt 8192", 16, 48, 1, 8192, fresh=True),
        # prompts of a batch, one value head to a key head
        _gdn("gdn 16 prompts 2048", 16, 16, 16, 2048, ragged=True, fresh=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "conv", "gdn", "gdn", "gdn"])
    if op == "norm":
        case = _norm("", _log(rng, 1, 16384), _log(rng, 64, 8192), rng.choice(["f32", "f32", "bf16"]), rng.choice(["f32", "bf16"]),
                     rng.choice(["f32", "bf16"]), rng.random() < 0.5, rng.choice(["none", "rows", "columns", "sigmoid"]),
                     rng.choice([1.0, 0.5, 0.22]), rng.choice([0.0, 1.0]))
        if rng.random() < 0.7:
            case["d"] = max(64, case["d"] // 64 * 64)
        while case["rows"] * case["d"] > 5120 << 14:
            case["rows"] -= case["rows"] // 2
    else:
        nk, nv = rng.choice([(16, 48), (16, 48), (16, 32), (16, 16), (4, 12), (2, 2), (1, 3), (5, 10)])
        seqs, new = _log(rng, 1, 64), 1 if rng.random() < 0.35 else _log(rng, 2, 8192)
        # not above the largest listed cases
        while seqs * new * nv > 8192 * 48:
            if seqs >= new:
                seqs -= seqs // 2
            else:
                new -= new // 2
        ragged, fresh = rng.random() < 0.7, rng.random() < 0.5
        case = (_conv("", nk, nv, seqs, new, rng.choice(["f32", "bf16"]), ragged, fresh) if op == "conv"
                else _gdn("", nk, nv, seqs, new, rng.choice(["f32", "bf16"]), rng.random() < 0.7, ragged, fresh))
    del case["name"]
    return case


def _lengths(case):
    """New rows of each sequence, and the positions that stand before them."""
    new, past = [], []
    for i in range(case["seqs"]):
        new.append(1 + (case["new"] - 1) * ((5 * i + 8) % 9) // 8 if case["ragged"] and case["seqs"] > 1 else case["new"])
        past.append(0 if case["fresh"] and i % 2 == 0 else 100 + 7 * i)
    return new, past


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, like=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=like)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    s = dict(case=case)
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        s["h"] = (3 * normal(rows, d)).to(TYPES[case["h"]])
        s["y"] = normal(rows, d).to(TYPES[case["y"]])
        s["n"] = torch.empty(rows, d, dtype=TYPES[case["n"]], device=dev)
        s["w"] = 1 - case["offset"] + 0.1 * normal(d)
        s["y_w"] = 1 - case["offset"] + 0.1 * normal(d)
        # a gate for each value, for each channel (a layer's scale), or one for each row (through a sigmoid)
        s["gate"] = {"none": None, "rows": normal(rows, d), "columns": 0.1 * normal(1, d).expand(rows, d),
                     "sigmoid": normal(rows, 1).expand(rows, d)}[case["gate"]]
        return s
    nk, nv, seqs = case["nk"], case["nv"], case["seqs"]
    new, past = _lengths(case)
    rows, chans = sum(new), (2 * nk + nv) * DH
    s["start"] = torch.tensor([sum(new[:i]) for i in range(seqs + 1)], dtype=torch.int32, device=dev)
    s["len"] = torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32, device=dev)
    # the sequences' states stand in the pool in no order, two places are another batch's
    s["slot"] = torch.randperm(seqs + 2, generator=g, device=dev)[:seqs].to(torch.int32)
    s["max_q"] = max(new)
    # the heads' decay rates and step sizes as such layers begin with: rates of 1 to 16, steps of 0.001 to 0.1
    a_log = torch.log(1 + 15 * uniform(nv))
    step = torch.exp(math.log(0.001) + math.log(100.0) * uniform(nv))
    dt_bias = step + torch.log(-torch.expm1(-step))
    if case["op"] == "conv":
        # the rows as the input projection leaves them: q | k | v | z | b | a
        t = normal(rows, chans + nv * DH + 2 * nv).to(TYPES[case["kind"]])
        s["x"], s["b"], s["a"] = t[:, :chans], t[:, -2 * nv : -nv], t[:, -nv:]
        s["conv_w"] = 0.5 * normal(chans, 4)
        s["a_log"], s["dt_bias"] = a_log, dt_bias
        s["state"] = normal(seqs + 2, 3, chans)
        for what, heads, dtype in (("q", nk, torch.float16), ("k", nk, torch.float16), ("v", nv, torch.bfloat16)):
            s[what] = torch.empty(rows, heads, DH, dtype=dtype, device=dev)
        s["g"], s["beta"] = torch.empty(rows, nv, device=dev), torch.empty(rows, nv, device=dev)
    else:
        # queries and keys of the convolution's silu (their means are above zero), of length 1
        for what in ("q", "k"):
            x = normal(rows, nk, DH)
            x = x * torch.sigmoid(x)
            s[what] = (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)).to(torch.float16)
            del x
        s["v"] = (1.5 * normal(rows, nv, DH)).to(torch.bfloat16)
        s["beta"] = torch.sigmoid(normal(rows, nv))
        s["g"] = -torch.exp(a_log) * torch.nn.functional.softplus(normal(rows, nv) + dt_bias)
        s["state"] = 0.3 * normal(seqs + 2, nv, DH, DH)
        s["z"] = normal(rows, nv * DH + 64)[:, : nv * DH].view(rows, nv, DH) if case["gate"] else None
        s["norm_w"] = 1 + 0.1 * normal(DH) if case["gate"] else None
        s["out"] = torch.empty(rows, nv, DH, dtype=TYPES[case["out"]], device=dev)
    if own:  # the handle on the batch, which a program keeps from call to call
        import q4_weight_quantized_block_gb300 as fak

        s["batch"] = fak.GDNBatch(s["start"], s["len"], s["slot"])
    return s


def run(s):
    return {"norm": _run_norm, "conv": _run_conv, "gdn": _run_gdn}[s["case"]["op"]](s)


def _run_norm(s):
    case = s["case"]
    if own:
        import q4_weight_quantized_block_gb300 as fak

        fak.fak_residual_norm(s["h"], s["y"], s["n"], w=s["w"], post_norm=case["post"], y_w=s["y_w"] if case["post"] else None,
                              gate=s["gate"], gate_sigmoid=case["gate"] == "sigmoid", scale=case["scale"], eps=EPS,
                              gain_offset=case["offset"])
        return [s["h"], s["n"]]
    y = s["y"].float()
    if case["post"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * (case["offset"] + s["y_w"])
    if case["gate"] != "none":
        y = y * (torch.sigmoid(s["gate"]) if case["gate"] == "sigmoid" else s["gate"])
    h = s["h"].float() + case["scale"] * y
    s["h"].copy_(h)
    s["n"].copy_(h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * (case["offset"] + s["w"]))
    return [s["h"], s["n"]]


def _rows(s, rows):
    """Sequence and index in its sequence of every new row."""
    start = s["start"].long()
    seq = torch.repeat_interleave(torch.arange(start.shape[0] - 1, device=start.device), start[1:] - start[:-1], output_size=rows)
    return seq, torch.arange(rows, device=start.device) - start[seq]


def _begins(s):
    """States of the sequences; those of sequences that begin at position 0 are empty."""
    start = s["start"].long()
    old = s["len"].long() > start[1:] - start[:-1]
    state = s["state"][s["slot"].long()]
    return torch.where(old.view(-1, *[1] * (state.dim() - 1)), state, 0.0)


def _run_conv(s):
    case = s["case"]
    nk, nv = case["nk"], case["nv"]
    if own:
        import q4_weight_quantized_block_gb300 as fak

        fak.fak_gdn_conv(s["batch"], s["x"], s["b"], s["a"], s["conv_w"], s["a_log"], s["dt_bias"], s["state"], s["q"], s["k"],
                         s["v"], s["g"], s["beta"], eps=EPS)
    else:
        rows = s["x"].shape[0]
        seq, i = _rows(s, rows)
        # every sequence's state and new rows, one after the other: three lines more for each sequence before
        line = torch.arange(rows, device=i.device) + 3 * (seq + 1)
        first = s["start"].long()[:-1] + 3 * torch.arange(s["start"].shape[0] - 1, device=i.device)
        x = torch.empty(rows + 3 * first.shape[0], s["x"].shape[1], device=i.device)
        x[line] = s["x"].float()
        x[first[:, None] + torch.arange(3, device=i.device)] = _begins(s)
        w = s["conv_w"]
        c = x[line - 3] * w[:, 0] + x[line - 2] * w[:, 1] + x[line - 1] * w[:, 2] + x[line] * w[:, 3]
        last = s["start"].long()[1:] + 3 * torch.arange(1, first.shape[0] + 1, device=i.device)
        s["state"][s["slot"].long()] = x[last[:, None] + torch.arange(-3, 0, device=i.device)]
        c = c * torch.sigmoid(c)
        q, k, v = c.split([nk * DH, nk * DH, nv * DH], 1)
        for what, t in (("q", q), ("k", k)):
            t = t.reshape(rows, nk, DH)
            s[what].copy_(t * torch.rsqrt(t.square().sum(-1, keepdim=True) + EPS))
        s["v"].copy_(v.reshape(rows, nv, DH))
        s["beta"].copy_(torch.sigmoid(s["b"].float()))
        u = s["a"].float() + s["dt_bias"]
        s["g"].copy_(-torch.exp(s["a_log"]) * (u.clamp(min=0) + torch.log1p(torch.exp(-u.abs()))))
    return [s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"]]


def _run_gdn(s):
    case = s["case"]
    nk, nv = case["nk"], case["nv"]
    if own:
        import q4_weight_quantized_block_gb300 as fak

        fak.fak_gdn_attn(s["batch"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["out"], s["max_q"], z=s["z"],
                         norm_w=s["norm_w"], eps=EPS)
        return [s["out"], s["state"]]
    # chunks of up to 64 rows, sequences padded to the longest: [chunk, sequence, head, row of the chunk, ...]; padding
    # rows write nothing (beta 0) and do not decay
    rows, seqs = s["q"].shape[0], s["start"].shape[0] - 1
    seq, i = _rows(s, rows)
    size = min(64, s["max_q"])
    chunks = -(-s["max_q"] // size)

    def padded(x, heads):
        t = torch.zeros(seqs, chunks * size, heads, *x.shape[2:], device=x.device)
        t[seq, i] = x.float()
        t = t.view(seqs, chunks, size, heads, *x.shape[2:]).transpose(2, 3).transpose(0, 1)
        return t.repeat_interleave(nv // heads, 2) if heads < nv else t

    q, k, v = padded(s["q"], nk) * DH**-0.5, padded(s["k"], nk), padded(s["v"], nv)
    beta = padded(s["beta"], nv)[..., None]
    G = padded(s["g"], nv).double().cumsum(-1)  # a row's decay since the chunk began: sums of 64 bits, whose differences matter
    low = torch.ones(size, size, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf).float())
    keep, left = torch.exp(G.float())[..., None], torch.exp((G[..., -1:] - G).float())[..., None]
    kt = k.transpose(-1, -2).contiguous()
    A = (beta * torch.matmul(k, kt) * decay).tril(-1)
    P = torch.matmul(q, kt) * decay
    eye = torch.eye(size, device=q.device)
    S, outs = _begins(s), []
    for c in range(chunks):
        r = beta[c] * (v[c] - keep[c] * torch.matmul(k[c], S))
        u = torch.linalg.solve_triangular(eye + A[c], r, upper=False, unitriangular=True)
        outs.append(keep[c] * torch.matmul(q[c], S) + torch.matmul(P[c], u))
        S = keep[c][..., -1:, :] * S + torch.matmul(kt[c], left[c] * u)
    s["state"][s["slot"].long()] = S
    o = torch.stack(outs, 1).transpose(2, 3).reshape(seqs, chunks * size, nv, DH)[seq, i]
    if case["gate"]:
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * s["norm_w"] * (s["z"] * torch.sigmoid(s["z"]))
    s["out"].copy_(o)
    return [s["out"], s["state"]]


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "norm":
        n = case["rows"] * case["d"]
        gate = {"none": 0, "rows": 4 * n, "columns": 4 * case["d"], "sigmoid": 4 * case["rows"]}[case["gate"]]
        return {"bytes": n * (2 * size[case["h"]] + size[case["y"]] + size[case["n"]]) + gate + 8 * case["d"],
                "flops": n * (6 + 4 * case["post"] + (case["gate"] != "none"))}
    nk, nv, seqs = case["nk"], case["nv"], case["seqs"]
    new, past = _lengths(case)
    rows, old, chans = sum(new), sum(p > 0 for p in past), (2 * nk + nv) * DH
    if case["op"] == "conv":
        return {"bytes": rows * (chans * (size[case["kind"]] + 2) + 2 * nv * (size[case["kind"]] + 4)) + (seqs + old) * 3 * chans * 4 + chans * 16,
                "flops": rows * chans * 12}
    a_row = 2 * nk * DH * 2 + nv * (DH * (2 + size[case["out"]] + (4 if case["gate"] else 0)) + 8)
    # by the recurrence a row and head take three products with the state; nothing can take fewer
    return {"bytes": rows * a_row + (seqs + old) * nv * DH * DH * 4, "flops": rows * nv * DH * DH * 6}


# ------------------------------------------------------------------ in 64 bits, from the definitions, row by row
def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64

    def rms(x):
        return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)

    def sigma(x):
        return 1 / (1 + torch.exp(-x))

    if case["op"] == "norm":
        y, h = s["y"].to(f), s["h"].to(f)
        if case["post"]:
            y = rms(y) * (s["y_w"].to(f) + case["offset"])
        if case["gate"] != "none":
            gate = s["gate"].to(f)
            y = y * (sigma(gate) if case["gate"] == "sigmoid" else gate)
        h = h + y * case["scale"]
        return [h, rms(h) * (s["w"].to(f) + case["offset"])]
    nk, nv = case["nk"], case["nv"]
    new, past = _lengths(case)
    slots, at = s["slot"].tolist(), [sum(new[:i]) for i in range(case["seqs"])]
    state = s["state"].to(f)
    if case["op"] == "conv":
        c = torch.empty(sum(new), (2 * nk + nv) * DH, dtype=f, device="cuda")
        for r, n, p, slot in zip(at, new, past, slots):
            before = state[slot] if p else torch.zeros_like(state[slot])
            x = torch.cat([before, s["x"][r : r + n].to(f)])
            y = sum(s["conv_w"][:, j].to(f) * x[j : j + n] for j in range(4))
            c[r : r + n] = y * sigma(y)
            state[slot] = x[-3:]
        c = c.view(len(c), -1, DH)
        unit = c / torch.sqrt((c * c).sum(-1, keepdim=True) + EPS)
        u = s["a"].to(f) + s["dt_bias"].to(f)
        g = -torch.exp(s["a_log"].to(f)) * torch.log1p(torch.exp(u))
        return [unit[:, :nk], unit[:, nk : 2 * nk], c[:, 2 * nk :], g, sigma(s["b"].to(f)), state]
    # all sequences that still have rows step together, the longest first
    order = sorted(range(case["seqs"]), key=lambda i: -new[i])
    S = torch.stack([state[slots[i]] if past[i] else torch.zeros_like(state[0]) for i in order])
    o = torch.empty(sum(new), nv, DH, dtype=f, device="cuda")
    first = torch.tensor([at[i] for i in order], device="cuda")
    q, k = (s[what].to(f).repeat_interleave(nv // nk, 1) for what in ("q", "k"))
    v, alpha, beta = s["v"].to(f), torch.exp(s["g"].to(f)), s["beta"].to(f)
    for t in range(max(new)):
        b = sum(n > t for n in new)
        r = first[:b] + t
        S[:b] *= alpha[r][..., None, None]
        kt = k[r][..., None, :]
        u = beta[r][..., None, None] * (v[r][..., None, :] - torch.matmul(kt, S[:b]))
        S[:b] += kt.transpose(-1, -2) * u
        o[r] = torch.matmul(q[r][..., None, :], S[:b])[..., 0, :]
    o /= math.sqrt(DH)
    for j, i in enumerate(order):
        state[slots[i]] = S[j]
    if case["gate"]:
        z = s["z"].to(f)
        o = rms(o) * s["norm_w"].to(f) * z * sigma(z)
    return [o, state]
