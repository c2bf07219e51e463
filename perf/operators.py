"""What is measured of the paged key / value cache and the attention over it.

Four operators, each as a serving program calls it between the Q4_K projections of a full-attention layer:
  write   fak_kv_append: RMSNorm and rotary embedding of the new rows, keys and values put into the cache
  read    fak_kv_read: positions of the cache back as rows
  attn    fak_paged_attn: new rows (single tokens, chunks, whole prompts) over the cache
  window  fak_paged_attn with a sliding window and a few first tokens that stay visible

A case holds the head layout, the cache's type and page, the number of sequences, the most new rows a
sequence has and the most positions that stand before them; with "ragged" the sequences differ in both.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 1e7
TOP = {"e4m3": 448.0, "i8": 127.0}


def _case(name, op, nq, nkv, dh, kind, page, seqs, new, ctx, ragged=False, rot=0, gate=False, window=0, sinks=0):
    return dict(name=name, op=op, nq=nq, nkv=nkv, dh=dh, kind=kind, page=page, seqs=seqs, new=new, ctx=ctx,
                ragged=ragged, rot=rot, gate=gate, window=window, sinks=sinks)


def listed():
    return [
        # one decoded token of one sequence: 24 query and 4 key heads of 256, qk-norm, rotary on 64 dims
        _case("write 1 token", "write", 24, 4, 256, "bf16", 64, 1, 1, 1000, rot=64),
        # chunks of eight prompts, quantised as they are written
        _case("write 8 chunks e4m3", "write", 24, 4, 256, "e4m3", 64, 8, 1024, 7000, ragged=True, rot=64),
        # a short prefix taken out of the cache
        _case("read 1000 e4m3", "read", 24, 4, 256, "e4m3", 64, 1, 1000, 0),
        # sixteen whole sequences taken out, to be moved
        _case("read 16x8192 i8", "read", 24, 4, 256, "i8", 32, 16, 8192, 0, ragged=True),
        # a decode step: one sequence with a short past, with the output gate
        _case("decode 1x1000", "attn", 24, 4, 256, "bf16", 64, 1, 1, 1000, gate=True),
        # a decode step of a full batch with pasts of all lengths
        _case("decode 64x8191 e4m3", "attn", 24, 4, 256, "e4m3", 64, 64, 1, 8191, ragged=True, gate=True),
        # a decode step of one sequence with a very long past, heads of 128
        _case("decode 1x131071 i8", "attn", 32, 8, 128, "i8", 64, 1, 1, 131071),
        # a chunk of a long prompt
        _case("chunk 512 over 8192", "attn", 24, 4, 256, "bf16", 64, 1, 512, 7680, gate=True),
        # chunks of several prompts in one call, eight-bit cache, heads of 128
        _case("chunks 8x1024 e4m3", "attn", 32, 8, 128, "e4m3", 16, 8, 1024, 4001, ragged=True),
        # a whole prompt at once
        _case("prompt 8192", "attn", 24, 4, 256, "bf16", 64, 1, 8192, 0, gate=True),
        # decode with a window: the past is long, what is seen of it is not
        _case("window decode 32x8191", "window", 24, 4, 256, "bf16", 64, 32, 1, 8191, ragged=True, window=1024, sinks=4),
        # a long chunk with a window, eight-bit cache
        _case("window chunk 2048 i8", "window", 32, 8, 128, "i8", 32, 1, 2048, 14000, window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn", "window", "window"])
    dh = rng.choice([64, 128, 256, 256])
    nq, nkv = rng.choice([(24, 4), (24, 4), (32, 8), (16, 16), (16, 2), (12, 3), (10, 1), (3, 1)])
    kind = rng.choice(["bf16", "e4m3", "i8"])
    page = rng.choice([16, 32, 64, 128])
    single = op in ("attn", "window") and rng.random() < 0.5
    seqs = _log(rng, 1, 64)
    new = 1 if single else _log(rng, 1, 8192)
    ctx = 0 if op == "read" else _log(rng, 1, 131072 if single else 16384)
    case = dict(op=op, nq=nq, nkv=nkv, dh=dh, kind=kind, page=page, seqs=seqs, new=new, ctx=ctx,
                ragged=rng.random() < 0.7, rot=0, gate=op in ("attn", "window") and rng.random() < 0.5, window=0, sinks=0)
    if op == "write" and kind != "i8":
        case["rot"] = rng.choice([0, 32, 64])
    if op == "window":
        case["window"], case["sinks"] = _log(rng, 1, 4096), rng.choice([0, 1, 4, 17])
    # not above the largest listed cases: 8192 x 8192 positions of 24 heads of 256, or 64 x 8192 cached ones
    while True:
        s, n, c = case["seqs"], case["new"], case["ctx"]
        if s * (n + c) <= 1 << 19 and (op in ("write", "read") or n * s * (n + c) * nq * dh <= 24 * 256 << 26) and s * n <= 1 << 16:
            return case
        if s > 1 and s >= n:
            case["seqs"] = s - s // 2
        elif n > c and n > 1:
            case["new"] = n - n // 2
        else:
            case["ctx"] = c - c // 2


def _lengths(case):
    """New rows and positions in all of each sequence."""
    new, past = [], []
    for i in range(case["seqs"]):
        a, b = ((5 * i + 8) % 9, (5 * i + 6) % 7) if case["ragged"] and case["seqs"] > 1 else (8, 6)
        new.append(1 + (case["new"] - 1) * a // 8)
        past.append(case["ctx"] * (1 + b) // 7)
    return new, [n + c for n, c in zip(new, past)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    nq, nkv, dh, page = case["nq"], case["nkv"], case["dh"], case["page"]
    new, total = _lengths(case)
    rows, seqs = sum(new), case["seqs"]
    per = [-(-t // page) for t in total]
    n_pages, most = sum(per) + 3, max(per)

    def normal(*shape, like=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=like)

    # the sequences' pages stand in the cache in no order
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([sum(per[:i]) for i in range(seqs)], device=dev)
    at = first[:, None] + torch.arange(most, device=dev)
    have = torch.arange(most, device=dev) < torch.tensor(per, device=dev)[:, None]
    table = torch.where(have, perm[torch.where(have, at, 0)], 0).to(torch.int32).contiguous()
    start = torch.tensor([sum(new[:i]) for i in range(seqs + 1)], dtype=torch.int32, device=dev)
    s = dict(case=case, table=table, start=start, kv_len=torch.tensor(total, dtype=torch.int32, device=dev),
             max_q=max(new), max_kv=max(total))

    # what the cache holds: normed keys (a few channels larger than the rest) and values of the projections' size
    kv = []
    for what in ("k", "v"):
        x = normal(n_pages, nkv, page, dh, like=torch.bfloat16)
        if what == "k":
            x[..., :: dh // 4] *= 3
        if case["kind"] == "bf16":
            kv.append((x, None))
            continue
        x = x.float()
        scale = x.abs().amax(-1) / TOP[case["kind"]]
        x /= scale[..., None]
        code = x.to(torch.float8_e4m3fn).view(torch.uint8) if case["kind"] == "e4m3" else x.round().to(torch.int8)
        kv.append((code, scale))
        del x
    (s["k"], s["k_scale"]), (s["v"], s["v_scale"]) = kv

    if case["op"] == "write":
        # the projections' rows as the input GEMM leaves them: query | gate per head, then keys, then values
        t = normal(rows, (2 * nq + 2 * nkv) * dh)
        s["q_in"] = t[:, : 2 * nq * dh].view(rows, nq, 2 * dh)[..., :dh]
        s["k_in"] = t[:, 2 * nq * dh : (2 * nq + nkv) * dh].view(rows, nkv, dh)
        s["v_in"] = t[:, (2 * nq + nkv) * dh :].view(rows, nkv, dh)
        s["q_out"] = torch.empty(rows, nq, dh, dtype=torch.bfloat16, device=dev)
        if case["rot"]:
            s["qw"], s["kw"] = 1 + 0.1 * normal(dh), 1 + 0.1 * normal(dh)
            i = torch.arange(case["rot"] // 2, dtype=torch.float64)
            # the rotary frequencies in turns per position, as 64-bit fractions of a turn
            f = torch.floor(THETA ** (-2 * i / case["rot"]) / (2 * math.pi) * 2.0**62 + 0.5).to(torch.int64) * 4
            s["rope"] = f.to(dev)
    elif case["op"] == "read":
        s["k_out"] = torch.empty(rows, nkv, dh, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        s["q"] = normal(rows, nq, dh, like=torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["gate"] = normal(rows, 2 * nq, dh)[:, 1::2] if case["gate"] else None
    if own:  # the handles on the cache and on the batch, and the workspace, which a program keeps from call to call
        import q4_weight_quantized_block_gb300 as fak

        kind = {"bf16": fak.FAK_KV_BF16, "e4m3": fak.FAK_KV_E4M3, "i8": fak.FAK_KV_I8}[case["kind"]]
        s["cache"] = fak.KVCache(kind, s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = fak.KVBatch(s["table"], s["start"], s["kv_len"])
        if case["op"] in ("attn", "window"):
            n = fak.fak_paged_attn_workspace_bytes(s["cache"], s["batch"], nq, rows, s["max_q"], s["max_kv"],
                                                   window=case["window"], sinks=case["sinks"])
            s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    return s


def run(s):
    return {"write": _write, "read": _read, "attn": _attn, "window": _attn}[s["case"]["op"]](s)


def _rows(s):
    """Sequence and position of every new row."""
    start, n = s["start"].long(), s["start"].shape[0] - 1
    new = start[1:] - start[:-1]
    seq = torch.repeat_interleave(torch.arange(n, device=start.device), new, output_size=s["rows"])
    return seq, torch.arange(s["rows"], device=start.device) - start[seq] + (s["kv_len"].long() - new)[seq]


def _places(s, seq, pos):
    page = s["case"]["page"]
    return s["table"].long()[seq, pos // page], pos % page


def _normed(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _turned(x, pos, rot):
    i = torch.arange(rot // 2, device=x.device, dtype=torch.float64)
    angle = pos[:, None].double() * THETA ** (-2 * i / rot)
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., rot:]], -1)


def _write(s):
    case = s["case"]
    if own:
        import q4_weight_quantized_block_gb300 as fak

        fak.fak_kv_append(s["cache"], s["batch"], s["k_in"], s["v_in"], q=s["q_in"], q_out=s["q_out"], q_norm_w=s.get("qw"),
                          k_norm_w=s.get("kw"), eps=EPS, rope=s.get("rope"), rot=case["rot"])
    else:
        s["rows"] = s["k_in"].shape[0]
        seq, pos = _rows(s)
        q, k, v = s["q_in"], s["k_in"], s["v_in"]
        if case["rot"]:
            q, k = _turned(_normed(q, s["qw"]), pos, case["rot"]), _turned(_normed(k, s["kw"]), pos, case["rot"])
        s["q_out"].copy_(q)
        pages, slot = _places(s, seq, pos)
        _put(s, "k", pages, slot, k)
        _put(s, "v", pages, slot, v)
    out = [s["q_out"], s["k"], s["v"]]
    if case["kind"] == "e4m3":
        out[1:] = [x.view(torch.float8_e4m3fn) for x in out[1:]]
    return out + [x for x in (s["k_scale"], s["v_scale"]) if x is not None]


def _put(s, what, pages, slot, x):
    kind = s["case"]["kind"]
    if kind == "bf16":
        s[what][pages, :, slot] = x.to(torch.bfloat16)
        return
    most = x.abs().amax(-1)
    x = x * (TOP[kind] / most)[..., None]
    s[what][pages, :, slot] = x.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "e4m3" else x.round().to(torch.int8)
    s[what + "_scale"][pages, :, slot] = most / TOP[kind]


def _values(s, what, pages, slot):
    """The cache's vectors at these places, in 32 bits: [..., n_kv, dh]."""
    x = s[what][pages, :, slot]
    if s["case"]["kind"] == "e4m3":
        x = x.view(torch.float8_e4m3fn)
    x = x.float()
    return x if s[what + "_scale"] is None else x * s[what + "_scale"][pages, :, slot][..., None]


def _read(s):
    if own:
        import q4_weight_quantized_block_gb300 as fak

        fak.fak_kv_read(s["cache"], s["batch"], s["k_out"], s["v_out"])
    else:
        s["rows"] = s["k_out"].shape[0]
        pages, slot = _places(s, *_rows(s))
        s["k_out"].copy_(_values(s, "k", pages, slot))
        s["v_out"].copy_(_values(s, "v", pages, slot))
    return [s["k_out"], s["v_out"]]


def _attn(s):
    case, q = s["case"], s["q"]
    nq, nkv, dh = case["nq"], case["nkv"], case["dh"]
    if own:
        import q4_weight_quantized_block_gb300 as fak

        fak.fak_paged_attn(s["cache"], s["batch"], q, s["out"], s["max_q"], s["max_kv"], scale=dh**-0.5, window=case["window"],
                           sinks=case["sinks"], gate=s["gate"], workspace=s["ws"])
        return s["out"]
    # padded to the longest: [sequence, key head, query head of the group, new row, position]
    s["rows"] = q.shape[0]
    seq, pos = _rows(s)
    row = torch.arange(s["rows"], device=q.device) - s["start"].long()[seq]
    b = s["start"].shape[0] - 1
    qp = torch.zeros(b, s["max_q"], nq, dh, device=q.device)
    qp[seq, row] = q.float()
    qpos = torch.full((b, s["max_q"]), -1, device=q.device)
    qpos[seq, row] = pos
    j = torch.arange(s["max_kv"], device=q.device)
    there = j < s["kv_len"].long()[:, None]
    pages, slot = _places(s, torch.arange(b, device=q.device)[:, None], torch.where(there, j, 0))
    k, v = (_values(s, what, pages, slot).permute(0, 2, 3, 1) for what in ("k", "v"))  # [b, n_kv, dh, position]
    sees = j <= qpos[..., None]
    if case["window"]:
        sees &= (j > qpos[..., None] - case["window"]) | (j < case["sinks"])
    qp = qp.view(b, -1, nkv, nq // nkv, dh).permute(0, 2, 3, 1, 4).reshape(b, nkv, -1, dh)
    w = torch.matmul(qp * dh**-0.5, k).view(b, nkv, nq // nkv, -1, s["max_kv"])
    w.masked_fill_(~sees[:, None, None], -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(b, nkv, -1, s["max_kv"]), v.transpose(2, 3)).view(b, nkv, nq // nkv, -1, dh)
    o = torch.where(total > 0, o / total, 0).permute(0, 3, 1, 2, 4).reshape(b, -1, nq, dh)[seq, row]
    if case["gate"]:
        o = o * torch.sigmoid(s["gate"])
    s["out"].copy_(o)
    return s["out"]


def _seen(case, first, count):
    """Pairs (row, position seen) of `count` rows at positions first, first + 1, ..., and positions that some row sees."""
    last = first + count - 1
    if not case["window"]:
        return (first + 1 + last + 1) * count // 2, last + 1
    w, k = case["window"], case["sinks"]
    pairs = sum(min(p + 1, w) + min(k, max(0, p + 1 - w)) for p in range(first, last + 1))
    low = max(0, first + 1 - w)
    return pairs, last + 1 - low + min(k, low)


def work(case):
    new, total = _lengths(case)
    nq, nkv, dh = case["nq"], case["nkv"], case["dh"]
    rows = sum(new)
    vector = dh * 2 if case["kind"] == "bf16" else dh + 4  # one cached vector
    if case["op"] == "write":
        return {"bytes": rows * ((nq + 2 * nkv) * dh * 4 + nq * dh * 2 + 2 * nkv * vector), "flops": 8 * rows * (nq + 2 * nkv) * dh}
    if case["op"] == "read":
        return {"bytes": rows * 2 * nkv * (vector + 2 * dh), "flops": 2 * rows * nkv * dh}
    seen = [_seen(case, t - n, n) for n, t in zip(new, total)]
    return {"bytes": sum(k for _, k in seen) * 2 * nkv * vector + rows * nq * dh * (8 if case["gate"] else 4),
            "flops": sum(p for p, _ in seen) * nq * dh * 4}


# ------------------------------------------------------------------ in 64 bits, sequence by sequence
def exact(case, seed):
    s = prepare(case, seed)
    new, total = _lengths(case)
    lines = [s["table"][i, torch.arange(total[i], device="cuda") // case["page"]].long() * case["page"]
             + torch.arange(total[i], device="cuda") % case["page"] for i in range(case["seqs"])]

    def flat(t):  # [n_pages, n_kv, page, ...] -> one line per place: [n_pages * page, n_kv, ...]
        return t.transpose(1, 2).flatten(0, 1)

    if case["op"] == "write":
        return _exact_write(case, s, new, total, lines)
    k, v = flat(s["k"]), flat(s["v"])
    ks, vs = (None, None) if s["k_scale"] is None else (flat(s["k_scale"]), flat(s["v_scale"]))

    def held(codes, scales, line):
        x = codes[line]
        x = (x.view(torch.float8_e4m3fn) if case["kind"] == "e4m3" else x).to(torch.float64)
        return x if scales is None else x * scales[line].double()[..., None]

    if case["op"] == "read":
        return [torch.cat([held(c, sc, line[-n:]) for line, n in zip(lines, new)]) for c, sc in ((k, ks), (v, vs))]
    group, outs, row = case["nq"] // case["nkv"], [], 0
    for n, t, line in zip(new, total, lines):
        p = torch.arange(t - n, t, device="cuda")[:, None]
        j = torch.arange(t, device="cuda")[None]
        dark = j > p
        if case["window"]:
            dark = dark | ((p - j >= case["window"]) & (j >= case["sinks"]))
        kk, vv = held(k, ks, line), held(v, vs, line)
        heads = []
        for h in range(case["nq"]):
            logit = s["q"][row : row + n, h].double() @ kk[:, h // group].T / math.sqrt(case["dh"])
            heads.append(torch.softmax(logit.masked_fill(dark, -math.inf), -1) @ vv[:, h // group])
        o = torch.stack(heads, 1)
        if case["gate"]:
            o = o / (1 + torch.exp(-s["gate"][row : row + n].double()))
        outs.append(o)
        row += n
    return torch.cat(outs)


def _exact_write(case, s, new, total, lines):
    pos = torch.cat([torch.arange(t - n, t, device="cuda") for n, t in zip(new, total)]).double()
    line = torch.cat([x[-n:] for x, n in zip(lines, new)])
    x = {"q": s["q_in"].double(), "k": s["k_in"].double(), "v": s["v_in"].double()}
    if case["rot"]:
        half = case["rot"] // 2
        turn = torch.exp(torch.arange(half, device="cuda").double() * (-2 * math.log(THETA) / case["rot"]))
        z = torch.polar(torch.ones(len(pos), half, device="cuda", dtype=torch.float64), pos[:, None] * turn)[:, None]
        for what, w in (("q", s["qw"]), ("k", s["kw"])):
            y = x[what] / torch.sqrt((x[what] ** 2).sum(-1, keepdim=True) / case["dh"] + EPS) * w.double()
            y[..., : 2 * half] = torch.view_as_real(torch.complex(y[..., :half], y[..., half : 2 * half]) * z).transpose(-1, -2).flatten(-2)
            x[what] = y
    out, scales = [x["q"]], []
    for what in ("k", "v"):
        held = s[what].view(torch.float8_e4m3fn) if case["kind"] == "e4m3" else s[what]
        held = held.to(torch.float64).transpose(1, 2).contiguous()  # [n_pages, page, n_kv, dh]
        y = x[what]
        if case["kind"] != "bf16":
            scale = s[what + "_scale"].double().transpose(1, 2).contiguous()
            scale.view(-1, case["nkv"])[line] = y.abs().amax(-1) / TOP[case["kind"]]
            y = y / (y.abs().amax(-1, keepdim=True) / TOP[case["kind"]])
            y = y.to(torch.float32).to(torch.float8_e4m3fn).double() if case["kind"] == "e4m3" else y
            scales.append(scale.transpose(1, 2).contiguous())
        held.view(-1, case["nkv"], case["dh"])[line] = y
        out.append(None if case["kind"] == "i8" else held.transpose(1, 2).contiguous())
    return out + scales
