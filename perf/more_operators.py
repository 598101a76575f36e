"""Cases that measure the router's balance loss and the operators on
microscaled 4-bit floats: their quantization, and the experts' products with
4-bit weights.

``run`` computes a case in plain torch operations, or, where ``own`` is set,
through the package's entry points.  Every buffer that a call writes is the
state's own, as in a serving or training loop that reuses its buffers: rows
that a call leaves untouched keep what the state holds there.

A 4-bit payload is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two
to a byte, the lower channel in the lower half; a scale byte b per 32 channels
means 2^(b - 127).  Rows of 8 bits are e4m3 with the same scales.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
G = 32  # channels of a scale


# ------------------------------------------------------------------- cases

def listed():
    return [
        # balance loss of one small expert-parallel rank's micro-batch, and
        # its gradient: latency alone
        dict(name="balance few tokens", op="balance", T=48, E=16, K=2, S=1,
             scoring="softmax", dtype="f32", z=True, pad=False, dead=0),
        # a training step's tokens through a sigmoid router, balanced over
        # the whole batch
        dict(name="balance batch", op="balance", T=8192, E=256, K=8, S=1,
             scoring="sigmoid", dtype="f32", z=False, pad=False, dead=0),
        # a long packed batch balanced sequence by sequence, padding behind
        # each, two experts out of service
        dict(name="balance sequences", op="balance", T=50000, E=160, K=6,
             S=23, scoring="softmax", dtype="bf16", z=True, pad=True, dead=2),
        # an odd matrix of master weights to 4 bits
        dict(name="quant odd weights", op="quant", rows=1431, H=1376,
             dtype="f32", rule="ocp_floor", wide="e4m3"),
        # the gate and up projections of four experts to 4 bits and back to
        # bf16, as quantization-aware training does
        dict(name="quant weights", op="quant", rows=16384, H=7168,
             dtype="bf16", rule="no_clip", wide="bf16"),
        # a decode batch's rows to the experts in 4 bits; the receiver's
        # product takes 8
        dict(name="dispatch decode", op="dispatch", T=128, K=8, E=32, H=7168,
             rule="no_clip"),
        # the same for a prefill chunk
        dict(name="dispatch prefill", op="dispatch", T=4096, K=8, E=64,
             H=7168, rule="no_clip"),
        # one token through eight of 32 experts: gate and up, gated and
        # quantized, and down
        dict(name="experts one token", op="experts", T=1, K=8, E=32, I=2048,
             H=7168, fmt="mxfp4", mid="mxfp4", bias=False, residual=False,
             cap=128),
        # a decode batch of 8-bit rows on a masked slab
        dict(name="experts decode 8-bit rows", op="experts", T=128, K=2, E=32,
             I=2048, H=7168, fmt="e8m0_g32", mid="e8m0_g32", bias=False,
             residual=False, cap=128),
        # a short prompt over small experts of odd sizes, with biases
        dict(name="experts odd", op="experts", T=777, K=6, E=24, I=736,
             H=1376, fmt="mxfp4", mid="e8m0_g32", bias=True, residual=False,
             cap=0),
        # a prefill chunk of all ranks' tokens in 4 bits
        dict(name="experts prefill", op="experts", T=8192, K=8, E=32, I=2048,
             H=7168, fmt="mxfp4", mid="mxfp4", bias=False, residual=False,
             cap=0),
        # half of it in 8 bits, with the shared branch added in the epilogue
        dict(name="experts prefill 8-bit rows", op="experts", T=4096, K=8,
             E=32, I=2048, H=7168, fmt="e8m0_g32", mid="e8m0_g32", bias=True,
             residual=True, cap=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance", "quant", "dispatch", "experts",
                     "experts", "experts"])
    if op == "balance":
        E = _log(rng, 4, 512)
        T = _log(rng, 1, 32768)
        return dict(op=op, T=T, E=E, K=min(rng.randint(1, 10), E),
                    S=min(T, _log(rng, 1, 64)) if rng.random() < 0.5 else 1,
                    scoring=rng.choice(["softmax", "sigmoid"]),
                    dtype=rng.choice(["bf16", "f32"]), z=rng.random() < 0.5,
                    pad=rng.random() < 0.5, dead=rng.randint(0, E // 4))
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 16384), H=G * _log(rng, 1, 224),
                    dtype=rng.choice(["bf16", "f32"]),
                    rule=rng.choice(["no_clip", "ocp_floor"]),
                    wide=rng.choice(["bf16", "e4m3"]))
    if op == "dispatch":
        E = _log(rng, 2, 256)
        return dict(op=op, T=_log(rng, 1, 4096), K=rng.randint(1, min(E, 8)),
                    E=E, H=G * _log(rng, 1, 224),
                    rule=rng.choice(["no_clip", "ocp_floor"]))
    E = _log(rng, 1, 32)
    T = _log(rng, 1, 8192)
    return dict(op=op, T=T, K=rng.randint(1, min(E, 8)), E=E,
                I=G * _log(rng, 2, 64), H=G * _log(rng, 4, 224),
                fmt=rng.choice(["mxfp4", "e8m0_g32"]),
                mid=rng.choice(["mxfp4", "e8m0_g32"]),
                bias=rng.random() < 0.3, residual=rng.random() < 0.3,
                cap=128 * math.ceil(T / 128) if rng.random() < 0.3 and
                T * E <= 65536 else 0)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _routing(g, T, K, E):
    """K distinct experts of E per token, some experts better liked."""
    like = 0.5 * _randn(g, E) + _randn(g, T, E)
    return like.topk(K, dim=1).indices


def _layout(ids, E, cap, block=128):
    """The layout's tensors for ids [T, K]: regions in whole blocks of rows,
    or a slab of `cap` rows an expert."""
    flat = ids.reshape(-1)
    counts = torch.bincount(flat, minlength=E)
    size = torch.full_like(counts, cap) if cap else \
        (counts + block - 1) // block * block
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = size.cumsum(0)
    order = torch.argsort(flat, stable=True)
    start = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    start[1:] = counts.cumsum(0)
    e = flat[order]
    dst = torch.empty_like(flat)
    at = torch.arange(flat.numel(), device=DEV)
    dst[order] = offsets[e] + at - start[e]
    A = flat.numel()
    n = min(A, E)
    rows = E * cap if cap else block * (n + (A - n) // block)
    return dict(counts=counts.int(), offsets=offsets.int(), rows=rows,
                src2dst=dst.reshape(ids.shape).int())


# e2m1 magnitudes, and where one rounds to the next: halfway, and halfway
# itself to the even code
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
HALF = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _exponent(amax, fmt, rule):
    """Exponent of a group's power-of-two scale: the smallest at which its
    largest value needs no clipping, or the value's own less the type's."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1
    top, border = (3, 0.75) if fmt == "mxfp4" else (9, 0.875)
    e = e - top if rule == "ocp_floor" else torch.where(m > border, e - top + 1,
                                                        e - top)
    return torch.where(amax == 0, torch.full_like(e, -127),
                       e.clamp(-127, 127))


def _scaled(x, fmt, rule):
    """Values over their group's scale, and the scale bytes."""
    v = x.reshape(x.shape[0], -1, G)
    e = _exponent(v.abs().amax(-1), fmt, rule)
    payload = torch.ldexp(v, -e.unsqueeze(-1).to(x.dtype)).reshape(x.shape)
    return payload, (e + 127).to(torch.uint8)


def _code(v):
    """e2m1 codes of payload values, to the nearest, ties to even."""
    a = v.abs()
    c = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    for i, h in enumerate(HALF):
        c += (a >= h) if i % 2 else (a > h)
    return c + 8 * torch.signbit(v).to(torch.uint8)


def _pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _quant(x, fmt, rule="no_clip"):
    """Bytes of the payload and scale bytes."""
    p, s = _scaled(x, fmt, rule)
    if fmt == "mxfp4":
        return _pack(_code(p)), s
    return p.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def _prepare_balance(c, g):
    T, E, K, S = c["T"], c["E"], c["K"], c["S"]
    t = DTYPES[c["dtype"]]
    # a trained router's: some experts better liked
    logits = (0.7 * _randn(g, E) + 1.5 * _randn(g, T, E)).to(t)
    dead = torch.randperm(E, generator=g, device=DEV)[:min(c["dead"], E - K)]
    logits[:, dead] = -math.inf
    s = dict(case=c, logits=logits, ids=logits.float().topk(K).indices.int())
    s["offsets"] = s["lens"] = None
    if S > 1:
        # ragged sequences that share the T tokens
        cuts = torch.randperm(T - 1, generator=g, device=DEV)[:S - 1] + 1
        s["offsets"] = torch.cat([cuts.new_zeros(1), cuts.sort().values,
                                  cuts.new_full((1,), T)]).int()
        if c["pad"]:
            full = s["offsets"][1:] - s["offsets"][:-1]
            keep = 0.8 + 0.2 * torch.rand(S, generator=g, device=DEV)
            s["lens"] = (full * keep).ceil().int()
    s["grad"] = torch.full((S,), 0.01 / S, device=DEV)
    s["grad_z"] = torch.full((S,), 0.001 / S, device=DEV) if c["z"] else None
    s["out"] = dict(loss=torch.zeros(S, device=DEV),
                    probs=torch.zeros((S, E), device=DEV),
                    counts=torch.zeros((S, E), dtype=torch.int32, device=DEV))
    if c["z"]:
        s["out"]["z_loss"] = torch.zeros(S, device=DEV)
    # the router's own gradient, which this one is added to
    s["add"] = (0.01 / (T * E) * _randn(g, T, E)).to(t)
    s["grad_logits"] = torch.zeros_like(logits)
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "balance":
        return _prepare_balance(c, g)
    H = c["H"]
    if c["op"] == "quant":
        rows, t = c["rows"], DTYPES[c["dtype"]]
        # weights: rows of their own size
        x = 0.02 * _randn(g, rows, H) * (0.5 * _randn(g, rows, 1)).exp()
        s = dict(case=c, x=x.to(t),
                 q=torch.zeros((rows, H // 2), dtype=torch.uint8, device=DEV),
                 scales=torch.zeros((rows, H // G), dtype=torch.uint8,
                                    device=DEV))
        s["out"] = torch.zeros((rows, H), device=DEV, dtype=torch.bfloat16
                               if c["wide"] == "bf16" else torch.uint8)
        return s
    lay = _layout(_routing(g, c["T"], c["K"], c["E"]), c["E"],
                  c.get("cap", 0))
    rows = lay["rows"]
    x = _randn(g, c["T"], H)
    # a few channels are a hundred times the others, as activations are
    x[:, torch.randperm(H, generator=g, device=DEV)[:max(1, H // 1000)]] *= 100
    if c["op"] == "dispatch":
        return dict(case=c, x=x.to(torch.bfloat16), src2dst=lay["src2dst"],
                    q=torch.zeros((rows, H // 2), dtype=torch.uint8,
                                  device=DEV),
                    scales=torch.zeros((rows, H // G), dtype=torch.uint8,
                                       device=DEV),
                    out=torch.zeros((rows, H), dtype=torch.uint8, device=DEV))
    E, I = c["E"], c["I"]
    q, scales = _quant(_randn(g, rows, H), c["fmt"])

    def weights(n, k):
        # expert by expert; one over sqrt(k): products of unit rows come out
        # near one
        out = torch.empty((E, n, k // 2), dtype=torch.uint8, device=DEV)
        # rows of scales start on 16 bytes, as the quantizer leaves them
        ld = -(-(k // G) // 16) * 16
        sc = torch.full((E, n, ld), 127, dtype=torch.uint8, device=DEV)
        for e in range(E):
            out[e], sc[e, :, :k // G] = _quant(_randn(g, n, k) / math.sqrt(k),
                                               "mxfp4")
        return out, sc[:, :, :k // G]

    w1, s1 = weights(2 * I, H)
    w2, s2 = weights(H, I)
    pay = I // 2 if c["mid"] == "mxfp4" else I
    return dict(case=c, q=q, scales=scales, w1=w1, s1=s1, w2=w2, s2=s2,
                offsets=lay["offsets"], counts=lay["counts"],
                most=int(lay["counts"].max()),
                b1=0.5 * _randn(g, E, 2 * I) if c["bias"] else None,
                b2=_randn(g, E, H) if c["bias"] else None,
                residual=_randn(g, rows, H).to(torch.bfloat16)
                if c["residual"] else None,
                mid=torch.zeros((rows, pay), dtype=torch.uint8, device=DEV),
                mid_scales=torch.zeros((rows, I // G), dtype=torch.uint8,
                                       device=DEV),
                out=torch.zeros((rows, H), dtype=torch.bfloat16, device=DEV),
                # rows an expert holds on average: what a scheduler knows
                expected=-(-c["T"] * c["K"] // E))


# ------------------------------------------------------------- plain forms

def _sequence_of(s):
    """Sequence of every token, S where it belongs to none, and the number
    of tokens of each."""
    c, S = s["case"], s["case"]["S"]
    t = torch.arange(c["T"], device=DEV)
    if s["offsets"] is None:
        return torch.zeros_like(t), t.new_full((1,), c["T"])
    off = s["offsets"].long()
    q = torch.searchsorted(off, t, right=True) - 1
    n = off[1:] - off[:-1] if s["lens"] is None else s["lens"].long()
    at = q.clamp(0, S - 1)
    live = (q >= 0) & (q < S) & (t - off[at] < n[at])
    return torch.where(live, q, S), n


def _balance(s):
    c = s["case"]
    T, E, S = c["T"], c["E"], c["S"]
    seq, n = _sequence_of(s)
    l = s["logits"].float()
    soft = torch.softmax(l, 1)
    if c["scoring"] == "softmax":
        p, back = soft, None
    else:
        sig = torch.sigmoid(l)
        p, back = sig / sig.sum(1, keepdim=True), torch.sigmoid(-l)
    # sums over a sequence's tokens in 64 bits: products with which tokens
    # are its own
    of = (seq == torch.arange(S, device=DEV).unsqueeze(1)).double()
    P = (of @ p.double()) / n.unsqueeze(1)
    taken = torch.zeros((T, E), dtype=torch.float64, device=DEV).scatter(
        1, s["ids"].long(), 1.0)
    counts = of @ taken
    total = counts.sum(1, keepdim=True).clamp(min=1)
    f = E * counts / total
    out = dict(loss=(f * P).sum(1).float(), probs=P.float(),
               counts=counts.int())
    # differences of counts in 64 bits: their mean takes most of them away
    a = torch.cat([(s["grad"].double() / n).unsqueeze(1) * f,
                   torch.zeros_like(f[:1])])[seq]
    grad = p * (a - (p * a).sum(1, keepdim=True))
    if back is not None:
        grad = grad * back
    if c["z"]:
        lse = torch.logsumexp(l, 1)
        out["z_loss"] = ((of @ lse.double() ** 2) / n).float()
        zc = torch.cat([s["grad_z"].double() / n, s["grad_z"].new_zeros(1)])
        grad = grad + (2 * zc[seq] * lse).unsqueeze(1) * soft
    return out, (grad + s["add"].float()).to(s["logits"].dtype)


def _e2m1(dtype):
    """[256, 2]: the two values of a byte."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device=DEV)
    b = torch.arange(256, device=DEV)
    return torch.stack([v[b & 15], v[b >> 4]], 1)


def _payload(q, fmt, dtype=torch.float32):
    if fmt == "mxfp4":
        return _e2m1(dtype)[q.int()].reshape(q.shape[:-1] + (-1,))
    return q.view(torch.float8_e4m3fn).to(dtype)


def _dequant(q, scales, fmt, dtype=torch.float32):
    v = _payload(q, fmt, dtype)
    e = (scales.to(dtype) - 127).unsqueeze(-1)
    return torch.ldexp(v.reshape(e.shape[:-1] + (G,)), e).reshape(v.shape)


def _quant_run(s):
    c = s["case"]
    q, b = _quant(s["x"].float(), "mxfp4", c["rule"])
    if c["wide"] == "bf16":
        return _dequant(q, b, "mxfp4").to(torch.bfloat16)
    return _payload(q, "mxfp4").to(torch.float8_e4m3fn), \
        b.view(torch.float8_e8m0fnu)


def _dispatch(s):
    q, b = _quant(s["x"].float(), "mxfp4", s["case"]["rule"])
    d = s["src2dst"].long()
    t = torch.arange(d.shape[0], device=DEV).unsqueeze(1).expand_as(d)
    rows = s["q"].index_copy(0, d.reshape(-1), q[t.reshape(-1)])
    scales = s["scales"].index_copy(0, d.reshape(-1), b[t.reshape(-1)])
    return _payload(rows, "mxfp4").to(torch.float8_e4m3fn), \
        scales.view(torch.float8_e8m0fnu)


def _silu_mul(y):
    gate, up = y.chunk(2, -1)
    return gate * torch.sigmoid(gate) * up


def _experts(s):
    c = s["case"]
    E, rows, M = c["E"], s["q"].shape[0], max(1, s["most"])
    first, count = s["offsets"][:-1].long(), s["counts"].long()
    at = (first.unsqueeze(1) + torch.arange(M, device=DEV)).clamp(max=rows - 1)
    x = _dequant(s["q"], s["scales"], c["fmt"])[at]
    w1 = _dequant(s["w1"], s["s1"], "mxfp4").transpose(1, 2).contiguous()
    y = torch.bmm(x, w1)
    if s["b1"] is not None:
        y = y + s["b1"].unsqueeze(1)
    y = _silu_mul(y).reshape(E * M, -1)
    y = _dequant(*_quant(y, c["mid"]), c["mid"]).reshape(E, M, -1)
    w2 = _dequant(s["w2"], s["s2"], "mxfp4").transpose(1, 2).contiguous()
    y = torch.bmm(y, w2)
    if s["b2"] is not None:
        y = y + s["b2"].unsqueeze(1)
    # back from [E, M] to the layout's rows
    r = torch.arange(rows, device=DEV)
    e = (torch.searchsorted(s["offsets"].long(), r, right=True) - 1).clamp(
        max=E - 1)
    j = r - first[e]
    live = ((j < count[e]) & (r < s["offsets"][-1])).unsqueeze(1)
    y = y.reshape(E * M, -1)[e * M + j.clamp(max=M - 1)]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return torch.where(live, y.to(torch.bfloat16), s["out"])


# --------------------------------------------------------------------- run

def run(state):
    s, c = state, state["case"]
    if own:
        import fp8_mx_activation_amd as mxq
        if c["op"] == "balance":
            out = mxq.moe_balance_loss(
                s["logits"], s["ids"], scoring=c["scoring"],
                seq_offsets=s["offsets"], seq_lens=s["lens"], z_loss=c["z"],
                out=s["out"])
            return out, mxq.moe_balance_loss_backward(
                s["grad"], s["logits"], out["counts"], scoring=c["scoring"],
                seq_offsets=s["offsets"], seq_lens=s["lens"],
                grad_z=s["grad_z"], add=s["add"],
                grad_logits=s["grad_logits"])
        if c["op"] == "quant":
            q, b = mxq.mxfp4_quant_rows(s["x"], rule=c["rule"], q=s["q"],
                                        scales=s["scales"])
            if c["wide"] == "bf16":
                return mxq.upscale_mxfp4_to_bf16(q, b, out=s["out"])
            return mxq.mxfp4_to_e4m3(q, out=s["out"]).view(
                torch.float8_e4m3fn), b.view(torch.float8_e8m0fnu)
        if c["op"] == "dispatch":
            q, b = mxq.moe_scatter_quant_mxfp4(
                s["x"], s["src2dst"], s["q"].shape[0], rule=c["rule"],
                q=s["q"], scales=s["scales"])
            return mxq.mxfp4_to_e4m3(q, out=s["out"]).view(
                torch.float8_e4m3fn), b.view(torch.float8_e8m0fnu)
        q, b = mxq.moe_expert_matmul_mxfp4_quant(
            s["q"], s["scales"], s["w1"], s["s1"], s["offsets"], s["counts"],
            fmt=c["fmt"], act="silu_mul", bias=s["b1"], out_fmt=c["mid"],
            q_out=s["mid"], scales_out=s["mid_scales"],
            expected_m=s["expected"])
        return mxq.moe_expert_matmul_mxfp4(
            q, b, s["w2"], s["s2"], s["offsets"], s["counts"], fmt=c["mid"],
            bias=s["b2"], residual=s["residual"], out=s["out"],
            expected_m=s["expected"])
    if c["op"] == "balance":
        return _balance(s)
    if c["op"] == "quant":
        return _quant_run(s)
    if c["op"] == "dispatch":
        return _dispatch(s)
    return _experts(s)


def work(case):
    c = case
    if c["op"] == "balance":
        T, E, K, S = c["T"], c["E"], c["K"], c["S"]
        size = 2 if c["dtype"] == "bf16" else 4
        # logits once for the loss and once for the gradient, which needs
        # the whole batch's counts; the gradient added to, and the result
        return {"bytes": 4 * T * E * size + 4 * T * K + 8 * S * E,
                "flops": 20 * T * E}
    H = c["H"]
    small = H / 2 + H / G  # a row in 4 bits
    if c["op"] == "quant":
        back = 2 * H if c["wide"] == "bf16" else H
        return {"bytes": c["rows"] * (H * (2 if c["dtype"] == "bf16" else 4) +
                                      2 * small + back),
                "flops": 4 * c["rows"] * H}
    A = c["T"] * c["K"]
    if c["op"] == "dispatch":
        return {"bytes": c["T"] * 2 * H + A * (2 * small + H),
                "flops": 4 * c["T"] * H}
    E, I = c["E"], c["I"]
    used = E * (1 - (1 - c["K"] / E) ** c["T"])  # experts that hold a row
    row = {"mxfp4": 1 / 2 + 1 / G, "e8m0_g32": 1 + 1 / G}
    per_row = H * row[c["fmt"]] + 2 * I * row[c["mid"]] + 2 * H + (
        2 * H if c["residual"] else 0)
    return {"bytes": A * per_row + used * 3 * I * H * row["mxfp4"],
            "flops": 2 * A * 3 * I * H}


# ------------------------------------------------------------------- exact

def _nearest(v):
    """e2m1 values nearest to v, by distance; of two as near the even one."""
    a = v.abs()
    table = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    hi = torch.searchsorted(table, a).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    dh, dl = table[hi] - a, a - table[lo]
    take = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.copysign(table[torch.where(take, hi, lo)], v)


def _exact_group(v, fmt, rule):
    """Values that a group's quantized form stands for, as payload and
    scale."""
    x = v.reshape(v.shape[0], -1, G)
    amax = x.abs().amax(-1)
    most, top = (6.0, 2) if fmt == "mxfp4" else (448.0, 8)
    e = torch.floor(torch.log2(amax)) - top if rule == "ocp_floor" else \
        torch.ceil(torch.log2(amax / most))
    # logarithms of values next to a power of two may round to either side
    if rule == "ocp_floor":
        e = torch.where(torch.exp2(e + top) > amax, e - 1, e)
        e = torch.where(torch.exp2(e + top + 1) <= amax, e + 1, e)
    else:
        e = torch.where(most * torch.exp2(e) < amax, e + 1, e)
        e = torch.where(most * torch.exp2(e - 1) >= amax, e - 1, e)
    e = torch.where(amax > 0, e, -127.0).clamp(-127, 127)
    scale = torch.exp2(e)
    p = x / scale.unsqueeze(-1)
    if fmt == "mxfp4":
        p = _nearest(p)
    else:
        _, k = torch.frexp(p)
        step = torch.exp2((k - 1).clamp(min=-6).double() - 3)
        p = (torch.round(p / step) * step).clamp(-448, 448)
    return p.reshape(v.shape), scale


def _exact_values(q, scales, fmt):
    """Rows from their bytes, bit by bit."""
    two = torch.tensor([2.0 ** (i - 127) for i in range(256)],
                       dtype=torch.float64, device=DEV)
    if fmt == "mxfp4":
        c = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1).long()
        e, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1).double(), m / 2)
        v = torch.where(c >= 8, -v, v)
    else:
        v = q.view(torch.float8_e4m3fn).double()
    return (v.reshape(v.shape[0], -1, G) *
            two[scales.long()].unsqueeze(-1)).reshape(v.shape)


def _exact_balance(s):
    """Sequence by sequence, the gradient by torch's differentiation."""
    c = s["case"]
    S, E = c["S"], c["E"]
    cut = [0, c["T"]] if s["offsets"] is None else s["offsets"].tolist()
    n = [b - a for a, b in zip(cut, cut[1:])] if s["lens"] is None else \
        s["lens"].tolist()
    out = dict(loss=[], probs=[], counts=None)
    if c["z"]:
        out["z_loss"] = []
    with torch.enable_grad():
        l = s["logits"].double().requires_grad_()
        total = 0.0
        for q in range(S):
            x = l[cut[q]:cut[q] + n[q]]
            # sigmoids' shares by their logarithms, for dead experts' sakes
            y = x if c["scoring"] == "softmax" else \
                torch.nn.functional.logsigmoid(x)
            p = (y - y.logsumexp(1, keepdim=True)).exp()
            P = p.sum(0) / n[q]
            k = torch.bincount(
                s["ids"][cut[q]:cut[q] + n[q]].reshape(-1).long(),
                minlength=E).double()
            loss = E * (k / k.sum() * P).sum()
            out["loss"].append(loss.detach())
            out["probs"].append(P.detach())
            total = total + s["grad"][q].double() * loss
            if c["z"]:
                z = (x.logsumexp(1) ** 2).sum() / n[q]
                out["z_loss"].append(z.detach())
                total = total + s["grad_z"][q].double() * z
        total.backward()
    for k in ("loss", "probs", "z_loss"):
        if k in out:
            out[k] = torch.stack(out[k])
    grad = torch.where(s["logits"] == -math.inf, 0.0, l.grad)
    return out, grad + s["add"].double()


def exact(case, seed):
    """The operators from their definitions in 64 bits, on the inputs that
    ``prepare`` makes."""
    s, c = prepare(case, seed), case
    if c["op"] == "balance":
        return _exact_balance(s)
    if c["op"] == "quant":
        p, scale = _exact_group(s["x"].double(), "mxfp4", c["rule"])
        if c["wide"] == "bf16":
            return (p.reshape(p.shape[0], -1, G) *
                    scale.unsqueeze(-1)).reshape(p.shape)
        return p, scale
    if c["op"] == "dispatch":
        p, scale = _exact_group(s["x"].double(), "mxfp4", c["rule"])
        d = s["src2dst"].long()
        # rows that hold nothing keep the state's bytes: 0 and 2^-127
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        sc = torch.full(s["scales"].shape, 2.0 ** -127, dtype=torch.float64,
                        device=DEV)
        for k in range(c["K"]):
            out[d[:, k]], sc[d[:, k]] = p, scale
        return out, sc
    out = s["out"].double()
    first, count = s["offsets"].tolist(), s["counts"].tolist()
    for e in range(c["E"]):
        a, b = first[e], first[e] + count[e]
        if a == b:
            continue
        x = _exact_values(s["q"][a:b], s["scales"][a:b], c["fmt"])
        y = x @ _exact_values(s["w1"][e], s["s1"][e], "mxfp4").t()
        if s["b1"] is not None:
            y += s["b1"][e].double()
        I = c["I"]
        y = y[:, :I] / (1 + (-y[:, :I]).exp()) * y[:, I:]
        p, scale = _exact_group(y, c["mid"], "no_clip")
        y = (p.reshape(b - a, -1, G) * scale.unsqueeze(-1)).reshape(b - a, I)
        y = y @ _exact_values(s["w2"][e], s["s2"][e], "mxfp4").t()
        if s["b2"] is not None:
            y += s["b2"][e].double()
        if s["residual"] is not None:
            y += s["residual"][a:b].double()
        out[a:b] = y
    return out
