"""What a rounded layer meets after the solve, measured case by case.

Four operators: the 4-bit layout of a layer's codes and grid steps (``pack4`` / ``unpack4``), the
product of such a layer with the activations of a few tokens (``matvec4``), the residual's addition
with the root-mean-square norm and an 8-bit output (``rms_norm_q8``), and the distillation loss from
a teacher's top logits with its gradient (``distill``). ``run`` computes each one in elementary
torch operations, or, where ``own`` is true, with the library.

The 4-bit layout: tiles of 16 rows x 64 columns, 512 bytes each, row tiles outermost; a 32-bit word
holds 8 neighbouring columns of one row, column c at the nibble whose index is c with its three bits
reversed; word (row r, columns 8 t + 32 h ..) sits at 16 (4 (r mod 8) + t) + 8 h + 4 (r div 8) of its
tile. Behind the tiles stand the grid steps, fp32, as (row tile, group, r mod 8, r div 8).
Rows and columns that pad the last tiles hold code 0, pad rows have step 0.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}
ORDER = [0, 4, 2, 6, 1, 5, 3, 7]      # nibble p holds column ORDER[p] of its word
EPS = 1e-6
# 16 entries at normal quantiles, the kind of sorted scalar codebook that the round takes
BOOK = [-1.0, -0.6962, -0.5251, -0.3949, -0.2844, -0.1848, -0.0911, 0.0, 0.0796, 0.1609, 0.2461,
        0.3379, 0.4407, 0.5626, 0.7230, 1.0]


def listed():
    mv = dict(op="matvec4")
    nq = dict(op="rms_norm_q8", eps=EPS)
    ds = dict(op="distill")
    return [
        # one decoding step of an attention projection behind the 8-bit norm
        dict(mv, name="matvec_attn_4096_step", m=4096, n=4096, tokens=1, x="i8", y="bf16", group=128,
             x_group=0, book=False),
        # a few sequences decoded together, down projection with a codebook
        dict(mv, name="matvec_down_book", m=4096, n=14336, tokens=5, x="f16", y="f16", group=64,
             x_group=0, book=True),
        # a batch of eight sequences on the largest layer
        dict(mv, name="matvec_upgate_batch", m=28672, n=8192, tokens=8, x="bf16", y="bf16", group=128,
             x_group=0, book=False),
        # sizes that fill no tile, the solver's own fp32 and one step per row
        dict(mv, name="matvec_ragged", m=1003, n=2500, tokens=3, x="f32", y="f32", group=0, x_group=0,
             book=False),
        # the norm of one decoding step
        dict(nq, name="norm_step", rows=1, n=4096, x="bf16", group=0, residual=True),
        # the norm over a prompt, one step per 128 columns
        dict(nq, name="norm_prompt", rows=2048, n=8192, x="bf16", group=128, residual=True),
        # fp32 calibration rows of odd length, nothing to add
        dict(nq, name="norm_ragged", rows=333, n=5003, x="f32", group=0, residual=False),
        # the loss alone, to see what a rounding cost
        dict(ds, name="distill_eval", rows=64, vocab=32000, x="f32", k=20, tau=1.0, grad=False,
             mass=True, ragged=False),
        # a step of recovery training: loss and gradient over a large vocabulary
        dict(ds, name="distill_step", rows=2048, vocab=131072, x="bf16", k=64, tau=2.0, grad=True,
             mass=False, ragged=False),
        # an odd vocabulary with masked entries, short lists and rows that do not count
        dict(ds, name="distill_ragged", rows=100, vocab=50001, x="f16", k=7, tau=1.5, grad=True,
             mass=True, ragged=True),
        # laying out one layer after its solve, and taking it apart again
        dict(op="pack4", name="pack_attn_4096", m=4096, n=4096, group=128, book=False),
        dict(op="pack4", name="pack_upgate", m=28672, n=8192, group=128, book=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec4", "matvec4", "rms_norm_q8", "distill", "pack4"])
    if op == "matvec4":
        m, n, tokens = _log(rng, 48, 28672), _log(rng, 64, 14336), _log(rng, 1, 32)
        while m * n * tokens > 28672 * 8192 * 8 or m * n > 28672 * 8192:
            m, n, tokens = _log(rng, 48, 28672), _log(rng, 64, 14336), _log(rng, 1, 32)
        x = rng.choice(["f32", "f16", "bf16", "i8"])
        return dict(op=op, m=m, n=n, tokens=tokens, x=x, y=rng.choice(["f16", "bf16"]) if x == "i8" else x,
                    group=rng.choice([0, 32, 64, 128]), x_group=rng.choice([0, 128]) if x == "i8" else 0,
                    book=rng.random() < 0.3)
    if op == "rms_norm_q8":
        rows, n = _log(rng, 1, 4096), _log(rng, 64, 16384)
        while rows * n > 2048 * 8192:
            rows, n = _log(rng, 1, 4096), _log(rng, 64, 16384)
        return dict(op=op, rows=rows, n=n, x=rng.choice(["f32", "f16", "bf16"]), eps=EPS,
                    group=rng.choice([0, 128]), residual=rng.random() < 0.7)
    if op == "distill":
        rows, vocab = _log(rng, 1, 2048), _log(rng, 4000, 131072)
        return dict(op=op, rows=rows, vocab=vocab, x=rng.choice(["f32", "f16", "bf16"]), k=_log(rng, 1, 256),
                    tau=rng.choice([1.0, 2.0]), grad=rng.random() < 0.7, mass=rng.random() < 0.5,
                    ragged=rng.random() < 0.5)
    m, n = _log(rng, 48, 28672), _log(rng, 64, 14336)
    while m * n > 28672 * 8192:
        m, n = _log(rng, 48, 28672), _log(rng, 64, 14336)
    return dict(op=op, m=m, n=n, group=rng.choice([0, 32, 64, 128]), book=rng.random() < 0.3)


# ------------------------------------------------------------------------------------- inputs
def _groups(n, group):
    g = n if group == 0 else min(group, n)
    return g, -(-n // g)


def _round_layer(m, n, group, book, gen):
    """(codes, steps) of a layer: N(0, 1/n) weights with rows of unequal size, rounded to nearest."""
    g, G = _groups(n, group)
    W = torch.randn(m, n, generator=gen, device="cuda") / math.sqrt(n)
    W *= torch.exp(0.3 * torch.randn(m, 1, generator=gen, device="cuda"))
    pad = torch.zeros(m, G * g, device="cuda")
    pad[:, :n] = W.abs()
    steps = pad.view(m, G, g).amax(dim=2) / (1.0 if book else 7.5)
    del pad
    W /= steps.repeat_interleave(g, dim=1)[:, :n]
    if book:
        b = torch.tensor(BOOK, device="cuda")
        return torch.bucketize(W, (b[1:] + b[:-1]) / 2).to(torch.int8), steps
    return W.round_().clamp_(-8, 7).to(torch.int8), steps


def _lay_out(codes, steps):
    m, n = codes.shape
    Mt, Kt, G = -(-m // 16), -(-n // 64), steps.shape[1]
    c = torch.zeros(Mt * 16, Kt * 64, dtype=torch.uint8, device="cuda")
    c[:m, :n] = codes.view(torch.uint8) & 15
    c = c.view(Mt, 2, 8, Kt, 2, 4, 8)[..., ORDER]
    c = c[..., 0::2] | (c[..., 1::2] << 4)
    c = c.permute(0, 3, 2, 5, 4, 1, 6).reshape(-1)
    s = torch.zeros(Mt * 16, G, device="cuda")
    s[:m] = steps
    s = s.view(Mt, 2, 8, G).permute(0, 3, 2, 1).reshape(-1)
    return torch.cat([c, s.view(torch.uint8)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    op = case["op"]
    st = {"case": case}
    if op in ("matvec4", "pack4"):
        m, n = case["m"], case["n"]
        codes, steps = _round_layer(m, n, case["group"], case["book"], gen)
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op == "pack4":
            st.update(codes=codes, steps=steps)
            return st
        st["packed"] = _lay_out(codes, steps)
        x = rnd(case["tokens"], n)
        x[:, :: 97] *= 8.0                       # a few large features, as activations have
        if case["x"] == "i8":
            g, G = _groups(n, case["x_group"])
            p = torch.zeros(case["tokens"], G * g, device="cuda")
            p[:, :n] = x
            s = p.view(-1, G, g).abs().amax(dim=2) / 127
            st["x_scales"] = s
            x = (x / s.repeat_interleave(g, dim=1)[:, :n]).round()
        st["x"] = x.to(DTYPES[case["x"]])
        return st
    if op == "rms_norm_q8":
        rows, n, dt = case["rows"], case["n"], DTYPES[case["x"]]
        st["x"] = rnd(rows, n).to(dt)
        st["weight"] = (1 + 0.1 * rnd(n)).to(dt)
        st["residual"] = (3 * rnd(rows, n)).to(dt) if case["residual"] else None
        return st
    rows, V, k, dt = case["rows"], case["vocab"], case["k"], DTYPES[case["x"]]
    z = 2.5 * rnd(rows, V)
    teacher = z + 0.7 * rnd(rows, V)
    if case["ragged"]:
        z[:, V - 33:] = -math.inf                # entries that pad the vocabulary
        teacher[:, V - 33:] = -math.inf
    val, idx = teacher.topk(k, dim=1)
    st["lse"] = torch.logsumexp(teacher / case["tau"], dim=1) if case["mass"] else None
    del teacher
    st["weights"] = None
    if case["ragged"]:
        keep = torch.rand(rows, k, generator=gen, device="cuda") < 0.8      # shorter lists
        idx = torch.where(keep, idx, torch.full_like(idx, -1))
        st["weights"] = (torch.rand(rows, generator=gen, device="cuda") < 0.7).float()
    elif case["grad"]:
        st["weights"] = torch.full((rows,), case["tau"] ** 2 / rows, device="cuda")
    st.update(logits=z.to(dt), idx=idx.to(torch.int32), top=val.contiguous(),
              status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return st


# -------------------------------------------------------------------------------- plain forms
def _take_apart(packed, m, n, G, book):
    """(codes, steps) from the 4-bit layout, codes as int8."""
    Mt, Kt = -(-m // 16), -(-n // 64)
    c = packed[: Mt * Kt * 512].view(Mt, Kt, 8, 4, 2, 2, 4).permute(0, 5, 2, 1, 4, 3, 6)
    c = torch.stack([c & 15, c >> 4], dim=-1).flatten(-2)[..., ORDER]
    c = c.reshape(Mt * 16, Kt * 64)[:m, :n].contiguous().view(torch.int8)
    s = packed[Mt * Kt * 512:].view(torch.float32).view(Mt, G, 8, 2).permute(0, 3, 2, 1)
    s = s.reshape(Mt * 16, G)[:m].contiguous()
    return (c if book else torch.where(c > 7, c - 16, c)), s


def _plain_matvec4(st):
    c = st["case"]
    m, n = c["m"], c["n"]
    g, G = _groups(n, c["group"])
    codes, steps = _take_apart(st["packed"], m, n, G, c["book"])
    W = torch.tensor(BOOK, device="cuda")[codes.to(torch.int32)] if c["book"] else codes.float()
    W = W * steps.repeat_interleave(g, dim=1)[:, :n]
    x = st["x"].float()
    if c["x"] == "i8":
        gx, _ = _groups(n, c["x_group"])
        x = x * st["x_scales"].repeat_interleave(gx, dim=1)[:, :n]
    return (x @ W.T).to(DTYPES[c["y"]])


def _plain_norm(st):
    c = st["case"]
    x, w, r = st["x"], st["weight"], st["residual"]
    rows, n = x.shape
    g, G = _groups(n, c["group"])
    h = x.float() if r is None else x.float() + r.float()
    rho = torch.rsqrt(h.square().mean(dim=1, keepdim=True) + c["eps"])
    # 64 bits: a quotient next to the border of two codes goes to its own side
    v = (x.double() if r is None else x.double() + r.double()) * w.double()
    pad = torch.zeros(rows, G * g, dtype=torch.float64, device="cuda")
    pad[:, :n] = v
    vmax = pad.view(rows, G, g).abs().amax(dim=2)
    t = v * 127 / vmax.repeat_interleave(g, dim=1)[:, :n]
    q = torch.where(vmax.repeat_interleave(g, dim=1)[:, :n] > 0, t.round(), 0.0).to(torch.int8)
    out = {"q": q, "scales": vmax.float() * rho / 127}
    if r is not None:
        out["sum"] = h.to(x.dtype)
    return out


def _plain_distill(st):
    c = st["case"]
    z = st["logits"].float() / c["tau"]
    idx, t = st["idx"].long(), st["top"] / c["tau"]
    there = idx >= 0
    t = torch.where(there, t, -math.inf)
    zmax = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - zmax)
    lse = zmax + e.sum(dim=1, keepdim=True).log()
    if st["lse"] is None:
        tmax = t.amax(dim=1, keepdim=True)
        tmax = torch.where(tmax > -math.inf, tmax, 0.0)
        tl = tmax + torch.exp(t - tmax).sum(dim=1, keepdim=True).log()
    else:
        tl = st["lse"][:, None]
    p = torch.where(t > -math.inf, torch.exp(t - tl), 0.0)
    at = idx.clamp(min=0)
    kl = torch.where(p > 0, p * ((t - tl) - (z.gather(1, at) - lse)), 0.0).sum(dim=1)
    w = st["weights"]
    out = {"loss": kl if w is None else torch.where(w != 0, w * kl, 0.0), "lse": lse[:, 0]}
    if w is not None:
        out["lse"] = torch.where(w != 0, out["lse"], 0.0)
    if c["grad"]:
        d = torch.exp(z - lse) * p.sum(dim=1, keepdim=True)
        d.scatter_add_(1, at, -p)
        d = d / c["tau"] if w is None else d * (w[:, None] / c["tau"])
        out["grad"] = d.to(st["logits"].dtype)
    return out


def _plain_pack4(st):
    c = st["case"]
    packed = _lay_out(st["codes"], st["steps"])
    codes, steps = _take_apart(packed, c["m"], c["n"], st["steps"].shape[1], c["book"])
    return {"packed": packed, "codes": codes, "steps": steps}


# --------------------------------------------------------------------------------- one pass
def _own_run(st):
    from two_sided_adaptive_bakron_b200 import bakron as bk
    c = st["case"]
    op = c["op"]
    if op == "matvec4":
        return bk.matvec4(st["packed"], c["m"], c["n"], st["x"], group_size=c["group"] or None,
                          codebook=BOOK if c["book"] else None, x_scales=st.get("x_scales"),
                          x_group_size=c["x_group"] or None, out_dtype=DTYPES[c["y"]])
    if op == "rms_norm_q8":
        q, s, h = bk.rms_norm_q8(st["x"], st["weight"], c["eps"], residual=st["residual"],
                                 group_size=c["group"] or None)
        return {"q": q, "scales": s} if h is None else {"q": q, "scales": s, "sum": h}
    if op == "distill":
        loss, lse, grad = bk.distill(st["logits"], st["idx"], st["top"], c["tau"], teacher_lse=st["lse"],
                                     row_weights=st["weights"], grad=c["grad"], status=st["status"])
        return {"loss": loss, "lse": lse, "grad": grad} if c["grad"] else {"loss": loss, "lse": lse}
    g = c["group"] or c["n"]        # steps stand as rows x steps, one step a row too
    packed = bk.pack4(st["codes"], st["steps"], group_size=g, unsigned=c["book"], status=st["status"])
    codes, steps = bk.unpack4(packed, c["m"], c["n"], group_size=g, unsigned=c["book"])
    return {"packed": packed, "codes": codes, "steps": steps}


def run(state):
    if own:
        return _own_run(state)
    return {"matvec4": _plain_matvec4, "rms_norm_q8": _plain_norm, "distill": _plain_distill,
            "pack4": _plain_pack4}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op in ("matvec4", "pack4"):
        m, n = case["m"], case["n"]
        _, G = _groups(n, case["group"])
        held = -(-m // 16) * -(-n // 64) * 512 + -(-m // 16) * G * 64
        if op == "pack4":       # codes and steps in, the layout out and in, codes and steps out
            return {"bytes": 2 * (m * n + 4 * m * G + held), "flops": 0}
        T = case["tokens"]
        xs = 4 * T * _groups(n, case["x_group"])[1] if case["x"] == "i8" else 0
        return {"bytes": held + T * n * BYTES[case["x"]] + xs + T * m * BYTES[case["y"]],
                "flops": 2 * T * m * n}
    if op == "rms_norm_q8":
        rows, n, b = case["rows"], case["n"], BYTES[case["x"]]
        _, G = _groups(n, case["group"])
        moved = 3 if case["residual"] else 1
        return {"bytes": rows * n * (b * moved + 1) + n * b + 4 * rows * G, "flops": 6 * rows * n}
    rows, V, b = case["rows"], case["vocab"], BYTES[case["x"]]
    return {"bytes": rows * V * b * (2 if case["grad"] else 1) + rows * (8 * case["k"] + 16),
            "flops": rows * V * (7 if case["grad"] else 4)}


# ------------------------------------------------------------------------------ in 64 bits
def _exact_weights(st):
    """The layer's weights, by index arithmetic on the layout, in float64."""
    c = st["case"]
    m, n, dev = c["m"], c["n"], "cuda"
    g, G = _groups(n, c["group"])
    Kt = -(-n // 64)
    j = torch.arange(n, device=dev)
    rev = (j & 1) * 4 + (j & 2) + (j & 4) // 4
    W = torch.empty(m, n, dtype=torch.float64, device=dev)
    book = torch.tensor(BOOK, dtype=torch.float32, device=dev).double()
    s0 = -(-m // 16) * Kt * 512
    steps = st["packed"][s0:].view(torch.float32)
    for lo in range(0, m, 4096):
        i = torch.arange(lo, min(m, lo + 4096), device=dev)[:, None]
        at = ((i // 16) * Kt + j // 64) * 512 + (4 * (i % 8) + (j % 32) // 8) * 16 \
            + 8 * ((j % 64) // 32) + 4 * ((i % 16) // 8) + rev // 2
        nib = (st["packed"][at] >> (4 * (rev % 2)).to(torch.uint8)) & 15
        del at
        val = book[nib.int()] if c["book"] else ((nib.double() + 8) % 16) - 8
        s = steps[(((i // 16) * G + torch.arange(G, device=dev)) * 8 + i % 8) * 2 + (i % 16) // 8].double()
        W[lo:lo + 4096] = val * s[:, j // g]
    return W


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "pack4":
        return {"packed": None, "codes": None, "steps": st["steps"].double()}
    if op == "matvec4":
        x = st["x"].double()
        if case["x"] == "i8":
            x = x * st["x_scales"].double()[:, torch.arange(case["n"], device="cuda") // _groups(case["n"], case["x_group"])[0]]
        return torch.einsum("tj,ij->ti", x, _exact_weights(st))
    if op == "rms_norm_q8":
        x, w = st["x"].double(), st["weight"].double()
        h = x + st["residual"].double() if case["residual"] else x
        rms = torch.sqrt((h * h).sum(dim=1) / case["n"] + case["eps"])
        g, G = _groups(case["n"], case["group"])
        y = (h / rms[:, None]) * w
        top = torch.stack([part.abs().amax(dim=1) for part in y.split(g, dim=1)], dim=1)
        out = {"q": None, "scales": top / 127}
        if case["residual"]:
            out["sum"] = h
        return out
    tau, rows, V = case["tau"], case["rows"], case["vocab"]
    w = torch.ones(rows, device="cuda") if st["weights"] is None else st["weights"]
    out = {"loss": torch.zeros(rows, dtype=torch.float64, device="cuda"),
           "lse": torch.zeros(rows, dtype=torch.float64, device="cuda")}
    if case["grad"]:
        out["grad"] = torch.zeros(rows, V, dtype=torch.float64, device="cuda")
    for lo in range(0, rows, 256):
        r = slice(lo, min(rows, lo + 256))
        on = (w[r] != 0)[:, None]
        logq = torch.log_softmax(st["logits"][r].double() / tau, dim=1)
        lse = torch.logsumexp(st["logits"][r].double() / tau, dim=1)
        i, t = st["idx"][r].long(), st["top"][r].double() / tau
        use = (i >= 0) & torch.isfinite(t)
        t = t.masked_fill(~use, -math.inf)
        if st["lse"] is None:
            logp = t - torch.logsumexp(t, dim=1, keepdim=True)
        else:
            logp = t - st["lse"][r].double()[:, None]
        p = logp.exp().masked_fill(~use, 0.0)
        lq = torch.take_along_dim(logq, i.clamp(min=0), dim=1)
        term = (p * (logp - lq)).masked_fill(~use, 0.0)
        out["loss"][r] = torch.where(on[:, 0], w[r].double() * term.sum(dim=1), 0.0)
        out["lse"][r] = torch.where(on[:, 0], lse, 0.0)
        if case["grad"]:
            full = torch.zeros_like(logq).scatter_add(1, i.clamp(min=0), p)
            out["grad"][r] = (w[r].double() / tau)[:, None] * (p.sum(dim=1, keepdim=True) * logq.exp() - full)
    return out
