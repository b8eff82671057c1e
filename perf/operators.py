"""The fine-tuning operators of packed weights, as cases to be measured.

A packed matrix holds b-bit codes q (LSB first along the row, in 32-bit words)
and one scale s and bias z per group of `gs` columns; w = q * s + z.  The cases
cover the lookup in a packed table and the gradient of its scales and biases,
the gated feed-forward block (SiLU(x Wg^T) * (x Wu^T)) with its backward pass,
and the backward pass of the quantized matmul.

With `own` false, run() computes them in their plain form from elementary torch
operations; with `own` true it calls the framework.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token of a decoding sequence looks up its row: latency
        dict(name="embed_one", op="embed", T=1, V=32768, D=4096, bits=4, gs=64, dt="bf16", out="bf16"),
        # a long packed prompt over a large vocabulary: bandwidth
        dict(name="embed_long", op="embed", T=16384, V=131072, D=4096, bits=4, gs=64, dt="bf16", out="bf16"),
        # one short training sequence, f32 gradients of the table's scales and biases
        dict(name="embed_grad_short", op="embed_grad", T=509, V=32768, D=2048, bits=6, gs=32, dt="f16", out="f32"),
        # a training batch over a large vocabulary
        dict(name="embed_grad_long", op="embed_grad", T=16384, V=131072, D=4096, bits=4, gs=64, dt="bf16", out="bf16"),
        # one decoding token through the gated block of an 8B dense layer
        dict(name="gate_up_one", op="gate_up", M=1, K=4096, F=14336, bits=4, gs=64, dt="bf16", save=False),
        # a decoding batch of a small layer with an odd number of rows
        dict(name="gate_up_few", op="gate_up", M=13, K=2048, F=1001, bits=6, gs=32, dt="f16", save=False),
        # a short prompt
        dict(name="gate_up_prompt", op="gate_up", M=200, K=4096, F=14336, bits=4, gs=64, dt="bf16", save=False),
        # the forward pass of a training step: pre-activations are kept
        dict(name="gate_up_train", op="gate_up", M=4096, K=4096, F=14336, bits=4, gs=64, dt="bf16", save=True),
        # the backward pass of a short ragged batch
        dict(name="gate_up_grad_short", op="gate_up_grad", M=77, K=2080, F=1001, bits=3, gs=32, dt="bf16"),
        # the backward pass of a training step
        dict(name="gate_up_grad_train", op="gate_up_grad", M=4096, K=4096, F=14336, bits=4, gs=64, dt="bf16"),
        # the backward pass of a projection, a short batch
        dict(name="matmul_grad_short", op="matmul_grad", M=33, K=2048, N=4096, bits=8, gs=128, dt="f16"),
        # the backward pass of the down projection of a training step
        dict(name="matmul_grad_train", op="matmul_grad", M=4096, K=14336, N=4096, bits=4, gs=64, dt="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "gate_up", "gate_up_grad", "matmul_grad"])
    bits, gs = rng.choice([2, 3, 4, 4, 6, 8]), rng.choice([32, 64, 64, 128])
    dt = rng.choice(["bf16", "bf16", "f16"])
    if op in ("embed", "embed_grad"):
        c = dict(op=op, T=_spread(rng, 1, 16384), V=_spread(rng, 1000, 131072), D=gs * rng.randint(1, 4096 // gs),
                 bits=bits, gs=gs, dt=dt, out=rng.choice([dt, dt, "f32"]))
        return c
    cols = gs * max(1, _spread(rng, 256, 4096) // gs)
    c = dict(op=op, M=_spread(rng, 1, 4096), K=cols, bits=bits, gs=gs, dt=dt)
    if op == "matmul_grad":
        c["N"] = _spread(rng, 64, 14336)
    else:
        c["F"] = _spread(rng, 64, 14336)
    if op == "gate_up":
        c["save"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs
def _pack(q, bits):
    """[rows, cols] codes -> [rows, cols * bits / 32] int32 words: 32 codes fill `bits` words."""
    rows, cols = q.shape
    step = max(1, (1 << 26) // (cols * bits))
    place = torch.arange(32, device=q.device)
    parts = []
    for r in range(0, rows, step):
        b = (q[r:r + step].view(-1, 32, 1) >> torch.arange(bits, device=q.device)) & 1
        w = (b.reshape(-1, bits, 32).to(torch.int64) << place).sum(-1)
        parts.append((w - ((w >> 31) << 32)).to(torch.int32).view(-1, cols * bits // 32))
    return torch.cat(parts)


def _weight(rows, cols, bits, gs, dt, gen, std=0.02):
    """Codes of normally distributed weights, with the scale and bias of a group's range."""
    top = 2 ** bits - 1
    q = torch.randn(rows, cols, device="cuda", generator=gen, dtype=torch.float16)
    q = (q.mul_(top / 6).add_(top / 2)).round_().clamp_(0, top).to(torch.int32)
    G = cols // gs
    s = (std * 6 / top) * (0.75 + 0.5 * torch.rand(rows, G, device="cuda", generator=gen))
    z = -s * (top / 2) * (0.9 + 0.2 * torch.rand(rows, G, device="cuda", generator=gen))
    return dict(packed=_pack(q, bits), scales=s.to(_DT[dt]), biases=z.to(_DT[dt]), rows=rows, cols=cols, gs=gs,
                bits=bits)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c, dt = case, _DT[case["dt"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std).to(dt)

    s = dict(case=dict(case))
    if c["op"] in ("embed", "embed_grad"):
        s["w"] = _weight(c["V"], c["D"], c["bits"], c["gs"], c["dt"], gen)
        # token frequencies of text: the probability of id i falls as 1 / (i + 1)
        u = torch.rand(c["T"], device="cuda", generator=gen, dtype=torch.float64)
        s["ids"] = (torch.exp(u * math.log(c["V"] + 1.0)) - 1.0).long().clamp_(0, c["V"] - 1).to(torch.int32)
        s["alpha"] = math.sqrt(c["D"])
        if c["op"] == "embed_grad":
            s["dy"] = normal(c["T"], c["D"], std=0.01)
        return s
    M, K = c["M"], c["K"]
    s["x"] = normal(M, K)
    if c["op"] == "matmul_grad":
        s["w"] = _weight(c["N"], K, c["bits"], c["gs"], c["dt"], gen)
        s["dy"] = normal(M, c["N"], std=0.01)
        return s
    s["gate"] = _weight(c["F"], K, c["bits"], c["gs"], c["dt"], gen)
    s["up"] = _weight(c["F"], K, c["bits"], c["gs"], c["dt"], gen)
    if c["op"] == "gate_up_grad":
        # the saved pre-activations of such a block, about unit scale
        s["g"], s["u"] = normal(M, c["F"]), normal(M, c["F"])
        s["dh"] = normal(M, c["F"], std=0.01)
    return s


# ---------------------------------------------------------------- the framework's calls
def _handle(s, key):
    """The framework's view of a packed weight that a program builds once."""
    from weight_only_quantized_qmm_b200 import QWeight
    h = s.setdefault("handles", {})
    if key not in h:
        w = s[key]
        h[key] = QWeight(w["packed"], w["scales"], w["biases"], w["rows"], w["cols"], w["gs"], w["bits"])
    return h[key]


def _run_own(s):
    import weight_only_quantized_qmm_b200 as q
    c = s["case"]
    op = c["op"]
    if op == "embed":
        return q.qmm_embedding(s["ids"], _handle(s, "w"), alpha=s["alpha"], y_dtype=_DT[c["out"]])
    if op == "embed_grad":
        return q.qmm_embedding_backward(s["dy"], s["ids"], _handle(s, "w"), alpha=s["alpha"], g_dtype=_DT[c["out"]])
    if op == "gate_up":
        return q.qmm_gate_up_silu(s["x"], _handle(s, "gate"), _handle(s, "up"), save=c["save"])
    if op == "gate_up_grad":
        return q.qmm_gate_up_silu_backward(s["dh"], s["x"], s["g"], s["u"], _handle(s, "gate"), _handle(s, "up"))
    return q.qmm_matmul_backward(s["dy"], s["x"], _handle(s, "w"))


# ---------------------------------------------------------------- the plain forms
def _codes(packed, cols, bits):
    """Codes of packed rows in 32-bit floats."""
    if bits in (2, 4, 8):
        at = torch.arange(32 // bits, device=packed.device, dtype=torch.int32) * bits
        q = (packed.unsqueeze(-1) >> at) & (2 ** bits - 1)
        return q.reshape(packed.shape[0], cols).to(torch.float32)
    bit = torch.arange(cols, device=packed.device) * bits
    word, sh = bit >> 5, bit & 31
    nxt = (word + 1).clamp_max(packed.shape[1] - 1)
    wide = (packed[:, word].to(torch.int64) & 0xFFFFFFFF) | (packed[:, nxt].to(torch.int64) << 32)
    return ((wide >> sh) & (2 ** bits - 1)).to(torch.float32)


def _dequant(w, rows=None):
    """(codes, values) of a packed weight (of some of its rows), [rows, groups, gs] each."""
    take = (lambda t: t) if rows is None else (lambda t: t[rows])
    q = _codes(take(w["packed"]), w["cols"], w["bits"]).view(-1, w["cols"] // w["gs"], w["gs"])
    return q, q * take(w["scales"]).float().unsqueeze(-1) + take(w["biases"]).float().unsqueeze(-1)


def _param_grads(dy, x, q):
    """Gradients of scales and biases, [rows, groups]."""
    dw = (dy.t() @ x).view(q.shape)
    return (dw * q).sum(-1), dw.sum(-1)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("embed", "embed_grad"):
        ids, out = s["ids"].long(), _DT[c["out"]]
        q, v = _dequant(s["w"], ids)
        if op == "embed":
            return (v * s["alpha"]).view(c["T"], c["D"]).to(out)
        dy = s["dy"].float().view(q.shape) * s["alpha"]
        zero = torch.zeros(c["V"], q.shape[1], device="cuda")
        ds = zero.index_add(0, ids, (dy * q).sum(-1))
        dz = zero.index_add(0, ids, dy.sum(-1))
        return ds.to(out), dz.to(out)
    dt, x = _DT[c["dt"]], s["x"].float()
    if op == "matmul_grad":
        q, v = _dequant(s["w"])
        dy = s["dy"].float()
        ds, dz = _param_grads(dy, x, q)
        return (dy @ v.view(c["N"], c["K"])).to(dt), ds.to(dt), dz.to(dt)
    qg, vg = _dequant(s["gate"])
    qu, vu = _dequant(s["up"])
    if op == "gate_up":
        g, u = x @ vg.view(c["F"], c["K"]).t(), x @ vu.view(c["F"], c["K"]).t()
        h = g / (1.0 + torch.exp(-g)) * u
        return (h.to(dt), g.to(dt), u.to(dt)) if c["save"] else h.to(dt)
    g, u, dh = s["g"].float(), s["u"].float(), s["dh"].float()
    p = 1.0 / (1.0 + torch.exp(-g))
    du = dh * (g * p)
    dg = dh * u * (p * (1.0 + g * (1.0 - p)))
    dx = dg @ vg.view(c["F"], c["K"]) + du @ vu.view(c["F"], c["K"])
    gs, gz = _param_grads(dg, x, qg)
    us, uz = _param_grads(du, x, qu)
    return dx.to(dt), (gs.to(dt), gz.to(dt)), (us.to(dt), uz.to(dt))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def _distinct(T, V):
    """Expected number of different ids among T (see prepare)."""
    i = torch.arange(1, V + 1, dtype=torch.float64)
    p = torch.log1p(1.0 / i) / math.log(V + 1.0)
    return float((1.0 - torch.exp(T * torch.log1p(-p))).sum())


def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2}

    def row(cols, with_scales=True):
        return cols * c["bits"] / 8 + (cols // c["gs"] * 4 if with_scales else 0)

    if c["op"] == "embed":
        n = c["T"] * c["D"]
        return dict(bytes=4 * c["T"] + _distinct(c["T"], c["V"]) * row(c["D"]) + n * size[c["out"]], flops=3 * n)
    if c["op"] == "embed_grad":
        n = c["T"] * c["D"]
        grads = 2 * c["V"] * (c["D"] // c["gs"]) * size[c["out"]]
        return dict(bytes=4 * c["T"] + 2 * n + _distinct(c["T"], c["V"]) * row(c["D"], False) + grads, flops=2 * n)
    M, K = c["M"], c["K"]
    if c["op"] == "matmul_grad":
        N = c["N"]
        return dict(bytes=2 * M * N + 4 * M * K + N * row(K) + 4 * N * (K // c["gs"]), flops=4 * M * N * K)
    F = c["F"]
    if c["op"] == "gate_up":
        return dict(bytes=2 * F * row(K) + 2 * M * K + 2 * M * F * (3 if c["save"] else 1), flops=4 * M * K * F)
    return dict(bytes=6 * M * F + 4 * M * K + 2 * F * row(K) + 8 * F * (K // c["gs"]), flops=8 * M * K * F)


# ---------------------------------------------------------------- from the definition, in 64 bits
def _exact_codes(packed, cols, bits):
    """Codes read off the row's bit string, as 64-bit floats."""
    step = max(1, (1 << 25) // (cols * bits))
    parts = []
    for r in range(0, packed.shape[0], step):
        string = torch.stack([(packed[r:r + step] >> k) & 1 for k in range(32)], dim=-1).to(torch.float64)
        digits = string.reshape(-1, cols, bits)
        parts.append(sum(digits[..., k] * 2.0 ** k for k in range(bits)))
    return torch.cat(parts)


def _exact_weight(w, rows=None):
    packed, s, z = w["packed"], w["scales"], w["biases"]
    if rows is not None:
        packed, s, z = packed[rows], s[rows], z[rows]
    q = _exact_codes(packed, w["cols"], w["bits"])
    return q, torch.addcmul(z.double().repeat_interleave(w["gs"], 1), q, s.double().repeat_interleave(w["gs"], 1))


def _by_group(t, gs):
    return t.unflatten(1, (-1, gs)).sum(2)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    gs = c["gs"]
    if c["op"] == "embed":
        return _exact_weight(s["w"], s["ids"].long())[1] * s["alpha"]
    if c["op"] == "embed_grad":
        # one dense row per different id, then its codes
        rows, where = torch.unique(s["ids"].long(), return_inverse=True)
        a = torch.zeros(rows.numel(), c["D"], dtype=torch.float64, device="cuda")
        a.index_add_(0, where, s["dy"].double())
        q = _exact_codes(s["w"]["packed"][rows], c["D"], c["bits"])
        ds = torch.zeros(c["V"], c["D"] // gs, dtype=torch.float64, device="cuda")
        dz = ds.clone()
        ds[rows] = s["alpha"] * _by_group(a * q, gs)
        dz[rows] = s["alpha"] * _by_group(a, gs)
        return ds, dz
    x = s["x"].double()

    def grads(dy, q):
        n = max(1, (1 << 27) // q.shape[1])
        d = [dy[:, r:r + n].t().matmul(x) for r in range(0, q.shape[0], n)]
        ds = torch.cat([_by_group(t * q[i * n:i * n + n], gs) for i, t in enumerate(d)])
        return ds, torch.cat([_by_group(t, gs) for t in d])

    if c["op"] == "matmul_grad":
        q, v = _exact_weight(s["w"])
        dy = s["dy"].double()
        return (dy.matmul(v),) + grads(dy, q)
    qg, vg = _exact_weight(s["gate"])
    qu, vu = _exact_weight(s["up"])
    if c["op"] == "gate_up":
        g, u = torch.einsum("mk,fk->mf", x, vg), torch.einsum("mk,fk->mf", x, vu)
        h = g * torch.sigmoid(g) * u
        return (h, g, u) if c["save"] else h
    g, u, dh = s["g"].double(), s["u"].double(), s["dh"].double()
    silu = g * torch.sigmoid(g)
    slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
    dg, du = dh * u * slope, dh * silu
    return dg.matmul(vg) + du.matmul(vu), grads(dg, qg), grads(du, qu)
