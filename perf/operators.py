"""The expert operators beside the layer call, as cases that can be timed and compared.

Three kinds of work on the experts' rows and weights:

* ``gmm``   matrix products grouped by expert over ragged row segments: the experts' linears
            (``nt``), their input gradient (``nn``) and their weight gradient (``tn``);
* ``ckpt``  8-bit activation checkpoints: ``step`` is the activation that saves its
            pre-activation in 8 bits, and its backward pass from that checkpoint; ``copy`` saves
            rows and reads them back;
* ``q4``    matrix-vector products of (token, slot) pairs with 4-bit expert weights.

``own`` false: the plain form, elementary torch operations in 32 bits.  ``own`` true: the calls a
user makes of this package.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# e2m1 values by code (sign in bit 3)
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a small GPT-2-width layer's up projection for a couple of hundred rows: latency
        dict(name="gmm_nt_small", op="gmm", kind="nt", groups=6, n=1536, k=768, rows=203, dtype="bf16", out="bf16",
             zipf=False),
        # one rank's 32 fine-grained experts, packed gate_up projection of a prefill or training batch
        dict(name="gmm_nt_large", op="gmm", kind="nt", groups=32, n=4096, k=7168, rows=16384, dtype="bf16",
             out="bf16", zipf=False),
        # the input gradient of eight wide experts under a skewed router, an expert without rows
        dict(name="gmm_nn_skewed", op="gmm", kind="nn", groups=8, n=14336, k=4096, rows=5003, dtype="bf16",
             out="bf16", zipf=True),
        # weight gradients of the fine-grained experts' down projection, fp32 for the optimizer
        dict(name="gmm_tn_large", op="gmm", kind="tn", groups=32, n=7168, k=2048, rows=16384, dtype="bf16",
             out="f32", zipf=False),
        # weight gradients at an odd width and odd segment lengths
        dict(name="gmm_tn_ragged", op="gmm", kind="tn", groups=8, n=2880, k=1000, rows=4099, dtype="bf16",
             out="bf16", zipf=True),
        # an fp32 layer's products
        dict(name="gmm_nt_f32", op="gmm", kind="nt", groups=8, n=1024, k=256, rows=1024, dtype="f32", out="f32",
             zipf=False),
        # activation and its backward for a few rows: latency
        dict(name="ckpt_step_small", op="ckpt", kind="step", rows=37, width=2880, act="swiglu", dtype="bf16",
             format="int8", group=64),
        # the same for the routed rows of a large training batch
        dict(name="ckpt_step_large", op="ckpt", kind="step", rows=65536, width=2048, act="swiglu", dtype="bf16",
             format="int8", group=128),
        # GELU experts, 8-bit floats, a width that ends inside a group
        dict(name="ckpt_step_gelu", op="ckpt", kind="step", rows=12289, width=2200, act="gelu", dtype="bf16",
             format="e4m3", group=64),
        # one token through four experts' packed gate_up projection
        dict(name="q4_up_one", op="q4", experts=32, n=5760, k=2880, tokens=1, topk=4, act="swiglu", format="int4",
             group=64, out="bf16", scaled=False),
        # eight tokens' down projection, rows weighted by their gates
        dict(name="q4_down_eight", op="q4", experts=32, n=2880, k=2880, tokens=8, topk=4, act="none", format="e2m1",
             group=32, out="f32", scaled=True),
        # a batch of 64 tokens: every expert is live with several rows
        dict(name="q4_up_many", op="q4", experts=32, n=5760, k=2880, tokens=64, topk=4, act="swiglu", format="int4",
             group=32, out="bf16", scaled=False),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["gmm", "gmm", "ckpt", "q4", "q4"])
    if op == "gmm":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        top = 7168 if dtype == "bf16" else 1536
        c = dict(op=op, kind=rng.choice(["nt", "nn", "tn"]), groups=_log(rng, 1, 48), n=_log(rng, 64, top, 8),
                 k=_log(rng, 64, top, 8), rows=_log(rng, 1, 16384 if dtype == "bf16" else 2048), dtype=dtype,
                 out="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]), zipf=rng.random() < 0.5)
        while c["groups"] * c["n"] * c["k"] > 32 * 4096 * 7168:   # no more weights than the largest listed case
            c["groups"] = max(1, c["groups"] // 2)
        return c
    if op == "ckpt":
        act = rng.choice(["swiglu", "gelu"])
        c = dict(op=op, kind=rng.choice(["step", "step", "copy"]), rows=_log(rng, 1, 32768),
                 width=_log(rng, 64, 8192, 8), act=act, dtype=rng.choice(["bf16", "bf16", "f32"]),
                 format=rng.choice(["int8", "e4m3"]), group=rng.choice([32, 64, 128]))
        while c["rows"] * c["width"] > 32768 * 2048:
            c["rows"] = max(1, c["rows"] // 2)
        return c
    fmt = rng.choice(["int4", "int4", "e2m1"])
    act = rng.choice(["none", "swiglu", "gelu"])
    experts = _log(rng, 2, 32)
    return dict(op=op, experts=experts, n=_log(rng, 64, 5760, 16), k=_log(rng, 64, 4096, 32),
                tokens=_log(rng, 1, 64), topk=min(experts, rng.choice([1, 2, 4, 8])), act=act, format=fmt,
                group=32 if fmt == "e2m1" else rng.choice([32, 64, 128]), out=rng.choice(["bf16", "f32"]),
                scaled=act == "none")


def work(case):
    c = case
    if c["op"] == "gmm":
        es, os_ = (2 if c["dtype"] == "bf16" else 4), (2 if c["out"] == "bf16" else 4)
        live = min(c["groups"], c["rows"])
        if c["kind"] == "tn":
            moved = c["rows"] * (c["n"] + c["k"]) * es + c["groups"] * c["n"] * c["k"] * os_
        else:
            moved = (c["rows"] * (c["k"] if c["kind"] == "nt" else c["n"]) + live * c["n"] * c["k"]) * es \
                + c["rows"] * (c["n"] if c["kind"] == "nt" else c["k"]) * os_
        return {"bytes": moved, "flops": 2 * c["rows"] * c["n"] * c["k"]}
    if c["op"] == "ckpt":
        es = 2 if c["dtype"] == "bf16" else 4
        halves = 2 if c["act"] == "swiglu" and c["kind"] == "step" else 1
        saved = halves * (c["width"] + -(-c["width"] // c["group"]))
        if c["kind"] == "copy":   # rows in, checkpoint out; checkpoint in, rows out
            return {"bytes": c["rows"] * (2 * c["width"] * es + 2 * saved), "flops": 2 * c["rows"] * c["width"]}
        # forward: u in, h and checkpoint out; backward: checkpoint, dh and weight in, du, w h and dw out
        moved = c["rows"] * (c["width"] * es * (halves + 1 + 1 + halves + 1) + 2 * saved + 8)
        return {"bytes": moved, "flops": 30 * c["rows"] * c["width"]}
    pairs = c["tokens"] * c["topk"]
    live = c["experts"] * (1 - (1 - c["topk"] / c["experts"]) ** c["tokens"])   # expected distinct experts
    per = c["n"] * (c["k"] / 2 + -(-c["k"] // c["group"]) * (2 if c["format"] == "int4" else 1))
    cols = c["n"] // 2 if c["act"] == "swiglu" else c["n"]
    return {"bytes": int(live * per + c["tokens"] * c["k"] * 2 + pairs * cols * (2 if c["out"] == "bf16" else 4)),
            "flops": 2 * pairs * c["n"] * c["k"]}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": c}
    if c["op"] == "gmm":
        G, n, k, rows = c["groups"], c["n"], c["k"], c["rows"]
        dt, out = _DTYPES[c["dtype"]], _DTYPES[c["out"]]
        p = 1.0 / torch.arange(1, G + 1, dtype=torch.float64) if c["zipf"] else torch.ones(G, dtype=torch.float64)
        if c["zipf"] and G > 2:
            p[G // 2] = 0.0   # an expert that no row was routed to
        chosen = torch.multinomial(p, rows, replacement=True, generator=h)
        s["counts"] = torch.bincount(chosen, minlength=G).tolist()   # as the router's host copy has them
        offsets = [0]
        for v in s["counts"]:
            offsets.append(offsets[-1] + v)
        s["row_offsets"] = torch.tensor(offsets, dtype=torch.int32).cuda()
        if c["kind"] == "tn":
            s["a"], s["b"] = randn(rows, n, std=0.01, dtype=dt), randn(rows, k, dtype=dt)
            s["c"] = torch.empty(G, n, k, dtype=out, device="cuda")
        else:
            wide = k if c["kind"] == "nt" else n
            s["a"] = randn(rows, wide, std=1.0 if c["kind"] == "nt" else 0.01, dtype=dt)
            s["b"] = torch.empty(G, n, k, dtype=dt, device="cuda")
            for e in range(G):
                s["b"][e] = randn(n, k, std=0.02, dtype=dt)
            s["c"] = torch.empty(rows, n if c["kind"] == "nt" else k, dtype=out, device="cuda")
        return s
    if c["op"] == "ckpt":
        rows, width, dt = c["rows"], c["width"], _DTYPES[c["dtype"]]
        cols = 2 * width if c["act"] == "swiglu" and c["kind"] == "step" else width
        # pre-activations: each row has a scale of its own, a few columns are outliers
        u = torch.randn(rows, cols, generator=g, device="cuda")
        u *= torch.empty(rows, 1, device="cuda").uniform_(0.5, 2.0, generator=g)
        u *= 1 + 7 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
        s["u"] = u.to(dt)
        scales = (cols // width) * -(-width // c["group"])
        s["q"] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        s["s"] = torch.empty(rows, scales, dtype=torch.uint8, device="cuda")
        if c["kind"] == "copy":
            s["back"] = torch.empty(rows, cols, dtype=dt, device="cuda")
            return s
        s["dh"] = randn(rows, width, std=0.01, dtype=dt)
        s["w"] = torch.rand(rows, generator=g, device="cuda")
        s["h"] = torch.empty(rows, width, dtype=dt, device="cuda")
        s["du"] = torch.empty(rows, cols, dtype=dt, device="cuda")
        s["hw"] = torch.empty(rows, width, dtype=dt, device="cuda")
        s["dw"] = torch.empty(rows, device="cuda")
        return s
    N, n, k, pairs = c["experts"], c["n"], c["k"], c["tokens"] * c["topk"]
    groups = -(-k // c["group"])
    s["x"] = randn(c["tokens"], k)
    s["codes"] = torch.randint(0, 256, (N, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    if c["format"] == "int4":
        s["scales"] = torch.empty(N, n, groups, device="cuda").uniform_(0.002, 0.006, generator=g).to(torch.bfloat16)
    else:
        s["scales"] = torch.randint(118, 122, (N, n, groups), generator=g, device="cuda", dtype=torch.uint8)
    s["expert"] = torch.rand(c["tokens"], N, generator=g, device="cuda").topk(c["topk"], 1).indices \
        .to(torch.int32).reshape(pairs)
    s["gate"] = torch.rand(pairs, generator=g, device="cuda") if c["scaled"] else None
    s["y"] = torch.empty(pairs, n // 2 if c["act"] == "swiglu" else n, dtype=_DTYPES[c["out"]], device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return {"gmm": _own_gmm, "ckpt": _own_ckpt, "q4": _own_q4}[c["op"]](state, c)
    return {"gmm": _plain_gmm, "ckpt": _plain_ckpt, "q4": _plain_q4}[c["op"]](state, c)


def _own_gmm(s, c):
    import sparse_mixture_experts_10_b200 as moe
    kind = {"nt": moe.MOE_GMM_NT, "nn": moe.MOE_GMM_NN, "tn": moe.MOE_GMM_TN}[c["kind"]]
    d = moe.make_gmm(kind, c["groups"], c["n"], c["k"], moe.dtype_code(s["a"].dtype), moe.dtype_code(s["c"].dtype))
    moe.check(moe.moe_grouped_mm(d, s["a"], s["b"], s["c"], s["row_offsets"], c["rows"]))
    return s["c"]


def _own_ckpt(s, c):
    import sparse_mixture_experts_10_b200 as moe
    form = moe.MOE_CKPT_INT8 if c["format"] == "int8" else moe.MOE_CKPT_E4M3
    act = moe.MOE_ACT_SWIGLU if c["act"] == "swiglu" else moe.MOE_ACT_GELU
    if c["kind"] == "copy":
        act = moe.MOE_ACT_NONE
    d = moe.make_ckpt(c["width"], act, moe.dtype_code(s["u"].dtype), form, c["group"])
    if c["kind"] == "copy":
        moe.check(moe.moe_ckpt_forward(d, s["u"], c["rows"], None, s["q"], s["s"]))
        moe.check(moe.moe_ckpt_load(d, s["q"], s["s"], c["rows"], s["back"]))
        return s["back"]
    moe.check(moe.moe_ckpt_forward(d, s["u"], c["rows"], s["h"], s["q"], s["s"]))
    moe.check(moe.moe_ckpt_backward(d, s["q"], s["s"], c["rows"], s["dh"], s["w"], s["du"], s["hw"], s["dw"]))
    return {"h": s["h"], "du": s["du"], "hw": s["hw"], "dw": s["dw"]}


def _own_q4(s, c):
    import sparse_mixture_experts_10_b200 as moe
    act = {"none": moe.MOE_ACT_NONE, "gelu": moe.MOE_ACT_GELU, "swiglu": moe.MOE_ACT_SWIGLU}[c["act"]]
    form = moe.MOE_Q4_INT4 if c["format"] == "int4" else moe.MOE_Q4_E2M1
    d = moe.make_q4(c["experts"], c["n"], c["k"], c["group"], form, act)
    moe.check(moe.moe_q4_matvec(d, s["x"], c["tokens"] * c["topk"], c["topk"], s["expert"], s["codes"], s["scales"],
                                s["gate"], s["y"], moe.dtype_code(s["y"].dtype)))
    return s["y"]


def _segments(s, c):
    """Group and place inside the group of every row."""
    r = torch.arange(c["rows"], device="cuda", dtype=torch.int32)
    gid = torch.searchsorted(s["row_offsets"][1:], r, right=True)
    return gid, r - s["row_offsets"][gid]


def _padded(x, gid, pos, groups, most):
    out = torch.zeros(groups, most, x.shape[1], device="cuda")
    out[gid, pos] = x.float()
    return out


def _plain_gmm(s, c):
    gid, pos = _segments(s, c)
    most = max(s["counts"])
    a = _padded(s["a"], gid, pos, c["groups"], most)
    if c["kind"] == "tn":
        b = _padded(s["b"], gid, pos, c["groups"], most)
        return torch.bmm(a.transpose(1, 2), b).to(s["c"].dtype)
    w = s["b"].float()
    y = torch.bmm(a, w.transpose(1, 2) if c["kind"] == "nt" else w)
    return y[gid, pos].to(s["c"].dtype)


def _pow2(e):
    """2^e exactly, for whole e from -126 to 127: the bits of the number."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _checkpoint(u, group, form):
    """The values that an 8-bit checkpoint of u [rows, cols] stands for: powers of two as scales."""
    rows, cols = u.shape
    x = torch.nn.functional.pad(u.float(), (0, -cols % group)).reshape(rows, -1, group)
    bits = x.abs().amax(2, keepdim=True).view(torch.int32)   # the smallest 2^e with amax <= most * 2^e
    lead, most = (6, 127 / 64) if form == "int8" else (8, 448 / 256)
    above = (bits & 0x7FFFFF) > int((most - 1) * (1 << 23))
    e = ((bits >> 23) - 127 - lead + above).clamp(min=-126)
    x = x * _pow2(-e)
    x = torch.round(x) if form == "int8" else x.to(torch.float8_e4m3fn).float()
    return (x * _pow2(e)).reshape(rows, -1)[:, :cols]


def _plain_ckpt(s, c):
    u, dt, width = s["u"], s["u"].dtype, c["width"]
    if c["kind"] == "copy":
        return _checkpoint(u, c["group"], c["format"]).to(dt)
    dh, w = s["dh"].float(), s["w"][:, None]
    if c["act"] == "gelu":
        x = u.float()
        h = 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
        x = _checkpoint(u, c["group"], c["format"])
        phi = 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
        again = x * phi
        du = dh * w * (phi + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi)))
    else:
        x, y = u[:, :width].float(), u[:, width:].float()
        h = x / (1 + torch.exp(-x)) * y
        x = _checkpoint(u[:, :width], c["group"], c["format"])
        y = _checkpoint(u[:, width:], c["group"], c["format"])
        sg = 1 / (1 + torch.exp(-x))
        again = x * sg * y
        du = torch.cat([dh * w * y * sg * (1 + x * (1 - sg)), dh * w * x * sg], 1)
    return {"h": h.to(dt), "du": du.to(dt), "hw": (w * again).to(dt), "dw": (dh * again).sum(1)}


def _dequantised(codes, scales, c):
    """Weights [.., n, k] in 32 bits from codes [.., n, k/2] (low nibble first) and group scales."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)
    if c["format"] == "int4":
        v, sc = (q - 8).float(), scales.float()
    else:
        v = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device="cuda")[q]
        sc = _pow2(scales.to(torch.int32) - 127)
    return v * sc.repeat_interleave(c["group"], -1, output_size=sc.shape[-1] * c["group"])[..., :c["k"]]


def _plain_q4(s, c):
    pairs = c["tokens"] * c["topk"]
    x = s["x"].float().repeat_interleave(c["topk"], 0, output_size=pairs)
    e = s["expert"].long()
    if pairs <= c["experts"]:   # each pair's own expert
        y = torch.bmm(_dequantised(s["codes"][e], s["scales"][e], c), x[:, :, None])[:, :, 0]
    else:                       # every expert's weights once, against every row
        y = torch.matmul(x, _dequantised(s["codes"], s["scales"], c).transpose(1, 2))[e, torch.arange(pairs, device="cuda")]
    if c["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "swiglu":
        gate, up = y.chunk(2, 1)
        y = gate / (1 + torch.exp(-gate)) * up
    if s["gate"] is not None:
        y = y * s["gate"][:, None]
    return y.to(s["y"].dtype)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gmm":
        out = torch.zeros(s["c"].shape, dtype=torch.float64, device="cuda")
        r0 = 0
        for g, m in enumerate(s["counts"]):
            if m:
                a = s["a"][r0:r0 + m].double()
                if c["kind"] == "tn":
                    out[g] = a.t() @ s["b"][r0:r0 + m].double()
                elif c["kind"] == "nt":
                    out[r0:r0 + m] = a @ s["b"][g].double().t()
                else:
                    out[r0:r0 + m] = a @ s["b"][g].double()
            r0 += m
        return out
    if c["op"] == "ckpt":
        return _exact_ckpt(s, c)
    lut = torch.tensor([i - 8.0 for i in range(16)] if c["format"] == "int4"
                       else [(-1.0) ** (i >> 3) * _E2M1[i & 7] for i in range(16)], dtype=torch.float64, device="cuda")
    y = torch.empty(c["tokens"] * c["topk"], c["n"], dtype=torch.float64, device="cuda")
    at = torch.arange(c["k"], device="cuda")
    experts = s["expert"].tolist()
    for e in sorted(set(experts)):
        q = (s["codes"][e][:, at // 2] >> (4 * (at % 2)).to(torch.uint8)) & 15
        sc = s["scales"][e].double() if c["format"] == "int4" else 2.0 ** (s["scales"][e].double() - 127)
        wt = lut[q.long()] * sc[:, at // c["group"]]
        mine = [p for p, v in enumerate(experts) if v == e]
        tok = torch.tensor(mine, device="cuda") // c["topk"]
        y[torch.tensor(mine, device="cuda")] = s["x"][tok].double() @ wt.t()
    if c["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    elif c["act"] == "swiglu":
        y = torch.nn.functional.silu(y[:, :c["n"] // 2]) * y[:, c["n"] // 2:]
    return y if s["gate"] is None else y * s["gate"].double()[:, None]


def _exact_saved(u, c):
    """Each group of values on its own grid: whole multiples of 2^e with at most 127 of them, or
    three bits behind the leading one, at 2^e from 448 downwards."""
    v, out = u.double(), torch.empty(u.shape, dtype=torch.float64, device="cuda")
    for lo in range(0, u.shape[1], c["group"]):
        part = v[:, lo:lo + c["group"]]
        m, ex = torch.frexp(part.abs().amax(1, keepdim=True) / (127.0 if c["format"] == "int8" else 448.0))
        e = torch.where(m > 0.5, ex, ex - 1).clamp(min=-126)
        step = ((e.long() + 1023) << 52).view(torch.float64)   # 2^e, exactly
        if c["format"] == "e4m3":
            lead = torch.frexp(part / step)[1] - 1          # exponent of the leading bit
            step = ((e + lead.clamp(min=-6) - 3 + 1023).long() << 52).view(torch.float64)
        out[:, lo:lo + c["group"]] = torch.round(part / step) * step
    return out


def _exact_ckpt(s, c):
    if c["kind"] == "copy":
        return _exact_saved(s["u"], c)
    if s["u"].numel() > 300e6:
        return None
    width, dh, w = c["width"], s["dh"].double(), s["w"].double()[:, None]
    if c["act"] == "gelu":
        v = s["u"].double()
        h = v * torch.special.ndtr(v)
        v = _exact_saved(s["u"], c).requires_grad_()
        again = v * torch.special.ndtr(v)
    else:
        h = torch.nn.functional.silu(s["u"][:, :width].double()) * s["u"][:, width:].double()
        v = torch.cat([_exact_saved(s["u"][:, :width], c), _exact_saved(s["u"][:, width:], c)], 1).requires_grad_()
        again = torch.nn.functional.silu(v[:, :width]) * v[:, width:]
    du, = torch.autograd.grad(again, v, w * dh)
    again = again.detach()
    return {"h": h, "du": du, "hw": w * again, "dw": (dh * again).sum(1)}
