"""Timed cases of the training operators: the norm's two passes, the 8-bit
activation checkpoints, a linear layer's weight gradient from them, and the
gated feed-forward block's two passes.

``run`` computes a case in plain torch operations (fp32) or, where ``own`` is
true, through the library's entry points.  The widths are those of the
workloads in ``workloads/``: 512/2048 (layout500), 1024/4096 (mixed50m) and
4096/12288 (kda_block).
"""
import math

import torch

own = False

GROUP = 32                       # columns that share a checkpoint's scale
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
SIZE = {"bf16": 2, "fp32": 4, "e4m3": 1 + 1 / GROUP, "int8": 1 + 1 / GROUP}
EPS = 1e-5


def listed():
    return [
        # one token's norm between two layers of a decode step: latency
        norm("layernorm_one_row", "fwd", "ln", 1, 1024, x="fp32", out="bf16"),
        # the norm before a KDA-style block's projections, keeping its input
        # and its output (the projections' input) in 8 bits
        norm("rmsnorm_kda_saved", "fwd", "rms", 16384, 4096, x="bf16", out="bf16", saved="e4m3"),
        # its backward pass, reading the 8-bit input
        norm("rmsnorm_kda_backward", "bwd", "rms", 16384, 4096, x="e4m3", out="bf16"),
        # a ragged micro-batch at a width that no vector divides, with bias gradients
        norm("layernorm_odd_backward", "bwd", "ln", 4099, 1001, x="bf16", out="bf16"),
        # the hidden activation of a KDA-style block put away in 8 bits
        dict(name="save_ffn_activation", op="save", rows=8192, cols=12288, x="bf16", saved="e4m3"),
        # a small odd activation read back
        dict(name="load_odd_activation", op="load", rows=333, cols=1000, x="bf16", saved="int8"),
        # a square projection's weight gradient in bf16 from its 8-bit input
        dict(name="weight_grad_kda_projection", op="wgrad", rows=8192, outs=4096, cols=4096, x="e4m3", dw="bf16"),
        # an up projection's weight gradient in fp32 (the reduction dtype), ragged tokens
        dict(name="weight_grad_layout500_up", op="wgrad", rows=2055, outs=2048, cols=512, x="int8", dw="fp32"),
        # one token through the gated block (sampling during training): bound by the weights
        gated("gated_one_token", "gfwd", 1, 1024, 4096, x="bf16", saved="none", act="silu"),
        # a training step's forward pass of a KDA-style block, projections kept in 8 bits
        gated("gated_kda_saved", "gfwd", 8192, 4096, 12288, x="bf16", saved="e4m3", act="silu"),
        # its backward pass from the 8-bit input and projections
        gated("gated_kda_backward", "gbwd", 4096, 4096, 12288, x="e4m3", saved="e4m3", act="silu"),
        # a narrow block's backward pass over a ragged micro-batch, nothing in 8 bits
        gated("gated_layout500_backward", "gbwd", 4099, 512, 2048, x="bf16", saved="bf16", act="gelu"),
    ]


def norm(name, way, kind, rows, cols, x, out, saved="none"):
    return dict(name=name, op="norm_" + way, kind=kind, rows=rows, cols=cols, x=x, out=out, saved=saved)


def gated(name, op, rows, cols, ffn, x, saved, act):
    return dict(name=name, op=op, rows=rows, cols=cols, ffn=ffn, x=x, saved=saved, act=act)


def draw(rng):
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        # half of the sizes as drawn (odd ones among them), half multiples of 64
        return n if rng.random() < 0.5 or n < 64 else n // 64 * 64

    op = rng.choice(["norm_fwd", "norm_bwd", "save", "load", "wgrad", "gfwd", "gbwd"])
    eight = rng.choice(["e4m3", "int8"])
    if op in ("norm_fwd", "norm_bwd"):
        c = norm("", op[5:], rng.choice(["ln", "rms"]), size(1, 16384), size(64, 4096), "bf16", rng.choice(["bf16", "fp32"]))
        c["x"] = rng.choice(["bf16", "fp32"] + ([eight] if op == "norm_bwd" else []))
        if op == "norm_fwd":
            c["saved"] = rng.choice(["none", eight])
    elif op in ("save", "load"):
        c = dict(op=op, rows=size(16, 8192), cols=size(64, 12288), x=rng.choice(["bf16", "fp32"]), saved=eight)
    elif op == "wgrad":
        c = dict(op=op, rows=size(64, 8192), outs=size(64, 4096), cols=size(64, 4096), x=eight, dw=rng.choice(["bf16", "fp32"]))
    else:
        c = gated("", op, size(1, 4096), size(64, 4096), size(64, 12288), "bf16", rng.choice(["bf16", eight]), rng.choice(["silu", "gelu"]))
        c["x"] = rng.choice(["bf16", eight]) if op == "gbwd" else "bf16"
        if op == "gfwd":
            c["saved"] = rng.choice(["none", c["saved"]])
    c.pop("name", None)
    return c


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype="bf16"):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(TYPES[dtype])

    def activation(rows, cols, kind, std=1.0):
        """An activation, dense or put away in 8 bits: a few columns larger than the rest, as in trained models."""
        x = torch.randn(rows, cols, generator=gen, device="cuda") * std
        x *= 1 + 15 * (torch.rand(cols, generator=gen, device="cuda") < 0.01)
        return x.to(TYPES[kind]) if kind in ("bf16", "fp32") else quantise(x.bfloat16().float(), kind)

    def empty(*shape, dtype="bf16"):
        return torch.empty(*shape, device="cuda", dtype=TYPES[dtype])

    op, s, rows, cols = case["op"], {"case": case}, case["rows"], case["cols"]
    if op.startswith("norm"):
        s["x"] = activation(rows, cols, case["x"])
        s["weight"] = 1 + normal(cols, std=0.2, dtype="fp32")
        s["bias"] = normal(cols, std=0.2, dtype="fp32") if case["kind"] == "ln" else None
        if op == "norm_fwd":
            s["out"] = empty(rows, cols, dtype=case["out"])
            s["stats"] = empty(rows, 2, dtype="fp32")
            s["saved"] = [empty_checkpoint(rows, cols, case["saved"]) for _ in range(2)] if case["saved"] != "none" else [None, None]
            s["back"] = [empty(rows, cols) for _ in range(2)] if case["saved"] != "none" else [None, None]
        else:
            x = dense(s["x"])
            mean = x.mean(1) if case["kind"] == "ln" else torch.zeros(rows, device="cuda")
            s["stats"] = torch.stack([mean, 1 / ((x - mean[:, None]).square().mean(1) + EPS).sqrt()], 1).contiguous()
            s["dout"] = normal(rows, cols, std=0.01, dtype=case["out"])
            s["dx"] = empty(rows, cols, dtype=case["out"])
            s["dweight"] = empty(cols, dtype="fp32")
            s["dbias"] = empty(cols, dtype="fp32") if case["kind"] == "ln" else None
    elif op == "save":
        s["x"] = activation(rows, cols, case["x"])
        s["saved"] = empty_checkpoint(rows, cols, case["saved"])
    elif op == "load":
        s["x"] = activation(rows, cols, case["saved"])
        s["out"] = empty(rows, cols, dtype=case["x"])
    elif op == "wgrad":
        s["x"] = activation(rows, cols, case["x"])
        s["dout"] = normal(rows, case["outs"], std=0.01)
        s["dw"] = empty(case["outs"], cols, dtype=case["dw"])
    else:
        ffn = case["ffn"]
        s["x"] = activation(rows, cols, case["x"], std=0.5)
        s["w_gate"] = normal(ffn, cols, std=1 / math.sqrt(cols))
        s["w_up"] = normal(ffn, cols, std=1 / math.sqrt(cols))
        if op == "gfwd":
            s["out"] = empty(rows, ffn)
            make = {"none": lambda: None, "bf16": lambda: empty(rows, ffn)}.get(case["saved"], lambda: empty_checkpoint(rows, ffn, case["saved"]))
            s["gate"], s["up"] = make(), make()
            s["back"] = [empty(rows, ffn) for _ in range(2)] if case["saved"] in ("e4m3", "int8") else [None, None]
        else:
            s["gate"] = activation(rows, ffn, case["saved"])
            s["up"] = activation(rows, ffn, case["saved"])
            s["dout"] = normal(rows, ffn, std=0.01)
            s["dx"] = empty(rows, cols)
            s["dw_gate"], s["dw_up"] = empty(ffn, cols), empty(ffn, cols)
    return s


def empty_checkpoint(rows, cols, kind):
    return (torch.empty(rows, cols, device="cuda", dtype=TYPES[kind]),
            torch.empty(rows, -(-cols // GROUP), device="cuda", dtype=torch.uint8))


# ------------------------------------------------------------------ one pass

def run(s):
    return (calls if own else plain)(s)


def calls(s):
    """The library's entry points, as a training program calls them."""
    import fsdp2_mixed_dtype_amd as fp

    c = s["case"]
    op = c["op"]

    def arg(v):
        return fp.Checkpoint(*v) if isinstance(v, tuple) else v

    def workspace(nbytes):
        if "workspace" not in s:
            s["workspace"] = torch.empty(nbytes(), device="cuda", dtype=torch.uint8)
        return s["workspace"]

    if op == "norm_fwd":
        kind = fp.LAYER_NORM if c["kind"] == "ln" else fp.RMS_NORM
        kept = [arg(v) for v in s["saved"]]
        fp.norm_forward(s["x"], s["weight"], s["out"], s["stats"], bias=s["bias"], kind=kind, eps=EPS,
                        x_checkpoint=kept[0], out_checkpoint=kept[1])
        for k, b in zip(kept, s["back"]):
            if k is not None:
                fp.checkpoint_load(k, b)
        return {"out": s["out"], "stats": s["stats"], "saved": s["back"]}
    if op == "norm_bwd":
        kind = fp.LAYER_NORM if c["kind"] == "ln" else fp.RMS_NORM
        ws = workspace(lambda: fp.norm_backward_workspace(c["rows"], c["cols"]))
        fp.norm_backward(s["dout"], arg(s["x"]), s["weight"], s["stats"], s["dx"], s["dweight"], ws, dbias=s["dbias"], kind=kind)
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if op == "save":
        fp.checkpoint_save(s["x"], arg(s["saved"]))
        return {"values": s["saved"][0], "scales": s["saved"][1]}
    if op == "load":
        fp.checkpoint_load(arg(s["x"]), s["out"])
        return s["out"]
    if op == "wgrad":
        ws = workspace(lambda: fp.weight_grad_workspace(c["rows"], c["outs"], c["cols"]))
        fp.weight_grad(s["dout"], arg(s["x"]), s["dw"], ws)
        return s["dw"]
    act = fp.SILU if c["act"] == "silu" else fp.GELU_TANH
    if op == "gfwd":
        gate, up = arg(s["gate"]), arg(s["up"])
        fp.gated_forward(s["x"], s["w_gate"], s["w_up"], s["out"], gate=gate, up=up, activation=act)
        for k, b in zip((gate, up), s["back"]):
            if b is not None:
                fp.checkpoint_load(k, b)
        back = s["back"] if s["back"][0] is not None else [s["gate"], s["up"]]
        return {"out": s["out"], "gate": back[0], "up": back[1]}
    ws = workspace(lambda: fp.gated_backward_workspace(c["rows"], c["ffn"], c["cols"]))
    fp.gated_backward(s["dout"], arg(s["x"]), s["w_gate"], s["w_up"], arg(s["gate"]), arg(s["up"]), s["dx"], s["dw_gate"],
                      s["dw_up"], ws, activation=act)
    return {"dx": s["dx"], "dw_gate": s["dw_gate"], "dw_up": s["dw_up"]}


def plain(s):
    """The same in elementary torch operations: 32 bits throughout, rounded once at the end."""
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True) if c["kind"] == "ln" else torch.zeros_like(x[:, :1])
        rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + EPS).sqrt()
        y = (x - mean) * rstd * s["weight"]
        if s["bias"] is not None:
            y = y + s["bias"]
        kept = [None, None]
        if c["saved"] != "none":
            kept = [dense(quantise(x, c["saved"])).bfloat16(), dense(quantise(y, c["saved"])).bfloat16()]
        return {"out": y.to(TYPES[c["out"]]), "stats": torch.cat([mean, rstd], 1), "saved": kept}
    if op == "norm_bwd":
        x, dy = dense(s["x"]), s["dout"].float()
        mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
        xh, wdy = (x - mean) * rstd, dy * s["weight"]
        dx = wdy - xh * (wdy * xh).mean(1, keepdim=True)
        if c["kind"] == "ln":
            dx = dx - wdy.mean(1, keepdim=True)
        return {"dx": (dx * rstd).to(TYPES[c["out"]]), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0) if c["kind"] == "ln" else None}
    if op == "save":
        values, scales = quantise(s["x"].float(), c["saved"])
        return {"values": values, "scales": scales}
    if op == "load":
        return dense(s["x"]).to(TYPES[c["x"]])
    if op == "wgrad":
        return (s["dout"].float().t() @ dense(s["x"])).to(TYPES[c["dw"]])
    if op == "gfwd":
        x = s["x"].float()
        g, u = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
        kept = [None, None]
        if c["saved"] == "bf16":
            kept = [g.bfloat16(), u.bfloat16()]
        elif c["saved"] != "none":
            kept = [dense(quantise(g, c["saved"])).bfloat16(), dense(quantise(u, c["saved"])).bfloat16()]
        return {"out": (activation_of(c["act"], g)[0] * u).bfloat16(), "gate": kept[0], "up": kept[1]}
    x, g, u, dh = dense(s["x"]), dense(s["gate"]), dense(s["up"]), s["dout"].float()
    a, da = activation_of(c["act"], g)
    dg, du = dh * u * da, dh * a
    dx = dg @ s["w_gate"].float() + du @ s["w_up"].float()
    return {"dx": dx.bfloat16(), "dw_gate": (dg.t() @ x).bfloat16(), "dw_up": (du.t() @ x).bfloat16()}


def activation_of(act, g):
    """The activation and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def quantise(x, kind):
    """fp32 [rows, cols] -> (8-bit values, scale bytes): the smallest power of
    two that brings each group of 32 columns within the format's range."""
    rows, cols = x.shape
    groups = torch.nn.functional.pad(x, (0, -cols % GROUP)).view(rows, -1, GROUP)
    top = groups.abs().amax(2)
    m, k = torch.frexp(top)                      # top = m * 2^k, m in [0.5, 1)
    limit, bits = (0.875, 9) if kind == "e4m3" else (127 / 128, 7)
    e = torch.where(top > 0, k - bits + (m > limit), -110).clamp(min=-110)
    q = groups * power_of_two(-e).unsqueeze(2)
    q = (q.to(torch.float8_e4m3fn) if kind == "e4m3" else q.round().to(torch.int8)).view(rows, -1)
    return q[:, :cols].contiguous(), (e + 127).to(torch.uint8)


def power_of_two(e):
    return ((e.int() + 127) << 23).view(torch.float32)


def dense(x):
    """An activation's values in fp32."""
    if not isinstance(x, tuple):
        return x.float()
    values, scales = x
    scale = (scales.int() << 23).view(torch.float32)
    return values.float() * scale.repeat_interleave(GROUP, 1)[:, :values.shape[1]]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, n = case, case["rows"] * case["cols"]
    op, rows, cols = c["op"], c["rows"], c["cols"]
    if op == "norm_fwd":
        kept = 2 * n * (SIZE[c["saved"]] + SIZE[c["saved"]] + 2) if c["saved"] != "none" else 0   # written, read back, values written
        return {"bytes": n * (SIZE[c["x"]] + SIZE[c["out"]]) + 8 * rows + 8 * cols + kept, "flops": 8 * n}
    if op == "norm_bwd":
        return {"bytes": n * (SIZE[c["x"]] + 2 * SIZE[c["out"]]) + 8 * rows + 12 * cols, "flops": 12 * n}
    if op in ("save", "load"):
        return {"bytes": n * (SIZE[c["x"]] + SIZE[c["saved"]]), "flops": 2 * n}
    if op == "wgrad":
        return {"bytes": n * SIZE[c["x"]] + 2 * rows * c["outs"] + c["outs"] * cols * SIZE[c["dw"]], "flops": 2 * n * c["outs"]}
    hidden, weights = rows * c["ffn"], c["ffn"] * cols
    if op == "gfwd":
        kept = {"none": 0, "bf16": 4}.get(c["saved"], 2 * (2 * SIZE["e4m3"] + 2))
        return {"bytes": 2 * n + 4 * weights + hidden * (2 + kept), "flops": 4 * n * c["ffn"]}
    return {"bytes": n * (SIZE[c["x"]] + 2) + 8 * weights + hidden * (2 + 2 * SIZE[c["saved"]]), "flops": 8 * n * c["ffn"]}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "save":
        codes, exponents = codes64(s["x"].double(), case["saved"])
        return {"values": codes, "scales": exponents + 127} if case["saved"] == "e4m3" else {"values": None, "scales": None}
    x = values64(s["x"])
    if op == "load":
        return x
    if op == "norm_fwd":
        centre = x.mean(dim=1) if case["kind"] == "ln" else x.new_zeros(len(x))
        spread = torch.rsqrt(((x - centre[:, None]) ** 2).sum(dim=1) / x.shape[1] + EPS)
        y = torch.einsum("rc,r,c->rc", x - centre[:, None], spread, s["weight"].double())
        if s["bias"] is not None:
            y += s["bias"].double()
        kept = [None, None]
        if case["saved"] != "none":
            kept = [rounded64(v, case["saved"]) for v in (x, y)]
        return {"out": y, "stats": torch.stack((centre, spread), dim=1), "saved": kept}
    dy = s.get("dout")
    dy = dy.double() if dy is not None else None
    if op == "norm_bwd":
        stats = s["stats"].double()
        unit = (x - stats[:, 0, None]) * stats[:, 1, None]
        dunit = dy * s["weight"].double()
        # the derivative of unit = (x - mean) * rstd through mean and rstd
        dx = dunit - (dunit.mean(dim=1, keepdim=True) if case["kind"] == "ln" else 0)
        dx = (dx - unit * ((dunit * unit).sum(dim=1, keepdim=True) / x.shape[1])) * stats[:, 1, None]
        return {"dx": dx, "dweight": torch.sum(dy * unit, dim=0), "dbias": dy.sum(dim=0) if case["kind"] == "ln" else None}
    if op == "wgrad":
        return torch.mm(dy.t().contiguous(), x)
    wg, wu = s["w_gate"].double(), s["w_up"].double()
    if op == "gfwd":
        g, u = torch.mm(x, wg.t().contiguous()), torch.mm(x, wu.t().contiguous())
        kept = [None, None]
        if case["saved"] != "none":
            kept = [g, u] if case["saved"] == "bf16" else [rounded64(v, case["saved"]) for v in (g, u)]
        return {"out": activation64(case["act"], g)[0] * u, "gate": kept[0], "up": kept[1]}
    a, slope = activation64(case["act"], values64(s["gate"]))
    dg, du = dy * values64(s["up"]) * slope, dy * a
    dx = torch.mm(dg, wg)
    dx += torch.mm(du, wu)
    return {"dx": dx, "dw_gate": torch.mm(dg.t().contiguous(), x), "dw_up": torch.mm(du.t().contiguous(), x)}


def activation64(act, g):
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    slope = math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)
    p = torch.sigmoid(2 * inner)                 # (1 + tanh(v)) / 2 = sigmoid(2 v)
    return g * p, p + g * 2 * p * (1 - p) * slope


def values64(x):
    if not isinstance(x, tuple):
        return x.double()
    each = torch.arange(x[0].shape[1], device="cuda") // GROUP
    return torch.ldexp(x[0].double(), x[1].double()[:, each] - 127)


def codes64(x, kind):
    """The 8-bit numbers and scale exponents of 64-bit values."""
    rows, cols = x.shape
    each = torch.arange(cols, device="cuda") // GROUP
    top = x.new_zeros(rows, -(-cols // GROUP)).scatter_reduce(1, each.expand(rows, cols), x.abs(), "amax")
    most = 448.0 if kind == "e4m3" else 127.0
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / most))
    e += (torch.ldexp(top, -e) > most).double()
    e -= (torch.ldexp(top, 1 - e) <= most).double()      # a logarithm's last bit may go either way
    e = e.clamp(min=-110)
    v = torch.ldexp(x, -e[:, each])
    if kind == "int8":
        return v.round(), e.long()
    # e4m3: three bits behind the leading one, none below 2^-9
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (v / step).round() * step, e.long()


def rounded64(x, kind):
    codes, e = codes64(x, kind)
    each = torch.arange(x.shape[1], device="cuda") // GROUP
    return torch.ldexp(codes, e.double()[:, each])
