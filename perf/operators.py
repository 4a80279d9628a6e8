"""Cases that measure the operators of ``include/adam_train.h``: 8-bit
activation checkpoints with the backward steps that read them, and softmax
cross entropy over a large vocabulary with its gradient.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end), or, where ``own`` is true, through the
package's entry points.  Widths are those of the 30B-class shard in
``workloads.py`` (hidden 4096, key/value 1024, feed-forward 14336, vocabulary
131072), and generic odd ones beside them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MAX8 = {"e4m3": 448.0, "e5m2": 57344.0}
TYPE8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
IGNORE = -100


def listed():
    return [
        # The input of the feed-forward block's second projection, one micro-batch: the largest activation kept.
        dict(name="act8_ffn_bf16", op="act8", rows=8192, cols=14336, pad=0, type="bf16", fmt="e4m3"),
        # A float activation that is a view of wider rows, neither of its sizes even.
        dict(name="act8_ragged_f32", op="act8", rows=1537, cols=4099, pad=29, type="f32", fmt="e5m2"),
        # The gated activation of one micro-batch, forward with checkpoints and backward from them.
        dict(name="glu_step_bf16", op="glu", rows=8192, cols=14336, type="bf16", fmt="e4m3", act="silu"),
        # A short ragged batch, width not a multiple of the scale block.
        dict(name="glu_step_odd_f16", op="glu", rows=333, cols=5003, type="f16", fmt="e4m3", act="gelu"),
        # A three-token batch: latency.
        dict(name="glu_step_tiny_bf16", op="glu", rows=3, cols=1000, type="bf16", fmt="e4m3", act="silu"),
        # Weight gradient of the second feed-forward projection into a float gradient buffer.
        dict(name="wgrad_ffn_bf16", op="wgrad", rows=8192, n=4096, k=14336, type="bf16", out="f32", fmt="e4m3"),
        # Weight gradient of a key/value projection: few output tiles over many tokens.
        dict(name="wgrad_kv_bf16", op="wgrad", rows=8192, n=1024, k=4096, type="bf16", out="bf16", fmt="e4m3"),
        # A ragged packed batch with odd widths in fp16.
        dict(name="wgrad_odd_f16", op="wgrad", rows=777, n=1003, k=2051, type="f16", out="f32", fmt="e5m2"),
        # Scoring one token: the weight is read once.
        dict(name="xent_one_token", op="xent", rows=1, hidden=4096, vocab=131072, type="bf16", grad=False, ignored=0.0),
        # Evaluation of a batch of tokens.
        dict(name="xent_eval_bf16", op="xent", rows=2048, hidden=4096, vocab=131072, type="bf16", grad=False, ignored=0.0),
        # The training step's loss and both gradients, a tenth of the rows padding.
        dict(name="xent_train_bf16", op="xent", rows=8192, hidden=4096, vocab=131072, type="bf16", grad=True, ignored=0.1),
        # The same at an odd token count and vocabulary, in fp16.
        dict(name="xent_train_odd_f16", op="xent", rows=1003, hidden=1000, vocab=50021, type="f16", grad=True, ignored=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["act8", "glu", "wgrad", "xent", "xent"])
    half = rng.choice(["bf16", "bf16", "f16"])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op == "act8":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 7, 14336), pad=rng.choice([0, 0, 1, 8, 61]),
                    type=rng.choice(["bf16", "f16", "f32"]), fmt=fmt)
    if op == "glu":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 7, 14336), type=rng.choice(["bf16", "f16", "f32"]),
                    fmt=fmt, act=rng.choice(["silu", "gelu"]))
    if op == "wgrad":
        return dict(op=op, rows=_log(rng, 1, 8192), n=_log(rng, 5, 4096), k=_log(rng, 33, 14336), type=half,
                    out=rng.choice(["f32", half]), fmt=fmt)
    return dict(op=op, rows=_log(rng, 1, 8192), hidden=rng.choice([4096, 1024, 2048, 8 * rng.randint(8, 512), rng.randint(64, 4096)]),
                vocab=_log(rng, 513, 131072), type=half, grad=rng.random() < 0.7, ignored=rng.choice([0.0, 0.1, 0.5]))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _activation(gen, rows, cols):
    """Activations: normal values whose columns differ in size, as trained ones do."""
    return _randn(gen, rows, cols) * torch.exp(0.7 * _randn(gen, 1, cols))


def _pad32(n):
    return (n + 31) // 32 * 32


def _checkpoint(x, fmt):
    """The checkpoint buffer that holds x (layout as adam_train.h states)."""
    rows, cols = x.shape
    pitch = _pad32(cols)
    wide = torch.zeros(rows, pitch, device=x.device)
    wide[:, :cols] = x
    blocks = wide.view(rows, pitch // 32, 32)
    e = _exponent(blocks.abs().amax(2), fmt)
    codes = torch.ldexp(blocks, -e[:, :, None]).to(TYPE8[fmt]).view(torch.uint8).view(rows, pitch)
    at = (rows * pitch + 255) // 256 * 256
    buf = torch.zeros(at + rows * (pitch // 32), dtype=torch.uint8, device=x.device)
    buf[: rows * pitch] = codes.reshape(-1)
    buf[at:] = (e + 127).to(torch.uint8).reshape(-1)
    return buf


def _exponent(amax, fmt):
    """The smallest e >= -127 with amax <= MAX * 2^e: amax = f 2^k with f in [0.5, 1) and MAX = g 2^j alike, so e is k - j,
    and one more where f > g."""
    f, k = torch.frexp(amax)
    g, j = math.frexp(MAX8[fmt])
    e = k - j + (f > g).to(k.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(min=-127)


def _values(buf, rows, cols, fmt):
    """The values a checkpoint buffer stands for, in 32 bits."""
    pitch = _pad32(cols)
    at = (rows * pitch + 255) // 256 * 256
    codes = buf[: rows * pitch].view(TYPE8[fmt]).view(rows, pitch // 32, 32).float()
    e = buf[at: at + rows * (pitch // 32)].view(rows, pitch // 32).to(torch.int32) - 127
    return torch.ldexp(codes, e[:, :, None]).view(rows, pitch)[:, :cols]


def prepare(case, seed):
    gen = _gen(seed)
    op, dt = case["op"], DTYPES[case["type"]]
    rows = case["rows"]
    s = dict(case=case)
    if op == "act8":
        cols = case["cols"]
        s["x"] = _activation(gen, rows, cols + case["pad"]).to(dt)[:, :cols]
        s["ckpt"] = torch.empty((rows * _pad32(cols) + 255) // 256 * 256 + rows * _pad32(cols) // 32, dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty(rows, cols, dtype=dt, device="cuda")
    elif op == "glu":
        cols = case["cols"]
        s["x"] = _activation(gen, rows, 2 * cols).to(dt)  # gate and up: the two halves of one projection's output
        s["dh"] = (1e-2 * _randn(gen, rows, cols)).to(dt)
        n8 = (rows * _pad32(cols) + 255) // 256 * 256 + rows * _pad32(cols) // 32
        s["ckpt"] = [torch.empty(n8, dtype=torch.uint8, device="cuda") for _ in range(2)]
        s["h"], s["again"] = (torch.empty(rows, cols, dtype=dt, device="cuda") for _ in range(2))
        s["dx"] = torch.empty(rows, 2 * cols, dtype=dt, device="cuda")
    elif op == "wgrad":
        s["ckpt"] = _checkpoint(_activation(gen, rows, case["k"]), case["fmt"])
        s["dy"] = (1e-2 * _randn(gen, rows, case["n"])).to(dt)
        s["dw"] = torch.empty(case["n"], case["k"], dtype=DTYPES[case["out"]], device="cuda")
    else:
        hidden, vocab = case["hidden"], case["vocab"]
        s["h"] = _randn(gen, rows, hidden).to(dt)
        s["w"] = (_randn(gen, vocab, hidden) * (2.5 / math.sqrt(hidden))).to(dt)
        target = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
        skip = torch.rand(rows, device="cuda", generator=gen) < case["ignored"]
        skip[0] = False  # a batch of padding alone has nothing to compute
        s["target"] = torch.where(skip, IGNORE, target)
        # a loss scale of 2^10 over the mean's count: what a mixed-precision step multiplies its loss by
        s["scale"] = 1024.0 / (s["target"] != IGNORE).sum().clamp(min=1).float().reshape(1)
        s["loss"], s["lse"] = (torch.empty(rows, device="cuda") for _ in range(2))
        if case["grad"]:
            s["dh"], s["dw"] = torch.empty_like(s["h"]), torch.empty_like(s["w"])
    return s


def _act(g, act):
    """a(g) and a'(g)."""
    if act == "silu":
        t = 1 / (1 + torch.exp(-g))
        return g * t, t * (1 + g * (1 - t))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _through8(x, fmt):
    rows, cols = x.shape
    return _values(_checkpoint(x, fmt), rows, cols, fmt)


def _plain(s, case):
    op = case["op"]
    if op == "act8":
        return _through8(s["x"].float(), case["fmt"]).to(s["x"].dtype)
    if op == "glu":
        dt = s["x"].dtype
        gate, up = s["x"].float().chunk(2, dim=1)
        h = (_act(gate, case["act"])[0] * up).to(dt)
        g, u, dh = _through8(gate, case["fmt"]), _through8(up, case["fmt"]), s["dh"].float()
        a, d = _act(g, case["act"])
        return h, torch.cat([dh * u * d, dh * a], dim=1).to(dt), (a * u).to(dt)
    if op == "wgrad":
        x = _values(s["ckpt"], case["rows"], case["k"], case["fmt"])
        return (s["dy"].float().t() @ x).to(s["dw"].dtype)
    h, w, target = s["h"].float(), s["w"].float(), s["target"]
    valid = target != IGNORE
    z = h @ w.t()
    top = z.amax(1, keepdim=True)
    lse = top.squeeze(1) + torch.log(torch.exp(z - top).sum(1))
    at = target.clamp(min=0)[:, None]
    loss = torch.where(valid, lse - z.gather(1, at).squeeze(1), 0.0)
    kept = torch.where(valid, lse, 0.0)
    if not case["grad"]:
        return loss, kept
    g = torch.exp(z.sub_(lse[:, None]))
    g.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
    g *= valid[:, None] * s["scale"]
    return loss, kept, (g @ w).to(s["h"].dtype), (g.t() @ h).to(s["w"].dtype)


def _own(s, case):
    import adamw_optimizer_step_tensor_amd as A

    op = case["op"]
    if op == "act8":
        A.adam_act8_store(s["x"], s["ckpt"], case["fmt"])
        A.adam_act8_load(s["ckpt"], s["out"], case["fmt"])
        return s["out"]
    if op == "glu":
        c = case["cols"]
        gate, up, dx = s["x"][:, :c], s["x"][:, c:], s["dx"]
        A.adam_glu_forward(gate, up, s["h"], case["act"], *s["ckpt"], fmt=case["fmt"])
        A.adam_glu_backward(s["dh"], *s["ckpt"], dx[:, :c], dx[:, c:], case["act"], h=s["again"], fmt=case["fmt"])
        return s["h"], dx, s["again"]
    if op == "wgrad":
        A.adam_act8_wgrad(s["dy"], s["ckpt"], s["dw"], case["fmt"])
        return s["dw"]
    if not case["grad"]:
        A.adam_xent(s["h"], s["w"], s["target"], s["loss"], lse=s["lse"], ignore_index=IGNORE)
        return s["loss"], s["lse"]
    A.adam_xent(s["h"], s["w"], s["target"], s["loss"], lse=s["lse"], dh=s["dh"], dw=s["dw"], d_loss_scale=s["scale"],
                ignore_index=IGNORE)
    return s["loss"], s["lse"], s["dh"], s["dw"]


def run(state):
    if own:
        return _own(state, state["case"])
    return _plain(state, state["case"])


def work(case):
    op, t = case["op"], case["rows"]
    b = SIZE[case["type"]]
    if op == "act8":  # x in, the checkpoint out; the checkpoint in, x out
        n = t * case["cols"]
        return {"bytes": 2 * n * b + 2 * n * 33 // 32, "flops": 4 * n}
    if op == "glu":  # gate and up in, h and two checkpoints out; dh and the checkpoints in, two gradients and h out
        n = t * case["cols"]
        return {"bytes": 7 * n * b + 4 * n * 33 // 32, "flops": 60 * n}
    if op == "wgrad":
        n, k = case["n"], case["k"]
        return {"bytes": t * n * b + t * k * 33 // 32 + n * k * SIZE[case["out"]], "flops": 2 * t * n * k}
    d, v = case["hidden"], case["vocab"]
    kept = t - int(t * case["ignored"])  # rows that are not padding
    if case["grad"]:  # h and w in, dh and dw out; the logits' product and one for each gradient
        return {"bytes": 2 * (t + v) * d * b, "flops": 6 * kept * v * d}
    return {"bytes": (t + v) * d * b, "flops": 2 * kept * v * d}


def _round8(x, fmt):
    """Values of the checkpoint of x, in 64 bits from the definition: per block of 32 the scale 2^e, then the nearest
    multiple of the format's spacing, ties to even."""
    rows, cols = x.shape
    bits, least = {"e4m3": (3, -6), "e5m2": (2, -14)}[fmt]
    pieces = torch.nn.functional.pad(x, (0, -cols % 32)).reshape(rows, -1, 32)
    amax = pieces.abs().max(dim=2, keepdim=True).values
    e = torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / MAX8[fmt]))
    e = torch.where(torch.exp2(e) * MAX8[fmt] < amax, e + 1, e)  # the logarithm may round across an integer
    e = torch.where(torch.exp2(e - 1) * MAX8[fmt] >= amax, e - 1, e)
    e = torch.clamp(e, min=-127.0)
    y = pieces / torch.exp2(e)
    spacing = torch.exp2(torch.clamp(torch.frexp(y).exponent.double() - 1, min=float(least)) - bits)
    return (torch.round(y / spacing) * spacing * torch.exp2(e)).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "act8":
        return _round8(s["x"].double(), case["fmt"])
    if op == "glu":
        x = s["x"].double()
        c = case["cols"]

        def gated(g):
            if case["act"] == "silu":
                return g * torch.sigmoid(g)
            return torch.nn.functional.gelu(g, approximate="tanh")

        h = gated(x[:, :c]) * x[:, c:]
        g = _round8(x[:, :c], case["fmt"]).requires_grad_()
        u = _round8(x[:, c:], case["fmt"]).requires_grad_()
        again = gated(g) * u
        dg, du = torch.autograd.grad(again, (g, u), s["dh"].double())
        return h, torch.cat([dg, du], dim=1), again.detach()
    if op == "wgrad":
        t, k = case["rows"], case["k"]
        p = _pad32(k)
        at = (t * p + 255) // 256 * 256
        x = s["ckpt"][: t * p].view(TYPE8[case["fmt"]]).double().view(t, p)
        scale = torch.exp2(s["ckpt"][at: at + t * p // 32].double() - 127).view(t, p // 32)
        x = (x * scale.repeat_interleave(32, dim=1))[:, :k]
        return torch.mm(s["dy"].double().t().contiguous(), x.contiguous())
    h, w = s["h"].double(), s["w"].double()
    keep = (s["target"] != IGNORE).nonzero().squeeze(1)
    hk, tk = h[keep], s["target"][keep]
    z = torch.mm(hk, w.t().contiguous())
    lse = torch.logsumexp(z, 1)
    rows = case["rows"]
    loss, kept = torch.zeros(rows, dtype=torch.float64, device="cuda"), torch.zeros(rows, dtype=torch.float64, device="cuda")
    loss[keep] = lse - z[torch.arange(len(keep), device="cuda"), tk]
    kept[keep] = lse
    if not case["grad"]:
        return loss, kept
    z -= lse[:, None]
    z.exp_()
    z[torch.arange(len(keep), device="cuda"), tk] -= 1
    z *= s["scale"].double()
    dh = torch.zeros_like(h)
    dh[keep] = torch.mm(z, w)
    dw = torch.mm(z.t().contiguous(), hk)
    return loss, kept, dh, dw
