"""The 8-bit operators' workloads: what is measured, each in a plain form.

Cases of four kinds:
  norm       root-mean-square norm of x + residual.  "serve" gives the new residual and the
             8-bit output (as the values it stands for), the step before an 8-bit product;
             "train" gives y, the new residual and 1/rms, then takes a backward pass from the
             residual and 1/rms that a forward pass has kept.
  quantize   rows to 8 bits with a scale each: a weight when it is loaded, an activation on its way
             into a product.  Returned as the values they stand for.
  product    activations in 8 bits times a weight [d_out, d_in] in 8 bits, a scale for each token
             and each channel; with "adapter" the DoRA composition with the adapter branch's
             output in the same call, with "bias" the layer's bias.
  train      a frozen 8-bit weight in a training step: output and gradient of the input.

Sizes are those of the workloads in dora_inputs.py (4096^2, 8192^2, 28672 x 8192, the 5120-wide
sweep; 2048 and 4096 tokens) and odd ones.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of decoding through the norm before an 8-bit projection: latency
        {"name": "norm serve 1x4096", "kind": "norm", "mode": "serve", "T": 1, "d": 4096, "dtype": "bf16"},
        # a prompt through the same norm
        {"name": "norm serve 4096x8192", "kind": "norm", "mode": "serve", "T": 4096, "d": 8192, "dtype": "bf16"},
        # a training step's norm of the 5120-wide sweep, forward and backward
        {"name": "norm train 2048x5120", "kind": "norm", "mode": "train", "T": 2048, "d": 5120, "dtype": "bf16"},
        # odd sizes in fp32
        {"name": "norm train 333x1003 f32", "kind": "norm", "mode": "train", "T": 333, "d": 1003, "dtype": "f32"},
        # a merged weight to 8 bits, when a server loads it
        {"name": "quantize 8192x8192", "kind": "quantize", "T": 8192, "d": 8192, "dtype": "bf16"},
        # a few tokens' wide activation on the way into the down projection
        {"name": "quantize 7x27648 f16", "kind": "quantize", "T": 7, "d": 27648, "dtype": "f16"},
        # one token through the widest projection: the weight's bytes count
        {"name": "product 1x28672x8192", "kind": "product", "T": 1, "d_out": 28672, "d_in": 8192,
         "dtype": "bf16", "adapter": False, "bias": False},
        # a decoding batch with its adapter unmerged
        {"name": "product 24x5120x5120 f16", "kind": "product", "T": 24, "d_out": 5120, "d_in": 5120,
         "dtype": "f16", "adapter": True, "bias": False},
        # ragged in every dimension, with a bias
        {"name": "product 333x4090x2056", "kind": "product", "T": 333, "d_out": 4090, "d_in": 2056,
         "dtype": "bf16", "adapter": False, "bias": True},
        # a prompt through a square projection, adapter unmerged
        {"name": "product 2048x8192x8192", "kind": "product", "T": 2048, "d_out": 8192, "d_in": 8192,
         "dtype": "bf16", "adapter": True, "bias": False},
        # the largest: a long prompt through the widest projection
        {"name": "product 4096x28672x8192", "kind": "product", "T": 4096, "d_out": 28672, "d_in": 8192,
         "dtype": "bf16", "adapter": False, "bias": False},
        # a training step's frozen weight, forward and the input's gradient
        {"name": "train 2048x5120x5120", "kind": "train", "T": 2048, "d_out": 5120, "d_in": 5120, "dtype": "bf16"},
    ]


WIDTHS = (1024, 2056, 4096, 5120, 8192, 27648, 28672)


def _spread(rng, lo, hi):
    """A whole number of lo..hi, evenly over the logarithm; odd ones among them."""
    n = int(round(lo * (hi / lo) ** rng.random()))
    if n > 64 and rng.random() < 0.5:
        n -= n % 8
    return n


def _width(rng):
    return rng.choice(WIDTHS) if rng.random() < 0.5 else _odd_width(rng)


def _odd_width(rng):
    n = _spread(rng, 64, 16384)
    return n + 8 if n == 3 << 10 else n


def draw(rng):
    kind = rng.choice(("norm", "norm", "quantize", "product", "product", "product", "train"))
    # fp32 where no output hangs on how one code was rounded: at a tie between two codes any fp32
    # evaluation may take either, a step that 32-bit comparison would not let pass
    dtype = rng.choice(("bf16", "bf16", "f16", "f32") if kind == "product" else ("bf16", "bf16", "f16"))
    T = _spread(rng, 1, 4096)
    T = T + 1 if T == 3 << 10 else T
    if kind in ("norm", "quantize"):
        case = {"kind": kind, "T": T, "d": _width(rng), "dtype": dtype}
        if kind == "norm":
            case["mode"] = rng.choice(("serve", "train"))
            if case["mode"] == "train" and rng.random() < 0.25:
                case["dtype"] = "f32"
        return case
    d_out, d_in = _width(rng), _width(rng)
    if d_out * d_in > 28672 * 8192:
        d_in = rng.choice((1024, 2056, 4096))
    case = {"kind": kind, "T": T, "d_out": d_out, "d_in": d_in, "dtype": dtype}
    if kind == "train":  # two products
        case["T"] = max(1, T // 2)
        case["T"] += case["T"] == 3 << 10
    else:
        case["adapter"], case["bias"] = rng.random() < 0.5, rng.random() < 0.3
    return case


def work(case):
    e = BYTES[case["dtype"]]
    T = case["T"]
    if case["kind"] == "norm":
        n, d = T * case["d"], case["d"]
        if case["mode"] == "serve":  # x, residual, w; h, values
            return {"bytes": 4 * n * e + d * e, "flops": 8 * n}
        # x, residual, w; y, h, rstd; dy, dh, the kept h and rstd; dx, dw
        return {"bytes": 8 * n * e + 2 * d * e + 8 * T + 4 * d, "flops": 16 * n}
    if case["kind"] == "quantize":
        n = T * case["d"]
        return {"bytes": 2 * n * e, "flops": 4 * n}
    N, K = case["d_out"], case["d_in"]
    if case["kind"] == "product":
        b = T * K + 4 * T + N * K + 4 * N + T * N * e
        b += (T * N * e + 4 * N if case["adapter"] else 0) + (4 * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * T * N * K}
    # x, codes, scales, y; dy, transposed codes, dx
    return {"bytes": 2 * T * K * e + 2 * T * N * e + 2 * N * K + 8 * N, "flops": 4 * T * N * K}


# ------------------------------------------------------------------ inputs
def _codes(w):
    """A weight's rows in 8 bits with a scale each, as they are kept after loading."""
    w = w.float()
    scale = w.abs().amax(dim=1) / 127
    return torch.round(w / scale[:, None]).to(torch.int8), scale


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    T = case["T"]
    s = {"case": case, "dtype": dt}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def hidden(rows, d):
        # the residual stream: a few channels far larger than the others
        width = torch.exp(0.5 * normal(d)) * torch.where(torch.rand(d, generator=gen, device=dev) < 0.002, 20.0, 1.0)
        return (normal(rows, d) * width).to(dt)

    if case["kind"] == "norm":
        d = case["d"]
        s["x"], s["residual"] = normal(T, d).to(dt), hidden(T, d)
        s["w"] = (1 + 0.1 * normal(d)).to(dt)
        if case["mode"] == "train":
            s["dy"], s["dh"] = normal(T, d).to(dt), normal(T, d).to(dt)
            # what a forward pass has kept for the backward pass
            s["h"] = (s["x"].float() + s["residual"].float()).to(dt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + EPS)
        return s
    if case["kind"] == "quantize":
        s["x"] = hidden(T, case["d"])
        return s
    N, K = case["d_out"], case["d_in"]
    s["wq"], s["ws"] = _codes((normal(N, K) / K ** 0.5).to(dt))
    if case["kind"] == "product":
        s["xq"], s["xs"] = _codes(hidden(T, K))
        s["g"] = 1 + 0.01 * normal(N) if case["adapter"] else None
        s["lora"] = (0.1 * normal(T, N)).to(dt) if case["adapter"] else None
        s["s"] = 2.0 if case["adapter"] else 1.0
        s["bias"] = normal(N) if case["bias"] else None
    else:
        s["x"], s["dy"] = hidden(T, K), normal(T, N).to(dt)
        s["wqt"] = s["wq"].t().contiguous()
    return s


# ------------------------------------------------------------------ the operators, plain
def _plain_quantize(p):
    scale = p.abs().amax(dim=1, keepdim=True) / 127
    return torch.where(scale > 0, torch.round(p / scale), 0.0), scale


def _plain(s):
    case, dt = s["case"], s["dtype"]
    if case["kind"] == "norm":
        h = s["x"].float() + s["residual"].float()
        w = s["w"].float()
        rstd = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        y = h * rstd * w
        if case["mode"] == "serve":
            q, scale = _plain_quantize(y)
            return {"h": h.to(dt), "values": (q * scale).to(dt)}
        dy, kept, r = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
        u = dy * w
        dx = r * (u - kept * (r * r) * (u * kept).mean(dim=1, keepdim=True)) + s["dh"].float()
        return {"y": y.to(dt), "h": h.to(dt), "rstd": rstd[:, 0], "dx": dx.to(dt), "dw": (dy * kept * r).sum(dim=0)}
    if case["kind"] == "quantize":
        q, scale = _plain_quantize(s["x"].float())
        return {"values": (q * scale).to(dt), "scale": scale[:, 0]}
    wq = s["wq"].float()
    if case["kind"] == "product":
        y = (s["xq"].float() @ wq.t()) * s["xs"][:, None] * s["ws"]
        if s["g"] is not None:
            y = y + ((s["g"] - 1) * y + (s["g"] * s["s"]) * s["lora"].float())
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"y": y.to(dt)}
    xq, xs = _plain_quantize(s["x"].float())
    y = (xq @ wq.t()) * xs * s["ws"]
    dq, ds = _plain_quantize(s["dy"].float() * s["ws"])
    dx = (dq @ wq) * ds
    return {"y": y.to(dt), "dx": dx.to(dt)}


def _own(s):
    import dora_adapter_factored_amd as D

    case, dt = s["case"], s["dtype"]
    if case["kind"] == "norm":
        if case["mode"] == "serve":
            q, scale, h = D.rmsnorm_q8(s["x"], s["w"], EPS, s["residual"])
            return {"h": h, "values": D.dequantize_rows(q, scale, dt)}
        y, h, rstd = D.rmsnorm(s["x"], s["w"], EPS, s["residual"])
        dx, dw = D.rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], s["dh"])
        return {"y": y, "h": h, "rstd": rstd, "dx": dx, "dw": dw}
    if case["kind"] == "quantize":
        q, scale = D.quantize_rows(s["x"])
        return {"values": D.dequantize_rows(q, scale, dt), "scale": scale}
    if case["kind"] == "product":
        y = D.matmul_q8(s["xq"], s["xs"], s["wq"], s["ws"], dt, bias=s["bias"], g=s["g"], lora_out=s["lora"], s=s["s"])
        return {"y": y}
    y = D.linear_q8(s["x"], s["wq"], s["ws"])
    return {"y": y, "dx": D.linear_q8_backward(s["dy"], s["wqt"], s["ws"])}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    a = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}

    def eight(v):
        top = v.abs().max(dim=1).values
        step = top / 127
        codes = torch.zeros_like(v)
        full = top > 0
        codes[full] = (v[full] / step[full].unsqueeze(1)).round()
        return codes, step

    if case["kind"] == "norm":
        h = a["x"] + a["residual"]
        rms = (h.square().sum(1) / case["d"] + EPS).sqrt()
        n = h / rms[:, None]
        y = n * a["w"]
        if case["mode"] == "serve":
            codes, step = eight(y)
            return {"h": h, "values": codes * step[:, None]}
        k = a["h"] * a["rstd"][:, None]
        dn = a["dy"] * a["w"]
        dx = (dn - k * ((dn * k).sum(1, keepdim=True) / case["d"])) * a["rstd"][:, None] + a["dh"]
        return {"y": y, "h": h, "rstd": 1 / rms, "dx": dx, "dw": (a["dy"] * k).sum(0)}
    if case["kind"] == "quantize":
        codes, step = eight(a["x"])
        return {"values": codes * step[:, None], "scale": step}
    W = a["wq"] * a["ws"][:, None]
    if case["kind"] == "product":
        base = (a["xq"] * a["xs"][:, None]) @ W.t()
        y = base if a["g"] is None else a["g"] * (base + a["s"] * a["lora"])
        return {"y": y if a["bias"] is None else y + a["bias"]}
    xc, xstep = eight(a["x"])
    dc, dstep = eight(a["dy"] * a["ws"])
    return {"y": (xc * xstep[:, None]) @ W.t(), "dx": (dc @ a["wq"]) * dstep[:, None]}
