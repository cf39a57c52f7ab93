"""Performance cases of the operators beside the convolution: group normalisation with an activation on NHWC
activations (wino.group_norm) and the matrix product with bias, activation and residual in its epilogue (wino.matmul).

Each case is one call as a program around the int8 convolutions makes it.  With `own` false, run() computes the
operator in plain fp32 torch operations, rounded once at the end; with `own` true it calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm(name, n, h, w, c, c2=0, groups=32, act="silu", add=False, dtype="bf16", eps=1e-5):
    return {"name": name, "op": "group_norm", "n": n, "h": h, "w": w, "c": c, "c2": c2, "groups": groups, "act": act,
            "add": add, "dtype": dtype, "eps": eps}


def _product(name, m, k, n, k2=0, act="none", bias=True, residual=False, dtype="bf16", out="bf16"):
    return {"name": name, "op": "matmul", "m": m, "k": k, "k2": k2, "n": n, "act": act, "bias": bias,
            "residual": residual, "dtype": dtype, "out": out}


def listed():
    return [
        # the norm before a conv of the innermost 8x8 level, one image: a few microseconds, latency only
        _norm("norm_n1_8x8_c1280", 1, 8, 8, 1280),
        # second norm of a residual block at 64x64: the time embedding's projection is added per image and channel
        _norm("norm_n8_64x64_c320_add", 8, 64, 64, 320, add=True),
        # first norm of an up-path block: the input is the concatenation with a skip tensor, groups of 30 channels
        # that straddle both; the largest norm
        _norm("norm_n8_64x64_c640+320", 8, 64, 64, 640, c2=320),
        # the norm in front of a 1x1 projection: no activation, small epsilon, fp32 activations
        _norm("norm_n2_32x32_c640_f32", 2, 32, 32, 640, act="none", dtype="f32", eps=1e-6),
        # an image whose sides are no multiple of anything, groups of 60 channels over a concatenation
        _norm("norm_n3_37x29_c1280+640", 3, 37, 29, 1280, c2=640),
        # the time embedding of a single image: one row, 1280 -> 1280
        _product("product_m1_1280_1280_silu", 1, 1280, 1280, act="silu"),
        # the same network's first layer in fp32 for a batch of 8
        _product("product_m8_320_1280_silu_f32", 8, 320, 1280, act="silu", dtype="f32", out="f32"),
        # the classifier of an image network: 32 images, 512 features, 1000 classes, logits in fp32
        _product("product_m32_512_1000_logits", 32, 512, 1000, out="f32"),
        # the 1x1 shortcut of an 8x8 up-path block over its concatenated input, added to the conv path's output
        _product("product_m512_1280+1280_1280_res", 512, 1280, 1280, k2=1280, residual=True),
        # the 1x1 shortcut of a 64x64 up-path block: bound by its activations' bytes
        _product("product_m32768_640+320_320_res", 32768, 640, 320, k2=320, residual=True),
        # a 1x1 projection with residual over three images of 37x29 pixels
        _product("product_m3219_640_640_res", 3219, 640, 640, residual=True),
        # the widening layer of a 32x32 block's per-pixel network: bound by the tensor cores
        _product("product_m8192_1280_5120_gelu", 8192, 1280, 5120, act="gelu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:   # up to the work of the largest listed norm
            n, h, w = rng.randint(1, 8), _log_int(rng, 4, 72), _log_int(rng, 4, 72)
            groups = rng.choice((8, 16, 32, 32, 32))
            c = 32 * _log_int(rng, 1, 40)
            c2 = 32 * _log_int(rng, 1, 40) if rng.random() < 0.35 else 0
            dtype = rng.choice(("bf16", "bf16", "f32"))
            if n * h * w * (c + c2) * (1 if dtype == "bf16" else 2) <= 8 * 64 * 64 * 960:
                case = _norm("", n, h, w, c, c2, groups, rng.choice(("silu", "silu", "none")), rng.random() < 0.4, dtype,
                             rng.choice((1e-5, 1e-6)))
                break
    else:
        while True:   # up to the work of the largest listed product
            m, n = _log_int(rng, 1, 33000), _log_int(rng, 10, 5120)
            k = 32 * _log_int(rng, 2, 40)
            k2 = 32 * _log_int(rng, 2, 40) if rng.random() < 0.3 else 0
            # fp32 operands are the small networks on embeddings
            dtype = "f32" if m <= 16 and rng.random() < 0.5 else "bf16"
            if m * n * (k + k2) <= 8192 * 1280 * 5120 and m * max(n, k + k2) <= 8192 * 5120:
                out = "f32" if dtype == "f32" or (m <= 64 and rng.random() < 0.3) else "bf16"
                case = _product("", m, k, n, k2, rng.choice(("none", "silu", "gelu")), rng.random() < 0.8,
                                rng.random() < 0.5, dtype, out)
                break
    del case["name"]
    return case


def _activations(gen, rows, c, dtype):
    """Activations as a network has them: each channel with its own mean and spread, a few wide channels."""
    spread = torch.exp(0.5 * torch.randn(c, generator=gen, device="cuda"))
    mean = 0.5 * torch.randn(c, generator=gen, device="cuda")
    x = torch.randn(rows, c, generator=gen, device="cuda")
    return x.mul_(spread).add_(mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "group_norm":
        n, h, w, c, c2 = (case[k] for k in ("n", "h", "w", "c", "c2"))
        return {"case": case,
                "x": _activations(gen, n * h * w, c, dtype).view(n, h, w, c),
                "x2": _activations(gen, n * h * w, c2, dtype).view(n, h, w, c2) if c2 else None,
                "add": 0.5 * rand(n, c + c2) if case["add"] else None,
                "gamma": 1.0 + 0.2 * rand(c + c2), "beta": 0.2 * rand(c + c2)}
    m, k, k2, n = (case[key] for key in ("m", "k", "k2", "n"))
    return {"case": case,
            "a": _activations(gen, m, k, dtype), "a2": _activations(gen, m, k2, dtype) if k2 else None,
            "w": (rand(n, k + k2) / math.sqrt(k + k2)).to(dtype),
            "bias": 0.1 * rand(n) if case["bias"] else None,
            "residual": rand(m, n).to(DTYPES[case["out"]]) if case["residual"] else None}


def _plain_act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v


def _plain_group_norm(s):
    case = s["case"]
    x = s["x"].float()
    if s["x2"] is not None:
        x = torch.cat([x, s["x2"].float()], dim=3)
    n, h, w, c = x.shape
    if s["add"] is not None:
        x = x + s["add"].view(n, 1, 1, c)
    g = x.view(n, h * w, case["groups"], c // case["groups"])
    d = g - g.mean(dim=(1, 3), keepdim=True)
    var = (d * d).mean(dim=(1, 3), keepdim=True)
    y = (d * torch.rsqrt(var + case["eps"])).view(n, h, w, c) * s["gamma"] + s["beta"]
    return _plain_act(y, case["act"]).to(s["x"].dtype)


def _plain_matmul(s):
    case = s["case"]
    a = s["a"].float()
    if s["a2"] is not None:
        a = torch.cat([a, s["a2"].float()], dim=1)
    v = a @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _plain_act(v, case["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(DTYPES[case["out"]])


def run(state):
    case = state["case"]
    if own:
        from group_wise_int8_b200 import wino
        act = {"none": wino.ACT_NONE, "silu": wino.ACT_SILU, "gelu": wino.ACT_GELU}[case["act"]]
        if case["op"] == "group_norm":
            return wino.group_norm(state["x"], case["groups"], state["gamma"], state["beta"], eps=case["eps"], act=act,
                                   add=state["add"], x2=state["x2"])
        return wino.matmul(state["a"], state["w"], bias=state["bias"], act=act, residual=state["residual"],
                           a2=state["a2"], out_dtype=DTYPES[case["out"]])
    return _plain_group_norm(state) if case["op"] == "group_norm" else _plain_matmul(state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "group_norm":
        c = case["c"] + case["c2"]
        values = case["n"] * case["h"] * case["w"] * c
        extra = 4 * c * (2 + (case["n"] if case["add"] else 0))
        return {"bytes": 2 * values * size + extra, "flops": values * (16 if case["act"] != "none" else 10)}
    m, k, n = case["m"], case["k"] + case["k2"], case["n"]
    out = 2 if case["out"] == "bf16" else 4
    return {"bytes": size * (m * k + n * k) + (4 * n if case["bias"] else 0) + out * m * n * (2 if case["residual"] else 1),
            "flops": 2 * m * n * k}


def _sigmoid(v):   # of either sign without overflow
    e = torch.exp(-v.abs())
    return torch.where(v >= 0, 1 / (1 + e), e / (1 + e))


def exact(case, seed):
    s = prepare(case, seed)
    act = {"none": lambda v: v, "silu": lambda v: v * _sigmoid(v),
           "gelu": lambda v: v * torch.special.ndtr(v)}[case["act"]]
    if case["op"] == "matmul":
        k = case["k"]
        w = s["w"].double()
        v = torch.einsum("mk,nk->mn", s["a"].double(), w[:, :k])
        if case["k2"]:
            v += torch.einsum("mk,nk->mn", s["a2"].double(), w[:, k:])
        v = act(v if s["bias"] is None else v + s["bias"].double()[None, :])
        return v if s["residual"] is None else v + s["residual"].double()
    parts = [s["x"].double()] + ([s["x2"].double()] if case["c2"] else [])
    x = torch.cat(parts, 3).flatten(1, 2).transpose(1, 2).contiguous()          # [n][channel][pixel]
    if case["add"]:
        x += s["add"].double()[:, :, None]
    rows = x.view(case["n"] * case["groups"], -1)
    var, mean = torch.var_mean(rows, dim=1, correction=0, keepdim=True)
    y = ((rows - mean) / torch.sqrt(var + case["eps"])).view_as(x)
    y = act(y * s["gamma"].double()[None, :, None] + s["beta"].double()[None, :, None])
    return y.transpose(1, 2).reshape(case["n"], case["h"], case["w"], -1)
