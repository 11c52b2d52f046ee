"""Operators around the vocabulary head: the linear layer with its epilogue, the
adjustments of logits before sampling, and the gradients' global norm and clipping.

Each case is one call (or one forward and backward pair) as a program makes it:
`prepare` makes what the program holds before the call, `run` makes the call.  With
`own` false `run` computes the operator in elementary torch operations in 32 bits,
with `own` true through the library; `exact` is the operator's definition in 64 bits.

kind "linear": z = hidden weight^T + bias;  out = residual + act(z); with "train" also
               dz = grad act'(z), dhidden = dz weight, dweight = dz^T hidden, dbias = sum_n dz.
kind "adjust": the logits of the tokens in a row's history are penalised (repetition, then
               frequency, then presence, as the sampler does it), biases are added to
               the listed tokens, and tokens whose mask bit is 0 become -inf.
kind "clip":   norm = sqrt(sum of all squares); where norm > max_norm every gradient is
               multiplied by max_norm / norm.
"""

import math

import torch

own = False

DEVICE = "cuda"
ROW_NOTHING_ALLOWED = 10


def listed():
    return [
        # The logits of one decoding sequence on a small model's head, capped, for
        # a sampler that takes float32: the weights are read once.
        dict(name="linear_head_one", kind="linear", N=1, V=32000, D=2048, dtype="bf16", bias=False, act="softcap",
             residual=False, out="f32", train=False),
        # The residual block of a draft head, h + silu(W h + b), for a few
        # sequences: a call where latency counts.
        dict(name="linear_block_few", kind="linear", N=8, V=4096, D=4096, dtype="bf16", bias=True, act="silu",
             residual=True, out="bf16", train=False),
        # The logits of the sampler's headline batch.
        dict(name="linear_head_batch", kind="linear", N=256, V=129280, D=4096, dtype="bf16", bias=False, act="none",
             residual=False, out="bf16", train=False),
        # A training step of the residual block: output and all gradients.
        dict(name="linear_train", kind="linear", N=4096, V=4096, D=4096, dtype="bf16", bias=True, act="silu",
             residual=True, out="bf16", train=True),
        # Odd sizes: columns that are no multiple of any tile, rows of odd length.
        dict(name="linear_train_odd", kind="linear", N=1037, V=5003, D=1000, dtype="bf16", bias=True, act="gelu_tanh",
             residual=False, out="bf16", train=True),
        # Fine-tuning in float32.
        dict(name="linear_train_f32", kind="linear", N=384, V=2048, D=1024, dtype="f32", bias=True, act="gelu",
             residual=True, out="f32", train=True),
        # One sequence under a grammar, with penalties for what it has written.
        dict(name="adjust_one", kind="adjust", B=1, V=32000, dtype="bf16", history=500, biases=20, narrow=0, wide=1),
        # A serving batch: penalties and biases for every row, a quarter of the rows at
        # a grammar's structural token (few tokens allowed), a quarter inside
        # free text of a grammar (most tokens allowed), the others without one.
        dict(name="adjust_batch", kind="adjust", B=256, V=129280, dtype="bf16", history=1024, biases=100, narrow=64,
             wide=64),
        # Odd sizes, float32 logits, long histories.
        dict(name="adjust_odd", kind="adjust", B=37, V=50001, dtype="f32", history=20000, biases=300, narrow=5,
             wide=8),
        # The gradients of a draft head's block and of its norms.
        dict(name="clip_block", kind="clip", sizes="block", count=12, largest=1048576, dtype="bf16", out="bf16",
             clipped=True),
        # Many small odd tensors (adapters) in float32.
        dict(name="clip_many", kind="clip", sizes="spread", count=1500, largest=40000, dtype="f32", out="f32",
             clipped=True),
        # A model's worth of gradients, the head's among them, to a float32 optimizer.
        dict(name="clip_model", kind="clip", sizes="block", count=48, largest=129280 * 4096, dtype="bf16", out="f32",
             clipped=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    kind = rng.choice(("linear", "linear", "adjust", "clip"))
    if kind == "linear":
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        train = rng.random() < 0.5
        N = _log_int(rng, 1, 512 if dtype == "f32" else 4096)
        V = _log_int(rng, 200, 4096 if dtype == "f32" else 8192 if train else 132000)
        D = _log_int(rng, 100, 1024 if dtype == "f32" else 4096)
        if rng.random() < 0.8:
            D = 8 * max(1, D // 8)
        while N * V * D > (4096 ** 3 if train else 256 * 129280 * 4096) * (0.02 if dtype == "f32" else 0.9):
            N = max(1, N // 2)
        return dict(kind="linear", N=N, V=V, D=D, dtype=dtype, bias=rng.random() < 0.6,
                    act=rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu", "softcap")),
                    residual=rng.random() < 0.5, out="f32" if dtype == "f32" else rng.choice(("bf16", "bf16", "f32")),
                    train=train)
    if kind == "adjust":
        B = _log_int(rng, 1, 256)
        V = _log_int(rng, 1000, 129280)
        narrow = rng.randint(0, B) // rng.choice((1, 2, 8))
        return dict(kind="adjust", B=B, V=V, dtype=rng.choice(("bf16", "bf16", "f32")) if B <= 128 else "bf16",
                    history=rng.choice((0, _log_int(rng, 1, 20000 if B <= 64 else 1024))),
                    biases=rng.choice((0, _log_int(rng, 1, 300))), narrow=narrow,
                    wide=rng.randint(0, B - narrow) // rng.choice((1, 2, 8)))
    return dict(kind="clip", sizes=rng.choice(("block", "spread")), count=_log_int(rng, 1, 1000),
                largest=_log_int(rng, 10, 100000), dtype=rng.choice(("bf16", "f32")), out=rng.choice(("bf16", "f32")),
                clipped=rng.random() < 0.8)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _counts(c):
    """Elements of each gradient of a clip case."""
    n, top = c["count"], c["largest"]
    if c["sizes"] == "block":
        # one large matrix, then smaller ones and vectors, as the parts of a block
        return [top if i == 0 else max(1, top // 32) if i % 3 == 1 else max(1, top // 64) if i % 3 == 2
                else max(1, min(top, 4096)) for i in range(n)]
    # sizes over the whole range, most of them odd
    return [max(1, int(math.exp(math.log(top) * ((i * 7919) % n + 1) / n))) for i in range(n)]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    if c["kind"] == "linear":
        N, V, D, t = c["N"], c["V"], c["D"], _type(c["dtype"])
        # a normalised hidden state; pre-activations of about one
        c["hidden"] = normal(N, D).to(t)
        c["weight"] = (normal(V, D) * (1.0 / math.sqrt(D))).to(t)
        c["cap"] = 3.0 if c["act"] == "softcap" else 0.0
        c["b"] = (normal(V) * 0.1).to(t) if c["bias"] else None
        c["r"] = normal(N, V).to(t) if c["residual"] else None
        c["grad"] = (normal(N, V) / N).to(_type(c["out"])) if c["train"] else None
        return c
    if c["kind"] == "adjust":
        B, V = c["B"], c["V"]
        # logits of a long-tailed distribution
        u = torch.rand(B, V, generator=g, device=DEVICE)
        c["logits"] = (-1.1 * torch.log(1.0 + u * V) + 0.5 * normal(B, V)).to(_type(c["dtype"]))
        c["presence"] = 0.5 * (torch.rand(B, generator=g, device=DEVICE) < 0.7).float()
        c["frequency"] = 0.3 * torch.rand(B, generator=g, device=DEVICE)
        c["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device=DEVICE)
        # sampling records as a server keeps them on the device
        record = torch.zeros(B, 8, dtype=torch.float32, device=DEVICE)
        record[:, 0], record[:, 2] = 0.7, 1.0
        record[:, 4], record[:, 5], record[:, 6] = c["presence"], c["frequency"], c["repetition"]
        c["params"] = record.view(torch.uint8).view(B, 32)
        every = torch.arange(B + 1, device=DEVICE, dtype=torch.int64)
        c["hist_ids"] = c["hist_offsets"] = None
        if c["history"]:
            # text repeats itself: most tokens come from the low ids
            spread = torch.rand(B * c["history"], generator=g, device=DEVICE)
            c["hist_ids"] = (spread * spread * spread * V).to(torch.int32).clamp_(0, V - 1)
            c["hist_offsets"] = every * c["history"]
        c["bias_ids"] = c["bias_values"] = c["bias_offsets"] = None
        if c["biases"]:
            # ids of one row are all different
            n = c["biases"]
            step = max(1, V // n)
            start = torch.randint(0, V, (B, 1), generator=g, device=DEVICE)
            c["bias_ids"] = ((start + step * torch.arange(n, device=DEVICE)) % V).to(torch.int32).reshape(-1)
            c["bias_values"] = 2.0 * normal(B * n)
            c["bias_offsets"] = every * n
        rows, words = c["narrow"] + c["wide"], (V + 31) // 32
        c["mask"] = c["mask_rows"] = None
        if rows:
            bits = torch.rand(rows, words * 32, generator=g, device=DEVICE)
            few = torch.arange(rows, device=DEVICE)[:, None] < c["narrow"]
            bits = torch.where(few, bits < 0.002, bits < 0.97)
            bits[:, 0] = True
            packed = (bits.view(rows, words, 32).long() << torch.arange(32, device=DEVICE)).sum(dim=2)
            c["mask"] = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)
            at = torch.full((B,), -1, dtype=torch.int32, device=DEVICE)
            at[torch.randperm(B, generator=g, device=DEVICE)[:rows]] = torch.arange(rows, dtype=torch.int32,
                                                                                     device=DEVICE)
            c["mask_rows"] = at
        c["status"] = torch.empty(B, dtype=torch.int32, device=DEVICE)
        return c
    counts = _counts(c)
    # gradients whose size differs from tensor to tensor
    c["grads"] = [normal(n).mul_(10.0 ** (-1 - i % 3)).to(_type(c["dtype"])) for i, n in enumerate(counts)]
    expected = math.sqrt(sum(n * 100.0 ** (-1 - i % 3) for i, n in enumerate(counts)))
    c["max_norm"] = expected * 0.25 if c["clipped"] else expected * 4.0 + 10.0
    # they go to an optimizer's buffer, one after the other
    c["flat"] = torch.empty(sum(counts), dtype=_type(c["out"]), device=DEVICE)
    c["outs"] = list(torch.split(c["flat"], counts))
    c["norm"] = torch.empty(1, dtype=torch.float32, device=DEVICE)
    if own:  # the list of its gradients that a program makes once
        import decode_step_token_row_amd as arcs
        c["plan"] = arcs.TensorList(c["grads"], outs=c["outs"])
    return c


_TANH_A, _TANH_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act, cap):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_TANH_A * (z + _TANH_B * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "softcap":
        return cap * torch.tanh(z / cap)
    return z


def _slope(z, act, cap):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_TANH_A * (z + _TANH_B * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _TANH_A * (1.0 + 3.0 * _TANH_B * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "softcap":
        t = torch.tanh(z / cap)
        return 1.0 - t * t
    return torch.ones_like(z)


def _plain_linear(s):
    h, w = s["hidden"].float(), s["weight"].float()
    z = h @ w.t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"], s["cap"])
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"out": y.to(_type(s["out"]))}
    if s["train"]:
        dz = s["grad"].float() * _slope(z, s["act"], s["cap"])
        out["dhidden"] = (dz @ w).to(s["hidden"].dtype)
        out["dweight"] = (dz.t() @ h).to(s["weight"].dtype)
        if s["b"] is not None:
            out["dbias"] = dz.sum(dim=0).to(s["b"].dtype)
    return out


def _rows_of(offsets, total):
    lengths = offsets[1:] - offsets[:-1]
    return torch.repeat_interleave(torch.arange(len(lengths), device=DEVICE), lengths, output_size=total)


def _plain_adjust(s):
    B, V = s["B"], s["V"]
    z = s["logits"].float()
    if s["hist_ids"] is not None:
        row = _rows_of(s["hist_offsets"], len(s["hist_ids"]))
        count = torch.zeros(B * V, dtype=torch.float32, device=DEVICE)
        count = count.scatter_add(0, row * V + s["hist_ids"].long(), torch.ones_like(row, dtype=torch.float32))
        count = count.view(B, V)
        r = s["repetition"][:, None]
        y = torch.where(z > 0, z / r, z * r)
        y = y - s["frequency"][:, None] * count
        y = y - s["presence"][:, None]
        z = torch.where(count > 0, y, z)
    if s["bias_ids"] is not None:
        row = _rows_of(s["bias_offsets"], len(s["bias_ids"]))
        add = torch.zeros(B * V, dtype=torch.float32, device=DEVICE)
        z = z + add.scatter_add(0, row * V + s["bias_ids"].long(), s["bias_values"]).view(B, V)
    status = torch.zeros(B, dtype=torch.int32, device=DEVICE)
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, dtype=torch.int32, device=DEVICE)) & 1
        allowed = (bits == 1).view(len(s["mask"]), -1)[:, :V]
        masked = (s["mask_rows"] >= 0)[:, None]
        allowed = allowed[s["mask_rows"].clamp(min=0).long()] | ~masked
        z = torch.where(allowed, z, torch.full_like(z, -math.inf))
        status = torch.where(allowed.any(dim=1), status, torch.full_like(status, ROW_NOTHING_ALLOWED))
    return {"logits": z.to(s["logits"].dtype), "status": status}


def _plain_clip(s):
    g = torch.cat(s["grads"]).float()
    norm = (g * g).sum(dtype=torch.float64).sqrt()
    scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm)).float()
    return {"norm": norm.float().view(1), "grads": (g * scale).to(_type(s["out"]))}


def _own_linear(arcs, s):
    args = dict(activation=s["act"], softcap=s["cap"])
    if not s["train"]:
        return {"out": arcs.linear(s["hidden"], s["weight"], bias=s["b"], residual=s["r"], out_dtype=_type(s["out"]),
                                   **args)}
    # the gradient of a linear layer without an activation needs no pre-activations
    keep = s["act"] != "none"
    y = arcs.linear(s["hidden"], s["weight"], bias=s["b"], residual=s["r"], out_dtype=_type(s["out"]),
                    want_pre=keep, **args)
    y, pre = y if keep else (y, None)
    dh, dw, db = arcs.linear_backward(s["hidden"], s["weight"], s["grad"], pre=pre, want_bias=s["b"] is not None,
                                      **args)
    out = {"out": y, "dhidden": dh, "dweight": dw}
    if s["b"] is not None:
        out["dbias"] = db
    return out


def _own_clip(arcs, s):
    return {"norm": arcs.clip_gradients(s["plan"], s["max_norm"], out_norm=s["norm"]), "grads": s["flat"]}


def run(state):
    s = state
    if own:
        import decode_step_token_row_amd as arcs
        if s["kind"] == "linear":
            return _own_linear(arcs, s)
        if s["kind"] == "clip":
            return _own_clip(arcs, s)
        return {"logits": arcs.adjust_logits(
            s["logits"], s["params"], hist_ids=s["hist_ids"], hist_offsets=s["hist_offsets"], bias_ids=s["bias_ids"],
            bias_values=s["bias_values"], bias_offsets=s["bias_offsets"], mask=s["mask"], mask_rows=s["mask_rows"],
            out_status=s["status"]), "status": s["status"]}
    return {"linear": _plain_linear, "adjust": _plain_adjust, "clip": _plain_clip}[s["kind"]](s)


def work(case):
    c, size = case, {"bf16": 2, "f32": 4}
    if c["kind"] == "linear":
        N, V, D, e, o = c["N"], c["V"], c["D"], size[c["dtype"]], size[c["out"]]
        bytes_ = (V * D + N * D + (V if c["bias"] else 0) + (N * V if c["residual"] else 0)) * e + N * V * o
        flops = 2 * N * V * D
        if c["train"]:
            # the gradient of the output comes in, the three gradients go out
            bytes_ += N * V * o + (N * D + V * D + (V if c["bias"] else 0)) * e
            flops *= 3
        return {"bytes": bytes_, "flops": flops}
    if c["kind"] == "adjust":
        B, V, e = c["B"], c["V"], size[c["dtype"]]
        # what a narrow mask takes away need not be read
        bytes_ = (B - c["narrow"]) * V * e + B * V * e + (c["narrow"] + c["wide"]) * ((V + 31) // 32) * 4
        bytes_ += B * (c["history"] * 4 + c["biases"] * 8 + 32 + 16 + 4 + 4)
        return {"bytes": bytes_, "flops": 4 * B * (c["history"] + c["biases"])}
    n = sum(_counts(c))
    return {"bytes": n * (size[c["dtype"]] + size[c["out"]]), "flops": 3 * n}


def _exact_linear(s):
    f8 = torch.float64
    h, w = s["hidden"].to(f8), s["weight"].to(f8)
    z = torch.mm(h, w.t().contiguous())
    if s["b"] is not None:
        z += s["b"].to(f8)
    # the activation and its derivative by torch's own differentiation in 64 bits
    z.requires_grad_(s["train"])
    act, cap = s["act"], s["cap"]
    if act == "relu":
        a = torch.relu(z)
    elif act == "gelu":
        a = z * torch.special.ndtr(z)
    elif act == "gelu_tanh":
        a = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    elif act == "silu":
        a = z * torch.sigmoid(z)
    elif act == "softcap":
        a = cap * (2.0 * torch.sigmoid(2.0 * z / cap) - 1.0)
    else:
        a = z * 1.0
    y = a.detach()
    out = {"out": y + s["r"].to(f8) if s["r"] is not None else y}
    if s["train"]:
        dz, = torch.autograd.grad(a, z, s["grad"].to(f8))
        out["dhidden"] = torch.mm(dz, w)
        out["dweight"] = torch.mm(dz.t().contiguous(), h)
        if s["b"] is not None:
            out["dbias"] = dz.sum(dim=0)
    return out


def _exact_adjust(s):
    f8, V = torch.float64, s["V"]
    y = s["logits"].to(f8)
    for b in range(s["B"]):
        if s["hist_ids"] is not None:
            lo, hi = b * s["history"], (b + 1) * s["history"]
            ids, times = torch.unique(s["hist_ids"][lo:hi].long(), return_counts=True)
            v = y[b, ids]
            v = torch.where(v > 0, v / s["repetition"][b].to(f8), v * s["repetition"][b].to(f8))
            y[b, ids] = v - times.to(f8) * s["frequency"][b].to(f8) - s["presence"][b].to(f8)
        if s["bias_ids"] is not None:
            lo, hi = b * s["biases"], (b + 1) * s["biases"]
            y[b, s["bias_ids"][lo:hi].long()] += s["bias_values"][lo:hi].to(f8)
    status = torch.zeros(s["B"], dtype=torch.int32, device=DEVICE)
    if s["mask"] is not None:
        token = torch.arange(V, device=DEVICE)
        for b, at in enumerate(s["mask_rows"].tolist()):
            if at >= 0:
                gone = (s["mask"][at].long()[token // 32] >> (token % 32)) % 2 == 0
                y[b, gone] = -math.inf
                if bool(gone.all()):
                    status[b] = ROW_NOTHING_ALLOWED
    return {"logits": y, "status": status}


def exact(case, seed):
    """The definition in 64 bits, from the inputs alone."""
    s = prepare(case, seed)
    if s["kind"] == "linear":
        return _exact_linear(s)
    if s["kind"] == "adjust":
        return _exact_adjust(s)
    f8 = torch.float64
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.to(f8))) ** 2 for g in s["grads"]))
    scale = min(1.0, s["max_norm"] / norm)
    return {"norm": torch.tensor([norm], dtype=f8, device=DEVICE),
            "grads": torch.cat([g.to(f8) * scale for g in s["grads"]])}
