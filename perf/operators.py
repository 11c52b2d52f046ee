"""The vocabulary head's operators: 4-bit head logits and the linear cross entropy.

Each case is one call (or one forward and backward pair) as a program makes
it: `prepare` makes what the program holds before the call, `run` makes the
call.  With `own` false `run` computes the operator in elementary torch
operations in 32 bits, with `own` true through the library; `exact` is the
operator's definition in 64 bits.

kind "w4": logits[b, v] = sum_g scale[v, g] * sum_{d in g} (q[v, d] - z[v, g]) * hidden[b, d].
kind "ce": z = hidden weight^T / T;  loss = logsumexp(z) - z[target], 0 for ignored rows;
           with "train" also the gradients of sum(grad_loss * loss).
"""

import math

import torch

own = False

IGNORE = -100
DEVICE = "cuda"


def listed():
    return [
        # One sequence decoding on a small model: the head's product at its
        # shortest, where the launch and the first loads count.
        dict(name="w4_one_row_small", kind="w4", B=1, V=32000, D=2048, group=64, zeros=False,
             scales="bf16", out="bf16"),
        # One sequence decoding with a large vocabulary: the 4-bit weights are
        # read once, everything else is small.
        dict(name="w4_one_row", kind="w4", B=1, V=129280, D=4096, group=128, zeros=True,
             scales="bf16", out="bf16"),
        # A few sequences, float32 scales and logits (a server that reports
        # log-probabilities).
        dict(name="w4_four_rows", kind="w4", B=4, V=151936, D=5120, group=64, zeros=False,
             scales="f32", out="f32"),
        # Odd sizes: a vocabulary that is no multiple of any tile, a batch in
        # between, the smallest groups with zero points.
        dict(name="w4_odd", kind="w4", B=19, V=50001, D=4064, group=32, zeros=True,
             scales="bf16", out="f32"),
        # A serving batch: still bound by the weights.
        dict(name="w4_batch_64", kind="w4", B=64, V=129280, D=7168, group=128, zeros=False,
             scales="bf16", out="bf16"),
        # The sampler's headline batch: the products count as much as the weights.
        dict(name="w4_batch_256", kind="w4", B=256, V=129280, D=7168, group=64, zeros=True,
             scales="bf16", out="bf16"),
        # The log-probability of one token, at its shortest.
        dict(name="score_one", kind="ce", N=1, V=32000, D=2048, dtype="bf16", train=False,
             temperature=False, ignored=0.0, weighted=False, head=True),
        # The log-probabilities of a decoded batch's tokens at their sampling temperatures.
        dict(name="score_batch", kind="ce", N=256, V=129280, D=4096, dtype="bf16", train=False,
             temperature=True, ignored=0.0, weighted=False, head=True),
        # A prompt's log-probabilities.
        dict(name="score_prompt", kind="ce", N=4096, V=129280, D=4096, dtype="bf16", train=False,
             temperature=False, ignored=0.0, weighted=False, head=True),
        # A training step of the head with a quarter of the rows masked
        # (prompt and padding): loss and both gradients.
        dict(name="train", kind="ce", N=4096, V=129280, D=4096, dtype="bf16", train=True,
             temperature=False, ignored=0.25, weighted=False, head=True),
        # Odd sizes, a weight per token and a temperature per row (a policy
        # gradient on sampled tokens).
        dict(name="train_odd", kind="ce", N=1037, V=50001, D=1000, dtype="bf16", train=True,
             temperature=True, ignored=0.1, weighted=True, head=True),
        # Fine-tuning in float32.
        dict(name="train_f32", kind="ce", N=384, V=32000, D=1024, dtype="f32", train=True,
             temperature=False, ignored=0.0, weighted=False, head=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: Products of a listed case at most, by kind.
_MOST = {"w4": 256 * 129280 * 7168, "ce": 4096 * 129280 * 4096}


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    if rng.random() < 0.5:
        group = rng.choice((32, 64, 128))
        B = _log_int(rng, 1, 256)
        V = _log_int(rng, 4096, 152000)
        D = group * _log_int(rng, 512 // group, 7168 // group)
        while B * V * D > _MOST["w4"]:
            B = max(1, B // 2)
        return dict(kind="w4", B=B, V=V, D=D, group=group, zeros=rng.random() < 0.5,
                    scales=rng.choice(("bf16", "f32")), out=rng.choice(("bf16", "f32")))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    N = _log_int(rng, 1, 512 if dtype == "f32" else 4096)
    V = _log_int(rng, 1000, 32000 if dtype == "f32" else 152000)
    D = 8 * _log_int(rng, 32, 128 if dtype == "f32" else 512)
    train = rng.random() < 0.6
    while N * V * D > _MOST["ce"] * 0.9:
        N = max(1, N // 2)
    return dict(kind="ce", N=N, V=V, D=D, dtype=dtype, train=train, temperature=rng.random() < 0.5,
                ignored=rng.choice((0.0, 0.0, 0.3, 0.6)) if N > 1 else 0.0,
                weighted=train and rng.random() < 0.5, head=rng.random() < 0.7)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _valid_rows(c):
    return c["N"] - int(c["ignored"] * c["N"])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    if c["kind"] == "w4":
        B, V, D, n = c["B"], c["V"], c["D"], c["D"] // c["group"]
        # a normalised hidden state; weights of a bell shape over the 16 levels
        hidden = torch.randn(B, D, generator=g, device=DEVICE).to(torch.bfloat16)
        q = torch.randn(V, D, generator=g, device=DEVICE, dtype=torch.bfloat16)
        q = q.mul_(2.7).round_().add_(8).clamp_(0, 15).to(torch.uint8)
        c["qweight"] = q[:, 0::2] | (q[:, 1::2] << 4)
        del q
        scale = (0.5 + torch.rand(V, n, generator=g, device=DEVICE)) * (1.0 / math.sqrt(D))
        c["scale"] = scale.to(_type(c["scales"]))
        c["zero"] = (torch.randint(6, 11, (V, n), generator=g, device=DEVICE, dtype=torch.uint8)
                     if c["zeros"] else None)
        c["hidden"] = hidden
        return c
    N, V, D, t = c["N"], c["V"], c["D"], _type(c["dtype"])
    weight = (torch.randn(V, D, generator=g, device=DEVICE) * (2.0 / math.sqrt(D))).to(t)
    target = torch.randint(0, V, (N,), generator=g, device=DEVICE)
    # hidden states that lean towards their targets, as a trained model's do
    lean = 4.0 * torch.rand(N, 1, generator=g, device=DEVICE)
    hidden = torch.randn(N, D, generator=g, device=DEVICE)
    hidden = (hidden + lean * 0.5 * weight[target].float()).to(t)
    valid = torch.ones(N, dtype=torch.bool, device=DEVICE)
    valid[torch.randperm(N, generator=g, device=DEVICE)[: N - _valid_rows(c)]] = False
    c["weight"], c["hidden"] = weight, hidden
    c["targets"] = torch.where(valid, target, torch.full_like(target, IGNORE)).to(torch.int32)
    c["T"] = 0.5 + torch.rand(N, generator=g, device=DEVICE) if c["temperature"] else None
    if c["train"]:
        grad = (torch.randn(N, generator=g, device=DEVICE) if c["weighted"]
                else torch.ones(N, device=DEVICE))
        c["grad_loss"] = grad / _valid_rows(c)
    return c


def _plain_w4(s):
    V, D, group = s["V"], s["D"], s["group"]
    q = torch.stack((s["qweight"] & 15, s["qweight"] >> 4), dim=2).view(V, D // group, group).float()
    q = q - (s["zero"].float()[:, :, None] if s["zero"] is not None else 8.0)
    w = (q * s["scale"].float()[:, :, None]).view(V, D)
    return (s["hidden"].float() @ w.t()).to(_type(s["out"]))


def _plain_ce(s):
    h, w, t = s["hidden"].float(), s["weight"].float(), s["targets"].long()
    valid = t != IGNORE
    t = torch.where(valid, t, torch.zeros_like(t))[:, None]
    z = h @ w.t()
    if s["T"] is not None:
        z = z / s["T"][:, None]
    m = z.max(dim=1, keepdim=True).values
    z_t = z.gather(1, t)
    e = torch.exp(z - m)
    total = e.sum(dim=1, keepdim=True)
    lse = m + torch.log(total)
    zero = torch.zeros_like(s["targets"], dtype=torch.float32)
    out = {"loss": torch.where(valid, (lse - z_t)[:, 0], zero), "lse": torch.where(valid, lse[:, 0], zero)}
    if not s["train"]:
        return out
    scale = s["grad_loss"] / s["T"] if s["T"] is not None else s["grad_loss"]
    scale = torch.where(valid, scale, zero)[:, None]
    p = e / total
    p = p.scatter_add(1, t, torch.full_like(p[:, :1], -1.0)) * scale
    out["dhidden"] = (p @ w).to(s["hidden"].dtype)
    if s["head"]:
        out["dweight"] = (p.t() @ h).to(s["weight"].dtype)
    return out


def run(state):
    s = state
    if own:
        import decode_step_token_row_amd as arcs
        if s["kind"] == "w4":
            return arcs.w4_logits(s["hidden"], s["qweight"], s["scale"], s["group"], zeros=s["zero"],
                                  out_dtype=_type(s["out"]))
        loss, lse = arcs.linear_cross_entropy(s["hidden"], s["weight"], s["targets"], temperature=s["T"],
                                              ignore_index=IGNORE)
        out = {"loss": loss, "lse": lse}
        if s["train"]:
            dh, dw = arcs.linear_cross_entropy_backward(
                s["hidden"], s["weight"], s["targets"], lse, s["grad_loss"], temperature=s["T"],
                ignore_index=IGNORE, want_weight=s["head"])
            out["dhidden"] = dh
            if s["head"]:
                out["dweight"] = dw
        return out
    return _plain_w4(s) if s["kind"] == "w4" else _plain_ce(s)


def work(case):
    c = case
    if c["kind"] == "w4":
        B, V, D, n = c["B"], c["V"], c["D"], c["D"] // c["group"]
        size = {"bf16": 2, "f32": 4}
        bytes_ = V * D // 2 + V * n * (size[c["scales"]] + (1 if c["zeros"] else 0))
        bytes_ += B * D * 2 + B * V * size[c["out"]]
        return {"bytes": bytes_, "flops": 2 * B * V * D}
    # ignored rows need no products; the logits are not kept, so a backward
    # pass computes them again
    N, V, D, size = _valid_rows(c), c["V"], c["D"], 2 if c["dtype"] == "bf16" else 4
    bytes_, products = V * D * size + N * D * size + c["N"] * 12, 1
    if c["train"]:
        bytes_ += c["N"] * D * size + c["N"] * 4 + (V * D * size if c["head"] else 0)
        products += 3 if c["head"] else 2
    return {"bytes": bytes_, "flops": 2 * products * N * V * D}


def exact(case, seed):
    """The definition in 64 bits, from the inputs alone."""
    s = prepare(case, seed)
    f8 = torch.float64
    if s["kind"] == "w4":
        V, D, n = s["V"], s["D"], s["D"] // s["group"]
        low, high = s["qweight"].bitwise_and(15), s["qweight"].bitwise_right_shift(4)
        level = torch.empty(V, D, dtype=f8, device=DEVICE)
        level[:, 0::2] = low.to(f8)
        level[:, 1::2] = high.to(f8)
        offset = s["zero"].to(f8) if s["zero"] is not None else torch.full((V, n), 8.0, dtype=f8, device=DEVICE)
        level -= offset.repeat_interleave(s["group"], dim=1)
        level *= s["scale"].to(f8).repeat_interleave(s["group"], dim=1)
        return torch.mm(level, s["hidden"].to(f8).t().contiguous()).t()
    rows = torch.nonzero(s["targets"] != IGNORE)[:, 0]
    h, w, t = s["hidden"][rows].to(f8), s["weight"].to(f8), s["targets"][rows].long()
    T = s["T"][rows].to(f8) if s["T"] is not None else torch.ones(len(rows), dtype=f8, device=DEVICE)
    z = torch.mm(w, h.t().contiguous()) / T  # [V, rows]
    lse = torch.logsumexp(z, dim=0)
    here = torch.arange(len(rows), device=DEVICE)

    def spread(x, *tail):
        full = torch.zeros((s["N"],) + tail, dtype=f8, device=DEVICE)
        full[rows] = x
        return full

    out = {"loss": spread(lse - z[t, here]), "lse": spread(lse)}
    if s["train"]:
        factor = s["grad_loss"][rows].to(f8) / T
        d = torch.exp(z - lse)
        d[t, here] -= 1.0
        d *= factor
        out["dhidden"] = spread(torch.mm(d.t().contiguous(), w), s["D"])
        if s["head"]:
            out["dweight"] = torch.mm(d, h)
    return out
