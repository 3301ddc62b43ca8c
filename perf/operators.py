"""The operators of an 8-bit mixture-of-experts layer, measured one pass at a time.

Five kinds of case, each one operator as a serving or training program calls it:

``quantize``  activations of 16 or 32 bits to int8 with one scale a token, in place or straight to
              the rows of their experts
``matmul``    Y = W . X in 8-bit integers with a scale for each token and channel; with ``E`` the
              tokens are sorted by expert and every expert has weights of its own
``dispatch``  tokens sorted by expert: positions and offsets from the chosen experts, rows moved
``combine``   the experts' outputs back in token order, weighted and summed, onto the shared
              expert's output where there is one
``backward``  the gradients of the last two

Sizes are those of the layers in ``workloads`` (a batch of 64 decode tokens, a prompt of 4096 or 8192,
widths 4096, 5120, 8192, 14336 and 16384, 128 experts) and ranges around them.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_handle = []


def listed():
    return [
        # one decode step's activations on their way into an 8-bit projection
        {"name": "quantize_decode", "op": "quantize", "T": 64, "K": 5120, "E": 0, "k": 0, "type": "bf16", "pad": 0, "drop": 0.0},
        # a prompt's activations quantised into their experts' rows
        {"name": "quantize_experts", "op": "quantize", "T": 8192, "K": 5120, "E": 128, "k": 1, "type": "bf16", "pad": 0, "drop": 0.0},
        # a dense layer's down projection for a single token
        {"name": "matmul_token", "op": "matmul", "T": 1, "M": 5120, "K": 16384, "E": 0, "k": 0, "type": "f16", "pad": 0, "drop": 0.0},
        # a dense layer's gate projection over a prompt
        {"name": "matmul_prompt", "op": "matmul", "T": 4096, "M": 14336, "K": 4096, "E": 0, "k": 0, "type": "bf16", "pad": 0, "drop": 0.0},
        # the experts' gate projections in a decode step of 64 requests: few tokens an expert
        {"name": "experts_decode", "op": "matmul", "T": 64, "M": 8192, "K": 5120, "E": 128, "k": 1, "type": "bf16", "pad": 0, "drop": 0.0},
        # the same over a prompt: ragged groups of a few to hundreds of tokens
        {"name": "experts_prompt", "op": "matmul", "T": 8192, "M": 8192, "K": 5120, "E": 128, "k": 1, "type": "bf16", "pad": 0, "drop": 0.0},
        # one token to its eight experts: nothing but latency
        {"name": "dispatch_token", "op": "dispatch", "T": 1, "K": 5120, "E": 128, "k": 8, "type": "bf16", "pad": 0, "drop": 0.0},
        # a training batch with padded tokens that go nowhere
        {"name": "dispatch_train", "op": "dispatch", "T": 8191, "K": 5120, "E": 128, "k": 2, "type": "bf16", "pad": 0, "drop": 0.03},
        # a decode step's expert outputs onto the shared expert's
        {"name": "combine_decode", "op": "combine", "T": 64, "K": 5120, "E": 128, "k": 1, "type": "bf16", "pad": 0, "drop": 0.0, "base": True},
        # a prompt's, in rows of an odd width
        {"name": "combine_prompt", "op": "combine", "T": 8192, "K": 4099, "E": 128, "k": 2, "type": "f32", "pad": 0, "drop": 0.0, "base": False},
        # the gradients of a small layer
        {"name": "backward_small", "op": "backward", "T": 128, "K": 256, "E": 4, "k": 2, "type": "f16", "pad": 0, "drop": 0.1},
        # and of a whole training batch
        {"name": "backward_train", "op": "backward", "T": 8192, "K": 5120, "E": 128, "k": 2, "type": "bf16", "pad": 0, "drop": 0.0},
    ]


def draw(rng):
    def size(lo, hi, step=1):  # evenly over the logarithm; a quarter of them odd where step allows
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if step > 1 and rng.random() < 0.75:
            n = max(1, n // step) * step
        return min(hi, max(lo, n))

    c = {"op": rng.choice(["quantize", "matmul", "matmul", "dispatch", "combine", "backward"])}
    c["T"] = size(1, 8192)
    c["K"] = size(64, 16384, 16)
    c["E"] = size(1, 256)
    c["k"] = rng.randint(1, min(8, c["E"]))
    if c["op"] in ("quantize", "matmul") and rng.random() < 0.5:
        c["E"] = c["k"] = 0
    if c["op"] == "matmul":
        # no more weights and products than the largest listed case
        c["M"] = size(64, 16384, 16)
        c["k"] = min(1, c["k"])
        while c["E"] * c["M"] * c["K"] > 128 * 8192 * 5120:
            c["E"] = (c["E"] + 1) // 2
        while c["T"] * c["M"] * c["K"] > 8192 * 8192 * 5120:
            c["T"] = (c["T"] + 1) // 2
    else:
        while c["T"] * max(1, c["k"]) * c["K"] > 8192 * 2 * 5120:
            c["T"] = (c["T"] + 1) // 2
    c["type"] = rng.choice(["f32", "f16", "bf16"])
    c["pad"] = rng.choice([0, 0, 16, 3])  # rows that are part of wider ones
    c["drop"] = rng.choice([0.0, 0.1]) if c["E"] else 0.0
    if c["op"] == "combine":
        c["base"] = rng.random() < 0.5
    return c


def _rows(n, width, pad, dtype, fill=None):
    """n rows of `width` values in rows of width + pad."""
    b = torch.zeros(n, width + pad, dtype=dtype, device="cuda")
    if fill is not None:
        b[:, :width] = fill
    return b[:, :width]


def _activations(g, T, K):
    """Activations as a layer's input has them: a spread of its own for every token, and a few
    channels that are far larger than the rest."""
    x = torch.randn(T, K, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device="cuda"))
    x *= torch.where(torch.rand(1, K, generator=g, device="cuda") < 0.005, 20.0, 1.0)
    return x


def _route(g, T, k, E, drop):
    """Each token's k experts by the largest of its logits, some experts more popular than others;
    tokens of padding go to none (-1)."""
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.2 * torch.randn(1, E, generator=g, device="cuda")
    w, e = logits.topk(k, dim=1)
    e = torch.where(torch.rand(T, 1, generator=g, device="cuda") < drop, -1, e).to(torch.int32)
    return e.contiguous(), torch.softmax(w, dim=1).contiguous()


def _positions(e, E):
    """Where each choice's row goes: by expert, then in the order of the choices; -1 for none."""
    n = e.numel()
    key = torch.where(e.reshape(-1) < 0, E, e.reshape(-1)).long()
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(n, device=e.device)
    pos = torch.where(key < E, place, -1).to(torch.int32).reshape(e.shape)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=e.device)
    counts.index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=e.device)
    offsets[1:] = counts[:E].cumsum(0).to(torch.int32)
    return offsets, pos


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, T, K, E, k, pad = case["op"], case["T"], case["K"], case["E"], case["k"], case["pad"]
    dt = TYPES[case["type"]]
    s = {"op": op, "E": E, "k": k}
    if E:
        e, s["weights"] = _route(g, T, k, E, case["drop"])
        offsets, pos = _positions(e, E)
    R = T * k if E else T
    if op == "quantize":
        s["x"] = _rows(T, K, pad, dt, _activations(g, T, K))
        s["pos"] = pos if E else None
        s["q"] = torch.zeros(R, K, dtype=torch.int8, device="cuda")
        s["scale"] = torch.zeros(R, device="cuda")
    elif op == "matmul":
        M = case["M"]
        s["w"] = torch.randint(-128, 128, (E, M, K) if E else (M, K), generator=g, device="cuda", dtype=torch.int8)
        s["w_scale"] = 1e-3 * torch.exp(0.3 * torch.randn((E, M) if E else (M,), generator=g, device="cuda"))
        s["x"] = _rows(R, K, pad, torch.int8, (32 * torch.randn(R, K, generator=g, device="cuda")).round().clamp(-127, 127).to(torch.int8))
        s["x_scale"] = 0.02 * torch.exp(0.5 * torch.randn(R, generator=g, device="cuda"))
        s["offsets"] = offsets if E else None
        s["y"] = torch.zeros(R, M, dtype=dt, device="cuda")
    elif op == "dispatch":
        s["e"] = e
        s["x"] = _rows(T, K, pad, dt, _activations(g, T, K))
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["pos"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        s["rows"] = torch.zeros(R, K, dtype=dt, device="cuda")
    else:
        s["pos"] = pos
        s["rows"] = _rows(R, K, pad, dt, _activations(g, R, K))
        if op == "combine":
            s["base"] = _activations(g, T, K).to(dt) if case["base"] else None
            s["out"] = torch.zeros(T, K, dtype=dt, device="cuda")
        else:
            s["dout"] = _rows(T, K, pad, dt, 0.1 * torch.randn(T, K, generator=g, device="cuda"))
            s["dinput"] = _rows(R, K, pad, dt, 0.1 * torch.randn(R, K, generator=g, device="cuda"))
            s["drows"] = torch.zeros(R, K, dtype=dt, device="cuda")
            s["dweights"] = torch.zeros(T, k, device="cuda")
            s["dx"] = torch.zeros(T, K, dtype=dt, device="cuda")
    return s


def _context():
    if not _handle:
        import sum_check_prover_b200 as fp

        _handle.append(fp.Context(torch.cuda.current_device()))
    return _handle[0]


def run(s):
    op = s["op"]
    if own:
        ctx = _context()
        if op == "quantize":
            ctx.quantize_rows(s["x"], s["q"], s["scale"], pos=s["pos"])
            return s["q"], s["scale"]
        if op == "matmul":
            ctx.matmul_i8(s["w"], s["x"], s["y"], s["w_scale"], s["x_scale"], offsets=s["offsets"])
            return s["y"]
        if op == "dispatch":
            ctx.moe_sort(s["e"], s["E"], s["offsets"], s["pos"])
            ctx.moe_dispatch(s["x"], s["pos"], s["rows"])
            return s["offsets"], s["pos"], s["rows"]
        if op == "combine":
            ctx.moe_combine(s["rows"], s["pos"], s["out"], weights=s["weights"], base=s["base"])
            return s["out"]
        ctx.moe_combine_grad(s["dout"], s["rows"], s["pos"], s["weights"], s["drows"], s["dweights"])
        ctx.moe_combine(s["dinput"], s["pos"], s["dx"])
        return s["drows"], s["dweights"], s["dx"]

    if op == "quantize":
        # 64 bits: a value halfway between two integers has to be seen as that
        x, pos = s["x"].double(), s["pos"]
        amax = x.abs().amax(dim=1, keepdim=True)
        q = torch.where(amax > 0, x * 127.0 / amax, 0.0).round().to(torch.int8)
        scale = (amax / 127.0).float()[:, 0]
        if pos is None:
            return q, scale
        return _scatter(q, pos, torch.zeros_like(s["q"])), _scatter(scale, pos, torch.zeros_like(s["scale"]))
    if op == "matmul":
        w, x, ws, xs, off = s["w"], s["x"].float(), s["w_scale"], s["x_scale"], s["offsets"]
        if off is None:
            return ((x @ w.float().T) * xs[:, None] * ws).to(s["y"].dtype)
        # every expert's rows padded to the largest group, one batched product
        E, R = s["E"], x.shape[0]
        counts = off[1:] - off[:-1]
        most = max(1, int(counts.max()))
        idx = off[:-1, None] + torch.arange(most, device=x.device)
        idx = torch.where(torch.arange(most, device=x.device) < counts[:, None], idx, R).long()
        padded = torch.cat([x * xs[:, None], x.new_zeros(1, x.shape[1])])[idx]
        y = torch.bmm(padded, w.float().transpose(1, 2)) * ws[:, None, :]
        out = torch.zeros(R + 1, w.shape[1], dtype=s["y"].dtype, device=x.device)
        out[idx] = y.to(out.dtype)
        return out[:R]
    if op == "dispatch":
        offsets, pos = _positions(s["e"], s["E"])
        return offsets, pos, _scatter(s["x"], pos, torch.zeros_like(s["rows"]))
    pos, w = s["pos"], s["weights"]
    if op == "combine":
        out = (_gather(s["rows"], pos) * w[:, :, None]).sum(dim=1)
        return (out if s["base"] is None else out + s["base"].float()).to(s["out"].dtype)
    dout = s["dout"].float()
    drows = _scatter((dout[:, None] * w[:, :, None]).to(s["drows"].dtype).flatten(0, 1), pos.reshape(-1, 1), torch.zeros_like(s["drows"]))
    dweights = (_gather(s["rows"], pos) * dout[:, None]).sum(dim=2)
    dx = _gather(s["dinput"], pos).sum(dim=1).to(s["dx"].dtype)
    return drows, dweights, dx


def _scatter(x, pos, out):
    """out with row t of x at its positions."""
    keep = pos >= 0
    src = torch.arange(pos.shape[0], device=pos.device)[:, None].expand(pos.shape)
    out[pos[keep].long()] = x[src[keep]]
    return out


def _gather(rows, pos):
    """The rows at the positions in 32 bits, nothing where there is none."""
    return torch.where((pos >= 0)[:, :, None], rows[pos.clamp(min=0).long()].float(), 0.0)


def work(case):
    op, T, K, E, k = case["op"], case["T"], case["K"], case["E"], case["k"]
    size = torch.finfo(TYPES[case["type"]]).bits // 8
    n = T * k if E else T
    kept = n * (1 - case["drop"])  # rows that are moved
    if op == "quantize":
        return {"bytes": T * K * size + kept * (K + 4) + (4 * n if E else 0), "flops": 3 * T * K}
    if op == "matmul":
        M = case["M"]
        # the expected number of experts with a token, were they chosen evenly
        used = E * (1 - (1 - 1 / E) ** kept) if E else 1
        return {"bytes": used * M * (K + 4) + kept * (K + 4) + kept * M * size, "flops": 2 * kept * M * K}
    if op == "dispatch":
        return {"bytes": 8 * n + 4 * E + (1 - case["drop"]) * T * K * size + kept * K * size, "flops": n}
    if op == "combine":
        return {"bytes": 8 * n + kept * K * size + T * K * size * (2 if case["base"] else 1), "flops": 2 * kept * K}
    # dout and the rows read, their gradients written; the rows' other gradients read, dx written
    return {"bytes": 12 * n + 2 * T * K * size + 3 * kept * K * size, "flops": 4 * kept * K}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        x = s["x"].double()
        top = torch.maximum(x.max(1).values, -x.min(1).values)
        safe = torch.where(top > 0, top, 1.0)
        q = torch.round(127 * x / safe[:, None])
        scale = top / 127
        if s["pos"] is not None:
            token, _, at = _choices(s["pos"])
            q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda").index_copy_(0, at, q[token])
            scale = torch.zeros(s["scale"].shape, dtype=torch.float64, device="cuda").index_copy_(0, at, scale[token])
        return q.to(torch.int8), scale
    if op == "matmul":
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        ends = [0, y.shape[0]] if s["offsets"] is None else s["offsets"].tolist()
        w, ws = s["w"].reshape(-1, *s["w"].shape[-2:]), s["w_scale"].reshape(-1, s["w"].shape[-2]).double()
        for i, (a, b) in enumerate(zip(ends, ends[1:])):
            if a < b:
                y[a:b] = torch.einsum("nk,mk->nm", s["x"][a:b].double(), w[i].double()) * ws[i] * s["x_scale"][a:b, None].double()
        return y
    if op == "dispatch":
        e = s["e"].reshape(-1).long()
        offsets = torch.stack([((e >= 0) & (e < j)).sum() for j in range(s["E"] + 1)]).to(torch.int32)
        pos = torch.full_like(e, -1)
        for j in range(s["E"]):
            mine = (e == j).nonzero()[:, 0]
            pos[mine] = offsets[j] + torch.arange(len(mine), device="cuda")
        pos = pos.reshape(s["e"].shape).to(torch.int32)
        token, _, at = _choices(pos)
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda").index_copy_(0, at, s["x"][token].double())
        return offsets, pos, rows
    token, choice, at = _choices(s["pos"])
    w = s["weights"][token, choice].double()[:, None]
    if op == "combine":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda") if s["base"] is None else s["base"].double()
        return out.index_add_(0, token, w * s["rows"][at].double())
    g = s["dout"].double()[token]
    drows = torch.zeros(s["drows"].shape, dtype=torch.float64, device="cuda").index_copy_(0, at, w * g)
    dweights = torch.zeros(s["dweights"].shape, dtype=torch.float64, device="cuda")
    dweights[token, choice] = torch.einsum("nk,nk->n", g, s["rows"][at].double())
    dx = torch.zeros(s["dx"].shape, dtype=torch.float64, device="cuda").index_add_(0, token, s["dinput"][at].double())
    return drows, dweights, dx


def _choices(pos):
    """(token, choice, row) of every choice that has a row."""
    token, choice = (pos >= 0).nonzero(as_tuple=True)
    return token, choice, pos[token, choice].long()
