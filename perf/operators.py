"""What is measured of the routing and adapter operators: their cases, inputs, plain forms and exact values.

Five operators beside the quantised-weight GEMMs:

``dispatch``      tokens sorted by expert (a stable counting sort of the expert ids) and copied into that order
``combine``       the experts' rows back in token order, weighted and summed, with an optional addend
``combine_grad``  the gradient of ``combine`` for the experts' rows and the weights
``lora``          low-rank adapters of many requests beside a shared projection: out = y + s (x A^T) B^T by row
``lora_grad``     its gradient for x, A and B

``own`` false: plain torch operations in 32 bits.  ``own`` true: the calls a user makes of the package.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a small batch: launch latency and little else
        dict(name="dispatch_decode", op="dispatch", tokens=16, top=2, experts=64, hidden=4096, dtype="bf16", drop=0.0),
        # expert parallelism: a rank holds some of the experts and drops the other tokens' copies
        dict(name="dispatch_ragged", op="dispatch", tokens=1027, top=6, experts=160, hidden=1024, dtype="f16", drop=0.2),
        # a long prompt batch: the copy bound by memory
        dict(name="dispatch_prompt", op="dispatch", tokens=8192, top=4, experts=64, hidden=8192, dtype="bf16", drop=0.0),
        dict(name="combine_decode", op="combine", tokens=16, top=2, experts=64, hidden=4096, dtype="bf16", drop=0.0,
             addend=False),
        # a prompt batch whose result joins a shared expert's output
        dict(name="combine_prompt", op="combine", tokens=4096, top=4, experts=64, hidden=8192, dtype="bf16", drop=0.0,
             addend=True),
        dict(name="combine_grad_ragged", op="combine_grad", tokens=1027, top=6, experts=160, hidden=1024, dtype="f16",
             drop=0.2),
        dict(name="combine_grad_batch", op="combine_grad", tokens=4096, top=4, experts=64, hidden=4096, dtype="bf16",
             drop=0.0),
        # sixteen requests decode one token each, beside a wide up projection
        dict(name="lora_decode", op="lora", rows=16, k=8192, n=28672, rank=16, adapters=16, requests=16, dtype="bf16",
             bare=0.1),
        # a few prompts at once
        dict(name="lora_prompt", op="lora", rows=4096, k=4096, n=4096, rank=16, adapters=4, requests=6, dtype="bf16",
             bare=0.1),
        # many requests, short prompts and single tokens mixed, a larger rank
        dict(name="lora_ragged", op="lora", rows=1043, k=4096, n=1024, rank=64, adapters=24, requests=40, dtype="f16",
             bare=0.1),
        # training one adapter
        dict(name="lora_grad_one", op="lora_grad", rows=4096, k=4096, n=4096, rank=16, adapters=1, requests=4,
             dtype="bf16", bare=0.0),
        # training several adapters at once
        dict(name="lora_grad_ragged", op="lora_grad", rows=2051, k=8192, n=1024, rank=64, adapters=6, requests=11,
             dtype="f16", bare=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


#: a drawn case moves no more than the largest listed one
_MOST_BYTES = 6.0e8


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "lora", "lora_grad"])
    dtype = rng.choice(["bf16", "f16"])
    while True:
        if op in ("lora", "lora_grad"):
            rows = _log(rng, 1, 8192)
            case = dict(op=op, rows=rows, k=32 * _log(rng, 8, 256), n=32 * _log(rng, 8, 896 if rows <= 512 else 256),
                        rank=rng.choice([8, 16, 16, 24, 32, 64, 128]),
                        adapters=_log(rng, 1, 64) if op == "lora" else _log(rng, 1, 16),
                        requests=rng.randint(1, min(rows, 96)), dtype=dtype, bare=rng.choice([0.0, 0.1, 0.5]))
        else:
            case = dict(op=op, tokens=_log(rng, 1, 8192), top=rng.randint(1, 8), experts=_log(rng, 2, 256),
                        hidden=8 * _log(rng, 32, 1024) + (rng.randint(1, 7) if rng.random() < 0.2 else 0), dtype=dtype,
                        drop=rng.choice([0.0, 0.0, 0.2, 0.9]))
            if op == "combine":
                case["addend"] = rng.random() < 0.5
        w = work(case)
        if w["bytes"] <= _MOST_BYTES and w["flops"] <= 5e10:
            return case


def work(case):
    e = 2
    if case["op"] in ("lora", "lora_grad"):
        m, k, n, r = case["rows"], case["k"], case["n"], case["rank"]
        with_one = 1 - case["bare"]
        used = case["adapters"] * (1 - (1 - with_one / case["adapters"]) ** case["requests"])
        flops = 2 * m * with_one * r * (k + n)
        weights = used * r * (k + n) * e
        if case["op"] == "lora":
            return {"bytes": m * with_one * k * e + weights + 2 * m * n * e, "flops": flops}
        given = case["adapters"] * r * (k + n) * e
        return {"bytes": m * with_one * (k + n) * e + weights + given + 2 * m * k * e, "flops": 3 * flops}
    t, j, h = case["tokens"], case["top"], case["hidden"]
    valid = t * j * (1 - case["drop"])
    if case["op"] == "dispatch":
        return {"bytes": t * h * e + valid * h * e + t * j * (8 + 8) + 4 * case["experts"], "flops": 0}
    if case["op"] == "combine":
        return {"bytes": valid * h * e + t * h * e * (2 if case["addend"] else 1) + t * j * 8, "flops": 2 * valid * h}
    return {"bytes": t * h * e + 2 * valid * h * e + t * j * 12, "flops": 3 * valid * h}


# ------------------------------------------------------------------------------------------------ inputs
def _order(ids, groups):
    """The stable order of the slots by group, those of no group behind: offsets, source and position, as the
    program that routes the tokens holds them."""
    flat = ids.reshape(-1).long()
    valid = (flat >= 0) & (flat < groups)
    key = torch.where(valid, flat, groups)
    by, source = torch.sort(key, stable=True)
    position = torch.empty_like(source)
    position[source] = torch.arange(source.numel(), device=ids.device)
    position = torch.where(valid, position, -1)
    offsets = torch.searchsorted(by, torch.arange(groups + 1, device=ids.device))
    return offsets.int(), source.int(), position.int().reshape(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case)
    if case["op"] in ("lora", "lora_grad"):
        m, k, n, r, count = case["rows"], case["k"], case["n"], case["rank"], case["adapters"]
        # the requests' lengths: rows dealt at random cuts; each has one adapter or none
        requests = case["requests"]
        cuts = torch.randperm(max(m - 1, 1), generator=g, device="cuda")[:requests - 1] + 1
        starts = torch.zeros(m, dtype=torch.long, device="cuda")
        starts[cuts[cuts < m]] = 1
        of = torch.randint(0, count, (requests,), generator=g, device="cuda")
        bare = torch.rand(requests, generator=g, device="cuda") < case["bare"]
        s["ids"] = torch.where(bare, -1, of)[starts.cumsum(0)].int()
        s["x"] = normal(m, k)
        s["a"] = normal(count, r, k, std=k ** -0.5)
        s["b"] = normal(count, n, r, std=0.05)
        s["scale"] = torch.rand(count, generator=g, device="cuda") * 1.5 + 0.5
        if case["op"] == "lora":
            s["y"] = normal(m, n)
        else:
            s["grad"] = normal(m, n, std=0.1)
            s["grad_x"] = normal(m, k, std=0.1)
        s["offsets"], s["source"], s["position"] = _order(s["ids"], count)
        return s
    t, j, h, experts = case["tokens"], case["top"], case["hidden"], case["experts"]
    # a router's choice: distinct experts of each token where there are enough, popular ones more often
    liking = torch.rand(experts, generator=g, device="cuda") * 2
    ids = (torch.rand(t, experts, generator=g, device="cuda") + liking * 0.2).topk(min(j, experts), dim=1).indices
    if j > experts:
        ids = torch.cat([ids, torch.randint(0, experts, (t, j - experts), generator=g, device="cuda")], 1)
    ids = torch.where(torch.rand(t, j, generator=g, device="cuda") < case["drop"], -1, ids)
    weights = torch.rand(t, j, generator=g, device="cuda") + 0.05
    s["weights"] = weights / weights.sum(1, keepdim=True)
    if case["op"] == "dispatch":
        s["ids"] = ids
        s["x"] = normal(t, h)
        s["out"] = torch.zeros(t * j, h, dtype=dtype, device="cuda")  # rows of no expert stay as they are
        return s
    s["offsets"], s["source"], s["position"] = _order(ids, experts)
    s["x_sorted"] = normal(t * j, h)
    if case["op"] == "combine":
        s["x3"] = normal(t, h) if case["addend"] else None
    else:
        s["grad"] = normal(t, h, std=0.1)
        s["grad_sorted"] = torch.zeros(t * j, h, dtype=dtype, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from weight_quantized_gemm_anti_b200 import lora, routing

    if s["op"] == "dispatch":
        order = routing.sort_tokens(s["ids"], s["experts"])
        rows = routing.dispatch_tokens(s["x"], order, out=s["out"])
        return {"rows": rows, "offsets": order.offsets, "source": order.source, "position": order.position}
    order = routing.TokenOrder(s["offsets"], s["source"], s["position"])
    if s["op"] == "combine":
        return routing.combine_tokens(s["x_sorted"], order, s["weights"], x3=s["x3"])
    if s["op"] == "combine_grad":
        rows, weights = routing.combine_tokens_grad(s["grad"], s["x_sorted"], order, s["weights"],
                                                    out=s["grad_sorted"])
        return {"rows": rows, "weights": weights}
    if s["op"] == "lora":
        return lora.lora_add(s["x"], s["a"], s["b"], order, s["scale"], y=s["y"])
    x, a, b = lora.lora_grad(s["grad"], s["x"], s["a"], s["b"], order, s["scale"], grad_x=s["grad_x"])
    return {"x": x, "a": a, "b": b}


def _plain(s):
    op = s["op"]
    if op == "dispatch":
        offsets, source, position = _order(s["ids"], s["experts"])
        out, slot = s["out"], source.long()
        has = (position.reshape(-1)[slot] >= 0)[:, None]  # the rows behind the last expert stay as they are
        torch.where(has, s["x"][slot // s["top"]], out, out=out)
        return {"rows": out, "offsets": offsets, "source": source, "position": position}
    if op == "combine":
        position = s["position"].long()
        w = torch.where(position >= 0, s["weights"], 0.0)
        rows = s["x_sorted"][position.clamp(min=0)].float()
        y = torch.where((position >= 0)[..., None], rows * w[..., None], 0.0).sum(1)
        return (y if s["x3"] is None else y + s["x3"].float()).to(s["x_sorted"].dtype)
    if op == "combine_grad":
        position = s["position"].long()
        has = position >= 0
        grad = s["grad"].float()
        rows = s["x_sorted"][position.clamp(min=0)].float()
        weights = torch.where(has, (rows * grad[:, None]).sum(2), 0.0)
        slot, out = s["source"].long(), s["grad_sorted"]
        of = grad[slot // s["top"]] * s["weights"].reshape(-1)[slot][:, None]
        torch.where(has.reshape(-1)[slot][:, None], of.to(out.dtype), out, out=out)
        return {"rows": s["grad_sorted"], "weights": weights}
    # adapters: every adapter's products side by side, and of each row only its own adapter's kept
    count, r = s["adapters"], s["rank"]
    ids = s["ids"].long()
    mine = (ids[:, None] == torch.arange(count, device=ids.device)).repeat_interleave(r, 1)
    scale = s["scale"].repeat_interleave(r)
    x, a = s["x"].float(), s["a"].float().reshape(count * r, -1)
    h = torch.where(mine, (x @ a.T) * scale, 0.0)
    b = s["b"].float().transpose(1, 2).reshape(count * r, -1)
    if op == "lora":
        return (s["y"].float() + h @ b).to(s["y"].dtype)
    grad, dtype = s["grad"].float(), s["x"].dtype
    g = torch.where(mine, (grad @ b.T) * scale, 0.0)
    grad_b = (h.T @ grad).reshape(count, r, -1).transpose(1, 2).contiguous()
    return {"x": (s["grad_x"].float() + g @ a).to(dtype), "a": (g.T @ x).reshape(s["a"].shape).to(dtype),
            "b": grad_b.to(dtype)}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("lora", "lora_grad"):
        x, ids = s["x"].double(), s["ids"].tolist()
        rows_of = [[i for i, v in enumerate(ids) if v == c] for c in range(case["adapters"])]
        if case["op"] == "lora":
            out = s["y"].double()
        else:
            grad, out = s["grad"].double(), s["grad_x"].double()
            da, db = torch.zeros_like(s["a"], dtype=torch.float64), torch.zeros_like(s["b"], dtype=torch.float64)
        for c, rows in enumerate(rows_of):
            if not rows:
                continue
            at = torch.tensor(rows, device=x.device)
            a, b, f = s["a"][c].double(), s["b"][c].double(), float(s["scale"][c])
            low = torch.einsum("mk,rk->mr", x[at], a)
            if case["op"] == "lora":
                out[at] += f * torch.einsum("mr,nr->mn", low, b)
            else:
                back = f * torch.einsum("mn,nr->mr", grad[at], b)
                out[at] += torch.einsum("mr,rk->mk", back, a)
                da[c] = torch.einsum("mr,mk->rk", back, x[at])
                db[c] = f * torch.einsum("mn,mr->nr", grad[at], low)
        return out if case["op"] == "lora" else {"x": out, "a": da, "b": db}
    top = case["top"]
    if case["op"] == "dispatch":
        ids = s["ids"].reshape(-1).tolist()
        by = [[] for _ in range(case["experts"])]
        none = []
        for slot, e in enumerate(ids):
            (by[e] if 0 <= e < case["experts"] else none).append(slot)
        offsets, source, position = [0], [], [-1] * len(ids)
        for slots in by:
            for slot in slots:
                position[slot] = len(source)
                source.append(slot)
            offsets.append(len(source))
        out = torch.zeros(len(ids), case["hidden"], dtype=torch.float64, device="cuda")
        if source:
            out[:len(source)] = s["x"].double()[torch.tensor(source, device="cuda") // top]
        whole = [torch.tensor(v, dtype=torch.int32) for v in (offsets, source + none, position)]
        return {"rows": out, "offsets": whole[0], "source": whole[1], "position": whole[2].reshape(-1, top)}
    slots, xs = s["position"].tolist(), s["x_sorted"].double()
    if case["op"] == "combine":
        y = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
        if s["x3"] is not None:
            y += s["x3"].double()
        for j in range(top):
            t = torch.tensor([i for i, p in enumerate(slots) if p[j] >= 0], dtype=torch.long, device="cuda")
            at = torch.tensor([p[j] for p in slots if p[j] >= 0], dtype=torch.long, device="cuda")
            y[t] += s["weights"].double()[t, j][:, None] * xs[at]
        return y
    grad = s["grad"].double()
    rows, weights = torch.zeros_like(xs), torch.zeros_like(s["weights"], dtype=torch.float64)
    for j in range(top):
        t = torch.tensor([i for i, p in enumerate(slots) if p[j] >= 0], dtype=torch.long, device="cuda")
        at = torch.tensor([p[j] for p in slots if p[j] >= 0], dtype=torch.long, device="cuda")
        rows[at] = s["weights"].double()[t, j][:, None] * grad[t]
        weights[t, j] = torch.einsum("th,th->t", grad[t], xs[at])
    return {"rows": rows, "weights": weights}
