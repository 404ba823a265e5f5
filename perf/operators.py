"""The decode loop's operators around token selection, as measured cases.

Three operators: the 4-bit output head (hidden states to logits rows), sampling
of 16-bit logits rows with a policy for each row, and the embedding lookup of
the drawn ids. `run` computes them in elementary torch operations, or, where
`own` is set, through the library's binding.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # A drafter's head, one token: the smallest call, where latency counts.
        head("head_draft_1row", rows=1, V=151936, H=1024, group=64, zeros=False, dtype="bf16", out="f32"),
        # Plain decoding of one sequence.
        head("head_decode_1row", rows=1, V=248320, H=4096, group=128, zeros=False, dtype="bf16", out="f32"),
        # A few sequences, an odd vocabulary slice (one shard's columns), a width that is not a power of two.
        head("head_shard_5rows", rows=5, V=93001, H=2880, group=32, zeros=True, dtype="f16", out="f32"),
        # The verify batch: every draft position of 7 x 7 in one call.
        head("head_verify_49rows", rows=49, V=248320, H=4096, group=64, zeros=False, dtype="bf16", out="f32"),
        # A full decode batch on a wide model, 16-bit logits.
        head("head_batch_64rows", rows=64, V=202048, H=8192, group=128, zeros=True, dtype="f16", out="f16"),
        # One request's token.
        sample("sample_1row", rows=1, V=151936, pad=0, dtype="bf16", masked=0.0),
        # A few requests under a grammar: most ids masked, an odd width inside padded rows.
        sample("sample_grammar_7rows", rows=7, V=93001, pad=23, dtype="f16", masked=0.9),
        # The verify batch's rows.
        sample("sample_verify_49rows", rows=49, V=248320, pad=0, dtype="bf16", masked=0.0),
        # A large serving batch, a policy for each request.
        sample("sample_batch_256rows", rows=256, V=202048, pad=0, dtype="bf16", masked=0.0),
        # The drawn ids of one step, from the tied 4-bit table.
        embed("embed_w4_49ids", n=49, V=248320, H=4096, group=64, zeros=False, dtype="bf16"),
        # A step of a small fp32 model, odd width.
        embed("embed_f32_7ids", n=7, V=32001, H=2049, group=0, zeros=False, dtype="f32"),
        # A prompt's tokens.
        embed("embed_prompt_16384ids", n=16384, V=151936, H=5120, group=0, zeros=False, dtype="bf16"),
    ]


def head(name, **kw):
    return {"name": name, "op": "head", **kw}


def sample(name, **kw):
    return {"name": name, "op": "sample", **kw}


def embed(name, **kw):
    return {"name": name, "op": "embed", **kw}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["head", "sample", "embed"])
    if op == "head":
        group = rng.choice([32, 64, 128])
        H = max(1, _log(rng, 512, 8192) // group) * group
        return {"op": op, "rows": _log(rng, 1, 64), "V": _log(rng, 2000, 170000), "H": H, "group": group,
                "zeros": rng.random() < 0.5, "dtype": rng.choice(["f16", "bf16"]),
                "out": rng.choice(["f32", "f32", "f16", "bf16"])}
    if op == "sample":
        return {"op": op, "rows": _log(rng, 1, 200), "V": _log(rng, 1000, 248320), "pad": rng.choice([0, 0, 1, 8, 57]),
                "dtype": rng.choice(["f16", "bf16"]), "masked": rng.choice([0.0, 0.0, 0.5, 0.99])}
    group = rng.choice([0, 0, 32, 64, 128])
    H = _log(rng, 256, 8192)
    H = max(1, H // group) * group if group else H
    return {"op": op, "n": _log(rng, 1, 8192), "V": _log(rng, 1000, 151936), "H": H, "group": group,
            "zeros": bool(group) and rng.random() < 0.5,
            "dtype": rng.choice(["f16", "bf16"] if group else ["f32", "f16", "bf16"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _weights(case, g, dev, spread):
    """4-bit rows, group scales and zero points of a [V, H] matrix with entries of about N(0, spread^2)."""
    V, H, group = case["V"], case["H"], case["group"]
    q = torch.randint(0, 256, (V, H // 2), generator=g, device=dev, dtype=torch.uint8)
    s = torch.rand((V, H // group), generator=g, device=dev) * 0.8 + 0.6
    s = (s * (spread / 4.6)).to(TYPES[case["dtype"]])
    z = None
    if case["zeros"]:
        z = torch.randint(5, 11, (V, H // group), generator=g, device=dev, dtype=torch.uint8)
    return q, s, z


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"case": dict(case)}
    if case["op"] == "head":
        rows, V, H, dt = case["rows"], case["V"], case["H"], TYPES[case["dtype"]]
        s["q"], s["scales"], s["zeros"] = _weights(case, g, dev, 3.0 / math.sqrt(H))
        x = torch.randn((rows, H), generator=g, device=dev)
        x[:, torch.randint(0, H, (4,), generator=g, device=dev)] *= 6.0  # the few large channels of hidden states
        s["hidden"] = x.to(dt)
        s["logits"] = torch.empty((rows, V), dtype=TYPES[case["out"]], device=dev)
    elif case["op"] == "sample":
        rows, V = case["rows"], case["V"]
        x = torch.randn((rows, V + case["pad"]), generator=g, device=dev) * 3.0
        # every other row: Zipf(1.1) log-probabilities with Gumbel noise, as a peaked model gives
        rank = torch.randperm(V, generator=g, device=dev).float() + 1.0
        e = torch.rand((rows, V), generator=g, device=dev).clamp_(min=1e-30)
        zipf = -1.1 * torch.log(rank) - torch.log(-torch.log(e)) + 4.0
        x[1::2, :V] = zipf[1::2]
        if case["masked"] > 0:
            x[:, :V].masked_fill_(torch.rand((rows, V), generator=g, device=dev) < case["masked"], -math.inf)
            x[:, V // 2] = 1.0  # a grammar state always leaves something
        s["rows"] = x.to(TYPES[case["dtype"]])
        pick = torch.rand((5, rows), generator=g, device=dev)
        s["temperature"] = torch.where(pick[0] < 0.1, 0.0, 0.4 + pick[1])
        ks = torch.tensor([0, 0, 1, 20, 40, 84, 1000, 5000], device=dev, dtype=torch.int32)
        s["top_k"] = ks[torch.randint(0, 8, (rows,), generator=g, device=dev)]
        s["top_p"] = torch.where(pick[2] < 0.3, 1.0, 0.5 + 0.49 * pick[3])
        s["min_p"] = torch.where(pick[4] < 0.5, 0.0, 0.1 * pick[4])
        s["u"] = torch.rand((rows,), generator=g, device=dev)
        s["ids"] = torch.empty((rows,), dtype=torch.int32, device=dev)
        s["probs"] = torch.empty((rows,), dtype=torch.float32, device=dev)
    else:
        n, V, H, dt = case["n"], case["V"], case["H"], TYPES[case["dtype"]]
        if case["group"]:
            s["q"], s["scales"], s["zeros"] = _weights(case, g, dev, 0.05)
        else:
            s["table"] = (torch.randn((V, H), generator=g, device=dev) * 0.05).to(dt)
        ids = torch.randint(0, V, (n,), generator=g, device=dev, dtype=torch.int32)
        # places behind a sequence's last accepted token hold the invalid id
        s["ids"] = torch.where(torch.rand((n,), generator=g, device=dev) < 0.1, -1, ids).to(torch.int32)
        s["scale"] = float(np.float32(math.sqrt(H)))
        s["out"] = torch.empty((n, H), dtype=dt, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _dequantised(q, scales, zeros, group):
    rows, half = q.shape
    w = torch.stack((q & 15, q >> 4), dim=2).view(rows, 2 * half // group, group).float()
    w -= zeros.float()[:, :, None] if zeros is not None else 8.0
    return w.mul_(scales.float()[:, :, None]).view(rows, 2 * half)


def _plain_head(s):
    w = _dequantised(s["q"], s["scales"], s["zeros"], s["case"]["group"])
    return {"logits": (s["hidden"].float() @ w.t()).to(TYPES[s["case"]["out"]])}


def _plain_sample(s):
    V = s["case"]["V"]
    v, order = torch.sort(s["rows"][:, :V].float() + 0.0, dim=1, descending=True, stable=True)
    greedy = s["temperature"] == 0
    T = torch.where(greedy, 1.0, s["temperature"]).double()[:, None]
    v = v.double()
    w = torch.exp((v - v[:, :1]) / T)
    cum = torch.cumsum(w, dim=1)
    n = torch.isfinite(v).sum(dim=1)
    k = s["top_k"].long()
    n = torch.where(k > 0, torch.minimum(k, n), n)
    Z = cum.gather(1, n[:, None] - 1)
    p = s["top_p"].double()[:, None]
    n_p = torch.where(p[:, 0] < 1, (cum < p * Z).sum(dim=1) + 1, n)
    n_m = (w >= s["min_p"].double()[:, None]).sum(dim=1)
    n = torch.minimum(n, torch.minimum(n_p, n_m))
    Zs = cum.gather(1, n[:, None] - 1)
    at = torch.minimum((cum <= s["u"].double()[:, None] * Zs).sum(dim=1), n - 1)
    at = torch.where(greedy, 0, at)[:, None]
    prob = torch.where(greedy, 1.0, (w.gather(1, at) / Zs)[:, 0])
    return {"ids": order.gather(1, at)[:, 0].to(torch.int32), "probs": prob.float()}


def _plain_embed(s):
    ids = s["ids"].long()
    at = ids.clamp(min=0)
    if s["case"]["group"]:
        z = s["zeros"][at] if s["zeros"] is not None else None
        rows = _dequantised(s["q"][at], s["scales"][at], z, s["case"]["group"])
    else:
        rows = s["table"][at].float()
    return {"out": torch.where(ids[:, None] >= 0, rows * s["scale"], 0.0).to(s["out"].dtype)}


def run(s):
    op = s["case"]["op"]
    if own:
        from sampling_row_fp32_gb300 import binding as B
        if op == "head":
            B.sel_head_w4(s["hidden"], s["q"], s["scales"], s["zeros"], s["case"]["group"], s["logits"])
            return {"logits": s["logits"]}
        if op == "sample":
            B.sel_sample16(s["rows"][:, :s["case"]["V"]], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"],
                           s["ids"], s["probs"])
            return {"ids": s["ids"], "probs": s["probs"]}
        if s["case"]["group"]:
            B.sel_embed_w4(s["ids"], s["q"], s["scales"], s["zeros"], s["case"]["group"], s["scale"], s["out"])
        else:
            B.sel_embed(s["ids"], s["table"], s["scale"], s["out"])
        return {"out": s["out"]}
    return {"head": _plain_head, "sample": _plain_sample, "embed": _plain_embed}[op](s)


def work(case):
    if case["op"] == "head":
        rows, V, H = case["rows"], case["V"], case["H"]
        groups = V * (H // case["group"])
        return {"bytes": V * H // 2 + groups * (3 if case["zeros"] else 2) + rows * H * 2 + rows * V * SIZE[case["out"]],
                "flops": 2 * rows * V * H}
    if case["op"] == "sample":
        return {"bytes": case["rows"] * (case["V"] * 2 + 28), "flops": case["rows"] * case["V"]}
    n, H = case["n"], case["H"]
    row = H * SIZE[case["dtype"]]
    if case["group"]:
        row = H // 2 + (H // case["group"]) * (3 if case["zeros"] else 2)
    return {"bytes": n * (4 + row + H * SIZE[case["dtype"]]), "flops": n * H}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "head":
        group, V = case["group"], case["V"]
        x = s["hidden"].double()
        out = torch.empty((case["rows"], V), dtype=torch.float64, device=x.device)
        for lo in range(0, V, 8192):
            hi = min(V, lo + 8192)
            q = s["q"][lo:hi].to(torch.int32)
            w = torch.empty((hi - lo, case["H"]), dtype=torch.float64, device=x.device)
            w[:, 0::2], w[:, 1::2] = (q % 16).double(), (q // 16).double()
            z = s["zeros"][lo:hi].double() if s["zeros"] is not None else torch.full_like(s["scales"][lo:hi], 8).double()
            w = (w - z.repeat_interleave(group, 1)) * s["scales"][lo:hi].double().repeat_interleave(group, 1)
            out[:, lo:hi] = torch.einsum("rh,vh->rv", x, w)
        return {"logits": out}
    if case["op"] == "sample":
        rows = s["rows"][:, :case["V"]].float().cpu().numpy().astype(np.float64)
        T, k, p, m, u = (s[n].cpu().numpy().astype(np.float64) for n in ("temperature", "top_k", "top_p", "min_p", "u"))
        probs = [_exact_row(rows[r], T[r], int(k[r]), p[r], m[r], u[r]) for r in range(case["rows"])]
        return {"ids": None, "probs": np.array(probs)}
    ids = s["ids"].cpu().numpy()
    if case["n"] * case["H"] > 1 << 27:
        return None
    at = torch.from_numpy(np.maximum(ids, 0)).to(s["out"].device).long()
    if case["group"]:
        group = case["group"]
        q = s["q"][at].to(torch.int32)
        rows = torch.empty((case["n"], case["H"]), dtype=torch.float64, device=q.device)
        rows[:, 0::2], rows[:, 1::2] = (q % 16).double(), (q // 16).double()
        z = s["zeros"][at].double() if s["zeros"] is not None else torch.full_like(s["scales"][at], 8).double()
        rows = (rows - z.repeat_interleave(group, 1)) * s["scales"][at].double().repeat_interleave(group, 1)
    else:
        rows = s["table"][at].double()
    rows = rows * s["scale"]
    rows[torch.from_numpy(ids < 0).to(rows.device)] = 0
    return {"out": rows}


def _exact_row(x, T, k, p, m, u):
    """The drawn token's probability: the row as its distinct values, from the largest, with their counts."""
    if T == 0:
        return 1.0
    val, count = np.unique(x[np.isfinite(x)], return_counts=True)
    val, count = val[::-1], count[::-1]
    w = np.exp((val - val[0]) / T)

    def first(total, n):
        """The prefix `count` cut to its first n ids."""
        before = np.concatenate(([0], np.cumsum(total)[:-1]))
        return np.clip(n - before, 0, total)

    c = first(count, k) if k > 0 else count
    if p < 1:
        mass = np.cumsum(c * w)
        b = int(np.searchsorted(mass, p * mass[-1]))
        b = min(b, len(c) - 1)
        need = p * mass[-1] - (mass[b] - c[b] * w[b])
        c = np.where(np.arange(len(c)) < b, c, 0)
        c[b] = max(1, math.ceil(need / w[b]))
    c = np.where(w >= m, c, 0)
    mass = np.cumsum(c * w)
    b = int(np.searchsorted(mass, u * mass[-1], side="right"))
    return w[min(b, np.nonzero(c)[0][-1])] / mass[-1]
