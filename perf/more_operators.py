"""What a drafter learns from the rows that selection works on, as measured cases.

Four operators: cross entropy through a 16-bit output head without its logits
rows, the gradient of that, and the divergence of logits rows from a teacher's
top logits (the lists that sel_topk writes), without and with its gradient.
`run` computes them in elementary torch operations, or, where `own` is set,
through the library's binding.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # The log-probability of one draft token: the smallest call, where latency counts.
        head("loss", "loss_1row", rows=1, V=151936, H=1024, dtype="bf16", ignored=0.0),
        # Scores of a verify batch (every position of 7 x 7).
        head("loss", "loss_verify_49rows", rows=49, V=248320, H=4096, dtype="bf16", ignored=0.0),
        # Ragged sequences packed into one batch, an odd vocabulary slice, a prompt's positions ignored.
        head("loss", "loss_ragged_777rows", rows=777, V=93001, H=2880, dtype="f16", ignored=0.3),
        # A training batch or a long document's log-probabilities.
        head("loss", "loss_batch_4096rows", rows=4096, V=151936, H=4096, dtype="bf16", ignored=0.05),
        # Online training of a small drafter on the positions of one verify step.
        head("grad", "grad_64rows", rows=64, V=151936, H=1024, dtype="bf16", ignored=0.1),
        # Ragged sequences again.
        head("grad", "grad_ragged_777rows", rows=777, V=93001, H=2880, dtype="f16", ignored=0.3),
        # A training batch.
        head("grad", "grad_batch_4096rows", rows=4096, V=151936, H=2048, dtype="bf16", ignored=0.05),
        # How far a drafter is from its target at the positions of one step.
        distill("distill", "distill_7rows", rows=7, V=151936, pad=0, dtype="f32", k=20, T=1.0, rest=False),
        # A held-out batch, with what the lists leave out as one more class.
        distill("distill", "distill_512rows", rows=512, V=202048, pad=0, dtype="bf16", k=64, T=2.0, rest=True),
        # Online distillation on the verify batch's rows.
        distill("distill_grad", "distill_grad_verify_49rows", rows=49, V=248320, pad=0, dtype="f32", k=20, T=1.0,
                rest=False),
        # Ragged sequences, an odd width inside padded rows, long lists.
        distill("distill_grad", "distill_grad_ragged_777rows", rows=777, V=93001, pad=23, dtype="f16", k=200, T=1.5,
                rest=True),
        # A training batch.
        distill("distill_grad", "distill_grad_batch_4096rows", rows=4096, V=151936, pad=0, dtype="bf16", k=64, T=1.0,
                rest=False),
    ]


def head(op, name, **kw):
    return {"name": name, "op": op, **kw}


def distill(op, name, **kw):
    return {"name": name, "op": op, **kw}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "grad", "distill", "distill_grad"])
    if op in ("loss", "grad"):
        return {"op": op, "rows": _log(rng, 1, 4096), "V": _log(rng, 2000, 151936),
                "H": 8 * _log(rng, 8, 512 if op == "loss" else 256), "dtype": rng.choice(["f16", "bf16"]),
                "ignored": rng.choice([0.0, 0.05, 0.5])}
    V = _log(rng, 1000, 248320)
    return {"op": op, "rows": _log(rng, 1, 2048), "V": V, "pad": rng.choice([0, 0, 1, 8, 57]),
            "dtype": rng.choice(["f32", "f16", "bf16"]), "k": _log(rng, 1, 512),
            "T": rng.choice([1.0, 1.0, 0.7, 2.0]), "rest": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

PIECE = 16384  # vocabulary columns at a time, where inputs need logits


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"case": dict(case)}
    rows, V, dt = case["rows"], case["V"], TYPES[case["dtype"]]
    gone = torch.rand((rows,), generator=g, device=dev)
    if case["op"] in ("loss", "grad"):
        H = case["H"]
        w = torch.empty((V, H), dtype=dt, device=dev)
        for lo in range(0, V, PIECE):
            n = min(V, lo + PIECE) - lo
            w[lo:lo + n] = (torch.randn((n, H), generator=g, device=dev) * (2.0 / math.sqrt(H))).to(dt)
        t = torch.randint(0, V, (rows,), generator=g, device=dev)
        x = torch.randn((rows, H), generator=g, device=dev)
        # every other row has learnt its token: its logit stands out, to probabilities up to nearly one
        lean = torch.rand((rows, 1), generator=g, device=dev) * 4.0
        lean[1::2] = 0.0
        x += lean * w[t].float()
        s["hidden"], s["weight"] = x.to(dt), w
        s["targets"] = torch.where(gone < case["ignored"], -1, t).to(torch.int32)
        s["loss"] = torch.empty((rows,), dtype=torch.float32, device=dev)
        s["lse"] = torch.empty((rows,), dtype=torch.float32, device=dev)
        if case["op"] == "grad":
            h = s["hidden"].float()
            parts = [torch.logsumexp(h @ w[lo:lo + PIECE].float().t(), dim=1) for lo in range(0, V, PIECE)]
            s["lse"] = torch.logsumexp(torch.stack(parts), dim=0)
            # the mean over the rows, with a weight for each, and f16's usual loss scale
            scale = 65536.0 if case["dtype"] == "f16" else 1.0
            s["grad"] = (0.5 + torch.rand((rows,), generator=g, device=dev)) * (scale / rows)
            s["hidden_grad"] = torch.empty_like(s["hidden"])
            s["weight_grad"] = torch.empty_like(w)
        if own:
            from sampling_row_fp32_gb300 import binding as B
            s["ws"] = B.workspace(B.SEL_OP_HEAD_LOSS_GRAD if case["op"] == "grad" else B.SEL_OP_HEAD_LOSS, rows, V, H)
        return s
    k, T = min(case["k"], V), case["T"]
    ld = V + case["pad"]
    s["logits"] = torch.empty((rows, ld), dtype=dt, device=dev)
    s["vals"] = torch.empty((rows, k), dtype=torch.float32, device=dev)
    s["ids"] = torch.empty((rows, k), dtype=torch.int32, device=dev)
    s["teacher_lse"] = torch.empty((rows,), dtype=torch.float32, device=dev) if case["rest"] else None
    for lo in range(0, rows, 512):  # a few rows at a time
        n = min(rows, lo + 512) - lo
        teacher = torch.randn((n, V), generator=g, device=dev) * 2.0
        # every other row peaked, as a model that knows its next token gives
        teacher[1::2, :V // 2] += 8.0 * torch.rand((n // 2, 1), generator=g, device=dev) * (
            torch.rand((n // 2, V // 2), generator=g, device=dev) < 4.0 / V)
        student = torch.randn((n, ld), generator=g, device=dev)
        student[:, :V] += 0.8 * teacher
        student[:, max(1, V - 64):V] = -math.inf  # columns past the tokenizer's last id
        teacher[:, max(1, V - 64):] = -math.inf
        s["logits"][lo:lo + n] = student.to(dt)
        v, i = torch.topk(teacher, k, dim=1)
        s["vals"][lo:lo + n], s["ids"][lo:lo + n] = v, i.to(torch.int32)
        if case["rest"]:
            s["teacher_lse"][lo:lo + n] = torch.logsumexp(teacher.double() / T, dim=1).float()
    # positions behind a sequence's end have no list; other lists may be shorter than k
    short = torch.randint(1, k + 1, (rows, 1), generator=g, device=dev)
    cut = torch.rand((rows, 1), generator=g, device=dev) < 0.1
    s["ids"].masked_fill_(cut & (torch.arange(k, device=dev)[None] >= short), -1)
    s["ids"].masked_fill_((gone < 0.1)[:, None], -1)
    s["loss"] = torch.empty((rows,), dtype=torch.float32, device=dev)
    if case["op"] == "distill_grad":
        scale = 1024.0 if case["dtype"] == "f16" else 1.0  # (a loss scale)
        s["grad"] = (0.5 + torch.rand((rows,), generator=g, device=dev)) * scale
        s["logits_grad"] = torch.empty_like(s["logits"])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_loss(s):
    t = s["targets"].long()
    z = s["hidden"].float() @ s["weight"].float().t()
    m = z.max(dim=1, keepdim=True).values
    lse = (m + (z - m).exp().sum(dim=1, keepdim=True).log())[:, 0]
    loss = torch.where(t >= 0, lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    return {"loss": loss, "lse": lse}


def _plain_grad(s):
    t, x, w = s["targets"].long(), s["hidden"].float(), s["weight"].float()
    p = ((x @ w.t()) - s["lse"][:, None]).exp()
    p[torch.arange(len(t), device=t.device), t.clamp(min=0)] -= 1.0
    p *= torch.where(t >= 0, s["grad"], 0.0)[:, None]
    return {"hidden": (p @ w).to(s["hidden"].dtype), "weight": (p.t() @ x).to(s["weight"].dtype)}


def _plain_distill(s):
    case, V = s["case"], s["case"]["V"]
    y = s["logits"][:, :V].float() / case["T"]
    y -= y.max(dim=1, keepdim=True).values
    q = y.exp()
    ids = s["ids"].long()
    there = ids >= 0
    ids = ids.clamp(min=0)
    listed = torch.zeros_like(y, dtype=torch.bool)
    listed.scatter_(1, torch.where(there, ids, ids.max(dim=1, keepdim=True).values), True)
    listed &= there.any(dim=1)[:, None]
    others = q.masked_fill(listed, 0.0).sum(dim=1, dtype=torch.float64)
    yi = torch.where(there, y.gather(1, ids), -math.inf).double()
    v = torch.where(there, s["vals"], -math.inf).double() / case["T"]
    Z = others + yi.exp().sum(dim=1)
    L = s["teacher_lse"].double() if case["rest"] else torch.logsumexp(v, dim=1)
    p = torch.where(there, (v - L[:, None]).exp(), 0.0)
    terms = torch.where(p > 0, p * ((v - L[:, None]) - (yi - Z.log()[:, None])), 0.0)
    loss = terms.sum(dim=1)
    live = there.any(dim=1)
    r = torch.zeros_like(loss)
    if case["rest"]:
        r = (1.0 - p.sum(dim=1)).clamp(min=0.0)
        loss = loss + torch.where(r > 0, r * (r.log() - (others / Z).log()), 0.0)
    out = {"loss": torch.where(live, loss, 0.0).float()}
    if case["op"] == "distill_grad":
        scale = torch.where(live, s["grad"].double() / case["T"], 0.0)
        mass = torch.where(r > 0, 1.0, p.sum(dim=1))
        # q / Z times the mass, less r / others for the ids that no list names
        q *= (scale / Z * (mass - torch.where(r > 0, r * Z / others, 0.0))).float()[:, None]
        at = ((yi.exp() / Z[:, None] * mass[:, None] - p) * scale[:, None]).float()
        rows = torch.arange(len(ids), device=ids.device)[:, None].expand_as(ids)
        q[rows[there], ids[there]] = at[there]
        out["logits"] = q.to(s["logits"].dtype)
    return out


def run(s):
    op, V = s["case"]["op"], s["case"]["V"]
    if own:
        from sampling_row_fp32_gb300 import binding as B
        if op == "loss":
            B.sel_head_loss(s["hidden"], s["weight"], s["targets"], s["loss"], s["lse"], s["ws"])
            return {"loss": s["loss"], "lse": s["lse"]}
        if op == "grad":
            B.sel_head_loss_grad(s["hidden"], s["weight"], s["targets"], s["lse"], s["grad"], s["hidden_grad"],
                                 s["weight_grad"], s["ws"])
            return {"hidden": s["hidden_grad"], "weight": s["weight_grad"]}
        if op == "distill":
            B.sel_distill(s["logits"][:, :V], s["vals"], s["ids"], s["teacher_lse"], s["case"]["T"], s["loss"])
            return {"loss": s["loss"]}
        out = s["logits_grad"][:, :V]
        B.sel_distill_grad(s["logits"][:, :V], s["vals"], s["ids"], s["teacher_lse"], s["case"]["T"], s["grad"],
                           s["loss"], out)
        return {"loss": s["loss"], "logits": out}
    return {"loss": _plain_loss, "grad": _plain_grad, "distill": _plain_distill, "distill_grad": _plain_distill}[op](s)


def work(case):
    rows, V = case["rows"], case["V"]
    if case["op"] == "loss":
        H = case["H"]
        return {"bytes": 2 * H * (rows + V) + 12 * rows, "flops": 2 * rows * V * H}
    if case["op"] == "grad":
        H = case["H"]
        return {"bytes": 4 * H * (rows + V) + 12 * rows, "flops": 6 * rows * V * H}
    passes = 2 if case["op"] == "distill_grad" else 1
    return {"bytes": rows * (passes * V * SIZE[case["dtype"]] + 8 * min(case["k"], V) + 12), "flops": 4 * passes * rows * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("loss", "grad"):
        if work(case)["flops"] > 1.2e13:
            return None
        return _exact_loss(s) if case["op"] == "loss" else _exact_grad(s)
    return _exact_distill(s)


def _exact_loss(s):
    x, t = s["hidden"].double(), s["targets"].long()
    V, rows = s["weight"].shape[0], x.shape[0]
    at = torch.einsum("rh,rh->r", x, s["weight"][t.clamp(min=0)].double())
    # ln of the sum of the other ids' weights over the target's own, so that a loss near 0 keeps its bits
    top = torch.full((rows,), -math.inf, dtype=torch.float64, device=x.device)
    rest = torch.zeros_like(top)
    for lo in range(0, V, 8192):
        z = torch.einsum("rh,vh->rv", x, s["weight"][lo:lo + 8192].double())
        mine = (t >= lo) & (t < lo + z.shape[1])
        z[torch.nonzero(mine)[:, 0], t[mine] - lo] = -math.inf
        high = torch.maximum(top, z.max(dim=1).values)
        rest = rest * torch.exp(top - high) + torch.exp(z - high[:, None]).sum(dim=1)
        top = high
    others = top + torch.log(rest)
    live = t >= 0
    loss = torch.where(live, torch.nn.functional.softplus(others - at, threshold=1e9), 0.0)
    return {"loss": loss, "lse": torch.where(live, torch.logaddexp(others, at), others)}


def _exact_grad(s):
    live = s["targets"] >= 0
    x, t = s["hidden"][live].double(), s["targets"][live].long()
    lse, g = s["lse"][live].double(), s["grad"][live].double()
    V, H = s["weight"].shape
    dx = torch.zeros_like(x)
    dw = torch.empty((V, H), dtype=torch.float64, device=x.device)
    for lo in range(0, V, 8192):
        w = s["weight"][lo:lo + 8192].double()
        a = torch.exp(torch.einsum("vh,rh->vr", w, x) - lse[None])
        mine = torch.nonzero((t >= lo) & (t < lo + len(w)))[:, 0]
        a[t[mine] - lo, mine] -= 1.0
        a *= g[None]
        dx += torch.einsum("vr,vh->rh", a, w)
        dw[lo:lo + len(w)] = torch.einsum("vr,rh->vh", a, x)
    out = torch.zeros((len(live), H), dtype=torch.float64, device=x.device)
    out[live] = dx
    return {"hidden": out, "weight": dw}


def _exact_distill(s):
    case, V, T = s["case"], s["case"]["V"], s["case"]["T"]
    grad = case["op"] == "distill_grad"
    rows = case["rows"]
    loss = torch.zeros((rows,), dtype=torch.float64, device=s["logits"].device)
    out = torch.empty((rows, V), dtype=torch.float64, device=s["logits"].device) if grad else None
    for lo in range(0, rows, 256):
        n = min(rows, lo + 256) - lo
        lq = torch.log_softmax(s["logits"][lo:lo + n, :V].double() / T, dim=1)
        ids = s["ids"][lo:lo + n].long()
        r, c = torch.nonzero(ids >= 0, as_tuple=True)
        # the teacher's row: probabilities where its list has them, nothing elsewhere
        lt = torch.full_like(lq, -math.inf)
        lt[r, ids[r, c]] = s["vals"][lo:lo + n][r, c].double() / T
        L = s["teacher_lse"][lo:lo + n].double() if case["rest"] else torch.logsumexp(lt, dim=1)
        lt -= L[:, None]
        live = (ids >= 0).any(dim=1)
        p = torch.where(live[:, None], torch.exp(lt), 0.0)
        kl = torch.where(p > 0, p * (lt - lq), 0.0).sum(dim=1)
        q = torch.exp(lq)
        left = torch.clamp(1.0 - p.sum(dim=1), min=0.0) if case["rest"] else torch.zeros_like(L)
        out_of = torch.where(lt == -math.inf, q, 0.0)
        s_out = out_of.sum(dim=1)
        kl = kl + torch.where(left > 0, left * torch.log(left / s_out), 0.0)
        loss[lo:lo + n] = torch.where(live, kl, 0.0)
        if grad:
            d = q * torch.where(left > 0, 1.0, p.sum(dim=1))[:, None] - p
            d -= torch.where(left > 0, left / s_out, 0.0)[:, None] * out_of
            out[lo:lo + n] = torch.where(live[:, None], d * (s["grad"][lo:lo + n].double() / T)[:, None], 0.0)
    return {"loss": loss, "logits": out} if grad else {"loss": loss}
