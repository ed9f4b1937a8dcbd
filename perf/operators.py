"""Cases of the drafter-training operators: the teacher's top logits of a row (spec_row_topk),
distillation from them (spec_topk_distill) and the LM head's cross entropy without its logits
(spec_lm_head_loss), with a plain form of each in elementary torch operations.

Sizes: vocabularies of 151,936 and 128,256 (the benchmark's workloads) and 32,003 (an odd one);
512 rows are the batch-64 workload's target rows (64 requests of 8 positions), 448 its draft rows;
a hidden size of 4096 is the LM head benchmark's.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# The work of the largest listed case of each operator, which a drawn case stays within.
MOST_LOGITS = 2048 * 151936
MOST_HEAD = 4096 * 128256 * 4096


def listed():
    return [
        # one request's next token is kept for the drafter: a single row, latency counts
        {"name": "topk-1row", "op": "topk", "R": 1, "V": 151936, "K": 16, "dt": "bf16", "T": 1.0},
        # the target rows of a batch of 64 requests, kept as the teacher's record of the round
        {"name": "topk-512", "op": "topk", "R": 512, "V": 151936, "K": 64, "dt": "bf16", "T": 1.0},
        # fp32 rows of an odd vocabulary, more rows than a multiple of anything, a long list
        {"name": "topk-f32-odd", "op": "topk", "R": 1027, "V": 32003, "K": 128, "dt": "f32", "T": 0.7},
        # the drafter's loss on one request's seven positions, as a signal during serving
        {"name": "distill-7rows", "op": "distill", "R": 7, "V": 151936, "K": 16, "dt": "bf16", "T": 1.0, "tail": True, "grad": True},
        # the loss alone over a batch's draft rows, to watch how the drafter fares
        {"name": "distill-448-loss", "op": "distill", "R": 448, "V": 151936, "K": 64, "dt": "bf16", "T": 1.0, "tail": True, "grad": False},
        # a training step's micro-batch of positions, loss and gradient
        {"name": "distill-2048", "op": "distill", "R": 2048, "V": 151936, "K": 64, "dt": "bf16", "T": 1.0, "tail": True, "grad": True},
        # fp32 logits of an odd vocabulary, renormalised short lists, softened
        {"name": "distill-f32-odd", "op": "distill", "R": 515, "V": 32003, "K": 17, "dt": "f32", "T": 2.0, "tail": False, "grad": True},
        # a small drafter's loss on a few positions
        {"name": "head-64-loss", "op": "head", "R": 64, "V": 32003, "D": 1024, "T": 1.0, "grad": False},
        # the loss of a batch's target rows under the benchmark's head
        {"name": "head-512-loss", "op": "head", "R": 512, "V": 151936, "D": 4096, "T": 1.0, "grad": False},
        # a small drafter's step on an odd number of positions, with gradients
        {"name": "head-333-odd", "op": "head", "R": 333, "V": 32003, "D": 1032, "T": 1.0, "grad": True},
        # adapting the head online on one round's positions: few rows, the whole head's gradient
        {"name": "head-448", "op": "head", "R": 448, "V": 151936, "D": 4096, "T": 1.0, "grad": True},
        # a training step's micro-batch of positions, with gradients
        {"name": "head-4096", "op": "head", "R": 4096, "V": 128256, "D": 4096, "T": 1.0, "grad": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk", "distill", "head"])
    T = rng.choice([0.5, 0.7, 1.0, 2.0])
    if op == "head":
        V, D = _log_int(rng, 1000, 151936), 8 * _log_int(rng, 16, 512)
        R = _log_int(rng, 1, max(1, min(4096, MOST_HEAD // (V * D))))
        return {"op": op, "R": R, "V": V, "D": D, "T": T, "grad": rng.random() < 0.75}
    V = _log_int(rng, 1000, 151936)
    R = _log_int(rng, 1, min(4096, MOST_LOGITS // V))
    case = {"op": op, "R": R, "V": V, "K": _log_int(rng, 1, 256 if op == "topk" else 128), "dt": rng.choice(["bf16", "bf16", "f32"]), "T": T}
    if op == "distill":
        case["tail"], case["grad"] = rng.random() < 0.6, rng.random() < 0.75
    return case


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    R, V = case["R"], case["V"]
    st = {"case": case}
    if case["op"] == "head":
        D = case["D"]
        # a head whose logits spread by about 1.3, hidden states that lean towards their target by
        # zero to ten units of logit; one position in sixteen is padding (target -1, weight 0)
        W = torch.randn((V, D), generator=g, device=DEV).mul_(1.28 / math.sqrt(D)).to(torch.bfloat16)
        y = torch.randint(0, V, (R,), generator=g, device=DEV)
        lean = 10.0 / 1.28 ** 2 * torch.rand((R, 1), generator=g, device=DEV)
        h = torch.randn((R, D), generator=g, device=DEV) + lean * W[y].float()
        pad = torch.rand(R, generator=g, device=DEV) < (1 / 16 if R > 16 else 0.0)
        st["hidden"], st["weight"] = h.to(torch.bfloat16), W
        st["targets"] = torch.where(pad, -1, y).to(torch.int32)
        st["row_weight"] = torch.where(pad, 0.0, 1.0 / R).to(torch.float32)
        return st
    # rows of N(0, 3^2) with a few favoured tokens, as a model's rows have them
    l = torch.randn((R, V), generator=g, device=DEV).mul_(3.0)
    hot = torch.randint(0, V, (R, 8), generator=g, device=DEV)
    l.scatter_add_(1, hot, torch.rand((R, 8), generator=g, device=DEV) * 12.0)
    if case["op"] == "topk":
        st["logits"] = l.to(DT[case["dt"]])
        return st
    # the drafter's row is the target's row plus N(0, 1); the record is the target's
    top, idx = torch.topk(l, case["K"], dim=1)
    st["index"], st["teacher"] = idx.to(torch.int32), top.contiguous()
    st["teacher_log_z"] = torch.logsumexp(l / case["T"], dim=1) if case["tail"] else None
    l += torch.randn((R, V), generator=g, device=DEV)
    st["logits"] = l.to(DT[case["dt"]])
    pad = torch.rand(R, generator=g, device=DEV) < (1 / 16 if R > 16 else 0.0)
    st["index"][pad] = -1                                  # padded positions hold an empty list
    st["row_weight"] = torch.where(pad, 0.0, 1.0 / R).to(torch.float32)
    return st


def run(state):
    c = state["case"]
    return {"topk": _topk, "distill": _distill, "head": _head}[c["op"]](state, c)


def _topk(st, c):
    if own:
        import lossless_draft_verification_row_amd as L
        return L.spec_row_topk(st["logits"], c["K"], temperature=c["T"])
    l = st["logits"].float()
    val, idx = torch.sort(l, dim=1, descending=True, stable=True)
    m = val[:, :1]
    z = torch.exp((l - m) / c["T"]).sum(dim=1)
    return {"index": idx[:, :c["K"]].to(torch.int32), "logit": val[:, :c["K"]].contiguous(), "log_z": m[:, 0] / c["T"] + torch.log(z)}


def _distill(st, c):
    if own:
        import lossless_draft_verification_row_amd as L
        return L.spec_topk_distill(st["logits"], st["index"], st["teacher"], teacher_log_z=st["teacher_log_z"], temperature=c["T"],
                                   row_weight=st["row_weight"], grad=c["grad"])
    T, V = c["T"], c["V"]
    s, x = st["logits"].float() / T, st["index"].long()
    ok = (x >= 0) & (x < V)
    x = torch.where(ok, x, 0)
    t = torch.where(ok, st["teacher"], -math.inf) / T
    some = ok.any(dim=1)
    m = s.amax(dim=1, keepdim=True)
    e = torch.exp(s - m)
    log_z = m + torch.log(e.sum(dim=1, keepdim=True))
    log_q = s.gather(1, x) - log_z
    if c["tail"]:
        log_p = t - st["teacher_log_z"][:, None]
        p = torch.exp(log_p)
        rho = torch.clamp(1.0 - p.double().sum(dim=1, keepdim=True), min=0.0).float()
        rho = torch.where((rho > 2.0 ** -20) & some[:, None], rho, 0.0)
    else:
        tm = torch.where(some, t.amax(dim=1), 0.0)[:, None]
        p = torch.exp(t - tm)
        zt = torch.where(some[:, None], p.sum(dim=1, keepdim=True), 1.0)
        log_p = t - tm - torch.log(zt)
        p = p / zt
        rho = torch.zeros_like(m)
    loss = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(dim=1)
    listed_v = torch.zeros((c["R"], V + 1), dtype=torch.bool, device=s.device).scatter_(1, torch.where(ok, x, V), True)[:, :V]
    q_rho = torch.where(listed_v, 0.0, torch.exp(s - log_z)).sum(dim=1, keepdim=True)
    loss = loss + torch.where(rho > 0, rho * (torch.log(rho) - torch.log(q_rho)), 0.0)[:, 0]
    out = {"loss": torch.where(some, loss, 0.0), "log_z": log_z[:, 0]}
    if c["grad"]:
        mass = p.sum(dim=1, keepdim=True) + rho
        scale = st["row_weight"][:, None] / T
        a_out = torch.where(rho > 0, mass - rho / q_rho, mass)
        d = torch.exp(s - log_z) * torch.where(listed_v, mass, a_out)
        d.scatter_add_(1, x, torch.where(ok, -p, 0.0))
        out["d_logits"] = torch.where(some[:, None], d * scale, 0.0).to(st["logits"].dtype)
    return out


def _head(st, c):
    if own:
        import lossless_draft_verification_row_amd as L
        return L.spec_lm_head_loss(st["hidden"], st["weight"], st["targets"], temperature=c["T"], row_weight=st["row_weight"], grad=c["grad"])
    T = c["T"]
    h, w, y = st["hidden"].float(), st["weight"].float(), st["targets"].long()
    l = h @ w.T
    l /= T
    m = l.amax(dim=1, keepdim=True)
    l -= m
    keep = (y >= 0) & (y < c["V"])
    y = torch.where(keep, y, 0)
    ly = l.gather(1, y[:, None])
    l.exp_()
    z = l.sum(dim=1, keepdim=True)
    out = {"loss": torch.where(keep, (torch.log(z) - ly)[:, 0], 0.0), "log_z": (m + torch.log(z))[:, 0]}
    if c["grad"]:
        scale = torch.where(keep, st["row_weight"], 0.0)[:, None] / T
        l *= scale / z
        l.scatter_add_(1, y[:, None], -scale)
        out["d_hidden"] = (l @ w).to(torch.bfloat16)
        out["d_weight"] = (l.T @ h).to(torch.bfloat16)
    return out


def work(case):
    R, V = case["R"], case["V"]
    if case["op"] == "head":
        D, f = case["D"], 3 if case["grad"] else 1
        return {"bytes": (R + V) * D * 2 * (2 if case["grad"] else 1) + R * 16, "flops": 2 * R * V * D * f}
    e = 2 if case["dt"] == "bf16" else 4
    if case["op"] == "topk":
        return {"bytes": R * V * e + R * case["K"] * 8 + R * 4, "flops": 4 * R * V}
    return {"bytes": R * V * e * (2 if case["grad"] else 1) + R * case["K"] * 8 + R * 16, "flops": 6 * R * V}


# ---- the definitions in 64 bits, on rows of the batch at a time ----


def exact(case, seed):
    st = prepare(case, seed)
    R, V = case["R"], case["V"]
    rows = max(1, (1 << 28) // V)
    parts = []
    if case["op"] == "head":
        return _exact_head(st, case)
    for a in range(0, R, rows):
        parts.append((_exact_topk if case["op"] == "topk" else _exact_distill)(st, case, slice(a, min(R, a + rows))))
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_topk(st, c, r):
    l = st["logits"][r].double()
    V = c["V"]
    # one whole number for each logit, larger for a larger value and, at equal values, for a lower index
    bits = (st["logits"][r].float() + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * (1 << 20) + (V - 1 - torch.arange(V, device=l.device))
    idx = torch.topk(key, c["K"], dim=1).indices
    return {"index": idx.to(torch.int32), "logit": l.gather(1, idx), "log_z": torch.logsumexp(l / c["T"], dim=1)}


def _exact_distill(st, c, r):
    T = c["T"]
    log_q = torch.log_softmax(st["logits"][r].double() / T, dim=1)
    log_z = torch.logsumexp(st["logits"][r].double() / T, dim=1)
    x, t = st["index"][r].cpu().numpy(), st["teacher"][r].double().cpu().numpy() / T
    lz = st["teacher_log_z"][r].double().cpu().numpy() if c["tail"] else None
    w = st["row_weight"][r].double().cpu().numpy()
    loss, rows = np.zeros(len(x)), []
    for i in range(len(x)):
        at = x[i] >= 0
        if not at.any():
            if c["grad"]:
                rows.append(torch.zeros_like(log_q[i]))
            continue
        xi = torch.from_numpy(x[i][at].astype(np.int64)).to(log_q.device)
        ti = t[i][at]
        lp = ti - (lz[i] if c["tail"] else np.logaddexp.reduce(ti))
        p = np.exp(lp)
        rho = max(0.0, 1.0 - math.fsum(p)) if c["tail"] else 0.0
        rho = rho if rho > 2.0 ** -20 else 0.0
        lq = log_q[i][xi].cpu().numpy()
        loss[i] = math.fsum(p * (lp - lq))
        outside = 0.0
        if rho:
            rest = log_q[i].clone()
            rest[xi] = -math.inf
            lq_rho = float(torch.logsumexp(rest, dim=0))
            loss[i] += rho * (math.log(rho) - lq_rho)
            outside = rho / math.exp(lq_rho)
        if c["grad"]:
            mass = math.fsum(p) + rho
            q = torch.exp(log_q[i])
            d = q * (mass - outside)
            d[xi] = q[xi] * mass - torch.from_numpy(p).to(q.device)
            rows.append(d * (w[i] / T))
    out = {"loss": torch.from_numpy(loss), "log_z": log_z.cpu()}
    if c["grad"]:
        out["d_logits"] = torch.stack(rows)
    return out


def _exact_head(st, c):
    R, V, T = c["R"], c["V"], c["T"]
    h, y = st["hidden"].double(), st["targets"].long()
    step = max(1, min(V, (1 << 28) // max(R, c["D"])))
    lz = torch.full((R,), -math.inf, dtype=torch.float64, device=DEV)
    for a in range(0, V, step):
        lz = torch.logaddexp(lz, torch.logsumexp(h @ st["weight"][a:a + step].double().T / T, dim=1))
    keep = y >= 0
    wy = st["weight"][torch.where(keep, y, 0)].double()
    loss = torch.where(keep, lz - (h * wy).sum(dim=1) / T, 0.0)
    out = {"loss": loss, "log_z": lz}
    if c["grad"]:
        scale = torch.where(keep, st["row_weight"].double(), 0.0) / T
        dh, dw = -scale[:, None] * wy, []
        for a in range(0, V, step):
            w = st["weight"][a:a + step].double()
            p = torch.exp(h @ w.T / T - lz[:, None]) * scale[:, None]
            dh += p @ w
            dw.append(p.T @ h)
        out["d_hidden"] = dh
        out["d_weight"] = torch.cat(dw).index_add_(0, torch.where(keep, y, 0), -scale[:, None] * h)
    return out
