"""The drafter-training operators in 64 bits, from their definitions, with the error that fp32
work and bf16 rounding can add.  Shares no code with the library.

How far a kernel's output may be off, counted in roundings (u = 2^-24 is half an fp32 step):
 * ln Z: a segment's sum is at most 32 + 8 fp32 additions (40 u relative); an exponent
   (l - m) c is off by 3 u of itself, which the sum weighs with its own term: |t| e / sum e stays
   below 20 for the rows here (60 u ln 2); the hardware exponential by 2 u; the fold over segments
   and the last rounding by 2 u and u |ln Z|.  LZ = 110 u covers them: 6.6e-6.
 * a probability: LZ, plus its own exponent, 3 u |t| with |t| <= 200 before it underflows.
"""
import math

import numpy as np
import torch

U = 2.0 ** -24
LZ = 110 * U
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def log_z_tolerance(ref):
    return LZ + 2 * U * np.abs(ref)


def topk(l, K, T):
    """l [R, V] float64 numpy -> index, logit, log_z as spec_row_topk defines them."""
    R, V = l.shape
    index, logit = np.full((R, K), -1, np.int32), np.full((R, K), -np.inf)
    log_z = np.full(R, np.nan)
    for r in range(R):
        x = l[r]
        if np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any():
            logit[r] = np.nan
            continue
        order = np.argsort(-x, kind="stable")
        order = order[x[order] > -np.inf][:K]
        index[r, :len(order)], logit[r, :len(order)] = order, x[order]
        m = x.max()
        log_z[r] = m / T + math.log(np.exp((x - m) / T).sum())
    return index, logit, log_z


def distill(s, index, t, lz_t, T, w):
    """s [R, V] float64, index [R, K], t [R, K], lz_t [R] or None, w [R] or None ->
    loss, log_z, d [R, V], and bounds of the loss's and the gradient's error before its last
    rounding."""
    R, V = s.shape
    w = np.ones(R) if w is None else w
    loss, log_z, d = np.zeros(R), np.full(R, np.nan), np.zeros((R, V))
    e_loss, e_d = np.zeros(R), np.zeros((R, V))
    for r in range(R):
        x = s[r]
        ok = not np.isnan(x).any() and not (x == np.inf).any() and (x > -np.inf).any()
        if ok:
            m = x.max()
            log_z[r] = m / T + math.log(np.exp((x - m) / T).sum())
        on = [j for j in range(index.shape[1]) if 0 <= index[r, j] < V and t[r, j] != -np.inf]
        if not on:
            continue
        if not ok:
            loss[r] = np.nan
            d[r] = 0.0 if w[r] == 0 else np.nan
            continue
        idx, tj = index[r, on], t[r, on].astype(np.float64) / T
        ln_p = tj - (lz_t[r] if lz_t is not None else tj.max() + math.log(np.exp(tj - tj.max()).sum()))
        p = np.exp(ln_p)
        rho = max(0.0, 1.0 - math.fsum(p)) if lz_t is not None else 0.0
        rho = rho if rho > 2.0 ** -20 else 0.0
        ln_q = x / T - log_z[r]
        q = np.exp(ln_q)
        listed = np.zeros(V, bool)
        listed[idx] = True
        mass = math.fsum(p) + rho
        with np.errstate(all="ignore"):
            loss[r] = math.fsum(np.where(p > 0, p * (ln_p - ln_q[idx]), 0.0))
        e_loss[r] = 3 * LZ * mass + 2 * U * abs(loss[r])
        off = 0.0
        if rho > 0:
            rest = x[~listed]
            if len(rest) == 0 or not (rest > -np.inf).any():
                loss[r] = np.inf
            else:
                mr = rest.max()
                z_rest = np.exp((rest - mr) / T).sum()
                loss[r] += rho * (math.log(rho) - (mr / T + math.log(z_rest) - log_z[r]))
                # q_v / q_rho from the logits' distances: where all of the rest is far down, ln q has
                # no digits left for them
                off = rho * np.exp(np.minimum((x - mr) / T, 0.0)) / z_rest
                e_loss[r] += 2 * U * abs(loss[r])
        g = mass * q - np.where(listed, 0.0, off)
        np.subtract.at(g, idx, p)
        d[r] = g * (w[r] / T)
        pl = np.zeros(V)
        np.add.at(pl, idx, p)
        t_abs = np.minimum(np.abs(x - x.max()) / T * 1.4427, 200.0)
        e_d[r] = abs(w[r] / T) * ((mass * q + np.where(listed, 0.0, off)) * (2 * LZ + 3 * U * np.where(np.isfinite(t_abs), t_abs, 0.0))
                                  + 8 * U * pl) + 1e-37
    return loss, log_z, d, e_loss, e_d


def head(h, wt, y, T, w):
    """Float64 torch tensors h [R, D], wt [V, D] (any device), y [R], w [R] or None -> a dict with
    loss, log_z, d_hidden, d_weight and the error that each may have before its last rounding
    (e_*).  A row that is left out gives zeros; hidden states of such rows are not looked at."""
    R, V = len(h), len(wt)
    y = y.to(h.device).long()
    keep = (y >= 0) & (y < V)
    w = torch.ones(R, dtype=torch.float64, device=h.device) if w is None else w.to(h.device).double()
    used = keep & (w != 0)
    l = h @ wt.T
    # fp32 accumulation of D products: D u sum |h w| for each logit
    delta = (h.shape[1] * U * (h.abs() @ wt.abs().T)).amax(dim=1) / T
    l = l / T
    m = l.amax(dim=1, keepdim=True)
    lz = (m + torch.log(torch.exp(l - m).sum(dim=1, keepdim=True)))[:, 0]
    yy = torch.where(keep, y, 0)
    loss = torch.where(keep, lz - l.gather(1, yy[:, None])[:, 0], 0.0)
    p = torch.exp(l - lz[:, None])
    # exponents are formed as (l - m) c - log2 sum: no more than 2 u of each of l c and log2 Z
    e_rel = (2 * delta + 2 * LZ)[:, None] + 4 * U * (l.abs() + lz.abs()[:, None])
    scale = torch.where(used, w, 0.0)[:, None] / T
    # Exponentials may be kept as fp16 of 2^15 e, e <= 1: below 2^-29 the step of e is fp16's
    # smallest, 2^-24 / 2^15, half of which is 2^-40; e / Z is off by no more, as Z >= 1 where e <= 1
    # is the distance from the row's maximum, and a wave's lower maximum scales both down.
    e_p = torch.where(used[:, None], (p * e_rel + 2.0 ** -40) * scale.abs(), 0.0)
    g = torch.where(used[:, None], p * scale, 0.0)
    g.scatter_add_(1, yy[:, None], -scale)
    # G is rounded to bf16
    e_g = e_p + HALF[torch.bfloat16] * (g.abs() + e_p) + 2.0 ** -133
    hz = torch.where(used[:, None], h, 0.0)
    aw, ah, ag = wt.abs(), hz.abs(), g.abs() + e_g
    return {"loss": loss, "log_z": lz, "d_hidden": g @ wt, "d_weight": g.T @ hz,
            "e_loss": 2 * delta + 2 * LZ + 4 * U * lz.abs() + 2 * U * loss.abs(),
            "e_log_z": delta + LZ + 2 * U * lz.abs(),
            # sums of V and of R products in fp32; a sum of n terms in n / 64 MFMA steps of the
            # longest chain is off by far less than n u, which is the bound taken
            "e_d_hidden": e_g @ aw + V * U * (ag @ aw), "e_d_weight": e_g.T @ ah + R * U * (ag.T @ ah)}
