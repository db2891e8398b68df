"""Operators in front of the low-bit products and beside the router: the
root-mean-square norm with the residual's addition and an 8-bit output, the
matrix product in 8-bit integers, and the router's balance loss.

``listed()`` names the measured cases, ``draw()`` gives further ones of the
same ranges, ``prepare()`` makes a case's inputs, ``run()`` is one pass (the
library's calls where ``own`` is true, elementary torch operations in float32
otherwise), ``work()`` the bytes and operations a pass cannot do without and
``exact()`` the outputs from the definitions in float64.

Definitions
  norm      h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * w;
            outputs h (where there is a residual), rstd and y, or y in 8 bits:
              fp8   E4M3 codes of y / s, s = max(amax, 1e-12) / 448 for a row's
                    block of 128 columns;
              int8  integers rint(y / s), s = max(amax, 1e-12) / 127 per row.
  norm_grad with g = d_y * w:  d_x = rstd * (g - h * rstd^2 * mean(g * h)) + d_h
            (d_h: the gradient that reaches h past the norm),
            d_w = sum over rows of d_y * h * rstd.
  int8      C[m, n] = sa[m] * sb[n] * sum_k qa[m, k] * qb[n, k]; with raw
            activations qa and sa are made in the pass (as norm's int8 form).
  balance   p[t] = softmax(logits[t]) (-inf masks an expert), n = tokens with an
            expert that is not masked, counts[e] = slots of expert e,
            f[e] = counts[e] * E / (n * k), P[e] = sum_t p[t, e] / n,
            loss = coeff * sum_e f[e] * P[e], counts' last entry is n;
            d_logits[t, e] = d_loss * coeff / n * p[t, e] * (f[e] - sum_j p[t, j] f[j]).
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
COEFF = 0.01


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a decode step's norm in front of an FP8 or W4A8 product: a few tokens, latency only
        dict(name="norm_decode", op="norm", rows=4, H=7168, dtype="bf16", residual=True, form="fp8"),
        # the norm of a long prefill (the prefill workload's 8192 x 8192 activations) in front of an FP8 product
        dict(name="norm_prefill", op="norm", rows=8192, H=8192, dtype="bf16", residual=True, form="fp8"),
        # the first norm of a block, no residual yet, in front of an INT8 product
        dict(name="norm_int8", op="norm", rows=4096, H=7168, dtype="f16", residual=False, form="int8"),
        # an odd width in float32, not quantized
        dict(name="norm_ragged", op="norm", rows=3001, H=2047, dtype="f32", residual=True, form="none"),
        # a training step's gradient at the grouped workload's tokens, joined with the residual stream's
        dict(name="norm_grad_train", op="norm_grad", rows=16384, H=7168, dtype="bf16", joined=True),
        # an odd width and row count, nothing to join
        dict(name="norm_grad_ragged", op="norm_grad", rows=9973, H=1411, dtype="bf16", joined=False),
        # one token through the decode workload's projection: bound by reading the weights
        dict(name="int8_decode", op="int8", M=1, N=8192, K=8192, dtype="bf16", raw=False),
        # a batch of decode requests, activations quantized in the pass, ragged output width
        dict(name="int8_batch", op="int8", M=100, N=4100, K=7168, dtype="bf16", raw=True),
        # the prefill workload's projection
        dict(name="int8_prefill", op="int8", M=8192, N=28672, K=8192, dtype="bf16", raw=False),
        # a short prompt through a small projection, float32 out, nothing a multiple of a tile
        dict(name="int8_ragged", op="int8", M=1001, N=2056, K=2064, dtype="f32", raw=False),
        # one microbatch's balance loss, watched but not trained on
        dict(name="balance_small", op="balance", T=1000, E=64, k=8, dtype="f32", backward=False),
        # a training step's balance loss and its gradient, many experts
        dict(name="balance_train", op="balance", T=65536, E=256, k=8, dtype="bf16", backward=True),
    ]


def _log(rng, lo, hi):
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "int8", "int8", "balance"])
    if op in ("norm", "norm_grad"):
        H = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 16 * 16)
        case = dict(op=op, rows=_log(rng, 1, 8192), H=H, dtype=rng.choice(["f32", "bf16", "f16"]))
        if op == "norm":
            case.update(residual=rng.random() < 0.6, form=rng.choice(["none", "fp8", "int8"]))
        else:
            case.update(joined=rng.random() < 0.6)
        return case
    if op == "int8":
        N = _log(rng, 64, 8192)
        return dict(op=op, M=_log(rng, 1, 4096), N=max(64, N // 16 * 16) if rng.random() < 0.6 else N,
                    K=16 * _log(rng, 4, 512), dtype=rng.choice(["f32", "bf16"]), raw=rng.random() < 0.4)
    E = _log(rng, 8, 512)
    return dict(op=op, T=_log(rng, 1, 65536), E=E, k=rng.randint(1, 8), dtype=rng.choice(["f32", "bf16", "f16"]),
                backward=rng.random() < 0.5)


def work(case):
    op, b = case["op"], _SIZE[case["dtype"]]
    if op == "norm":
        rows, H = case["rows"], case["H"]
        n = rows * H
        moved = b * n * (3 if case["residual"] else 1) + b * H + 4 * rows
        moved += {"none": b * n, "fp8": n + 4 * rows * -(-H // 128), "int8": n + 4 * rows}[case["form"]]
        return {"bytes": moved, "flops": (5 if case["form"] == "none" else 8) * n}
    if op == "norm_grad":
        n = case["rows"] * case["H"]
        return {"bytes": b * n * (4 if case["joined"] else 3) + (b + 4) * case["H"] + 4 * case["rows"], "flops": 12 * n}
    if op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        moved = N * K + 4 * N + b * M * N + (2 * M * K if case["raw"] else M * K) + 4 * M
        return {"bytes": moved, "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    moved = b * T * E + 4 * T * k + 8 * E
    if case["backward"]:
        moved += b * T * E
    return {"bytes": moved, "flops": (10 if case["backward"] else 5) * T * E}


# ------------------------------------------------------------------ inputs

def _gen(seed, tag):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + tag) % (1 << 62))
    return g


def _normal(seed, tag, shape, std=1.0):
    return torch.randn(shape, generator=_gen(seed, tag), device="cuda", dtype=torch.float32) * std


def _uniform(seed, tag, shape):
    return torch.rand(shape, generator=_gen(seed, tag), device="cuda", dtype=torch.float32)


def _activations(seed, tag, rows, K):
    """N(0, 1) with one column in 200 scaled by 20, as activations have them."""
    x = _normal(seed, tag, (rows, K))
    x[:, _uniform(seed, tag + 1, (K,)) < 0.005] *= 20.0
    return x


def _integers(x):
    """x in 8-bit integers, one scale per row."""
    scale = torch.clamp(x.abs().amax(dim=1), min=1e-12) / 127.0
    return torch.clamp(torch.round(x / scale.unsqueeze(1)), -127, 127).to(torch.int8), scale


def prepare(case, seed):
    op, dt, st = case["op"], _DT[case["dtype"]], {"case": case}
    if op in ("norm", "norm_grad"):
        rows, H = case["rows"], case["H"]
        st["weight"] = (1.0 + _normal(seed, 5, (H,), 0.2)).to(dt)
        x = _activations(seed, 1, rows, H)
        if op == "norm":
            st["x"] = x.to(dt)
            st["residual"] = (4.0 * _normal(seed, 3, (rows, H))).to(dt) if case["residual"] else None
        else:
            st["h"] = x.to(dt)
            st["rstd"] = torch.rsqrt(st["h"].to(torch.float32).square().mean(dim=1) + EPS)
            st["d_y"] = _normal(seed, 6, (rows, H), 0.01).to(dt)
            st["d_h"] = _normal(seed, 7, (rows, H), 0.01).to(dt) if case["joined"] else None
    elif op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        st["qb"], st["sb"] = _integers(_normal(seed, 2, (N, K), 0.02))
        x = _activations(seed, 3, M, K)
        if case["raw"]:
            st["x"] = x.to(torch.bfloat16)
        else:
            st["qa"], st["sa"] = _integers(x)
    else:
        T, E, k = case["T"], case["E"], case["k"]
        logits = _normal(seed, 1, (T, E)) + 0.5 * _normal(seed, 2, (1, E))
        if E >= 2 * k:  # a few experts switched off for a few tokens, a few tokens of padding
            logits = torch.where(_uniform(seed, 3, (T, E)) < 0.01, torch.full_like(logits, -math.inf), logits)
        pad = _uniform(seed, 4, (T, 1)) < 0.02
        pad[0] = False
        st["logits"] = torch.where(pad, torch.full_like(logits, -math.inf), logits).to(dt)
        k = min(k, E)
        ids = torch.sort(st["logits"], dim=1, descending=True, stable=True).indices[:, :k]
        st["ids"] = torch.where(pad, torch.full_like(ids, -1), ids).to(torch.int32).contiguous()
        st["d_loss"] = torch.ones(1, device="cuda") * 0.5
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import int4_gemm_gb300 as q4
    case = st["case"]
    op = case["op"]
    if op == "norm":
        x, w, r = st["x"], st["weight"], st["residual"]
        if case["form"] == "none":
            y, h, rstd = q4.rms_norm(x, w, residual=r, eps=EPS)
            return {"y": y, "h": h, "rstd": rstd}
        if case["form"] == "fp8":
            codes, scales, _, h, rstd = q4.rms_norm_fp8(x, w, residual=r, eps=EPS)
            return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales, "h": h, "rstd": rstd}
        codes, scales, _, h, rstd = q4.rms_norm_int8(x, w, residual=r, eps=EPS)
        return {"codes": codes.to(torch.bfloat16), "scales": scales, "h": h, "rstd": rstd}
    if op == "norm_grad":
        d_x, d_w = q4.rms_norm_backward(st["d_y"], st["h"], st["rstd"], st["weight"], d_h=st["d_h"])
        return {"d_x": d_x, "d_w": d_w}
    if op == "int8":
        qa, sa = q4.quantize_int8(st["x"]) if case["raw"] else (st["qa"], st["sa"])
        return {"C": q4.gemm_w8a8_int8(qa, sa, st["qb"], st["sb"], out_dtype=_DT[case["dtype"]]), "sa": sa}
    loss, counts, mean = q4.moe_balance_loss(st["logits"], st["ids"], COEFF)
    out = {"loss": loss, "counts": counts, "mean": mean}
    if case["backward"]:
        out["d_logits"] = q4.moe_balance_loss_backward(st["logits"], counts, st["ids"].shape[1], st["d_loss"], COEFF)
    return out


def _run_plain(st):
    case = st["case"]
    op, dt, f32 = case["op"], _DT[case["dtype"]], torch.float32
    if op == "norm":
        h, H = st["x"].to(f32), case["H"]
        if st["residual"] is not None:
            h = h + st["residual"].to(f32)
        rstd = 1.0 / torch.sqrt((h * h).mean(dim=1) + EPS)
        y = h * rstd.unsqueeze(1) * st["weight"].to(f32)
        out = {"h": h.to(dt) if case["residual"] else None, "rstd": rstd}
        if case["form"] == "none":
            out["y"] = y.to(dt)
        elif case["form"] == "int8":
            codes, out["scales"] = _integers(y)
            out["codes"] = codes.to(torch.bfloat16)
        else:
            blocks = -(-H // 128)
            padded = torch.zeros((case["rows"], blocks * 128), dtype=f32, device=y.device)
            padded[:, :H] = y
            padded = padded.reshape(case["rows"], blocks, 128)
            s = torch.clamp(padded.abs().amax(dim=2), min=1e-12) / 448.0
            codes = (padded / s.unsqueeze(2)).to(torch.float8_e4m3fn)
            out["codes"] = codes.reshape(case["rows"], blocks * 128)[:, :H].contiguous()
            out["scales"] = s
        return out
    if op == "norm_grad":
        h, dy, r = st["h"].to(f32), st["d_y"].to(f32), st["rstd"].unsqueeze(1)
        g = dy * st["weight"].to(f32)
        d = r * (g - h * (r * r) * (g * h).mean(dim=1, keepdim=True))
        if st["d_h"] is not None:
            d = d + st["d_h"].to(f32)
        return {"d_x": d.to(dt), "d_w": (dy * h * r).sum(dim=0)}
    if op == "int8":
        qa, sa = _integers(st["x"].to(f32)) if case["raw"] else (st["qa"], st["sa"])
        C = qa.to(f32) @ st["qb"].to(f32).t()
        C *= sa.unsqueeze(1)
        C *= st["sb"]
        return {"C": C.to(dt), "sa": sa}
    T, E = st["logits"].shape
    k = st["ids"].shape[1]
    x = st["logits"].to(f32)
    top = torch.clamp(x.amax(dim=1, keepdim=True), min=torch.finfo(f32).min)
    p = torch.exp(x - top)
    total = p.sum(dim=1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    n = (total > 0).sum()
    flat = st["ids"].reshape(-1).to(torch.int64)
    live = (flat >= 0) & (flat < E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device)
    counts.index_add_(0, torch.where(live, flat, torch.full_like(flat, E)), torch.ones_like(flat))
    counts[E] = n
    f = counts[:E].to(f32) * E / (n.to(f32) * k)
    mean = p.sum(dim=0) / n.to(f32)
    out = {"loss": (COEFF * (f * mean).sum()).reshape(1), "counts": counts.to(torch.int32), "mean": mean}
    if case["backward"]:
        d = p * (f - (p * f).sum(dim=1, keepdim=True)) * (st["d_loss"] * COEFF / n.to(f32))
        out["d_logits"] = d.to(dt)
    return out


# ------------------------------------------------------------------ float64

def _e4m3_values(v):
    """v rounded to the nearest E4M3 number, ties to even: steps of 2^-9 below
    2^-6, else of 1/8 of the power of two."""
    a = v.abs()
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(a + 1e-300)), min=-6.0) - 3.0)
    return torch.sign(v) * torch.clamp(torch.round(a / step) * step, max=448.0)


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "norm":
        h, H = st["x"].to(f64), case["H"]
        if case["residual"]:
            h = torch.add(h, st["residual"].to(f64))
        rstd = torch.pow(torch.einsum("ij,ij->i", h, h) / H + EPS, -0.5)
        y = torch.einsum("ij,i,j->ij", h, rstd, st["weight"].to(f64))
        out = {"h": h if case["residual"] else None, "rstd": rstd}
        floor = float(np.float32(1e-12))
        if case["form"] == "none":
            out["y"] = y
        elif case["form"] == "int8":
            out["scales"] = torch.clamp(torch.linalg.vector_norm(y, ord=math.inf, dim=1), min=floor) / 127.0
            out["codes"] = torch.round(y / out["scales"][:, None])
        else:
            scales, values = [], []
            for lo in range(0, H, 128):
                b = y[:, lo:lo + 128]
                s = torch.clamp(torch.linalg.vector_norm(b, ord=math.inf, dim=1), min=floor) / 448.0
                scales.append(s)
                values.append(_e4m3_values(b / s[:, None]))
            out["scales"], out["codes"] = torch.stack(scales, 1), torch.cat(values, 1)
        return out
    if op == "norm_grad":
        # through the normalised rows u = h rstd:  d u = d_y w,  d h = rstd (d u - u <d u, u> / H)
        r = st["rstd"].to(f64)
        u = st["h"].to(f64) * r[:, None]
        dy = st["d_y"].to(f64)
        du = dy * st["weight"].to(f64)
        d = (du - u * (torch.einsum("ij,ij->i", du, u) / case["H"])[:, None]) * r[:, None]
        if case["joined"]:
            d += st["d_h"].to(f64)
        return {"d_x": d, "d_w": torch.einsum("ij,ij->j", dy, u)}
    if op == "int8":
        if 2.0 * case["M"] * case["N"] * case["K"] > 4e12:
            return None
        if case["raw"]:
            x = st["x"].to(f64)
            sa = torch.linalg.vector_norm(x, ord=math.inf, dim=1).clamp(min=float(np.float32(1e-12))) / 127.0
            qa = torch.round(x / sa.to(torch.float32).to(f64)[:, None])
        else:
            qa, sa = st["qa"].to(f64), st["sa"].to(f64)
        C = torch.einsum("mk,nk->mn", qa, st["qb"].to(f64))
        return {"C": C * torch.outer(sa, st["sb"].to(f64)), "sa": sa}
    x = st["logits"].double().cpu().numpy()
    T, E = x.shape
    k = st["ids"].shape[1]
    there = np.isfinite(x).any(axis=1)
    n = int(there.sum())
    p = np.zeros((T, E))
    live = x[there]
    live = np.exp(live - live.max(axis=1, keepdims=True))
    p[there] = live / live.sum(axis=1, keepdims=True)
    ids = st["ids"].cpu().numpy().reshape(-1)
    counts = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    f = counts * (E / (n * k))
    mean = p.mean(axis=0) * (T / n)
    out = {"loss": np.array([COEFF * float(f @ mean)]), "counts": np.append(counts, n).astype(np.int32), "mean": mean}
    if case["backward"]:
        out["d_logits"] = float(st["d_loss"]) * COEFF / n * p * (f[None, :] - (p @ f)[:, None])
    return out
