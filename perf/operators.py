"""Operators around the routed-expert products: routing, tokens sorted by expert
and back, 8-bit activation checkpoints, and the weight gradient that reads them.

``listed()`` names the measured cases, ``draw()`` gives further ones of the
same ranges, ``prepare()`` makes a case's inputs, ``run()`` is one pass (the
library's calls where ``own`` is true, elementary torch operations in float32
otherwise), ``work()`` the bytes and operations a pass cannot do without and
``exact()`` the outputs from the definitions in float64.

Definitions
  route     top-k experts of every token by logit (ties to the lower index,
            -inf masks an expert, a slot without an expert has id -1 and
            weight 0); weights are the softmax over the chosen logits
            ("topk") or over all logits ("all").
  sort      slots (token, j) ordered by expert, then token, then j.  An id
            outside [0, E) drops its slot: dropped slots take the last rows
            and are marked by ~row in slot_row.
  dispatch  rows[slot_row[t, j]] = x[t]; rows of dropped slots are zero.
  combine   out[t] = sum_j weights[t, j] * rows[slot_row[t, j]] over the slots
            that are not dropped, with its gradients.
  checkpoint  E4M3 codes of x / s, one power-of-two scale s per row and 128
            columns: the smallest 2^e with max(amax, 1e-12) <= 448 * 2^e.
  swiglu    h = silu(gate) * up of gate_up = [gate | up] with both halves
            checkpointed; the gradient is taken at the checkpointed values.
  wgrad     dW[e] = sum over the rows r of expert e of
            d_y[r]^T (codes * scales)[row_token[r]].
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a decode step's router: a handful of tokens, latency only
        dict(name="route_decode", op="route", T=4, E=64, k=8, dtype="f32", normalize="topk", backward=False),
        # a training microbatch's router and its gradient, many experts, some masked
        dict(name="route_train", op="route", T=16384, E=256, k=8, dtype="bf16", normalize="all", backward=True),
        # the sort of a decode step
        dict(name="sort_decode", op="sort", T=16, E=64, k=8, drop=0.0),
        # the sort of a long batch, a few slots dropped at their experts' capacity
        dict(name="sort_long", op="sort", T=65536, E=256, k=8, drop=0.03),
        # tokens of the grouped workload (4096 x 7168, 64 experts, top-8) into expert order
        dict(name="dispatch_grouped", op="dispatch", T=4096, H=7168, E=64, k=8, dtype="bf16", drop=0.0),
        # one sequence's decode step back into token order
        dict(name="combine_decode", op="combine", T=1, H=7168, E=64, k=8, dtype="bf16", drop=0.0),
        # an odd width in float32, with dropped slots
        dict(name="combine_ragged", op="combine", T=3001, H=2047, E=64, k=4, dtype="f32", drop=0.05),
        # the grouped workload's gradients of rows and routing weights
        dict(name="combine_grad_grouped", op="combine_grad", T=4096, H=7168, E=64, k=8, dtype="bf16", drop=0.0),
        # the grouped workload's expert activations (2 x 2048 wide), checkpointed on the way
        dict(name="swiglu_grouped", op="swiglu", rows=32768, inner=2048, dtype="bf16", backward=False),
        # their gradient at an odd width and row count
        dict(name="swiglu_grad_ragged", op="swiglu", rows=9973, inner=1411, dtype="bf16", backward=True),
        # a fine-tuning step's small experts, gradient kept in float32
        dict(name="wgrad_small", op="wgrad", T=1000, E=16, k=2, N=520, K=1024, dtype="f32"),
        # the grouped workload's expert weights (64 of 2048 x 7168), token rows gathered
        dict(name="wgrad_grouped", op="wgrad", T=4096, E=64, k=8, N=2048, K=7168, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    return n - 1 if n in (3072, 6144) else n


def draw(rng):
    op = rng.choice(["route", "sort", "dispatch", "combine", "combine_grad", "swiglu", "wgrad"])
    if op == "route":
        E = _log(rng, 8, 512)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 10)),
                    dtype=rng.choice(["f32", "bf16", "f16"]), normalize=rng.choice(["topk", "all"]),
                    backward=rng.random() < 0.5)
    if op == "sort":
        E = _log(rng, 8, 512)
        return dict(op=op, T=_log(rng, 1, 65536), E=E, k=rng.randint(1, 8),
                    drop=rng.choice([0.0, 0.02, 0.1]))
    if op in ("dispatch", "combine", "combine_grad"):
        H = _log(rng, 64, 7168)
        if rng.random() < 0.6:
            H = max(64, H // 16 * 16)
        return dict(op=op, T=_log(rng, 1, 2048), H=H - 16 if H in (3072, 6144) else H, E=_log(rng, 8, 256),
                    k=rng.randint(1, 8), dtype=rng.choice(["f32", "bf16", "f16"]),
                    drop=rng.choice([0.0, 0.0, 0.05]))
    if op == "swiglu":
        inner = _log(rng, 64, 2048)
        if rng.random() < 0.6:
            inner = max(64, inner // 16 * 16)
        return dict(op=op, rows=_log(rng, 1, 16384), inner=inner - 16 if inner in (1536, 3072) else inner,
                    dtype=rng.choice(["f32", "bf16", "f16"]), backward=rng.random() < 0.5)
    N, K = 8 * _log(rng, 16, 256), 16 * _log(rng, 8, 256)
    return dict(op=op, T=_log(rng, 16, 4096), E=_log(rng, 4, 48), k=rng.randint(1, 4),
                N=N - 8 if N in (3072, 6144) else N, K=K - 16 if K in (3072, 6144) else K,
                dtype=rng.choice(["f32", "bf16"]))


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, b = case["T"], case["E"], case["k"], _SIZE[case["dtype"]]
        n = T * E * b + 8 * T * k
        if case["backward"]:  # the upstream gradient in, d_logits out
            n += 4 * T * k + T * E * b
        return {"bytes": n, "flops": (4 if case["backward"] else 2) * T * E}
    if op == "sort":
        S = case["T"] * case["k"]
        return {"bytes": 4 * (3 * S + case["E"] + 1), "flops": 2 * S}
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, H, b = case["T"], case["k"], case["H"], _SIZE[case["dtype"]]
        live = T * k * (1.0 - case["drop"])
        if op == "dispatch":
            return {"bytes": b * H * T * (1 + k) + 4 * T * k, "flops": T * k * H}
        if op == "combine":
            return {"bytes": b * H * (live + T) + 8 * T * k, "flops": 2 * live * H}
        return {"bytes": b * H * (T + live + T * k) + 12 * T * k, "flops": 3 * live * H}
    if op == "swiglu":
        n, b = case["rows"] * case["inner"], _SIZE[case["dtype"]]
        scales = 8 * case["rows"] * -(-case["inner"] // 128)
        if case["backward"]:
            return {"bytes": (b + 2 + 2 * b) * n + scales, "flops": 12 * n}
        return {"bytes": (2 * b + b + 2) * n + scales, "flops": 10 * n}
    T, E, k, N, K = (case[x] for x in "TEkNK")
    R = T * k
    out = E * N * K * _SIZE[case["dtype"]]
    return {"bytes": T * K + 4 * T * -(-K // 128) + 2 * R * N + 4 * (R + E + 1) + out, "flops": 2 * R * N * K}


# ------------------------------------------------------------------ inputs

def _gen(seed, tag):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + tag) % (1 << 62))
    return g


def _normal(seed, tag, shape, std=1.0):
    return torch.randn(shape, generator=_gen(seed, tag), device="cuda", dtype=torch.float32) * std


def _uniform(seed, tag, shape):
    return torch.rand(shape, generator=_gen(seed, tag), device="cuda", dtype=torch.float32)


def _experts(seed, T, E, k, drop):
    """Expert ids [T, k], distinct within a token and unevenly spread; -1 where dropped."""
    score = _normal(seed, 11, (T, E)) + 0.5 * _normal(seed, 12, (1, E))
    ids = torch.sort(score, dim=1, descending=True).indices[:, :k].to(torch.int32)
    if drop > 0.0:
        ids = torch.where(_uniform(seed, 13, (T, k)) < drop, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def _sorted_slots(ids, E):
    """(expert_offsets, row_token, slot_row) of ids [T, k]; the definition in torch."""
    T, k = ids.shape
    flat = ids.reshape(-1).to(torch.int64)
    live = (flat >= 0) & (flat < E)
    key = torch.where(live, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    count.index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), torch.cumsum(count[:E], 0)])
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=ids.device)
    slot = torch.where(live, row, -1 - row).reshape(T, k)
    return offsets.to(torch.int32), (order // k).to(torch.int32), slot.to(torch.int32)


def _activations(seed, tag, rows, K):
    """N(0, 1) with one column in 200 scaled by 20, as activations have them."""
    x = _normal(seed, tag, (rows, K))
    x[:, _uniform(seed, tag + 1, (K,)) < 0.005] *= 20.0
    return x


def _checkpoint(x, pieces=1):
    """E4M3 codes (as float8) and power-of-two scales of x, each of `pieces`
    equal column ranges cut into blocks of 128 (the last one shorter)."""
    rows, cols = x.shape
    width = cols // pieces
    blocks = -(-width // 128)
    padded = torch.zeros((rows, pieces, blocks * 128), dtype=torch.float32, device=x.device)
    padded[:, :, :width] = x.to(torch.float32).reshape(rows, pieces, width)
    padded = padded.reshape(rows, pieces, blocks, 128)
    top = torch.clamp(padded.abs().amax(dim=3), min=1e-12)
    mantissa, exponent = torch.frexp(top)
    exponent = exponent - 9 + (mantissa > 0.875).to(exponent.dtype)
    scale = torch.ldexp(torch.ones_like(top), exponent)
    codes = torch.ldexp(padded, -exponent.unsqueeze(3)).to(torch.float8_e4m3fn)
    codes = codes.reshape(rows, pieces, blocks * 128)[:, :, :width].reshape(rows, cols)
    return codes.contiguous(), scale.reshape(rows, pieces * blocks).contiguous()


def _restore(codes, scales, pieces, dtype):
    rows, cols = codes.shape
    width = cols // pieces
    s = scales.to(dtype).reshape(rows, pieces, -1).repeat_interleave(128, dim=2)[:, :, :width]
    return codes.view(torch.float8_e4m3fn).to(torch.float32).to(dtype) * s.reshape(rows, cols)


def prepare(case, seed):
    op, st = case["op"], {"case": case}
    if op == "route":
        T, E = case["T"], case["E"]
        logits = _normal(seed, 1, (T, E)) + 0.2 * _normal(seed, 2, (1, E))
        if E >= 2 * case["k"]:  # a few experts switched off for a few tokens
            logits = torch.where(_uniform(seed, 3, (T, E)) < 0.01, torch.full_like(logits, -math.inf), logits)
        st["logits"] = logits.to(_DT[case["dtype"]])
        st["d_weights"] = _normal(seed, 4, (T, case["k"]))
    elif op == "sort":
        st["ids"] = _experts(seed, case["T"], case["E"], case["k"], case["drop"])
    elif op in ("dispatch", "combine", "combine_grad"):
        T, H, k, dt = case["T"], case["H"], case["k"], _DT[case["dtype"]]
        ids = _experts(seed, T, case["E"], k, case["drop"])
        st["offsets"], st["row_token"], st["slot_row"] = _sorted_slots(ids, case["E"])
        if op == "dispatch":
            st["x"] = _activations(seed, 1, T, H).to(dt)
        else:
            st["rows"] = _normal(seed, 1, (T * k, H)).to(dt)
            st["weights"] = torch.softmax(_normal(seed, 3, (T, k)), dim=1)
            if op == "combine_grad":
                st["d_out"] = _normal(seed, 4, (T, H), 0.01).to(dt)
    elif op == "swiglu":
        gate_up = _activations(seed, 1, case["rows"], 2 * case["inner"]).to(_DT[case["dtype"]])
        if case["backward"]:
            codes, st["scales"] = _checkpoint(gate_up, 2)
            st["codes"] = codes.view(torch.uint8)
            st["d_h"] = _normal(seed, 3, (case["rows"], case["inner"]), 0.01).to(_DT[case["dtype"]])
        else:
            st["gate_up"] = gate_up
    else:
        T, E, k, N, K = (case[x] for x in "TEkNK")
        ids = _experts(seed, T, E, min(k, E), 0.0)
        st["offsets"], st["row_token"], _ = _sorted_slots(ids, E)
        st["bounds"] = st["offsets"].tolist()
        codes, st["scales"] = _checkpoint(_activations(seed, 1, T, K))
        st["codes"] = codes.view(torch.uint8)
        st["d_y"] = _normal(seed, 3, (T * k, N), 0.01).to(torch.bfloat16)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import int4_gemm_gb300 as q4
    case = st["case"]
    op = case["op"]
    if op == "route":
        ids, weights = q4.moe_route_topk(st["logits"], case["k"], normalize=case["normalize"])
        if not case["backward"]:
            return ids, weights
        return ids, weights, q4.moe_route_topk_backward(st["logits"], ids, st["d_weights"],
                                                        normalize=case["normalize"])
    if op == "sort":
        return q4.moe_sort_tokens(st["ids"], case["E"])
    if op == "dispatch":
        return q4.moe_dispatch(st["x"], st["slot_row"])
    if op == "combine":
        return q4.moe_combine(st["rows"], st["slot_row"], st["weights"])
    if op == "combine_grad":
        return q4.moe_combine_backward(st["d_out"], st["rows"], st["slot_row"], st["weights"])
    if op == "swiglu":
        if case["backward"]:
            return q4.swiglu_fp8_backward(st["d_h"], st["codes"], st["scales"])
        h, codes, scales = q4.swiglu_fp8(st["gate_up"])
        return h, codes.view(torch.float8_e4m3fn), scales
    return q4.grouped_wgrad_fp8(st["d_y"], st["codes"], st["scales"], st["offsets"],
                                row_token=st["row_token"], out_dtype=_DT[case["dtype"]])


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route":
        k, x = case["k"], st["logits"].to(torch.float32)
        value, order = torch.sort(x, dim=1, descending=True, stable=True)
        value, order = value[:, :k], order[:, :k]
        found = value > -math.inf
        ids = torch.where(found, order, torch.full_like(order, -1)).to(torch.int32)
        top = torch.clamp(value[:, :1], min=torch.finfo(torch.float32).min)
        e = torch.exp(value - top)
        if case["normalize"] == "topk":
            total = e.sum(dim=1, keepdim=True)
        else:
            p = torch.exp(x - top)
            total = p.sum(dim=1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        weights = e / total
        if not case["backward"]:
            return ids, weights
        dw = torch.where(found, st["d_weights"], torch.zeros_like(st["d_weights"]))
        dot = (dw * weights).sum(dim=1, keepdim=True)
        if case["normalize"] == "topk":
            d = torch.zeros_like(x)
            d.scatter_(1, order, weights * (dw - dot))
        else:
            p = p / total
            g = torch.zeros_like(x)
            g.scatter_(1, order, dw)
            d = p * (g - dot)
        return ids, weights, d.to(st["logits"].dtype)
    if op == "sort":
        return _sorted_slots(st["ids"], case["E"])
    if op == "dispatch":
        x, slot = st["x"], st["slot_row"].reshape(-1).to(torch.int64)
        rows = torch.zeros((slot.numel(), x.shape[1]), dtype=x.dtype, device=x.device)
        live = (slot >= 0).nonzero().reshape(-1)
        rows[slot[live]] = x[live // case["k"]]
        return rows
    if op == "combine":
        slot = st["slot_row"].to(torch.int64)
        out = torch.zeros((case["T"], case["H"]), dtype=torch.float32, device=slot.device)
        for j in range(case["k"]):
            live = slot[:, j] >= 0
            y = st["rows"][torch.where(live, slot[:, j], torch.zeros_like(slot[:, j]))].to(torch.float32)
            out = out + torch.where(live.unsqueeze(1), y * st["weights"][:, j:j + 1], torch.zeros_like(y))
        return out.to(st["rows"].dtype)
    if op == "combine_grad":
        slot, d = st["slot_row"].to(torch.int64), st["d_out"].to(torch.float32)
        d_rows = torch.zeros_like(st["rows"])
        d_weights = torch.zeros_like(st["weights"])
        for j in range(case["k"]):
            live = slot[:, j] >= 0
            at = torch.where(live, slot[:, j], -1 - slot[:, j])
            keep = live.to(torch.float32).unsqueeze(1)
            d_rows[at] = (d * (st["weights"][:, j:j + 1] * keep)).to(d_rows.dtype)
            d_weights[:, j] = (d * st["rows"][at].to(torch.float32) * keep).sum(dim=1)
        return d_rows, d_weights
    if op == "swiglu":
        inner = case["inner"]
        if case["backward"]:
            x = _restore(st["codes"], st["scales"], 2, torch.float32)
            g, u, d = x[:, :inner], x[:, inner:], st["d_h"].to(torch.float32)
            s = 1.0 / (1.0 + torch.exp(-g))
            dg = d * u * s * (1.0 + g * (1.0 - s))
            du = d * g * s
            return torch.cat([dg, du], dim=1).to(st["d_h"].dtype)
        x = st["gate_up"].to(torch.float32)
        g, u = x[:, :inner], x[:, inner:]
        h = (g / (1.0 + torch.exp(-g)) * u).to(st["gate_up"].dtype)
        return (h,) + _checkpoint(x, 2)
    x = _restore(st["codes"], st["scales"], 1, torch.float32)
    token = st["row_token"].to(torch.int64)
    out = torch.empty((case["E"], case["N"], case["K"]), dtype=_DT[case["dtype"]], device=x.device)
    for e, (lo, hi) in enumerate(zip(st["bounds"][:-1], st["bounds"][1:])):
        out[e] = (st["d_y"][lo:hi].to(torch.float32).t() @ x[token[lo:hi]]).to(out.dtype)
    return out


# ------------------------------------------------------------------ float64

def _exact_route(case, st):
    x = st["logits"].double().cpu().numpy()
    T, E = x.shape
    k = case["k"]
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    value = np.take_along_axis(x, order, axis=1)
    found = np.isfinite(value)
    ids = np.where(found, order, -1).astype(np.int32)
    top = np.where(np.isfinite(value[:, :1]), value[:, :1], 0.0)
    p = np.exp(x - top)
    if case["normalize"] == "topk":
        chosen = np.zeros((T, E), bool)
        np.put_along_axis(chosen, order, found, axis=1)
        p = np.where(chosen, p, 0.0)
    p = p / np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
    w = np.where(found, np.take_along_axis(p, order, axis=1), 0.0)
    if not case["backward"]:
        return ids, w
    g = np.zeros((T, E))
    np.put_along_axis(g, order, np.where(found, st["d_weights"].double().cpu().numpy(), 0.0), axis=1)
    return ids, w, p * (g - (p * g).sum(axis=1, keepdims=True))


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "route":
        return _exact_route(case, st)
    if op == "sort":
        ids = st["ids"].cpu().numpy().reshape(-1)
        key = np.where((ids >= 0) & (ids < case["E"]), ids, case["E"])
        order = np.lexsort((np.arange(key.size), key))
        row = np.empty(key.size, np.int32)
        row[order] = np.arange(key.size)
        offsets = np.searchsorted(key[order], np.arange(case["E"] + 1)).astype(np.int32)
        return (offsets, (order // case["k"]).astype(np.int32),
                np.where(key < case["E"], row, ~row).reshape(case["T"], case["k"]))
    if op == "dispatch":
        token = st["row_token"].to(torch.int64)
        rows = st["x"].to(f64)[token]
        rows[int(st["offsets"][-1]):] = 0.0
        return rows
    if op in ("combine", "combine_grad"):
        # from the rows' side: each row belongs to one slot
        T, k = case["T"], case["k"]
        slot = st["slot_row"].reshape(-1).to(torch.int64)
        of_row = torch.empty_like(slot)
        of_row[torch.where(slot >= 0, slot, -1 - slot)] = torch.arange(slot.numel(), device=slot.device)
        live = int(st["offsets"][-1])
        of_row = of_row[:live]
        w = st["weights"].to(f64).reshape(-1)[of_row].unsqueeze(1)
        y = st["rows"][:live].to(f64)
        if op == "combine":
            return torch.zeros((T, case["H"]), dtype=f64, device=w.device).index_add_(0, of_row // k, y * w)
        d = st["d_out"].to(f64)[of_row // k]
        d_rows = torch.zeros((T * k, case["H"]), dtype=f64, device=w.device)
        d_rows[:live] = d * w
        d_weights = torch.zeros(T * k, dtype=f64, device=w.device)
        d_weights[of_row] = torch.einsum("rh,rh->r", d, y)
        return d_rows, d_weights.reshape(T, k)
    if op == "swiglu":
        inner = case["inner"]
        if case["backward"]:
            x = _restore(st["codes"], st["scales"], 2, f64)
            g, u, d = x[:, :inner], x[:, inner:], st["d_h"].to(f64)
            s = torch.sigmoid(g)
            return torch.cat([d * u * (s + g * s * torch.sigmoid(-g)), d * g * s], dim=1)
        x = st["gate_up"].to(f64)
        scales, values = [], []
        for half in (x[:, :inner], x[:, inner:]):
            for lo in range(0, inner, 128):
                b = half[:, lo:lo + 128]
                top = torch.clamp(b.abs().amax(dim=1, keepdim=True), min=float(np.float32(1e-12)))
                s = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
                s = torch.where(top <= 224.0 * s, s * 0.5, torch.where(top > 448.0 * s, s * 2.0, s))
                v = (b / s).abs()
                # E4M3: steps of 2^-9 below 2^-6, else of 1/8 of the power of two
                step = torch.exp2(torch.clamp(torch.floor(torch.log2(v + 1e-300)), min=-6.0) - 3.0)
                values.append(torch.round(v / step) * step * torch.sign(b))
                scales.append(s)
        return x[:, :inner] * torch.sigmoid(x[:, :inner]) * x[:, inner:], torch.cat(values, 1), torch.cat(scales, 1)
    if 2.0 * case["T"] * case["k"] * case["N"] * case["K"] > 4e12:
        return None
    x = _restore(st["codes"], st["scales"], 1, f64)
    token, bounds = st["row_token"].to(torch.int64), st["bounds"]
    return torch.stack([torch.einsum("rn,rk->nk", st["d_y"][lo:hi].to(f64), x[token[lo:hi]])
                        for lo, hi in zip(bounds[:-1], bounds[1:])])
