"""The layer's slot-sorting and 8-bit checkpoint operators: cases, inputs, plain forms and exact results.

Six operators (see include/moe_null.h for their definitions):
  sort              slots sorted by expert: counts, offsets, row -> token, slot -> row
  permute           rows of x copied to their slots' places; with grad, the gradient of that
  unpermute         rows brought back to their tokens with the gates applied, onto a base
  unpermute_grad    its gradient: rows' upstream gradients and the gates' gradients, the rows
                    held in their own type or (codes) as 8-bit blocks
  checkpoint8       an activation stored in 8 bits with one scale per 32 columns, and restored
  swiglu8           SwiGLU's backward from pre-activations stored that way

Slots without an expert (null copies, padding) carry an id outside [0, N) and have no row.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 32


def listed():
    return [
        # one decode step of 64 sequences with the 0.6B layer's routing: launch latency
        {"name": "sort_decode", "op": "sort", "T": 64, "K": 4, "N": 64, "drop": 0.5, "skew": False, "wide_ids": False},
        # the skewed 16 x 8192-token training batch: Zipf-distributed experts, many null slots
        {"name": "sort_skew", "op": "sort", "T": 131072, "K": 8, "N": 64, "drop": 0.4, "skew": True, "wide_ids": False},
        # rows gathered for the expert products of a 16384-token batch (0.6B layer)
        {"name": "permute_prefill", "op": "permute", "grad": False, "T": 16384, "K": 4, "N": 64, "d": 1024,
         "drop": 0.5, "skew": False, "dtype": "bf16"},
        # the gather's gradient at an odd width in fp32 (a user's own experts)
        {"name": "permute_grad_odd", "op": "permute", "grad": True, "T": 5003, "K": 6, "N": 40, "d": 1001,
         "drop": 0.25, "skew": False, "dtype": "fp32"},
        # one decode step of the 1.7B layer: latency of bringing the rows back onto the shared output
        {"name": "unpermute_decode", "op": "unpermute", "T": 64, "K": 8, "N": 64, "d": 2048, "drop": 0.75,
         "skew": False, "dtype": "bf16"},
        # a 65536-token training batch at the 1.7B width, every second slot null
        {"name": "unpermute_train", "op": "unpermute", "T": 65536, "K": 8, "N": 64, "d": 2048, "drop": 0.5,
         "skew": True, "dtype": "bf16"},
        # the backward of a 16384-token batch at the 1.7B width
        {"name": "unpermute_grad_train", "op": "unpermute_grad", "codes": False, "T": 16384, "K": 8, "N": 64,
         "d": 2048, "drop": 0.5, "skew": False, "dtype": "bf16"},
        # the same backward at the 0.6B width with the experts' outputs stored in 8 bits
        {"name": "unpermute_grad_codes", "op": "unpermute_grad", "codes": True, "T": 16384, "K": 4, "N": 64,
         "d": 1024, "drop": 0.5, "skew": False, "dtype": "bf16"},
        # the 0.6B layer's gate/up pre-activations of a 16384-token batch; half of the rows in use
        {"name": "checkpoint8_preact", "op": "checkpoint8", "rows": 65536, "cols": 1536, "used": 0.5, "dtype": "bf16"},
        # an activation of odd width in fp16
        {"name": "checkpoint8_odd", "op": "checkpoint8", "rows": 4099, "cols": 1001, "used": 1.0, "dtype": "fp16"},
        # SwiGLU's backward of the same pre-activations in the packed order of the layer
        {"name": "swiglu8_train", "op": "swiglu8", "rows": 65536, "F": 768, "used": 0.5, "packed": True, "dtype": "bf16"},
        # a small ragged batch of a user's own products: gate and up as two halves, odd width
        {"name": "swiglu8_odd", "op": "swiglu8", "rows": 513, "F": 499, "used": 1.0, "packed": False, "dtype": "fp16"},
    ]


# A drawn case's work() and slot elements stay below the largest listed case's.
MOST_BYTES, MOST_ELEMENTS = 1.5e9, 1.0e9


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """Widths as they occur: half of them multiples of 64, the others as drawn (odd ones among them)."""
    w = _log_int(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.5 else w


def draw(rng):
    op = rng.choice(["sort", "permute", "unpermute", "unpermute_grad", "checkpoint8", "swiglu8"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "sort":
        N = _log_int(rng, 1, 512)
        K = rng.randint(1, min(16, N))
        return {"op": op, "T": _log_int(rng, 1, 131072), "K": K, "N": N, "drop": rng.choice([0.0, 0.3, 0.6]),
                "skew": rng.random() < 0.5, "wide_ids": rng.random() < 0.5}
    if op in ("permute", "unpermute", "unpermute_grad"):
        N = _log_int(rng, 1, 256)
        case = {"op": op, "T": _log_int(rng, 1, 65536), "K": rng.randint(1, min(16, N)), "N": N,
                "d": _width(rng, 1, 8192), "drop": rng.choice([0.0, 0.3, 0.6]), "skew": rng.random() < 0.5,
                "dtype": dtype}
        if op == "permute":
            case["grad"] = rng.random() < 0.5
        if op == "unpermute_grad":
            case["codes"] = rng.random() < 0.5
    elif op == "checkpoint8":
        case = {"op": op, "rows": _log_int(rng, 1, 262144), "cols": _width(rng, 1, 16384),
                "used": rng.choice([0.4, 0.8, 1.0]), "dtype": dtype}
    else:
        packed = rng.random() < 0.5
        F = _width(rng, 1, 8192)
        case = {"op": op, "rows": _log_int(rng, 1, 262144), "F": max(64, F // 64 * 64) if packed else F,
                "used": rng.choice([0.4, 0.8, 1.0]), "packed": packed, "dtype": dtype}
    first = "T" if "T" in case else "rows"
    elements = case["T"] * case["K"] * case["d"] if "T" in case else case["rows"] * case.get("cols", 2 * case.get("F", 0))
    over = max(work(case)["bytes"] / MOST_BYTES, elements / MOST_ELEMENTS)
    if over > 1.0:
        case[first] = max(1, int(case[first] / over))
    return case


def _slots(case):
    return case["T"] * case["K"]


def _used(case):
    return max(0, min(case["rows"], int(case["rows"] * case["used"])))


def work(case):
    """Bytes that the operator has to read and write once, and its multiplications and additions
    (those of one token or pre-activation; slots with an expert are counted at their expected number)."""
    op = case["op"]
    if op == "sort":
        S = _slots(case)
        return {"bytes": S * (8 if case["wide_ids"] else 4) + 4 * S + 4 * S * (1 - case["drop"]) + 8 * case["N"],
                "flops": 2 * S}
    e = 4 if case["dtype"] == "fp32" else 2
    if "T" in case:
        T, S, d = case["T"], _slots(case), case["d"]
        R = S * (1 - case["drop"])
        if op == "permute":
            return {"bytes": (T + R) * d * e + 4 * S, "flops": R * d if case["grad"] else 0}
        if op == "unpermute":
            return {"bytes": (2 * T + R) * d * e + 8 * S, "flops": 2 * R * d}
        rows = R * (d + -(-d // BLOCK)) if case["codes"] else R * d * e
        return {"bytes": (T + R) * d * e + rows + 12 * S, "flops": 3 * R * d}
    U = _used(case)
    if op == "checkpoint8":
        c = case["cols"]
        return {"bytes": U * (2 * c * e + 2 * (c + -(-c // BLOCK))), "flops": 4 * U * c}
    F = case["F"]
    return {"bytes": U * (4 * F * e + 2 * F + -(-2 * F // BLOCK)), "flops": 16 * U * F}


# ---------------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _ids(case, g):
    """Each token's K different experts in the order of their scores; slots that took a null copy
    hold N, padding holds -1."""
    T, K, N = case["T"], case["K"], case["N"]
    score = torch.rand((T, N), generator=g, device="cuda").clamp_(1e-9, 1.0 - 1e-7)
    score = -torch.log(-torch.log(score))
    if case["skew"]:
        score -= 1.1 * torch.log(torch.arange(1, N + 1, device="cuda", dtype=torch.float32))
    ids = torch.topk(score, K, dim=1).indices
    lost = torch.rand((T, K), generator=g, device="cuda") < case["drop"]
    pad = torch.rand((T, K), generator=g, device="cuda") < 0.5
    return torch.where(lost, torch.where(pad, N, -1), ids)


def _plain_sort(ids, N):
    T, K = ids.shape
    flat = ids.reshape(-1).long()
    has = (flat >= 0) & (flat < N)
    key = torch.where(has, flat, N)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(N + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    ends = torch.cumsum(counts, 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends[:N]])
    at = torch.arange(T * K, device=ids.device)
    row = torch.empty_like(order)
    row[order] = at
    slot_row = torch.where(has, row, -1).reshape(T, K)
    perm_tok = torch.where(at < offsets[N], torch.div(order, K, rounding_mode="floor"), -1)
    return counts[:N].int(), offsets.int(), perm_tok.int(), slot_row.int()


def _quantise(x):
    """codes int8 and scale bytes of each block of 32 columns (the last one may be shorter)."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = torch.zeros((rows, nb * BLOCK), dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    v = v.reshape(rows, nb, BLOCK)
    bits = v.abs().amax(2).contiguous().view(torch.int32)
    e = bits >> 23
    byte = torch.where(e == 255, 255, (e - 6).clamp(min=1))
    inv = ((254 - byte.clamp(max=253)) << 23).to(torch.int32).view(torch.float32)
    code = torch.round(v * inv[..., None]).clamp(-127, 127)
    code = torch.where((byte == 255)[..., None], 0.0, code)
    return code.reshape(rows, nb * BLOCK)[:, :cols].to(torch.int8).contiguous(), byte.to(torch.uint8)


def _values(codes, byte):
    """The fp32 values that codes and scale bytes stand for."""
    rows, cols = codes.shape
    scale = (byte.to(torch.int32) << 23).view(torch.float32)
    scale = torch.where(byte == 255, float("nan"), scale)
    return codes.float() * scale.repeat_interleave(BLOCK, 1, output_size=scale.shape[1] * BLOCK)[:, :cols]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    dev = "cuda"
    s = {"case": dict(case)}
    if op == "sort":
        T, K, N = case["T"], case["K"], case["N"]
        s["ids"] = _ids(case, g).to(torch.int64 if case["wide_ids"] else torch.int32)
        s["counts"] = torch.zeros(N, dtype=torch.int32, device=dev)
        s["offsets"] = torch.zeros(N + 1, dtype=torch.int32, device=dev)
        s["perm_tok"] = torch.full((T * K,), -1, dtype=torch.int32, device=dev)
        s["slot_row"] = torch.zeros((T, K), dtype=torch.int32, device=dev)
        return s
    dt = DTYPES[case["dtype"]]
    if op in ("permute", "unpermute", "unpermute_grad"):
        T, K, N, d = case["T"], case["K"], case["N"], case["d"]
        s["slot_row"] = _plain_sort(_ids(case, g), N)[3]
        if op == "permute" and not case["grad"]:
            s["x"] = _normal((T, d), g, dt)
            s["xs"] = torch.zeros((T * K, d), dtype=dt, device=dev)
        elif op == "permute":
            s["dxs"] = _normal((T * K, d), g, dt)
            s["base"] = _normal((T, d), g, dt)
            s["dx"] = torch.zeros((T, d), dtype=dt, device=dev)
        else:
            w = torch.softmax(_normal((T, K), g), 1)
            s["weights"] = torch.where(s["slot_row"] >= 0, w, 0.0)
            ys = _normal((T * K, d), g, dt)
            if op == "unpermute":
                s["ys"] = ys
                s["base"] = _normal((T, d), g, dt)
                s["y"] = torch.zeros((T, d), dtype=dt, device=dev)
            else:
                if case["codes"]:
                    s["codes"], s["scales"] = _quantise(ys)
                else:
                    s["ys"] = ys
                s["dy"] = _normal((T, d), g, dt, 0.1)
                s["dys"] = torch.zeros((T * K, d), dtype=dt, device=dev)
                s["dweights"] = torch.zeros((T, K), dtype=torch.float32, device=dev)
        return s
    rows = case["rows"]
    s["used"] = torch.full((1,), _used(case), dtype=torch.int32, device=dev)
    if op == "checkpoint8":
        cols = case["cols"]
        # rows of different magnitude, as tokens have them
        s["x"] = (_normal((rows, cols), g) * torch.exp(_normal((rows, 1), g))).to(dt)
        s["codes"] = torch.zeros((rows, cols), dtype=torch.int8, device=dev)
        s["scales"] = torch.zeros((rows, -(-cols // BLOCK)), dtype=torch.uint8, device=dev)
        s["restored"] = torch.zeros((rows, cols), dtype=dt, device=dev)
    else:
        F = case["F"]
        s["codes"], s["scales"] = _quantise(_normal((rows, 2 * F), g, dt, 1.5))
        s["dh"] = _normal((rows, F), g, dt, 0.1)
        s["dz"] = torch.zeros((rows, 2 * F), dtype=dt, device=dev)
        s["h"] = torch.zeros((rows, F), dtype=dt, device=dev)
    return s


# ------------------------------------------------------------------------------ plain forms


def _rows_of(slot_row, rows):
    """Index of each slot's row, with a row past the end for the slots that have none."""
    return torch.where(slot_row >= 0, slot_row, rows).reshape(-1).long()


def _place(values, slot_row, dtype):
    """values [T, K, d] at their slots' rows; zeros in the rows behind the last one."""
    T, K, d = values.shape
    out = torch.zeros((T * K + 1, d), dtype=dtype, device=values.device)
    out[_rows_of(slot_row, T * K)] = values.reshape(T * K, d).to(dtype)
    return out[:T * K]


def _fetch(rows, slot_row):
    """[T, K, d] fp32 rows of the slots, zeros where a slot has none."""
    has = (slot_row >= 0)[..., None]
    return torch.where(has, rows[slot_row.clamp(min=0).long()].float(), 0.0)


def _split(z, F, packed):
    """Gate and up columns of z [rows, 2F]: 64-column panels of each in turn, or two halves."""
    if packed:
        p = z.reshape(z.shape[0], F // 64, 2, 64)
        return p[:, :, 0].reshape(-1, F), p[:, :, 1].reshape(-1, F)
    return z[:, :F], z[:, F:]


def _join(a, b, F, packed):
    if packed:
        return torch.stack([a.reshape(-1, F // 64, 64), b.reshape(-1, F // 64, 64)], 2).reshape(-1, 2 * F)
    return torch.cat([a, b], 1)


def _below(used, v):
    """v in the rows in use, zeros behind them."""
    return torch.where((torch.arange(v.shape[0], device=v.device) < used)[:, None], v, torch.zeros((), dtype=v.dtype, device=v.device))


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "sort":
        counts, offsets, perm_tok, slot_row = _plain_sort(s["ids"], case["N"])
        return {"counts": counts, "offsets": offsets, "perm_tok": perm_tok, "slot_row": slot_row}
    dt = DTYPES[case["dtype"]]
    if op == "permute":
        if not case["grad"]:
            K = case["K"]
            return {"xs": _place(s["x"][:, None].expand(-1, K, -1), s["slot_row"], dt)}
        return {"dx": (s["base"].float() + _fetch(s["dxs"], s["slot_row"]).sum(1)).to(dt)}
    if op == "unpermute":
        y = s["base"].float() + (_fetch(s["ys"], s["slot_row"]) * s["weights"][..., None]).sum(1)
        return {"y": y.to(dt)}
    if op == "unpermute_grad":
        ys = _values(s["codes"], s["scales"]) if case["codes"] else s["ys"]
        dy = s["dy"].float()[:, None]
        dw = (_fetch(ys, s["slot_row"]) * dy).sum(2)
        return {"dys": _place(s["weights"][..., None] * dy, s["slot_row"], dt), "dweights": dw}
    if op == "checkpoint8":
        return {"restored": _below(s["used"], _values(*_quantise(s["x"])).to(dt))}
    F, packed = case["F"], case["packed"]
    a, b = _split(_values(s["codes"], s["scales"]), F, packed)
    dh = s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-a))
    da = dh * b * sig * (1.0 + a * (1.0 - sig))
    dz = _join(da, dh * a * sig, F, packed)
    return {"dz": _below(s["used"], dz.to(dt)), "h": _below(s["used"], (a * sig * b).to(dt))}


# -------------------------------------------------------------------- the framework's calls


def _workspace(s):
    """The caller's workspace, allocated once."""
    from token_choice_routing_b200 import binding as B
    if "ws" not in s:
        c = s["case"]
        s["ws"] = torch.empty(B.sort_workspace_bytes(c["T"], c["K"], c["N"]), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    from token_choice_routing_b200 import binding as B
    case = s["case"]
    op = case["op"]
    if op == "sort":
        B.sort_slots(s["ids"], case["N"], s["counts"], s["offsets"], s["perm_tok"], s["slot_row"], _workspace(s))
        return {k: s[k] for k in ("counts", "offsets", "perm_tok", "slot_row")}
    if op == "permute":
        if not case["grad"]:
            B.permute(s["x"], s["slot_row"], s["xs"])
            return {"xs": s["xs"]}
        B.permute_backward(s["dxs"], s["slot_row"], s["dx"], base=s["base"])
        return {"dx": s["dx"]}
    if op == "unpermute":
        B.unpermute(s["ys"], s["weights"], s["slot_row"], s["y"], base=s["base"])
        return {"y": s["y"]}
    if op == "unpermute_grad":
        if case["codes"]:
            B.unpermute_backward8(s["dy"], s["codes"], s["scales"], s["weights"], s["slot_row"], s["dys"], s["dweights"])
        else:
            B.unpermute_backward(s["dy"], s["ys"], s["weights"], s["slot_row"], s["dys"], s["dweights"])
        return {"dys": s["dys"], "dweights": s["dweights"]}
    if op == "checkpoint8":
        B.checkpoint8(s["x"], s["codes"], s["scales"], rows_used=s["used"])
        B.restore8(s["codes"], s["scales"], s["restored"], rows_used=s["used"])
        return {"restored": s["restored"]}
    B.swiglu_backward8(s["codes"], s["scales"], s["dh"], s["dz"], s["h"], packed=case["packed"], rows_used=s["used"])
    return {"dz": s["dz"], "h": s["h"]}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# --------------------------------------------------------------------- results in 64 bits


def _exact_values(codes, scales):
    """Values of 8-bit blocks in 64 bits: code * 2^(byte - 127), NaN for byte 255."""
    e = scales.double() - 127.0
    scale = torch.exp2(e)
    scale[scales == 255] = float("nan")
    col = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    return codes.double() * scale[:, col]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        import numpy as np
        ids = s["ids"].cpu().numpy().astype(np.int64)
        T, K = ids.shape
        N = case["N"]
        flat = ids.reshape(-1)
        rows = np.full(T * K, -1, dtype=np.int64)
        counts = np.zeros(N, dtype=np.int64)
        toks = []
        for e in range(N):
            slots = np.nonzero(flat == e)[0]
            rows[slots] = counts[:e].sum() + np.arange(slots.size)
            counts[e] = slots.size
            toks.append(slots // K)
        perm = np.concatenate(toks + [np.full(T * K - int(counts.sum()), -1, dtype=np.int64)])
        offsets = np.concatenate([[0], np.cumsum(counts)])
        out = {"counts": counts, "offsets": offsets, "perm_tok": perm, "slot_row": rows.reshape(T, K)}
        return {k: torch.from_numpy(v).int() for k, v in out.items()}
    if op in ("permute", "unpermute", "unpermute_grad"):
        T, K, d = case["T"], case["K"], case["d"]
        sr = s["slot_row"].long()
        f64 = dict(dtype=torch.float64, device="cuda")
        if op == "permute" and not case["grad"]:
            xs = torch.zeros((T * K, d), **f64)
            for k in range(K):
                t = torch.nonzero(sr[:, k] >= 0)[:, 0]
                xs[sr[t, k]] = s["x"][t].double()
            return {"xs": xs}
        if op in ("permute", "unpermute"):
            rows = s["dxs"] if op == "permute" else s["ys"]
            acc = s["base"].double()
            for k in range(K):
                t = torch.nonzero(sr[:, k] >= 0)[:, 0]
                part = rows[sr[t, k]].double()
                if op == "unpermute":
                    part *= s["weights"][t, k].double()[:, None]
                acc.index_add_(0, t, part)
            return {"dx" if op == "permute" else "y": acc}
        dys = torch.zeros((T * K, d), **f64)
        dw = torch.zeros((T, K), **f64)
        for k in range(K):
            t = torch.nonzero(sr[:, k] >= 0)[:, 0]
            r = sr[t, k]
            ys = _exact_values(s["codes"][r], s["scales"][r]) if case["codes"] else s["ys"][r].double()
            dy = s["dy"][t].double()
            dw[t, k] = (dy * ys).sum(1)
            dys[r] = dy * s["weights"][t, k].double()[:, None]
        return {"dys": dys, "dweights": dw}
    U = _used(case)
    if op == "checkpoint8":
        x = s["x"][:U].double()
        out = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
        for c0 in range(0, case["cols"], BLOCK):
            blk = x[:, c0:c0 + BLOCK]
            top = blk.abs().amax(1, keepdim=True)
            e = torch.frexp(top)[1].double() - 1.0 - 6.0  # floor(log2) - 6
            step = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -126.0)).clamp(min=-126.0))
            out[:U, c0:c0 + BLOCK] = torch.round(blk / step).clamp(-127.0, 127.0) * step
        return {"restored": out}
    F = case["F"]
    dz = torch.zeros((case["rows"], 2 * F), dtype=torch.float64, device="cuda")
    h = torch.zeros((case["rows"], F), dtype=torch.float64, device="cuda")
    j = torch.arange(F, device="cuda")
    ca = j // 64 * 128 + j % 64 if case["packed"] else j
    cb = ca + 64 if case["packed"] else j + F
    step = max(1, (1 << 26) // F)
    for r0 in range(0, U, step):
        r = slice(r0, min(U, r0 + step))
        z = _exact_values(s["codes"][r], s["scales"][r])
        a, b, g = z[:, ca], z[:, cb], s["dh"][r].double()
        sig = torch.sigmoid(a)
        dz[r, ca] = g * b * (sig + a * sig * (1.0 - sig))
        dz[r, cb] = g * a * sig
        h[r] = a * sig * b
    return {"dz": dz, "h": h}
