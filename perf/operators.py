"""Measured cases of the grouped expert products, the 8-bit activation
checkpoints and the 4-bit expert products: what each computes in plain torch,
and the calls a user makes of the library for the same.

Rows are grouped by expert: row i belongs to the expert e with
offsets[e] <= i < offsets[e+1].  The routing draws top_k experts per token
from random logits (some with a Zipf-like preference), and `ids` lists the
token-expert pairs in that order.

Operators ("op"):
  fwd    y = W[e] a            gather: a = x[ids / top_k]; scatter: y to pair order
  dgrad  da = W[e]^T dy        gather: dy of the token; scatter: da to pair order
  wgrad  dW[e] = sum dy a^T    gather: a = x[ids / top_k]
  save   h = w SiLU(g) u, and (g, u) kept in 8 bits
  grad   gradients of the same from the 8 bits
  w4     y = W[e] a with 4-bit weights ("mxfp4" or "int4")
"""
import math

import torch

own = False

GROUP = 32  # values per scale of a checkpoint
W4_GROUP = {"mxfp4": 32, "int4": 128}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _product(op, name, tokens, top_k, E, N, K, skew, gather, scatter, out, fmt="bf16"):
    return dict(name=name, op=op, tokens=tokens, top_k=top_k, E=E, N=N, K=K, skew=skew, gather=gather,
                scatter=scatter, out=out, fmt=fmt)


def listed():
    return [
        # four decoding users of a 128-expert layer with bf16 experts: latency and the weights' stream
        _product("fwd", "fwd_few_tokens", 4, 8, 128, 1536, 2048, 0.0, True, False, "bf16"),
        # the same layer's gate/up product over a 4096-token training batch
        _product("fwd", "fwd_gate_up_128", 4096, 8, 128, 1536, 2048, 0.5, True, False, "bf16"),
        # the down product of an 8-expert layer, results back in pair order
        _product("fwd", "fwd_down_8", 4096, 2, 8, 4096, 14336, 0.0, False, True, "bf16"),
        # a small layer of odd sizes, some experts nearly empty
        _product("dgrad", "dgrad_small_odd", 77, 2, 8, 520, 264, 1.0, True, False, "bf16"),
        # gradient of the hidden states through the 8-expert layer's gate/up weights
        _product("dgrad", "dgrad_gate_up_8", 4096, 2, 8, 28672, 4096, 0.0, False, True, "bf16"),
        # weight gradients of a middling layer of odd sizes, in bf16
        _product("wgrad", "wgrad_odd", 333, 3, 7, 776, 1032, 0.5, True, False, "bf16"),
        # weight gradients of the 8-expert layer's down product, fp32 as the optimizer keeps them
        _product("wgrad", "wgrad_down_8", 4096, 2, 8, 4096, 14336, 0.0, False, False, "fp32"),
        # activation of the 128-expert layer's training batch, kept in 8 bits
        dict(name="save_128", op="save", rows=32768, I=768, weighted=False),
        # its gradient for the 8-expert layer, with the routing weights' gradient
        dict(name="grad_8", op="grad", rows=8192, I=14336, weighted=True),
        # one decoding user, 8-expert layer in MXFP4
        _product("w4", "w4_one_token_8", 1, 2, 8, 28672, 4096, 0.0, True, False, "bf16", "mxfp4"),
        # 32 users, the 128-expert layer's down product in int4 with scales per 128
        _product("w4", "w4_down_128", 32, 8, 128, 2048, 768, 0.0, False, True, "bf16", "int4"),
        # 64 users, the 256-expert layer's gate/up product in MXFP4
        _product("w4", "w4_gate_up_256", 64, 8, 256, 4096, 7168, 0.5, True, False, "bf16", "mxfp4"),
    ]


def _log(rng, lo, hi, step=1):
    return max(step, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(("fwd", "fwd", "dgrad", "dgrad", "wgrad", "wgrad", "save", "grad", "w4", "w4"))
    if op in ("save", "grad"):
        while True:
            rows, I = _log(rng, 1, 65536), _log(rng, 64, 16384, 8)
            if rows * I <= 8192 * 14336:
                return dict(op=op, rows=rows, I=I, weighted=rng.random() < 0.5)
    while True:
        E = _log(rng, 2, 256)
        top_k = rng.randint(1, min(8, E))
        fmt = rng.choice(("mxfp4", "int4")) if op == "w4" else "bf16"
        step = W4_GROUP.get(fmt, 8)
        N = _log(rng, 128, 16384, 8)
        K = _log(rng, 128, 16384, step)
        tokens = _log(rng, 1, 256 if op == "w4" else 8192)
        work = tokens * top_k * N * K
        if E * N * K <= 8 * 4096 * 14336 and work <= 8192 * 4096 * 14336:
            case = _product(op, "", tokens, top_k, E, N, K, rng.choice((0.0, 0.5, 1.0)), rng.random() < 0.5,
                            op != "wgrad" and rng.random() < 0.3, "fp32" if rng.random() < 0.3 else "bf16", fmt)
            del case["name"]
            return case


def _active(case):
    """Expected number of experts that hold rows (uniform routing)."""
    return case["E"] * (1.0 - (1.0 - case["top_k"] / case["E"]) ** case["tokens"])


def work(case):
    if case["op"] in ("save", "grad"):
        n = case["rows"] * case["I"]
        scales = 2 * case["rows"] * -(-case["I"] // GROUP)
        vec = 4 * case["rows"] if case["weighted"] else 0
        if case["op"] == "save":  # gate and up in, h and the codes out
            return {"bytes": 4 * n + 2 * n + 2 * n + scales + vec, "flops": 8 * n}
        return {"bytes": 2 * n + scales + 2 * n + 6 * n + 4 * case["rows"] + vec, "flops": 20 * n}
    R, E, N, K = case["tokens"] * case["top_k"], case["E"], case["N"], case["K"]
    src, dst = (N, K) if case["op"] == "dgrad" else (K, N)
    out = 4 if case["out"] == "fp32" else 2
    rows_in = case["tokens"] if case["gather"] else R
    index = 4 * R * (int(case["gather"]) + int(case["scatter"])) + 4 * (E + 1)
    if case["op"] == "wgrad":
        return {"bytes": 2 * (R * N + rows_in * K) + out * E * N * K + index, "flops": 2 * R * N * K}
    weight = {"bf16": 2.0, "mxfp4": 0.5 + 1 / 32, "int4": 0.5 + 2 / 128}[case["fmt"]] * _active(case) * N * K
    return {"bytes": int(2 * rows_in * src + weight + out * R * dst + index), "flops": 2 * R * N * K}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    st = {"case": case}
    if case["op"] in ("save", "grad"):
        R, I = case["rows"], case["I"]
        # gate and up values of a layer with unit-variance hidden states; rows of different size
        gu = _normal(g, R, 2 * I) * torch.exp(0.5 * _normal(g, R, 1))
        st["gu"] = gu
        st["row_weight"] = torch.rand(R, generator=g, device="cuda") if case["weighted"] else None
        if case["op"] == "grad":
            st["codes"], st["scales"] = _encode(gu)
            st["dh"] = _normal(g, R, I)
            del st["gu"]
        return st
    T, k, E, N, K = case["tokens"], case["top_k"], case["E"], case["N"], case["K"]
    R = T * k
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits -= case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    experts = torch.topk(logits, k, dim=1).indices.reshape(-1)
    order = torch.argsort(experts, stable=True)
    counts = torch.bincount(experts, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    st["offsets"] = offsets
    st["bounds"] = offsets.tolist()  # the routing's result as the host has it in the plain form
    st["ids"] = order.to(torch.int32)
    src = N if case["op"] == "dgrad" else K
    rows = T if case["gather"] else R
    if case["op"] == "wgrad":
        st["dy"] = _normal(g, R, N) * 0.125
        st["a"] = _normal(g, rows, K)
    else:
        st["a"] = _normal(g, rows, src)
    if case["op"] in ("fwd", "dgrad"):
        st["w"] = _normal(g, E, N, K) * (K ** -0.5)
    if case["op"] == "w4":
        st["w4"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        groups = K // W4_GROUP[case["fmt"]]
        if case["fmt"] == "mxfp4":
            st["scales"] = torch.randint(118, 122, (E, N, groups), generator=g, device="cuda", dtype=torch.uint8)
        else:
            st["scales"] = (torch.rand(E, N, groups, generator=g, device="cuda") * 0.01 + 0.002).to(torch.bfloat16)
    return st


# ------------------------------------------------------------------ plain forms
def _scale_code(amax):
    """E8M0 code of the smallest power of two under which amax (fp32) does not
    pass 448: its exponent - 8, one more where its mantissa is above 1.75."""
    bits = amax.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp(min=0)


def _pow2(code):
    """2^(code - 127) of E8M0 codes (int32), made from the bits."""
    return torch.where(code > 0, code << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _encode(gu):
    """bf16 [R, 2I] -> e4m3 codes [R, 2I] and E8M0 scale codes [R, 2, ceil(I/32)]."""
    R, I = gu.shape[0], gu.shape[1] // 2
    v = torch.nn.functional.pad(gu.float().view(R, 2, I), (0, -I % GROUP)).view(R, 2, -1, GROUP)
    code = _scale_code(v.abs().amax(-1))
    q = (v * _pow2(254 - code)[..., None]).to(torch.float8_e4m3fn)
    return q.reshape(R, 2, -1)[:, :, :I].reshape(R, 2 * I).view(torch.uint8), code.to(torch.uint8)


def _decode(codes, scales):
    """The values that a checkpoint stands for, fp32 [R, 2, I]."""
    R, I = codes.shape[0], codes.shape[1] // 2
    s = _pow2(scales.to(torch.int32)).repeat_interleave(GROUP, dim=2)[:, :, :I]
    return codes.view(torch.float8_e4m3fn).float().view(R, 2, I) * s


def _save_plain(gu, row_weight):
    I = gu.shape[1] // 2
    g, u = gu[:, :I].float(), gu[:, I:].float()
    h = g / (1.0 + torch.exp(-g)) * u
    if row_weight is not None:
        h = h * row_weight[:, None]
    return (h.to(torch.bfloat16),) + _encode(gu)


def _grad_plain(codes, scales, dh, row_weight):
    v = _decode(codes, scales)
    g, u, d = v[:, 0], v[:, 1], dh.float()
    s = 1.0 / (1.0 + torch.exp(-g))
    silu = g * s
    h = silu * u
    dw = (d * h).sum(1)
    if row_weight is not None:
        d = d * row_weight[:, None]
        h = h * row_weight[:, None]
    dgu = torch.cat((d * u * s * (1.0 + g * (1.0 - s)), d * silu), dim=1)
    return dgu.to(torch.bfloat16), h.to(torch.bfloat16), dw


def _w4_values(codes, scales, fmt):
    """4-bit codes [N, K/2] (low nibble first) and their scales -> fp32 [N, K]."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).view(codes.shape[0], -1)
    if fmt == "mxfp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        v, s = table[q.int()], _pow2(scales.int())
    else:
        v, s = q.float() - 8.0, scales.float()
    return (v.view(codes.shape[0], scales.shape[1], -1) * s[..., None]).view(codes.shape[0], -1)


def _product_plain(st):
    c = st["case"]
    dtype = torch.float32 if c["out"] == "fp32" else torch.bfloat16
    a = st["a"][st["ids"].long() // c["top_k"]].float() if c["gather"] else st["a"].float()
    R, E, N, K = c["tokens"] * c["top_k"], c["E"], c["N"], c["K"]
    if c["op"] == "wgrad":
        out, dy = torch.zeros(E, N, K, device=a.device, dtype=dtype), st["dy"].float()
    else:
        out = torch.empty(R, K if c["op"] == "dgrad" else N, device=a.device, dtype=torch.float32)
    # one matrix product for each expert that holds rows
    for e, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        if lo == hi:
            continue
        if c["op"] == "wgrad":
            out[e] = (dy[lo:hi].t() @ a[lo:hi]).to(dtype)
        elif c["op"] == "dgrad":
            out[lo:hi] = a[lo:hi] @ st["w"][e].float()
        else:
            w = st["w"][e].float() if c["op"] == "fwd" else _w4_values(st["w4"][e], st["scales"][e], c["fmt"])
            out[lo:hi] = a[lo:hi] @ w.t()
    out = out.to(dtype)
    if c["scatter"]:
        placed = torch.empty_like(out)
        placed[st["ids"].long()] = out
        return placed
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "save":
            h, codes, scales = _save_plain(state["gu"], state["row_weight"])
        elif c["op"] == "grad":
            return dict(zip(("dgu", "h", "dweight"), _grad_plain(state["codes"], state["scales"], state["dh"],
                                                                  state["row_weight"])))
        else:
            return _product_plain(state)
    else:
        import moe_layer_align_amd as moe
        dtype = torch.float32 if c.get("out") == "fp32" else torch.bfloat16
        if c["op"] == "save":
            h, codes, scales = moe.swiglu_checkpoint(state["gu"], row_weight=state["row_weight"])
        elif c["op"] == "grad":
            dgu, h, dw = moe.swiglu_checkpoint_grad(state["codes"], state["scales"], state["dh"],
                                                    row_weight=state["row_weight"])
            return {"dgu": dgu, "h": h, "dweight": dw}
        else:
            rows = state["ids"] if c["gather"] else None
            to = state["ids"] if c["scatter"] else None
            if c["op"] == "fwd":
                return moe.grouped_gemm(state["a"], state["w"], state["offsets"], a_rows=rows, a_div=c["top_k"],
                                        out_rows=to, out_dtype=dtype)
            if c["op"] == "dgrad":
                return moe.grouped_gemm_dgrad(state["a"], state["w"], state["offsets"], dy_rows=rows,
                                              dy_div=c["top_k"], out_rows=to, out_dtype=dtype)
            if c["op"] == "wgrad":
                return moe.grouped_gemm_wgrad(state["dy"], state["a"], state["offsets"], a_rows=rows,
                                              a_div=c["top_k"], out_dtype=dtype)
            return moe.grouped_gemm_w4(state["a"], state["w4"], state["scales"], state["offsets"], a_rows=rows,
                                       a_div=c["top_k"], out_rows=to, out_dtype=dtype)
    return {"h": h, "codes": codes.view(torch.float8_e4m3fn), "scales": scales}


# ------------------------------------------------------------------ 64 bits
def _grid_round(v):
    """float64 -> the nearest e4m3 value (ties to even), |v| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] == "save":
        I, gu = case["I"], st["gu"].to(d)
        g, u = gu[:, :I], gu[:, I:]
        h = g * torch.sigmoid(g) * u
        if st["row_weight"] is not None:
            h = h * st["row_weight"].to(d)[:, None]
        halves = torch.stack((g, u), 1)
        n = -(-I // GROUP)
        full = torch.zeros(case["rows"], 2, n * GROUP, dtype=d, device=gu.device)
        full[:, :, :I] = halves
        blocks = full.view(case["rows"], 2, n, GROUP)
        top = blocks.abs().amax(-1)
        scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -126) / 448.0)))
        scale = torch.where(top > 448.0 * scale, 2 * scale, scale).clamp(min=2.0 ** -127)
        values = _grid_round(blocks / scale[..., None])
        values = values.view(case["rows"], 2, -1)[:, :, :I].reshape(case["rows"], 2 * I)
        return {"h": h, "codes": values, "scales": None}
    if case["op"] == "grad":
        R, I = case["rows"], case["I"]
        bits = st["codes"].to(torch.int64)
        e, m = (bits >> 3) & 15, bits & 7
        mag = torch.where(e > 0, torch.ldexp((8 + m).to(d), e - 10), torch.ldexp(m.to(d), torch.full_like(e, -9)))
        v = torch.where(bits >= 128, -mag, mag).view(R, 2, I)
        of = torch.arange(I, device=v.device) // GROUP
        v = torch.ldexp(v, (st["scales"].to(torch.int64) - 127)[:, :, of])
        g, u, dh = v[:, 0], v[:, 1], st["dh"].to(d)
        w = st["row_weight"].to(d)[:, None] if st["row_weight"] is not None else 1.0
        s = torch.sigmoid(g)
        return {"dgu": torch.cat((w * dh * u * (s + g * s * torch.sigmoid(-g)), w * dh * g * s), 1),
                "h": w * g * s * u, "dweight": (dh * g * s * u).sum(1)}
    T, k, E, N, K = (case[n] for n in ("tokens", "top_k", "E", "N", "K"))
    pos = torch.arange(T * k, device="cuda")
    owner = torch.searchsorted(st["offsets"][1:].contiguous(), pos.to(torch.int32), right=True)
    ids = st["ids"].long()
    pick = (lambda sel: st["a"][torch.div(ids[sel], k, rounding_mode="floor")].to(d)) if case["gather"] else \
        (lambda sel: st["a"][sel].to(d))
    out = torch.zeros((E, N, K) if case["op"] == "wgrad" else (T * k, K if case["op"] == "dgrad" else N), dtype=d,
                      device="cuda")
    for e in torch.unique(owner).tolist():
        sel = torch.nonzero(owner == e).flatten()
        if case["op"] == "wgrad":
            out[e] = torch.matmul(pick(sel).t(), st["dy"][sel].to(d)).t()
            continue
        if case["op"] == "w4":
            c = st["w4"][e].to(torch.int64)
            q = torch.empty(N, K, dtype=torch.int64, device="cuda")
            q[:, 0::2], q[:, 1::2] = c % 16, c // 16
            if case["fmt"] == "int4":
                w = (q - 8).to(d) * st["scales"][e].to(d)[:, torch.arange(K, device="cuda") // 128]
            else:
                ex, m = (q >> 1) & 3, q & 1
                mag = torch.where(ex > 0, torch.ldexp((2 + m).to(d), ex - 2), m.to(d) / 2)
                w = torch.where(q >= 8, -mag, mag)
                w = torch.ldexp(w, (st["scales"][e].to(torch.int64) - 127)[:, torch.arange(K, device="cuda") // 32])
        else:
            w = st["w"][e].to(d)
        r = torch.matmul(w.t() if case["op"] == "dgrad" else w, pick(sel).t()).t()
        out[ids[sel] if case["scatter"] else sel] = r
    return out
