"""What is measured of the operators around the expert layer: tokens copied into
expert order and back with their weights, with the gradients of both, and the
MXFP4 (E2M1 codes, one UE8M0 scale per 32) quantisation and grouped product.

A case's "op" is one of
  permute    rows[inv[t, j]] = x[t]
  unpermute  out[t] = sum_j w[t, j] * rows[inv[t, j]]; with weighted = False the
             weights are 1, which is permute's gradient
  backward   unpermute's gradient: drows[inv[t, j]] = w[t, j] * dout[t] and
             dw[t, j] = <dout[t], rows[inv[t, j]]>
  quantize   x (each token's row once, or once per slot in expert order) to E2M1
             codes and UE8M0 scales, and the values that they stand for
  product    out[r] = a[r] @ w[e]^T for the rows r of each expert e, both operands
             in MXFP4, fp32 sums
with inv[t, j] the position of slot (t, j) in expert order, -1 for a masked slot.
Sizes are those of the layer's configurations (hidden size 7168, expert sizes 2048
and 1536, 32 to 64 experts, top-4 to top-8) and odd ones around them.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # One token of a decode step, sent to its experts: latency.
        dict(name="permute_one_token", op="permute", T=1, H=7168, k=8, E=32, dtype="bf16", masked=0.0),
        # A prefill batch copied into expert order: the largest copy.
        dict(name="permute_prefill", op="permute", T=8192, H=7168, k=8, E=32, dtype="bf16", masked=0.0),
        # permute's gradient in a small fp32 training step of odd sizes, some slots masked.
        dict(name="unpermute_ones_odd", op="unpermute", T=515, H=1544, k=4, E=64, dtype="fp32",
             masked=0.1, weighted=False),
        # A prefill batch's expert rows back in token order with their weights.
        dict(name="unpermute_prefill", op="unpermute", T=8192, H=7168, k=8, E=32, dtype="bf16",
             masked=0.05, weighted=True),
        # The gradient of a decode-sized fine-tuning batch: few tokens, latency.
        dict(name="backward_small", op="backward", T=37, H=7168, k=6, E=48, dtype="fp16", masked=0.0),
        # The gradient of a full training batch.
        dict(name="backward_large", op="backward", T=4096, H=7168, k=8, E=32, dtype="bf16", masked=0.05),
        # Activations of a small ragged batch, quantised in token order.
        dict(name="quantize_ragged", op="quantize", T=333, H=1568, k=1, E=1, dtype="fp16", masked=0.0,
             gathered=False),
        # A prefill batch quantised straight into expert order.
        dict(name="quantize_prefill", op="quantize", T=8192, H=7168, k=8, E=32, dtype="bf16",
             masked=0.0, gathered=True),
        # One token through the gate and up projections of its 8 experts: the weights of 8 experts stream.
        dict(name="product_one_token", op="product", T=1, H=7168, N=4096, k=8, E=32, out="bf16", skew=False),
        # A skewed decode batch: a few experts busy, some idle.
        dict(name="product_decode", op="product", T=128, H=7168, N=4096, k=8, E=32, out="bf16", skew=True),
        # A plain linear layer (one group) of odd sizes.
        dict(name="product_dense_odd", op="product", T=1001, H=2080, N=1544, k=1, E=1, out="fp16", skew=False),
        # A prefill batch through the gate and up projections: tensor-bound.
        dict(name="product_prefill", op="product", T=8192, H=7168, N=4096, k=8, E=32, out="bf16", skew=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["permute", "unpermute", "backward", "quantize", "product"])
    E = rng.choice([1, 8, 32, 48, 64, 256])
    k = rng.randint(1, min(8, E))
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    masked = rng.choice([0.0, 0.05, 0.5])
    if op == "product":
        H = 32 * _log(rng, 4, 224)
        N = 8 * _log(rng, 8, 512)
        E = min(E, 64)
        T = _log(rng, 1, 4096)
        k = min(k, E)
        return dict(op=op, T=T, H=H, N=N, k=k, E=E, out=rng.choice(["bf16", "fp16"]),
                    skew=E >= 16 and rng.random() < 0.5)
    if op == "quantize":
        gathered = rng.random() < 0.5
        T = _log(rng, 1, 8192 if dtype != "fp32" else 4096)
        k, E = (k, E) if gathered else (1, 1)
        return dict(op=op, T=T, H=32 * _log(rng, 1, 224), k=k, E=E, dtype=dtype,
                    masked=masked if gathered and T * k >= 32 else 0.0, gathered=gathered)
    T = _log(rng, 1, 4096 if dtype != "fp32" else 2048)
    # Masks in batches only: a few slots could all be masked, and nothing would be left to compare.
    c = dict(op=op, T=T, H=8 * _log(rng, 8, 896), k=k, E=E, dtype=dtype, masked=masked if T * k >= 32 else 0.0)
    if op == "unpermute":
        c["weighted"] = rng.random() < 0.6
    return c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _route(c, g):
    """Expert ids [T, k] (distinct within a token, -1 masked), and what routing makes of
    them: inv i32 [T, k], offsets i32 [E + 1], and the counts on the host."""
    T, k, E = c["T"], c["k"], c["E"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    if c.get("skew"):
        # Popularity falls with rank and the last eighth of the experts is idle.
        rank = torch.arange(1, E + 1, device="cuda", dtype=torch.float32)
        logits = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))
        logits = logits - 1.2 * rank.log()
        logits[:, E - E // 8:] = float("-inf")
        logits = logits[:, torch.randperm(E, generator=g, device="cuda")]
    ids = logits.topk(k, dim=1).indices
    if c.get("masked"):
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < c["masked"], -1, ids)
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    perm = torch.sort(key, stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device="cuda")
    inv = torch.where(flat < 0, -1, inv)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return inv.reshape(T, k).to(torch.int32), offsets.to(torch.int32), counts


def _activations(rows, cols, g, dtype):
    """Normal values with a few channels much larger than the rest."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    gain = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return (x * gain).to(dtype)


def _to_mxfp4(v):
    """fp32 [R, K] -> (E2M1 codes, two to a byte, [R, K/2]; UE8M0 bytes [R, K/32])."""
    R, K = v.shape
    b = v.reshape(R, K // 32, 32)
    n = _exponent(b.abs().amax(2))
    y = torch.ldexp(b, -n.unsqueeze(2)).reshape(R, K)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    code = code | (torch.signbit(y).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), (n + 127).to(torch.uint8)


def _exponent(amax):
    """The smallest n >= -127 with amax <= 6 * 2^n."""
    m, e = torch.frexp(amax)
    n = torch.where(m <= 0.75, e - 3, e - 2)
    return torch.where(amax > 0, n, -127).clamp(min=-127)


def _from_mxfp4(codes, scales):
    """The values of codes [..., K/2] and scales [..., K/32], fp32."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = table[nib.int()]
    s = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _group_major(scales):
    """Scale bytes [R, K/32] -> [ceil(K/128), R, 4], missing blocks 0: the product's layout."""
    R, nb = scales.shape
    g = (nb + 3) // 4
    s = torch.zeros(R, g * 4, dtype=torch.uint8, device=scales.device)
    s[:, :nb] = scales
    return s.reshape(R, g, 4).transpose(0, 1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    c = case
    s = {"case": c}
    if own:
        import moe_expert_ffn_permute_b200 as moe
        s["moe"] = moe
    T, H, k, E = c["T"], c["H"], c["k"], c["E"]
    s["inv"], s["offsets"], counts = _route(c, g)
    S = T * k
    if c["op"] == "product":
        N = c["N"]
        x = _activations(T, H, g, torch.float32)
        codes, scales = _to_mxfp4(x)
        # Each token's row at its slots' positions, as the gathering quantiser leaves them.
        token = torch.empty(S, dtype=torch.int64, device="cuda")
        token[s["inv"].reshape(-1).long()] = torch.arange(S, device="cuda") // k
        s["codes"], s["row_scales"] = codes[token], scales[token]
        s["scales"] = _group_major(s["row_scales"])
        w = torch.empty(E, N, H // 2, dtype=torch.uint8, device="cuda")
        ws = torch.empty(E, N, H // 32, dtype=torch.uint8, device="cuda")
        for e in range(E):
            w[e], ws[e] = _to_mxfp4(torch.randn(N, H, generator=g, device="cuda") * 0.02)
        s["most"] = int(counts.max())
        if own:
            # Weights are laid out once, when a model is loaded.
            s["w"] = torch.empty(moe.moe_mxfp4_weight_bytes(E, N, H), dtype=torch.uint8, device="cuda")
            s["ws"] = torch.empty(moe.moe_mxfp4_weight_scale_bytes(E, N, H), dtype=torch.uint8, device="cuda")
            moe.moe_mxfp4_prepack(w, ws, E, N, H, s["w"], s["ws"])
            s["workspace"] = torch.zeros(moe.moe_mxfp4_workspace_bytes(S, E, N, H), dtype=torch.uint8,
                                         device="cuda")
            s["out"] = torch.empty(S, N, dtype=DTYPES[c["out"]], device="cuda")
        else:
            s["w"], s["ws"] = w, ws
        return s
    dt = DTYPES[c["dtype"]]
    if c["op"] in ("permute", "quantize"):
        s["x"] = _activations(T, H, g, dt)
    else:
        s["rows"] = torch.randn(S, H, generator=g, device="cuda").to(dt)
        s["topk_w"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    if c["op"] == "backward":
        s["dout"] = torch.randn(T, H, generator=g, device="cuda").to(dt)
    if own:
        # Buffers that a program keeps; rows behind the last routed one stay zero.
        if c["op"] == "permute":
            s["rows"] = torch.zeros(S, H, dtype=dt, device="cuda")
        elif c["op"] == "unpermute":
            s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
        elif c["op"] == "backward":
            s["drows"] = torch.zeros(S, H, dtype=dt, device="cuda")
            s["dw"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
        else:
            s["codes"] = torch.zeros(S, H // 2, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.zeros((H + 127) // 128, S, 4, dtype=torch.uint8, device="cuda")
            s["values"] = torch.empty(S, H, dtype=torch.bfloat16, device="cuda")
    return s


def _kernels(s, c):
    moe, T, H, k, E = s["moe"], c["T"], c["H"], c["k"], c["E"]
    if c["op"] == "permute":
        moe.moe_permute(s["x"], T, H * s["x"].element_size(), k, s["inv"], s["rows"])
        return s["rows"]
    if c["op"] == "unpermute":
        if c["weighted"]:
            moe.moe_unpermute(s["rows"], c["dtype"], T, H, k, s["inv"], s["topk_w"], s["out"])
        else:
            moe.moe_permute_backward(s["rows"], c["dtype"], T, H, k, s["inv"], s["out"])
        return s["out"]
    if c["op"] == "backward":
        moe.moe_unpermute_backward(s["dout"], s["rows"], c["dtype"], T, H, k, s["inv"], s["topk_w"],
                                   s["drows"], s["dw"])
        return {"drows": s["drows"], "dw": s["dw"]}
    if c["op"] == "quantize":
        inv = s["inv"] if c["gathered"] else None
        moe.moe_quantize_mxfp4(s["x"], c["dtype"], T, H, k, inv, s["codes"], s["scales"], "group")
        moe.moe_dequantize_mxfp4(s["codes"], s["scales"], "group", T * k, H, "bf16", s["values"])
        return s["values"]
    moe.moe_mxfp4_gemm(s["codes"], s["scales"], s["offsets"], T * k, E, c["N"], H, s["w"], s["ws"],
                       c["out"], s["out"], s["workspace"])
    return s["out"]


def _slots(inv):
    """Positions and flat slots of the routed slots."""
    flat = inv.reshape(-1).long()
    slot = (flat >= 0).nonzero().squeeze(1)
    return flat[slot], slot


def run(state):
    s, c = state, state["case"]
    if own:
        return _kernels(s, c)
    T, H, k, E = c["T"], c["H"], c["k"], c["E"]
    if c["op"] == "permute":
        pos, slot = _slots(s["inv"])
        rows = torch.zeros(T * k, H, dtype=s["x"].dtype, device="cuda")
        rows[pos] = s["x"][slot // k]
        return rows
    if c["op"] == "unpermute":
        inv = s["inv"].long()
        r = s["rows"][inv.clamp(min=0)].float()
        w = s["topk_w"] if c["weighted"] else torch.ones_like(s["topk_w"])
        r = torch.where((inv >= 0).unsqueeze(2), r * w.unsqueeze(2), 0.0)
        return r.sum(1).to(s["rows"].dtype)
    if c["op"] == "backward":
        inv = s["inv"].long()
        pos, slot = _slots(s["inv"])
        dout = s["dout"].float()
        drows = torch.zeros(T * k, H, dtype=s["rows"].dtype, device="cuda")
        drows[pos] = (dout[slot // k] * s["topk_w"].reshape(-1)[slot].unsqueeze(1)).to(drows.dtype)
        dot = (s["rows"][inv.clamp(min=0)].float() * dout.unsqueeze(1)).sum(2)
        return {"drows": drows, "dw": torch.where(inv >= 0, dot, 0.0)}
    if c["op"] == "quantize":
        codes, scales = _to_mxfp4(s["x"].float())
        v = _from_mxfp4(codes, scales).to(torch.bfloat16)
        if not c["gathered"]:
            return v
        pos, slot = _slots(s["inv"])
        out = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
        out[pos] = v[slot // k]
        return out
    # Each expert's rows, filled up to the longest group, times its weights.
    a = _from_mxfp4(s["codes"], s["row_scales"])
    off = s["offsets"].long()
    row = torch.arange(T * k, device="cuda")
    e = torch.searchsorted(off[1:], row, right=True)
    at = row - off[e]
    pad = torch.zeros(E, s["most"], H, device="cuda")
    pad[e, at] = a
    out = torch.bmm(pad, _from_mxfp4(s["w"], s["ws"]).transpose(1, 2))
    return out[e, at].to(DTYPES[c["out"]])


def work(case):
    c = case
    T, H, k, E = c["T"], c["H"], c["k"], c["E"]
    S = T * k
    if c["op"] == "product":
        N = c["N"]
        live = E - E // 8 if c["skew"] else E
        active = live * (1.0 - (1.0 - min(1.0, k / live)) ** T)   # experts that get a row
        per = H / 2 + H / 32
        return {"bytes": active * N * per + S * per + S * N * 2, "flops": 2.0 * S * N * H}
    size = 4 if c["dtype"] == "fp32" else 2
    R = S * (1.0 - c["masked"])                                   # routed slots
    if c["op"] == "permute":
        return {"bytes": (T + R) * H * size + 4 * S, "flops": 0.0}
    if c["op"] == "unpermute":
        return {"bytes": (T + R) * H * size + 8 * S, "flops": 2.0 * R * H}
    if c["op"] == "backward":
        return {"bytes": (T + 2 * R) * H * size + 12 * S, "flops": 3.0 * R * H}
    # x once, the codes and scales, and the values that they stand for.
    return {"bytes": T * H * size + R * (H / 2 + H / 32) + S * H * 2, "flops": 4.0 * T * H}


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    c, s = case, prepare(case, seed)
    T, H, k, E = c["T"], c["H"], c["k"], c["E"]
    inv = s["inv"].reshape(-1).long()
    if c["op"] == "product":
        grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        value = torch.tensor(grid + [-v for v in grid], dtype=torch.float64, device="cuda")

        def decode(codes, scales):
            v = torch.empty(codes.shape[0], H, dtype=torch.float64, device="cuda")
            v[:, 0::2] = value[(codes % 16).long()]
            v[:, 1::2] = value[(codes // 16).long()]
            return v * torch.pow(2.0, scales.double() - 127.0).repeat_interleave(32, 1)

        out = torch.zeros(T * k, c["N"], dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        w = s["w"]
        for e in range(E):
            if off[e + 1] > off[e]:
                rows = slice(off[e], off[e + 1])
                out[rows] = decode(s["codes"][rows], s["row_scales"][rows]) @ decode(w[e], s["ws"][e]).T
        return out
    if c["op"] == "permute":
        out = torch.zeros(T * k + 1, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            out[inv[j::k]] = s["x"].double()       # -1 is the spare last row
        return out[:-1]
    if c["op"] == "unpermute":
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            p = inv[j::k]
            got = (p >= 0).nonzero().squeeze(1)
            w = s["topk_w"][got, j].double() if c["weighted"] else torch.ones(len(got), device="cuda").double()
            out[got] += s["rows"][p[got]].double() * w[:, None]
        return out
    if c["op"] == "backward":
        drows = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        dout = s["dout"].double()
        for j in range(k):
            p = inv[j::k]
            got = (p >= 0).nonzero().squeeze(1)
            drows[p[got]] = dout[got] * s["topk_w"][got, j].double()[:, None]
            dw[got, j] = torch.linalg.vecdot(dout[got], s["rows"][p[got]].double())
        return {"drows": drows, "dw": dw}
    x = s["x"].double().reshape(T, H // 32, 32)
    amax = x.abs().amax(2, keepdim=True)
    n = torch.ceil(torch.log2((amax / 6.0).clamp(min=2.0 ** -127)))
    n = torch.where(amax > 6.0 * torch.pow(2.0, n), n + 1, n)
    n = torch.where((amax <= 6.0 * torch.pow(2.0, n - 1)) & (n > -127), n - 1, n)
    y = x / torch.pow(2.0, n)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).double()
    v = (torch.round(y / step) * step * torch.pow(2.0, n)).reshape(T, H)   # round: ties to even
    if not c["gathered"]:
        return v
    out = torch.zeros(T * k + 1, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        out[inv[j::k]] = v
    return out[:-1]
