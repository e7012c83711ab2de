"""The training operators around the experts, as measured cases.

A mixture block in training form is: layer norm (with the residual stream
added in front of it), routing, tokens copied into expert order (permute), the
experts' products, the rows weighted and summed back into tokens (unpermute);
then the gradients of all of these, and an AdamW step over the block's
parameters.  Each case below is one of these calls at one size.

``own`` False computes a case in elementary torch operations in 32 bits;
True makes the framework's calls on the same state.
"""
import math
import random

import torch

own = False

_DT = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
_BYTES = {"bfloat16": 2, "float16": 2, "float32": 4}

# The prefill batch of the benchmark: 32768 tokens, 16 picks, hidden 3584.
_MOST_ROW_ELEMS = 32768 * 16 * 3584
_MOST_NORM_ELEMS = 32768 * 3584
_MOST_PARAMS = 144_000_000


# ------------------------------------------------------------------ the cases
def _norm(name, which, rows, cols, dtype, w_dtype, residual):
    c = {"op": "norm", "pass": which, "rows": rows, "cols": cols, "dtype": dtype, "w_dtype": w_dtype,
         "residual": residual}
    return dict(c, name=name) if name else c


def _tokens(name, op, which, T, E_global, E_local, offset, top_k, shared, hidden, dtype, zipf):
    c = {"op": op, "pass": which, "T": T, "E_global": E_global, "E_local": E_local, "offset": offset, "top_k": top_k,
         "shared": shared, "hidden": hidden, "dtype": dtype, "zipf": zipf}
    return dict(c, name=name) if name else c


def _route(name, T, E_global, top_k, shared):
    c = {"op": "route", "pass": "backward", "T": T, "E_global": E_global, "top_k": top_k, "shared": shared}
    return dict(c, name=name) if name else c


def _adamw(name, tensors, params, grad, state, clip):
    c = {"op": "adamw", "pass": "step", "tensors": tensors, "params": params, "grad": grad, "state": state,
         "clip": clip}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode batch in front of the layer: only latency counts
        _norm("norm_decode", "forward", 32, 3584, "bfloat16", "same", True),
        # the prefill batch
        _norm("norm_prefill", "forward", 32768, 3584, "bfloat16", "same", True),
        # a row length that no vector width divides, in full precision (a small model's test or a probe head)
        _norm("norm_grad_ragged", "backward", 4099, 1021, "float32", "float32", False),
        # the prefill batch's gradient: the residual gradient joined, weights kept in 32 bits
        _norm("norm_grad_prefill", "backward", 32768, 3584, "bfloat16", "float32", True),
        # a decode batch sorted into 896 experts
        _tokens("permute_decode", "permute", "forward", 32, 896, 896, 0, 16, 0, 3584, "bfloat16", 0.0),
        # the gradient of an expert-parallel rank's half of the experts, with a shared expert, at an odd length
        _tokens("permute_grad_slice", "permute", "backward", 8189, 896, 448, 448, 16, 1, 3584, "bfloat16", 0.0),
        # the prefill batch summed back into tokens
        _tokens("unpermute_prefill", "unpermute", "forward", 32768, 896, 896, 0, 16, 0, 3584, "bfloat16", 0.0),
        # a skewed training batch: gradients of the rows and of the routing weights
        _tokens("unpermute_grad_skewed", "unpermute", "backward", 4096, 896, 896, 0, 16, 1, 3584, "bfloat16", 1.1),
        # the router's gradient of a short batch with a shared expert, and of the prefill batch
        _route("route_grad_short", 256, 896, 16, 1),
        _route("route_grad_prefill", 32768, 896, 16, 0),
        # a few large matrices with 32-bit states; many tensors of all sizes with 8-bit states
        _adamw("adamw_large", 5, 128_000_000, "bfloat16", "float32", True),
        _adamw("adamw_many_8bit", 320, 96_000_000, "bfloat16", "mxfp8", False),
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over its logarithm: half of them odd, half a multiple of 56, as the block's
    usual hidden sizes are (small ones as they come)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v < 112:
        return max(lo, min(hi, v))
    return min(hi, v // 56 * 56) if rng.random() < 0.5 else min(hi - 1 + hi % 2, v | 1)


def draw(rng):
    op = rng.choice(("norm", "norm", "permute", "permute", "unpermute", "unpermute", "route", "adamw"))
    if op == "norm":
        cols = _size(rng, 64, 8192)
        rows = _size(rng, 1, min(32768, _MOST_NORM_ELEMS // cols))
        dtype = rng.choice(("bfloat16", "bfloat16", "float16", "float32"))
        if dtype == "float32":
            rows = max(1, rows // 2)
        return _norm(None, rng.choice(("forward", "backward")), rows, cols, dtype, rng.choice(("same", "float32")),
                     rng.random() < 0.5)
    if op in ("permute", "unpermute"):
        hidden = _size(rng, 64, 7168)
        shared = rng.choice((0, 0, 1))
        E = rng.choice((8, 60, 128, 256, 384, 896))
        parts = rng.choice((1, 1, 2, 4))
        local = E // parts
        top_k = min(rng.choice((1, 2, 4, 6, 8, 10, 16)), E)
        most = min(32768, _MOST_ROW_ELEMS // (2 * hidden * (top_k + shared)))
        least = 1 if parts == 1 else 56  # a slice of the experts takes a batch that has tokens for it
        return _tokens(None, op, rng.choice(("forward", "backward")), _size(rng, least, most), E, local,
                       local * rng.randrange(parts), top_k, shared, hidden,
                       rng.choice(("bfloat16", "bfloat16", "float16", "float32")), rng.choice((0.0, 0.0, 1.1)))
    if op == "route":
        E = rng.choice((8, 60, 127, 256, 384, 896, 1024))
        return _route(None, _size(rng, 1, 32768), E, min(rng.choice((2, 6, 8, 16, 32)), E), rng.choice((0, 1)))
    tensors = _size(rng, 1, 400)
    return _adamw(None, tensors, max(tensors * 64, _size(rng, 4096, _MOST_PARAMS // 2)),
                  rng.choice(("bfloat16", "float32")), rng.choice(("float32", "mxfp8")), rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _filled(g, rows, cols, dt, scale=1.0):
    """Normal values of a large matrix, written in its own type."""
    out = torch.empty((rows, cols), device="cuda", dtype=dt)
    out.normal_(0.0, scale, generator=g)
    return out


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm":
        _prepare_norm(case, g, s)
    elif case["op"] in ("permute", "unpermute"):
        _prepare_tokens(case, g, s)
    elif case["op"] == "route":
        _prepare_route(case, g, s)
    else:
        _prepare_adamw(case, g, s)
    return s


def _prepare_norm(case, g, s):
    rows, cols, dt = case["rows"], case["cols"], _DT[case["dtype"]]
    wdt = dt if case["w_dtype"] == "same" else torch.float32
    # a residual stream: some channels are much larger than the rest, and the mean is not zero
    channel = 1.0 + 3.0 * _randn(g, cols).square()
    s["weight"] = (1.0 + 0.1 * _randn(g, cols)).to(wdt)
    s["bias"] = (0.1 * _randn(g, cols) + 0.02).to(wdt)
    s["x"] = _filled(g, rows, cols, dt)
    s["x"].mul_(channel.to(dt)).add_(0.25)
    s["residual"] = None
    s["eps"] = 1e-5
    like = torch.empty_like
    if case["pass"] == "forward":
        if case["residual"]:
            s["residual"] = _filled(g, rows, cols, dt, 0.5)
        s["y"], s["h"] = like(s["x"]), like(s["x"]) if case["residual"] else None
        s["mean"] = torch.empty(rows, device="cuda")
        s["rstd"] = torch.empty(rows, device="cuda")
        return
    x = s["x"].float()
    s["mean"] = x.mean(1)
    s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + s["eps"])
    del x
    s["dy"] = _filled(g, rows, cols, dt, 0.1)
    s["dh"] = _filled(g, rows, cols, dt, 0.1) if case["residual"] else None
    s["dx"] = like(s["x"])
    s["dweight"] = torch.empty(cols, device="cuda")
    s["dbias"] = torch.empty(cols, device="cuda")
    if own:  # the scratch that a program keeps
        import mxfp4_mixture_experts_02_gb300 as moe

        s["ws"] = moe.layer_norm_workspace(rows, cols)


def _pick(case, g):
    """Routing of normal logits (with a popularity bias where the case has one): ids and renormalised weights, the
    shared expert last."""
    T, E, k = case["T"], case["E_global"], case["top_k"]
    logits = _randn(g, T, E)
    if case.get("zipf"):
        logits -= case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    top, ids = torch.topk(logits, k, dim=1)
    w = torch.softmax(top, dim=1)
    ids = ids.to(torch.int32)
    z = None
    if case["shared"]:
        z = _randn(g, T, 1).to(torch.bfloat16)
        ids = torch.cat([ids, torch.full((T, 1), E, device="cuda", dtype=torch.int32)], 1)
        w = torch.cat([w, torch.sigmoid(z.float()) * _SHARED_SCALE], 1)
    return ids.contiguous(), w.contiguous(), z


_SHARED_SCALE = 0.5


def _slots_to_rows(case, ids):
    """c_map [T, k']: the expert-order row of each slot, -1 without one; and a_map, offsets."""
    flat = ids.reshape(-1).long()
    n, E, lo, local = flat.numel(), case["E_global"], case["offset"], case["E_local"]
    total = local + case["shared"]
    e = torch.where((flat >= lo) & (flat < lo + local), flat - lo, torch.where(flat >= E, flat - E + local, total))
    by, order = torch.sort(e, stable=True)
    here = by < total
    rows = torch.arange(n, device="cuda")
    c_map = torch.empty(n, device="cuda", dtype=torch.int32)
    c_map[order] = torch.where(here, rows, -1).int()
    a_map = torch.where(here, order, -1).int()
    offsets = torch.searchsorted(by, torch.arange(total + 1, device="cuda")).int()
    return c_map.view_as(ids), a_map, offsets


def _prepare_tokens(case, g, s):
    T, H, dt = case["T"], case["hidden"], _DT[case["dtype"]]
    kp = case["top_k"] + case["shared"]
    s["ids"], s["w"], _ = _pick(case, g)
    c_map, a_map, offsets = _slots_to_rows(case, s["ids"])
    if own:
        import mxfp4_mixture_experts_02_gb300 as moe

        s["shape"] = moe.MoeTokenShape(T=T, E_global=case["E_global"], E_local=case["E_local"],
                                       expert_offset=case["offset"], top_k=case["top_k"], num_shared=case["shared"],
                                       hidden=H)
        s["ws"] = moe.token_map_workspace(s["shape"])
        s["maps"] = moe.MoeTokenMap(a_map, c_map, offsets)
    s["c_map"] = c_map
    if case["op"] == "permute" and case["pass"] == "forward":
        s["x"] = _filled(g, T, H, dt)
        # rows past the last expert's stay as they are: zero here
        s["rows"] = torch.zeros((T * kp, H), device="cuda", dtype=dt)
        s["a_out"] = torch.full((T * kp,), -1, device="cuda", dtype=torch.int32)
        s["c_out"] = torch.empty((T, kp), device="cuda", dtype=torch.int32)
        s["o_out"] = torch.empty(case["E_local"] + case["shared"] + 1, device="cuda", dtype=torch.int32)
        if own:
            s["maps"] = moe.MoeTokenMap(s["a_out"], s["c_out"], s["o_out"])
        return
    s["y"] = _filled(g, T * kp, H, dt)
    s["out"] = torch.empty((T, H), device="cuda", dtype=dt)
    if case["op"] == "unpermute" and case["pass"] == "backward":
        s["dout"] = _filled(g, T, H, dt, 0.1)
        s["dy"] = torch.zeros((T * kp, H), device="cuda", dtype=dt)
        s["dw"] = torch.empty((T, kp), device="cuda")


def _prepare_route(case, g, s):
    T, E, kp = case["T"], case["E_global"], case["top_k"] + case["shared"]
    s["ids"], s["w"], s["z"] = _pick(case, g)
    s["dw"] = _randn(g, T, kp)
    s["dlogits"] = torch.empty((T, E), device="cuda")
    s["dz"] = torch.empty((T, 1), device="cuda") if case["shared"] else None
    if own:
        import mxfp4_mixture_experts_02_gb300 as moe

        s["shape"] = moe.MoeTokenShape(T=T, E_global=E, E_local=E, expert_offset=0, top_k=case["top_k"],
                                       num_shared=case["shared"], hidden=512)


def _parts(case):
    """Sizes of the case's tensors: two thirds of the parameters in a few matrices, the rest spread over three
    orders of magnitude, odd ones among them; each starts at a multiple of 32 in the flat buffers."""
    n, total = case["tensors"], case["params"]
    r = random.Random(n * 1_000_003 + total)
    share = [math.exp(r.uniform(0.0, 7.0)) for _ in range(n)]
    for i in range(0, n, max(1, n // 3)):
        share[i] += 2.0 * sum(share) / 3
    unit = total / sum(share)
    return [max(1, int(v * unit) - r.randrange(0, 3)) for v in share]


def _prepare_adamw(case, g, s):
    sizes = _parts(case)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // 32) * 32
    s["n"] = at

    def flat(scale, dt=torch.float32):
        v = torch.empty(at, device="cuda", dtype=dt).normal_(0.0, scale, generator=g)
        for b, n in zip(starts, sizes):  # nothing between the tensors
            v[b + n:b + -(-n // 32) * 32] = 0
        return v

    s["p"] = flat(0.02)
    s["g"] = flat(1e-3, _DT[case["grad"]])
    m, r = flat(3e-4), flat(1e-3).abs_()
    s["hyper"] = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1, "step": 100}
    s["seed"] = 0x5EED
    s["clip"] = torch.tensor([0.73], device="cuda") if case["clip"] else None
    if case["state"] == "float32":
        s["m"], s["v"] = m, r.square_()
        s["ms"] = s["vs"] = None
    else:
        # 8-bit states: E4M3 codes with a power-of-two scale for 32 values; the second moment as its square root
        half = torch.full((at,), 0x8000, device="cuda", dtype=torch.int32)
        s["m"], s["ms"] = _mx_store(m, half, False)
        s["v"], s["vs"] = _mx_store(r, half, True)
    if own:
        import mxfp4_mixture_experts_02_gb300 as moe

        def cut(t, per=1):
            return None if t is None else [t[b // per:b // per + -(-n // per)] for b, n in zip(starts, sizes)]

        s["handle"] = moe.MoeAdamwTensors(cut(s["p"]), cut(s["g"]), cut(s["m"]), cut(s["v"]), cut(s["ms"], 32),
                                          cut(s["vs"], 32))


# ------------------------------------------------------------------ the pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import mxfp4_mixture_experts_02_gb300 as moe

    op, back = s["case"]["op"], s["case"]["pass"] == "backward"
    if op == "norm" and not back:
        y, h, mean, rstd = moe.moe_layer_norm(s["x"], s["weight"], s["bias"], s["residual"], s["eps"], y=s["y"],
                                              h=s["h"], mean=s["mean"], rstd=s["rstd"])
        return {"y": y, "h": h if s["residual"] is not None else None, "mean": mean, "rstd": rstd}
    if op == "norm":
        dx, dw, db = moe.moe_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], dh=s["dh"],
                                                 dx=s["dx"], dweight=s["dweight"], dbias=s["dbias"], ws=s["ws"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "permute" and not back:
        maps = moe.moe_token_map(s["shape"], s["ids"], ws=s["ws"], maps=s["maps"])
        rows = moe.moe_permute(s["shape"], s["x"], maps, rows=s["rows"])
        return {"rows": rows, "a_map": maps.a_map, "c_map": maps.c_map, "offsets": maps.expert_offsets}
    if op == "permute":
        return {"dx": moe.moe_permute_backward(s["shape"], s["y"], s["maps"], dx=s["out"])}
    if op == "unpermute" and not back:
        return {"out": moe.moe_unpermute(s["shape"], s["y"], s["w"], s["maps"], out=s["out"])}
    if op == "unpermute":
        dy, dw = moe.moe_unpermute_backward(s["shape"], s["dout"], s["y"], s["w"], s["maps"], dy=s["dy"], dw=s["dw"])
        return {"dy": dy, "dw": dw}
    if op == "route":
        dl, dz = moe.moe_route_backward(s["shape"], s["ids"], s["w"], s["dw"], s["z"], _SHARED_SCALE,
                                        dlogits=s["dlogits"], dshared=s["dz"])
        return {"dlogits": dl, "dshared": dz}
    h = s["hyper"]
    moe.moe_adamw(s["handle"], h["step"], h["lr"], (h["beta1"], h["beta2"]), h["eps"], h["weight_decay"],
                  grad_scale=s["clip"], seed=s["seed"])
    return _adamw_state(s)


def _adamw_state(s):
    out = {"p": s["p"]}
    if s["ms"] is None:
        return dict(out, m=s["m"], v=s["v"])
    # each 8-bit value as the number it is, and each block's scale as the power of two it is
    return dict(out, m=s["m"].view(torch.float8_e4m3fn), root_v=s["v"].view(torch.float8_e4m3fn),
                m_scale=_pow2(s["ms"].int() - 127), root_v_scale=_pow2(s["vs"].int() - 127))


def _plain(s):
    case = s["case"]
    op, back = case["op"], case["pass"] == "backward"
    if op == "norm" and not back:
        h = s["x"].float()
        if s["residual"] is not None:
            h = (h + s["residual"].float()).to(s["x"].dtype)  # the stream is stored in its type, and normalised from there
            stored, h = h, h.float()
        mean = h.mean(1)
        d = h - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(1) + s["eps"])
        y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "h": stored if s["residual"] is not None else None, "mean": mean, "rstd": rstd}
    if op == "norm":
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dy"].float()
        wdy = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}
    if op == "permute" and not back:
        c_map, a_map, offsets = _slots_to_rows(case, s["ids"])
        kp = s["ids"].shape[1]
        rows = s["x"][a_map.clamp_min(0).long() // kp]
        return {"rows": torch.where((a_map >= 0)[:, None], rows, 0), "a_map": a_map, "c_map": c_map, "offsets": offsets}
    if op == "permute":
        return {"dx": _rows_of_slots(s).sum(1).to(s["y"].dtype)}
    if op == "unpermute" and not back:
        return {"out": (_rows_of_slots(s) * s["w"][:, :, None]).sum(1).to(s["y"].dtype)}
    if op == "unpermute":
        there = s["c_map"] >= 0
        dout = s["dout"].float()
        dw = torch.where(there, (_rows_of_slots(s) * dout[:, None, :]).sum(2), 0.0)
        n, H = s["y"].shape
        dy = torch.zeros((n + 1, H), device="cuda", dtype=s["y"].dtype)  # the last row takes what has none
        dy[torch.where(there, s["c_map"], n).view(-1).long()] = \
            (dout[:, None, :] * s["w"][:, :, None]).to(dy.dtype).view(n, H)
        return {"dy": dy[:n], "dw": dw}
    if op == "route":
        k = case["top_k"]
        w, dw = s["w"][:, :k], s["dw"][:, :k]
        dl = torch.zeros_like(s["dlogits"])
        dl.scatter_(1, s["ids"][:, :k].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
        dz = None
        if s["z"] is not None:
            a = 1.0 / (1.0 + torch.exp(-s["z"].float()))
            dz = s["dw"][:, k:] * _SHARED_SCALE * a * (1.0 - a)
        return {"dlogits": dl, "dshared": dz}
    return _plain_adamw(s)


def _rows_of_slots(s):
    """[T, k', H] in 32 bits: each slot's row, zero without one."""
    c = s["c_map"]
    return torch.where((c >= 0)[:, :, None], s["y"][c.clamp_min(0).long()].float(), 0.0)


def _plain_adamw(s):
    h = s["hyper"]
    b1, b2 = h["beta1"], h["beta2"]
    g = s["g"].float()
    if s["clip"] is not None:
        g = g * s["clip"]
    if s["ms"] is None:
        m, v = s["m"], s["v"]
    else:
        m, v = _mx_load(s["m"], s["ms"]), _mx_load(s["v"], s["vs"]).square()
    m = m + (g - m) * (1.0 - b1)
    v = v + (g * g - v) * (1.0 - b2)
    root = torch.sqrt(v)
    den = root * (1.0 / math.sqrt(1.0 - b2 ** h["step"])) + h["eps"]
    s["p"].copy_(s["p"] * (1.0 - h["lr"] * h["weight_decay"]) - (m / den) * (h["lr"] / (1.0 - b1 ** h["step"])))
    if s["ms"] is None:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        bits = _random_bits(s["seed"], s["n"])
        for name, scale, value, shift, up in (("m", "ms", m, 0, False), ("v", "vs", root, 16, True)):
            codes, scales = _mx_store(value, (bits >> shift) & 0xFFFF, up)
            s[name].copy_(codes)
            s[scale].copy_(scales)
    return _adamw_state(s)


# ------------------------------------------------------------------ 8-bit states
def _pow2(e):
    """2^e as 32-bit floats, for whole e from -126 to 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _mx_load(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().view(-1, 32)
    return (v * _pow2(scales.int() - 127)[:, None]).view(-1)


def _mx_store(value, rand, up):
    """Blocks of 32: a scale 2^e with the largest magnitude between 128 and 256 times it, and E4M3 codes rounded up or
    down at random (by 16 random bits each), so that small changes are kept on average.  `up`: what is not zero does
    not become zero."""
    block = value.view(-1, 32)
    _, ex = torch.frexp(block.abs().amax(1))
    e = torch.where(block.abs().amax(1) > 0, ex - 8, -126).clamp(-126, 126)
    x = (block * _pow2(-e)[:, None]).view(-1)
    a = x.abs()
    low = 2.0 ** -6  # below it codes are 2^-9 apart: moved up by 2^-6 they are where the steps have that size
    small = a < low
    shifted = torch.where(small, a + low, a)
    kept = (shifted.view(torch.int32) + (rand.int() << 4)) & ~0xFFFFF
    a = kept.view(torch.float32) - torch.where(small, low, 0.0)
    if up:
        a = torch.where(x != 0, a.clamp_min(2.0 ** -9), a)
    codes = torch.copysign(a, x).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _shr(v, n):
    return (v >> n) & ((1 << (64 - n)) - 1)


def _signed(v):
    return v - (1 << 64) if v >= 1 << 63 else v


def _random_bits(seed, n):
    """32 random bits for each of n elements: the SplitMix64 sequence that starts at `seed`, one 64-bit number for
    two elements."""
    i = torch.arange(1, n // 2 + 1, device="cuda", dtype=torch.int64)
    z = i * _signed(0x9E3779B97F4A7C15) + seed
    z = (z ^ _shr(z, 30)) * _signed(0xBF58476D1CE4E5B9)
    z = (z ^ _shr(z, 27)) * _signed(0x94D049BB133111EB)
    z = z ^ _shr(z, 31)
    return torch.stack([z & 0xFFFFFFFF, _shr(z, 32)], 1).view(-1)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    op, back = case["op"], case["pass"] == "backward"
    if op == "norm":
        x = d(s["x"])
        if not back:
            if s["residual"] is not None:
                x = d((x + d(s["residual"])).to(s["x"].dtype))
            n = x.shape[1]
            mean = x.sum(1) / n
            var = (x - mean.unsqueeze(1)).pow(2).sum(1) / n
            rstd = (var + s["eps"]).pow(-0.5)
            y = torch.addcmul(d(s["bias"]), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), d(s["weight"]))
            return {"y": y, "h": x if s["residual"] is not None else None, "mean": mean, "rstd": rstd}
        dy, n = d(s["dy"]), x.shape[1]
        x.sub_(d(s["mean"]).unsqueeze(1)).mul_(d(s["rstd"]).unsqueeze(1))
        dweight, dbias = torch.einsum("rc,rc->c", dy, x), dy.sum(0)
        dy.mul_(d(s["weight"]))
        a, b = dy.sum(1) / n, torch.einsum("rc,rc->r", dy, x) / n
        dx = (dy - a.unsqueeze(1) - x * b.unsqueeze(1)) * d(s["rstd"]).unsqueeze(1)
        if s["dh"] is not None:
            dx += d(s["dh"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op in ("permute", "unpermute"):
        return _exact_tokens(case, s)
    if op == "route":
        k = case["top_k"]
        w, dw = d(s["w"][:, :k]), d(s["dw"][:, :k])
        # the softmax's Jacobian, applied
        jac = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)
        grad = torch.bmm(jac, dw.unsqueeze(2)).squeeze(2)
        dl = torch.zeros((case["T"], case["E_global"]), device="cuda", dtype=torch.float64)
        rows = torch.arange(case["T"], device="cuda").unsqueeze(1)
        dl[rows, s["ids"][:, :k].long()] = grad
        dz = None
        if s["z"] is not None:
            a = torch.sigmoid(d(s["z"]))
            dz = d(s["dw"][:, k:]) * _SHARED_SCALE * (a - a * a)
        return {"dlogits": dl, "dshared": dz}
    return _exact_adamw(case, s)


def _exact_tokens(case, s):
    T, H = case["T"], case["hidden"]
    kp = case["top_k"] + case["shared"]
    if case["op"] == "permute" and case["pass"] == "forward":
        rows = torch.zeros((T * kp, H), device="cuda", dtype=torch.float64)
        for j in range(kp):
            t = torch.nonzero(s["c_map"][:, j] >= 0).squeeze(1)
            rows[s["c_map"][t, j].long()] = s["x"][t].double()
        return {"rows": rows, "a_map": None, "c_map": None, "offsets": None}
    if case["op"] == "unpermute" and case["pass"] == "backward":
        dout = s["dout"].double()
        dy = torch.zeros((T * kp, H), device="cuda", dtype=torch.float64)
        dw = torch.zeros((T, kp), device="cuda", dtype=torch.float64)
        for j in range(kp):
            t = torch.nonzero(s["c_map"][:, j] >= 0).squeeze(1)
            r = s["c_map"][t, j].long()
            dy[r] = dout[t] * s["w"][t, j].double().unsqueeze(1)
            dw[t, j] = torch.einsum("th,th->t", dout[t], s["y"][r].double())
        return {"dy": dy, "dw": dw}
    out = torch.zeros((T, H), device="cuda", dtype=torch.float64)
    for j in range(kp):
        t = torch.nonzero(s["c_map"][:, j] >= 0).squeeze(1)
        v = s["y"][s["c_map"][t, j].long()].double()
        out[t] += v if case["op"] == "permute" else v * s["w"][t, j].double().unsqueeze(1)
    return {"dx" if case["op"] == "permute" else "out": out}


def _exact_adamw(case, s):
    h = s["hyper"]
    g = s["g"].double()
    if s["clip"] is not None:
        g.mul_(s["clip"].double())
    eight = s["ms"] is not None
    m, v = s["m"], s["v"]
    if eight:
        m, v = ((c.view(torch.float8_e4m3fn).double().view(-1, 32) * torch.exp2(e.double() - 127).unsqueeze(1)).view(-1)
                for c, e in ((s["m"], s["ms"]), (s["v"], s["vs"])))
        v = v.pow(2)
    m = torch.lerp(g, m.double(), h["beta1"])
    v = torch.lerp(g.pow(2), v.double(), h["beta2"])
    mhat, vhat = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
    p = s["p"].double()
    p = p - h["lr"] * (h["weight_decay"] * p + mhat / (vhat.sqrt() + h["eps"]))
    if not eight:
        return {"p": p, "m": m, "v": v}
    bits = _random_bits(s["seed"], s["n"])
    out = {"p": p}
    for name, x, u in (("m", m, bits & 0xFFFF), ("root_v", v.sqrt(), bits >> 16)):
        blocks = x.view(-1, 32)
        top = blocks.abs().amax(1)
        e = torch.where(top > 0, torch.floor(torch.log2(top)) - 7, -126).clamp(-126, 126)
        q = blocks / torch.exp2(e).unsqueeze(1)
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
        q = torch.sign(q) * torch.floor(q.abs() / step + u.double().view(-1, 32) / 65536) * step
        if name == "root_v":
            q = torch.where(blocks != 0, q.clamp_min(2.0 ** -9), q)
        out[name], out[name + "_scale"] = q.view(-1), torch.exp2(e)
    return {k: out[k] for k in ("p", "m", "root_v", "m_scale", "root_v_scale")}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, back = case["op"], case["pass"] == "backward"
    if op == "norm":
        n, rows, cols, b = case["rows"] * case["cols"], case["rows"], case["cols"], _BYTES[case["dtype"]]
        wb = b if case["w_dtype"] == "same" else 4
        if not back:  # x (and the residual) in, y (and the sum) out
            return {"bytes": n * b * (4 if case["residual"] else 2) + 2 * cols * wb + 8 * rows, "flops": 8 * n}
        return {"bytes": n * b * (4 if case["residual"] else 3) + cols * (wb + 8) + 8 * rows, "flops": 14 * n}
    if op == "route":
        T, kp = case["T"], case["top_k"] + case["shared"]
        return {"bytes": T * (case["E_global"] * 4 + kp * 12 + case["shared"] * 6), "flops": 5 * T * kp}
    if op == "adamw":
        n = sum(_parts(case))
        states = 16 if case["state"] == "float32" else 4 + 4 / 32
        return {"bytes": n * (8 + _BYTES[case["grad"]] + states), "flops": 14 * n}
    T, H, b = case["T"], case["hidden"], _BYTES[case["dtype"]]
    picked = T * case["top_k"] * case["E_local"] / case["E_global"]  # rows on this rank, on average
    if case["zipf"]:
        share = [1.0 / (e + 1) ** case["zipf"] for e in range(case["E_global"])]
        if case["E_local"] < case["E_global"]:
            part = sum(share[case["offset"]:case["offset"] + case["E_local"]]) / sum(share)
            picked = T * min(case["top_k"] * part, case["E_local"])
    rows = picked + T * case["shared"]
    slots = T * (case["top_k"] + case["shared"])
    if op == "permute" and not back:
        return {"bytes": (T + rows) * H * b + 8 * slots + 4 * rows, "flops": 0}
    if op == "permute":
        return {"bytes": (T + rows) * H * b + 4 * slots, "flops": rows * H}
    if not back:
        return {"bytes": (T + rows) * H * b + 8 * slots, "flops": 2 * rows * H}
    return {"bytes": (T + 2 * rows) * H * b + 12 * slots, "flops": 3 * rows * H}
