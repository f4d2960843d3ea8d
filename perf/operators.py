"""Measured cases of the packed-sequence operators: ``qk_norm_rope`` and packed attention.

Two operators that run one after the other in an attention layer on packed sequences:

* ``rope``: every query and key vector normalized over the head dimension, multiplied by a
  gain and rotated by its token's position (one axis, or several for images and video);
  mode ``fwd`` returns the rotated q and k, mode ``train`` also the gradients of q, k and of
  both gains;
* ``attn``: softmax attention over sequences of different lengths laid end to end, with
  grouped heads; mode ``fwd`` returns the output and the log-sum-exp of the scores, mode
  ``train`` the output and the gradients of q, k and v.

``run`` computes them in elementary torch operations, or with the framework's calls where
``own`` is true; ``exact`` computes the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_BASE = 10000.0
_EPS = 1e-6


def _ints(text):
    return [int(x) for x in text.split(",")]


# ---- cases -----------------------------------------------------------------------------------
def _rope(mode, tokens, hq, hkv, d, dtype="bf16", rotary=None, sections="", interleaved=False,
          far=0, fused=True):
    return {"op": "rope", "mode": mode, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "rotary": d if rotary is None else rotary, "sections": sections,
            "interleaved": interleaved, "far": far, "fused": fused}


def _attn(mode, lengths, hq, hkv, d, dtype="bf16", causal=True, fused=True):
    return {"op": "attn", "mode": mode, "lengths": ",".join(str(n) for n in lengths), "hq": hq,
            "hkv": hkv, "d": d, "dtype": dtype, "causal": causal, "fused": fused}


# document lengths of one packed training row of 16384 tokens: a few long ones, many short
_DOCS = [5021, 3407, 2290, 1777, 1311, 866, 590, 431, 288, 170, 111, 64, 37, 12, 7, 2]


def listed():
    return [
        # one new token of one sequence: launch and latency only
        {"name": "rope_token", **_rope("fwd", 1, 16, 16, 64)},
        # the 325M Llama layer's step: 8 sequences of 2048 tokens, 16 heads of 64
        {"name": "rope_llama325m", **_rope("train", 16384, 16, 16, 64)},
        # video tokens (time, height, width): 13 frames of 45 x 61 patches, half precision
        {"name": "rope_video", **_rope("train", 35685, 12, 12, 128, "fp16", sections="16,24,24",
                                       fused=False)},
        # a prompt far into a long context, part of each head rotated, neighbouring pairs
        {"name": "rope_far", **_rope("fwd", 12345, 32, 8, 128, rotary=64, interleaved=True,
                                     far=1 << 20)},
        # the 262144-token training step of the tokens-per-step sweep, grouped heads
        {"name": "rope_sweep", **_rope("train", 262144, 16, 4, 128)},
        # a few short prompts, one of a single token: latency
        {"name": "attn_short", **_attn("fwd", [1, 37, 90], 16, 16, 64)},
        # the 325M Llama layer's training step
        {"name": "attn_llama325m", **_attn("train", [2048] * 8, 16, 16, 64)},
        # packed documents of very different lengths, grouped heads, training
        {"name": "attn_docs", **_attn("train", _DOCS, 16, 4, 128)},
        # images of different sizes seen whole (no causal mask), half precision, odd group
        {"name": "attn_images", **_attn("train", [1369, 1024, 777, 777, 576, 333, 196, 49], 15, 5,
                                        64, "fp16", causal=False)},
        # a batch of prompts before decoding, grouped heads
        {"name": "attn_prompts", **_attn("fwd", [4099, 2048, 1500, 731, 517, 128, 33, 8], 32, 8,
                                         128, "fp16", fused=False)},
        # the sweep's longest sequences, one per head, training
        {"name": "attn_sweep8192", **_attn("train", [8192] * 4, 16, 16, 128)},
        # one long prompt
        {"name": "attn_long16k", **_attn("fwd", [16384], 32, 8, 128)},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    mode = rng.choice(["fwd", "train"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * hkv <= 32])
    fused = rng.random() < 0.6
    if rng.random() < 0.4:
        tokens = _spread(rng, 1, 262144 * 20 * 128 // ((hq + hkv) * d))
        sections = ""
        rotary = rng.choice([d, d, d // 2])
        if rng.random() < 0.4:
            a = rng.randrange(1, rotary // 4)
            b = rng.randrange(1, rotary // 4)
            sections = "%d,%d,%d" % (a, b, rotary // 2 - a - b)
        return _rope(mode, tokens, hq, hkv, d, dtype, rotary, sections, rng.random() < 0.3,
                     rng.choice([0, 0, 1 << 15, 1 << 20]), fused)
    causal = rng.random() < 0.75
    longest = 8192 if hq <= 16 else 5000
    # a row that sees one key has no gradient but rounding: training draws hold longer ones too
    least = 1 if mode == "fwd" else 32
    total = _spread(rng, least, 24000)
    lengths = []
    while total > 0 and len(lengths) < 24:
        n = min(total, _spread(rng, 1 if lengths else least, longest))
        lengths.append(n)
        total -= n
    return _attn(mode, lengths, hq, hkv, d, dtype, causal, fused)


# ---- inputs ----------------------------------------------------------------------------------
def _heads(case, tokens, g, extra):
    """q, k and, with ``extra``, v: slices of one projection's rows, or tensors of their own."""
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], _DT[case["dtype"]]
    n = hq + hkv * (2 if extra else 1)
    if case["fused"]:
        x = torch.randn((tokens, hq + 2 * hkv, d), generator=g, device="cuda").to(dt)
        parts = [x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]]
        return parts if extra else parts[:2]
    x = torch.randn((n, tokens, d), generator=g, device="cuda").to(dt).transpose(0, 1)
    parts = [x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]]
    return [p.contiguous() for p in (parts if extra else parts[:2])]


def _buckets(lengths, hq, device):
    """Tokens of sequences of like length, padded to the longest of their group: [(index,
    present)], each [sequences, length], small enough for one batch of score matrices."""
    starts, at = [], 0
    for n in lengths:
        starts.append(at)
        at += n
    order = sorted(range(len(lengths)), key=lambda i: -lengths[i])
    out, i = [], 0
    while i < len(order):
        top = lengths[order[i]]
        most = max(1, (1 << 30) // (top * top * hq))
        group = [j for j in order[i:i + most] if lengths[j] * 3 >= top * 2 or top <= 128]
        i += len(group)
        index = torch.tensor([starts[j] for j in group])[:, None] + torch.arange(top)
        present = torch.arange(top) < torch.tensor([lengths[j] for j in group])[:, None]
        index = torch.where(present, index, torch.tensor([starts[j] for j in group])[:, None])
        out.append((index.to(device), present.to(device)))
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    d, dt = case["d"], _DT[case["dtype"]]
    state = {"case": case}
    if case["op"] == "rope":
        T = case["tokens"]
        state["q"], state["k"] = _heads(case, T, g, False)
        state["gq"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        state["gk"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        if case["sections"]:
            # time, height and width of the tokens of a grid 45 high and 61 wide
            t = torch.arange(T, device="cuda")
            pos = torch.stack([t // (45 * 61), t // 61 % 45, t % 61])
        else:
            pos = torch.arange(T, device="cuda") % 8192
        state["pos"] = (pos + case["far"]).to(torch.int32)
        if case["mode"] == "train":
            state["dq"] = torch.randn((T, case["hq"], d), generator=g, device="cuda").to(dt)
            state["dk"] = torch.randn((T, case["hkv"], d), generator=g, device="cuda").to(dt)
        half = case["rotary"] // 2
        state["freq"] = _BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        if own:
            from fwd_bwd_b200 import rope
            state["rope"] = rope.Rope(d, base=_BASE, rotary_dim=case["rotary"],
                                      sections=_ints(case["sections"]) if case["sections"] else None,
                                      interleaved=case["interleaved"], eps=_EPS)
        return state
    lengths = _ints(case["lengths"])
    T = sum(lengths)
    state["q"], state["k"], state["v"] = _heads(case, T, g, True)
    if case["mode"] == "train":
        state["do"] = (torch.randn((T, case["hq"], d), generator=g, device="cuda") * 1e-2).to(dt)
    state["buckets"] = _buckets(lengths, case["hq"], "cuda")
    if own:
        from fwd_bwd_b200 import packed
        state["batch"] = packed.Batch(lengths, device="cuda")
    return state


# ---- the operators ---------------------------------------------------------------------------
def _own_rope(s):
    from fwd_bwd_b200 import rope
    q, k = rope.qk_norm_rope_fwd(s["q"], s["k"], s["pos"], s["rope"], s["gq"], s["gk"])
    if s["case"]["mode"] == "fwd":
        return {"q": q, "k": k}
    dq, dk, dgq, dgk = rope.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["pos"], s["rope"],
                                             s["gq"], s["gk"])
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dgq": dgq, "dgk": dgk}


def _own_attn(s):
    from fwd_bwd_b200 import packed
    causal = s["case"]["causal"]
    o, lse = packed.attn_fwd(s["q"], s["k"], s["v"], s["batch"], causal=causal)
    if s["case"]["mode"] == "fwd":
        return {"o": o, "lse": lse}
    dq, dk, dv = packed.attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], s["batch"],
                                 causal=causal)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv}


def _turn(x, cos, sin, rotary, interleaved):
    """The first ``rotary`` channels of x [T, H, d] turned by the angles [T, rotary / 2]."""
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rotary // 2], x[..., rotary // 2:rotary]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return y if rotary == x.shape[-1] else torch.cat([y, x[..., rotary:]], -1)


def _angles(s):
    """cos and sin [T, rotary / 2] of position times frequency, the angle in 64 bits."""
    pos, freq, case = s["pos"], s["freq"], s["case"]
    if case["sections"]:
        axis = torch.repeat_interleave(torch.arange(pos.shape[0], device=pos.device),
                                       torch.tensor(_ints(case["sections"]), device=pos.device))
        angle = pos[axis].t().double() * freq
    else:
        angle = pos[:, None].double() * freq
    return angle.cos().float(), angle.sin().float()


def _plain_rope_one(x, gain, grad, cos, sin, case):
    rotary, inter, dt = case["rotary"], case["interleaved"], x.dtype
    x = x.float()
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    xh = x * inv
    y = _turn(xh * gain, cos, sin, rotary, inter).to(dt)
    if grad is None:
        return y, None, None
    gy = _turn(grad.float(), cos, -sin, rotary, inter)
    dgain = (gy * xh).sum((0, 1), dtype=torch.float64).float()
    gx = gy * gain
    dx = (gx - xh * (gx * xh).mean(-1, keepdim=True)) * inv
    return y, dx.to(dt), dgain


def _plain_rope(s):
    case = s["case"]
    cos, sin = _angles(s)
    q, dq, dgq = _plain_rope_one(s["q"], s["gq"], s.get("dq"), cos, sin, case)
    k, dk, dgk = _plain_rope_one(s["k"], s["gk"], s.get("dk"), cos, sin, case)
    if case["mode"] == "fwd":
        return {"q": q, "k": k}
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dgq": dgq, "dgk": dgk}


def _plain_attn(s):
    case, q, k, v = s["case"], s["q"], s["k"], s["v"]
    train, hkv, group = case["mode"] == "train", case["hkv"], case["hq"] // case["hkv"]
    tau = 1.0 / math.sqrt(case["d"])
    T, hq, d = q.shape
    o = q.new_empty((T, hq, d))
    lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    dq, dk, dv = q.new_empty((T, hq, d)), k.new_empty((T, hkv, d)), k.new_empty((T, hkv, d))
    for index, present in s["buckets"]:
        n, L = index.shape
        # heads in pieces, so that no score matrix passes 2^30 values
        step = max(1, min(hkv, (1 << 30) // (n * group * L * L)))
        seen = present[:, None, None, None, :].expand(n, 1, 1, L, L)
        if case["causal"]:
            at = torch.arange(L, device=q.device)
            seen = seen & (at[None, :] <= at[:, None])
        rows = index[present]
        for h in range(0, hkv, step):
            kv, qh = slice(h, min(hkv, h + step)), slice(h * group, min(hkv, h + step) * group)

            def split(x, heads):  # [n, kv heads, heads of one kv head, L, d]
                x = x[:, heads][index].float().unflatten(2, (kv.stop - kv.start, -1))
                return x.permute(0, 2, 3, 1, 4)

            def join(x, out, heads):
                out[rows, heads] = x.permute(0, 3, 1, 2, 4).flatten(2, 3)[present].to(out.dtype)

            qs, ks, vs = split(q, qh), split(k, kv), split(v, kv)
            z = (qs @ ks.mT).mul_(tau).masked_fill_(~seen, -math.inf)
            top = z.amax(-1, keepdim=True)
            p = z.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            p /= total
            os = p @ vs
            join(os, o, qh)
            if not train:
                lse[qh, rows] = (top + total.log()).permute(1, 2, 0, 3, 4)[..., 0].flatten(0, 1)[
                    :, present]
                continue
            dos = split(s["do"], qh)
            dos = dos * present[:, None, None, :, None]
            join((p.mT @ dos).sum(2, keepdim=True), dv, kv)
            ds = (dos @ vs.mT).sub_((dos * os).sum(-1, keepdim=True)).mul_(p).mul_(tau)
            join(ds @ ks, dq, qh)
            join((ds.mT @ qs).sum(2, keepdim=True), dk, kv)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv} if train else {"o": o, "lse": lse}


def run(state):
    if state["case"]["op"] == "rope":
        return _own_rope(state) if own else _plain_rope(state)
    return _own_attn(state) if own else _plain_attn(state)


# ---- what the operators cannot do without ----------------------------------------------------
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    train = case["mode"] == "train"
    if case["op"] == "rope":
        rows = case["tokens"] * (hq + hkv)
        pos = 4 * case["tokens"] * max(1, len(case["sections"].split(",")))
        # q, k in and out; then also their gradients in and out (q and k are read once)
        return {"bytes": rows * d * 2 * (4 if train else 2) + pos + 8 * d * (2 if train else 1),
                "flops": rows * d * (18 if train else 8)}
    lengths = _ints(case["lengths"])
    T = sum(lengths)
    # scores a row sees: all, or those up to its own position
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lengths)
    matrix = 2 * pairs * d * hq
    if train:  # q, dq, do, o; k, v, dk, dv
        return {"bytes": T * d * 2 * (4 * hq + 4 * hkv), "flops": 7 * matrix}
    return {"bytes": T * d * 2 * (2 * hq + 2 * hkv) + 4 * T * hq, "flops": 2 * matrix}


# ---- the same from the definitions, in 64 bits -----------------------------------------------
def _exact_rope_one(x, gain, grad, unit, case):
    """Rotation as multiplication by a complex unit; the norm's gradient as the projection of
    the incoming one off the vector itself."""
    rotary, d = case["rotary"], x.shape[-1]
    if case["interleaved"]:
        re, im = torch.arange(0, rotary, 2), torch.arange(1, rotary, 2)
    else:
        re, im = torch.arange(rotary // 2), torch.arange(rotary // 2, rotary)

    def turned(y, u):
        y = y.clone()
        z = torch.complex(y[..., re], y[..., im]) * u[:, None]
        y[..., re], y[..., im] = z.real, z.imag
        return y

    outs, grads, dgain = [], [], torch.zeros(d, dtype=torch.float64, device=x.device)
    for t in range(0, x.shape[0], 16384):
        part = x[t:t + 16384].double()
        length = (part.pow(2).sum(-1, keepdim=True) / d + _EPS).sqrt()
        outs.append(turned(part / length * gain.double(), unit[t:t + 16384]).float())
        if grad is not None:
            back = turned(grad[t:t + 16384].double(), unit[t:t + 16384].conj())
            dgain += (back * part / length).sum((0, 1))
            back = back * gain.double()
            along = (back * part).sum(-1, keepdim=True) / (d * length.pow(2))
            grads.append(((back - part * along) / length).float())
    return torch.cat(outs), (torch.cat(grads) if grads else None), dgain


def _exact_rope(s, case):
    pos, half = s["pos"].double(), case["rotary"] // 2
    freq = torch.exp(torch.arange(half, dtype=torch.float64, device="cuda") * (-math.log(_BASE) / half))
    if case["sections"]:
        parts, at = [], 0
        for axis, n in enumerate(_ints(case["sections"])):
            parts.append(torch.outer(pos[axis], freq[at:at + n]))
            at += n
        angle = torch.cat(parts, 1)
    else:
        angle = torch.outer(pos, freq)
    unit = torch.polar(torch.ones_like(angle), angle)
    q, dq, dgq = _exact_rope_one(s["q"], s["gq"], s.get("dq"), unit, case)
    k, dk, dgk = _exact_rope_one(s["k"], s["gk"], s.get("dk"), unit, case)
    if case["mode"] == "fwd":
        return {"q": q, "k": k}
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dgq": dgq, "dgk": dgk}


def _exact_attn(s, case):
    q, k, v = s["q"], s["k"], s["v"]
    T, hq, d = q.shape
    train, group = case["mode"] == "train", hq // case["hkv"]
    o = torch.zeros((T, hq, d), device=q.device)
    lse = torch.zeros((hq, T), dtype=torch.float64, device=q.device)
    dq = torch.zeros_like(o)
    dk, dv = (torch.zeros(k.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    at = 0
    for n in _ints(case["lengths"]):
        rows = slice(at, at + n)
        at += n
        for h in range(hq):
            kh, vh = k[rows, h // group].double(), v[rows, h // group].double()
            for i in range(0, n, 2048):  # queries i .. j-1
                j = min(n, i + 2048)
                end = j if case["causal"] else n
                qh = q[rows][i:j, h].double()
                z = torch.einsum("id,jd->ij", qh, kh[:end]) / math.sqrt(d)
                if case["causal"]:
                    z += torch.full_like(z, -math.inf).triu(i + 1)
                log = torch.logsumexp(z, 1, keepdim=True)
                p = torch.exp(z - log)
                oh = p @ vh[:end]
                o[rows][i:j, h] = oh.float()
                lse[h, rows][i:j] = log[:, 0]
                if train:
                    g = s["do"][rows][i:j, h].double()
                    dv[rows][:end, h // group] += p.T @ g
                    dz = p * (g @ vh[:end].T - (g * oh).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[rows][i:j, h] = (dz @ kh[:end]).float()
                    dk[rows][:end, h // group] += dz.T @ qh
    if train:
        return {"o": o, "dq": dq, "dk": dk.float(), "dv": dv.float()}
    return {"o": o, "lse": lse}


def exact(case, seed):
    w = work(case)
    # 64-bit products run at some 30 TFLOP/s and the masked half is computed too
    if w["flops"] > 2e14:
        return None
    s = prepare(case, seed)
    return _exact_rope(s, case) if case["op"] == "rope" else _exact_attn(s, case)
