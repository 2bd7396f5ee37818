"""The token-mixer operators next to the MoE-FFN step, as workloads that can be timed.

Two operators, each in the forms a server calls:

* ``matvec``: y = W x (+ bias) (+ y) for a matrix held in 4-bit blocks with group scales
  (``moe_q4_matvec``): the projections around the step and the vocabulary head.
* ``prefill`` and ``step``: linear attention with a decay for each head, over whole prompts
  (``moe_linattn_prefill``) and for one token of each sequence (``moe_linattn_step``), on
  the same state: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale * S_t^T q_t.

``own`` false computes them with elementary torch operations; ``own`` true calls this package.
``exact`` gives the definition in 64 bits, written apart from both.
"""

import math

import torch

own = False

F16, BF16, F32 = "f16", "bf16", "f32"
TORCH = {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32}
SIZE = {F16: 2, BF16: 2, F32: 4}
BLOCK_VALUES = {"q4_0": 32, "q4_1": 32, "q4_k": 256}
BLOCK_BYTES = {"q4_0": 18, "q4_1": 20, "q4_k": 144}
CHUNK = 64  # tokens of a chunk in the plain form

# ------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------


def matvec(name, qtype, rows, cols, vecs, x, y, group=0, mins=False, bias=False, add=False, pad=0):
    c = dict(op="matvec", qtype=qtype, rows=rows, cols=cols, vecs=vecs, x=x, y=y, group=group, mins=mins,
             bias=bias, add=add, pad=pad)
    return dict(c, name=name) if name else c


def attn(name, op, lens, heads, qk_heads, dk, dv, type, decay, fresh=False, slots="all", fused=False):
    """``lens``: the sequences' token counts ("2048*3,17,0"); a step has one token each ("1*64").
    ``decay``: "head" (one per head), "token" (one per token and head) or "reset" (per token, with
    some -inf). ``slots``: "all", "pool" (a permutation inside a larger pool) or "holes" (and every
    seventh sequence inactive). ``fused``: q, k and v are views of one buffer."""
    c = dict(op=op, lens=lens, heads=heads, qk_heads=qk_heads, dk=dk, dv=dv, type=type, decay=decay,
             fresh=fresh, slots=slots, fused=fused)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the key projection of one decoded token, Flint's hidden size: the smallest call of a layer
        matvec("matvec_kv_q41_t1", "q4_1", 512, 2048, 1, F32, BF16),
        # the output projection of one token, added into the residual stream; Ling's hidden size, K-quant rows
        matvec("matvec_out_q4k_t1", "q4_k", 2560, 2560, 1, BF16, F32, add=True),
        # the vocabulary head for one token: the largest matrix a decoded token reads
        matvec("matvec_head_q40_t1", "q4_0", 128000, 2048, 1, F32, F32),
        # a fused q/k/v projection for a small batch of sequences
        matvec("matvec_qkv_q41_t8", "q4_1", 8192, 2560, 8, F32, BF16),
        # planes with a scale and an offset per 64 values, ragged row count, odd batch, padded vectors
        matvec("matvec_planes_t5", "planes", 4999, 2112, 5, F16, F16, group=64, mins=True, bias=True, pad=24),
        # one decoded token of one sequence: latency
        attn("step_b1", "step", "1*1", 16, 16, 128, 128, BF16, "head"),
        # a full batch of sequences out of a state pool, shared q/k heads: bandwidth of the states
        attn("step_b96", "step", "1*96", 32, 8, 128, 128, BF16, "token", slots="pool"),
        # small odd heads in f32, some sequences inactive
        attn("step_odd_f32", "step", "1*37", 10, 10, 72, 40, F32, "token", slots="holes"),
        # one long prompt: the sequence axis has to be split to fill the GPU
        attn("prefill_16k", "prefill", "16384", 32, 32, 128, 128, BF16, "head", fresh=True),
        # a packed batch of prompts of every length, document resets inside, q/k/v views of one buffer
        attn("prefill_ragged", "prefill", "2048,0,1,777,64,3001,63,65,1500", 20, 20, 128, 128, F16, "reset",
             slots="pool", fused=True),
        # f32 activations, a second turn that continues from its states
        attn("prefill_f32", "prefill", "1024*2", 16, 4, 64, 128, F32, "token"),
        # a short prompt: latency
        attn("prefill_short", "prefill", "40", 16, 16, 128, 128, BF16, "head", fresh=True),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "step", "prefill", "prefill"])
    if op == "matvec":
        qtype = rng.choice(["q4_0", "q4_1", "q4_k", "planes"])
        group = rng.choice([32, 64, 128]) if qtype == "planes" else 0
        unit = BLOCK_VALUES.get(qtype, group)
        cols = max(unit, log_int(rng, 256, 8192) // unit * unit)
        vecs = rng.choice([1, 1, 1, 2, 3, 4, 6, 8, 13, 16])
        rows = max(1, log_int(rng, 64, 64000) * 2048 // (2048 + cols))
        x = rng.choice([F32, BF16, F16])
        return matvec(None, qtype, rows, cols, vecs, x, rng.choice([F32, BF16, x]), group=group,
                      mins=qtype == "planes" and rng.random() < 0.5, bias=rng.random() < 0.3,
                      add=rng.random() < 0.3, pad=rng.choice([0, 0, 8, 24]))
    qk = rng.choice([1, 2, 4, 5, 8, 16])
    heads = qk * rng.choice([1, 1, 2, 4])
    heads = heads if heads <= 32 else qk
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64), (96, 96), (72, 40), (32, 112)])
    type = rng.choice([BF16, BF16, F16, F32])
    decay = rng.choice(["head", "token", "reset"])
    slots = rng.choice(["all", "pool", "holes"])
    if op == "step":
        return attn(None, op, "1*%d" % log_int(rng, 1, 96), heads, qk, dk, dv, type, decay, slots=slots)
    total = log_int(rng, 24, 16384)
    left, lens = total, []
    for _ in range(rng.randrange(6)):
        n = rng.randrange(0, left // 2 + 1)
        lens.append(n)
        left -= n
    lens.append(left)
    return attn(None, op, ",".join(map(str, lens)), heads, qk, dk, dv, type, decay, fresh=rng.random() < 0.5,
                slots=slots, fused=rng.random() < 0.5)


def lengths(case):
    out = []
    for part in case["lens"].split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * int(times or 1)
    return out


# ------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------


def weights(case, gen):
    """Random weights in the case's form: block scales as 4-bit models have them."""
    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def f16_bytes(t):
        return t.half().contiguous().view(torch.uint8).reshape(*t.shape, 2)

    def nibbles(*shape):
        return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)

    rows, cols = case["rows"], case["cols"]
    if case["qtype"] == "planes":
        groups = cols // case["group"]
        s = (0.005 + 0.015 * rand(rows, groups)).half()
        m = (-0.15 * rand(rows, groups)).half() if case["mins"] else None
        return nibbles(rows, cols // 2), s, m
    n = cols // BLOCK_VALUES[case["qtype"]]
    w = nibbles(rows, n, BLOCK_BYTES[case["qtype"]])
    if case["qtype"] == "q4_k":
        w[..., 0:2] = f16_bytes(1.5e-4 + 5e-4 * rand(rows, n))
        w[..., 2:4] = f16_bytes(5e-4 + 2e-3 * rand(rows, n))
    else:
        w[..., 0:2] = f16_bytes(0.005 + 0.015 * rand(rows, n))
        if case["qtype"] == "q4_1":
            w[..., 2:4] = f16_bytes(-0.1 * rand(rows, n))
    return w.reshape(rows, -1), None, None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = dict(case=case)
    if case["op"] == "matvec":
        s["w"], s["scales"], s["mins"] = weights(case, gen)
        x = randn(case["vecs"], case["cols"] + case["pad"])
        x = x * (1 + 30 * (torch.rand(x.shape[1], generator=gen, device="cuda") < 0.004))  # outlier channels
        s["x"] = x.to(TORCH[case["x"]])[:, :case["cols"]]
        s["bias"] = randn(case["rows"]) if case["bias"] else None
        s["y"] = randn(case["vecs"], case["rows"]).to(TORCH[case["y"]]) if case["add"] else None
        return s

    lens, H, G, dk, dv, t = lengths(case), case["heads"], case["qk_heads"], case["dk"], case["dv"], TORCH[case["type"]]
    n, total = len(lens), sum(lens)
    q, k, v = randn(total, G, dk), randn(total, G, dk), randn(total, H, dv)
    k = k / k.norm(dim=-1, keepdim=True)
    if case["fused"]:
        buf = torch.cat([a.reshape(total, -1) for a in (q, k, v)], 1).to(t)
        s["q"], s["k"], s["v"] = (a.unflatten(1, (-1, d)) for a, d in
                                  zip(buf.split([G * dk, G * dk, H * dv], 1), (dk, dk, dv)))
    else:
        s["q"], s["k"], s["v"] = q.to(t), k.to(t), v.to(t)
    if case["decay"] == "head":  # slopes in a geometric series over the heads
        s["g"] = -torch.exp2(-8 * (1 + torch.arange(H, device="cuda", dtype=torch.float64)) / H).float()
    else:
        s["g"] = -torch.nn.functional.softplus(randn(total, H) - 2)
        if case["decay"] == "reset":
            s["g"][torch.rand(total, generator=gen, device="cuda") < 0.002] = -math.inf
    s["offsets"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    pool = n if case["slots"] == "all" else n + n // 3 + 1
    s["state"] = randn(pool, H, dk, dv) * 0.3
    if case["slots"] == "all":
        s["slots"] = None
    else:
        slots = torch.randperm(pool, generator=gen, device="cuda")[:n].to(torch.int32)
        if case["slots"] == "holes":
            slots[6::7] = -1
        s["slots"] = slots
    s["lens"], s["max_len"] = lens, max(lens)
    return s


# ------------------------------------------------------------------------------------------
# Plain forms
# ------------------------------------------------------------------------------------------


def as_f16(b):
    """The f16 numbers of byte pairs."""
    return b.contiguous().view(torch.float16)[..., 0]


def dequantised(s, real):
    """The weight matrix as `real` numbers: value = scale * nibble + offset."""
    case, w = s["case"], s["w"]
    rows, cols, qtype = case["rows"], case["cols"], case["qtype"]
    if qtype == "q4_k":
        b = w.reshape(rows, -1, 144)
        low, high = b[..., 4:8], b[..., 8:12]  # scales and mins of sub-blocks 0..3
        mix = b[..., 12:16]
        sc = torch.cat([low & 63, (mix & 15) | (low >> 6) << 4], -1).to(real) * as_f16(b[..., 0:2]).to(real)[..., None]
        mn = torch.cat([high & 63, (mix >> 4) | (high >> 6) << 4], -1).to(real) * as_f16(b[..., 2:4]).to(real)[..., None]
        q = b[..., 16:].reshape(rows, -1, 4, 1, 32)
        q = torch.cat([q & 15, q >> 4], -2).reshape(rows, -1, 8, 32).to(real)
        return (q * sc[..., None] - mn[..., None]).reshape(rows, cols)
    if qtype == "planes":
        q, g = w.reshape(rows, -1, 16), case["group"]
        sc = s["scales"].to(real).repeat_interleave(g // 32, 1)
        off = -8 * sc if s["mins"] is None else s["mins"].to(real).repeat_interleave(g // 32, 1)
    else:
        b = w.reshape(rows, -1, BLOCK_BYTES[qtype])
        sc = as_f16(b[..., 0:2]).to(real)
        off = -8 * sc if qtype == "q4_0" else as_f16(b[..., 2:4]).to(real)
        q = b[..., -16:]
    q = torch.cat([q & 15, q >> 4], -1).to(real)
    return (q * sc[..., None] + off[..., None]).reshape(rows, cols)


def plain_matvec(s):
    y = s["x"].float() @ dequantised(s, torch.float32).T
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["y"] is None:
        return y.to(TORCH[s["case"]["y"]])
    s["y"].copy_((s["y"].float() + y).to(s["y"].dtype))
    return s["y"]


def active(s):
    """The sequences that have a state, and its place in the pool."""
    n = len(s["lens"])
    slots = torch.arange(n, device="cuda") if s["slots"] is None else s["slots"].long()
    return slots >= 0, slots.clamp(min=0)


def padded(s):
    """q, k, v [n][H][C][chunk][d] in f32, g (f64) and whether a place holds a token, the tokens
    padded to whole chunks."""
    case, n = s["case"], len(s["lens"])
    chunks = max(1, -(-s["max_len"] // CHUNK))
    at = s["offsets"][:-1, None].long() + torch.arange(chunks * CHUNK, device="cuda")
    real = at < s["offsets"][1:, None]
    at = torch.where(real, at, 0)

    def take(a):  # [tokens][heads][d] -> [n][heads][chunks][CHUNK][d]
        a = a.float()[at] * real[..., None, None]
        return a.reshape(n, chunks, CHUNK, a.shape[2], -1).permute(0, 3, 1, 2, 4)

    rep = case["heads"] // case["qk_heads"]
    q, k = (take(s[name]).repeat_interleave(rep, 1) for name in "qk")
    g = s["g"].double()
    g = g.expand(at.shape + g.shape) if g.dim() == 1 else g[at]
    g = (g * real[..., None]).nan_to_num(nan=0.0).clamp(min=-1e5)  # exp(-1e5) is 0: a reset
    return q, k, take(s["v"]), g.reshape(n, chunks, CHUNK, -1).permute(0, 3, 1, 2), at, real


def plain_attn(s):
    """Chunks of tokens: within a chunk as masked products, between chunks through states that
    are summed with their decays by one more product."""
    case, t = s["case"], TORCH[s["case"]["type"]]
    scale = case["dk"] ** -0.5
    act, slots = active(s)
    total = sum(s["lens"])
    o = torch.zeros(total, case["heads"], case["dv"], device="cuda")
    if total == 0:
        if case["fresh"]:
            s["state"][slots[act]] = 0
        return {"o": o.to(t), "state": s["state"]}
    q, k, v, g, at, real = padded(s)
    G = g.cumsum(-1)                                        # [n][H][C][chunk]
    end = G[..., -1]
    tri = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    D = torch.where(tri, (G[..., :, None] - G[..., None, :]).clamp(max=0), -math.inf).exp().float()
    inner = ((q @ k.transpose(-1, -2)) * D) @ v
    local = (k * (end[..., None] - G).exp().float()[..., None]).transpose(-1, -2) @ v  # [n][H][C][dk][dv]
    first = torch.zeros_like(s["state"][slots]) if case["fresh"] else s["state"][slots]
    states = torch.cat([first[:, :, None], local], 2)       # what each chunk, and the start, adds
    E = torch.cat([torch.zeros_like(end[..., :1]), end.cumsum(-1)], -1)
    C = E.shape[-1]
    ctri = torch.ones(C, C, device="cuda", dtype=torch.bool).tril()
    W = torch.where(ctri, (E[..., :, None] - E[..., None, :]).clamp(max=0), -math.inf).exp().float()
    states = (W @ states.flatten(3)).unflatten(3, states.shape[3:])
    outer = (q @ states[:, :, :-1]) * G.exp().float()[..., None]
    out = ((inner + outer) * scale).permute(0, 2, 3, 1, 4).flatten(1, 2)  # [n][places][H][dv]
    keep = real & act[:, None]
    o[at[keep]] = out[keep]
    s["state"][slots[act]] = states[:, :, -1][act]
    return {"o": o.to(t), "state": s["state"]}


def plain_step(s):
    case, t = s["case"], TORCH[s["case"]["type"]]
    act, slots = active(s)
    rep = case["heads"] // case["qk_heads"]
    q, k = (s[name].float().repeat_interleave(rep, 1) for name in "qk")
    new = s["state"][slots] * s["g"].exp()[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
    o = (q[..., None] * new).sum(-2) * case["dk"] ** -0.5 * act[:, None, None]
    s["state"][slots[act]] = new[act]
    return {"o": o.to(t), "state": s["state"]}


# ------------------------------------------------------------------------------------------
# This package's operators
# ------------------------------------------------------------------------------------------


def own_matvec(s):
    import expert_ffn_decode_gb300 as ffn
    case, x = s["case"], s["x"]
    if "cfg" not in s:
        types = {F32: ffn.MOE_F32, F16: ffn.MOE_F16, BF16: ffn.MOE_BF16}
        qtype = {"q4_0": ffn.MOE_Q4_0, "q4_1": ffn.MOE_Q4_1, "q4_k": ffn.MOE_Q4_K, "planes": ffn.MOE_Q4_PLANES}
        s["cfg"] = ffn.make_matvec_cfg(case["rows"], case["cols"], case["vecs"], qtype=qtype[case["qtype"]],
                                       group=case["group"], x_type=types[case["x"]], y_type=types[case["y"]],
                                       x_stride=x.stride(0), flags=ffn.MOE_ACCUMULATE if case["add"] else 0)
    y = s["y"]
    if y is None:
        y = torch.empty(case["vecs"], case["rows"], dtype=TORCH[case["y"]], device="cuda")
    ffn.check(ffn.moe_q4_matvec(x, s["w"], s["scales"], s["mins"], s["bias"], s["cfg"], y,
                                torch.cuda.current_stream()))
    return y


def own_cfg(s):
    import expert_ffn_decode_gb300 as ffn
    case = s["case"]
    types = {F32: ffn.MOE_F32, F16: ffn.MOE_F16, BF16: ffn.MOE_BF16}
    flags = (ffn.MOE_FRESH_STATE if case["fresh"] else 0) | (0 if case["decay"] == "head" else ffn.MOE_TOKEN_DECAY)
    return ffn.make_linattn_cfg(len(s["lens"]), sum(s["lens"]), case["heads"], case["dk"], case["dv"],
                                n_qk_heads=case["qk_heads"], n_states=s["state"].shape[0], type=types[case["type"]],
                                scale=case["dk"] ** -0.5, flags=flags, q_stride=s["q"].stride(0),
                                k_stride=s["k"].stride(0), v_stride=s["v"].stride(0))


def own_attn(s):
    import expert_ffn_decode_gb300 as ffn
    if "cfg" not in s:
        s["cfg"] = own_cfg(s)
        s["ws"] = torch.zeros(ffn.moe_linattn_workspace_size(s["cfg"]), dtype=torch.uint8, device="cuda")
    o = torch.empty(s["v"].shape, dtype=s["v"].dtype, device="cuda")
    ffn.check(ffn.moe_linattn_prefill(s["q"], s["k"], s["v"], s["g"], s["offsets"], s["slots"], s["cfg"], s["state"],
                                      o, s["ws"], s["ws"].numel(), torch.cuda.current_stream()))
    return {"o": o, "state": s["state"]}


def own_step(s):
    import expert_ffn_decode_gb300 as ffn
    if "cfg" not in s:
        s["cfg"] = own_cfg(s)
    o = torch.empty(s["v"].shape, dtype=s["v"].dtype, device="cuda")
    ffn.check(ffn.moe_linattn_step(s["q"], s["k"], s["v"], s["g"], s["slots"], s["cfg"], s["state"], o,
                                   torch.cuda.current_stream()))
    return {"o": o, "state": s["state"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"matvec": own_matvec, "prefill": own_attn, "step": own_step}[op](state)
    return {"matvec": plain_matvec, "prefill": plain_attn, "step": plain_step}[op](state)


# ------------------------------------------------------------------------------------------
# Work and definition
# ------------------------------------------------------------------------------------------


def work(case):
    if case["op"] == "matvec":
        rows, cols, vecs = case["rows"], case["cols"], case["vecs"]
        if case["qtype"] == "planes":
            b = rows * cols // 2 + rows * cols // case["group"] * (4 if case["mins"] else 2)
        else:
            b = rows * cols // BLOCK_VALUES[case["qtype"]] * BLOCK_BYTES[case["qtype"]]
        b += vecs * cols * SIZE[case["x"]] + vecs * rows * SIZE[case["y"]] * (2 if case["add"] else 1)
        return {"bytes": b + (4 * rows if case["bias"] else 0), "flops": 2 * rows * cols * vecs}
    lens = lengths(case)
    H, G, dk, dv = case["heads"], case["qk_heads"], case["dk"], case["dv"]
    alive = [n for i, n in enumerate(lens) if not (case["slots"] == "holes" and i % 7 == 6)]
    tokens, states = sum(alive), sum(n > 0 or case["fresh"] for n in alive)
    b = tokens * (2 * G * dk + H * dv) * SIZE[case["type"]] + sum(lens) * H * dv * SIZE[case["type"]]
    b += 4 * (H if case["decay"] == "head" else tokens * H)
    b += states * H * dk * dv * 4 * (1 if case["fresh"] else 2)
    return {"bytes": b, "flops": 4 * tokens * H * dk * dv}


def exact(case, seed):
    """The definitions, in 64 bits: every weight from its own nibble, every token in its turn."""
    s = prepare(case, seed)
    if case["op"] == "matvec":
        i = torch.arange(case["cols"], device="cuda")
        qtype, x = case["qtype"], s["x"].double()
        out = torch.zeros(case["vecs"], case["rows"], dtype=torch.float64, device="cuda")
        for lo in range(0, case["rows"], 8192):  # rows in parts, for memory
            w = s["w"][lo:lo + 8192].long()

            def half(pos):  # the f16 number whose bytes start at each place
                bits = w[:, pos] | w[:, pos + 1] << 8
                e, f = bits >> 10 & 31, (bits & 1023).double()
                v = torch.where(e == 0, f * 2.0 ** -24, (1 + f / 1024) * torch.exp2(e.double() - 15))
                return torch.where(bits >> 15 == 1, -v, v)

            if qtype == "q4_k":
                base, j = i // 256 * 144, i % 256 // 32
                byte = w[:, base + 16 + j // 2 * 32 + i % 32]
                at = base + 4
                sc = torch.where(j < 4, w[:, at + j % 4] & 63, w[:, at + 8 + j % 4] & 15 | w[:, at + j % 4] >> 6 << 4)
                mn = torch.where(j < 4, w[:, at + 4 + j % 4] & 63,
                                 w[:, at + 8 + j % 4] >> 4 | w[:, at + 4 + j % 4] >> 6 << 4)
                W = half(base) * sc * (byte >> 4 * (j % 2) & 15) - half(base + 2) * mn
            elif qtype == "planes":
                nib = w[:, i // 32 * 16 + i % 16] >> i % 32 // 16 * 4 & 15
                sc = s["scales"][lo:lo + 8192].double()[:, i // case["group"]]
                W = sc * (nib - 8) if s["mins"] is None else sc * nib + s["mins"][lo:lo + 8192].double()[:, i // case["group"]]
            else:
                size = BLOCK_BYTES[qtype]
                base = i // 32 * size
                nib = w[:, base + size - 16 + i % 16] >> i % 32 // 16 * 4 & 15
                W = half(base) * (nib - 8) if qtype == "q4_0" else half(base) * nib + half(base + 2)
            out[:, lo:lo + 8192] = x @ W.T
        if s["bias"] is not None:
            out = out + s["bias"].double()
        return out if s["y"] is None else out + s["y"].double()
    lens, H, rep = s["lens"], case["heads"], case["heads"] // case["qk_heads"]
    q, k = (s[name].double().repeat_interleave(rep, 1) for name in "qk")
    v, g, pool = s["v"].double(), s["g"].double(), s["state"].double()
    o = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    slots = list(range(len(lens))) if s["slots"] is None else s["slots"].tolist()
    begin = s["offsets"].tolist()
    alive = [b for b in range(len(lens)) if slots[b] >= 0]
    if case["op"] == "step":
        begin = list(range(len(lens)))
    S = {b: torch.zeros_like(pool[0]) if case["fresh"] else pool[slots[b]].clone() for b in alive}
    if case["op"] == "step":
        at = torch.tensor(alive, device="cuda")
        lam = (g if case["decay"] == "head" else g[at]).exp()
        new = torch.stack([S[b] for b in alive]) * lam[..., None, None] + k[at][..., None] * v[at][..., None, :]
        o[at] = torch.einsum("bhd,bhde->bhe", q[at], new) * case["dk"] ** -0.5
        pool[[slots[b] for b in alive]] = new
        return {"o": o, "state": pool}
    # all sequences advance together, longest first, so the ones still running are a prefix
    alive.sort(key=lambda b: -lens[b])
    run_state = torch.stack([S[b] for b in alive])
    start = torch.tensor([begin[b] for b in alive], device="cuda")
    lam_head = g.exp() if case["decay"] == "head" else None
    for t in range(max((lens[b] for b in alive), default=0)):
        m = sum(lens[b] > t for b in alive)
        at = start[:m] + t
        lam = lam_head if lam_head is not None else g[at].exp()
        now = run_state[:m]
        now.mul_(lam[..., None, None]).addcmul_(k[at][..., None], v[at][..., None, :])
        o[at] = (q[at][..., None, :] @ now)[..., 0, :]
    pool[[slots[b] for b in alive]] = run_state
    return {"o": o * case["dk"] ** -0.5, "state": pool}
