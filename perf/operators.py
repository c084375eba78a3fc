"""Cases that measure the gated delta rule with one decay per head (chunked forward and
backward, recurrent) and the backward passes of the prologue and of the output epilogue.

With ``own`` false, ``run`` computes an operator in its plain form, elementary torch
operations in fp32; with ``own`` true it calls the library.  Sequences are packed:
``lens`` lists their lengths, ``HK`` key heads serve ``HV`` value heads (value head h
reads key head h // (HV / HK)), ``D`` is the head dimension of keys and values.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
C = 64
F64 = torch.float64


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # Prefill of one prompt with a carried state, as many key heads as value heads.
        {"name": "chunk one prompt", "op": "chunk", "lens": "4096", "HK": 8, "HV": 8, "D": 128,
         "dt": "bf16", "state": True},
        # A serving batch of packed prompts, two value heads to a key head.
        {"name": "chunk packed prompts", "op": "chunk",
         "lens": "8192,512,16384,3333,1024,6001,12288,2047,9000,777", "HK": 16, "HV": 32,
         "D": 128, "dt": "bf16", "state": True},
        # The shortest prompts: one not a whole chunk, one a single token, one empty.
        {"name": "chunk short prompts", "op": "chunk", "lens": "37,1,0,90", "HK": 2, "HV": 4,
         "D": 64, "dt": "f16", "state": True},
        # A training step's backward over whole sequences.
        {"name": "chunk backward", "op": "chunk_bwd", "lens": "2048,2048,2048,2048", "HK": 16,
         "HV": 16, "D": 128, "dt": "bf16", "state": False},
        # The same over ragged sequences with carried states and shared key heads.
        {"name": "chunk backward ragged", "op": "chunk_bwd", "lens": "200,0,1,64,63,1030,517",
         "HK": 4, "HV": 8, "D": 128, "dt": "f16", "state": True},
        # One new token for every sequence of a large batch.
        {"name": "decode large batch", "op": "recurrent", "lens": ",".join(["1"] * 256),
         "HK": 96, "HV": 96, "D": 128, "dt": "bf16", "state": True},
        # One new token for one user: latency.
        {"name": "decode one sequence", "op": "recurrent", "lens": "1", "HK": 4, "HV": 8,
         "D": 128, "dt": "bf16", "state": True},
        # A few drafted tokens for each sequence, shared key heads.
        {"name": "decode drafted tokens", "op": "recurrent",
         "lens": ",".join(str(1 + i % 5) for i in range(32)), "HK": 16, "HV": 32, "D": 128,
         "dt": "f16", "state": True},
        # Gradients of the conv, SiLU and norm over a training batch.
        {"name": "prologue backward", "op": "prologue_bwd", "lens": "4096,2048,2048", "H": 32,
         "D": 128, "dt": "bf16", "grad": "bf16", "cache": False},
        # The same for a few tokens with the conv history of an earlier call, fp32 gradients.
        {"name": "prologue backward small", "op": "prologue_bwd", "lens": "33,2,0,70", "H": 3,
         "D": 64, "dt": "f16", "grad": "f32", "cache": True},
        # Gradients of the norm and the gate over a training batch.
        {"name": "epilogue backward", "op": "epilogue_bwd", "lens": "8192", "H": 32, "D": 128,
         "dt": "bf16"},
        # The same for a few rows, all in fp32.
        {"name": "epilogue backward small", "op": "epilogue_bwd", "lens": "17", "H": 3, "D": 64,
         "dt": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(rng, n, total):
    w = [rng.random() + 0.05 for _ in range(n)]
    lens = [max(1, int(total * x / sum(w))) for x in w]
    if n > 3 and rng.random() < 0.5:
        lens[rng.randrange(n)] = rng.choice([0, 1, 64, 65])
    return ",".join(map(str, lens))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk_bwd", "recurrent", "prologue_bwd", "epilogue_bwd"])
    if op in ("chunk", "chunk_bwd"):
        D = rng.choice([128, 128, 64])
        hk = _log(rng, 1, 16)
        hv = hk * rng.choice([1, 1, 2, 4])
        most = (1 << 20) if op == "chunk" else (1 << 17)  # value heads x tokens
        total = _log(rng, 40, max(64, min(24000, most // hv)))
        return {"op": op, "lens": _lens(rng, rng.choice([1, 1, 3, 7]), total), "HK": hk, "HV": hv,
                "D": D, "dt": rng.choice(["bf16", "bf16", "f16"]), "state": rng.random() < 0.6}
    if op == "recurrent":
        hk = _log(rng, 1, 32)
        hv = hk * rng.choice([1, 2, 4])
        n = _log(rng, 1, max(1, min(300, 16384 // hv)))
        most = rng.choice([1, 1, 5])
        return {"op": op, "lens": ",".join(str(rng.randint(1, most)) for _ in range(n)), "HK": hk,
                "HV": hv, "D": rng.choice([128, 128, 64, 32]),
                "dt": rng.choice(["bf16", "f16", "f32"]), "state": True}
    h = _log(rng, 1, 48)
    total = _log(rng, 20, 200000 // h)
    D = rng.choice([128, 128, 64, 32])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "prologue_bwd":
        return {"op": op, "lens": _lens(rng, rng.choice([1, 2, 5]), total), "H": h, "D": D,
                "dt": dt, "grad": rng.choice([dt, "f32"]), "cache": rng.random() < 0.4}
    return {"op": op, "lens": str(total), "H": h, "D": D, "dt": dt}


def _sizes(case):
    lens = [int(x) for x in case["lens"].split(",")]
    return lens, len(lens), sum(lens)


def work(case):
    lens, N, T = _sizes(case)
    D, op = case["D"], case["op"]
    es = 4 if case["dt"] == "f32" else 2
    if op == "epilogue_bwd":  # o, d_o in fp32; gate, d_out, d_gate
        n = T * case["H"] * D
        return {"bytes": n * (8 + 3 * es) + 8 * D, "flops": 20 * n}
    if op == "prologue_bwd":  # x, dx; the gradients of q, k, v; taps and their gradients
        n, ch = 3 * T * case["H"] * D, 3 * case["H"] * D
        gs = 4 if case["grad"] == "f32" else 2
        rows = 3 * N * ch * es * (2 if case["cache"] else 0)
        return {"bytes": n * (2 * es + gs) + 32 * ch + rows, "flops": 40 * n}
    HK, HV = case["HK"], case["HV"]
    qkv = T * (2 * HK + HV) * D * es
    state = 4 * N * HV * D * D * (2 if case["state"] else 0)
    if op == "chunk_bwd":  # q, k, v, g, beta, d_o in; their gradients out; the states' four
        return {"bytes": 2 * qkv + T * HV * (16 + 4 * D) + 2 * state, "flops": 21 * T * HV * D * D}
    return {"bytes": qkv + T * HV * (8 + 4 * D) + state, "flops": 7 * T * HV * D * D}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------

def prepare(case, seed):
    r = torch.Generator(DEV).manual_seed(int(seed) * 7919 + 13)

    def randn(*shape):
        return torch.randn(shape, generator=r, device=DEV)

    lens, N, T = _sizes(case)
    dt, D = TYPES[case["dt"]], case["D"]
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens).cumsum(0)
    s = {"op": case["op"], "N": N, "T": T, "D": D, "dt": dt, "cu": cu.to(DEV), "scale": D ** -0.5}
    if s["op"] == "epilogue_bwd":
        H = case["H"]
        s.update(o=0.3 * randn(T, H, D), gate=randn(T, H, D).to(dt), weight=1 + 0.1 * randn(D),
                 d_out=randn(T, H, D).to(dt), eps=1e-5)
        s["d_o"], s["d_gate"] = torch.empty_like(s["o"]), torch.empty_like(s["gate"])
        s["d_weight"] = torch.empty_like(s["weight"])
        if own:
            import gated_delta_rule_prologue_b200 as kda
            n = kda.kda_output_epilogue_bwd_workspace_bytes(T, H, D)
            s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        return s
    # Where each sequence's tokens stand in a batch padded to whole chunks (row T: padding).
    L = max(C, -(-max(lens) // C) * C) if "chunk" in s["op"] else max(lens)
    at = torch.arange(L)[None, :]
    idx = torch.where(at < torch.tensor(lens)[:, None], cu[:-1, None] + at, torch.tensor(T))
    s["idx"] = idx.to(DEV)
    s["back"] = torch.nonzero(idx.reshape(-1) < T)[:, 0].to(DEV)
    if s["op"] == "prologue_bwd":
        H = case["H"]
        ch = 3 * H * D
        gt = TYPES[case["grad"]]
        s.update(H=H, x=randn(T, ch).to(dt), w=0.5 * randn(ch, 4), cache=None, d_cache=None)
        for name in ("dq", "dk", "dv"):
            s[name] = randn(T, H, D).to(gt)
        s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
        if case["cache"]:
            s["cache"] = randn(N, 3, ch).to(dt)
            s["d_cache"] = torch.empty_like(s["cache"])
        if own:
            import gated_delta_rule_prologue_b200 as kda
            n = kda.kda_prologue_bwd_workspace_bytes(N, T, H, D, dt)
            s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        return s
    HK, HV = case["HK"], case["HV"]
    unit = lambda z: z / z.square().sum(-1, keepdim=True).add(1e-6).sqrt()  # noqa: E731
    silu = lambda z: z * torch.sigmoid(z)  # noqa: E731
    s["q"], s["k"] = (unit(silu(randn(T, HK, D))).to(dt) for _ in range(2))
    s["v"] = silu(randn(T, HV, D)).to(dt)
    # One rate per head, from almost no decay to a half-life of a token or so.
    rate = torch.exp(torch.rand(HV, generator=r, device=DEV) * math.log(1500.0) + math.log(1e-3))
    s["g"] = -rate * torch.log1p(torch.exp(randn(T, HV)))
    s["beta"] = torch.sigmoid(randn(T, HV))
    s["s0"] = 0.3 * randn(N, HV, D, D) if case["state"] else None
    s["o"] = torch.empty(T, HV, D, device=DEV)
    if s["op"] == "chunk_bwd":
        s["d_o"] = randn(T, HV, D)
        s["d_sN"] = randn(N, HV, D, D) if case["state"] else None
        for name, like in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "beta")):
            s[name] = torch.empty_like(s[like])
        s["d_s0"] = torch.empty_like(s["s0"]) if case["state"] else None
    else:
        s["sN"] = torch.empty(N, HV, D, D, device=DEV) if case["state"] else None
    if own and s["op"] != "recurrent":
        import gated_delta_rule_prologue_b200 as kda
        size = (kda.kda_gdr_chunk_fwd_workspace_bytes if s["op"] == "chunk"
                else kda.kda_gdr_chunk_bwd_workspace_bytes)
        s["ws"] = torch.empty(max(size(N, T, HK, HV, D, dt), 16), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------

def run(s):
    return _OPS[s["op"]][own](s)


def _own_chunk(s):
    import gated_delta_rule_prologue_b200 as kda
    kda.kda_gdr_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], scale=s["scale"],
                          initial_state=s["s0"], final_state=s["sN"], cu_seqlens=s["cu"],
                          workspace=s["ws"])
    return {"o": s["o"], "state": s["sN"]}


def _own_recurrent(s):
    import gated_delta_rule_prologue_b200 as kda
    kda.kda_gdr_recurrent(s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"], scale=s["scale"],
                          initial_state=s["s0"], final_state=s["sN"], cu_seqlens=s["cu"])
    return {"o": s["o"], "state": s["sN"]}


def _own_chunk_bwd(s):
    import gated_delta_rule_prologue_b200 as kda
    kda.kda_gdr_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["d_o"], scale=s["scale"],
                          initial_state=s["s0"], d_final_state=s["d_sN"], cu_seqlens=s["cu"],
                          dq=s["dq"], dk=s["dk"], dv=s["dv"], dg=s["dg"], dbeta=s["dbeta"],
                          d_initial_state=s["d_s0"], want_d_initial_state=s["d_s0"] is not None,
                          workspace=s["ws"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"], "dg": s["dg"], "dbeta": s["dbeta"],
            "d_state": s["d_s0"]}


def _own_prologue_bwd(s):
    import gated_delta_rule_prologue_b200 as kda
    kda.kda_prologue_bwd(s["x"], s["w"], s["dq"], s["dk"], s["dv"], s["dx"], s["dw"], H=s["H"],
                         D=s["D"], cache_in=s["cache"], d_cache_in=s["d_cache"],
                         cu_seqlens=s["cu"], workspace=s["ws"])
    return {"dx": s["dx"], "dw": s["dw"], "d_cache": s["d_cache"]}


def _own_epilogue_bwd(s):
    import gated_delta_rule_prologue_b200 as kda
    kda.kda_output_epilogue_bwd(s["o"], s["gate"], s["weight"], s["d_out"], s["d_o"], s["d_gate"],
                                s["d_weight"], eps=s["eps"], workspace=s["ws"])
    return {"d_o": s["d_o"], "d_gate": s["d_gate"], "d_weight": s["d_weight"]}


# ---- plain forms ------------------------------------------------------------------------

def _padded(x, idx, pad=0.0):
    """[T, ...] to fp32 [N, L, ...] with `pad` where a sequence has ended."""
    return torch.cat([x.float(), x.new_full((1,) + x.shape[1:], pad, dtype=torch.float32)])[idx]


def _chunks(x, idx, H):
    """[T, h, ...] to fp32 [N, H, chunks, C, ...], key heads repeated for their value heads."""
    x = _padded(x, idx)
    x = x.reshape(x.shape[0], -1, C, *x.shape[2:]).movedim(3, 1)
    return x.repeat_interleave(H // x.shape[1], 1) if x.shape[1] != H else x


def _packed(x, s):
    """[N, H, chunks, C, ...] back to [T, H, ...]."""
    x = x.movedim(1, 3)
    return x.reshape(-1, *x.shape[3:])[s["back"]]


def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower A [..., 64, 64]: the inverses of the diagonal blocks of
    size b give those of size 2 b, [[X, 0], [-Y A21 X, Y]], from b = 1 to 64."""
    n = A.shape[-1]
    lead = A.shape[:-2]
    T = torch.ones(*lead, n, 1, 1, device=A.device, dtype=A.dtype)
    b = 1
    while b < n:
        m = n // (2 * b)
        blocks = A.reshape(*lead, m, 2, b, m, 2, b)[..., 1, :, :, 0, :].diagonal(
            dim1=-4, dim2=-2).movedim(-1, -3)
        X, Y = T[..., 0::2, :, :], T[..., 1::2, :, :]
        low = -(Y @ blocks @ X)
        T = torch.cat([torch.cat([X, torch.zeros_like(X)], -1), torch.cat([low, Y], -1)], -2)
        b *= 2
    return T[..., 0, :, :]


def _chunk_terms(s):
    """What a chunk's products need and no state enters."""
    H = s["v"].shape[1]
    t = {n: _chunks(s[n], s["idx"], H) for n in ("q", "k", "v", "g", "beta")}
    gamma = t["g"].double().cumsum(-1)
    lower = torch.ones(C, C, device=gamma.device, dtype=torch.bool).tril()
    dec = torch.exp((gamma[..., :, None] - gamma[..., None, :]).masked_fill(~lower, -math.inf)).float()
    t["G"], t["E"] = torch.exp(gamma).float(), torch.exp(gamma[..., -1:] - gamma).float()
    t["dec"], t["low"] = dec, dec * lower.tril(-1)
    t["KK"] = t["k"] @ t["k"].mT
    t["P"] = (t["q"] @ t["k"].mT) * dec
    t["A"] = t["beta"][..., None] * t["low"] * t["KK"]
    t["inv"] = _unit_lower_inverse(t["A"])
    return t


def _states(t, S, keep=None):
    """The chunks in order: the read-outs (before the scale), the corrected values U, what
    the write of each token misses (R = V - G K S) and the last state."""
    o, u, r = (torch.empty_like(t["v"]) for _ in range(3))
    for c in range(t["v"].shape[2]):
        k, G = t["k"][:, :, c], t["G"][:, :, c, :, None]
        if keep is not None:
            keep[:, :, c] = S
        r[:, :, c] = t["v"][:, :, c] - G * (k @ S)
        u[:, :, c] = t["inv"][:, :, c] @ (t["beta"][:, :, c, :, None] * r[:, :, c])
        o[:, :, c] = G * (t["q"][:, :, c] @ S) + t["P"][:, :, c] @ u[:, :, c]
        S = G[:, :, -1:] * S + k.mT @ (t["E"][:, :, c, :, None] * u[:, :, c])
    return o, u, r, S


def _start(s):
    N, H, D = s["N"], s["v"].shape[1], s["D"]
    return s["s0"].mT if s["s0"] is not None else torch.zeros(N, H, D, D, device=DEV)


def _plain_chunk(s):
    t = _chunk_terms(s)
    o, _, _, S = _states(t, _start(s))
    return {"o": s["scale"] * _packed(o, s),
            "state": S.mT.contiguous() if s["sN"] is not None else None}


def _plain_chunk_bwd(s):
    t = _chunk_terms(s)
    N, H, n = t["v"].shape[:3]
    D = s["D"]
    S = torch.empty(N, H, n, D, D, device=DEV)
    _, u, r, _ = _states(t, _start(s), keep=S)
    do = s["scale"] * _chunks(s["d_o"], s["idx"], H)
    dS_out = torch.empty_like(S)
    dx = torch.empty_like(u)  # the gradient of (I + A) U = beta R's right-hand side
    dS = s["d_sN"].mT if s["d_sN"] is not None else torch.zeros(N, H, D, D, device=DEV)
    for c in range(n - 1, -1, -1):
        k, G = t["k"][:, :, c], t["G"][:, :, c, :, None]
        dS_out[:, :, c] = dS
        du = t["P"][:, :, c].mT @ do[:, :, c] + t["E"][:, :, c, :, None] * (k @ dS)
        dx[:, :, c] = t["inv"][:, :, c].mT @ du
        dr = t["beta"][:, :, c, :, None] * dx[:, :, c]
        dS = G[:, :, -1:] * dS + t["q"][:, :, c].mT @ (G * do[:, :, c]) - k.mT @ (G * dr)
    G, E, beta = t["G"][..., None], t["E"][..., None], t["beta"][..., None]
    dr = beta * dx
    dA = -(dx @ u.mT)
    dP = do @ u.mT
    from_q, from_r, from_u = (G * do) @ S.mT, (G * dr) @ S.mT, (E * u) @ dS_out.mT
    W = dP * t["dec"]
    M = dA * beta * t["low"]
    dq = from_q + W @ t["k"]
    dk = W.mT @ t["q"] + from_u - from_r + (M + M.mT) @ t["k"]
    dbeta = (dx * r).sum(-1) + (dA * t["low"] * t["KK"]).sum(-1)
    rows = dP * t["P"] + dA * t["A"]
    tail = (from_u * t["k"]).sum(-1)
    dgamma = rows.sum(-1) - rows.sum(-2) + (from_q * t["q"]).sum(-1) - (from_r * t["k"]).sum(-1) - tail
    dgamma[..., -1] += tail.sum(-1) + t["G"][..., -1] * (dS_out * S).sum((-1, -2))
    dg = dgamma.flip(-1).cumsum(-1).flip(-1)
    hk = s["q"].shape[1]
    dq, dk = (x.reshape(N, hk, H // hk, *x.shape[2:]).sum(2) for x in (dq, dk))
    return {"dq": _packed(dq, s).to(s["dt"]), "dk": _packed(dk, s).to(s["dt"]),
            "dv": _packed(dr, s).to(s["dt"]), "dg": _packed(dg, s), "dbeta": _packed(dbeta, s),
            "d_state": dS.mT.contiguous() if s["d_s0"] is not None else None}


def _plain_recurrent(s):
    H = s["v"].shape[1]
    q, k, v, g, beta = (_padded(s[n], s["idx"]) for n in ("q", "k", "v", "g", "beta"))
    q, k = (x.repeat_interleave(H // x.shape[2], 2) for x in (q, k))
    S = s["s0"]  # value-major, as it is stored
    o = torch.empty_like(v)
    for t in range(v.shape[1]):
        S = torch.exp(g[:, t])[..., None, None] * S
        e = v[:, t] - (S * k[:, t, :, None, :]).sum(-1)
        S = S + (beta[:, t, :, None] * e)[..., None] * k[:, t, :, None, :]
        o[:, t] = (S * q[:, t, :, None, :]).sum(-1)
    return {"o": s["scale"] * o.reshape(-1, H, s["D"])[s["back"]], "state": S}


def _conv_inputs(s, dtype=torch.float32):
    """[N, L + 3, 3 H D]: each sequence's inputs behind its three rows of history."""
    x = torch.cat([s["x"], s["x"].new_zeros(1, s["x"].shape[1])]).to(dtype)[s["idx"]]
    past = x.new_zeros(x.shape[0], 3, x.shape[2]) if s["cache"] is None else s["cache"].to(dtype)
    return torch.cat([past, x], 1)


def _plain_prologue_bwd(s):
    H, D = s["H"], s["D"]
    x, w = _conv_inputs(s), s["w"]
    N, L = x.shape[0], x.shape[1] - 3
    c = sum(w[:, j] * x[:, j:j + L] for j in range(4))
    sig = torch.sigmoid(c)
    y = (c * sig).reshape(N, L, 3, H, D)
    dn = torch.stack([_padded(s[n], s["idx"]) for n in ("dq", "dk", "dv")], 2)
    qk = y[:, :, :2]
    r = torch.rsqrt(qk.square().sum(-1, keepdim=True) + 1e-6)
    unit = qk * r
    dqk = r * (dn[:, :, :2] - unit * (dn[:, :, :2] * unit).sum(-1, keepdim=True))
    dy = torch.cat([dqk, dn[:, :, 2:]], 2).reshape(N, L, -1)
    dc = dy * sig * (1 + c * (1 - sig))
    dx = torch.zeros_like(x)
    for j in range(4):
        dx[:, j:j + L] += w[:, j] * dc
    dw = torch.stack([(dc * x[:, j:j + L]).double().sum((0, 1)) for j in range(4)], -1).float()
    out = {"dx": dx[:, 3:].reshape(N * L, -1)[s["back"]].to(s["dt"]), "dw": dw, "d_cache": None}
    if s["cache"] is not None:
        out["d_cache"] = dx[:, :3].to(s["dt"])
    return out


def _plain_epilogue_bwd(s):
    o, z, d = s["o"], s["gate"].float(), s["d_out"].float()
    r = torch.rsqrt(o.square().mean(-1, keepdim=True) + s["eps"])
    unit, sig = o * r, torch.sigmoid(z)
    dn = d * sig * s["weight"]
    d_o = r * (dn - unit * (dn * unit).mean(-1, keepdim=True))
    d_gate = d * unit * s["weight"] * sig * (1 - sig)
    d_weight = (d * sig * unit).double().sum((0, 1)).float()
    return {"d_o": d_o, "d_gate": d_gate.to(s["dt"]), "d_weight": d_weight}


_OPS = {"chunk": (_plain_chunk, _own_chunk), "chunk_bwd": (_plain_chunk_bwd, _own_chunk_bwd),
        "recurrent": (_plain_recurrent, _own_recurrent),
        "prologue_bwd": (_plain_prologue_bwd, _own_prologue_bwd),
        "epilogue_bwd": (_plain_epilogue_bwd, _own_epilogue_bwd)}


# ---------------------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------------------

def _by_token(x, s, H):
    """[T, h, ...] to fp64 [L, N, H, ...]; a token that a sequence lacks is all zeros, which
    leaves its state as it is."""
    x = torch.cat([x, x.new_zeros((1,) + x.shape[1:])]).to(F64)[s["idx"].T]
    return torch.stack([x[:, :, h * x.shape[2] // H] for h in range(H)], 2)


def _token(S, q, k, v, a, b):
    """One token of the recurrence on S [N, H, Dk, Dv]: the decayed state, the error, the new
    state."""
    Sd = a[..., None, None] * S
    e = v - torch.einsum("nhkv,nhk->nhv", Sd, k)
    return Sd, e, Sd + b[..., None, None] * k[..., :, None] * e[..., None, :]


def exact(case, seed):
    lens, N, T = _sizes(case)
    if case["op"] in ("chunk", "chunk_bwd") and max(lens) * N * case["HV"] * case["D"] ** 2 > 2e11:
        return None
    s = prepare(case, seed)
    if s["op"] == "epilogue_bwd":
        o, z, w, d = (s[n].to(F64) for n in ("o", "gate", "weight", "d_out"))
        D = s["D"]
        norm = (o.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt()
        gate = 1 / (1 + torch.exp(-z))
        up = d * gate * w
        d_o = up / norm - o * (up * o).sum(-1, keepdim=True) / (D * norm ** 3)
        d_gate = d * w * o / norm * torch.exp(-z) * gate ** 2
        return {"d_o": d_o, "d_gate": d_gate, "d_weight": (d * gate * o / norm).sum((0, 1))}
    if s["op"] == "prologue_bwd":
        H, D = s["H"], s["D"]
        dx, dw, dcache = torch.zeros(T, 3 * H * D, dtype=F64, device=DEV), 0, []
        x, w = s["x"].to(F64), s["w"].to(F64)
        up = torch.cat([s[n].to(F64).reshape(T, -1) for n in ("dq", "dk", "dv")], -1)
        a = 0
        for n, m in enumerate(lens):
            past = x.new_zeros(3, x.shape[1]) if s["cache"] is None else s["cache"][n].to(F64)
            row = torch.cat([past, x[a:a + m]])
            win = row.unfold(0, 4, 1) if m else row.new_zeros(0, row.shape[1], 4)
            c = (win * w).sum(-1)
            sig = 1 / (1 + torch.exp(-c))
            y, gr = (c * sig).reshape(m, 3, H, D), up[a:a + m].reshape(m, 3, H, D)
            norm = (y.square().sum(-1, keepdim=True) + 1e-6).sqrt()
            normed = gr / norm - y * (gr * y).sum(-1, keepdim=True) / norm ** 3
            dy = torch.where(torch.arange(3, device=DEV)[None, :, None, None] < 2, normed, gr)
            dc = dy.reshape(m, 3 * H * D) * (sig + c * sig * (1 - sig))
            drow = torch.zeros_like(row)
            for j in range(4):
                drow[j:j + m] += dc * w[:, j]
            dx[a:a + m] = drow[3:]
            dcache.append(drow[:3])
            dw = dw + (dc[..., None] * win).sum(0)
            a += m
        return {"dx": dx, "dw": dw, "d_cache": torch.stack(dcache) if s["cache"] is not None else None}
    HV, D = case["HV"], s["D"]
    q, k, v, b = (_by_token(s[n], s, HV) for n in ("q", "k", "v", "beta"))
    a = torch.exp(_by_token(s["g"], s, HV))
    S = torch.zeros(N, HV, D, D, dtype=F64, device=DEV)
    if s["s0"] is not None:
        S = s["s0"].to(F64).transpose(-1, -2)
    L = q.shape[0]
    rows = lambda x: x.transpose(0, 1).reshape(N * L, *x.shape[2:])[s["back"]]  # noqa: E731
    if s["op"] != "chunk_bwd":
        o = torch.zeros_like(v)
        for t in range(L):
            _, _, S = _token(S, q[t], k[t], v[t], a[t], b[t])
            o[t] = s["scale"] * torch.einsum("nhkv,nhk->nhv", S, q[t])
        return {"o": rows(o), "state": S.transpose(-1, -2) if s["sN"] is not None else None}
    # The adjoint of the recurrence, the states recomputed from one kept every 64 tokens.
    do = _by_token(s["d_o"], s, HV)
    kept = []
    for t in range(L):
        if t % 64 == 0:
            kept.append(S)
        S = _token(S, q[t], k[t], v[t], a[t], b[t])[2]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(a), torch.zeros_like(b)
    dS = torch.zeros(N, HV, D, D, dtype=F64, device=DEV)
    if s["d_sN"] is not None:
        dS = s["d_sN"].to(F64).transpose(-1, -2)
    for block in range(len(kept) - 1, -1, -1):
        seen, S = [], kept.pop()
        span = range(64 * block, min(L, 64 * block + 64))
        for t in span:
            Sd, e, S = _token(S, q[t], k[t], v[t], a[t], b[t])
            seen.append((Sd, e, S))
        for t in reversed(span):
            Sd, e, S = seen.pop()
            dS = dS + s["scale"] * q[t][..., :, None] * do[t][..., None, :]
            dq[t] = s["scale"] * torch.einsum("nhkv,nhv->nhk", S, do[t])
            m = torch.einsum("nhkv,nhk->nhv", dS, k[t])
            db[t] = (m * e).sum(-1)
            de = b[t][..., None] * m
            dv[t] = de
            dk[t] = torch.einsum("nhkv,nhv->nhk", dS, b[t][..., None] * e) - torch.einsum("nhkv,nhv->nhk", Sd, de)
            dS = dS - k[t][..., :, None] * de[..., None, :]
            dg[t] = (dS * Sd).sum((-1, -2))
            dS = a[t][..., None, None] * dS
    HK = case["HK"]
    dq, dk = (x.reshape(L, N, HK, HV // HK, D).sum(3) for x in (dq, dk))
    return {"dq": rows(dq), "dk": rows(dk), "dv": rows(dv), "dg": rows(dg), "dbeta": rows(db),
            "d_state": dS.transpose(-1, -2) if s["d_s0"] is not None else None}
