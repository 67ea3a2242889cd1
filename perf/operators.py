"""Cases and plain forms of the decayed linear attention and the multi-axis rotary embedding.

Three operators of ``block_causal_linear_rope_b200``:

``decay_prefill``  causal linear attention over a prompt with one decay per head,
                   S_n = g_h S_{n-1} + k_n^T v_n,   o_n = scale * q_n S_n,
                   ragged rows, states read from and written to slots of a pool;
``decay_step``     the same recurrence for one token per request;
``rope``           rotary positions over the axes (t, y, x) of q and k, from a
                   latent grid or from given positions, forward or inverse
                   (the inverse rotation is also the gradient).

``own = False`` computes them with elementary torch operations in 32 bits,
``own = True`` through the package's entry points; ``exact`` gives the definition
in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 128  # tokens per block of the plain chunked form


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # a chat turn's first prompt: a launch-bound call, odd length
        dict(name="prefill-short", op="prefill", B=1, H=16, N=77, d=64, dtype="bf16", decay="slopes", ragged=False,
             pool=1, fused=False),
        # a serving batch of prompts of unequal lengths (one empty, one row idle) into a pool of states
        dict(name="prefill-ragged", op="prefill", B=8, H=32, N=2048, d=128, dtype="bf16", decay="retention",
             ragged=True, pool=12, fused=False),
        # one long document
        dict(name="prefill-long", op="prefill", B=1, H=32, N=32768, d=128, dtype="bf16", decay="retention",
             ragged=False, pool=1, fused=False),
        # the 480p video's tokens, read in place from a fused projection [B, N, 3, H, d]
        dict(name="prefill-480p", op="prefill", B=1, H=70, N=32760, d=32, dtype="bf16", decay="retention",
             ragged=False, pool=1, fused=True),
        # the wide video workload: four sequences, 64-wide heads
        dict(name="prefill-wide", op="prefill", B=4, H=32, N=32760, d=64, dtype="bf16", decay="slopes", ragged=False,
             pool=4, fused=False),
        # full precision, two sequences
        dict(name="prefill-f32", op="prefill", B=2, H=16, N=4000, d=64, dtype="f32", decay="retention", ragged=False,
             pool=2, fused=False),
        # one request's next token
        dict(name="step-one", op="step", B=1, H=32, d=128, dtype="bf16", decay="retention", pool=1, idle=0),
        # a decode batch out of a larger pool of states, some of its rows idle
        dict(name="step-batch", op="step", B=128, H=32, d=128, dtype="bf16", decay="retention", pool=160, idle=5),
        # narrow heads in full precision
        dict(name="step-f32", op="step", B=32, H=70, d=32, dtype="f32", decay="slopes", pool=40, idle=1),
        # q and k of the 720p video, positions from the latent grid
        dict(name="rope-720p", op="rope", B=1, Hq=70, Hk=70, N=75600, Hg=45, Wg=80, t0=0, d=32, dtype="bf16",
             split_t=8, split_y=12, split_x=12, inverse=False),
        # one token of each of 64 requests, given positions, fewer key heads
        dict(name="rope-decode", op="rope", B=64, Hq=32, Hk=8, N=1, Hg=0, Wg=0, t0=0, d=128, dtype="bf16",
             split_t=32, split_y=48, split_x=48, inverse=False),
        # the gradient's rotation of a prompt of text and images, a part of each head left alone
        dict(name="rope-inverse-f32", op="rope", B=2, Hq=24, Hk=24, N=4099, Hg=0, Wg=0, t0=0, d=64, dtype="f32",
             split_t=16, split_y=16, split_x=16, inverse=True),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "rope"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "prefill":
        d = rng.choice([32, 64, 128])
        B, H = _spread(rng, 1, 16), _spread(rng, 1, 70)
        room = (130_000_000 if dtype == "bf16" else 20_000_000) // (B * H * d)
        N = _spread(rng, 1, max(1, min(40000, room)))
        return dict(op=op, B=B, H=H, N=N, d=d, dtype=dtype, decay=rng.choice(["retention", "slopes"]),
                    ragged=rng.random() < 0.5, pool=B + rng.choice([0, 0, 3]), fused=rng.random() < 0.3)
    if op == "step":
        d = rng.choice([32, 64, 128])
        H = _spread(rng, 1, 70)
        B = _spread(rng, 1, max(1, min(256, 60_000_000 // (H * d * d))))
        return dict(op=op, B=B, H=H, d=d, dtype=dtype, decay=rng.choice(["retention", "slopes"]),
                    pool=B + rng.choice([0, 2, 17]), idle=rng.choice([0, 0, min(B - 1, 2)]))
    d = rng.choice([32, 64, 96, 128])
    parts = [2 * rng.randint(1, d // 6) for _ in range(3)]
    B, Hq = _spread(rng, 1, 16), _spread(rng, 1, 70)
    Hk = Hq if rng.random() < 0.6 else max(1, Hq // 4)
    room = (130_000_000 if dtype == "bf16" else 60_000_000) // (B * Hq * d)
    if rng.random() < 0.5:
        Hg, Wg = _spread(rng, 1, 60), _spread(rng, 1, 90)
        T = _spread(rng, 1, max(1, min(60, room // (Hg * Wg))))
        N, t0 = T * Hg * Wg, rng.choice([0, 5, 240])
        if N * B * Hq * d > 300_000_000:
            B = Hq = Hk = 1
    else:
        N, Hg, Wg, t0 = _spread(rng, 1, max(1, min(40000, room))), 0, 0, 0
    return dict(op="rope", B=B, Hq=Hq, Hk=Hk, N=N, Hg=Hg, Wg=Wg, t0=t0, d=d, dtype=dtype, split_t=parts[0],
                split_y=parts[1], split_x=parts[2], inverse=rng.random() < 0.4)


# ----------------------------------------------------------------------------- inputs
def _log_decay(case):
    """log g_h: retention heads 1 - 2^(-5 ... -12), or slopes 2^(-8 (h+1) / H)."""
    h = torch.arange(case["H"], dtype=torch.float64)
    if case["decay"] == "retention":
        lg = torch.log1p(-torch.exp2(-5.0 - 7.0 * h / max(1, case["H"] - 1)))
    else:
        lg = -torch.exp2(-8.0 * (h + 1.0) / case["H"])
    return lg.float().cuda()


def _pool(case, lg, gen):
    """States as a running service holds them: the recurrence's standard deviation for unit inputs."""
    std = torch.rsqrt(1.0 - torch.exp(2.0 * lg)).view(1, -1, 1, 1)
    return torch.randn(case["pool"], case["H"], case["d"], case["d"], generator=gen, device="cuda") * std


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed + 1)
    dt, d, B = DT[case["dtype"]], case["d"], case["B"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dt)

    if case["op"] == "rope":
        N = case["N"]
        s = dict(q=normal(B, case["Hq"], N, d), k=normal(B, case["Hk"], N, d), positions=None)
        if not case["Hg"]:
            # text and images in turn: text advances all three axes together, an image's tokens share a time
            n = torch.arange(N)
            base = torch.randint(0, 30000, (B, 1), generator=host)
            image = (n // 256) % 2 == 1
            at = n % 256
            t = base + torch.where(image, n - at, n)
            y = torch.where(image, base + n - at + at // 16, t)
            x = torch.where(image, base + n - at + at % 16, t)
            s["positions"] = torch.stack([t, y, x], dim=-1).to(torch.int32).cuda()
    else:
        H = case["H"]
        lg = _log_decay(case)
        s = dict(log_decay=lg, scale=d ** -0.5, state=_pool(case, lg, gen), lengths=None, slots=None)
        if case["op"] == "prefill":
            N = case["N"]
            if case["fused"]:
                s["q"], s["k"], s["v"] = normal(B, N, 3, H, d).permute(2, 0, 3, 1, 4).unbind(0)
            else:
                s["q"], s["k"], s["v"] = normal(B, H, N, d), normal(B, H, N, d), normal(B, H, N, d)
            if case["ragged"]:
                n = torch.randint(0, N + 1, (B,), generator=host)
                n[0] = N
                if B > 2:
                    n[1] = 0
                s["lengths"] = n.to(torch.int32).cuda()
            idle = 1 if case["ragged"] and B > 3 else 0
        else:
            s["q"], s["k"], s["v"] = normal(B, H, d), normal(B, H, d), normal(B, H, d)
            idle = case["idle"]
        if case["pool"] > B or idle:
            slots = torch.randperm(case["pool"], generator=host)[:B]
            slots[torch.randperm(B, generator=host)[:idle]] = -1
            s["slots"] = slots.to(torch.int32).cuda()
    s["case"] = dict(case)
    return s


# ----------------------------------------------------------------------------- the operators, plain
def _rows_of(state, slots):
    """The rows' states (zeros for idle rows) and which rows are served."""
    if slots is None:
        return state, None
    served = (slots >= 0).view(-1, 1, 1, 1)
    return torch.where(served, state[slots.clamp(min=0).long()], 0.0), served


def _store(state, slots, new):
    """Writes the rows' new states to their slots."""
    if slots is None:
        state.copy_(new)
        return
    match = slots.view(1, -1) == torch.arange(state.shape[0], device=state.device).view(-1, 1)
    row = match.to(torch.int32).argmax(dim=1)
    state.copy_(torch.where(match.any(dim=1).view(-1, 1, 1, 1), new[row], state))


def _powers(lg, n):
    """exp(lg * n) in 32 bits, the exponent in 64 (lg and n broadcast)."""
    return torch.exp(lg.double() * n).float()


def _plain_prefill(s):
    q, k, v, lg, state = s["q"], s["k"], s["v"], s["log_decay"], s["state"]
    B, H, N, d = q.shape
    C = min(CHUNK, N)
    nc = -(-N // C)
    n = torch.arange(N, device=q.device)
    L = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), N, device=q.device)
    given = (n.view(1, 1, N, 1) < L.view(B, 1, 1, 1))

    def chunks(x):
        x = torch.where(given, x.float(), 0.0)
        return torch.nn.functional.pad(x, (0, 0, 0, nc * C - N)).view(B, H, nc, C, d)

    qc, kc, vc = chunks(q), chunks(k), chunks(v)
    S0, served = _rows_of(state, s["slots"])
    i = torch.arange(C, device=q.device)
    g = lg.view(H, 1, 1)
    D = torch.where(i.view(C, 1) >= i, _powers(g, (i.view(C, 1) - i).clamp(min=0)), 0.0)  # [H, C, C]
    intra = (qc @ kc.transpose(-1, -2) * D.view(1, H, 1, C, C)) @ vc
    own_kv = (kc * _powers(g, (C - 1 - i).view(1, C, 1)).view(1, H, 1, C, 1)).transpose(-1, -2) @ vc
    # states entering each chunk: all earlier chunks' products and the cache, weighted by distance
    c = torch.arange(nc, device=q.device)
    W = torch.where(c.view(nc, 1) > c, _powers(g, C * (c.view(nc, 1) - c - 1).clamp(min=0)), 0.0)  # [H, nc, nc]
    before = (W @ own_kv.view(B, H, nc, d * d)).view(B, H, nc, d, d)
    before = before + _powers(g, C * c).view(1, H, nc, 1, 1) * S0.view(B, H, 1, d, d)
    inter = (qc @ before) * _powers(g, (i + 1).view(1, C, 1)).view(1, H, 1, C, 1)
    o = s["scale"] * (intra + inter).view(B, H, nc * C, d)[:, :, :N]
    o = torch.where(given if served is None else given & served, o, 0.0).to(q.dtype)
    # the states after each row's last token
    left = (L.view(B, 1, 1) - 1 - n.view(1, 1, N))
    w = torch.where(left >= 0, _powers(lg.view(1, H, 1), left.clamp(min=0)), 0.0)
    w = torch.nn.functional.pad(w, (0, nc * C - N)).view(B, H, nc, C, 1)
    new = ((kc * w).transpose(-1, -2) @ vc).sum(dim=2) + _powers(lg.view(1, H), L.view(B, 1)).view(B, H, 1, 1) * S0
    _store(state, s["slots"], new)
    return o, state


def _plain_step(s):
    q, k, v = (s[x].float() for x in "qkv")
    S0, served = _rows_of(s["state"], s["slots"])
    new = torch.exp(s["log_decay"]).view(1, -1, 1, 1) * S0 + k.unsqueeze(-1) * v.unsqueeze(-2)
    o = s["scale"] * (q.unsqueeze(-2) @ new).squeeze(-2)
    if served is not None:
        o = torch.where(served.squeeze(-1), o, 0.0)
    _store(s["state"], s["slots"], new)
    return o.to(s["q"].dtype), s["state"]


def _positions(s):
    """[1 or B, N, 3] positions of the tokens: given, or of the grid (t-major, then y, then x)."""
    case = s["case"]
    if s["positions"] is not None:
        return s["positions"].view(-1, case["N"], 3)
    n = torch.arange(case["N"], device="cuda")
    hw = case["Hg"] * case["Wg"]
    return torch.stack([case["t0"] + n // hw, n % hw // case["Wg"], n % case["Wg"]], dim=-1).unsqueeze(0)


def _plain_rope(s):
    case, d = s["case"], s["case"]["d"]
    split = [case["split_t"], case["split_y"], case["split_x"]]
    pos = _positions(s).double()
    turn = torch.cat([pos[..., a:a + 1] * 1e4 ** (-torch.arange(0, n, 2, device="cuda", dtype=torch.float64) / n)
                      for a, n in enumerate(split)], dim=-1).unsqueeze(1)
    c, sn = torch.cos(turn).float(), torch.sin(turn).float()
    if case["inverse"]:
        sn = -sn
    m = sum(split)

    def rotate(x):
        a, b = x[..., 0:m:2].float(), x[..., 1:m:2].float()
        y = torch.stack([a * c - b * sn, a * sn + b * c], dim=-1).flatten(-2).to(x.dtype)
        return torch.cat([y, x[..., m:]], dim=-1) if m < d else y

    return rotate(s["q"]), rotate(s["k"])


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"prefill": _plain_prefill, "step": _plain_step, "rope": _plain_rope}[case["op"]](s)
    import block_causal_linear_rope_b200 as blin
    if case["op"] == "prefill":
        return blin.decay_prefill(s["q"], s["k"], s["v"], s["log_decay"], state=s["state"], slots=s["slots"],
                                  lengths=s["lengths"], scale=s["scale"]), s["state"]
    if case["op"] == "step":
        return blin.decay_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], slots=s["slots"],
                               scale=s["scale"]), s["state"]
    split = (case["split_t"], case["split_y"], case["split_x"])
    if s["positions"] is not None:
        return blin.rope(s["q"], s["k"], positions=s["positions"], rope_split=split, inverse=case["inverse"])
    grid = (case["N"] // (case["Hg"] * case["Wg"]), case["Hg"], case["Wg"])
    return blin.rope(s["q"], s["k"], grid=grid, t0=case["t0"], rope_split=split, inverse=case["inverse"])


# ----------------------------------------------------------------------------- work and definition
def work(case):
    es, d = 2 if case["dtype"] == "bf16" else 4, case["d"]
    if case["op"] == "rope":
        n = case["B"] * (case["Hq"] + case["Hk"]) * case["N"]
        m = case["split_t"] + case["split_y"] + case["split_x"]
        return {"bytes": 2 * n * d * es + (0 if case["Hg"] else 12 * case["B"] * case["N"]), "flops": 3 * n * m}
    heads = case["B"] * case["H"]
    if case["op"] == "step":
        live = (case["B"] - case["idle"]) * case["H"]
        return {"bytes": 8 * live * d * d + 4 * heads * d * es, "flops": 5 * live * d * d}
    # ragged rows: lengths are drawn from [0, N], so half the tokens are there
    tokens = heads * case["N"] * (0.5 if case["ragged"] and case["B"] > 1 else 1.0)
    return {"bytes": 4 * tokens * d * es + 8 * heads * d * d, "flops": 4 * tokens * d * d}


def _exact_recurrence(s, tokens):
    """The recurrence in 64 bits, 64 tokens of every row and head at a time."""
    q, k, v = s["q"], s["k"], s["v"]
    if tokens is None:
        q, k, v = (x.unsqueeze(2) for x in (q, k, v))
    B, H, N, d = q.shape
    lens = [N] * B if s["lengths"] is None else s["lengths"].tolist()
    slots = list(range(B)) if s["slots"] is None else s["slots"].tolist()
    lens = torch.tensor([n if p >= 0 else 0 for n, p in zip(lens, slots)], device="cuda")
    pool = s["state"].double()
    rows = torch.tensor([max(p, 0) for p in slots], device="cuda")
    S, g = pool[rows], s["log_decay"].double().view(1, H, 1, 1)
    out = torch.zeros(B, H, N, d, dtype=torch.float64, device="cuda")
    for a in range(0, N, 64):
        m = min(64, N - a)
        i = torch.arange(m, device="cuda")
        here = (lens - a).clamp(0, m).view(B, 1, 1, 1)
        live = i.view(1, 1, m, 1) < here
        qs, ks, vs = (torch.where(live, x[:, :, a:a + m].double(), 0.0) for x in (q, k, v))
        far = (i.view(m, 1) - i).view(1, 1, m, m)
        score = torch.where(far >= 0, torch.exp(g * far.clamp(min=0)) * (qs @ ks.mT), 0.0)
        rest = torch.exp(g * (i + 1).view(1, 1, m, 1)) * (qs @ S)
        out[:, :, a:a + m] = torch.where(live, s["scale"] * (score @ vs + rest), 0.0)
        S = torch.exp(g * here) * S + (torch.exp(g * (here - 1 - i.view(1, 1, m, 1)).clamp(min=0)) * ks).mT @ vs
    for b, p in enumerate(slots):
        if p >= 0:
            pool[p] = S[b]
    return out if tokens is not None else out.squeeze(2), pool


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "rope":
        return _exact_recurrence(s, case.get("N"))
    angle, sections = [], (case["split_t"], case["split_y"], case["split_x"])
    pos = _positions(s).double()
    for a, n in enumerate(sections):
        for j in range(n // 2):
            angle.append(pos[..., a] * math.pow(1e4, -2.0 * j / n))
    angle = torch.stack(angle, dim=-1).unsqueeze(1)
    w = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)
    m = sum(sections)
    outs = []
    for x in (s["q"].double(), s["k"].double()):
        x[..., :m] = torch.view_as_real(torch.view_as_complex(x[..., :m].unflatten(-1, (-1, 2)).contiguous()) * w).flatten(-2)
        outs.append(x)
    return tuple(outs)
