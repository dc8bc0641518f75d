"""Cases for the gated delta rule over the paged state pool (packed varlen extend, one-token
decode, chain verify) and for the packed state store (8-bit snapshots of pool slots).

Per request and value head h, with key head h // (H / Hk), D = 128 and an fp32 state S [D, D]
(rows: k, columns: v):

    S <- e^{g_t} S;  u_t = beta_t (v_t - S^T k_t);  S <- S + k_t u_t^T;  o_t = D^-0.5 S^T q_t

with q and k divided by sqrt(sum x^2 + 1e-6) first where ``l2`` is set.  The packed store keeps a
state in blocks of 32 along v: int8 codes and a power-of-two scale 2^(s - 127) per block.
"""
import math
import random

import torch

own = False

D = 128
CHUNK = 64
EPS = 1e-6
DEV = "cuda"


def listed():
    return [
        # one short prompt on a small model: latency of a single request's prefill
        dict(name="extend_one_short", op="extend", B=1, lo=37, hi=37, lens=0, Hk=4, H=8, l2=True, prefix=0),
        # a prefill step of eight prompts of mixed length, every other one continuing a cached prefix
        dict(name="extend_varlen", op="extend", B=8, lo=512, hi=4096, lens=1, Hk=16, H=16, l2=True, prefix=2),
        # one long document, grouped value heads
        dict(name="extend_long", op="extend", B=1, lo=32768, hi=32768, lens=0, Hk=16, H=32, l2=True, prefix=0),
        # a large batch of short prompts, keys normalised by the model itself
        dict(name="extend_many", op="extend", B=256, lo=32, hi=512, lens=2, Hk=16, H=16, l2=False, prefix=2),
        # interactive decoding of one request
        dict(name="decode_one", op="decode", B=1, Hk=8, H=16, l2=True),
        # a full decode batch
        dict(name="decode_batch", op="decode", B=256, Hk=16, H=16, l2=True),
        # an odd batch with grouped value heads
        dict(name="decode_grouped", op="decode", B=61, Hk=16, H=32, l2=False),
        # speculative decoding: the draft tokens of three requests
        dict(name="verify_small", op="verify", B=3, N=4, Hk=4, H=8, l2=True),
        # speculative decoding of a full batch
        dict(name="verify_batch", op="verify", B=128, N=5, Hk=16, H=64, l2=True),
        # one request's snapshot into the prefix cache and back
        dict(name="pack_one", op="pack", B=1, H=16),
        # a batch of evicted requests' states into the prefix cache and back
        dict(name="pack_batch", op="pack", B=128, H=32),
        # prefix-cache hits of an arriving batch: packed states back into pool slots
        dict(name="unpack_batch", op="unpack", B=96, H=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "extend", "decode", "verify", "pack", "unpack"])
    Hk = rng.choice([1, 2, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 3, 4])
    l2 = rng.random() < 0.6
    if op == "extend":
        B = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, min(16384, 260000 // (B * max(1, H // 4)))))
        lo = rng.randint(0, hi) if B > 1 else hi
        return dict(op=op, B=B, lo=lo, hi=hi, lens=rng.randrange(1 << 20), Hk=Hk, H=H, l2=l2,
                    prefix=rng.choice([0, 1, 2, 3]))
    if op == "decode":
        return dict(op=op, B=_log(rng, 1, 4096 // H), Hk=Hk, H=H, l2=l2)
    if op == "verify":
        N = rng.randint(1, 9)
        return dict(op=op, B=_log(rng, 1, max(1, 16384 // (H * N))), N=N, Hk=Hk, H=H, l2=l2)
    return dict(op=op, B=_log(rng, 1, 4096 // H), H=H)


def _lens(case):
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _slots(case):
    return case["B"] + 3


def work(case):
    H, B = case["H"], case["B"]
    mat = D * D * 4
    if case["op"] in ("pack", "unpack"):
        packed = D * D + D * D // 32
        return {"bytes": B * H * (mat + packed) * (2 if case["op"] == "pack" else 1), "flops": 0}
    if case["op"] == "extend":
        lens = _lens(case)
        tokens = sum(lens)
        prefixed = sum(bool(_prefixed(case, b)) for b in range(B))
        states = (prefixed + B) * H * mat
    else:
        tokens = B * case.get("N", 1)
        states = B * H * mat * (2 if case["op"] == "decode" else 1 + case["N"])
    rows = tokens * (2 * case["Hk"] * D * 2 + 2 * H * D * 2 + 8 * H)
    return {"bytes": rows + states, "flops": 6 * D * D * tokens * H}


def _prefixed(case, b):
    return case["prefix"] > 0 and b % case["prefix"] == 0


def _unit(x):
    return x / (x * x).sum(-1, keepdim=True).add(EPS).sqrt()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    B, H, slots = case["B"], case["H"], _slots(case)
    s = {"case": case, "idx": torch.randperm(slots, generator=gen, device=DEV)[:B].int()}
    if case["op"] in ("pack", "unpack"):
        # states of different heads and rows differ in size by orders of magnitude
        size = torch.exp(1.5 * rand(slots, H, D, 1))
        pool = rand(slots, H, D, D) * 0.05 * size
        s["sidx"] = torch.randperm(B + 2, generator=gen, device=DEV)[:B].int()
        s["codes"] = torch.zeros(B + 2, H, D, D, dtype=torch.int8, device=DEV)
        s["scales"] = torch.zeros(B + 2, H, D, D // 32, dtype=torch.uint8, device=DEV)
        if case["op"] == "unpack":
            s["codes"] = torch.randint(-127, 128, s["codes"].shape, generator=gen, device=DEV).to(torch.int8)
            s["scales"] = torch.randint(110, 128, s["scales"].shape, generator=gen, device=DEV).to(torch.uint8)
            s["pool"] = torch.zeros_like(pool)
        else:
            s["pool"], s["back"] = pool, torch.zeros_like(pool)
        return s
    Hk, N = case["Hk"], case.get("N", 1)
    if case["op"] == "extend":
        lens = _lens(case)
        tokens = sum(lens)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["lens"], s["cu"] = lens, torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["prefix"] = torch.tensor([int(_prefixed(case, b)) for b in range(B)], dtype=torch.uint8, device=DEV)
    else:
        tokens = B * N
    q, k = rand(tokens, Hk, D), torch.nn.functional.silu(rand(tokens, Hk, D))
    if not case["l2"]:
        q, k = _unit(q), _unit(k)
    s["q"], s["k"] = (x.reshape(tokens, Hk * D).bfloat16() for x in (q, k))
    s["v"] = rand(tokens, H * D).bfloat16()
    # g = -A softplus(x + bias), softplus(bias) between 0.001 and 0.1, A between 1 and 16 per head
    a = 1 + 15 * torch.rand(H, generator=gen, device=DEV)
    dt = torch.exp(torch.rand(H, generator=gen, device=DEV) * math.log(100.0) + math.log(1e-3))
    s["g"] = -a * torch.nn.functional.softplus(torch.log(torch.expm1(dt)) + 0.5 * rand(tokens, H))
    s["beta"] = torch.sigmoid(rand(tokens, H))
    s["pool"] = rand(slots, H, D, D) * 0.05
    if case["op"] == "verify":
        s["inter"] = torch.zeros(B, N, H, D, D, device=DEV)
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import lightning_attention_gb300 as la

    c = s["case"]
    if c["op"] == "pack":
        la.pack_states(s["pool"], s["idx"], s["codes"], s["scales"], s["sidx"])
        la.unpack_states(s["codes"], s["scales"], s["sidx"], s["back"], s["idx"])
        return s["back"]
    if c["op"] == "unpack":
        la.unpack_states(s["codes"], s["scales"], s["sidx"], s["pool"], s["idx"])
        return s["pool"]
    if c["op"] == "decode":
        return [la.delta_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["idx"],
                                qk_l2norm=c["l2"]), s["pool"]]
    if c["op"] == "verify":
        out, inter = la.delta_verify_chain(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["idx"],
                                           c["N"], inter_states=s["inter"], qk_l2norm=c["l2"])
        return [out, inter]
    out = la.delta_extend(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["idx"], s["cu"],
                          s["prefix"], max_seqlen=max(s["lens"]), qk_l2norm=c["l2"])
    return [out, s["pool"]]


def _plain(s):
    c = s["case"]
    idx = s["idx"].long()
    if c["op"] == "pack":
        codes, scales = _quantise(s["pool"][idx])
        s["codes"][s["sidx"].long()], s["scales"][s["sidx"].long()] = codes, scales
    if c["op"] in ("pack", "unpack"):
        to = s["back"] if c["op"] == "pack" else s["pool"]
        to[idx] = _restore(s["codes"][s["sidx"].long()], s["scales"][s["sidx"].long()])
        return to
    H, Hk = c["H"], c["Hk"]
    q, k = (x.float().reshape(-1, Hk, D) for x in (s["q"], s["k"]))
    if c["l2"]:
        q, k = _unit(q), _unit(k)
    q, k = (x.repeat_interleave(H // Hk, 1) for x in (q, k))
    v = s["v"].float().reshape(-1, H, D)
    if c["op"] == "extend":
        return _plain_extend(s, q, k, v)
    N = c.get("N", 1)
    B = c["B"]
    q, k, v = (x.reshape(B, N, H, D) for x in (q, k, v))
    decay, beta = s["g"].exp().reshape(B, N, H, 1, 1), s["beta"].reshape(B, N, H, 1)
    S, out = s["pool"][idx], torch.empty_like(v)
    for t in range(N):
        S = S * decay[:, t]
        u = beta[:, t] * (v[:, t] - (S * k[:, t, :, :, None]).sum(-2))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        out[:, t] = (S * q[:, t, :, :, None]).sum(-2)
        if c["op"] == "verify":
            s["inter"][:, t] = S
    if c["op"] == "decode":
        s["pool"][idx] = S
    out = (out * D ** -0.5).reshape(B * N, H * D).bfloat16()
    return [out, s["inter"] if c["op"] == "verify" else s["pool"]]


def _plain_extend(s, q, k, v):
    """The chunked form: within a chunk of 64 tokens u = (I + A)^-1 (beta v - beta e^G k S)."""
    c, lens = s["case"], s["lens"]
    B, H = c["B"], c["H"]
    n = max(1, -(-max(lens) // CHUNK))
    L = n * CHUNK
    cu = s["cu"].long()
    length = (cu[1:] - cu[:-1])[:, None]
    at = torch.arange(L, device=DEV)[None]
    valid = at < length
    rows = (cu[:-1, None] + at).clamp(max=max(0, q.shape[0] - 1))

    def pad(x, width):
        if not x.shape[0]:
            return torch.zeros(B, H, n, CHUNK, width, device=DEV)
        x = torch.where(valid[..., None, None], x.reshape(-1, H, width)[rows], 0.0)
        return x.reshape(B, n, CHUNK, H, width).permute(0, 3, 1, 2, 4).contiguous()

    q, k, v, g, beta = pad(q, D), pad(k, D), pad(v, D), pad(s["g"], 1), pad(s["beta"], 1)
    G = g[..., 0].double().cumsum(-1)  # differences of long sums of log decays
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    decay = (G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf).exp().float()
    A = (beta * (k @ k.transpose(-1, -2)) * decay).tril(-1)
    X = -A
    for i in range(1, CHUNK):  # rows of (I + A)^-1 - I by forward substitution
        X[..., i, :i] = X[..., i, :i] + (X[..., i, :i, None] * X[..., :i, :i]).sum(-2)
    X = X + torch.eye(CHUNK, device=DEV)
    gam = G.exp().float()[..., None]
    lam = (G[..., -1:] - G).exp().float()[..., None]
    W, V, P = X @ (beta * gam * k), X @ (beta * v), (q @ k.transpose(-1, -2)) * decay
    qg, kl, end = q * gam, (k * lam).transpose(-1, -2), gam[:, :, :, -1:, :]
    idx = s["idx"].long()
    S = torch.where(s["prefix"].bool()[:, None, None, None], s["pool"][idx], 0.0)
    out = torch.empty_like(v)
    for i in range(n):
        U = V[:, :, i] - W[:, :, i] @ S
        out[:, :, i] = qg[:, :, i] @ S + P[:, :, i] @ U
        S = end[:, :, i] * S + kl[:, :, i] @ U
    s["pool"][idx] = S
    out = (out * D ** -0.5).permute(0, 2, 3, 1, 4).reshape(B, L, H * D)
    return [out[valid].bfloat16(), s["pool"]]


def _pow2(e):
    """2^e in 64 bits, put together from its bits: library powers may be off in the last one."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise(x):
    """Codes in [-127, 127] and scale exponents (scale 2^(s - 127)) of blocks of 32 along the last
    axis: the smallest power of two that keeps the largest code at 127 or less, at least 2^-127; a
    block that is not finite has s = 255."""
    x = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32).double()
    top = x.abs().amax(-1)
    fine = torch.isfinite(top)
    e = torch.frexp(torch.where(fine, top, 1.0))[1] - 7  # top / 2^e is in [64, 128)
    e = torch.where(top == 0, -127, e).clamp(min=-127)
    e = e + (torch.round(torch.where(fine, top, 1.0) * _pow2(-e)) > 127).to(e.dtype)
    codes = torch.where(fine[..., None], torch.round(x * _pow2(-e)[..., None]), 0.0).to(torch.int8)
    return codes.flatten(-2), torch.where(fine, e + 127, 255).to(torch.uint8)


def _restore(codes, scales):
    x = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32).double()
    x = x * _pow2(scales.int() - 127)[..., None]
    return torch.where(scales[..., None] == 255, math.nan, x).float().flatten(-2)


def exact(case, seed):
    """The recurrence token by token in 64 bits."""
    s = prepare(case, seed)
    idx = s["idx"].long()
    if case["op"] in ("pack", "unpack"):
        at = s["sidx"].long()
        powers = torch.tensor([2.0 ** e for e in range(-200, 201)], dtype=torch.float64, device=DEV)
        if case["op"] == "unpack":
            scale = powers[s["scales"][at].long() - 127 + 200].repeat_interleave(32, -1)
            to = s["pool"].double()
            to[idx] = s["codes"][at].double() * scale
            return to
        to = s["back"].double()
        x = s["pool"][idx].double().unflatten(-1, (D // 32, 32))
        step = powers[torch.floor(torch.log2(x.abs().amax(-1, keepdim=True))).long() - 6 + 200]
        step = torch.where(torch.round(x.abs().amax(-1, keepdim=True) / step) > 127, 2 * step, step)
        to[idx] = (torch.round(x / step) * step).flatten(-2)
        return to
    H, Hk, B = case["H"], case["Hk"], case["B"]
    rep = H // Hk
    q, k = (x.double().reshape(-1, Hk, D) for x in (s["q"], s["k"]))
    if case["l2"]:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS) for x in (q, k))
    v, g, beta = s["v"].double().reshape(-1, H, D), s["g"].double(), s["beta"].double()
    first = s["cu"][:-1].long() if case["op"] == "extend" else torch.arange(B, device=DEV) * case.get("N", 1)
    lens = s["lens"] if case["op"] == "extend" else [case.get("N", 1)] * B
    order = sorted(range(B), key=lambda b: -lens[b])  # the requests still running are a prefix of it
    perm = torch.tensor(order, device=DEV)
    S = s["pool"][idx].double()
    if case["op"] == "extend":
        S[s["prefix"] == 0] = 0
    S = S[perm].transpose(-1, -2).contiguous()  # [B, H, v, k]
    out = torch.zeros_like(v)
    inter = s["inter"].double() if case["op"] == "verify" else None
    live = B
    for t in range(max(lens)):
        while live and lens[order[live - 1]] <= t:
            live -= 1
        rows = first[perm[:live]] + t
        kt, qt = (x[rows].repeat_interleave(rep, 1)[..., None] for x in (k, q))
        M = S[:live]
        M *= g[rows].exp()[..., None, None]
        u = beta[rows][..., None, None] * (v[rows][..., None] - M @ kt)
        M += u * kt.transpose(-1, -2)
        out[rows] = (M @ qt)[..., 0]
        if inter is not None:
            inter[perm[:live], t] = M.transpose(-1, -2)
    out = (out * D ** -0.5).reshape(-1, H * D)
    if inter is not None:
        return [out, inter]
    pool = s["pool"].double()
    pool[idx[perm]] = S.transpose(-1, -2)
    return [out, pool]
