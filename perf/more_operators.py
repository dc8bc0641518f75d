"""Cases for the softmax-attention layers of a hybrid model over a paged key/value cache: rotary
positions (alone, and with the keys and values stored into pages), attention of packed prompts,
attention of single tokens and of drafted trees over the cache, and the commit of accepted drafts.

D = 128, H query heads on Hkv key/value heads, pages bf16 [pages, Hkv, P, D]; position j of request
b is row j % P of page page_table[b, j // P].

  rotary     a pair (x, y) of a head at position p, angle a = p f_i:
             (x, y) -> m (x cos a - y sin a, x sin a + y cos a)
  attention  o_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale q_i . k_j) over the keys j that row i sees:
             in a prompt those at and before it, in a tree the context, its ancestors and itself
"""
import math
import random

import torch

own = False

D = 128
DEV = "cuda"
SCALE = D ** -0.5


def listed():
    return [
        # the prompt of a linear-attention layer, half of each head rotated
        dict(name="rope_prompt", op="rope", T=16384, H=32, Hkv=32, rot=64, inter=True, scaling="none", far=16384),
        # a decode batch of a softmax layer: q rotated, keys and values into their pages, far positions
        dict(name="store_decode", op="store", T=256, H=32, Hkv=4, rot=128, inter=False, scaling="yarn", far=131072, P=64),
        # one short prompt on a small model: latency
        dict(name="extend_one_short", op="extend", B=1, lo=37, hi=37, plo=0, phi=0, lens=0, H=16, Hkv=4, P=16),
        # a prefill step of eight prompts of mixed length
        dict(name="extend_varlen", op="extend", B=8, lo=512, hi=4096, plo=0, phi=0, lens=1, H=32, Hkv=4, P=64),
        # one long document
        dict(name="extend_long", op="extend", B=1, lo=16384, hi=16384, plo=0, phi=0, lens=0, H=32, Hkv=8, P=128),
        # the next chunk of three long prompts, six query heads a group
        dict(name="extend_chunked", op="extend", B=3, lo=400, hi=600, plo=6000, phi=20000, lens=2, H=24, Hkv=4, P=32),
        # interactive decoding of one request
        dict(name="decode_one", op="decode", B=1, lo=1000, hi=1000, lens=0, H=32, Hkv=4, P=64),
        # a full decode batch of mixed lengths
        dict(name="decode_batch", op="decode", B=128, lo=500, hi=8000, lens=3, H=32, Hkv=4, P=64),
        # two requests over very long documents
        dict(name="decode_long", op="decode", B=2, lo=100000, hi=131072, lens=4, H=64, Hkv=8, P=16),
        # speculative decoding of a batch with trees of eight drafts
        dict(name="tree_batch", op="tree", B=64, N=8, lo=1000, hi=8000, lens=5, H=64, Hkv=8, P=64),
        # the step after it, for one request of a small model: accepted drafts to the end of the context
        dict(name="commit_one", op="commit", B=1, N=6, lo=700, hi=700, lens=7, Hkv=4, P=64),
        # and for a full batch
        dict(name="commit_batch", op="commit", B=256, N=16, lo=20, hi=300, lens=6, Hkv=8, P=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "store", "extend", "extend", "decode", "tree", "commit"])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * max(rng.choice([1, 2, 3, 4, 5, 6, 8, 16]), -(-8 // Hkv))
    P, lens = rng.choice([16, 32, 64, 128]), rng.randrange(1 << 20)
    if op in ("rope", "store"):
        case = dict(op=op, T=_log(rng, 1, 1 << 19) // (H + 2 * Hkv) + 1, H=H, Hkv=Hkv, rot=16 * rng.randint(1, 8),
                    inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    far=_log(rng, 64, 1 << 20))
        return dict(case, P=P) if op == "store" else case
    if op == "extend":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 8192 // math.isqrt(B))
        phi = rng.choice([0, _log(rng, 1, max(1, min(32768, (1 << 26) // (hi * B))))])
        return dict(op=op, B=B, lo=rng.randint(0, hi) if B > 1 else hi, hi=hi, plo=rng.randint(0, phi), phi=phi,
                    lens=lens, H=min(H, 32), Hkv=Hkv if H <= 32 else 2, P=P)
    if op == "commit":
        B = _log(rng, 1, 512)
        return dict(op=op, B=B, N=rng.randint(1, 32), lo=0, hi=_log(rng, 1, max(2, 65536 // B)), lens=lens, Hkv=Hkv, P=P)
    B = _log(rng, 1, 256)
    hi = _log(rng, 1, (1 << 21) // (B * Hkv))
    case = dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, lens=lens, H=H, Hkv=Hkv, P=P)
    return dict(case, N=rng.randint(2, 16)) if op == "tree" else case


def _lens(case):
    """(new tokens, positions before them) of each request."""
    r = random.Random(case["lens"])
    B = case["B"]
    if case["op"] == "extend":
        return ([case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(B - 1)],
                [r.randint(case["plo"], case["phi"]) for _ in range(B)])
    return [case.get("N", 1)] * B, [r.randint(case["lo"], case["hi"]) for _ in range(B)]


def work(case):
    op, Hkv = case["op"], case["Hkv"]
    if op in ("rope", "store"):
        heads = case["H"] + Hkv * (2 if op == "store" else 1)
        return {"bytes": case["T"] * (heads * D * 4 + (8 if op == "store" else 4)) + 4 * case["rot"],
                "flops": 3 * case["T"] * (case["H"] + Hkv) * case["rot"]}
    new, old = _lens(case)
    if op == "commit":
        paths = sum(_accepts(case)[1])
        return {"bytes": paths * Hkv * D * 2 * 2 * 2 + case["B"] * (case["N"] + 3) * 4, "flops": 0}
    H = case["H"]
    keys = sum(n + m for n, m in zip(new, old) if n)
    pairs = sum(n * m + n * (n + 1) // 2 for n, m in zip(new, old))  # of a tree at most, little beside the context
    return {"bytes": sum(new) * H * D * 2 * 2 + keys * Hkv * D * 2 * 2, "flops": 4 * D * H * pairs}


def _trees(case):
    """Parents of every request's drafts: token t hangs on a random earlier one or on the context."""
    r = random.Random(case["lens"] + 1)
    return [[r.randint(max(-1, t - 4), t - 1) for t in range(case["N"])] for _ in range(case["B"])]


def _accepts(case):
    """(last accepted draft or -1, drafts on its path) of each request."""
    r = random.Random(case["lens"] + 2)
    last, paths = [], []
    for tree in _trees(case):
        a = at = r.randint(-1, case["N"] - 1)
        n = 0
        while at >= 0:
            at, n = tree[at], n + 1
        last.append(a)
        paths.append(n)
    return last, paths


def _frequencies(case):
    """(inverse frequencies in 64 bits, factor on the rotated values)."""
    R, base, factor, orig = case["rot"], 10000.0, 8.0, 8192
    i = torch.arange(R // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * factor ** (R / max(R - 2, 1))
    f = base ** (-2 * i / R)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":
        # few turns over the original length: interpolated; many: kept; a ramp between
        at = [R * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=gen, device=DEV).int()  # noqa: E731
    op, Hkv = case["op"], case["Hkv"]
    s = {"case": case}
    if op in ("rope", "store"):
        T = case["T"]
        s["q"], s["k"] = rand(T, case["H"] * D), rand(T, Hkv * D)
        s["pos"] = torch.randint(0, case["far"], (T,), generator=gen, device=DEV).int()
        f, s["mscale"] = _frequencies(case)
        s["freq"] = f.to(DEV)
        if op == "store":
            P = case["P"]
            s["v"] = rand(T, Hkv * D)
            pages = -(-T // P) + 2
            s["kp"], s["vp"] = rand(pages, Hkv, P, D), rand(pages, Hkv, P, D)
            s["loc"] = perm(pages * P)[:T].contiguous()
        return s
    new, old = _lens(case)
    P, B = case["P"], case["B"]
    need = [-(-(n + m) // P) for n, m in zip(new, old)]
    width, pages = max(1, max(need)), sum(need) + 2
    order, table, at = perm(pages), torch.zeros(B, width, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    s["table"] = order[table.long().to(DEV)].contiguous()
    s["kp"], s["vp"] = rand(pages, Hkv, P, D), rand(pages, Hkv, P, D)
    total = [n + m for n, m in zip(new, old)]
    s["kv"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    if op != "commit":
        s["q"] = rand(sum(new), case["H"] * D) * 2
    if op == "extend":
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["new"], s["total"], s["cu"] = new, total, torch.tensor(cu, dtype=torch.int32, device=DEV)
    if op in ("tree", "commit"):
        s["parents"] = torch.tensor(_trees(case), dtype=torch.int32, device=DEV)
    if op == "commit":
        s["accept"] = torch.tensor(_accepts(case)[0], dtype=torch.int32, device=DEV)
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import lightning_attention_gb300 as la

    c = s["case"]
    if c["op"] == "rope":
        return list(la.rope(s["q"], s["k"], s["pos"], s["freq"], interleaved=c["inter"], mscale=s["mscale"]))
    if c["op"] == "store":
        out = la.kv_store(s["q"], s["k"], s["v"], s["pos"], s["freq"], s["kp"], s["vp"], s["loc"],
                          interleaved=c["inter"], mscale=s["mscale"])
        return [out, s["kp"], s["vp"]]
    if c["op"] == "extend":
        return la.attn_extend(s["q"], s["kp"], s["vp"], s["table"], s["cu"], s["kv"], max_seqlen=max(s["new"]))
    if c["op"] == "decode":
        return la.attn_decode(s["q"], s["kp"], s["vp"], s["table"], s["kv"])
    if c["op"] == "tree":
        return la.attn_verify_tree(s["q"], s["kp"], s["vp"], s["table"], s["kv"], s["parents"], c["N"])
    lens = la.kv_commit(s["kp"], s["vp"], s["table"], s["kv"], s["parents"], s["accept"])
    return [lens, s["kp"], s["vp"]]


def _rotate(x, s):
    c = s["case"]
    R = c["rot"]
    x = x.float().reshape(x.shape[0], -1, D)
    angle = (s["pos"].double()[:, None] * s["freq"][None])[:, None]  # far positions: 64 bits
    cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if c["inter"] else (x[..., : R // 2], x[..., R // 2 : R])
    y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1 if c["inter"] else -2).flatten(-2)
    return torch.cat((y, x[..., R:]), -1).flatten(1).bfloat16()


def _plain(s):
    c = s["case"]
    if c["op"] == "rope":
        return [_rotate(s["q"], s), _rotate(s["k"], s)]
    if c["op"] == "store":
        page, row = s["loc"].long() // c["P"], s["loc"].long() % c["P"]
        s["kp"][page, :, row] = _rotate(s["k"], s).reshape(-1, c["Hkv"], D)
        s["vp"][page, :, row] = s["v"].reshape(-1, c["Hkv"], D)
        return [_rotate(s["q"], s), s["kp"], s["vp"]]
    if c["op"] == "extend":
        return _plain_extend(s)
    if c["op"] == "commit":
        return _plain_commit(s)
    B, N, Hkv = c["B"], c.get("N", 1), c["Hkv"]
    G = c["H"] // Hkv
    k, v = (p[s["table"].long()].transpose(1, 2).flatten(2, 3) for p in (s["kp"], s["vp"]))  # [B, Hkv, keys, D]
    q = s["q"].float().reshape(B, N, Hkv, G, D).transpose(1, 2).flatten(2, 3)
    at, kv = torch.arange(k.shape[2], device=DEV), s["kv"].long()[:, None, None]
    seen = (at < kv - N).expand(B, N, -1)
    draft = at - (kv - N)  # number of the draft at a key
    if c["op"] == "tree":
        up = _ancestors(s["parents"])
        seen = seen | ((draft >= 0) & (draft < N) & up.gather(2, draft.clamp(0, N - 1).expand(B, N, -1)))
    else:
        seen = seen | (draft == 0)
    w = q @ k.float().transpose(-1, -2) * SCALE
    w = torch.where(seen.repeat_interleave(G, 1)[:, None], w, -math.inf)
    w = (w - w.amax(-1, keepdim=True)).exp()
    o = (w @ v.float()) / w.sum(-1, keepdim=True)
    return o.reshape(B, Hkv, N, G, D).transpose(1, 2).reshape(B * N, -1).bfloat16()


def _ancestors(parents):
    """[B, N, N]: whether draft j is draft t or one of its ancestors."""
    N = parents.shape[1]
    step = torch.nn.functional.one_hot(parents.long() + 1, N + 1)[..., 1:].float()
    up = step + torch.eye(N, device=DEV)
    for _ in range(max(1, N.bit_length())):
        up = (up @ up).clamp(max=1)
    return up > 0


def _plain_extend(s):
    c = s["case"]
    Hkv, H = c["Hkv"], c["H"]
    G, outs = H // Hkv, []
    q = s["q"].reshape(-1, Hkv, G, D)
    first = 0
    for b, (n, total) in enumerate(zip(s["new"], s["total"])):
        k, v = (p[s["table"][b].long()].transpose(0, 1).flatten(1, 2)[:, :total].float() for p in (s["kp"], s["vp"]))
        step = max(1, (1 << 29) // max(1, H * total))
        for i in range(0, n, step):
            m = min(step, n - i)
            end = total - n + i + m  # the block's last query sees the keys before this one
            x = q[first + i : first + i + m].float().permute(1, 2, 0, 3).flatten(1, 2)
            w = (x @ k[:, :end].transpose(-1, -2) * SCALE).view(Hkv, G, m, end)
            hidden = torch.ones(m, end, dtype=torch.bool, device=DEV).triu(end - m + 1)
            w = w.masked_fill_(hidden, -math.inf)
            w = w.sub_(w.amax(-1, keepdim=True)).exp_().flatten(1, 2)
            o = (w @ v[:, :end]) / w.sum(-1, keepdim=True)
            outs.append(o.view(Hkv, G, m, D).permute(2, 0, 1, 3).reshape(m, H * D).bfloat16())
        first += n
    return torch.cat(outs) if outs else torch.empty_like(s["q"])


def _plain_commit(s):
    c = s["case"]
    N, P = c["N"], c["P"]
    up = _ancestors(s["parents"])
    on = up.gather(1, s["accept"].clamp(min=0).long()[:, None, None].expand(-1, 1, N))[:, 0]
    on = on & (s["accept"] >= 0)[:, None]  # the drafts of the accepted path
    count = on.sum(1)
    # a path's drafts in order, then row i onto itself
    order = torch.argsort((~on).int(), dim=1, stable=True)
    at = torch.arange(N, device=DEV)[None]
    order = torch.where(at < count[:, None], order, at)
    start = (s["kv"].long() - N)[:, None]
    src, dst = start + order, start + at
    table = s["table"].long()
    sp, dp = table.gather(1, src // P), table.gather(1, dst // P)
    for p in (s["kp"], s["vp"]):
        p[dp, :, dst % P] = p[sp, :, src % P]
    return [(start[:, 0] + count).int(), s["kp"], s["vp"]]


def exact(case, seed):
    """The definitions in 64 bits, request by request and head by head."""
    s = prepare(case, seed)
    op, Hkv = case["op"], case["Hkv"]
    if op in ("rope", "store"):
        R = case["rot"]
        turn = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device=DEV).expand(case["T"], R // 2),
                           torch.outer(s["pos"].double(), s["freq"]))

        def spin(x):
            y = x.double().unflatten(1, (-1, D)).clone()
            a, b = (slice(0, R, 2), slice(1, R, 2)) if case["inter"] else (slice(0, R // 2), slice(R // 2, R))
            z = torch.complex(y[..., a], y[..., b]) * turn[:, None]
            y[..., a], y[..., b] = z.real.clone(), z.imag.clone()
            return y

        q, k = spin(s["q"]), spin(s["k"])
        if op == "rope":
            return [q.flatten(1), k.flatten(1)]
        kp, vp = (p.double().transpose(1, 2).flatten(0, 1) for p in (s["kp"], s["vp"]))
        kp[s["loc"].long()], vp[s["loc"].long()] = k, s["v"].double().unflatten(1, (Hkv, D))
        return [q.flatten(1)] + [p.unflatten(0, (-1, case["P"])).transpose(1, 2).contiguous() for p in (kp, vp)]
    new, old = _lens(case)
    P, B = case["P"], case["B"]
    table = s["table"].tolist()

    def places(b, lo, hi):
        j = range(lo, hi)
        return (torch.tensor([table[b][x // P] for x in j], dtype=torch.long, device=DEV),
                torch.tensor([x % P for x in j], dtype=torch.long, device=DEV))

    if op == "commit":
        kp, vp, lens = s["kp"].double(), s["vp"].double(), []
        for b, (a, tree) in enumerate(zip(_accepts(case)[0], _trees(case))):
            path = []
            while a >= 0:
                path.insert(0, a)
                a = tree[a]
            pg, row = places(b, old[b], old[b] + case["N"])
            for p in (kp, vp):
                p[pg[: len(path)], :, row[: len(path)]] = p[pg[path], :, row[path]]
            lens.append(old[b] + len(path))
        return [torch.tensor(lens, dtype=torch.int32, device=DEV), kp, vp]
    H = case["H"]
    G = H // Hkv
    out = torch.zeros(sum(new), H, D, dtype=torch.float64, device=DEV)
    trees = _trees(case) if op == "tree" else None
    first = 0
    for b, (n, m) in enumerate(zip(new, old)):
        if n == 0:
            continue
        pg, row = places(b, 0, n + m)
        sees = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        if trees:
            rows = []
            for t, up in enumerate(trees[b]):
                rows.append([x == t or (up >= 0 and rows[up][x]) for x in range(n)])
            sees = torch.tensor(rows, device=DEV)
        for h in range(Hkv):
            k, v = s["kp"][pg, h, row].double(), s["vp"][pg, h, row].double()
            x = s["q"][first : first + n].unflatten(1, (H, D))[:, h * G : (h + 1) * G].double()
            for i in range(0, n, 1024):
                e = min(n, i + 1024)
                z = torch.einsum("tgd,jd->gtj", x[i:e], k) / math.sqrt(D)
                z[:, :, m:] = z[:, :, m:].masked_fill(~sees[i:e], -math.inf)
                out[first + i : first + e, h * G : (h + 1) * G] = torch.einsum("gtj,jd->tgd", z.softmax(-1), v)
        first += n
    return out.flatten(1)
