"""What the operators around the folded MLA decode are measured on: the listed
cases, further ones drawn from the same ranges, the operators' plain forms and
their exact values.

* ``append``: the new tokens of every request enter the paged FP8 latent cache:
  RMS norm of the 512 latent dims, rotation of the 64 rope dims at the token's
  position, E4M3 codes written through the block table.
* ``absorb``: the query side of the same step: the 128 nope dims of every
  (token, head) times that head's W_UK, the 64 rope dims rotated, E4M3 codes in
  the [R*k, H, 576] layout that the decode reads.
* ``prefix``: the decode of a batch whose requests all begin with one shared
  prefix: its keys are read once for all requests, each request's own keys
  follow, one softmax over both.
"""
import math

import torch

own = False

PAGE, LATENT, ROPE, NOPE = 64, 512, 64, 128
DQK = LATENT + ROPE
E4M3_MAX = 448.0
SM_SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
LOG2E = 1.4426950408889634


# ---------------------------------------------------------------- cases
def listed():
    return [
        # The smallest decode batch (two requests, four draft tokens): launch latency.
        dict(name="append R2 k4", op="append", R=2, k=4, lo=37, hi=100, ahead=0, rows=0,
             stride=576, norm=True, interleaved=True),
        # A full decode step of 128 requests with seven draft tokens behind a shared prefix of
        # 64k tokens (positions go on from there); the rows come out of a wider fused projection,
        # so they are strided.
        dict(name="append R128 k7", op="append", R=128, k=7, lo=0, hi=128, ahead=65536, rows=0,
             stride=2112, norm=True, interleaved=True),
        # Prompts of 24 requests in one ragged batch, padded rows at its end, half-split rotation.
        dict(name="append prompts 24", op="append", R=24, k=0, lo=0, hi=8192, ahead=0, rows=64,
             stride=576, norm=True, interleaved=False),
        # Queries of the smallest batch.
        dict(name="absorb R2 k4 H8", op="absorb", R=2, k=4, H=8, hi=128, stride=192,
             interleaved=True),
        # One tensor-parallel rank's eight heads, 64 requests.
        dict(name="absorb R64 k7 H8", op="absorb", R=64, k=7, H=8, hi=32768, stride=192,
             interleaved=True),
        # All 64 heads of a few requests: the weights are most of the bytes.
        dict(name="absorb R16 k4 H64", op="absorb", R=16, k=4, H=64, hi=65536, stride=192,
             interleaved=False),
        # All 64 heads of the large batch.
        dict(name="absorb R128 k7 H64", op="absorb", R=128, k=7, H=64, hi=131072, stride=256,
             interleaved=True),
        # Two requests behind a short system prompt: latency.
        dict(name="prefix R2 k4 H8 300", op="prefix", R=2, k=4, H=8, prefix=300, lo=37, hi=100,
             std=1.0),
        # 32 chats behind one long system prompt.
        dict(name="prefix R32 k4 H8 4k", op="prefix", R=32, k=4, H=8, prefix=4096, lo=0, hi=2048,
             std=0.5),
        # 64 requests on one shared document, its last page partly filled.
        dict(name="prefix R64 k7 H8 16k", op="prefix", R=64, k=7, H=8, prefix=16330, lo=256,
             hi=4096, std=1.0),
        # All 64 heads, plain decode of one token per request behind a shared document.
        dict(name="prefix R24 k1 H64 64k", op="prefix", R=24, k=1, H=64, prefix=65536, lo=1,
             hi=700, std=1.0),
        # All 64 heads, seven draft tokens, a large batch.
        dict(name="prefix R128 k7 H64 16k", op="prefix", R=128, k=7, H=64, prefix=16384, lo=512,
             hi=4096, std=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "absorb", "prefix", "prefix"])
    inter = rng.random() < 0.5
    if op == "append":
        c = dict(op=op, ahead=rng.choice([0, _log(rng, 1, 131072)]),
                 stride=rng.choice([576, 584, 1000, 2112]), norm=rng.random() < 0.8,
                 interleaved=inter)
        if rng.random() < 0.5:
            return dict(c, R=_log(rng, 1, 256), k=rng.randint(1, 8), lo=rng.choice([0, 1, 60]),
                        hi=_log(rng, 64, 1024), rows=0)
        return dict(c, R=_log(rng, 1, 24), k=0, lo=rng.choice([0, 1, 7]), hi=_log(rng, 16, 8192),
                    rows=rng.randint(0, 100))
    if op == "absorb":
        return dict(op=op, R=_log(rng, 1, 128), k=rng.randint(1, 7),
                    H=rng.choice([1, 3, 8, 12, 16, 20, 32, 64]), hi=_log(rng, 64, 131072),
                    stride=rng.choice([192, 200, 256]), interleaved=inter)
    while True:
        c = dict(op=op, R=_log(rng, 1, 128), k=rng.randint(1, 7),
                 H=rng.choice([1, 3, 8, 12, 16, 20, 32, 64]), prefix=_log(rng, 1, 131072),
                 lo=rng.choice([0, 1, 30]), hi=_log(rng, 32, 16384),
                 std=rng.choice([0.5, 0.7, 1.0]))
        if 2048 < c["prefix"] and rng.random() < 0.5:
            c["prefix"] -= c["prefix"] % PAGE
        if c["R"] * c["k"] * c["H"] * (c["prefix"] + c["hi"]) <= 9e8 and c["R"] * c["hi"] <= 524288:
            return c


# ---------------------------------------------------------------- inputs
def _lengths(case, g):
    return torch.randint(case["lo"], case["hi"] + 1, (case["R"],), generator=g)


def _tables(pages, total, g):
    """Block table [R, widest] of requests of `pages` pages each: one random permutation of all
    `total` pages handed out in order; and the pages left over."""
    R, width = len(pages), max(1, int(pages.max()))
    perm = torch.randperm(total, generator=g)
    slot = torch.arange(width)[None, :] < pages[:, None]
    table = torch.zeros((R, width), dtype=torch.int32)
    table[slot] = perm[:int(pages.sum())].to(torch.int32)
    return table, perm[int(pages.sum()):].to(torch.int32)


def _rope_table(rows):
    """cos and sin of position * 10000^(-2 i / 64), [rows, 32 cos + 32 sin] FP32; angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _codes(x):
    """Values -> E4M3 codes (as uint8) under the per-tensor scale amax / 448, and that scale."""
    scale = float(x.abs().max()) / E4M3_MAX
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed + 1)
    dev = "cuda"
    R = case["R"]
    rand = lambda *s: torch.randn(s, generator=gd, device=dev)  # noqa: E731
    s = dict(case=case)
    if case["op"] == "append":
        if case["k"]:
            starts, new = _lengths(case, g), torch.full((R,), case["k"])
            s["cu"] = None
        else:                                     # prompts: ragged, a few of them continued
            new = _lengths(case, g)
            starts = torch.where(torch.rand(R, generator=g) < 0.7, 0,
                                 torch.randint(0, 300, (R,), generator=g))
            s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).int().to(dev)
        T = int(new.sum()) + case["rows"]
        # A cache of a fixed size for the case, whatever lengths the seed draws.
        pages = R * ((case["hi"] + (case["k"] or 300)) // PAGE + 1)
        table, _ = _tables((starts + new + PAGE - 1) // PAGE, pages, g)
        # Latents of very different sizes from token to token, as projections give them.
        wide = rand(max(T, 1), case["stride"]).mul_(torch.exp(0.7 * rand(max(T, 1), 1)))
        s["new"] = wide.to(torch.bfloat16)[:T, :DQK]
        s["weight"] = (1 + 0.1 * rand(LATENT)).to(torch.bfloat16) if case["norm"] else None
        s["scale"] = (6.0 if case["norm"] else 12.0) / E4M3_MAX
        s["kv"] = (rand(pages, PAGE, DQK) * 70).clamp(-E4M3_MAX, E4M3_MAX).to(
            torch.float8_e4m3fn).view(torch.uint8)
        s["table"], s["starts"] = table.to(dev), starts.int().to(dev)
        s["turns"] = (s["starts"] + case["ahead"]) if case["ahead"] else None
        s["rope"] = _rope_table(case["ahead"] + int((starts + new).max()) + 1)
    elif case["op"] == "absorb":
        k, H, st = case["k"], case["H"], case["stride"]
        s["q"] = rand(R * k, H, st).to(torch.bfloat16)[:, :, :NOPE + ROPE]
        s["w"] = (rand(H, NOPE, LATENT) / math.sqrt(NOPE)).to(torch.bfloat16)
        s["starts"] = torch.randint(0, case["hi"], (R,), generator=g).int().to(dev)
        s["rope"] = _rope_table(case["hi"] + k)
        s["scale"] = 6.0 / E4M3_MAX
    else:
        k, H, P = case["k"], case["H"], case["prefix"]
        lens = _lengths(case, g)
        pp = (P + PAGE - 1) // PAGE
        pages = int(((lens + PAGE - 1) // PAGE).sum()) + pp + 2
        table, rest = _tables((lens + PAGE - 1) // PAGE, pages, g)
        s["prefix_table"] = rest[:pp].contiguous().to(dev)
        s["prefix_len"] = torch.tensor([P], dtype=torch.int32, device=dev)
        s["table"], s["lens"] = table.to(dev), lens.int().to(dev)
        s["q"], qs = _codes(rand(R * k, H, DQK) * case["std"])
        s["kv"], s["bmm2"] = _codes(rand(pages, PAGE, DQK) * case["std"])
        s["bmm1"] = SM_SCALE * qs * s["bmm2"]
        s["most"] = int(lens.max())
        if own:
            import mla_decode_attention_folded_gb300 as mla
            s["engine"] = mla.PrefixMla(R, k, H, table.shape[1], pp, pages, dev)
    return s


# ---------------------------------------------------------------- plain forms
def _rotate(x, cs, interleaved):
    """x [..., 64] rotated by the angles whose cos | sin are cs [..., 64]."""
    c, n = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    u, v = a * c - b * n, b * c + a * n
    return torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)


def _tokens(s, T):
    """(request, index among its new tokens, whether it belongs to any) of every new row."""
    t = torch.arange(T, device="cuda")
    if s["cu"] is None:
        k = s["case"]["k"]
        return t // k, t % k, torch.ones_like(t, dtype=torch.bool)
    cu = s["cu"].long()
    r = (t[:, None] >= cu[None, 1:]).sum(1)
    live = t < cu[-1]
    r = r.clamp(max=s["case"]["R"] - 1)
    return r, t - cu[r], live


def _plain_append(s):
    x, kv = s["new"].float(), s["kv"]
    r, i, live = _tokens(s, x.shape[0])
    pos = s["starts"].long()[r] + i
    lat = x[:, :LATENT]
    if s["weight"] is not None:
        lat = lat * torch.rsqrt((lat * lat).mean(1, keepdim=True) + EPS) * s["weight"].float()
    pos = torch.where(live, pos, 0)
    pe = _rotate(x[:, LATENT:], s["rope"][pos + s["case"]["ahead"]], s["case"]["interleaved"])
    y = (torch.cat([lat, pe], 1) / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX)
    row = s["table"].long()[r, pos // PAGE] * PAGE + pos % PAGE
    kv.view(-1, DQK)[row[live]] = y[live].to(torch.float8_e4m3fn).view(torch.uint8)
    return kv.view(torch.float8_e4m3fn)


def _plain_absorb(s):
    c, q = s["case"], s["q"].float()
    lat = torch.einsum("thd,hdl->thl", q[..., :NOPE], s["w"].float())
    pos = (s["starts"].long()[:, None] + torch.arange(c["k"], device="cuda")).flatten()
    pe = _rotate(q[..., NOPE:], s["rope"][pos][:, None], c["interleaved"])
    y = torch.cat([lat, pe], -1) / s["scale"]
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_prefix(s):
    c = s["case"]
    R, M, P = c["R"], c["k"] * c["H"], c["prefix"]
    val = lambda codes: codes.view(torch.float8_e4m3fn).float()  # noqa: E731
    q = val(s["q"]).view(R, M, DQK) * (s["bmm1"] * LOG2E)
    shared = val(s["kv"][s["prefix_table"].long()]).view(-1, DQK)[:P]
    mine = val(s["kv"][s["table"].long()]).view(R, -1, DQK)[:, :max(1, s["most"])]
    a = (q.view(R * M, DQK) @ shared.T).view(R, M, P)
    b = q @ mine.transpose(1, 2)
    seen = torch.arange(mine.shape[1], device="cuda") < s["lens"][:, None]
    b = torch.where(seen[:, None], b, -math.inf)
    top = torch.maximum(a.amax(-1), b.amax(-1))[..., None]
    a, b = torch.exp2(a - top), torch.exp2(b - top)
    z = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    o = (a.view(R * M, P) @ shared[:, :LATENT]).view(R, M, LATENT) + b @ mine[..., :LATENT]
    out = (o / z * s["bmm2"]).to(torch.bfloat16)
    return out, (top + torch.log2(z))[..., 0]


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "absorb": _plain_absorb, "prefix": _plain_prefix}[op](s)
    import mla_decode_attention_folded_gb300 as mla
    inter = s["case"].get("interleaved")
    if op == "append":
        mla.kv_append(s["new"], s["kv"], s["table"], s["starts"], s["rope"], s["scale"],
                      norm_weight=s["weight"], norm_eps=EPS, cu_tokens=s["cu"], rope_starts=s["turns"],
                      interleaved=inter)
        return s["kv"].view(torch.float8_e4m3fn)
    if op == "absorb":
        return mla.query_absorb(s["q"], s["w"], s["rope"], s["starts"], s["scale"],
                                interleaved=inter).view(torch.float8_e4m3fn)
    eng = s["engine"]
    eng.plan(s["lens"])
    return eng.decode(s["q"], s["kv"], s["prefix_table"], s["prefix_len"], s["table"], s["lens"],
                      s["bmm1"], s["bmm2"])


# ---------------------------------------------------------------- work
def _drawn_lengths(case):
    """The mean total of the case's drawn lengths."""
    return case["R"] * (case["lo"] + case["hi"]) / 2


def work(case):
    R, k = case["R"], case["k"]
    if case["op"] == "append":
        T = R * k if k else _drawn_lengths(case)
        # Each new row, its angles and its codes; the norm's square, sum and two products, the
        # scale, the rotation.
        return dict(bytes=T * (DQK * 2 + ROPE * 4 + DQK) + LATENT * 2, flops=T * (LATENT * 5 + ROPE * 4))
    H = case["H"]
    N = R * k * H
    if case["op"] == "absorb":
        return dict(bytes=N * ((NOPE + ROPE) * 2 + DQK) + H * NOPE * LATENT * 2 + R * k * ROPE * 4,
                    flops=N * (2 * NOPE * LATENT + ROPE * 4))
    keys = _drawn_lengths(case)
    return dict(bytes=N * (DQK + LATENT * 2 + 4) + (case["prefix"] + keys) * DQK,
                flops=2 * (DQK + LATENT) * (N * case["prefix"] + k * H * keys))


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    """64-bit values, token by token and request by request, from the definitions."""
    if case["op"] == "prefix" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    f64 = torch.float64

    def angles(pos):
        inv = 10000.0 ** (-2.0 * torch.arange(32, dtype=f64, device="cuda") / 64.0)
        return pos.to(f64)[:, None] * inv

    def turned(pe, pos):                      # [n, ..., 64], complex numbers of 32 planes
        if case["interleaved"]:
            z = torch.view_as_complex(pe.unflatten(-1, (32, 2)).contiguous())
        else:
            z = torch.complex(pe[..., :32].contiguous(), pe[..., 32:].contiguous())
        th = angles(pos)
        w = torch.polar(torch.ones_like(th), th)
        z = z * w.view(w.shape[0], *([1] * (z.dim() - 2)), 32)
        flat = torch.view_as_real(z)
        return flat.flatten(-2) if case["interleaved"] else torch.cat([flat[..., 0], flat[..., 1]], -1)

    limit = lambda y: (y / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX)  # noqa: E731
    if case["op"] == "append":
        cache = s["kv"].view(torch.float8_e4m3fn).to(f64)
        if s["cu"] is None:
            cuts = [case["k"] * i for i in range(case["R"] + 1)]
        else:
            cuts = s["cu"].tolist()
        for r, first in enumerate(s["starts"].tolist()):
            x = s["new"][cuts[r]:cuts[r + 1]].to(f64)
            if not len(x):
                continue
            pos = first + torch.arange(len(x), device="cuda")
            lat = x[:, :LATENT]
            if s["weight"] is not None:
                lat = lat / ((lat ** 2).sum(1, keepdim=True) / LATENT + EPS).sqrt() * s["weight"].to(f64)
            y = limit(torch.cat([lat, turned(x[:, LATENT:], pos + case["ahead"])], 1))
            cache[s["table"][r].long()[pos // PAGE], pos % PAGE] = y
        return cache
    if case["op"] == "absorb":
        q, k = s["q"].to(f64), case["k"]
        pos = s["starts"].long().repeat_interleave(k) + torch.arange(k, device="cuda").repeat(case["R"])
        lat = torch.stack([q[:, h, :NOPE] @ s["w"][h].to(f64) for h in range(case["H"])], 1)
        return limit(torch.cat([lat, turned(q[..., NOPE:], pos)], -1))
    M = case["k"] * case["H"]
    code = lambda c: c.view(torch.float8_e4m3fn).to(f64)  # noqa: E731
    out, lse = [], []
    shared = code(s["kv"][s["prefix_table"].long()]).reshape(-1, DQK)[:case["prefix"]]
    for r, n in enumerate(s["lens"].tolist()):
        keys = code(s["kv"][s["table"][r].long()]).reshape(-1, DQK)[:n]
        keys = torch.cat([shared, keys])
        sc = code(s["q"]).view(case["R"], M, DQK)[r] @ keys.T * s["bmm1"]
        out.append(torch.softmax(sc, -1) @ keys[:, :LATENT] * s["bmm2"])
        lse.append(torch.logsumexp(sc, -1) * LOG2E)
    return torch.stack(out), torch.stack(lse)
