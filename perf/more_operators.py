"""What the operators that begin and bound a cache are measured on: the listed
cases, further ones drawn from the same ranges, the operators' plain forms and
their exact values.

* ``prompt``: attention over whole prompts of different lengths, packed: per
  (token, head) 128 nope and 64 rope dims against keys whose rope dims all heads
  share, values of 128 dims; causal or not, with cached keys before the new ones.
* ``weigh``: after a decode of the paged FP8 latent cache, the attention weight
  that each cached key got from the step's query rows, added to what it had.
* ``evict``: of every request's keys the first, the newest and those of most
  weight stay, so many in all; the cache's rows move together.
"""
import math

import torch

own = False

PAGE, LATENT, ROPE, NOPE, DV = 64, 512, 64, 128, 128
DQK = LATENT + ROPE
DP = NOPE + ROPE
E4M3_MAX = 448.0
SM_SCALE = 1.0 / math.sqrt(192.0)
LOG2E = 1.4426950408889634


# ---------------------------------------------------------------- cases
def listed():
    return [
        # The smallest batch's two prompts: launch latency.
        dict(name="prompt R2 H8", op="prompt", R=2, H=8, Hkv=8, lo=37, hi=100, ctx=0, causal=True,
             fused=True),
        # One tensor-parallel rank's eight heads, 24 prompts of very different lengths.
        dict(name="prompt R24 H8 2k", op="prompt", R=24, H=8, Hkv=8, lo=0, hi=2048, ctx=0,
             causal=True, fused=True),
        # A chunk of a long prompt: few queries, many cached keys.
        dict(name="prompt chunk 512 on 16k H8", op="prompt", R=1, H=8, Hkv=8, lo=512, hi=512,
             ctx=15871, causal=True, fused=True),
        # A non-causal drafter over its whole context, with grouped heads and separate K and V.
        dict(name="prompt R4 H32 grouped full", op="prompt", R=4, H=32, Hkv=4, lo=900, hi=1500,
             ctx=0, causal=False, fused=False),
        # All 64 heads of one long prompt.
        dict(name="prompt 8k H64", op="prompt", R=1, H=64, Hkv=64, lo=8192, hi=8192, ctx=0,
             causal=True, fused=True),
        # Weights after a step of the smallest decode batch: latency.
        dict(name="weigh R2 k4 H8", op="weigh", R=2, k=4, H=8, lo=37, hi=100, std=1.0),
        # One rank's eight heads, 64 requests with seven draft tokens: the cache's bytes.
        dict(name="weigh R64 k7 H8", op="weigh", R=64, k=7, H=8, lo=256, hi=8192, std=1.0),
        # All 64 heads of a few long requests.
        dict(name="weigh R16 k4 H64", op="weigh", R=16, k=4, H=64, lo=16384, hi=65536, std=0.7),
        # All 64 heads, seven draft tokens, a large batch.
        dict(name="weigh R128 k7 H64", op="weigh", R=128, k=7, H=64, lo=512, hi=4096, std=0.5),
        # Every step of a bounded cache: 128 requests drop the seven keys that they got too many.
        dict(name="evict R128 step of 7", op="evict", R=128, lo=2055, hi=2055, keep=2048, recent=64,
             sinks=4, mixed=True),
        # Prompts cut down to an eighth once they are read.
        dict(name="evict R8 32k to 4k", op="evict", R=8, lo=20000, hi=32768, keep=4096, recent=512,
             sinks=4, mixed=False),
        # One very long request halved.
        dict(name="evict R1 128k to 64k", op="evict", R=1, lo=131072, hi=131072, keep=65536,
             recent=1000, sinks=16, mixed=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "weigh", "evict"])
    if op == "prompt":
        while True:
            Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32, 64])
            c = dict(op=op, R=_log(rng, 1, 40), H=Hkv * rng.choice([1, 1, 1, 2, 4, 5]), Hkv=Hkv,
                     hi=_log(rng, 1, 8192), ctx=rng.choice([0, 0, _log(rng, 1, 32768)]),
                     causal=rng.random() < 0.75, fused=rng.random() < 0.6)
            c["lo"] = rng.choice([0, 1, c["hi"] // 2, c["hi"]])
            if c["R"] * c["H"] * c["hi"] * (c["hi"] + c["ctx"]) <= 2.5e9 and c["H"] <= 64 and \
                    c["R"] * (c["hi"] + c["ctx"]) * c["H"] <= 4e6:
                return c
    if op == "weigh":
        while True:
            c = dict(op=op, R=_log(rng, 1, 128), k=rng.randint(1, 7),
                     H=rng.choice([1, 3, 8, 12, 16, 20, 32, 64]), hi=_log(rng, 16, 65536),
                     std=rng.choice([0.5, 0.7, 1.0]))
            c["lo"] = rng.choice([0, 1, c["hi"] // 3])
            if c["R"] * c["k"] * c["H"] * c["hi"] <= 2.6e8 and c["R"] * c["hi"] <= 1.04e6:
                return c
    while True:
        c = dict(op=op, R=_log(rng, 1, 128), hi=_log(rng, 8, 131072), mixed=rng.random() < 0.5,
                 recent=rng.choice([0, 1, 32, 333]), sinks=rng.choice([0, 1, 4, 100]))
        c["lo"] = rng.choice([0, c["hi"] // 2, c["hi"]])
        c["keep"] = max(1, int(c["hi"] * rng.choice([0.1, 0.3, 0.5, 0.9, 0.995])))
        if c["R"] * c["hi"] <= 2.6e5:
            return c


# ---------------------------------------------------------------- inputs
def _sizes(case):
    """The case's lengths: even from the longest down to the shortest."""
    lo, hi, R = case["lo"], case["hi"], case["R"]
    return [hi - (hi - lo) * i // max(1, R - 1) for i in range(R)]


def _lengths(case, g):
    """The lengths in the seed's order: totals do not go by the seed."""
    return torch.tensor(_sizes(case))[torch.randperm(case["R"], generator=g)]


def _cu(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).int().cuda()


def _tables(lens, g, spare=2):
    """Block table [R, widest] of requests of so many keys: one random permutation of all pages
    handed out in order; and the number of pages, which goes by the widest request alone."""
    pages = (lens + PAGE - 1) // PAGE
    R, width = len(pages), max(1, int(pages.max()))
    total = R * width + spare
    perm = torch.randperm(total, generator=g)
    slot = torch.arange(width)[None, :] < pages[:, None]
    table = torch.zeros((R, width), dtype=torch.int32)
    table[slot] = perm[:int(pages.sum())].to(torch.int32)
    return table.cuda(), total


def _codes(x):
    """Values -> E4M3 codes (as uint8) under the per-tensor scale amax / 448, and that scale."""
    scale = float(x.abs().max()) / E4M3_MAX
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed + 1)
    rand = lambda *s: torch.randn(s, generator=gd, device="cuda")  # noqa: E731
    R = case["R"]
    lens = _lengths(case, g)
    s = dict(case=case, most=int(lens.max()))
    if case["op"] == "prompt":
        H, Hkv = case["H"], case["Hkv"]
        T = int(lens.sum())
        s["cu"] = _cu(lens)
        s["cu_keys"] = _cu(lens + case["ctx"]) if case["ctx"] else None
        Tk = T + R * case["ctx"]
        # Rotated rope dims and projected nope dims, as the projections before the attention give
        # them; queries twice as large, so that some keys stand out.
        s["q"] = rand(T, H, DP).mul_(2.0).to(torch.bfloat16)
        s["k_rope"] = rand(Tk, ROPE).to(torch.bfloat16)
        if case["fused"]:                   # one projection's output: nope and value side by side
            kv = rand(Tk, Hkv, NOPE + DV).to(torch.bfloat16)
            s["k_nope"], s["v"] = kv[..., :NOPE], kv[..., NOPE:]
        else:
            s["k_nope"] = rand(Tk, Hkv, NOPE).to(torch.bfloat16)
            s["v"] = rand(Tk, Hkv, DV).to(torch.bfloat16)
    elif case["op"] == "weigh":
        k, H = case["k"], case["H"]
        s["table"], pages = _tables(lens, g)
        s["lens"] = lens.int().cuda()
        # k of the keys are the step's own and carry no weight yet.
        s["starts"] = (lens - k).clamp(min=0).int().cuda()
        s["turns"] = s["starts"] + 5000
        s["q"], qs = _codes(rand(R * k, H, DQK) * case["std"])
        s["kv"], kvs = _codes(rand(pages, PAGE, DQK) * case["std"])
        s["bmm1"] = SM_SCALE * qs * kvs
        x, seen = _scores(s)
        s["lse"] = (torch.logsumexp(torch.where(seen[:, None], x, -math.inf) * math.log(2.0), -1)
                    * LOG2E).contiguous()
        S = s["table"].shape[1] * PAGE
        # As some steps before gave it: rows times steps over keys, more to some than to others.
        s["weights"] = torch.exp(rand(R, S)) * (3.0 * k * H / max(1, s["most"]))
        s["positions"] = torch.full((R, S), -1, dtype=torch.int32, device="cuda")
    else:
        s["table"], pages = _tables(lens, g)
        s["lens"] = lens.int().cuda()
        S = s["table"].shape[1] * PAGE
        # Summed attention weights: a few keys hold most, some hold none at all.
        w = torch.exp(2.0 * rand(R, S))
        s["weights"] = torch.where(torch.rand((R, S), generator=gd, device="cuda") < 0.1, 0.0, w)
        p = torch.arange(S, device="cuda").expand(R, S)
        if case["mixed"]:                   # a cache that has dropped keys before
            top = torch.where(p < s["lens"][:, None], torch.rand((R, S), generator=gd, device="cuda"),
                              2.0)
            p = top.argsort(1).argsort(1)
        s["positions"] = p.int().contiguous()
        s["keep"] = torch.full((R,), case["keep"], dtype=torch.int32, device="cuda")
        s["kv"] = (rand(pages, PAGE, DQK) * 70).clamp(-E4M3_MAX, E4M3_MAX).to(
            torch.float8_e4m3fn).view(torch.uint8)
        s["new_weights"] = torch.zeros_like(s["weights"])
        s["new_positions"] = torch.full_like(s["positions"], -1)
    return s


# ---------------------------------------------------------------- plain forms
def _rows(cu, most, R):
    """Row of token i of every request [R, most], and whether there is one."""
    cu = cu.long()
    i = torch.arange(most, device="cuda")
    return cu[:R, None] + i, i < (cu[1:] - cu[:-1])[:, None]


def _plain_prompt(s):
    c = s["case"]
    R, H, n, m = c["R"], c["H"], s["most"], s["most"] + c["ctx"]
    rows, live = _rows(s["cu"], n, R)
    keys, there = _rows(s["cu"] if s["cu_keys"] is None else s["cu_keys"], m, R)
    G = H // c["Hkv"]
    at, of = rows.clamp(max=len(s["q"]) - 1), keys.clamp(max=len(s["v"]) - 1)
    q = (s["q"][at].float() * (SM_SCALE * LOG2E)).transpose(1, 2)                # [R, H, n, 192]
    k = s["k_nope"][of].float().repeat_interleave(G, 2).transpose(1, 2)          # [R, H, m, 128]
    v = s["v"][of].float().repeat_interleave(G, 2).transpose(1, 2)
    x = q[..., :NOPE] @ k.transpose(2, 3)
    x += q[..., NOPE:] @ s["k_rope"][of].float()[:, None].transpose(2, 3)
    seen = there[:, None, :].expand(R, n, m)
    if c["causal"]:
        last = torch.arange(n, device="cuda")[None] + (there.sum(1) - live.sum(1))[:, None]
        seen = seen & (torch.arange(m, device="cuda") <= last[..., None])
    x = x.masked_fill_(~seen[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(base).exp2_()
    z = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(z == 0, 1.0, z)
    lse = (base + torch.log2(z))[..., 0]
    return o.transpose(1, 2)[live].to(torch.bfloat16), lse.transpose(1, 2)[live]


def _scores(s):
    """Base-2 scores [R, k H, keys] of every row against its request's cached keys, and which keys
    there are."""
    c = s["case"]
    val = lambda codes: codes.view(torch.float8_e4m3fn).float()  # noqa: E731
    q = val(s["q"]).view(c["R"], c["k"] * c["H"], DQK) * (s["bmm1"] * LOG2E)
    keys = val(s["kv"][s["table"].long()]).view(c["R"], -1, DQK)
    return q @ keys.transpose(1, 2), torch.arange(keys.shape[1], device="cuda") < s["lens"][:, None]


DECAY = 0.875


def _plain_weigh(s):
    x, seen = _scores(s)
    got = torch.exp2(x - s["lse"][..., None]).sum(1)
    slot = torch.arange(x.shape[2], device="cuda")
    new = slot >= s["starts"][:, None]
    w, p = s["weights"], s["positions"]
    w.copy_(torch.where(seen, torch.where(new, 0.0, w * DECAY) + got, w))
    p.copy_(torch.where(seen & new, s["turns"][:, None] + slot - s["starts"][:, None], p))
    return w, p


def _plain_evict(s):
    c, w, p = s["case"], s["weights"], s["positions"]
    n, keep = s["lens"].long()[:, None], s["keep"].long()[:, None]
    R, S = w.shape
    slot = torch.arange(S, device="cuda").expand(R, S)
    there = slot < n
    end = torch.where(there, p.long(), -1).amax(1, keepdim=True) + 1
    held = (p < c["sinks"]) | (p >= end - c["recent"])
    v = torch.where(there, torch.where(held, math.inf, w), -math.inf)
    rank = v.argsort(dim=1, descending=True, stable=True).argsort(dim=1)
    kept = (rank < keep) & there
    hole, mover = ~kept & (slot < keep) & there, kept & (slot >= keep)
    # The i-th mover goes to the i-th hole.
    order = torch.where(hole, slot, S).sort(1).values
    to = order.gather(1, (mover.cumsum(1) - 1).clamp(min=0))
    r, a = mover.nonzero(as_tuple=True)
    b = to[r, a]
    table, rows = s["table"].long(), s["kv"].view(-1, DQK)
    rows[table[r, b // PAGE] * PAGE + b % PAGE] = rows[table[r, a // PAGE] * PAGE + a % PAGE]
    nw, np = s["new_weights"], s["new_positions"]
    nw.copy_(torch.where(there, torch.where(kept & (slot < keep), w, 0.0), nw))
    np.copy_(torch.where(there, torch.where(kept & (slot < keep), p, -1), np))
    nw[r, b], np[r, b] = w[r, a], p[r, a]
    return s["kv"].view(torch.float8_e4m3fn), torch.minimum(n, keep)[:, 0].int(), nw, np


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if not own:
        return {"prompt": _plain_prompt, "weigh": _plain_weigh, "evict": _plain_evict}[c["op"]](s)
    import mla_decode_attention_folded_gb300 as mla
    if c["op"] == "prompt":
        return mla.prompt_attention(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu"], SM_SCALE,
                                    cu_keys=s["cu_keys"], causal=c["causal"])
    if c["op"] == "weigh":
        mla.kv_weigh(s["q"], s["kv"], s["table"], s["lens"], s["lse"], s["bmm1"], s["weights"],
                     s["starts"], decay=DECAY, positions=s["positions"], rope_starts=s["turns"])
        return s["weights"], s["positions"]
    lens = mla.kv_evict(s["kv"], s["table"], s["lens"], s["weights"], s["keep"],
                        positions=s["positions"], recent=c["recent"], sinks=c["sinks"],
                        weights_out=s["new_weights"], positions_out=s["new_positions"])
    return s["kv"].view(torch.float8_e4m3fn), lens, s["new_weights"], s["new_positions"]


# ---------------------------------------------------------------- work
def work(case):
    n = _sizes(case)
    R, T = case["R"], sum(n)
    if case["op"] == "prompt":
        H, Hkv, ctx = case["H"], case["Hkv"], case["ctx"]
        Tk = T + R * ctx
        pairs = sum(x * ctx + (x * (x + 1) // 2 if case["causal"] else x * x) for x in n)
        return dict(bytes=T * H * (DP * 2 + DV * 2 + 4) + Tk * (Hkv * (NOPE + DV) * 2 + ROPE * 2),
                    flops=pairs * H * 2 * (DP + DV))
    if case["op"] == "weigh":
        M = case["k"] * case["H"]
        return dict(bytes=T * (DQK + 8) + R * M * (DQK + 4) + R * case["k"] * 4,
                    flops=T * M * 2 * DQK)
    # Of the kept keys, as many lie behind slot `keep` as chance has it.
    keep = case["keep"]
    moved = sum(keep * (x - keep) / x for x in n if x > keep)
    return dict(bytes=T * 16 + moved * DQK * 2, flops=T * 4)


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    """64-bit values, request by request, from the definitions."""
    s = prepare(case, seed)
    f64 = torch.float64
    R = case["R"]
    if case["op"] == "prompt":
        H, G = case["H"], case["H"] // case["Hkv"]
        cu = s["cu"].tolist()
        ck = cu if s["cu_keys"] is None else s["cu_keys"].tolist()
        out = torch.zeros((cu[-1], H, DV), dtype=f64, device="cuda")
        lse = torch.full((cu[-1], H), -math.inf, dtype=f64, device="cuda")
        for r in range(R):
            a, b, c, d = cu[r], cu[r + 1], ck[r], ck[r + 1]
            for h in range(H if b > a and d > c else 0):
                for i in range(a, b, 2048):
                    e = min(b, i + 2048)
                    kk = torch.cat([s["k_nope"][c:d, h // G], s["k_rope"][c:d]], 1).to(f64)
                    x = s["q"][i:e, h].to(f64) @ kk.T * SM_SCALE
                    if case["causal"]:
                        far = torch.arange(d - c, device="cuda")[None] - (d - c - (b - a)) > \
                            torch.arange(i - a, e - a, device="cuda")[:, None]
                        x[far] = -math.inf
                    lse[i:e, h] = torch.logsumexp(x, 1) * LOG2E
                    out[i:e, h] = torch.softmax(x, 1) @ s["v"][c:d, h // G].to(f64)
        return out, lse
    code = lambda x: x.view(torch.float8_e4m3fn).to(f64)  # noqa: E731
    lens = s["lens"].tolist()
    if case["op"] == "weigh":
        M = case["k"] * case["H"]
        w = s["weights"].to(f64)
        q = code(s["q"]).view(R, M, DQK)
        for r, n in enumerate(lens):
            if n:
                a = int(s["starts"][r])
                keys = code(s["kv"][s["table"][r].long()]).reshape(-1, DQK)[:n]
                x = q[r] @ keys.T * s["bmm1"] * LOG2E - s["lse"][r].to(f64)[:, None]
                w[r, a:n] = 0
                w[r, :a] *= DECAY
                w[r, :n] += torch.exp2(x).sum(0)
        return w, None
    kv, nw = code(s["kv"]), torch.zeros_like(s["weights"], dtype=f64)
    flat = kv.view(-1, DQK)
    for r, n in enumerate(lens):
        keep = case["keep"]
        w, p = s["weights"][r, :n].tolist(), s["positions"][r, :n].tolist()
        end = max(p, default=-1) + 1
        first = sorted(range(n), key=lambda j: (not (p[j] < case["sinks"] or p[j] >= end - case["recent"]),
                                                -w[j], j))
        # Keys held by their position all come first; among them the lower slot wins.
        held = [j for j in range(n) if p[j] < case["sinks"] or p[j] >= end - case["recent"]]
        first = held + first[len(held):]
        kept = set(first[:keep])
        where = {j: j for j in kept if j < keep}
        holes = [j for j in range(min(n, keep)) if j not in kept]
        where.update(zip(sorted(j for j in kept if j >= keep), holes))
        if where:
            a, b = (torch.tensor(list(x), device="cuda") for x in (where.keys(), where.values()))
            tab = s["table"][r].long()
            flat[tab[b // PAGE] * PAGE + b % PAGE] = flat[tab[a // PAGE] * PAGE + a % PAGE]
            nw[r, b] = s["weights"][r, a].to(f64)
    return kv, None, nw, None
