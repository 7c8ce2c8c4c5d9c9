"""What the library's rotary, shared-prefix and scored attention calls are measured on.

Four entry points: ``rswa_rope_1d`` (rotary positions, both pair layouts, part of the head, scaled
frequencies, and the transposed rotation of a gradient), ``rswa_decode_shared`` (one decode step of
sequences that share long prefixes), ``rswa_decode_scored`` and ``rswa_prefill_scored`` (attention
whose scores are capped by a tanh, biased by distance and limited to each query's own document).
``run`` computes a case in elementary torch operations, or, with ``own`` set, through the library.
"""
import math
import random

import torch

own = False  # set from outside: True runs the library's calls, False the plain forms

D = 128


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _rope(B, Hq, Hk, T, D=128, rot=128, layout="half", dtype="bf16", scaling="none", packed=False, inverse=False,
          far=0):
    return dict(op="rope", B=B, Hq=Hq, Hk=Hk, T=T, D=D, rot=rot, layout=layout, dtype=dtype, scaling=scaling,
                packed=packed, inverse=inverse, far=far)


def _shared(B, P, H, scap, n=128, cap=0, groups="even", lens="full", fill="full"):
    return dict(op="shared", B=B, P=P, H=H, scap=scap, n=n, cap=cap, groups=groups, lens=lens, fill=fill)


def _decode(B, H, cap, n=128, lens="full", fill="full", softcap=0.0, slopes=False, ranges="none", qstd=1.0):
    return dict(op="decode", B=B, H=H, cap=cap, n=n, lens=lens, fill=fill, softcap=softcap, slopes=slopes,
                ranges=ranges, qstd=qstd)


def _prefill(B, H, T, cap, n=128, lens="full", ring=True, softcap=0.0, slopes=False, ranges="none", qstd=1.0):
    return dict(op="prefill", B=B, H=H, T=T, cap=cap, n=n, lens=lens, ring=ring, softcap=softcap, slopes=slopes,
                ranges=ranges, qstd=qstd)


def listed():
    return [
        # rotary: the q and k rows of one decode step of 16 sequences
        dict(_rope(16, 16, 16, 1, scaling="by_parts", far=100000), name="rope_step"),
        # a ragged chunk read in place from a packed q/k/v projection, half of each head, pairs side by side
        dict(_rope(3, 16, 4, 777, rot=64, layout="interleaved", packed=True, scaling="linear"), name="rope_packed"),
        # the gradient of an encoded chunk in f32
        dict(_rope(2, 16, 16, 1024, dtype="f32", inverse=True, scaling="by_parts", far=30000), name="rope_gradient"),
        # the benchmark's chunk: 4 sequences x 4096 tokens
        dict(_rope(4, 16, 16, 4096), name="rope_chunk"),
        # shared prefix: eight questions about one page
        dict(_shared(8, 1, 16, 288), name="shared_one_page"),
        # odd sizes: five documents, some sequences with none, private prompts, part-filled rings of 100
        dict(_shared(37, 5, 12, 1999, n=100, cap=77, groups="random", lens="ragged", fill="ragged"),
             name="shared_ragged"),
        # 64 readers of one 400-page document
        dict(_shared(64, 1, 16, 102400), name="shared_long"),
        # 512 sequences over 64 ten-page documents
        dict(_shared(512, 64, 16, 2592), name="shared_batch"),
        # scored decode: one sequence, capped scores
        dict(_decode(1, 16, 288, softcap=30.0, qstd=4.0), name="decode_capped_one"),
        # 64 sequences whose query sees one document of its 32K history, distance bias
        dict(_decode(64, 16, 32768, lens="ragged", fill="ragged", softcap=50.0, slopes=True, ranges="window",
                     qstd=4.0), name="decode_documents"),
        # scored prefill: a small ragged chunk over packed pages
        dict(_prefill(3, 16, 333, 2592, lens="ragged", softcap=50.0, slopes=True, ranges="window", qstd=4.0),
             name="prefill_documents"),
        # a full chunk over a 40-page prefix, capped scores
        dict(_prefill(2, 16, 4096, 10272, softcap=50.0, qstd=4.0), name="prefill_capped"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "shared", "decode", "prefill"])
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128, 256) if r <= dim])
        B, T = _log(rng, 1, 64), _log(rng, 1, 4096)
        while B * T > 16384:
            T = max(1, T // 2)
        Hq = rng.randint(1, 16)
        return _rope(B, Hq, rng.randint(0, Hq), T, dim, rot, rng.choice(["half", "interleaved"]),
                     "f32" if B * T < 4096 and rng.random() < 0.4 else "bf16",
                     rng.choice(["none", "linear", "by_parts"]), rng.random() < 0.4, rng.random() < 0.4,
                     rng.choice([0, 1000, 100000]))
    H = rng.randint(1, 16)
    n = rng.choice([128, 128, 100, rng.randint(1, 256)])
    if op == "shared":
        B, P, scap = _log(rng, 1, 512), _log(rng, 1, 64), _log(rng, 1, 102400)
        while P * scap > 165888:
            P = max(1, P // 2)
            scap = scap if P > 1 else min(scap, 102400)
        if scap > 2592:
            B = min(B, 64)
        P = min(P, B)
        return _shared(B, P, H, scap, n, rng.choice([0, 0, _log(rng, 1, 600)]), rng.choice(["even", "random", "one"]),
                       rng.choice(["full", "ragged"]), rng.choice(["full", "ragged"]))
    softcap = rng.choice([0.0, 20.0, 50.0])
    slopes, ranges = rng.random() < 0.5, rng.choice(["none", "window", "window"])
    lens, qstd = rng.choice(["full", "ragged"]), rng.choice([1.0, 4.0])
    if op == "decode":
        B, cap = _log(rng, 1, 64), _log(rng, 1, 32768)
        while ranges == "none" and B * cap > 165888:
            B //= 2
        return _decode(B, H, cap, n, lens, rng.choice(["full", "ragged"]), softcap, slopes, ranges, qstd)
    B, T, cap = rng.randint(1, 3), _log(rng, 1, 2000), _log(rng, 1, 10272)
    return _prefill(B, H, T, cap, n, lens, rng.random() < 0.6, softcap, slopes, ranges, qstd)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _sizes(case):
    """The case's lengths, ring states, groups and documents: by the case alone, so that work() knows them."""
    r = random.Random("sizes:" + ",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))
    z = {}

    def lengths(count, cap, how):
        return [cap if how == "full" else r.randint(cap // 3, cap) for _ in range(count)]

    B, n = case["B"], case.get("n", 0)
    if case["op"] == "rope":
        z["start"] = [r.randint(0, case["far"]) for _ in range(B)]
        return z
    ring = case.get("ring", True)
    full = case.get("fill", "full") == "full"
    z["fill"] = [n if full else r.randint(0, n) for _ in range(B)] if ring else [0] * B
    z["wp"] = [r.randrange(n) for _ in range(B)]
    if case["op"] == "shared":
        P = case["P"]
        z["shared_len"] = lengths(P, case["scap"], case["lens"])
        z["share_of"] = ([b % P for b in range(B)] if case["groups"] == "even" else
                         [0] * B if case["groups"] == "one" else [r.randint(-1, P - 1) for _ in range(B)])
        z["len"] = lengths(B, case["cap"], "ragged")
        return z
    z["len"] = lengths(B, case["cap"], case["lens"])
    T = case.get("T", 1)
    z["pos"] = [m + r.randint(0, 2000) for m in z["len"]]
    z["ranges"] = []
    for m in z["len"]:
        # documents of up to 2592 rows laid end to end; the chunk's queries go through them in order
        cuts = [0]
        while cuts[-1] < m:
            cuts.append(min(m, cuts[-1] + r.randint(max(1, min(2592, m) // 3), max(1, min(2592, m)))))
        docs = list(zip(cuts, cuts[1:])) or [(0, 0)]
        first = r.randrange(len(docs))
        each = max(1, T // 3 + 1)
        if case["ranges"] == "none":
            z["ranges"].append([(0, m)] * T)
        else:
            z["ranges"].append([docs[(first + i // each) % len(docs)] for i in range(T)])
    return z


def _inv_freq(case):
    """Pair frequencies in f64: base^(-2i/rot), divided for positions beyond the trained length."""
    rot = case["rot"]
    f = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if case["scaling"] == "linear":
        return f / 8.0, 1.0
    if case["scaling"] == "by_parts":  # slow pairs are divided, fast ones kept, a ramp between
        factor, trained = 16.0, 4096.0
        turns = trained * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _randn(shape, gen, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    z = _sizes(case)
    s = {"case": case}
    if case["op"] == "rope":
        B, Hq, Hk, T, dim = case["B"], case["Hq"], case["Hk"], case["T"], case["D"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["packed"]:  # the rows of one [tokens][heads] projection: q, k and v heads side by side
            x = torch.randn((B, T, Hq + 2 * Hk, dim), generator=gen, device="cuda").to(dt).transpose(1, 2)
            s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hk]
        else:
            s["q"] = torch.randn((B, Hq, T, dim), generator=gen, device="cuda").to(dt)
            s["k"] = torch.randn((B, Hk, T, dim), generator=gen, device="cuda").to(dt)
        s["q_out"] = torch.empty((B, Hq, T, dim), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((B, Hk, T, dim), dtype=dt, device="cuda")
        s["pos"] = _int(z["start"])[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")
        s["freq"], s["mscale"] = _inv_freq(case)
        s["freq_gpu"] = s["freq"].cuda()
        return s
    B, H, n = case["B"], case["H"], case["n"]
    T = case.get("T", 1)
    q_shape = (B, H, T, D) if case["op"] == "prefill" else (B, H, D)
    s["q"] = _randn(q_shape, gen, case.get("qstd", 1.0))
    s["wp"], s["fill"], s["len"] = _int(z["wp"]), _int(z["fill"]), _int(z["len"])
    cap = case["cap"]
    s["pk"], s["pv"] = _randn((B, H, cap, D), gen), _randn((B, H, cap, D), gen)
    # rows past a sequence's end and empty ring slots hold whatever memory held: NaN here
    past = torch.arange(cap, device="cuda")[None, :] >= s["len"][:, None]
    s["pk"].masked_fill_(past[:, None, :, None], math.nan)
    s["pv"].masked_fill_(past[:, None, :, None], math.nan)
    s["rk"], s["rv"] = _randn((B, H, n, D), gen), _randn((B, H, n, D), gen)
    empty = _age(s["wp"], n) > s["fill"][:, None]
    s["rk"].masked_fill_(empty[:, None, :, None], math.nan)
    s["rv"].masked_fill_(empty[:, None, :, None], math.nan)
    s["lse"] = torch.empty(q_shape[:-1], device="cuda")
    if case["op"] == "shared":
        P, scap = case["P"], case["scap"]
        s["sk"], s["sv"] = _randn((P, H, scap, D), gen), _randn((P, H, scap, D), gen)
        s["shared_len"], s["share_of"] = _int(z["shared_len"]), _int(z["share_of"])
        past = torch.arange(scap, device="cuda")[None, :] >= s["shared_len"][:, None]
        s["sk"].masked_fill_(past[:, None, :, None], math.nan)
        s["sv"].masked_fill_(past[:, None, :, None], math.nan)
        s["most"] = max([z["share_of"].count(p) for p in range(P)] + [1])  # readers of the widest group
        s["out"] = torch.empty(q_shape, dtype=torch.bfloat16, device="cuda")
        return s
    s["softcap"] = case["softcap"]
    s["pos"] = _int(z["pos"])
    s["slopes"] = (2.0 ** (-8.0 * (torch.arange(H, device="cuda") + 1) / H)).float() if case["slopes"] else None
    s["ranges"] = _int(z["ranges"]).view(q_shape[0], T, 2) if case["ranges"] != "none" else None
    if case["op"] == "decode":
        s["ranges"] = s["ranges"][:, 0].contiguous() if s["ranges"] is not None else None
        s["out"] = torch.empty(q_shape, device="cuda")
    else:
        s["out"] = torch.empty(q_shape, dtype=torch.bfloat16, device="cuda")
        s["ko"], s["vo"] = _randn(q_shape, gen), _randn(q_shape, gen)
    return s


_workspaces = {}


def _workspace(rswa, c):
    """The zero-filled scratch of these dims, which a user's program makes once."""
    key = (c["op"], c["B"], c["H"], c["n"], c["cap"], c.get("P"), c.get("scap"))
    if key not in _workspaces:
        dims = rswa.Dims(c["B"], c["H"], D, c["n"], c["cap"])
        _workspaces[key] = (rswa.new_shared_workspace(dims, c["P"]) if c["op"] == "shared" else
                            rswa.new_workspace(dims, rswa.OP_DECODE_SCORED if c["op"] == "decode" else rswa.OP_PREFILL))
    return _workspaces[key]


def _age(wp, n):
    """Age of each ring slot: 1 for the most recently written one."""
    return torch.remainder(wp[:, None].long() - 1 - torch.arange(n, device=wp.device), n) + 1


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import long_context_decode_swa_b200 as rswa
    c = s["case"]
    if c["op"] == "rope":
        k = dict(k=s["k"], k_out=s["k_out"]) if c["Hk"] else {}
        rswa.rswa_rope_1d(s["q"], s["pos"], s["freq"], q_out=s["q_out"], layout=c["layout"], mscale=s["mscale"],
                          inverse=c["inverse"], **k)
        return s["q_out"], s["k_out"]
    ws = _workspace(rswa, c)
    if c["op"] == "shared":
        rswa.rswa_decode_shared(s["q"], s["sk"], s["sv"], s["shared_len"], s["share_of"], s["rk"], s["rv"], s["wp"],
                                s["fill"], s["out"], ws, pk=s["pk"], pv=s["pv"], prefix_len=s["len"],
                                lse=s["lse"])
    elif c["op"] == "decode":
        rswa.rswa_decode_scored(s["q"], s["pk"], s["pv"], s["len"], s["rk"], s["rv"], s["wp"], s["fill"], s["out"],
                                ws, softcap=s["softcap"], slopes=s["slopes"], pos=s["pos"], ranges=s["ranges"],
                                lse=s["lse"])
    else:
        ring = dict(ring_k=s["rk"], ring_v=s["rv"], wp=s["wp"], fill=s["fill"]) if c["ring"] else dict(ring=c["n"])
        rswa.rswa_prefill_scored(s["q"], s["ko"], s["vo"], s["pk"], s["pv"], s["len"], s["out"], ws,
                                 softcap=s["softcap"], slopes=s["slopes"], pos=s["pos"], ranges=s["ranges"],
                                 lse=s["lse"], **ring)
    return s["out"], s["lse"]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rope":
        return _plain_rope(s, s["q"]), _plain_rope(s, s["k"])
    if c["op"] == "shared":
        return _plain_shared(s)
    return _plain_decode(s) if c["op"] == "decode" else _plain_prefill(s)


def _plain_rope(s, x):
    c, rot = s["case"], s["case"]["rot"]
    angle = s["pos"].double()[:, None, :, None] * s["freq_gpu"]
    sign = -1.0 if c["inverse"] else 1.0
    cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * (sign * s["mscale"])).float()
    f = x.float()
    if c["layout"] == "half":
        a, b = f[..., :rot // 2], f[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, f[..., rot:]], -1).to(x.dtype)


def _softmax_v(score, seen, v, dtype):
    """softmax over the last axis of `score` where `seen`, times v, and its log-sum-exp."""
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = weight.sum(-1)
    out = weight.to(v.dtype) @ v / total.clamp_min(1e-37)[..., None].to(v.dtype)
    lse = top[..., 0] + total.log()
    return out.to(dtype), lse.float()


def _rows(x, seen):
    """Rows in f32, zero where nothing may read them."""
    return x.float().masked_fill_(~seen[:, None, :, None], 0.0)


def _readers(x, none):
    """[P][H][most].. -> [P * most + 1][H]..: the last row, all `none`, is for sequences without a prefix."""
    x = x.transpose(1, 2).flatten(0, 1)
    return torch.cat([x, torch.full_like(x[:1], none)])


def _plain_shared(s):
    c = s["case"]
    scale = 1.0 / math.sqrt(D)
    B, P, H, n, most = c["B"], c["P"], c["H"], c["n"], s["most"]
    dev = s["q"].device
    # readers of each prefix side by side: [P][most] rows, most = the widest group
    order = torch.argsort(s["share_of"], stable=True)
    group = s["share_of"].long()[order]
    first = torch.searchsorted(group, group)
    place = torch.where(group >= 0, group * most + torch.arange(B, device=dev) - first, P * most)
    q = s["q"].float()
    grouped = torch.zeros((P * most + 1, H, D), device=dev)
    grouped[place] = q[order]
    grouped = grouped[:P * most].view(P, most, H, D).transpose(1, 2)
    seen = torch.arange(c["scap"], device=dev)[None, :] < s["shared_len"][:, None]
    score = (grouped @ _rows(s["sk"], seen).transpose(-1, -2)).mul_(scale)
    score.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1)
    top = top.masked_fill(top == -math.inf, -1e30)
    weight = score.sub_(top[..., None]).exp_()
    total, mixed = weight.sum(-1), weight @ _rows(s["sv"], seen)
    # back to sequences; a sequence without a prefix reads a row of zeros
    back = torch.empty_like(place)
    back[order] = place
    top, total, mixed = _readers(top, -1e30)[back], _readers(total, 0.0)[back], _readers(mixed, 0.0)[back]
    # each sequence's private rows and ring
    seen = torch.cat([torch.arange(c["cap"], device=dev)[None, :] < s["len"][:, None],
                      _age(s["wp"], n) <= s["fill"][:, None]], 1)
    k = _rows(torch.cat([s["pk"], s["rk"]], 2), seen)
    v = _rows(torch.cat([s["pv"], s["rv"]], 2), seen)
    score = (q[:, :, None] @ k.transpose(-1, -2))[:, :, 0] * scale
    score.masked_fill_(~seen[:, None], -math.inf)
    both = torch.maximum(top, score.amax(-1))
    weight = (score - both[..., None]).exp()
    shrink = (top - both).exp()
    total = total * shrink + weight.sum(-1)
    mixed = mixed * shrink[..., None] + (weight[:, :, None] @ v)[:, :, 0]
    out = (mixed / total.clamp_min(1e-37)[..., None]).to(torch.bfloat16)
    return out, torch.where(total > 0, both + total.log(), -math.inf)


def _capped(score, softcap):
    return score.div_(softcap).tanh_().mul_(softcap) if softcap > 0 else score


def _plain_decode(s):
    c, dev = s["case"], s["q"].device
    x = torch.arange(c["cap"], device=dev)
    seen = x[None, :] < s["len"][:, None]
    if s["ranges"] is not None:
        seen = seen & (x >= s["ranges"][:, :1]) & (x < s["ranges"][:, 1:])
    age = _age(s["wp"], c["n"])
    seen = torch.cat([seen, age <= s["fill"][:, None]], 1)
    k = _rows(torch.cat([s["pk"], s["rk"]], 2), seen)
    v = _rows(torch.cat([s["pv"], s["rv"]], 2), seen)
    score = (s["q"].float()[:, :, None] @ k.transpose(-1, -2))[:, :, 0].mul_(1.0 / math.sqrt(D))
    score = _capped(score, s["softcap"]).double()  # in 64 bits: a far document's bias is large
    if s["slopes"] is not None:
        away = torch.cat([s["pos"][:, None] - x, age - 1], 1)
        score.sub_(s["slopes"].double()[None, :, None] * away[:, None])
    top = score.masked_fill_(~seen[:, None], -math.inf).amax(-1, keepdim=True)
    weight = score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_().float()
    total = weight.sum(-1)
    out = (weight[:, :, None] @ v)[:, :, 0] / total.clamp_min(1e-37)[..., None]
    return out, (top[..., 0] + total.double().log()).float()


def _plain_prefill(s):
    c, dev = s["case"], s["q"].device
    n, T = c["n"], c["T"]
    x, i = torch.arange(c["cap"], device=dev), torch.arange(T, device=dev)
    inside = x[None, :] < s["len"][:, None]
    seen = inside[:, None, :].expand(-1, T, -1)
    if s["ranges"] is not None:
        seen = seen & (x >= s["ranges"][..., :1]) & (x < s["ranges"][..., 1:])
    band = (i[None, :] <= i[:, None]) & (i[None, :] > i[:, None] - n)
    away = s["pos"][:, None, None] + i[:, None] - x
    ks, vs, live = [s["pk"]], [s["pv"]], [inside]
    seens, aways = [seen], [away]
    if c["ring"]:
        age = _age(s["wp"], n)
        written = age <= s["fill"][:, None]
        ks.append(s["rk"]), vs.append(s["rv"]), live.append(written)
        seens.append(written[:, None, :] & (age[:, None, :] < n - i[:, None]))
        aways.append(i[:, None] + age[:, None, :])
    ks.append(s["ko"]), vs.append(s["vo"]), live.append(torch.ones_like(s["pos"], dtype=torch.bool)[:, None].expand(-1, T))
    seens.append(band[None].expand(c["B"], -1, -1))
    aways.append((i[:, None] - i)[None].expand(c["B"], -1, -1))
    live = torch.cat(live, 1)
    k, v = _rows(torch.cat(ks, 2), live), _rows(torch.cat(vs, 2), live)
    score = _capped((s["q"].float() @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)), s["softcap"])
    if s["slopes"] is not None:
        score.sub_(s["slopes"][None, :, None, None] * torch.cat(aways, 2)[:, None])
    return _softmax_v(score, torch.cat(seens, 2)[:, None], v, torch.bfloat16)


# ---------------------------------------------------------------------------------------------
# the cost that no form can do without
# ---------------------------------------------------------------------------------------------

def work(case):
    z = _sizes(case)
    if case["op"] == "rope":
        rows = case["B"] * (case["Hq"] + case["Hk"]) * case["T"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2.0 * size * rows * case["D"] + 4.0 * case["B"] * case["T"], "flops": 3.0 * rows * case["rot"]}
    B, H, T = case["B"], case["H"], case.get("T", 1)
    row = 4.0 * D * H  # one key and one value row of every head
    ring = sum(min(f, case["n"]) for f in z["fill"])
    if case["op"] == "shared":
        used = sorted(set(p for p in z["share_of"] if p >= 0))
        pairs = sum(z["shared_len"][p] for p in z["share_of"] if p >= 0) + sum(z["len"]) + ring
        rows = sum(z["shared_len"][p] for p in used) + sum(z["len"]) + ring
        return {"bytes": row * rows + B * H * (4.0 * D + 4.0), "flops": 4.0 * D * H * pairs}
    n, pairs, rows = case["n"], 0, 0
    for b in range(B):
        spans = sorted(set(z["ranges"][b]))
        rows += sum(hi - lo for lo, hi in spans) + z["fill"][b]
        pairs += sum(hi - lo for lo, hi in z["ranges"][b])
        if T == 1 and case["op"] == "decode":
            pairs += z["fill"][b]
        else:
            rows += T
            pairs += sum(min(i + 1, n) + max(0, min(z["fill"][b], n - 1 - i)) for i in range(T))
    out = 6.0 if case["op"] == "decode" else 4.0
    return {"bytes": row * rows + B * H * T * (out * D + 4.0), "flops": 4.0 * D * H * pairs}


# ---------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------------------------

def _reference(q, k, v, bias=None, softcap=0.0):
    """Attention of queries q [.., T, D] over rows k, v [.., K, D]: bias is -inf where a row is not seen."""
    z = torch.einsum("...td,...kd->...tk", q, k) / math.sqrt(D)
    if softcap > 0:
        z = softcap * torch.tanh(z / softcap)
    if bias is not None:
        z = z + bias
    if z.shape[-1] == 0 or bool(torch.isneginf(z).all(-1).any()):
        z = torch.cat([z, torch.full_like(z[..., :1] if z.shape[-1] else q[..., :1], -1e300)], -1)
        v = torch.cat([v, torch.zeros_like(v[..., :1, :]) if v.shape[-2] else torch.zeros_like(q[..., :1, :])], -2)
    lse = torch.logsumexp(z, -1)
    out = torch.einsum("...tk,...kd->...td", torch.exp(z - lse[..., None]), v)
    return out, torch.where(lse < -1e299, -math.inf, lse)


def exact(case, seed):
    s, z = prepare(case, seed), _sizes(case)
    if case["op"] == "rope":
        freq = s["freq"].cuda()
        spin = torch.polar(torch.full_like(freq, s["mscale"]).expand(case["B"], 1, case["T"], -1),
                           s["pos"].double()[:, None, :, None] * freq)
        spin = spin.conj() if case["inverse"] else spin
        outs = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            rot = case["rot"]
            if case["layout"] == "half":
                w = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * spin
                y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
            else:
                w = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * spin
                y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
            outs.append(y)
        return tuple(outs)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:-1], dtype=torch.float64, device="cuda")
    n, H = case["n"], case["H"]
    for b in range(case["B"]):
        m, f, w = z["len"][b], z["fill"][b], z["wp"][b]
        slots = torch.tensor([(w - f + j) % n for j in range(f)], dtype=torch.long, device="cuda")  # oldest first
        rk, rv = s["rk"][b][:, slots], s["rv"][b][:, slots]
        if case["op"] == "shared":
            p = z["share_of"][b]
            some = z["shared_len"][p] if p >= 0 else 0
            k = torch.cat([s["sk"][p][:, :some], s["pk"][b][:, :m], rk], 1).double()
            v = torch.cat([s["sv"][p][:, :some], s["pv"][b][:, :m], rv], 1).double()
            o, e = _reference(s["q"][b][:, None].double(), k, v)
            out[b], lse[b] = o[:, 0], e[:, 0]
        elif case["op"] == "decode":
            lo, hi = z["ranges"][b][0]
            k = torch.cat([s["pk"][b][:, lo:hi], rk], 1).double()
            v = torch.cat([s["pv"][b][:, lo:hi], rv], 1).double()
            at = torch.cat([torch.arange(lo, hi, device="cuda"), z["pos"][b] - f + 1 + torch.arange(f, device="cuda")])
            bias = None
            if s["slopes"] is not None:
                bias = -s["slopes"].double()[:, None, None] * (z["pos"][b] - at).double()
            o, e = _reference(s["q"][b][:, None].double(), k, v, bias, case["softcap"])
            out[b], lse[b] = o[:, 0], e[:, 0]
        else:
            T = case["T"]
            # one line of positions: the prefix's own, then the chunk's, the ring's just before it
            at = torch.cat([torch.arange(m), z["pos"][b] - f + torch.arange(f), z["pos"][b] + torch.arange(T)]).cuda()
            here = z["pos"][b] + torch.arange(T, device="cuda")[:, None]
            recent = (at <= here) & (at > here - n)
            lohi = torch.tensor(z["ranges"][b], device="cuda")
            row = torch.arange(m + f + T, device="cuda")
            seen = torch.where(row < m, (row >= lohi[:, :1]) & (row < lohi[:, 1:]), recent)
            for h in range(H):
                k = torch.cat([s["pk"][b, h, :m], rk[h], s["ko"][b, h]]).double()
                v = torch.cat([s["pv"][b, h, :m], rv[h], s["vo"][b, h]]).double()
                bias = torch.zeros(T, m + f + T, dtype=torch.float64, device="cuda")
                if s["slopes"] is not None:
                    bias = -s["slopes"][h].double() * (here - at).double()
                bias = bias.masked_fill(~seen, -math.inf)
                out[b, h], lse[b, h] = _reference(s["q"][b, h].double(), k, v, bias, case["softcap"])
    return out, lse
