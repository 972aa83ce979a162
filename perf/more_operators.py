"""A cache in 8 or 4 bits with what is around it, and what it measures.

Four operators of a server that keeps its keys and values in few bits:

  rotary  positions turned into q and k: each pair of channels is rotated by the
          position on its axis (text has one; images and video time, height and
          width) times its frequency; or back
  write   k and v of new tokens into the paged cache, as codes of 8 bits (a row
          of a head shares a lowest value and a step) or 4 (32 channels do),
          rotated on the way or not, and read back as the values they stand for,
          as the next chunk of a prompt needs them
  attend  attention of one new token of every sequence over its cache: capped or
          biased scores, all tokens or a window of the newest
  step    a decode step of the three together: q and k of one token of every
          sequence rotated, k and v written, all attended; returned are the
          rotated q and the new row as the cache holds it, too

Where `own` is false the operators are computed from elementary torch operations
in 32 bits (angles in 64) and rounded once; where it is true through the library.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BASE = 500000.0  # of the frequencies


# ---- cases -------------------------------------------------------------------

def listed():
    r = dict(op="rotary", hq=32, hkv=8, d=128, rot=128, dtype="bf16", sections="64", turns=False,
             neighbours=False, inverse=False)
    w = dict(op="write", hq=32, hkv=8, d=128, dtype="bf16", rotary=True, page=256)
    a = dict(op="attend", hq=32, hkv=8, d=128, dtype="bf16", out="same", softcap=0.0, slopes=False,
             window=0, page=256)
    s = dict(op="step", hq=32, hkv=8, d=128, dtype="bf16", out="same", page=256)
    return [
        # one token of five requests, far apart in long texts: latency counts
        dict(r, name="rotary-step", n=5, far=131072),
        # a prompt of video frames: time, height and width take the pairs in turn
        dict(r, name="rotary-video", n=20011, far=20011, sections="24 20 20", turns=True),
        # images on two axes, half of 64 channels, neighbours paired, rotated back
        # (the gradient, or keys that move to another place)
        dict(r, name="rotary-image-back", n=3001, far=1024, hq=16, hkv=16, d=64, rot=32,
             dtype="fp16", sections="8 8", neighbours=True, inverse=True),
        # a long prompt rotated into 8 bits, and back for its next chunk
        dict(w, name="write-prompt-8", bits=8, n=1, tokens=16385),
        # short prompts of a batch into 4 bits, small pages, 64 channels
        dict(w, name="write-batch-4", bits=4, n=6, tokens=1111, hq=32, hkv=4, d=64, dtype="fp16",
             rotary=False, page=64),
        # a short question: latency counts
        dict(a, name="attend-short-8", bits=8, n=1, len_max=77),
        # one request about a very long document
        dict(a, name="attend-long-4", bits=4, n=1, len_max=131072),
        # a batch of ragged chats, scores capped
        dict(a, name="attend-batch-4", bits=4, n=48, len_max=8192, softcap=50.0),
        # the sliding layers of a model with biased scores, eight heads a key, fp32 out
        dict(a, name="attend-window-8", bits=8, n=16, len_max=32768, hq=64, dtype="fp16",
             out="fp32", slopes=True, window=4096),
        # decode steps: one request, and a batch of ragged chats
        dict(s, name="step-one-4", bits=4, n=1, len_max=4096),
        dict(s, name="step-batch-8", bits=8, n=32, len_max=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _sections(rng, pairs):
    axes = rng.choice([1, 1, 2, 3])
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    return " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))


def draw(rng):
    op = rng.choice(["rotary", "write", "attend", "step"])
    dtype = rng.choice(["bf16", "fp16"])
    hkv, g = rng.choice([(8, 4), (8, 1), (4, 8), (2, 2), (16, 1), (8, 2), (1, 8), (8, 8)])
    d = rng.choice([128, 128, 64])
    c = dict(op=op, hq=hkv * g, hkv=hkv, d=d, dtype=dtype)
    rows = hkv * d  # channels of a token's keys; the largest listed cases have 1,024
    if op == "rotary":
        rot = rng.choice([d, d, d // 2, 16])
        return dict(c, n=_log(rng, 1, min(20000, 20011 * 40 * 128 // (hkv * (g + 1) * d))),
                    far=_log(rng, 16, 1 << 20), rot=rot, sections=_sections(rng, rot // 2),
                    turns=rng.random() < 0.5, neighbours=rng.random() < 0.4,
                    inverse=rng.random() < 0.3)
    c.update(bits=rng.choice([8, 4]), page=rng.choice([16, 64, 256, 1024]))
    if op == "write":
        tokens = _log(rng, 1, 16384 * 1024 // max(rows, 1024))
        return dict(c, rotary=rng.random() < 0.6, tokens=tokens,
                    n=_log(rng, 1, max(1, min(48, 16384 * 1024 // rows // tokens))))
    c.update(len_max=_log(rng, 1, 131072 * 1024 // max(rows, 1024)), out=rng.choice(["same", "fp32"]))
    c.update(n=_log(rng, 1, max(1, min(96, 131072 * 1024 // max(rows, 1024) // c["len_max"]))))
    if op == "attend":
        c.update(softcap=rng.choice([0.0, 0.0, 50.0]), slopes=rng.random() < 0.3,
                 window=rng.choice([0, 0, _log(rng, 1, c["len_max"])]))
    return c


# ---- what a case holds -----------------------------------------------------------

def _lengths(case):
    r = random.Random("lengths %d %d" % (case["n"], case["len_max"]))
    return [case["len_max"]] + [r.randint(max(1, case["len_max"] // 8), case["len_max"])
                                for _ in range(case["n"] - 1)]


def _sizes(case):
    """How many pairs of channels each axis has."""
    return [int(x) for x in case["sections"].split()]


def _axes(case):
    """For every pair of channels the axis whose position turns it."""
    left = _sizes(case)
    if not case["turns"]:
        return [a for a, k in enumerate(left) for _ in range(k)]
    out, a = [], 0
    while sum(left):
        if left[a]:
            left[a] -= 1
            out.append(a)
        a = (a + 1) % len(left)
    return out


def _row_bytes(case):
    d = case["d"]
    return d + 4 if case["bits"] == 8 else d // 2 + d // 32 * 4


def work(case):
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "rotary":
        return {"bytes": case["n"] * ((hq + hkv) * d * 4 + 4 * len(_sizes(case))),
                "flops": case["n"] * (hq + hkv) * case["rot"] * 3}
    if case["op"] == "write":
        t = case["n"] * case["tokens"]
        return {"bytes": t * hkv * 2 * (4 * d + 2 * _row_bytes(case)) +
                (t * (hq * d * 4 + 4) if case["rotary"] else 0),
                "flops": t * (hkv * 2 * d * 4 + ((hq + hkv) * d * 3 if case["rotary"] else 0))}
    lens, n = _lengths(case), case["n"]
    window = case.get("window") or max(lens) + 1
    seen = sum(min(x, window) for x in lens)
    ob = 4 if case["out"] == "fp32" else 2
    b, f = seen * hkv * 2 * _row_bytes(case) + n * hq * d * (2 + ob), 4 * seen * hq * d
    if case["op"] == "step":  # q and k rotated, k and v written and attended
        b += n * (hkv * 2 * (4 * d + 2 * _row_bytes(case)) + hq * d * 2 + 4)
        f += n * ((hq + hkv) * d * 3 + 4 * hq * d)
    return {"bytes": b, "flops": f}


# ---- inputs ------------------------------------------------------------------

def _slopes(hq, dev):
    """The usual geometric slopes of a distance bias."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32,
                        device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g, dtype=torch.float32)

    def far(*shape, to):
        return torch.randint(0, to, shape, device=dev, generator=g, dtype=torch.int32)

    # keys have a few channels that stand far from zero in every token
    shift = normal(hkv, d) * (torch.rand(hkv, d, device=dev, generator=g) < 0.1) * 4.0

    def keys(*shape):
        return normal(*shape, hkv, d).add_(shift).to(dt)

    def values(*shape):
        return normal(*shape, hkv, d).to(dt)

    s = dict(case)
    if case["op"] == "rotary":
        s.update(q=normal(case["n"], hq, d).to(dt), k=keys(case["n"]),
                 positions=far(len(_sizes(case)), case["n"], to=case["far"]))
        if own:
            import sparse_paged_decode_logical_gb300 as spd
            s["rule"] = spd.Rotary(d, rotary_dim=case["rot"], sections=_sizes(case),
                                   axes_in_turn=case["turns"], neighbours=case["neighbours"],
                                   base=BASE)
        return s
    if case["op"] == "write":
        n, t = case["n"], case["tokens"]
        s.update(k=keys(n, t), v=values(n, t))
        if case["rotary"]:  # after a first chunk of another length for every sequence
            first = far(n, 1, to=100000)
            s.update(q=normal(n, t, hq, d).to(dt),
                     positions=first + torch.arange(t, device=dev, dtype=torch.int32))
        if own:
            s["cache"] = _cache(case, n, -(-t // case["page"]) * n, t)
            s["rule"] = _text_rule(d) if case["rotary"] else None
        return s
    lens, n = _lengths(case), case["n"]
    gain = 4.0 if case.get("softcap") else 1.0
    step = case["op"] == "step"
    s.update(q=(normal(n, hq, d) * gain).to(dt),
             slope=_slopes(hq, dev) if case.get("slopes") else None)
    if step:
        s.update(k_new=keys(n, 1), v_new=values(n, 1),
                 positions=torch.tensor(lens, dtype=torch.int32, device=dev)[:, None])
    longest = max(lens) + 1
    if own:
        c = _cache(case, n, sum(-(-(x + 1) // case["page"]) for x in lens), longest)
        s.update(cache=c, ids=[c.seq_create() for _ in lens], held=lens,
                 rule=_text_rule(d) if step else None,
                 out_dtype=torch.float32 if case["out"] == "fp32" else dt)
    else:
        groups, at = (1 if case["bits"] == 8 else d // 32), []
        for _ in range(2):
            at.append([torch.zeros(n, longest, hkv, d, dtype=torch.uint8, device=dev)] +
                      [torch.zeros(n, longest, hkv, groups, dtype=dt, device=dev) for _ in range(2)])
        s.update(kc=at[0], vc=at[1], lens=torch.tensor(lens, device=dev))
        if case.get("keep"):
            s["raw"] = []
    for i, x in enumerate(lens):
        k, v = keys(x), values(x)
        if own:
            c.kv_append([s["ids"][i]], k[None], v[None])
            continue
        if case.get("keep"):  # (for the definition in 64 bits)
            s["raw"].append((k, v))
        for to, x16 in ((s["kc"], k), (s["vc"], v)):
            for a, b in zip(to, _quantise(x16, case["bits"])):
                a[i, :x] = b
    return s


def _text_rule(d):
    import sparse_paged_decode_logical_gb300 as spd
    return spd.Rotary(d, base=BASE)


def _cache(case, seqs, pages, longest):
    import sparse_paged_decode_logical_gb300 as spd
    return spd.SparsePagedKVCache(
        device="cuda", num_q_heads=case["hq"], num_kv_heads=case["hkv"], head_dim=case["d"],
        dtype=case["dtype"], logical_page=16, physical_page=case["page"],
        num_physical_pages=pages, max_seqs=seqs, max_context=longest, kv_quant=case["bits"])


# ---- one pass -----------------------------------------------------------------

def run(s):
    if s["op"] == "rotary":
        return _rotary_own(s) if own else _rotary(s)
    if s["op"] == "write":
        return _write_own(s) if own else _write(s)
    if s["op"] == "attend":
        return _attend_own(s, s["q"]) if own else _attend(s, s["q"])
    return _step_own(s) if own else _step(s)


def _rotary_own(s):
    import sparse_paged_decode_logical_gb300 as spd
    return spd.rotary(s["rule"], s["positions"], s["q"], s["k"], inverse=s["inverse"])


def _write_own(s):
    c = s["cache"]
    ids = [c.seq_create() for _ in range(s["n"])]
    q = None
    if s["rotary"]:
        q = c.kv_append_rotary(ids, s["rule"], s["q"], s["k"], s["v"], positions=s["positions"])
    else:
        c.kv_append(ids, s["k"], s["v"])
    k, v = c.kv_read(ids)
    for i in ids:
        c.seq_free(i)
    return (k, v) if q is None else (q, k, v)


def _attend_own(s, q):
    return s["cache"].quant_decode_attention(q, s["ids"], window=s.get("window", 0),
                                             softcap=s.get("softcap", 0.0), slopes=s["slope"],
                                             out_dtype=s["out_dtype"])


def _step_own(s):
    c = s["cache"]
    q = c.kv_append_rotary(s["ids"], s["rule"], s["q"][:, None], s["k_new"], s["v_new"],
                           positions=s["positions"])
    out = _attend_own(s, q[:, 0])
    k, v = c.kv_read(s["ids"], begin=-1)
    for i, x in zip(s["ids"], s["held"]):  # taken back, as a token that is rejected
        c.seq_truncate(i, x)
    return out, q[:, 0], k[:, 0], v[:, 0]


def _angles(positions, rot, axes):
    """cos and sin [tokens][rot / 2] in 32 bits of angles in 64."""
    dev = positions.device
    freq = torch.tensor([BASE ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64,
                        device=dev)
    angle = positions[torch.tensor(axes, device=dev)].t().double() * freq
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(x, cos, sin, rot, neighbours):
    """x [tokens][heads][d] with its first rot channels rotated, in the type of x."""
    y = x.float()
    cos, sin = cos[:, None], sin[:, None]
    if neighbours:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([z, y[..., rot:]], -1).to(x.dtype)


def _rotary(s):
    cos, sin = _angles(s["positions"], s["rot"], _axes(s))
    if s["inverse"]:
        sin = -sin
    return tuple(_turn(s[x], cos, sin, s["rot"], s["neighbours"]) for x in ("q", "k"))


def _turn_text(x, positions):
    """x [n][tokens][heads][d] rotated over all its channels by positions [n][tokens]."""
    d = x.shape[-1]
    cos, sin = _angles(positions.reshape(1, -1), d, [0] * (d // 2))
    return _turn(x.flatten(0, 1), cos, sin, d, False).view(x.shape)


def _quantise(x, bits):
    """Codes, lowest values and steps of x [...][heads][d]: a step is the least
    number of the type of x that reaches from the lowest value to the highest in
    2^bits - 1 steps."""
    d = x.shape[-1]
    y = x.float().unflatten(-1, (1, d) if bits == 8 else (d // 32, 32))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    levels = torch.full_like(lo, 2 ** bits - 1)  # (a scalar divisor would be a product)
    step = ((hi - lo) / levels).to(x.dtype)
    up = (step.view(torch.int16) + 1).view(x.dtype)
    step = torch.where(step.float() * levels < hi - lo, up, step)
    f = torch.where(step == 0, torch.ones_like(lo), step.float())
    codes = torch.round((y - lo) / f).flatten(-2).to(torch.uint8)
    return codes, lo.squeeze(-1).to(x.dtype), step.squeeze(-1)


def _values(codes, lo, step):
    """The values that codes stand for, in 32 bits."""
    y = codes.float().unflatten(-1, (lo.shape[-1], -1))
    return (lo.float()[..., None] + step.float()[..., None] * y).flatten(-2)


def _write(s):
    k = _turn_text(s["k"], s["positions"]) if s["rotary"] else s["k"]
    k, v = (_values(*_quantise(x, s["bits"])).to(x.dtype) for x in (k, s["v"]))
    return (_turn_text(s["q"], s["positions"]), k, v) if s["rotary"] else (k, v)


def _attend(s, q, more=0):
    n, hq, d = q.shape
    k, v = _values(*s["kc"]), _values(*s["vc"])
    longest, hkv = k.shape[1:3]
    g = hq // hkv
    x = torch.matmul(q.float().view(n, hkv, g, d), k.permute(0, 2, 3, 1)) * d ** -0.5
    if s.get("softcap"):
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    back = (s["lens"] + more - 1)[:, None] - torch.arange(longest, device=q.device)
    if s["slope"] is not None:
        x -= s["slope"].view(1, hkv, g, 1) * back.view(n, 1, 1, longest)
    hidden = (back < 0) | (back >= (s.get("window") or longest))
    x.masked_fill_(hidden.view(n, 1, 1, longest), float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x /= x.sum(-1, keepdim=True)
    o = torch.matmul(x, v.permute(0, 2, 1, 3)).reshape(n, hq, d)
    return o if s["out"] == "fp32" else o.to(q.dtype)


def _step(s):
    q = _turn_text(s["q"][:, None], s["positions"])[:, 0]
    k = _turn_text(s["k_new"], s["positions"])
    row, kept = torch.arange(len(q), device=q.device), []
    for to, x in ((s["kc"], k), (s["vc"], s["v_new"])):
        new = _quantise(x[:, 0], s["bits"])
        for a, b in zip(to, new):
            a[row, s["lens"]] = b
        kept.append(_values(*new).to(q.dtype))
    return (_attend(s, q, 1), q, *kept)


# ---- the definition in 64 bits -----------------------------------------------------

def exact(case, seed):
    global own
    held, own = own, False
    try:
        s = prepare(dict(case, keep=True), seed)
    finally:
        own = held
    if case["op"] == "rotary":
        return tuple(_exact_turn(s[x], s["positions"], case["rot"], _axes(case),
                                 case["neighbours"], case["inverse"]) for x in ("q", "k"))
    if case["op"] == "write":
        def turned(x):
            p = s["positions"].reshape(1, -1)
            return _exact_turn(x.flatten(0, 1), p, x.shape[-1], None, False, False).view(x.shape)

        if not case["rotary"]:
            return tuple(_exact_kept(s[x], case["bits"]) for x in ("k", "v"))
        k = turned(s["k"]).to(s["k"].dtype)  # (a key is rounded to its type when it is rotated)
        return turned(s["q"]), _exact_kept(k, case["bits"]), _exact_kept(s["v"], case["bits"])
    q = s["q"]
    step = case["op"] == "step"
    if step:
        p = s["positions"].reshape(1, -1)
        turned_q = _exact_turn(q, p, case["d"], None, False, False)
        q = turned_q.to(q.dtype)
        k_new = _exact_turn(s["k_new"][:, 0], p, case["d"], None, False, False).to(q.dtype)
    out = torch.zeros(*q.shape, dtype=torch.float64, device=q.device)
    g = case["hq"] // case["hkv"]
    for i, (k, v) in enumerate(s["raw"]):
        if step:
            k, v = torch.cat([k, k_new[i][None]]), torch.cat([v, s["v_new"][i]])
        first = max(0, len(k) - (case.get("window") or len(k)))
        for c in range(case["hkv"]):
            kd, vd = (_exact_kept(x[first:, c], case["bits"]) for x in (k, v))
            x = q[i, c * g:(c + 1) * g].double() @ kd.t() / math.sqrt(case["d"])
            if case.get("softcap"):
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            if s["slope"] is not None:
                back = torch.arange(len(kd) - 1, -1, -1, device=x.device, dtype=torch.float64)
                x = x - s["slope"][c * g:(c + 1) * g, None].double() * back
            out[i, c * g:(c + 1) * g] = torch.softmax(x, 1) @ vd
    if step:
        return (out, turned_q, _exact_kept(k_new, case["bits"]),
                _exact_kept(s["v_new"][:, 0], case["bits"]))
    return out


def _exact_turn(x, positions, rot, axes, neighbours, inverse):
    """Each pair as a complex number times e^(i angle)."""
    y = x.double().clone()
    first = torch.arange(rot // 2, device=x.device) * (2 if neighbours else 1)
    second = first + (1 if neighbours else rot // 2)
    axes = torch.tensor(axes or [0] * (rot // 2), device=x.device)
    turn = torch.pow(torch.tensor(BASE, dtype=torch.float64, device=x.device),
                     torch.arange(rot // 2, device=x.device, dtype=torch.float64) * (-2.0 / rot))
    angle = positions.double()[axes].t() * turn * (-1.0 if inverse else 1.0)
    z = torch.complex(y[..., first], y[..., second]) * \
        torch.polar(torch.ones_like(angle), angle)[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_kept(x, bits):
    """What is read back of x [...][d] in 64 bits."""
    size, most = (x.shape[-1], 255) if bits == 8 else (32, 15)
    y = x.double().unflatten(-1, (-1, size))
    lo = y.min(-1, keepdim=True)[0]
    span = y.max(-1, keepdim=True)[0] - lo
    below = (span / most).to(x.dtype)
    for _ in range(2):  # the least number of the type that reaches
        below = torch.where(below.double() * most < span,
                            (below.view(torch.int16) + 1).view(x.dtype), below)
    step = below.double()
    code = torch.where(step > 0, torch.round((y - lo) / torch.where(step > 0, step, 1.0)), 0.0)
    return (lo + step * code).flatten(-2)
