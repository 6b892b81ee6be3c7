"""The operators that decode over a cache which is scored, evicted from and held in 4 bits.

Four operators, measured at the sizes of this repository's workloads (a compressed layer, the ragged
decode batch, grouped queries over 16384 rows, a 131072-row cache) and at drawn ones:

  attend   decode attention over a dense cache that adds every row's weight to a running score
  q4       the same over a cache whose rows are held in 4 bits (with or without the score)
  write    rows quantised into a 4-bit cache, and read back as the values they stand for
  evict    the lightest rows of a full cache dropped in place, dense or 4-bit

A 4-bit row is, for each group of 64 channels, a step h and a centre z in bf16 and a level
t = 2u - 15 (u = 0..15) per channel; it stands for z + h t.
"""
import math

import torch

own = False

GROUP = 64
SIGN_BIT = (15, 14, 7, 6)     # of channels 2j (low half) and 2j + 1 (high half) of a 32-bit word
MAG_BIT = (3, 0, 11, 8)


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: one short fp32 head per query, where latency is all
        dict(name="attend tiny fp32", op="attend", batch=1, heads=4, group=1, d=64, cap=83, short=0.0, dtype="fp32",
             decay=1.0),
        # one layer of a 7B-shaped model right after its prompt was compressed to 1024 + 32 rows
        dict(name="attend layer", op="attend", batch=1, heads=32, group=1, d=128, cap=1057, short=0.0, dtype="bf16",
             decay=1.0),
        # grouped queries, uncompressed caches of ragged lengths
        dict(name="attend grouped", op="attend", batch=8, heads=8, group=4, d=128, cap=16384, short=0.5,
             dtype="bf16", decay=0.9),
        # the same layer as above with its cache in 4 bits
        dict(name="q4 layer scored", op="q4", batch=1, heads=32, group=1, d=128, cap=1057, short=0.0, dtype="bf16",
             decay=1.0, scored=True),
        # the decode batch: 64 sequences, 2048 + 32 kept rows and up to 128 new ones
        dict(name="q4 decode batch", op="q4", batch=64, heads=32, group=1, d=128, cap=2208, short=0.06,
             dtype="bf16", decay=1.0, scored=False),
        dict(name="q4 grouped scored", op="q4", batch=8, heads=8, group=4, d=128, cap=16384, short=0.5,
             dtype="bf16", decay=1.0, scored=True),
        # one sequence's long context, uncompressed
        dict(name="q4 long", op="q4", batch=1, heads=32, group=1, d=128, cap=131072, short=0.0, dtype="bf16",
             decay=1.0, scored=False),
        # the new token of every sequence of the decode batch
        dict(name="write step", op="write", batch=64, heads=32, rows=1, d=128, cap=2208, dtype="bf16"),
        # a whole prompt's keys and values
        dict(name="write prompt", op="write", batch=1, heads=32, rows=16384, d=128, cap=16385, dtype="bf16"),
        # a short cache in 4 bits
        dict(name="evict tiny q4", op="evict", batch=1, heads=4, d=64, cap=97, keep=49, recent=32, q4=True,
             dtype="fp32"),
        # the decode batch's caches, full after 128 steps, back to 2048 + 32 rows
        dict(name="evict decode batch", op="evict", batch=64, heads=32, d=128, cap=2208, keep=2048, recent=32,
             q4=False, dtype="bf16"),
        # a long cache brought down by an eighth
        dict(name="evict long", op="evict", batch=1, heads=32, d=128, cap=131072, keep=114624, recent=64, q4=False,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "q4", "q4", "write", "evict"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    batch = _log_int(rng, 1, 64)
    heads = rng.choice([1, 2, 4, 5, 8, 12, 16, 32])
    most = (1 << 22) // (batch * heads)          # cached rows over all heads: 4 Mi, as the largest listed case
    if dtype == "fp32":
        most //= 2
    cap = _log_int(rng, 17, max(18, min(131072, most)))
    case = dict(op=op, batch=batch, heads=heads, d=d, cap=cap, dtype=dtype)
    if op in ("attend", "q4"):
        case.update(group=rng.choice([1, 1, 2, 3, 4, 7, 8, 16]), short=rng.choice([0.0, 0.1, 0.5, 1.0]),
                    decay=rng.choice([1.0, 1.0, 0.9, 0.0]))
        if op == "q4":
            case.update(scored=rng.random() < 0.5)
    elif op == "write":
        # rows over all heads: 512 Ki, as the prompt of the listed cases
        case.update(rows=_log_int(rng, 1, max(1, min(cap - 1, (1 << 19) // (batch * heads)))))
    else:
        held = max(2, int(cap * rng.uniform(0.5, 0.98)))
        recent = min(held - 1, rng.choice([0, 1, 16, 32, 64, 200]))
        case.update(keep=held - recent, recent=recent, q4=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _rows(g, shape, dtype, scale=None):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if scale is not None:
        x *= scale
    return x.to(dtype)


def _pack(u):
    """Level numbers u (0..15) [..., d] as the cache's words, returned as bytes [..., d / 2]."""
    d = u.shape[-1]
    e = u.to(torch.int32).reshape(*u.shape[:-1], d // GROUP, GROUP // 8, 4, 2)   # group, word, pair, half
    neg = (e < 8).to(torch.int32)
    mag = torch.where(e < 8, 7 - e, e - 8)
    half = torch.zeros_like(e[..., 0, :])
    for j in range(4):
        half |= (neg[..., j, :] << SIGN_BIT[j]) | (mag[..., j, :] << MAG_BIT[j])
    word = half[..., 0] | (half[..., 1] << 16)
    return word.transpose(-1, -2).flatten(-2).contiguous().view(torch.uint8)


def _cache_tensors(g, case):
    """A 4-bit cache's codes and (h, z) pairs: rows of normal values, quantised sequence by sequence."""
    B, H, cap, d = case["batch"], case["heads"], case["cap"], case["d"]
    out = {}
    for name in ("k", "v"):
        scale = torch.rand((H, 1, d), generator=g, device="cuda") * 1.5 + 0.5 if name == "k" else None
        codes = torch.empty((B, H, cap, d // 2), dtype=torch.uint8, device="cuda")
        meta = torch.empty((B, H, cap, d // GROUP, 2), dtype=torch.bfloat16, device="cuda")
        step = max(1, (1 << 25) // (H * d))
        for b in range(B):
            for r in range(0, cap, step):
                n = min(step, cap - r)
                u, h, z = _levels(_rows(g, (H, n, d), torch.bfloat16, scale))
                codes[b, :, r:r + n] = _pack(u)
                meta[b, :, r:r + n, :, 0] = h
                meta[b, :, r:r + n, :, 1] = z
        out[name + "_codes"], out[name + "_meta"] = codes, meta
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, d, cap, dt = case["batch"], case["heads"], case["d"], case["cap"], _dtype(case)
    s = {"case": dict(case)}
    if case["op"] in ("attend", "q4"):
        # lengths: full, or down to a share `short` below it
        cut = torch.rand((B,), generator=g, device="cuda") * case["short"]
        s["len"] = (cap - (cut * cap).floor()).clamp_(1, cap).to(torch.int32)
        s["q"] = _rows(g, (B, H * case["group"], d), dt, 1.5)
        if case["op"] == "q4":
            s.update(_cache_tensors(g, case))
        else:
            s["k"] = _rows(g, (B, H, cap, d), dt, torch.rand((H, 1, d), generator=g, device="cuda") * 1.5 + 0.5)
            s["v"] = _rows(g, (B, H, cap, d), dt)
        if case.get("scored", True):
            # what the steps so far have left: weights of a few dozen queries
            s["score"] = torch.rand((B, H, cap), generator=g, device="cuda").pow_(4) * (64.0 / cap)
            s["score"].masked_fill_(torch.arange(cap, device="cuda") >= s["len"][:, None, None], 0.0)
    elif case["op"] == "write":
        s["k"] = _rows(g, (B, H, case["rows"], d), dt, torch.rand((H, 1, d), generator=g, device="cuda") * 1.5 + 0.5)
        s["v"] = _rows(g, (B, H, case["rows"], d), dt)
        room = cap - case["rows"]
        s["len"] = torch.randint(0, room + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        for n in ("k", "v"):
            s[n + "_codes"] = torch.zeros((B, H, cap, d // 2), dtype=torch.uint8, device="cuda")
            s[n + "_meta"] = torch.zeros((B, H, cap, d // GROUP, 2), dtype=torch.bfloat16, device="cuda")
    else:
        s["len"] = torch.full((B,), cap, dtype=torch.int32, device="cuda")
        if B > 1:   # one sequence is not full yet and keeps all its rows
            s["len"][-1] = case["keep"] + case["recent"]
        # a running score: a few heavy rows, many light ones, some never attended (equal: the lower slot stays)
        score = torch.rand((B, H, cap), generator=g, device="cuda").pow_(6)
        score.masked_fill_(torch.rand((B, H, cap), generator=g, device="cuda") < 0.02, 0.0)
        score.masked_fill_(torch.arange(cap, device="cuda") >= s["len"][:, None, None], 0.0)
        s["score_now"], s["score"] = score, torch.empty_like(score)
        if case["q4"]:
            s.update(_cache_tensors(g, case))
        else:
            s["k"], s["v"] = _rows(g, (B, H, cap, d), dt), _rows(g, (B, H, cap, d), dt)
    return s


# -------------------------------------------------------------------------------------- plain forms

def _levels(x):
    """Level numbers and the bf16 pair (h, z) of rows x [..., d]: in 64 bits, as rows of 16-bit values meet ties."""
    x = x.double().unflatten(-1, (-1, GROUP))
    hi, lo = x.amax(-1), x.amin(-1)
    h = ((hi - lo) / 30.0).float().to(torch.bfloat16)
    h = torch.where(h.float() < 2.0 ** -126, torch.zeros_like(h), h)
    z = ((hi + lo) / 2.0).float().to(torch.bfloat16)
    step = torch.where(h > 0, 2.0 * h.double(), torch.full_like(hi, torch.inf))
    u = ((x - z.double()[..., None]) / step[..., None] + 7.5).round().clamp(0, 15)
    return u.flatten(-2).float(), h, z


def _values(codes, meta):
    """The fp32 values that codes [..., d / 2] with pairs [..., d / 64, 2] stand for."""
    ng = meta.shape[-2]
    word = codes.contiguous().view(torch.int32).unflatten(-1, (GROUP // 8, ng)).transpose(-1, -2)
    e = torch.arange(8, device=word.device, dtype=torch.int32)
    half = (word[..., None] >> (16 * (e & 1))) & 0xFFFF
    sign = torch.tensor(SIGN_BIT, dtype=torch.int32, device=word.device)[(e >> 1).long()]
    mag = torch.tensor(MAG_BIT, dtype=torch.int32, device=word.device)[(e >> 1).long()]
    t = (1 - 2 * ((half >> sign) & 1)) * (2 * ((half >> mag) & 7) + 1)
    t = t.flatten(-2).float()
    return (meta[..., 1:].float() + meta[..., :1].float() * t).flatten(-2)


def _attend(s, k, v, length, score, decay):
    """softmax attention of q over k, v [B, H, cap, d] in fp32; adds the weights to score in place."""
    q = s["q"].float()
    B, H, cap, d = k.shape
    group = q.shape[1] // H
    seen = torch.arange(cap, device=q.device) < length[:, None, None, None]                  # [B, 1, 1, cap]
    logits = (q.view(B, H, group, d) @ k.transpose(-1, -2)) / math.sqrt(d)
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = (logits - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = p @ v.masked_fill(~seen.transpose(-1, -2), 0.0)
    if score is not None:
        added = p.sum(2) + (decay * score if decay else 0.0)
        score.copy_(torch.where(seen[:, :, 0], added, score))
    return out.view(B, H * group, d).to(s["q"].dtype)


def _evict_source(case, score, length):
    """The slot that each slot's row comes from, and the new lengths."""
    B, H, cap = score.shape
    keep, recent = case["keep"], case["recent"]
    at = torch.arange(cap, device=score.device)
    n = (length - recent)[:, None, None]                                  # rows up to here may go
    full = (length > keep + recent)[:, None, None]
    ranked = torch.where(at < n, score, -torch.inf).sort(dim=-1, descending=True, stable=True).indices
    stays = torch.zeros((B, H, cap), dtype=torch.bool, device=score.device)
    stays.scatter_(-1, ranked[..., :keep], True)
    hole, mover = ~stays & (at < keep), stays & (at >= keep)
    # the i-th hole takes the i-th mover
    order = torch.where(mover, at, cap).sort(dim=-1).values
    nth = (hole.cumsum(-1) - 1).clamp_min(0)
    source = torch.where(hole, order.gather(-1, nth), at)
    source = torch.where((at >= keep) & (at < keep + recent), at - keep + n, source)
    source = torch.where(full, source, at)
    return source.clamp_max(cap - 1), torch.minimum(length, torch.full_like(length, keep + recent))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "attend":
        out = _attend(s, s["k"].float(), s["v"].float(), s["len"], s["score"], case["decay"])
        return {"out": out, "score": s["score"]}
    if op == "q4":
        score = s.get("score")
        out = _attend(s, _values(s["k_codes"], s["k_meta"]), _values(s["v_codes"], s["v_meta"]), s["len"], score,
                      case["decay"])
        return {"out": out} if score is None else {"out": out, "score": score}
    if op == "write":
        B, H, rows, d = s["k"].shape
        res = {"len": s["len"] + rows}
        for n in ("k", "v"):
            u, h, z = _levels(s[n])
            t = (2.0 * u - 15.0).unflatten(-1, (-1, GROUP))
            res[n] = (z.float()[..., None] + h.float()[..., None] * t).flatten(-2).to(s[n].dtype)
        return res
    s["score"].copy_(s["score_now"])
    source, length = _evict_source(case, s["score"], s["len"])
    res = {"len": length}
    for n in ("k", "v", "k_codes", "k_meta", "v_codes", "v_meta"):
        if n in s:
            flat = s[n].flatten(3)
            flat.copy_(flat.gather(2, source[..., None].expand(-1, -1, -1, flat.shape[-1])))
    moved = s["score"].gather(-1, source)
    s["score"].copy_(moved.masked_fill(torch.arange(case["cap"], device=source.device) >= length[:, None, None], 0.0))
    res["score"] = s["score"]
    res["source"] = source[..., :case["keep"] + case["recent"]].to(torch.int32)
    if case["q4"]:
        res["k"] = _values(s["k_codes"], s["k_meta"]).to(_dtype(case))
        res["v"] = _values(s["v_codes"], s["v_meta"]).to(_dtype(case))
    else:
        res["k"], res["v"] = s["k"], s["v"]
    return res


def _kernels(s):
    import kv_cache_compression_gb300 as kv
    case = s["case"]
    op = case["op"]
    if op == "attend":
        out = kv.decode_attend_scored(s["q"], s["k"], s["v"], s["len"], s["score"], decay=case["decay"])
        return {"out": out, "score": s["score"]}
    cache = kv.Q4Cache(s["k_codes"], s["k_meta"], s["v_codes"], s["v_meta"]) if "k_codes" in s else None
    if op == "q4":
        score = s.get("score")
        out = kv.q4_decode_attend(s["q"], cache, s["len"], score, decay=case["decay"])
        return {"out": out} if score is None else {"out": out, "score": score}
    if op == "write":
        length = kv.q4_append(cache, s["k"], s["v"], s["len"])
        k, v = kv.q4_read(cache, s["k"].shape[2], start=s["len"], dtype=s["k"].dtype)
        return {"len": length, "k": k, "v": v}
    s["score"].copy_(s["score_now"])
    if case["q4"]:
        length, source = kv.q4_evict(cache, s["score"], s["len"], keep=case["keep"], recent=case["recent"])
        k, v = kv.q4_read(cache, case["cap"], dtype=_dtype(case))
    else:
        length, source = kv.evict(s["k"], s["v"], s["score"], s["len"], keep=case["keep"], recent=case["recent"])
        k, v = s["k"], s["v"]
    return {"len": length, "score": s["score"], "source": source, "k": k, "v": v}


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------- floors

def work(case):
    B, H, d, cap = case["batch"], case["heads"], case["d"], case["cap"]
    e = 4 if case["dtype"] == "fp32" else 2
    q4_row = d // 2 + 4 * (d // GROUP)
    if case["op"] in ("attend", "q4"):
        held = cap * (1.0 - case["short"] / 2) * B * H
        row = 2 * (q4_row if case["op"] == "q4" else d * e)
        if case.get("scored", True):
            row += 8 if case["decay"] else 4
        return {"bytes": held * row + 2 * B * H * case["group"] * d * e, "flops": 4.0 * held * case["group"] * d}
    if case["op"] == "write":
        rows = B * H * case["rows"]
        # rows in, the 4-bit rows out, and in again for the values that are returned
        return {"bytes": rows * 2 * (2 * d * e + 2 * q4_row), "flops": 10.0 * rows * 2 * d}
    full = B - 1 if B > 1 else 1
    keep, recent = case["keep"], case["recent"]
    gone = cap - keep - recent
    # of the keep + gone rows in question, those below `keep` that go are replaced
    moved = keep * gone / (keep + gone) + recent
    row = 2 * (q4_row if case["q4"] else d * e) + 4
    data = full * H * (4 * cap + 2 * moved * row) + B * H * 4 * (keep + recent)
    if case["q4"]:   # the values that the cache then stands for
        data += B * H * cap * 2 * (q4_row + e * d)
    return {"bytes": data, "flops": 4.0 * B * H * cap}


# ------------------------------------------------------------------------------------------- exact

def _exact_row_values(codes, meta):
    """float64 values of rows [..., d / 2], channel by channel from the words' bit fields."""
    d, ng = 2 * codes.shape[-1], meta.shape[-2]
    word = codes.contiguous().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
    out = torch.empty((*codes.shape[:-1], d), dtype=torch.float64, device=codes.device)
    h, z = meta[..., 0].double(), meta[..., 1].double()
    for c in range(d):
        g, e = c // GROUP, c % 8
        bits = word[..., ng * ((c % GROUP) // 8) + g] >> (16 * (e % 2))
        t = 2 * ((bits >> MAG_BIT[e // 2]) & 7) + 1
        t = torch.where(((bits >> SIGN_BIT[e // 2]) & 1) == 1, -t, t)
        out[..., c] = z[..., g] + h[..., g] * t
    return out


def exact(case, seed):
    s = prepare(case, seed)
    B, H, cap, d = case["batch"], case["heads"], case["cap"], case["d"]
    op = case["op"]
    if op in ("attend", "q4"):
        group = case["group"]
        out = torch.zeros((B, H * group, d), dtype=torch.float64, device="cuda")
        score = s["score"].double() if "score" in s else None
        for b in range(B):
            n = int(s["len"][b])
            if op == "q4":
                k = _exact_row_values(s["k_codes"][b, :, :n], s["k_meta"][b, :, :n])
                v = _exact_row_values(s["v_codes"][b, :, :n], s["v_meta"][b, :, :n])
            else:
                k, v = s["k"][b, :, :n].double(), s["v"][b, :, :n].double()
            for h in range(H):
                for i in range(group):
                    w = torch.softmax(torch.mv(k[h], s["q"][b, h * group + i].double()) * d ** -0.5, 0)
                    out[b, h * group + i] = torch.mv(v[h].t(), w)
                    if score is not None:
                        if i == 0:
                            score[b, h, :n] *= case["decay"]
                        score[b, h, :n] += w
        return {"out": out} if score is None else {"out": out, "score": score}
    if op == "write":
        res = {"len": s["len"] + case["rows"]}
        for n in ("k", "v"):
            full = torch.empty(s[n].shape, dtype=torch.float64, device="cuda")
            for g in range(d // GROUP):
                x = s[n][..., g * GROUP:(g + 1) * GROUP].double()
                top, low = x.max(-1, keepdim=True).values, x.min(-1, keepdim=True).values
                h = ((top - low) / 30).to(torch.bfloat16).double()
                z = ((top + low) / 2).to(torch.bfloat16).double()
                u = torch.clamp(torch.round((x - z) / (2 * h) + 7.5), 0, 15)
                full[..., g * GROUP:(g + 1) * GROUP] = z + h * (2 * u - 15)
            res[n] = full
        return res
    # rows are only moved: the values are the inputs' own, put where a slot-by-slot walk puts them
    import numpy as np
    keep, recent = case["keep"], case["recent"]
    score, length = s["score_now"].cpu().numpy(), s["len"].cpu().numpy()
    source = np.tile(np.arange(cap), (B, H, 1))
    for b in range(B):
        n = int(length[b]) - recent
        if length[b] <= keep + recent:
            continue
        for h in range(H):
            kept = np.sort(np.argsort(-score[b, h, :n], kind="stable")[:keep])
            free = np.setdiff1d(np.arange(keep), kept)
            source[b, h, free] = kept[kept >= keep]
            source[b, h, keep:keep + recent] = np.arange(n, n + recent)
    new = np.minimum(length, keep + recent)
    moved = np.take_along_axis(score.astype(np.float64), source, -1)
    for b in range(B):
        moved[b, :, new[b]:] = 0.0
    res = {"len": torch.from_numpy(new), "score": torch.from_numpy(moved),
           "source": torch.from_numpy(source[..., :keep + recent].astype(np.int32))}
    at = torch.from_numpy(source).cuda()
    for n in ("k", "v"):
        x = _exact_row_values(s[n + "_codes"], s[n + "_meta"]) if case["q4"] else s[n].double()
        res[n] = x.gather(2, at[..., None].expand(-1, -1, -1, d))
    return res
