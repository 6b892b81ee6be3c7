"""The operators that verify several drafted tokens at a time over a cache, dense or held in 8 bits.

Five operators, measured at the sizes of this repository's workloads (a compressed layer, the decode batch of 64
sequences, grouped queries over 16384 rows, a 131072-row cache, a 16384-row prompt) and at drawn ones:

  tree     attention of a tree of drafted tokens: every token sees the cached rows and, of the drafted ones, those
           that its mask names (its ancestors and itself)
  cross    several tokens' attention to cached states alone, of another length (an encoder's), without drafted rows
  q8       tree over a cache whose rows are held in 8 bits
  write    a prompt's rows quantised to 8 bits, and read back as the values they stand for
  commit   the accepted tokens' rows, picked out of the drafted ones and appended to the cache (dense or 8 bits)

An 8-bit row is a step h (fp32) and, for each channel, a sign (bit 7) and a magnitude u of 0..127; it stands for
the values +-u h.
"""
import math

import torch

own = False

SMALLEST_STEP = 2.0 ** -80   # rows whose step would be smaller are held as zeros


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: one token's cross attention to a few fp32 states, where latency is all
        dict(name="cross tiny fp32", op="cross", batch=1, heads=4, group=1, d=64, tokens=1, cap=83, short=0.0,
             ragged=False, dtype="fp32"),
        # a batch of prompts that read their encoders' states
        dict(name="cross prompt", op="cross", batch=16, heads=16, group=1, d=64, tokens=440, cap=1500, short=0.3,
             ragged=True, dtype="bf16"),
        # one layer of a 7B-shaped model whose prompt was compressed to 1024 + 32 rows, eight drafted tokens
        dict(name="tree layer", op="tree", batch=1, heads=32, group=1, d=128, tokens=8, cap=1057, short=0.0,
             ragged=False, dtype="bf16"),
        # grouped queries over uncompressed caches of ragged lengths, sixteen drafted tokens
        dict(name="tree grouped", op="tree", batch=8, heads=8, group=4, d=128, tokens=16, cap=16384, short=0.5,
             ragged=True, dtype="bf16"),
        # a wide tree over long caches
        dict(name="tree wide", op="tree", batch=4, heads=8, group=4, d=128, tokens=64, cap=32768, short=0.1,
             ragged=False, dtype="bf16"),
        # the same shape of call in fp32
        dict(name="tree grouped fp32", op="tree", batch=8, heads=8, group=4, d=128, tokens=7, cap=8192, short=0.5,
             ragged=True, dtype="fp32"),
        # a single new token over one sequence's long context
        dict(name="q8 token", op="q8", batch=1, heads=32, group=1, d=128, tokens=1, cap=131072, short=0.0,
             ragged=False, dtype="bf16"),
        # the decode batch: 64 sequences, 2048 + 32 kept rows and up to 128 new ones, six drafted tokens each
        dict(name="q8 decode batch", op="q8", batch=64, heads=32, group=1, d=128, tokens=6, cap=2208, short=0.06,
             ragged=True, dtype="bf16"),
        # a tree of 32 tokens with grouped queries
        dict(name="q8 grouped", op="q8", batch=8, heads=8, group=4, d=128, tokens=32, cap=16384, short=0.5,
             ragged=False, dtype="bf16"),
        # a whole prompt's keys and values
        dict(name="write prompt", op="write", batch=1, heads=32, d=128, rows=16384, cap=16385, dtype="bf16"),
        # what the decode batch accepts of sixteen drafted tokens, up to six, in 8 bits
        dict(name="commit q8 batch", op="commit", batch=64, heads=32, d=128, tokens=16, most=6, cap=2208, q8=True,
             dtype="bf16"),
        # longer accepted runs of a wide tree, dense
        dict(name="commit dense", op="commit", batch=16, heads=8, d=128, tokens=64, most=33, cap=4111, q8=False,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "cross", "q8", "q8", "write", "commit"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    batch = _log_int(rng, 1, 64)
    heads = rng.choice([1, 2, 4, 5, 8, 12, 16, 32])
    case = dict(op=op, batch=batch, heads=heads, d=d, dtype=dtype)
    most = (1 << 22) // (batch * heads)          # cached rows over all heads: 4 Mi, as the longest listed case
    if op in ("tree", "cross", "q8"):
        if op != "q8":
            most //= 4 if dtype == "bf16" else 8
        group = rng.choice([1, 1, 2, 3, 4, 7, 8])
        tokens = _log_int(rng, 1, 512 if op == "cross" else 96)
        cap = _log_int(rng, 17, max(18, min(131072, most)))
        # products in all: as the wide tree's, fp32 an eighth
        limit = (1 << 30) if dtype == "bf16" else (1 << 27)
        while batch * heads * group * tokens * cap > limit:
            if tokens > 1:
                tokens = (tokens + 1) // 2
            else:
                cap = max(17, cap // 2)
                if cap == 17:
                    break
        case.update(group=group, tokens=tokens, cap=cap, short=rng.choice([0.0, 0.1, 0.5, 1.0]),
                    ragged=rng.random() < 0.5)
    elif op == "write":
        if dtype == "fp32":
            most //= 2
        cap = _log_int(rng, 17, max(18, min(131072, most)))
        case.update(cap=cap, rows=_log_int(rng, 1, max(1, min(cap - 1, (1 << 18) // (batch * heads)))))
    else:
        tokens = _log_int(rng, 1, 128)
        cap = _log_int(rng, 17, max(18, min(32768, most // 8)))
        case.update(tokens=tokens, most=min(cap - 1, tokens, _log_int(rng, 1, 48)), cap=cap, q8=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _rows(g, shape, dtype, scale=None):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if scale is not None:
        x *= scale
    return x.to(dtype)


def _codes(u):
    """Signed level numbers as bytes of sign and magnitude."""
    u = u.to(torch.int16)
    return (u.abs() + (u < 0).to(torch.int16) * 128).to(torch.uint8)


def _q8_tensors(g, case, scale):
    """An 8-bit cache's codes and steps: rows of normal values, quantised piece by piece."""
    B, H, cap, d = case["batch"], case["heads"], case["cap"], case["d"]
    out = {}
    for name in ("k", "v"):
        codes = torch.empty((B, H, cap, d), dtype=torch.uint8, device="cuda")
        steps = torch.empty((B, H, cap), dtype=torch.float32, device="cuda")
        piece = max(1, (1 << 25) // (H * d))
        for b in range(B):
            for r in range(0, cap, piece):
                n = min(piece, cap - r)
                u, h = _levels(_rows(g, (H, n, d), torch.bfloat16, scale if name == "k" else None))
                codes[b, :, r:r + n] = _codes(u)
                steps[b, :, r:r + n] = h
        out[name + "_codes"], out[name + "_step"] = codes, steps
    return out


def _tree(g, B, T):
    """Masks [B, T, T] of random trees: token i hangs on one of the last few before it, or on the cached text."""
    parent = torch.arange(T, device="cuda") - 1 - torch.randint(0, 4, (B, T), generator=g, device="cuda")
    seq = torch.arange(B, device="cuda")
    mask = torch.zeros((B, T, T), dtype=torch.bool, device="cuda")
    for i in range(T):
        p = parent[:, i]
        mask[:, i] = mask[seq, p.clamp_min(0)] & (p >= 0)[:, None]
        mask[:, i, i] = True
    return mask


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, d, cap, dt = case["batch"], case["heads"], case["d"], case["cap"], _dtype(case)
    s = {"case": dict(case)}
    scale = torch.rand((H, 1, d), generator=g, device="cuda") * 1.5 + 0.5      # channels of K differ in size
    if case["op"] in ("tree", "cross", "q8"):
        T = case["tokens"]
        # lengths: full, or down to a share `short` below it
        cut = torch.rand((B,), generator=g, device="cuda") * case["short"]
        s["len"] = (cap - (cut * cap).floor()).clamp_(0, cap).to(torch.int32)
        if case["ragged"]:    # sequences with fewer tokens than the call has room for
            s["n"] = torch.randint(1, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["q"] = _rows(g, (B, H * case["group"], T, d), dt, 1.5)
        if case["op"] != "cross":
            s["k_new"] = _rows(g, (B, H, T, d), dt, scale)
            s["v_new"] = _rows(g, (B, H, T, d), dt)
            s["mask"] = _tree(g, B, T)
        if case["op"] == "q8":
            s.update(_q8_tensors(g, case, scale))
        else:
            s["k"] = _rows(g, (B, H, cap, d), dt, scale)
            s["v"] = _rows(g, (B, H, cap, d), dt)
        return s
    rows = case["rows"] if case["op"] == "write" else case["tokens"]
    most = case.get("most", rows)
    s["k_new"] = _rows(g, (B, H, rows, d), dt, scale)
    s["v_new"] = _rows(g, (B, H, rows, d), dt)
    s["len"] = torch.randint(0, cap - most + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] == "commit":
        # a path down the tree: ascending tokens, of which a sequence takes the first few (or none)
        s["pick"] = torch.rand((B, rows), generator=g, device="cuda").argsort(-1)[:, :most].sort(-1).values.to(torch.int32)
        s["n"] = torch.randint(0, most + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] == "write" or case["q8"]:
        for n in ("k", "v"):
            s[n + "_codes"] = torch.zeros((B, H, cap, d), dtype=torch.uint8, device="cuda")
            s[n + "_step"] = torch.zeros((B, H, cap), dtype=torch.float32, device="cuda")
    else:
        s["k"], s["v"] = _rows(g, (B, H, cap, d), dt, scale), _rows(g, (B, H, cap, d), dt)
    return s


# -------------------------------------------------------------------------------------- plain forms

def _levels(x):
    """Signed level numbers and steps of rows x [..., d]: in 64 bits, as rows of 16-bit values meet ties."""
    x = x.double()
    h = (x.abs().amax(-1) / 127.0).float()
    h = torch.where(h < SMALLEST_STEP, torch.zeros_like(h), h)
    step = torch.where(h > 0, h.double(), torch.full_like(h, torch.inf, dtype=torch.float64))
    return (x / step[..., None]).round().clamp(-127, 127).float(), h


def _values(codes, step):
    """The fp32 values that codes [..., d] with steps [...] stand for."""
    c = codes.to(torch.int16)
    u = torch.where(c > 127, 128 - c, c)
    return u.float() * step[..., None]


def _attend(s, k, v):
    """Attention of all tokens to k, v [B, H, cap, d] and to the drafted rows that the mask names, in fp32."""
    B, H, cap, d = k.shape
    q = s["q"].float()
    T, G = q.shape[2], q.shape[1] // H
    count = s["n"] if "n" in s else torch.full((B,), T, dtype=torch.int32, device="cuda")
    at, token = torch.arange(cap, device="cuda"), torch.arange(T, device="cuda")
    live = token < count[:, None]                                                           # [B, T]
    seen = (at < s["len"][:, None])[:, None, :].expand(B, T, cap)                           # [B, T, rows]
    v = v.masked_fill(~(at < s["len"][:, None])[:, None, :, None], 0.0)
    if "k_new" in s:
        seen = torch.cat([seen, s["mask"] & live[:, None, :]], -1)
        k = torch.cat([k, s["k_new"].float()], 2)
        v = torch.cat([v, s["v_new"].float()], 2)
    seen = (seen & live[:, :, None])[:, None, None]                                         # [B, 1, 1, T, rows]
    logits = (q.view(B, H, G * T, d) @ k.transpose(-1, -2)).view(B, H, G, T, -1) / math.sqrt(d)
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = (logits - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).view(B, H * G, T)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = p.view(B, H, G * T, -1) @ v
    return {"out": out.view(B, H * G, T, d).to(s["q"].dtype), "lse": lse}


def _picked(s, name):
    """The rows that a call appends, [B, H, most, d], and how many of them each sequence takes."""
    x = s[name + "_new"]
    if "pick" not in s:
        return x, torch.full((x.shape[0],), x.shape[2], dtype=torch.int32, device="cuda")
    index = s["pick"].long()[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3])
    return x.gather(2, index), s["n"]


def _put(s, name, rows, count):
    """rows [B, H, most, ...] into the state's tensor at slots len .. len + count - 1."""
    old = s[name]
    most = rows.shape[2]
    slot = s["len"].long()[:, None] + torch.arange(most, device="cuda")                     # [B, most]
    index = slot.view(slot.shape[0], 1, most, *([1] * (old.dim() - 3))).expand_as(rows)
    taken = (torch.arange(most, device="cuda") < count[:, None]).view(index.shape[0], 1, most, *([1] * (old.dim() - 3)))
    old.scatter_(2, index, torch.where(taken, rows, old.gather(2, index)))


def _read(s, name, most, dtype):
    slot = s["len"].long()[:, None] + torch.arange(most, device="cuda")
    step = s[name + "_step"]
    index = slot[:, None, :].expand(-1, step.shape[1], -1)
    codes = s[name + "_codes"].gather(2, index[..., None].expand(-1, -1, -1, s[name + "_codes"].shape[-1]))
    return _values(codes, step.gather(2, index)).to(dtype)


def _plain(s):
    case = s["case"]
    if case["op"] in ("tree", "cross"):
        return _attend(s, s["k"].float(), s["v"].float())
    if case["op"] == "q8":
        return _attend(s, _values(s["k_codes"], s["k_step"]), _values(s["v_codes"], s["v_step"]))
    res = {}
    for n in ("k", "v"):
        rows, count = _picked(s, n)
        if "k_codes" in s:
            u, h = _levels(rows)
            _put(s, n + "_codes", _codes(u), count)
            _put(s, n + "_step", h, count)
            res[n] = _read(s, n, rows.shape[2], rows.dtype)
        else:
            _put(s, n, rows, count)
            res[n] = s[n]
    res["len"] = s["len"] + count
    return res


def _kernels(s):
    import kv_cache_compression_gb300 as kv
    case = s["case"]
    if case["op"] in ("tree", "cross", "q8"):
        lse = torch.empty(s["q"].shape[:3], dtype=torch.float32, device="cuda")
        drafts = (s["k_new"], s["v_new"], s["mask"]) if "k_new" in s else ()
        if case["op"] == "q8":
            cache = kv.Q8Cache(s["k_codes"], s["k_step"], s["v_codes"], s["v_step"])
            out = kv.q8_tree_attend(s["q"], cache, s["len"], *drafts, n_new=s.get("n"), lse=lse)
        else:
            out = kv.tree_attend(s["q"], s["k"], s["v"], s["len"], *drafts, n_new=s.get("n"), lse=lse)
        return {"out": out, "lse": lse}
    if "k_codes" in s:
        cache = kv.Q8Cache(s["k_codes"], s["k_step"], s["v_codes"], s["v_step"])
        length = kv.q8_append(cache, s["k_new"], s["v_new"], s["len"], n_new=s.get("n"), pick=s.get("pick"))
        k, v = kv.q8_read(cache, case.get("most", case.get("rows")), start=s["len"], dtype=s["k_new"].dtype)
    else:
        k, v = s["k"], s["v"]
        length = kv.append_rows(k, v, s["k_new"], s["v_new"], s["len"], n_new=s.get("n"), pick=s.get("pick"))
    return {"k": k, "v": v, "len": length}


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------- floors

def work(case):
    B, H, d, cap = case["batch"], case["heads"], case["d"], case["cap"]
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("tree", "cross", "q8"):
        T = case["tokens"] * (0.5 if case["ragged"] else 1.0)     # tokens that are there, on average
        M = B * H * case["group"]
        held = B * H * cap * (1.0 - case["short"] / 2)
        data = held * 2 * (d + 4 if case["op"] == "q8" else d * e)
        data += M * T * d * e + M * case["tokens"] * (d * e + 4)
        flops = 4.0 * held * case["group"] * T * d
        if case["op"] != "cross":
            data += 2 * B * H * T * d * e + B * T * T
            flops += 4.0 * M * T * T * d
        return {"bytes": data, "flops": flops}
    if case["op"] == "write":
        # rows in, the 8-bit rows out, and in again for the values that are returned
        rows = B * H * case["rows"]
        return {"bytes": rows * 2 * (2 * d * e + 2 * (d + 4)), "flops": 6.0 * rows * 2 * d}
    rows = B * H * case["most"] / 2
    data = rows * 2 * (d * e + (d + 4 if case["q8"] else d * e)) + B * 4 * (case["most"] / 2 + 3)
    if case["q8"]:
        data += B * H * case["most"] * 2 * (d + 4 + d * e)
    return {"bytes": data, "flops": 6.0 * rows * 2 * d}


# ------------------------------------------------------------------------------------------- exact

def _exact_rows(s, n, b, h, upto):
    """float64 rows 0 .. upto - 1 of one head of K or V."""
    if n in s:
        return s[n][b, h, :upto].double()
    codes = s[n + "_codes"][b, h, :upto]
    return (codes & 127).double() * (1.0 - 2.0 * (codes >> 7).double()) * s[n + "_step"][b, h, :upto, None].double()


def exact(case, seed):
    s = prepare(case, seed)
    B, H, d = case["batch"], case["heads"], case["d"]
    if case["op"] in ("tree", "cross", "q8"):
        G, T = case["group"], case["tokens"]
        out = torch.zeros((B, H * G, T, d), dtype=torch.float64, device="cuda")
        lse = torch.full((B, H * G, T), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            rows = int(s["len"][b])
            n = int(s["n"][b]) if "n" in s else T
            for h in range(H):
                k, v = _exact_rows(s, "k", b, h, rows), _exact_rows(s, "v", b, h, rows)
                hidden = torch.zeros((n, rows), dtype=torch.float64, device="cuda")
                if "k_new" in s:
                    k = torch.cat([k, s["k_new"][b, h, :n].double()])
                    v = torch.cat([v, s["v_new"][b, h, :n].double()])
                    drafted = torch.zeros((n, n), dtype=torch.float64, device="cuda")
                    drafted[~s["mask"][b, :n, :n]] = -math.inf
                    hidden = torch.cat([hidden, drafted], 1)
                if k.shape[0] == 0:
                    continue
                for i in range(h * G, (h + 1) * G):
                    x = torch.einsum("td,rd->tr", s["q"][b, i, :n].double(), k) * d ** -0.5 + hidden
                    lse[b, i, :n] = torch.logsumexp(x, 1)
                    out[b, i, :n] = torch.softmax(x, 1) @ v
        return {"out": out, "lse": lse}
    res = {"len": s["len"] + (s["n"] if "n" in s else case["rows"])}
    for n in ("k", "v"):
        new = s[n + "_new"]
        most = case.get("most", case.get("rows"))
        q8 = n + "_codes" in s
        full = torch.zeros((B, H, most, d), dtype=torch.float64, device="cuda") if q8 else s[n].double()
        for b in range(B):
            count = int(s["n"][b]) if "n" in s else most
            x = new[b, :, s["pick"][b, :count].long()] if "pick" in s else new[b]
            x = x.double()
            if not q8:
                at = int(s["len"][b])
                full[b, :, at:at + count] = x
                continue
            h = (x.abs().max(-1, keepdim=True).values / 127).float().double()
            u = torch.round(x.abs() / h) * torch.sign(x)
            full[b, :, :count] = torch.where(h >= SMALLEST_STEP, u * h, torch.zeros_like(u))
        res[n] = full
    return res
