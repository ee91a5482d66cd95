"""Measured cases of the 8-bit cache operators: writing rows into a cache held in
8 bits, attending over it, accounting for the attention each row received, and
evicting the rows that received least.

``own`` false: every operator in its plain form, elementary torch operations in
32 bits.  ``own`` true: the calls a user makes of this package.
"""

import math

import torch

own = False

#: Largest code of each 8-bit format: a block's largest magnitude maps onto it.
TOP = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "bf16": torch.bfloat16}
#: A block's largest magnitude is taken as at least this, so that its inverse is finite.
TINY = 2.0 ** -100


def listed():
    return [
        # one new token, few heads, a short selection: pure latency
        dict(name="attend_one_token", op="attend", batch=1, heads=16, kv_heads=1, d=128, T=500, k=64, W=0, block=16,
             fmt="e4m3", shared=False, sink=False, holes=0.0),
        # the decode step of 8 sequences: 128 heads on one embedding of 512, 1024 selected rows and a window of 128
        dict(name="attend_decode", op="attend", batch=8, heads=128, kv_heads=1, d=512, T=32768, k=1024, W=128, block=64,
             fmt="e4m3", shared=False, sink=True, holes=0.0),
        # grouped heads on several KV heads, odd lengths, skipped slots and ragged windows
        dict(name="attend_grouped_ragged", op="attend", batch=5, heads=40, kv_heads=8, d=192, T=5001, k=333, W=77,
             block=32, fmt="int8", shared=False, sink=True, holes=0.2),
        # a prompt piece of 512 tokens over one shared cache, the longest selection
        dict(name="attend_prompt", op="attend", batch=512, heads=128, kv_heads=1, d=512, T=32768, k=2048, W=0,
             block=128, fmt="e4m3", shared=True, sink=False, holes=0.0),
        # a decode step's new row of each of 8 sequences, a scale for each row
        dict(name="write_append", op="write", batch=8, n=1, kv_heads=1, d=512, T=32768, block=1, fmt="e4m3", ragged=False),
        # ragged prompts written into a grouped-head cache
        dict(name="write_grouped_ragged", op="write", batch=3, n=1001, kv_heads=8, d=192, T=2048, block=16, fmt="int8",
             ragged=True),
        # long prompts of 8 sequences, written whole
        dict(name="write_prompt", op="write", batch=8, n=16384, kv_heads=1, d=512, T=32768, block=64, fmt="e4m3",
             ragged=False),
        # the account after a decode step
        dict(name="mass_decode", op="mass", batch=8, heads=128, kv_heads=1, d=512, T=32768, k=1024, block=64,
             fmt="e4m3", shared=False, holes=0.0),
        # the account over a grouped-head cache in 16 bits, odd sizes, skipped slots
        dict(name="mass_grouped_bf16", op="mass", batch=5, heads=40, kv_heads=8, d=192, T=5001, k=333, block=1,
             fmt="bf16", shared=False, holes=0.2),
        # one sequence, row by row
        dict(name="evict_one_rows", op="evict", batch=1, T=4096, kv_heads=1, d=128, block=1, budget=2048, first=4,
             last=128, fmt="int8", ragged=False),
        # 5 ragged sequences with an open last block, grouped heads
        dict(name="evict_grouped_ragged", op="evict", batch=5, T=10007, kv_heads=8, d=192, block=16, budget=301, first=1,
             last=3, fmt="int8", ragged=True),
        # 8 full caches halved
        dict(name="evict_half", op="evict", batch=8, T=32768, kv_heads=1, d=512, block=64, budget=256, first=1, last=2,
             fmt="e4m3", ragged=False),
    ]


def _log(rng, lo, hi):
    """A whole number, uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "mass", "evict"])
    d = 64 * rng.randint(1, 8)
    block = 2 ** rng.randint(0, 7)
    kv_heads = rng.choice([1, 1, 1, 2, 4, 8])
    fmt = rng.choice(["e4m3", "int8"])
    if op in ("attend", "mass"):
        heads = kv_heads * _log(rng, 1, 128 // kv_heads)
        shared = rng.random() < 0.3
        batch = _log(rng, 1, 512 if shared else 16)
        T = _log(rng, 64, 32768)
        k = _log(rng, 1, min(T, 2048))
        c = dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, d=d, T=T, k=k, block=block, fmt=fmt, shared=shared,
                 holes=rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.5), 2)]))
        while kv_heads * batch * k * d > 512 * 2048 * 512 // 2:
            batch = c["batch"] = max(1, batch // 2)
        while kv_heads * T * d * (1 if shared else batch) > 8 * 32768 * 512:
            T = c["T"] = max(k, T // 2)
            if T == k:
                batch = c["batch"] = max(1, batch // 2)
        if op == "attend":
            c.update(W=rng.choice([0, _log(rng, 1, 256)]), sink=rng.random() < 0.5)
        elif rng.random() < 0.4:
            c.update(fmt="bf16", block=1)
        return c
    batch = _log(rng, 1, 16)
    T = _log(rng, 128, 32768)
    while kv_heads * batch * T * d > 8 * 32768 * 512:
        T //= 2
    c = dict(op=op, batch=batch, kv_heads=kv_heads, d=d, T=T, block=block, fmt=fmt, ragged=rng.random() < 0.5)
    if op == "write":
        c.update(n=_log(rng, 1, T // 2))
    else:
        blocks = -(-T // block)
        budget = max(1, int(blocks * rng.uniform(0.2, 0.9)))
        c.update(budget=budget, first=rng.randint(0, min(4, budget // 2)), last=rng.randint(0, min(8, budget // 2)))
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, *shape):
    """Embedding rows: unit normal, each row at a level of its own."""
    return (_normal(g, *shape) * torch.exp(0.3 * _normal(g, *shape[:-1], 1))).to(torch.bfloat16)


def _write_plain(x, block, fmt):
    """Codes and scales of whole rows x [B, n, heads, d] (the last block may be short)."""
    B, n, H, d = x.shape
    nb = -(-n // block)
    pad = torch.zeros(B, nb * block, H, d, device=x.device)
    pad[:, :n] = x.float()
    y = pad.view(B, nb, block, H, d)
    a = y.abs().amax(dim=(2, 4)).clamp_min(TINY)
    top = torch.full_like(a, TOP[fmt])
    inv, s = torch.div(top, a), torch.div(a, top)
    v = y * inv[:, :, None, :, None]
    v = v.round() if fmt == "int8" else v
    return v.to(DTYPE[fmt]).view(B, nb * block, H, d)[:, :n], s


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"] in ("attend", "mass"):
        B, H, K, d, T, k = c["batch"], c["heads"], c["kv_heads"], c["d"], c["T"], c["k"]
        x = _rows(g, 1 if c["shared"] else B, T, K, d)
        if c["fmt"] == "bf16":
            cache, s["scales"] = x, None
        else:
            cache, s["scales"] = _write_plain(x, c["block"], c["fmt"])
            cache = cache.contiguous()
        if c["shared"]:
            cache = cache[0] if c["fmt"] != "bf16" or K == 1 else cache[0].expand(B, T, K, d)
            s["scales"] = None if s["scales"] is None else s["scales"][0]
        if c["fmt"] == "bf16" and K == 1:
            cache = cache.reshape(cache.shape[:-2] + (d,))
        s["cache"] = cache
        s["q"] = _normal(g, B, H, d).to(torch.bfloat16)
        idx = torch.rand(B, T, generator=g, device="cuda").topk(k, dim=1).indices
        hole = torch.rand(B, k, generator=g, device="cuda") < c["holes"]
        s["idx"] = torch.where(hole, -1, idx).to(torch.int32)
        s["scale"] = 1.0 / math.sqrt(d)
        if c["op"] == "attend":
            W = c["W"]
            s["win"] = _rows(g, B, W, K, d) if W else None
            s["win_len"] = torch.randint(0, W + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if W and c["holes"] else None
            s["sink"] = _normal(g, H) if c["sink"] else None
        else:
            # the log of a softmax's normaliser over these rows: log k + 1/2 in the mean
            s["lse"] = math.log(k) + 0.5 + 0.3 * _normal(g, B, H)
            s["mass"] = 20.0 * torch.rand(B, T, generator=g, device="cuda")
        return s
    B, K, d, T, block = c["batch"], c["kv_heads"], c["d"], c["T"], c["block"]
    nb = -(-T // block)
    if c["op"] == "write":
        n = c["n"]
        s["rows"] = _rows(g, B, n, K, d)
        s["codes"] = torch.zeros(B, T, K, d, dtype=DTYPE[c["fmt"]], device="cuda")
        s["scales"] = torch.zeros(B, nb, K, device="cuda")
        # each sequence starts at a block of its own, so that the rows fit
        s["pos"] = (torch.randint(0, (T - n) // block + 1, (B,), generator=g, device="cuda") * block).to(torch.int32)
        s["length"] = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if c["ragged"] else None
        return s
    s["codes"], s["scales"] = _write_plain(_rows(g, B, T, K, d), block, c["fmt"])
    s["codes"] = s["codes"].contiguous()
    # attention received: a long tail over the rows
    s["mass"] = torch.exp(2.0 * _normal(g, B, T))
    lo = T // 2
    s["length"] = torch.randint(lo, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if c["ragged"] else \
        torch.full((B,), T, dtype=torch.int32, device="cuda")
    m = c["budget"]
    s["to_codes"] = torch.zeros(B, m * block, K, d, dtype=DTYPE[c["fmt"]], device="cuda")
    s["to_scales"] = torch.zeros(B, m, K, device="cuda")
    s["to_mass"] = torch.zeros(B, m * block, device="cuda")
    return s


# ---------------------------------------------------------------- the operators

def _gathered(s):
    """The selected rows in 32 bits [B, kv_heads, k, d], zero where the slot is skipped, and which are not."""
    c = s["case"]
    B, K, d, T = c["batch"], c["kv_heads"], c["d"], c["T"]
    ok = s["idx"] >= 0
    r = torch.where(ok, s["idx"], 0).long()
    cache = s["cache"].view(s["cache"].shape[:-1] + (1, d)) if s["cache"].dim() == (2 if c["shared"] else 3) and c["fmt"] == "bf16" else s["cache"]
    b = torch.arange(B, device="cuda")[:, None]
    alone = cache.dim() == 3
    rows = (cache[r] if alone else cache[b, r]).float()
    if s["scales"] is not None:
        n = r // c["block"]
        rows = rows * (s["scales"][n] if alone else s["scales"][b, n])[..., None]
    return torch.where(ok[:, :, None, None], rows, 0.0).transpose(1, 2), ok


def _scores(s, rows):
    c = s["case"]
    q = s["q"].float().view(c["batch"], c["kv_heads"], -1, c["d"])
    return torch.matmul(q, rows.transpose(-1, -2)) * s["scale"]


def _attend(s):
    c = s["case"]
    B, H, d = c["batch"], c["heads"], c["d"]
    rows, ok = _gathered(s)
    if s["win"] is not None:
        w = torch.arange(c["W"], device="cuda")
        has = (w < s["win_len"][:, None]) if s["win_len"] is not None else (w >= 0).expand(B, c["W"])
        win = torch.where(has[:, :, None, None], s["win"].float(), 0.0)
        rows, ok = torch.cat([rows, win.transpose(1, 2)], 2), torch.cat([ok, has], 1)
    z = torch.where(ok[:, None, None, :], _scores(s, rows), -math.inf)
    top = z.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, c["kv_heads"], -1, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - top)
    out = torch.matmul(e, rows) / torch.where(total == 0.0, 1.0, total)
    return out.reshape(B, H, d).to(torch.bfloat16), (top + torch.log(total)).reshape(B, H)


def _mass(s):
    c = s["case"]
    rows, ok = _gathered(s)
    w = torch.exp(_scores(s, rows) - s["lse"].view(c["batch"], c["kv_heads"], -1, 1)).sum((1, 2))
    return s["mass"].scatter_add_(1, torch.where(ok, s["idx"], 0).long(), torch.where(ok, w, 0.0))


def _write(s):
    c = s["case"]
    B, K, d, n, block = c["batch"], c["kv_heads"], c["d"], c["n"], c["block"]
    length = s["length"] if s["length"] is not None else torch.full((B,), n, device="cuda")
    r = torch.arange(n, device="cuda")
    has = r < length[:, None]
    codes, scales = _write_plain(torch.where(has[:, :, None, None], s["rows"], 0.0), block, c["fmt"])
    b = torch.arange(B, device="cuda")[:, None]
    at = s["pos"][:, None].long() + r
    s["codes"].view(torch.uint8)[b, at] = torch.where(has[:, :, None, None], codes.view(torch.uint8), s["codes"].view(torch.uint8)[b, at])
    m = torch.arange(scales.shape[1], device="cuda")
    at = s["pos"][:, None].long() // block + m
    s["scales"][b, at] = torch.where((m * block < length[:, None])[:, :, None], scales, s["scales"][b, at])
    return s["codes"], s["scales"]


def _evict(s):
    c = s["case"]
    B, T, block, m = c["batch"], c["T"], c["block"], c["budget"]
    nb = -(-T // block)
    length = s["length"][:, None].long()
    r = torch.arange(nb * block, device="cuda")
    mass = torch.zeros(B, nb * block, dtype=torch.float64, device="cuda")
    mass[:, :T] = s["mass"]
    # in 64 bits: a block next to the border of what stays must not change sides with the order of its sum
    key = torch.where(r < length, mass, 0.0).view(B, nb, block).sum(-1).float()
    n, has = torch.arange(nb, device="cuda"), -(-length // block)
    key = torch.where((n < c["first"]) | (n >= has - c["last"]), math.inf, key)
    key = torch.where(n < has, key, -math.inf)
    kept = key.sort(dim=1, descending=True, stable=True).indices[:, :m]
    kept = torch.where(kept < has, kept, nb).sort(dim=1).values
    there = kept < nb
    src = (kept[:, :, None] * block + torch.arange(block, device="cuda")).view(B, -1)
    stays = there.repeat_interleave(block, 1) & (src < length)
    src, blk, b = torch.where(stays, src, 0), torch.where(there, kept, 0), torch.arange(B, device="cuda")[:, None]
    u8 = torch.uint8
    s["to_codes"].view(u8).copy_(torch.where(stays[:, :, None, None], s["codes"].view(u8)[b, src], s["to_codes"].view(u8)))
    s["to_scales"].copy_(torch.where(there[:, :, None], s["scales"][b, blk], s["to_scales"]))
    s["to_mass"].copy_(torch.where(stays, s["mass"][b, src], s["to_mass"]))
    return torch.where(there, kept, -1).to(torch.int32), stays.sum(1).to(torch.int32), s["to_codes"], s["to_scales"], s["to_mass"]


def run(state):
    s, c = state, state["case"]
    if own:
        import sparse_attention_top_ds_b200 as ds
        if c["op"] == "attend":
            return ds.ds_sparse_attention_q8(s["q"], s["cache"], s["scales"], s["idx"], c["block"], scale=s["scale"], win=s["win"],
                                             win_len=s["win_len"], sink=s["sink"], return_lse=True)
        if c["op"] == "mass":
            return ds.ds_attention_mass(s["q"], s["cache"], s["idx"], s["lse"], s["mass"], scales=s["scales"], block=c["block"],
                                        scale=s["scale"])
        if c["op"] == "write":
            return ds.ds_cache_quantize(s["rows"], s["codes"], s["scales"], c["block"], pos=s["pos"], length=s["length"])
        kept, new_length = ds.ds_cache_evict(s["mass"], c["budget"], block=c["block"], length=s["length"], keep_first=c["first"],
                                             keep_last=c["last"])
        ds.ds_cache_compact(kept, block=c["block"], length=s["length"], rows=[(s["codes"], s["to_codes"]), (s["mass"], s["to_mass"])],
                            blocks=[(s["scales"], s["to_scales"])])
        return kept, new_length, s["to_codes"], s["to_scales"], s["to_mass"]
    return {"attend": _attend, "mass": _mass, "write": _write, "evict": _evict}[c["op"]](s)


def work(case):
    c = case
    B, K, d, T, block = c["batch"], c["kv_heads"], c["d"], c["T"], c["block"]
    if c["op"] in ("attend", "mass"):
        H, k = c["heads"], c["k"]
        live = max(1, int(k * (1.0 - c["holes"])))
        rows = min(T, B * live) if c["shared"] else B * live
        size = 2 if c["fmt"] == "bf16" else 1
        b = rows * K * (d * size + (0 if size == 2 else 4.0 / block)) + 4 * B * k + 2 * B * H * d + 4 * B * H
        if c["op"] == "mass":
            return {"bytes": b + 8 * B * live, "flops": 2 * B * H * live * d}
        W = c["W"] / 2 if c["holes"] else c["W"]
        return {"bytes": b + 2 * B * H * d + 2 * B * W * K * d, "flops": 4 * B * H * (live + W) * d}
    if c["op"] == "write":
        n = c["n"] / 2 if c["ragged"] else c["n"]
        return {"bytes": B * K * n * (3 * d + 4.0 / block) + 8 * B, "flops": 2 * B * K * n * d}
    m = c["budget"]
    L = 0.75 * T if c["ragged"] else T
    stay = min(m * block, L)
    return {"bytes": B * (4 * L + 2 * stay * (K * d + 4) + 8 * K * m + 4 * m + 8), "flops": B * L}


# ---------------------------------------------------------------- in 64 bits

def _exact_rows(s, b):
    """The rows that batch row b selects, [slots, kv_heads, d] in 64 bits, and their positions."""
    c = s["case"]
    idx = s["idx"][b].long()
    idx = idx[idx >= 0]
    cache = s["cache"]
    mine = cache if (c["shared"] and cache.dim() < 4) else cache[b]
    rows = mine.index_select(0, idx) if c["fmt"] == "bf16" else mine.view(torch.uint8).index_select(0, idx).view(DTYPE[c["fmt"]])
    rows = rows.double().reshape(len(idx), c["kv_heads"], c["d"])
    if s["scales"] is not None:
        sc = s["scales"] if s["scales"].dim() == 2 else s["scales"][b]
        rows = rows * sc.double().index_select(0, torch.div(idx, c["block"], rounding_mode="floor")).unsqueeze(-1)
    return rows, idx


def _exact_e4m3(v):
    """v in 64 bits at the nearest e4m3 value, ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    B, K, d = c["batch"], c["kv_heads"], c["d"]
    if c["op"] == "attend":
        G = c["heads"] // K
        out, lse = [], []
        for b in range(B):
            rows, _ = _exact_rows(s, b)
            if s["win"] is not None:
                live = c["W"] if s["win_len"] is None else int(s["win_len"][b])
                rows = torch.cat([rows, s["win"][b, :live].double()])
            z = torch.einsum("kgd,nkd->kgn", s["q"][b].double().view(K, G, d), rows) * s["scale"]
            both = z if s["sink"] is None else torch.cat([z, s["sink"].double().view(K, G, 1)], -1)
            if both.shape[-1] == 0:
                out.append(torch.zeros(K * G, d, dtype=torch.float64, device="cuda"))
                lse.append(torch.full((K * G,), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            total = torch.logsumexp(both, -1, keepdim=True)
            out.append(torch.einsum("kgn,nkd->kgd", torch.exp(z - total), rows).reshape(K * G, d))
            lse.append(total.reshape(-1))
        return torch.stack(out), torch.stack(lse)
    if c["op"] == "mass":
        G = c["heads"] // K
        acc = s["mass"].double()
        for b in range(B):
            rows, idx = _exact_rows(s, b)
            z = torch.einsum("kgd,nkd->kgn", s["q"][b].double().view(K, G, d), rows) * s["scale"]
            acc[b, idx] += torch.exp(z - s["lse"][b].double().view(K, G, 1)).sum((0, 1))
        return acc
    if c["op"] == "write":
        codes, scales, n, block = s["codes"].double(), s["scales"].double(), c["n"], c["block"]
        top = TOP[c["fmt"]]
        for b in range(B):
            live, p = n if s["length"] is None else int(s["length"][b]), int(s["pos"][b])
            x = s["rows"][b, :live].double()
            if live == 0:
                continue
            whole = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -live % block)).view(-1, block, K, d)
            sc = whole.abs().amax((1, 3)).clamp_min(TINY) / top
            scales[b, p // block : p // block + len(sc)] = sc
            if c["fmt"] == "e4m3":
                codes[b, p : p + live] = _exact_e4m3(x / sc.repeat_interleave(block, 0)[:live, :, None])
        return (codes if c["fmt"] == "e4m3" else None), scales
    return None
