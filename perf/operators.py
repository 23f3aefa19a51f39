"""Measured cases of the exact token cache's operators: rotary positions, the
append that rotates and stores a step's tokens, the attention of a batch over
one shared prefix and each sequence's own tokens (with the tokens' accumulated
attention weight), and the eviction of a cache's least-attended tokens.

`run` computes a case in plain torch operations (`own` false) or through the
package's entry points (`own` true); `exact` is the same result from the
definitions in 64 bits, one sequence or head at a time.
"""
import math

import numpy as np
import torch

own = False

D = 128  # head dimension of the cache
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the new token's query and key heads of 16 sequences (32 + 8 heads)
        _rotary("rotary_step_16", B=16, T=1, heads=40, dtype="bf16", dim=128, interleaved=False,
                scaling="bands", start=131000, heads_first=False, inverse=False),
        # one layer's keys of a 128K prompt, written in the index build's layout
        _rotary("rotary_prompt_128k", B=1, T=131072, heads=8, dtype="bf16", dim=128,
                interleaved=False, scaling="bands", start=0, heads_first=True, inverse=False),
        # half of the head rotated in pairs, backwards (gradients of rotated heads)
        _rotary("rotary_part_backward", B=3, T=5001, heads=28, dtype="fp16", dim=64,
                interleaved=True, scaling="yarn", start=7, heads_first=False, inverse=True),
        # a decode step of 16 sequences: rotate q and k, store k and v
        _append("append_step_16", B=16, T=1, H=8, G=4, cap=4096, length=2047, scaling="bands"),
        # a chunk of two prompts
        _append("append_chunk_4k", B=2, T=4096, H=8, G=4, cap=16384, length=8191,
                scaling="none"),
        # one short sequence, nothing shared: the smallest step
        _attend("attend_short", B=1, H=8, G=4, P=0, pad=0, cap=512, length=200, spread=0),
        # 16 sequences behind one 32K prefix
        _attend("attend_16_32k", B=16, H=8, G=4, P=32768, pad=0, cap=4096, length=2048,
                spread=700),
        # 5 sequences of 7 query heads per KV head, odd lengths, some without own tokens
        _attend("attend_odd_100k", B=5, H=4, G=7, P=100003, pad=61, cap=1600, length=1500,
                spread=1500),
        # a full batch behind a 128K prefix: the largest step
        _attend("attend_64_128k", B=64, H=8, G=4, P=131072, pad=0, cap=2048, length=1024,
                spread=300),
        # a full cache gives up one token per head, each step
        _evict("evict_one", B=16, H=8, cap=2112, length=2049, spread=0, budget=2048, into=0),
        # a cache of 8K tokens halved in place, ragged
        _evict("evict_half", B=16, H=8, cap=8192, length=8192, spread=2000, budget=4096, into=0),
        # a 128K prompt reduced to 8K tokens in a cache of its own
        _evict("evict_prompt_128k", B=1, H=8, cap=131072, length=131072, spread=0, budget=8192,
               into=9216),
    ]


def _rotary(name, **c):
    return {"name": name, "op": "rotary", **c}


def _append(name, **c):
    return {"name": name, "op": "append", **c}


def _attend(name, **c):
    return {"name": name, "op": "attend", **c}


def _evict(name, **c):
    return {"name": name, "op": "evict", **c}


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend", "evict"])
    scaling = rng.choice(["none", "linear", "ntk", "bands", "yarn"])
    if op == "rotary":
        heads = rng.randint(1, 40)
        T = _log(rng, 1, 131072)
        B = max(1, min(_log(rng, 1, 64), 1048576 // (T * heads)))
        return {"op": op, "B": B, "T": T, "heads": heads,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "dim": rng.choice([128, 128, 64, 96, 32, 20]),
                "interleaved": rng.random() < 0.5, "scaling": scaling,
                "start": rng.randint(0, 1000000), "heads_first": rng.random() < 0.5,
                "inverse": rng.random() < 0.3}
    H, G = rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
    if op == "append":
        T = _log(rng, 1, 4096)
        B = max(1, min(_log(rng, 1, 64), 8192 // T))
        length = rng.randint(0, 2048)
        return {"op": op, "B": B, "T": T, "H": H, "G": G, "cap": length + T + rng.randint(0, 300),
                "length": length, "scaling": scaling}
    if op == "attend":
        B = _log(rng, 1, 64)
        P = 0 if rng.random() < 0.15 else _log(rng, 1, 131072)
        length = _log(rng, 1, 4096)
        if B * H * length > 524288:
            length = 524288 // (B * H)
        return {"op": op, "B": B, "H": H, "G": G if B * H * G * P <= 1 << 28 else 1 + G // 2,
                "P": P, "pad": rng.choice([0, 0, 1, 77]), "cap": length + rng.randint(0, 500),
                "length": length, "spread": rng.randint(0, length)}
    length = _log(rng, 1, 131072)
    B = max(1, min(_log(rng, 1, 32), 1048576 // (H * length)))
    budget = max(1, int(length * rng.uniform(0.05, 1.1)))
    return {"op": op, "B": B, "H": H, "cap": length + rng.randint(0, 100), "length": length,
            "spread": rng.randint(0, length // 2), "budget": budget,
            "into": 0 if rng.random() < 0.6 else budget + rng.randint(0, 64)}


# -------------------------------------------------------------------- inputs
def _lengths(case):
    """Tokens of every (sequence, KV head): `length` minus a fixed share of `spread`."""
    b = np.arange(case["B"], dtype=np.int64)[:, None]
    h = np.arange(case["H"], dtype=np.int64)[None, :]
    cut = (b * 7919 + h * 104729) % (case["spread"] + 1) if case["spread"] else 0 * (b + h)
    return np.maximum(0, case["length"] - cut)


ORIGINAL = 8192  # trained length of the scaled variants
BASE = 500000.0
FACTOR = 16.0


def frequencies(dim, scaling):
    """Radians per position of each rotated pair, and the factor on the rotated values."""
    i = np.arange(dim // 2, dtype=np.float64)
    base = BASE
    if scaling == "ntk":
        base = BASE * FACTOR ** (dim / max(1.0, dim - 2.0))
    f = base ** (-2.0 * i / dim)
    if scaling == "linear":
        f = f / FACTOR
    elif scaling == "bands":  # long wavelengths slowed, short ones kept, a ramp between
        t = np.clip((ORIGINAL * f / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = (1 - t) * f / FACTOR + t * f
    elif scaling == "yarn":  # the ramp runs over the pairs' indices
        def turn(n):
            return dim * math.log(ORIGINAL / (n * 2 * math.pi)) / (2 * math.log(BASE))
        lo = max(math.floor(turn(32.0)), 0)
        hi = min(math.ceil(turn(1.0)), dim - 1)
        slow = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        f = slow * f / FACTOR + (1 - slow) * f
        return f, 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _cache(case, g, dev):
    B, H, cap = case["B"], case["H"], case["cap"]
    lens = torch.from_numpy(_lengths(case).astype(np.int32)).to(dev)
    centres = torch.randn((H, 64, D), generator=g, device=dev)
    pick = torch.randint(0, 64, (B, H, cap), generator=g, device=dev)
    K = torch.empty((B, H, cap, D), dtype=torch.bfloat16, device=dev)
    V = torch.empty((B, H, cap, D), dtype=torch.bfloat16, device=dev)
    for b in range(B):
        for h in range(H):
            K[b, h] = centres[h][pick[b, h]] + 0.3 * torch.randn((cap, D), generator=g, device=dev)
            V[b, h] = torch.randn((cap, D), generator=g, device=dev)
    return K, V, lens, centres


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 2 + 1)
    s = {"op": case["op"], "case": case}
    if case["op"] in ("rotary", "append"):
        dim = case.get("dim", D)
        f, s["mag"] = frequencies(dim, case["scaling"])
        s["freq"] = torch.from_numpy(f).to(dev)
        s["interleaved"] = bool(case.get("interleaved", False))
    if case["op"] == "rotary":
        B, T, heads = case["B"], case["T"], case["heads"]
        s["x"] = torch.randn((B, T, heads, D), generator=g, device=dev).to(DTYPES[case["dtype"]])
        s["pos"] = (case["start"] + torch.arange(T, device=dev, dtype=torch.int32)[None]
                    + torch.randint(0, 64, (B, 1), generator=g, device=dev, dtype=torch.int32))
        shape = (B, heads, T, D) if case["heads_first"] else (B, T, heads, D)
        out = torch.empty(shape, dtype=s["x"].dtype, device=dev)
        s["out"] = out.transpose(1, 2) if case["heads_first"] else out
        s["sign"] = -1.0 if case["inverse"] else 1.0
    elif case["op"] == "append":
        B, T, H, G, cap = case["B"], case["T"], case["H"], case["G"], case["cap"]
        # q, k and v are slices of one projection's output
        qkv = torch.randn((B, T, (G + 2) * H, D), generator=g, device=dev).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :, :G * H], qkv[:, :, G * H:(G + 1) * H], \
            qkv[:, :, (G + 1) * H:]
        s["K"] = torch.zeros((B, H, cap, D), dtype=torch.bfloat16, device=dev)
        s["V"] = torch.zeros_like(s["K"])
        s["pos"] = torch.full((B, H, cap), -1, dtype=torch.int32, device=dev)
        s["weight"] = torch.rand((B, H, cap), generator=g, device=dev)
        s["lens"] = torch.full((B, H), case["length"], dtype=torch.int32, device=dev)
        s["lens_out"] = torch.zeros_like(s["lens"])
        s["at"] = (100000 + torch.arange(T, device=dev, dtype=torch.int32)[None]
                   + torch.randint(0, 5000, (B, 1), generator=g, device=dev, dtype=torch.int32))
        s["q_out"] = torch.empty((B, T, G * H, D), dtype=torch.bfloat16, device=dev)
    elif case["op"] == "attend":
        B, H, G, P = case["B"], case["H"], case["G"], case["P"]
        s["K"], s["V"], s["lens"], centres = _cache(case, g, dev)
        s["pos"] = (P + torch.arange(case["cap"], device=dev, dtype=torch.int32)).expand(
            B, H, -1).contiguous()
        s["weight"] = torch.rand((B, H, case["cap"]), generator=g, device=dev)
        s["PK"] = s["PV"] = None
        if P:
            pk = torch.empty((H, P + case["pad"], D), dtype=torch.bfloat16, device=dev)
            pv = torch.empty_like(pk)
            for h in range(H):
                pick = torch.randint(0, 64, (pk.shape[1],), generator=g, device=dev)
                pk[h] = centres[h][pick] + 0.3 * torch.randn(pk[h].shape, generator=g, device=dev)
                pv[h] = torch.randn(pv[h].shape, generator=g, device=dev)
            s["PK"], s["PV"] = pk[:, :P], pv[:, :P]
        pick = torch.randint(0, 64, (B, H, G), generator=g, device=dev)
        q = 0.7 * centres[torch.arange(H, device=dev)[None, :, None], pick]
        q = q + 0.3 * torch.randn((B, H, G, D), generator=g, device=dev)
        s["q"] = q.reshape(B, H * G, D).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, H * G), dtype=torch.float32, device=dev)
    else:
        B, H, cap = case["B"], case["H"], case["cap"]
        s["K"], s["V"], s["lens"], _ = _cache(case, g, dev)
        # positions in no order, as earlier evictions leave them
        s["pos"] = torch.rand((B, H, cap), generator=g, device=dev).argsort(-1).to(torch.int32)
        w = torch.rand((B, H, cap), generator=g, device=dev)
        # a few tokens hold most of the weight; many share small values
        s["weight"] = torch.where(w > 0.5, (w ** 8) * 30.0, (w * 64).floor() / 256.0)
        s["first"], s["recent"] = (4, 64) if case["budget"] >= 128 else (0, 1)
        if case["into"]:
            s["oK"] = torch.zeros((B, H, case["into"], D), dtype=torch.bfloat16, device=dev)
            s["oV"] = torch.zeros_like(s["oK"])
        else:
            s["oK"], s["oV"] = s["K"], s["V"]
        rows = s["oK"].shape[2]
        s["opos"] = torch.full((B, H, rows), -1, dtype=torch.int32, device=dev)
        s["oweight"] = torch.zeros((B, H, rows), dtype=torch.float32, device=dev)
        s["olens"] = torch.zeros((B, H), dtype=torch.int32, device=dev)
    if own:
        _handles(s, case, dev)
    return s


def _handles(s, case, dev):
    """What a user's program keeps beside its tensors: the table, the cache, the scratch."""
    import kv_cache_vector_segmented_b200 as R
    if "freq" in s:
        s["table"] = R.RotaryTable.make(case.get("dim", D), base=BASE, scaling=case["scaling"],
                                        factor=FACTOR, original_len=ORIGINAL,
                                        interleaved=s["interleaved"], device=dev)
    if "K" in s:
        s["cache"] = R.TokenCache(s["K"], s["V"], s["pos"], s["weight"], s["lens"],
                                  group_size=case.get("G", 1))
    if case["op"] == "attend":
        s["ws"] = R.alloc_workspace(R.token_attend_workspace_bytes(s["cache"], case["P"]), dev)
        s["prefix"] = (s["PK"], s["PV"]) if case["P"] else None
    if case["op"] == "evict":
        s["ocache"] = R.TokenCache(s["oK"], s["oV"], s["opos"], s["oweight"], s["olens"],
                                   group_size=1)
        s["ws"] = R.alloc_workspace(R.token_evict_workspace_bytes(s["cache"], case["budget"]), dev)


# ----------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"rotary": _plain_rotary, "append": _plain_append, "attend": _plain_attend,
            "evict": _plain_evict}[s["op"]](s)


def _run_own(s):
    import kv_cache_vector_segmented_b200 as R
    if s["op"] == "rotary":
        return R.rotary(s["x"], s["pos"], s["table"], out=s["out"], inverse=s["sign"] < 0)
    if s["op"] == "append":
        R.token_append(s["cache"], s["k"], s["v"], s["at"], s["table"], q=s["q"],
                       q_out=s["q_out"], lens_out=s["lens_out"])
        return [s["q_out"], s["K"], s["V"], s["pos"], s["weight"], s["lens_out"]]
    if s["op"] == "attend":
        R.token_attend(s["q"], s["cache"], prefix=s["prefix"], out=s["out"], lse=s["lse"],
                       workspace=s["ws"])
        return [s["out"], s["lse"], s["weight"]]
    R.token_evict(s["cache"], s["case"]["budget"], keep_first=s["first"],
                  keep_recent=s["recent"], out=s["ocache"], workspace=s["ws"])
    return [s["oK"], s["oV"], s["opos"], s["oweight"], s["olens"]]


def _rotate(x, pos, freq, mag, sign, interleaved):
    """x [..., T, heads, d] in 32 bits, angles pos * freq in 64."""
    ang = pos.double()[..., None] * freq
    c, s = (ang.cos() * mag).float()[..., None, :], (ang.sin() * (mag * sign)).float()[..., None, :]
    n = freq.numel()
    x = x.float()
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _plain_rotary(s):
    s["out"].copy_(_rotate(s["x"], s["pos"], s["freq"], s["mag"], s["sign"], s["interleaved"]))
    return s["out"]


def _plain_append(s):
    T = s["at"].shape[1]
    B, H = s["lens"].shape
    q = _rotate(s["q"], s["at"], s["freq"], s["mag"], 1.0, False)
    k = _rotate(s["k"], s["at"], s["freq"], s["mag"], 1.0, False)
    slot = s["lens"].long()[..., None] + torch.arange(T, device=q.device)
    rows = slot[..., None].expand(B, H, T, D)
    s["q_out"].copy_(q)
    s["K"].scatter_(2, rows, k.transpose(1, 2).to(s["K"].dtype))
    s["V"].scatter_(2, rows, s["v"].transpose(1, 2))
    s["pos"].scatter_(2, slot, s["at"][:, None].expand(B, H, T))
    s["weight"].scatter_(2, slot, 0.0)
    torch.add(s["lens"], T, out=s["lens_out"])
    return [s["q_out"], s["K"], s["V"], s["pos"], s["weight"], s["lens_out"]]


def _plain_attend(s):
    B, H = s["lens"].shape
    cap = s["K"].shape[2]
    q = s["q"].float().view(B, H, -1, D) * D ** -0.5
    live = torch.arange(cap, device=q.device) < s["lens"][..., None]
    x = torch.matmul(q, s["K"].float().transpose(-1, -2))
    x = x.masked_fill(~live[:, :, None], float("-inf"))
    top = x.amax(-1)
    if s["PK"] is not None:
        y = torch.matmul(q.transpose(0, 1).reshape(H, -1, D), s["PK"].float().transpose(-1, -2))
        top = torch.maximum(top, y.amax(-1).view(H, B, -1).transpose(0, 1))
    base = top.masked_fill(top == float("-inf"), 0.0)
    e = torch.exp(x - base[..., None])
    den = e.sum(-1)
    num = torch.matmul(e, s["V"].float())
    if s["PK"] is not None:
        f = torch.exp(y - base.transpose(0, 1).reshape(H, -1, 1))
        den = den + f.sum(-1).view(H, B, -1).transpose(0, 1)
        num = num + torch.matmul(f, s["PV"].float()).view(H, B, -1, D).transpose(0, 1)
    safe = den.masked_fill(den == 0, 1.0)
    s["out"].copy_((num / safe[..., None]).reshape(B, -1, D))
    s["lse"].copy_((base + torch.log(den)).reshape(B, -1))
    s["weight"].add_((e / safe[..., None]).sum(2))
    return [s["out"], s["lse"], s["weight"]]


def _plain_evict(s):
    K, V, pos, weight, lens = s["K"], s["V"], s["pos"], s["weight"], s["lens"].long()
    B, H, cap = pos.shape
    i = torch.arange(cap, device=K.device)
    live = i < lens[..., None]
    newest = pos.masked_fill(~live, -2 ** 31).amax(-1, keepdim=True).long()
    held = live & ((pos < s["first"]) | (pos.long() > newest - s["recent"]))
    w = torch.where(weight.isnan(), float("-inf"), weight + 0.0)
    # by class (held, live, free), then weight, then place
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank = (live.int() + held.int()).gather(-1, order)
    order = order.gather(-1, torch.sort(rank, dim=-1, descending=True, stable=True).indices)
    keep = lens.clamp(max=s["case"]["budget"])[..., None]
    kept = torch.zeros_like(live).scatter_(-1, order, (i < keep).expand(B, H, cap))
    # the kept rows behind the first `keep` fill the gaps before them, in order
    hole, moved = ~kept & (i < keep), kept & (i >= keep)
    source = torch.sort(moved.int(), dim=-1, descending=True, stable=True).indices
    place = torch.where(hole, source.gather(-1, (hole.long().cumsum(-1) - 1).clamp(min=0)), i)
    W = min(s["case"]["budget"], cap)
    place = place[..., :W]
    used = (i[:W] < keep)
    rows = place[..., None].expand(B, H, W, D)
    s["oK"][:, :, :W] = torch.where(used[..., None], K.gather(2, rows), s["oK"][:, :, :W])
    s["oV"][:, :, :W] = torch.where(used[..., None], V.gather(2, rows), s["oV"][:, :, :W])
    s["opos"][:, :, :W] = torch.where(used, pos.gather(2, place), s["opos"][:, :, :W])
    s["oweight"][:, :, :W] = torch.where(used, weight.gather(2, place), s["oweight"][:, :, :W])
    s["olens"].copy_(keep[..., 0])
    return [s["oK"], s["oV"], s["opos"], s["oweight"], s["olens"]]


# ------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "attend": _exact_attend,
            "evict": _exact_evict}[case["op"]](s)


def _turned(x, pos, s, sign, interleaved):
    """Rotated heads in 64 bits, one complex product per pair."""
    n = s["freq"].numel()
    turn = torch.polar(torch.full((), s["mag"], dtype=torch.float64, device=x.device),
                       sign * pos.double()[..., None] * s["freq"])[..., None, :]
    y = x.double()
    pair = y[..., :2 * n].unflatten(-1, (n, 2) if interleaved else (2, n))
    pair = pair if interleaved else pair.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    z = z if interleaved else z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), y[..., 2 * n:]), -1)


def _exact_rotary(s):
    return _turned(s["x"], s["pos"], s, s["sign"], s["interleaved"])


def _exact_append(s):
    T, length = s["at"].shape[1], s["case"]["length"]
    K, V = s["K"].double(), s["V"].double()
    K[:, :, length:length + T] = _turned(s["k"], s["at"], s, 1.0, False).transpose(1, 2)
    V[:, :, length:length + T] = s["v"].transpose(1, 2).double()
    pos, weight = s["pos"].clone(), s["weight"].double()
    pos[:, :, length:length + T] = s["at"][:, None]
    weight[:, :, length:length + T] = 0.0
    return [_turned(s["q"], s["at"], s, 1.0, False), K, V, pos, weight, s["lens"] + T]


def _exact_attend(s):
    lens = s["lens"].cpu().tolist()
    B, H = s["lens"].shape
    G = s["q"].shape[1] // H
    q = s["q"].double().view(B, H, G, D)
    out, lse = torch.zeros_like(q), torch.full((B, H, G), float("-inf"), dtype=torch.float64,
                                               device=q.device)
    weight = s["weight"].double()
    for h in range(H):
        pk = s["PK"][h].double() if s["PK"] is not None else q.new_zeros((0, D))
        pv = s["PV"][h].double() if s["PK"] is not None else q.new_zeros((0, D))
        for b in range(B):
            n = lens[b][h]
            if n + pk.shape[0] == 0:
                continue
            x = torch.cat((q[b, h] @ pk.T, q[b, h] @ s["K"][b, h, :n].double().T), 1)
            x = x / math.sqrt(D)
            lse[b, h] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b, h][:, None])
            out[b, h] = p[:, :pk.shape[0]] @ pv + p[:, pk.shape[0]:] @ s["V"][b, h, :n].double()
            weight[b, h, :n] += p[:, pk.shape[0]:].sum(0)
    return [out.view(B, H * G, D), lse.view(B, H * G), weight]


def _exact_evict(s):
    lens, pos = s["lens"].cpu().numpy(), s["pos"].cpu().numpy()
    weight = s["weight"].double().cpu().numpy()
    oK, oV = s["oK"].clone(), s["oV"].clone()
    opos, oweight, olens = s["opos"].clone(), s["oweight"].double(), s["olens"].clone()
    for b in range(lens.shape[0]):
        for h in range(lens.shape[1]):
            n = int(lens[b, h])
            m = min(n, s["case"]["budget"])
            olens[b, h] = m
            if m == 0:
                continue
            p, w = pos[b, h, :n].astype(np.int64), weight[b, h, :n]
            held = (p < s["first"]) | (p > p.max() - s["recent"])
            best = np.lexsort((np.arange(n), -w, ~held))[:m]
            place = np.arange(m)
            kept = np.zeros(n, dtype=bool)
            kept[best] = True
            place[~kept[:m]] = m + np.nonzero(kept[m:])[0]
            at = torch.from_numpy(place).to(oK.device)
            oK[b, h, :m], oV[b, h, :m] = s["K"][b, h][at], s["V"][b, h][at]
            opos[b, h, :m], oweight[b, h, :m] = s["pos"][b, h][at], s["weight"][b, h][at].double()
    return [oK, oV, opos, oweight, olens]


# ---------------------------------------------------------------------- work
def work(case):
    if case["op"] == "rotary":
        n = case["B"] * case["T"] * case["heads"]
        size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
        return {"bytes": 2 * n * D * size + 4 * case["B"] * case["T"], "flops": 3 * n * case["dim"]}
    if case["op"] == "append":
        n = case["B"] * case["T"] * case["H"]
        return {"bytes": n * (case["G"] + 2) * D * 4 + n * 8 + 8 * case["B"] * case["H"],
                "flops": 3 * n * (case["G"] + 1) * D}
    lens = _lengths(case)
    units = case["B"] * case["H"]
    if case["op"] == "attend":
        rows = case["H"] * case["P"] + int(lens.sum())
        heads = units * case["G"]
        return {"bytes": rows * D * 4 + int(lens.sum()) * 8 + heads * (D * 4 + 4) + units * 4,
                "flops": 4 * D * case["G"] * (units * case["P"] + int(lens.sum()))}
    keep = np.minimum(lens, case["budget"])
    # into another cache every kept row moves; in place, about the kept share of those behind
    moved = keep if case["into"] else (lens - keep) * keep / np.maximum(lens, 1)
    return {"bytes": int(lens.sum()) * 8 + int(moved.sum()) * D * 8 + int(keep.sum()) * 8
            + units * 8, "flops": int(lens.sum())}
