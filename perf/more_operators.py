"""Operators between a decoder block's Q/K/V layers and its O layer: the cases they are measured at.

Three operators, each with the plain form that says what it computes and the call that a user makes of the library:

  rotate  every head of queries and keys RMS-normalised and rotated by its token's position
  append  new keys and values rounded to 8 bits into the pages of a cache, with a scale per page and head (a power of two;
          a page whose scale has to grow has its earlier codes rounded again), queries and keys normalised and rotated in the
          same call where the case says so
  attend  causal attention of new tokens over such a cache, all of it or a sliding window and a few first tokens

A batch holds B sequences; the new tokens of sequence b are rows offsets[b] .. offsets[b+1]-1, at the last of its lens[b]
positions.  A sequence's tokens lie in the pages that its row of the table names, `page` tokens each.  Keys are stored
(page, head, token, dim), values (page, head, dim, token).

Sizes follow the library's block workload (4096 wide: 32 heads of 128) and generic ones with fewer key/value heads.
"""
import math

import torch

own = False

INT8, E4M3 = 0, 1
TOP = {INT8: 127.0, E4M3: 448.0}                           # the largest code's value
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # rotation
        # one decoded token, fewer key heads than query heads
        dict(name="rotate_t1_h32_8_d128", op="rotate", T=1, H=32, Hkv=8, D=128, dims=128, paired=False, norm=True,
             packed=True),
        # a prefill batch of the block workload
        dict(name="rotate_t2048_h32_32_d128", op="rotate", T=2048, H=32, Hkv=32, D=128, dims=128, paired=False, norm=True,
             packed=False),
        # append
        # one decoded token of the block workload, with norm and rotation of its queries and keys
        dict(name="append_b1_n1_h32_32_rot", op="append", B=1, n=1, len=777, H=32, Hkv=32, D=128, page=64, fmt=E4M3,
             rotary=True),
        # a decoded batch: one token for each of 64 sequences in small pages
        dict(name="append_b64_n1_h32_8_p16", op="append", B=64, n=1, len=2049, H=32, Hkv=8, D=128, page=16, fmt=INT8,
             rotary=False),
        # a prefill of 2048 tokens with norm and rotation
        dict(name="append_b1_n2048_h32_32_rot", op="append", B=1, n=2048, len=2048, H=32, Hkv=32, D=128, page=64, fmt=E4M3,
             rotary=True),
        # attention
        # one decoded token, a short context: nothing but latency
        dict(name="attend_b1_n1_l333_h32_32", op="attend", B=1, n=1, len=333, H=32, Hkv=32, D=128, page=64, fmt=INT8,
             window=0, sinks=0),
        # one decoded token, a long context
        dict(name="attend_b1_n1_l32768_h32_8", op="attend", B=1, n=1, len=32768, H=32, Hkv=8, D=128, page=64, fmt=E4M3,
             window=0, sinks=0),
        # a decoded batch of ragged contexts in small pages
        dict(name="attend_b64_n1_l8192_h32_8_p16", op="attend", B=64, n=1, len=8192, H=32, Hkv=8, D=128, page=16, fmt=INT8,
             window=0, sinks=0),
        # a decoded batch over a sliding window with first tokens that stay
        dict(name="attend_b16_n1_w4096_s4_h32_32", op="attend", B=16, n=1, len=20000, H=32, Hkv=32, D=128, page=128,
             fmt=INT8, window=4096, sinks=4),
        # a few drafted tokens for each of a few sequences, narrow heads
        dict(name="attend_b4_n5_l4100_h16_4_d64", op="attend", B=4, n=5, len=4100, H=16, Hkv=4, D=64, page=32, fmt=E4M3,
             window=0, sinks=0),
        # a prefill of the block workload
        dict(name="attend_b1_n2048_l2048_h32_32", op="attend", B=1, n=2048, len=2048, H=32, Hkv=32, D=128, page=64, fmt=INT8,
             window=0, sinks=0),
        # chunks of two long prompts over a sliding window
        dict(name="attend_b2_n1000_l9000_w1024_h64_8", op="attend", B=2, n=1000, len=9000, H=64, Hkv=8, D=128, page=128,
             fmt=E4M3, window=1024, sinks=16),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "attend", "attend", "attend", "attend"])
    D = rng.choice([64, 128, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 32])
    H = Hkv * rng.choice([1, 1, 2, 3, 4, 7, 8] if Hkv < 32 else [1, 2])
    if op == "rotate":
        T = _log(rng, 1, 2048)
        while T * (H + Hkv) * D > 2048 * 64 * 128:
            T //= 2
        return dict(op=op, T=T, H=H, Hkv=Hkv, D=D, dims=rng.choice([D, D, D // 2]), paired=rng.random() < 0.4,
                    norm=rng.random() < 0.8, packed=rng.random() < 0.5)
    page, B = rng.choice([16, 32, 64, 128]), _log(rng, 1, 64)
    if op == "append":
        n = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
        length = n + (0 if rng.random() < 0.3 else _log(rng, 1, 2048))
        while B * n * (H + 2 * Hkv) * D > 2048 * 96 * 128 or B * length * Hkv * D > 2048 * 64 * 128:
            B, n = (B + 1) // 2, (n + 1) // 2
            length = max(n, length // 2)
        rotary = rng.random() < 0.5
        return dict(op=op, B=B, n=n, len=length, H=H, Hkv=Hkv, D=D, page=page,
                    fmt=E4M3 if rotary else rng.choice([INT8, E4M3]), rotary=rotary)
    kind = rng.random()
    n = 1 if kind < 0.55 else rng.randint(2, 8) if kind < 0.7 else _log(rng, 16, 2048)
    length = max(n, _log(rng, 16, 32768))
    window = 0 if rng.random() < 0.6 else _log(rng, 64, 4096)
    # up to the largest listed cases' cache and products
    while B * length * Hkv * D > 47 * 8192 * 8 * 128 or B * n * min(length, (window + n) if window else length) * H * D > \
            2 * 1000 * 900 * 64 * 128 or B * n * length * H > 2 * 1000 * 9000 * 64:
        if B > 1:
            B = (B + 1) // 2
        else:
            n, length = (n + 1) // 2, max(16, length // 2)
    return dict(op=op, B=B, n=n, len=max(n, length), H=H, Hkv=Hkv, D=D, page=page, fmt=rng.choice([INT8, E4M3]),
                window=window, sinks=rng.choice([0, 1, 4, 50]) if window else 0)


def _ragged(case):
    """New tokens and lengths of a case's sequences: the first one's are the case's, the others' are less."""
    B, n, length = case["B"], case["n"], case["len"]
    new = [max(1, n - (n // 2) * ((7 * b) % B) // B) for b in range(B)]
    lens = [max(m, length - (length // 2) * ((5 * b) % B) // B) for b, m in enumerate(new)]
    return new, lens


def _visible(p, window, sinks):
    """How many tokens position p sees."""
    return p + 1 if not window else min(window, p + 1) + min(sinks, max(0, p + 1 - window))


def work(case):
    op, H, Hkv, D = case["op"], case["H"], case["Hkv"], case["D"]
    if op == "rotate":
        T = case["T"]
        return dict(bytes=4 * T * (H + Hkv) * D + 4 * T * case["dims"] + 4 * T, flops=10 * T * (H + Hkv) * D)
    new, lens = _ragged(case)
    T = sum(new)
    if op == "append":
        more = (4 * T * H * D + 4 * T * D) if case["rotary"] else 0
        return dict(bytes=6 * T * Hkv * D + more, flops=(10 * T * H * D if case["rotary"] else 0) + 4 * T * Hkv * D)
    window, sinks = case["window"], case["sinks"]
    # a sequence's visible tokens are those of its first new one and the new ones behind it
    seen = sum(_visible(s - m, window, sinks) + m - 1 for m, s in zip(new, lens))
    pairs = sum(_visible(p, window, sinks) for m, s in zip(new, lens) for p in range(s - m, s))
    return dict(bytes=2 * seen * Hkv * D + 4 * T * H * D, flops=4 * pairs * H * D)


# ------------------------------------------------------------------------------------------------ inputs

def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 64 + salt)


def _table(rows, dims):
    """Cosines and sines of rows positions, (rows, dims / 2, 2), made in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, dims, 2, device=DEV, dtype=torch.float64) / dims)
    a = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.stack([torch.cos(a), torch.sin(a)], -1).float()


def _codes(shape, fmt, g):
    """Codes of a filled cache: the largest of a page near the top."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    for i in range(0, shape[0], 4096):                     # (in pieces: the cache may be large)
        x = torch.randn((min(4096, shape[0] - i),) + tuple(shape[1:]), device=DEV, generator=g, dtype=torch.float16)
        x = (x * 30).round_().clamp_(-127, 127).to(torch.int8) if fmt == INT8 else \
            (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        out[i:i + 4096] = x.view(torch.uint8)
    return out


def _batch(s, case, g):
    """The sequences' offsets, lengths and pages (in no order; no page where a sequence has none yet), and the cache."""
    new, lens = _ragged(case)
    B, page, Hkv, D = case["B"], case["page"], case["Hkv"], case["D"]
    width = -(-case["len"] // page)
    need = torch.tensor([-(-x // page) for x in lens], device=DEV)
    total = sum(-(-x // page) for x in lens)
    has = torch.arange(width, device=DEV)[None] < need[:, None]
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[has] = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    i32 = dict(dtype=torch.int32, device=DEV)
    off = [0]
    for m in new:
        off.append(off[-1] + m)
    s.update(offsets=torch.tensor(off, **i32), lens=torch.tensor(lens, **i32), table=table, T=off[-1], pages=total,
             max_new=max(new))
    s["K"] = _codes((total, Hkv, page, D), case["fmt"], g)
    s["V"] = _codes((total, Hkv, D, page), case["fmt"], g)
    # a head's scales: of one size over its pages, some of them twice or half of it
    for name in ("K_scale", "V_scale"):
        base = 2.0 ** torch.randint(-7, -4, (1, Hkv), device=DEV, generator=g)
        some = 2.0 ** torch.randint(-1, 2, (total, Hkv), device=DEV, generator=g)
        s[name] = (base * some * (1.0 if case["fmt"] == INT8 else 0.25)).float()


def prepare(case, seed):
    op, H, Hkv, D = case["op"], case["H"], case["Hkv"], case["D"]
    g = _gen(seed, 2)
    s = dict(case)

    def rows(T, heads):
        return torch.randn((T, heads, D), device=DEV, generator=g, dtype=torch.float16)

    def gain():
        return (1.0 + 0.2 * torch.randn(D, device=DEV, generator=g)).half()

    if op == "rotate":
        T = case["T"]
        x = rows(T, H + Hkv)
        # the layers' outputs lie in one buffer, or each in its own
        s["Q"], s["Kx"] = (x[:, :H], x[:, H:]) if case["packed"] else (x[:, :H].contiguous(), x[:, H:].contiguous())
        s["angles"] = _table(4096, case["dims"])
        s["positions"] = ((torch.arange(T, device=DEV) + 1000) % 4096).to(torch.int32)
        s["gains"] = (gain(), gain()) if case["norm"] else None
        s["out"] = (torch.empty((T, H, D), dtype=torch.float16, device=DEV),
                    torch.empty((T, Hkv, D), dtype=torch.float16, device=DEV))
        return _plan(s) if own else s
    _batch(s, case, g)
    T = s["T"]
    if op == "append":
        s["Kx"], s["Vx"] = rows(T, Hkv), rows(T, Hkv)
        s["Kx"] *= (0.5 + torch.rand((1, Hkv, D), device=DEV, generator=g)).half()     # channels of different sizes
        if case["rotary"]:
            s["Q"], s["out"] = rows(T, H), torch.empty((T, H, D), dtype=torch.float16, device=DEV)
            s["angles"], s["gains"] = _table(4096, D), (gain(), gain())
        return _plan(s) if own else s
    s["Q"] = rows(T, H)
    s["out"] = torch.empty((T, H, D), dtype=torch.float16, device=DEV)
    s["sm_scale"] = D ** -0.5
    return _plan(s) if own else s


def _plan(s):
    """The handles that a user's program keeps: the cache, the batch, the rotation, the workspace."""
    import bit_mixed_precision_tri_amd as tri
    if "angles" in s:
        s["rotary"] = tri.Rotary(s["angles"], gains=s["gains"], norm=s["gains"] is not None, eps=1e-5,
                                 interleaved=s.get("paired", False))
    if s["op"] != "rotate":
        s["cache"] = tri.KVCache(s["K"], s["V"], s["K_scale"], s["V_scale"], s["fmt"])
        s["seqs"] = tri.Sequences(s["offsets"], s["lens"], s["table"], max_new=s["max_new"], max_len=s["len"])
    if s["op"] == "attend":
        need = tri.cache_attend_workspace_bytes(s["cache"], s["seqs"], s["T"], s["H"], window=s["window"], sinks=s["sinks"])
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    return {"rotate": _plain_rotate, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)


def _held(s):
    """The cache's codes as the values they stand for, without their scales, and the scales."""
    kind = torch.int8 if s["fmt"] == INT8 else torch.float8_e4m3fn
    return dict(K=s["K"].view(kind), V=s["V"].view(kind), K_scale=s["K_scale"], V_scale=s["V_scale"])


def _own(s):
    import bit_mixed_precision_tri_amd as tri
    if s["op"] == "rotate":
        return tri.heads_rotate((s["Q"], s["Kx"]), s["rotary"], s["positions"], out=s["out"])
    if s["op"] == "append":
        if not s["rotary"]:
            tri.cache_append(s["cache"], s["seqs"], s["Kx"], s["Vx"])
            return _held(s)
        q = tri.cache_append(s["cache"], s["seqs"], s["Kx"], s["Vx"], rotary=s["rotary"], Q=s["Q"], out=s["out"])
        return dict(_held(s), Q=q)
    return tri.cache_attend(s["cache"], s["seqs"], s["Q"], scale=s["sm_scale"], window=s["window"], sinks=s["sinks"],
                            workspace=s["ws"], out=s["out"])


def _rotated(x, gain, angles, positions, paired):
    """(T, heads, D) normalised where there is a gain, and rotated; in 32 bits, rounded once."""
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * gain.float()
    cs = angles[positions.long()].unsqueeze(1)             # (T, 1, dims / 2, 2)
    dims = 2 * cs.shape[2]
    r = x[..., :dims]
    a, b = (r[..., 0::2], r[..., 1::2]) if paired else (r[..., :dims // 2], r[..., dims // 2:])
    u, v = a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]
    r = torch.stack([u, v], -1).flatten(-2) if paired else torch.cat([u, v], -1)
    return torch.cat([r, x[..., dims:]], -1).half()


def _plain_rotate(s):
    gains = s["gains"] or (None, None)
    return tuple(_rotated(x, g, s["angles"], s["positions"], s["paired"]) for x, g in zip((s["Q"], s["Kx"]), gains))


def _places(s):
    """Of every new token: its sequence, position, page (that many of the cache) and place in the page."""
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(s["offsets"].long(), t, right=True) - 1
    p = s["lens"].long()[b] - s["offsets"].long()[b + 1] + t
    return b, p, s["table"].long()[b, p // s["page"]], p % s["page"]


def _to_codes(x, fmt):
    """Values over their scale (exact: the scales are powers of two), rounded to the nearest code, ties to even."""
    x = x.clamp(-TOP[fmt], TOP[fmt])
    return x.round().to(torch.int8) if fmt == INT8 else x.to(torch.float8_e4m3fn)


def _plain_append(s):
    fmt, page = s["fmt"], s["page"]
    _, p, at, place = _places(s)
    K, V, q = s["Kx"], s["Vx"], None
    if s["rotary"]:
        q = _rotated(s["Q"], s["gains"][0], s["angles"], p, False)
        K = _rotated(K, s["gains"][1], s["angles"], p, False)
    # the first new place of every page that gets one (all of it is new where that is 0)
    first = torch.full((s["pages"],), page, device=DEV).scatter_reduce(0, at, place, "amin")
    kind = torch.int8 if fmt == INT8 else torch.float8_e4m3fn
    earlier = (torch.arange(page, device=DEV) < first[:, None]) & (first[:, None] < page)
    for x, codes, scale in ((K, s["K"], s["K_scale"]), (V, s["V"], s["V_scale"])):
        x = x.float()
        most = torch.zeros_like(scale).scatter_reduce(0, at[:, None].expand(-1, s["Hkv"]), x.abs().amax(-1), "amax")
        f, e = torch.frexp(most)                           # most = f 2^e, 0.5 <= f < 1; the top is c 2^d likewise
        c, d = math.frexp(TOP[fmt])
        need = torch.ldexp(torch.ones_like(f), torch.where(most > 0, e - d + (f > c), -40).clamp(min=-30))
        now = torch.where(first[:, None] == 0, need, torch.maximum(need, scale))
        now = torch.where(first[:, None] == page, scale, now)
        # the codes of earlier tokens where the scale grew
        old = codes.view(kind).float() * torch.where(first[:, None] == 0, torch.ones_like(now), scale / now)[..., None, None]
        held = earlier[:, None, :, None] if codes is s["K"] else earlier[:, None, None]
        codes.copy_(torch.where((now > scale)[..., None, None] & held, _to_codes(old, fmt).view(torch.uint8), codes))
        scale.copy_(now)
        new = _to_codes(x / now[at][..., None], fmt).view(torch.uint8)
        if codes is s["K"]:
            codes[at, :, place] = new
        else:
            codes[at, :, :, place] = new
    return _held(s) if q is None else dict(_held(s), Q=q)


def _plain_attend(s):
    B, H, Hkv, D, page, fmt, n = (s[x] for x in ("B", "H", "Hkv", "D", "page", "fmt", "max_new"))
    kind, G = torch.int8 if fmt == INT8 else torch.float8_e4m3fn, H // Hkv
    table = s["table"].long().clamp(min=0)                 # (pages that are not there lie behind every position)
    L = table.shape[1] * page
    K = s["K"][table].view(kind).float() * s["K_scale"][table][..., None, None]      # (B, pages, Hkv, page, D)
    K = K.permute(0, 2, 4, 1, 3).reshape(B * Hkv, D, L)
    V = s["V"][table].view(kind).float() * s["V_scale"][table][..., None, None]      # (B, pages, Hkv, D, page)
    V = V.permute(0, 2, 1, 4, 3).reshape(B * Hkv, L, D)
    # queries padded to the longest
    row = s["offsets"].long()[:-1, None] + torch.arange(n, device=DEV)
    live = row < s["offsets"].long()[1:, None]
    q = s["Q"][row.clamp(max=s["T"] - 1)].float()          # (B, n, H, D)
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B * Hkv, n * G, D)
    p = (s["lens"].long() - s["offsets"].long()[1:])[:, None] + row      # positions, (B, n)
    j = torch.arange(L, device=DEV)
    sees = (j <= p[..., None]) & live[..., None]
    if s["window"]:
        sees &= (j > p[..., None] - s["window"]) | (j < s["sinks"])
    sees = sees.view(B, 1, n, 1, L)
    x = (torch.bmm(q, K) * s["sm_scale"]).view(B, Hkv, n, G, L).masked_fill_(~sees, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    y = torch.bmm(x.view(B * Hkv, n * G, L), V).view(B, Hkv, n, G, D) / x.sum(-1, keepdim=True).clamp(min=1e-30)
    y = y.permute(0, 2, 1, 3, 4).reshape(B, n, H, D)
    out = torch.empty_like(s["out"])
    out[row[live]] = y[live].half()
    return out


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_heads(x, gain, angles, positions, paired):
    y = x.double()
    if gain is not None:
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + 1e-5) * gain.double()
    half = angles.shape[1]
    turn = torch.complex(angles[..., 0].double(), angles[..., 1].double())[positions.long()]
    z = y.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if paired else (i, half + i)
        w = torch.complex(y[..., a], y[..., b]) * turn[:, i, None]
        z[..., a], z[..., b] = w.real, w.imag
    return z


def _exact_rotate(s):
    gains = s["gains"] if s["gains"] is not None else (None, None)
    return (_exact_heads(s["Q"], gains[0], s["angles"], s["positions"], s["paired"]),
            _exact_heads(s["Kx"], gains[1], s["angles"], s["positions"], s["paired"]))


def _code_values(fmt):
    """What the 256 codes stand for, from the formats' definitions."""
    if fmt == INT8:
        v = [b - 256 if b > 127 else b for b in range(256)]
    else:
        v = [(-1.0 if b & 128 else 1.0) * ((b & 7) * 2.0 ** -9 if b & 120 == 0 else (8 + (b & 7)) * 2.0 ** ((b >> 3 & 15) - 10))
             for b in range(256)]
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _nearest(x, fmt):
    """The nearest value of a code, ties to the even one."""
    if fmt == INT8:
        return torch.round(x).clamp(-127, 127)
    step = 2.0 ** (torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
    """Page by page for whole numbers of pages; int8 codes are whole numbers and have no such value."""
    fmt, page, Hkv, D = s["fmt"], s["page"], s["Hkv"], s["D"]
    values = _code_values(fmt)
    off, lens, table = s["offsets"].tolist(), s["lens"].tolist(), s["table"].tolist()
    pos = torch.tensor([lens[b] - off[b + 1] + t for b in range(s["B"]) for t in range(off[b], off[b + 1])], device=DEV)
    K, V, out = s["Kx"].double(), s["Vx"].double(), {}
    if s["rotary"]:
        out["Q"] = _exact_heads(s["Q"], s["gains"][0], s["angles"], pos, False)
        K = _exact_heads(s["Kx"], s["gains"][1], s["angles"], pos, False).half().double()
    k, v = values[s["K"].long()], values[s["V"].long()].transpose(2, 3).contiguous()
    ks, vs = s["K_scale"].double(), s["V_scale"].double()
    for b in range(s["B"]):
        t, p = off[b], lens[b] - (off[b + 1] - off[b])
        while t < off[b + 1]:
            at, i = table[b][p // page], p % page
            m = min(page - i, off[b + 1] - t)
            for x, c, sc in ((K, k, ks), (V, v, vs)):
                most = x[t:t + m].abs().amax(dim=(0, 2))
                e = torch.log2(most.clamp(min=2.0 ** -40) / TOP[fmt]).ceil()
                need = 2.0 ** torch.where(most <= TOP[fmt] * 2.0 ** (e - 1), e - 1, e).clamp(min=-30)
                grown = need if i == 0 else torch.maximum(need, sc[at])
                if i > 0:
                    c[at, :, :i] = torch.where((grown > sc[at])[:, None, None],
                                               _nearest(c[at, :, :i] * (sc[at] / grown)[:, None, None], fmt), c[at, :, :i])
                sc[at] = grown
                c[at, :, i:i + m] = _nearest(x[t:t + m].transpose(0, 1) / grown[:, None, None], fmt)
            t, p = t + m, p + m
    out.update(K_scale=ks, V_scale=vs, K=None if fmt == INT8 else k, V=None if fmt == INT8 else v.transpose(2, 3).contiguous())
    return out


def _exact_attend(s):
    H, Hkv, D, page, fmt, window, sinks = (s[x] for x in ("H", "Hkv", "D", "page", "fmt", "window", "sinks"))
    values, G = _code_values(fmt), H // Hkv
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["Q"].shape, dtype=torch.float64, device=DEV)
    for b in range(s["B"]):
        n, L = off[b + 1] - off[b], lens[b]
        pages = s["table"][b, :-(-L // page)].long()
        p = torch.arange(L - n, L, device=DEV)[:, None]
        j = torch.arange(L, device=DEV)[None]
        hidden = j > p
        if window > 0:
            hidden = hidden | ((p - j >= window) & (j >= sinks))
        for h in range(Hkv):
            k = (values[s["K"][pages, h].long()] * s["K_scale"][pages, h].double()[:, None, None]).reshape(-1, D)[:L]
            v = (values[s["V"][pages, h].long()] * s["V_scale"][pages, h].double()[:, None, None])
            v = v.transpose(1, 2).reshape(-1, D)[:L]
            for i in range(h * G, (h + 1) * G):
                x = (s["Q"][off[b]:off[b + 1], i].double() @ k.t() * s["sm_scale"]).masked_fill(hidden, -math.inf)
                out[off[b]:off[b + 1], i] = torch.softmax(x, dim=1) @ v
    return out
