"""What is measured of the operators around a user's history kept in 4 bits.

A recommender that ranks candidates for a user reads the user's history as
keys and values.  Between requests the history stays in a paged cache of 4-bit
values, shared by all of the user's candidates: rotary positions are applied to
queries and keys, block tables and slot maps follow from the lengths, new
events are quantised into their slots, and attention reads the cache.

A case is one call of one operator; `op` says which.  Lengths and the number
of candidates of each user follow from the case alone (so that the work does),
values and orders from the seed.

The cache's layout: uint8 [n_pages][H_kv][page / 16][2560]; the 2560 bytes of
16 tokens of one head are the keys' codes [16][64] (element j in nibble j, the
low one first), the keys' (s, z) pairs [16][4] of two bf16 for groups of 32
elements, then the same for the values.  A code c stands for
bf16(z + (16 + c) s).
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension of the attention
GROUP = 32       # elements that share a scale
BLOCK = 2560     # bytes of 16 tokens of one head


# ------------------------------------------------------------------ cases
def listed():
    return [
        # queries of a 1024-candidate request (15 users, 70:1): each candidate at its user's position
        dict(name="rope_queries", op="rope", n=1024, users=15, H=8, L=32, d=128, rot=128, interleaved=False, dtype="bf16",
             scaling="none", factor=1.0, far=4096, backward=False),
        # the gradient of the histories' keys, one row each (16 users x 2048), half of the head, stretched context, 32 bits
        dict(name="rope_keys_gradient", op="rope", n=32768, users=0, H=8, L=1, d=128, rot=64, interleaved=True, dtype="fp32",
             scaling="turns", factor=8.0, far=1000000, backward=True),
        # the newest event of one user, one row: latency
        dict(name="rope_one_token", op="rope", n=1, users=0, H=8, L=1, d=128, rot=128, interleaved=False, dtype="bf16",
             scaling="linear", factor=4.0, far=100000, backward=False),
        # a request's 15 users each grow by a few events: latency
        dict(name="tables_request", op="tables", users=15, page=16, old=2000, spread=900, grow=24, shrink=0),
        # 2048 users after a training day: some grow by hundreds, every fourth one is cut
        dict(name="tables_many_users", op="tables", users=2048, page=64, old=1500, spread=1400, grow=300, shrink=4),
        # the new events of a request (15 users, 1..3 pages) written and read back
        dict(name="store_events", op="store", users=15, H=8, page=16, len=24, spread=20),
        # whole histories of 15 users x 2048
        dict(name="store_histories", op="store", users=15, H=8, page=64, len=2048, spread=0),
        # one candidate of one user: latency
        dict(name="attend_one", op="attend", cands=1, users=1, H=8, Hkv=8, Lq=8, len=1000, spread=0, page=16, skew=1, lse=False),
        # one candidate for each of 64 long histories: the cache's bytes count
        dict(name="attend_one_each", op="attend", cands=64, users=64, H=8, Hkv=8, Lq=8, len=4096, spread=1000, page=64, skew=1, lse=False),
        # few users with very long histories, heads that share keys, log-sum-exp wanted
        dict(name="attend_long_shared", op="attend", cands=8, users=4, H=32, Hkv=8, Lq=8, len=50001, spread=20000, page=128, skew=1, lse=True),
        # ten candidates a user, ragged histories
        dict(name="attend_ten_each", op="attend", cands=1024, users=102, H=8, Hkv=8, Lq=16, len=2048, spread=1800, page=32, skew=1, lse=False),
        # the 70:1 request: 1024 candidates of 15 users
        dict(name="attend_request", op="attend", cands=1024, users=15, H=8, Hkv=8, Lq=32, len=2048, spread=0, page=64, skew=1, lse=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "tables", "store", "attend", "attend"])
    if op == "rope":
        users = rng.choice([0, _log(rng, 1, 100)])
        L = 8 * rng.randint(1, 8) if users else rng.choice([1, 1, rng.randint(2, 300)])
        H = rng.randint(1, 12)
        d = rng.choice([64, 80, 96, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        n = _log(rng, 1, max(1, 30000000 // (L * H * d * (2 if dtype == "fp32" else 1))))
        return dict(op=op, n=n, users=min(users, n), H=H, L=L, d=d, rot=rng.choice([d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                    interleaved=rng.random() < 0.5, dtype=dtype, scaling=rng.choice(["none", "linear", "base", "turns"]),
                    factor=round(rng.uniform(1.0, 16.0), 2), far=_log(rng, 1, 1000000), backward=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        users = _log(rng, 1, 4096)
        old = _log(rng, 1, max(1, min(8000, 4000000 // users)))
        return dict(op=op, users=users, page=page, old=old, spread=rng.randint(0, old), grow=_log(rng, 1, max(1, min(2000, 600000 // users))),
                    shrink=rng.choice([0, 0, 2, 5]))
    if op == "store":
        users, H = _log(rng, 1, 64), rng.choice([1, 2, 4, 5, 8])
        length = _log(rng, 1, max(1, min(8192, 245760 // (users * H))))
        return dict(op=op, users=users, H=H, page=page, len=length, spread=rng.randint(0, length))
    group = rng.choice([1, 1, 1, 2, 4])
    Hkv = rng.choice([1, 2, 4, 8])
    Lq = 8 * rng.randint(1, 4)
    users = _log(rng, 1, 120)
    cands = _log(rng, users, max(users, min(1024, 70 * users)))
    rows = cands * Hkv * group * Lq
    most = min(50000, 260000 * 2048 // rows, 1600000 // (users * Hkv))
    length = _log(rng, 1, max(1, most))
    return dict(op=op, cands=cands, users=users, H=Hkv * group, Hkv=Hkv, Lq=Lq, len=length, spread=rng.randint(0, length), page=page,
                skew=rng.choice([1, 1, 2]), lse=rng.random() < 0.3)


def _spread(count, longest, spread):
    """Lengths longest - spread .. longest, the first the longest; a spread as long as the longest leaves some empty."""
    i = np.arange(count, dtype=np.int64)
    return longest - (i * 7919) % (spread + 1)


def _tables_lens(c):
    i = np.arange(c["users"], dtype=np.int64)
    old = _spread(c["users"], c["old"], c["spread"])
    new = old + (i * 613) % (c["grow"] + 1) + (1 if c["grow"] else 0)
    if c["shrink"]:
        new = np.where(i % c["shrink"] == c["shrink"] - 1, old // 2, new)
    return old, new


def _users_of(cands, users, skew):
    """The user of each candidate before they are shuffled: even, or with the first users taking most."""
    i = np.arange(cands, dtype=np.int64)
    return i * users // cands if skew == 1 else (i * i * users) // (cands * cands)


# ---------------------------------------------------------------- prepare
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _keys(shape, g):
    """Keys: a few channels are several times as large as the others, as trained keys have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., 5::41] *= 4.0
    return x.to(torch.bfloat16)


def _pages(lens, page, g):
    """A table of distinct pages in shuffled order for these lengths, and how many pages there are."""
    blocks = (lens + page - 1) // page
    total, most = int(blocks.sum()), max(1, int(blocks.max()))
    n_pages = total + total // 8 + 4
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = np.concatenate([[0], np.cumsum(blocks)])[:-1]
    at = first[:, None] + np.arange(most)[None, :]
    used = torch.from_numpy(np.arange(most)[None, :] < blocks[:, None]).cuda()
    at = torch.from_numpy(np.minimum(at, max(0, total - 1))).cuda()
    table = torch.where(used, order[at], torch.full_like(order[at], -1)).contiguous()
    return table, n_pages, order, total


def prepare(c, seed):
    g = _gen(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": c}
    if c["op"] == "rope":
        s["x"] = torch.randn((c["n"], c["H"], c["L"], c["d"]), generator=g, device="cuda").to(_TYPES[c["dtype"]])
        s["start"] = torch.randint(0, c["far"] + 1, (c["users"] or c["n"],), generator=g, **i32)
        if c["users"]:
            m = torch.from_numpy(_users_of(c["n"], c["users"], 1)).cuda().to(torch.int32)
            s["map"] = m[torch.randperm(c["n"], generator=g, device="cuda")].contiguous()
        return s
    if c["op"] == "tables":
        old, new = _tables_lens(c)
        P = c["page"]
        most = int(max((old + P - 1).max(), (new + P - 1).max()) // P)
        have, need = (old + P - 1) // P, (new + P - 1) // P
        n_pages = int(np.maximum(have, need).sum()) + 7
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        first = np.concatenate([[0], np.cumsum(have)])[:-1]
        at = np.minimum(first[:, None] + np.arange(most)[None, :], n_pages - 1)
        used = torch.from_numpy(np.arange(most)[None, :] < have[:, None]).cuda()
        table = torch.where(used, order[torch.from_numpy(at).cuda()], -1).to(torch.int32)
        n_free = n_pages - int(have.sum())
        free = torch.full((n_pages,), -1, **i32)
        free[:n_free] = order[int(have.sum()):]
        # the program's own state in one array: table, free pages, their number, lengths
        s["state"] = torch.cat([table.reshape(-1), free, torch.tensor([n_free], **i32), torch.from_numpy(old).cuda().to(torch.int32)])
        s["sizes"] = (table.numel(), n_pages, 1, c["users"])
        s["new"] = torch.from_numpy(new).cuda().to(torch.int32)
        s["most"], s["max_new"] = most, int(np.maximum(new - old, 0).sum()) + 5
        return s
    lens = _spread(c["users"], c["len"], c["spread"])
    P, Hkv = c["page"], c.get("Hkv", c.get("H"))
    table, n_pages, order, used = _pages(lens, P, g)
    s.update(table=table, lens=torch.from_numpy(lens).cuda().to(torch.int32), n_pages=n_pages, rows=int(lens.sum()))
    off = np.concatenate([[0], np.cumsum(lens)])
    s["offsets"] = torch.from_numpy(off).cuda().to(torch.int32)
    if c["op"] == "store":
        n = s["rows"]
        s["K"], s["V"] = _keys((n, Hkv, D), g), torch.randn((n, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        user = np.repeat(np.arange(c["users"]), lens)
        at = torch.from_numpy(np.arange(n) - off[user]).cuda()
        pages = table[torch.from_numpy(user).cuda(), at // P].to(torch.int64)
        s["slots"] = (pages * P + at % P).to(torch.int32)
        s["data"] = torch.zeros((n_pages, Hkv, P // 16, BLOCK), dtype=torch.uint8, device="cuda")
        return s
    s["Q"] = torch.randn((c["cands"], c["H"], c["Lq"], D), generator=g, device="cuda").to(torch.bfloat16)
    users = torch.from_numpy(_users_of(c["cands"], c["users"], c["skew"])).cuda().to(torch.int32)
    s["map"] = users[torch.randperm(c["cands"], generator=g, device="cuda")].contiguous()
    # the cache as earlier requests left it: every page holds something, also behind a history's end
    data = torch.empty((n_pages, Hkv, P // 16, BLOCK), dtype=torch.uint8, device="cuda")
    tokens = n_pages * Hkv * P
    step = max(1, tokens // max(1, -(-tokens // (1 << 19))))
    flat = data.view(-1, BLOCK)
    for a in range(0, tokens // 16, max(1, step // 16)):
        b = min(tokens // 16, a + max(1, step // 16))
        k = _keys(((b - a) * 16, D), g)
        v = torch.randn(((b - a) * 16, D), generator=g, device="cuda").to(torch.bfloat16)
        flat[a:b] = torch.cat([_pack(x).view(b - a, -1) for x in (k, v)], dim=1)
    s["data"] = data
    return s


# ------------------------------------------------------------ plain forms
def _quantise(x):
    """Codes (0..15, fp32) and (s, z) (bf16) of groups of 32 elements of bf16 x."""
    v = x.float().view(*x.shape[:-1], -1, GROUP)
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    s = ((hi * 0.5 - lo * 0.5) / torch.full_like(lo, 7.5)).to(torch.bfloat16).float()
    z = (lo - 16.0 * s).to(torch.bfloat16).float()
    q = torch.where(s > 0, ((v - z) / s).round() - 16.0, torch.zeros_like(v)).clamp(0.0, 15.0)
    return q, s, z


def _pack(x):
    """[tokens, 128] bf16 -> the bytes of tokens / 16 half blocks (codes, then (s, z))."""
    q, s, z = _quantise(x)
    q = q.view(-1, 16, D // 2, 2).to(torch.uint8)
    codes = (q[..., 0] | (q[..., 1] << 4)).view(-1, 16 * 64)
    sz = torch.cat([s, z], dim=-1).to(torch.bfloat16).view(torch.uint8).view(-1, 256)
    return torch.cat([codes, sz], dim=1)


def _unpack(data):
    """The cache's bytes [..., 2560] as fp32 values [..., 2, 16, 128] (keys, values)."""
    half = data.view(*data.shape[:-1], 2, BLOCK // 2)
    codes = half[..., :1024].view(*half.shape[:-1], 16, 64)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).view(*half.shape[:-1], 16, 4, GROUP).float()
    sz = half[..., 1024:].contiguous().view(torch.bfloat16).float().view(*half.shape[:-1], 16, 4, 2)
    v = sz[..., 1:] + (c + 16.0) * sz[..., :1]
    return v.to(torch.bfloat16).float().view(*half.shape[:-1], 16, D)


def _histories(data, table, P):
    """Keys and values [users, H, blocks * page, 128] in fp32 of every user's pages (absent ones read page 0)."""
    kv = _unpack(data[table.clamp(min=0).to(torch.int64)])   # [users, blocks, H, page / 16, 2, 16, 128]
    kv = kv.permute(4, 0, 2, 1, 3, 5, 6)
    return kv.reshape(2, table.shape[0], data.shape[1], -1, D)


def _frequencies(c):
    """Radians a position for each pair, in 64 bits."""
    j = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    rot, base = c["rot"], 10000.0
    if c["scaling"] == "base" and rot > 2:
        base = base * c["factor"] ** (rot / (rot - 2.0))
    f = base ** (-2.0 * j / rot)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "turns":
        keep = ((8192.0 * f / (2.0 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / c["factor"]
    return f


def _rope(s):
    c, x = s["case"], s["x"]
    start = s["start"][s["map"].to(torch.int64)] if c["users"] else s["start"]
    pos = start.to(torch.float64)[:, None] + torch.arange(c["L"], dtype=torch.float64, device="cuda")
    angle = (pos[:, :, None] * _frequencies(c))[:, None]                     # [n, 1, L, rot / 2]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if c["backward"]:
        sin = -sin
    v = x[..., :c["rot"]].float()
    if c["interleaved"]:
        a, b = v[..., 0::2], v[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = v.chunk(2, dim=-1)
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y.to(x.dtype), x[..., c["rot"]:]], dim=-1)


def _tables(s):
    c, new = s["case"], s["new"].to(torch.int64)
    table, free, n_free, old = (t.to(torch.int64) for t in s["state"].split(s["sizes"]))
    P, U, n_pages = c["page"], c["users"], free.numel()
    table = table.view(U, -1)
    need, have = (new + P - 1) // P, (old + P - 1) // P
    take, give = (need - have).clamp(min=0), (have - need).clamp(min=0)
    blk = torch.arange(s["most"], device="cuda")[None, :]
    kth = (take.cumsum(0) - take)[:, None] + blk - have[:, None]
    takes = (blk >= have[:, None]) & (blk < need[:, None])
    gives = (blk >= need[:, None]) & (blk < have[:, None])
    grown = torch.where(takes, free[(n_free - 1 - kth).clamp(0, n_pages - 1)], table)
    at = n_free - take.sum() + (give.cumsum(0) - give)[:, None] + blk - need[:, None]
    at = torch.where(gives, at, torch.full_like(at, n_pages))
    free = torch.cat([free, free.new_zeros(1)]).scatter(0, at.reshape(-1), table.reshape(-1))[:n_pages]
    grown = torch.where(gives, torch.full_like(grown, -1), grown)
    count = (new - old).clamp(min=0)
    ends = count.cumsum(0)
    i = torch.arange(s["max_new"], device="cuda")
    u = torch.searchsorted(ends, i, right=True).clamp(max=U - 1)
    pos = old[u] + i - (ends - count)[u]
    there = i < ends[-1]
    slot = grown[u, (pos // P).clamp(0, s["most"] - 1)] * P + pos % P
    out = dict(table=grown, free=free, n_free=n_free - take.sum() + give.sum(), lens=new, slots=torch.where(there, slot, -1),
               offsets=torch.cat([ends.new_zeros(1), ends]), positions=torch.where(there, pos, 0))
    return {k: v.to(torch.int32) for k, v in out.items()}


def _store(s):
    c = s["case"]
    P, Hkv = c["page"], c["H"]
    n = s["rows"]
    block, row = (s["slots"] // 16).to(torch.int64), (s["slots"] % 16).to(torch.int64)
    per = P // 16
    flat = ((block // per)[:, None] * Hkv + torch.arange(Hkv, device="cuda")[None, :]) * per + (block % per)[:, None]
    data = s["data"].view(-1, 2, BLOCK // 2)
    codes, sz = data[..., :1024].view(-1, 2, 16, 64), data[..., 1024:].view(-1, 2, 16, 16)
    q, sc, z = _quantise(torch.stack([s["K"], s["V"]], dim=2))
    q = q.view(n, Hkv, 2, 64, 2).to(torch.uint8)
    codes[flat, :, row[:, None]] = q[..., 0] | (q[..., 1] << 4)
    sz[flat, :, row[:, None]] = torch.cat([sc, z], dim=-1).to(torch.bfloat16).view(torch.uint8).view(n, Hkv, 2, 16)
    kv = _unpack(s["data"].view(-1, BLOCK))[flat]                            # [n, H, 2, 16, 128]
    kv = kv.gather(3, row.view(n, 1, 1, 1, 1).expand(n, Hkv, 2, 1, D))[:, :, :, 0]
    return [kv[:, :, 0].to(torch.bfloat16).contiguous(), kv[:, :, 1].to(torch.bfloat16).contiguous()]


def _attend(s):
    c, Q, m = s["case"], s["Q"].float(), s["map"].to(torch.int64)
    n, H, Lq, U, Hkv = c["cands"], c["H"], c["Lq"], c["users"], c["Hkv"]
    K, V = _histories(s["data"], s["table"], c["page"])
    L = K.shape[2]
    # candidates grouped by user, each group padded to the largest
    order = torch.argsort(m, stable=True)
    count = torch.bincount(m, minlength=U)
    place = torch.arange(n, device="cuda") - (count.cumsum(0) - count)[m[order]]
    most = int(count.max())
    where = m[order] * most + place
    rows = Q.new_zeros((U * most, H, Lq, D)).index_copy(0, where, Q[order])
    rows = rows.view(U, most, Hkv, H // Hkv, Lq, D).permute(0, 2, 1, 3, 4, 5).reshape(U, Hkv, -1, D)
    there = torch.arange(L, device="cuda")[None, :] < s["lens"][:, None]
    V = torch.where(there[:, None, :, None], V, V.new_zeros(()))
    S = torch.matmul(rows, K.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    S = torch.where(there[:, None, None, :], S, S.new_full((), -math.inf))
    top = S.amax(-1, keepdim=True)
    p = torch.exp(S - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    O = torch.matmul(p, V) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + torch.log(total)

    def back(x):
        x = x.view(U, Hkv, most, H // Hkv, Lq, -1).permute(0, 2, 1, 3, 4, 5).reshape(U * most, H, Lq, -1)
        return x.new_empty((n,) + x.shape[1:]).index_copy(0, order, x[where])

    out = [back(O).to(torch.bfloat16)]
    if c["lse"]:
        out.append(back(lse)[..., 0])
    return out


# -------------------------------------------------- the framework's calls
_idle = []  # plans that no state holds: a server keeps a few, made once for its largest request


class _Held:
    def __init__(self, plan):
        self.plan = plan

    def __del__(self):
        _idle.append(self.plan)


def _plan(s):
    """The state's plan: taken once, and bound to the state's request where it has one."""
    if "plan" not in s:
        from broadcast_gemm_attention_gb300 import binding
        plan = _idle.pop() if _idle else binding.Plan(65536, 8192, 32)
        c = s["case"]
        if "map" in s:
            plan.plan(s["map"], c["users"], c["H"], c.get("Lq", 8))
        s["plan"] = _Held(plan)
        if c["op"] == "rope":
            freqs = binding.ikbo_rope_frequencies(c["rot"], base=10000.0, scaling=c["scaling"], factor=c["factor"],
                                                  original_len=8192.0, low_turns=1.0, high_turns=4.0)
            s["rope"] = binding.Rope(c["rot"], freqs, interleaved=c["interleaved"])
    return s["plan"].plan


def _own(s):
    c, p = s["case"], _plan(s)
    if c["op"] == "rope":
        y = torch.empty_like(s["x"])
        call = p.rope_backward if c["backward"] else p.rope_forward
        call(s["rope"], s["x"], y, start=s["start"], broadcast=bool(c["users"]))
        return y
    if c["op"] == "tables":
        new = s["state"].clone()
        table, free, n_free, lens = new.split(s["sizes"])
        table = table.view(c["users"], -1)
        slots = new.new_empty(s["max_new"])
        positions = new.new_empty(s["max_new"])
        offsets = new.new_empty(c["users"] + 1)
        p.qcache_resize(lens, s["new"], table, c["page"], free, n_free, slots, offsets, positions)
        return dict(table=table, free=free, n_free=n_free, lens=lens, slots=slots, offsets=offsets, positions=positions)
    if c["op"] == "store":
        K, V = torch.empty_like(s["K"]), torch.empty_like(s["V"])
        p.qcache_append(s["K"], s["V"], s["slots"], s["data"], c["page"])
        p.qcache_load(s["data"], c["page"], s["table"], s["lens"], s["offsets"], K, V)
        return [K, V]
    O = torch.empty_like(s["Q"])
    lse = s["Q"].new_empty(s["Q"].shape[:3], dtype=torch.float32) if c["lse"] else None
    p.attn_qcache_forward(s["Q"], s["data"], c["page"], s["table"], s["lens"], O, lse=lse, Lkv=s["rows"])
    return [O] if lse is None else [O, lse]


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "rope":
        return _rope(s)
    if op == "tables":
        out = _tables(s)
        return dict(out, n_free=out["n_free"].view(1))
    return _store(s) if op == "store" else _attend(s)


# ------------------------------------------------------------------- work
def work(c):
    if c["op"] == "rope":
        values = c["n"] * c["H"] * c["L"] * c["d"]
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * values * size + 4 * (c["users"] or c["n"]) + (4 * c["n"] if c["users"] else 0),
                "flops": 3 * c["n"] * c["H"] * c["L"] * c["rot"]}
    if c["op"] == "tables":
        old, new = _tables_lens(c)
        P = c["page"]
        moved = int(np.abs((new + P - 1) // P - (old + P - 1) // P).sum())
        tokens = int(np.maximum(new - old, 0).sum())
        return {"bytes": 4 * (4 * c["users"] + 2 * moved + 2 * tokens), "flops": 0}
    lens = _spread(c["users"], c["len"], c["spread"])
    if c["op"] == "store":
        values = int(lens.sum()) * c["H"] * D * 2
        return {"bytes": values * 2 * (2 + 0.625) + 4 * int(lens.sum()), "flops": 0}
    keys = int(lens.sum())
    per = np.bincount(_users_of(c["cands"], c["users"], c["skew"]), minlength=c["users"])
    read = int(lens[per > 0].sum())
    values = c["cands"] * c["H"] * c["Lq"] * D
    return {"bytes": read * c["Hkv"] * 160 + 4 * values + (4 * values // D if c["lse"] else 0) + 4 * (keys // c["page"] + c["cands"]),
            "flops": 4 * D * c["H"] * c["Lq"] * int((per * lens).sum())}


# ------------------------------------------------- the definition, 64 bits
def exact(c, seed):
    if c["op"] == "tables":
        return None
    s = prepare(c, seed)
    if c["op"] == "rope":
        x = s["x"].double()
        half = c["rot"] // 2
        pos = s["start"].double() if not c["users"] else s["start"].double()[s["map"].long()]
        out = x.clone()
        l = torch.arange(c["L"], device="cuda").double()
        for j in range(half):
            base = 10000.0
            if c["scaling"] == "base" and c["rot"] > 2:
                base *= math.pow(c["factor"], c["rot"] / (c["rot"] - 2))
            f = math.exp(-2.0 * j / c["rot"] * math.log(base))
            if c["scaling"] == "linear":
                f /= c["factor"]
            elif c["scaling"] == "turns":
                turns = 8192.0 * f / (2 * math.pi)
                f = f if turns >= 4.0 else f / c["factor"] if turns <= 1.0 else f * ((turns - 1) / 3 + (4 - turns) / 3 / c["factor"])
            a = (pos[:, None] + l[None, :])[:, None, :] * (-f if c["backward"] else f)
            i, k = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
            out[..., i] = x[..., i] * torch.cos(a) - x[..., k] * torch.sin(a)
            out[..., k] = x[..., i] * torch.sin(a) + x[..., k] * torch.cos(a)
        return out
    if c["op"] == "store":
        got = []
        for x in (s["K"], s["V"]):
            w = x.double().reshape(-1, GROUP)
            lo, hi = w.min(1).values, w.max(1).values
            step = ((hi - lo) / 15.0).to(torch.bfloat16).double()
            zero = (lo - 16.0 * step).to(torch.bfloat16).double()
            code = torch.round((w - zero[:, None]) / torch.where(step > 0, step, 1.0)[:, None]) - 16.0
            code = torch.where(step[:, None] > 0, code.clamp(0.0, 15.0), 0.0)
            got.append((zero[:, None] + (16.0 + code) * step[:, None]).to(torch.bfloat16).double().view(x.shape))
        return got
    n, H, Lq, Hkv, P = c["cands"], c["H"], c["Lq"], c["Hkv"], c["page"]
    O = torch.zeros((n, H, Lq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((n, H, Lq), -math.inf, dtype=torch.float64, device="cuda")
    lens, m = s["lens"].tolist(), s["map"].long()
    for u in range(c["users"]):
        who = torch.nonzero(m == u).flatten()
        if not lens[u] or not len(who):
            continue
        blocks = (lens[u] + P - 1) // P
        raw = s["data"][s["table"][u, :blocks].long()].transpose(0, 1).reshape(Hkv, -1, BLOCK)  # [Hkv, 16-token blocks, 2560]
        kv = []
        for a in (0, 1280):
            codes = raw[..., a:a + 1024].reshape(Hkv, -1, 64)
            code = torch.empty((Hkv, codes.shape[1], D), dtype=torch.float64, device="cuda")
            code[..., 0::2], code[..., 1::2] = (codes % 16).double(), (codes // 16).double()
            pair = raw[..., a + 1024:a + 1280].contiguous().view(torch.bfloat16).reshape(Hkv, -1, 4, 2).double()
            step, zero = (pair[..., i].repeat_interleave(GROUP, dim=-1) for i in (0, 1))
            kv.append((zero + (16.0 + code) * step).to(torch.bfloat16).double()[:, :lens[u]])
        for h in range(Hkv):
            heads = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
            q = s["Q"][who][:, heads].double().reshape(-1, D)
            logits = q @ kv[0][h].T / math.sqrt(D)
            total = torch.logsumexp(logits, dim=-1)
            part = torch.exp(logits - total[:, None]) @ kv[1][h]
            O[who, heads] = part.view(len(who), -1, Lq, D)
            lse[who, heads] = total.view(len(who), -1, Lq)
    return [O, lse] if c["lse"] else [O]
