"""What is measured of the operators that let candidates be more than rows of their own beside a kept history.

Four operators stand beside broadcast attention and the 4-bit cache:

  axes   rotary positions with several axes (an item's time, height and width, a
         drafted token's depth), forward and gradient
  tree   attention of a tree of drafted tokens: a row reads its user's history in
         the cache, its ancestors in the draft, and itself
  scan   linear attention with a decay for each head over users' events,
           S_t = decay S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t,
         from a kept state to a kept state: whole histories, a few new events,
         single ones, and the gradient
  read   candidates' queries of their user's state through the map,
           O[i] = scale Q[i] S[map[i]],  and the gradient

A case is one call of one operator; `op` says which.  Lengths and the number of
candidates of each user follow from the case alone (so that the work does), values
and orders from the seed.

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

D = 128          # head dimension
GROUP = 32       # elements of the cache that share a scale
BLOCK = 2560     # bytes of 16 tokens of one head
CHUNK = 128      # tokens of a chunk of the plain scan


# ------------------------------------------------------------------ cases
def listed():
    return [
        # patches of 256 image or video candidates (8 x 8 each) at their users' time: time, height, width
        dict(name="axes_patches", op="axes", n=256, users=15, H=8, L=64, d=128, rot=128, axes=3, shared=True, interleaved=False,
             dtype="bf16", far=100000, backward=False),
        # the gradient of keys with a time and a place, half of the head, 32 bits
        dict(name="axes_keys_gradient", op="axes", n=20000, users=0, H=8, L=1, d=128, rot=64, axes=2, shared=False,
             interleaved=True, dtype="fp32", far=1000000, backward=True),
        # a draft of 8 tokens for one user: latency
        dict(name="tree_one", op="tree", cands=1, users=1, H=8, Hkv=8, Lq=8, len=1000, spread=0, page=16, branch=2, lse=False),
        # a draft of 32 tokens for each of 64 users, four heads share keys, log-sum-exp wanted
        dict(name="tree_each", op="tree", cands=64, users=64, H=16, Hkv=4, Lq=32, len=4096, spread=1000, page=64, branch=3, lse=True),
        # ten drafts of 16 tokens a user, ragged histories
        dict(name="tree_ten_each", op="tree", cands=1024, users=102, H=8, Hkv=8, Lq=16, len=2048, spread=1800, page=32, branch=2, lse=False),
        # one new event of each of 256 users, with its query: the states are the bytes
        dict(name="scan_step", op="scan", users=256, H=8, len=1, spread=0, queries=True, start=True, fused=True, backward=False),
        # 0 to 24 new events of a request's 15 users go into the states: latency
        dict(name="scan_events", op="scan", users=15, H=8, len=24, spread=24, queries=False, start=True, fused=False, backward=False),
        # whole histories of 15 users, 1200 to 2048 events
        dict(name="scan_histories", op="scan", users=15, H=8, len=2048, spread=848, queries=True, start=False, fused=True, backward=False),
        # two users with very long histories, few heads
        dict(name="scan_long", op="scan", users=2, H=4, len=30001, spread=10000, queries=True, start=False, fused=False, backward=False),
        # the gradient of 15 users' histories, between states
        dict(name="scan_gradient", op="scan", users=15, H=8, len=1024, spread=500, queries=True, start=True, fused=False, backward=True),
        # 1024 candidates of 15 users read their user's state
        dict(name="read_request", op="read", cands=1024, users=15, H=8, Lq=32, skew=1, backward=False),
        # its gradient, candidates spread unevenly over 64 users
        dict(name="read_gradient", op="read", cands=1024, users=64, H=8, Lq=16, skew=2, backward=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["axes", "tree", "tree", "scan", "scan", "scan", "read"])
    if op == "axes":
        users = rng.choice([0, _log(rng, 1, 100)])
        L, H, d = rng.choice([1, rng.randint(2, 100)]), rng.randint(1, 12), rng.choice([64, 80, 96, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        n = _log(rng, 1, max(1, 16000000 // (L * H * d * (2 if dtype == "fp32" else 1))))
        return dict(op=op, n=n, users=min(users, n), H=H, L=L, d=d, rot=rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)]),
                    axes=rng.randint(1, 4), shared=rng.random() < 0.5, interleaved=rng.random() < 0.5, dtype=dtype,
                    far=_log(rng, 1, 1000000), backward=rng.random() < 0.5)
    if op == "tree":
        group, Hkv, Lq = rng.choice([1, 1, 2, 4]), rng.choice([1, 2, 4, 8]), 8 * rng.choice([1, 1, 2, 3, 4, 8, 16])
        users = _log(rng, 1, 120)
        cands = _log(rng, users, max(users, min(1024, 20 * users, 131072 // (Hkv * group * Lq))))
        rows = cands * Hkv * group * Lq
        most = min(50000, 130000 * 2048 // rows, 1600000 // (users * Hkv))
        length = _log(rng, 1, max(1, most))
        return dict(op=op, cands=cands, users=users, H=Hkv * group, Hkv=Hkv, Lq=Lq, len=length, spread=rng.randint(0, length),
                    page=rng.choice([16, 32, 64, 128]), branch=rng.randint(1, 5), lse=rng.random() < 0.4)
    if op == "read":
        users, H, Lq = _log(rng, 1, 200), rng.randint(1, 12), 8 * rng.choice([1, 2, 3, 4])
        cands = _log(rng, users, max(users, min(1024, 200000 // (H * Lq))))
        return dict(op=op, cands=cands, users=users, H=H, Lq=Lq, skew=rng.choice([1, 1, 2]), backward=rng.random() < 0.5)
    users, H = _log(rng, 1, 800), rng.randint(1, 12)
    users = min(users, 4096 // H)
    backward = rng.random() < 0.35
    length = _log(rng, 1, max(1, min(30000, (120000 if backward else 240000) // (users * H))))
    return dict(op=op, users=users, H=H, len=length, spread=rng.randint(0, length), queries=backward or rng.random() < 0.8,
                start=rng.random() < 0.6, fused=rng.random() < 0.5, backward=backward)


def _spread(count, longest, spread):
    """Lengths longest - spread .. longest, the first the longest; a spread as long as the longest leaves some empty."""
    i = np.arange(count, dtype=np.int64)
    return longest - (i * 7919) % (spread + 1)


def _users_of(cands, users, skew):
    """The user of each candidate before they are shuffled: even, or with the first users taking most."""
    i = np.arange(cands, dtype=np.int64)
    return i * users // cands if skew == 1 else (i * i * users) // (cands * cands)


def _axis_of_pair(c):
    """The axis of each pair: the pairs in runs, one for each axis, the first axes a pair longer."""
    half = c["rot"] // 2
    return [j * c["axes"] // half for j in range(half)]


def _decays(c):
    """The decay of each head, as bits of 32: from slow to fast, one head of several without any."""
    h = np.arange(c["H"], dtype=np.float64)
    lam = 1.0 - 2.0 ** (-8.0 + 6.0 * h / c["H"])
    if c["H"] > 2:
        lam[1] = 1.0
    return lam.astype(np.float32)


# ---------------------------------------------------------------- prepare
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda")


def _keys(shape, g):
    """Keys: a few channels are several times as large as the others, as trained keys have them."""
    x = _randn(shape, g)
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
    return torch.where(used, order[at], torch.full_like(order[at], -1)).contiguous(), n_pages


def _shuffled_map(c, g):
    users = torch.from_numpy(_users_of(c["cands"], c["users"], c.get("skew", 1))).cuda().to(torch.int32)
    return users[torch.randperm(c["cands"], generator=g, device="cuda")].contiguous()


def prepare(c, seed):
    g = _gen(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = torch.bfloat16
    s = {"case": c}
    if c["op"] == "axes":
        s["x"] = _randn((c["n"], c["H"], c["L"], c["d"]), g).to(_TYPES[c["dtype"]])
        s["start"] = torch.randint(0, c["far"] + 1, (c["users"] or c["n"], c["axes"]), generator=g, **i32)
        shape = (c["L"], c["axes"]) if c["shared"] else (c["n"], c["L"], c["axes"])
        s["positions"] = torch.randint(-8, 57, shape, generator=g, **i32)
        s["axis"] = _axis_of_pair(c)
        if c["users"]:
            m = torch.from_numpy(_users_of(c["n"], c["users"], 1)).cuda().to(torch.int32)
            s["map"] = m[torch.randperm(c["n"], generator=g, device="cuda")].contiguous()
        return s
    if c["op"] == "read":
        s["map"] = _shuffled_map(c, g)
        s["Q"] = _randn((c["cands"], c["H"], c["Lq"], D), g).to(bf)
        s["S"] = _randn((c["users"], c["H"], D, D), g) * 5.0
        if c["backward"]:
            s["dO"] = _randn(s["Q"].shape, g).to(bf)
        return s
    lens = _spread(c["users"], c["len"], c["spread"])
    off = np.concatenate([[0], np.cumsum(lens)])
    s["lens"], s["rows"] = torch.from_numpy(lens).cuda().to(torch.int32), int(off[-1])
    if c["op"] == "scan":
        H, n = c["H"], s["rows"]
        s["offsets"] = torch.from_numpy(off).cuda().to(torch.int32)
        if c["fused"]:  # slices of one projection
            qkv = _randn((n, 3, H, D), g).to(bf)
            s["Q"], s["K"], s["V"] = qkv[:, 0], qkv[:, 1], qkv[:, 2]
        else:
            s["Q"], s["K"], s["V"] = (_randn((n, H, D), g).to(bf) for _ in range(3))
        s["decay"] = torch.from_numpy(_decays(c)).cuda()
        s["S"] = _randn((c["users"], H, D, D), g) * 3.0 if c["start"] else None
        if c["backward"]:
            s["dO"] = _randn((n, H, D), g).to(bf)
            s["dS"] = _randn((c["users"], H, D, D), g)
        return s
    P, Hkv, n, Lq = c["page"], c["Hkv"], c["cands"], c["Lq"]
    table, n_pages = _pages(lens, P, g)
    s.update(table=table, n_pages=n_pages)
    s["map"] = _shuffled_map(c, g)
    s["Q"] = _randn((n, c["H"], Lq, D), g).to(bf)
    s["K"], s["V"] = _keys((n, Lq, Hkv, D), g), _randn((n, Lq, Hkv, D), g).to(bf)
    # trees of different sizes: each row's parent among the last few before it (or a second root now and then), then rows that are not there
    row = torch.arange(Lq, device="cuda")[None, :]
    back = torch.randint(1, c["branch"] + 1, (n, Lq), generator=g, device="cuda")
    parent = (row - back).clamp(min=-1)
    size = torch.randint((Lq + 1) // 2, Lq + 1, (n, 1), generator=g, device="cuda")
    s["parents"] = torch.where(row < size, parent, torch.full_like(parent, -2)).to(torch.int32)
    # the cache as earlier requests left it: every page holds something, also behind a history's end
    data = torch.empty((n_pages, Hkv, P // 16, BLOCK), dtype=torch.uint8, device="cuda")
    flat = data.view(-1, BLOCK)
    for a in range(0, flat.shape[0], 32768):
        b = min(flat.shape[0], a + 32768)
        k, v = _keys(((b - a) * 16, D), g), _randn(((b - a) * 16, D), g).to(bf)
        flat[a:b] = torch.cat([_pack(x).view(b - a, -1) for x in (k, v)], dim=1)
    s["data"] = data
    return s


# ------------------------------------------------------------ plain forms
def _pack(x):
    """[tokens, 128] bf16 -> the bytes of tokens / 16 half blocks (codes, then (s, z))."""
    v = x.float().view(*x.shape[:-1], -1, GROUP)
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    s = ((hi * 0.5 - lo * 0.5) / torch.full_like(lo, 7.5)).to(torch.bfloat16).float()
    z = (lo - 16.0 * s).to(torch.bfloat16).float()
    q = torch.where(s > 0, ((v - z) / s).round() - 16.0, torch.zeros_like(v)).clamp(0.0, 15.0)
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


def _histories(data, table):
    """Keys and values [users, H, blocks * page, 128] in fp32 of every user's pages (absent ones read page 0)."""
    kv = _unpack(data[table.clamp(min=0).to(torch.int64)])   # [users, blocks, H, page / 16, 2, 16, 128]
    kv = kv.permute(4, 0, 2, 1, 3, 5, 6)
    return kv.reshape(2, table.shape[0], data.shape[1], -1, D)


def _axes(s):
    c, x = s["case"], s["x"]
    f = 10000.0 ** (-2.0 * torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda") / c["rot"])
    start = s["start"][s["map"].to(torch.int64)] if c["users"] else s["start"]
    pos = start.to(torch.float64)[:, None] + s["positions"].to(torch.float64)              # [n, L, axes]
    angle = (pos[:, :, torch.tensor(s["axis"], device="cuda")] * f)[:, None]                # [n, 1, L, rot / 2]
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


def _sees(parents):
    """[n, Lq, Lq] truth: row i reads row j (itself and its ancestors); rows that are not there read nothing."""
    n, L = parents.shape
    there = parents >= -1
    up = (parents[:, :, None] == torch.arange(L, device="cuda")).float()
    step = up + torch.eye(L, device="cuda")
    for _ in range(max(1, (L - 1).bit_length())):
        step = (step @ step > 0).float()
    return (step > 0) & there[:, :, None]


def _tree(s):
    c, Q, m = s["case"], s["Q"].float(), s["map"].to(torch.int64)
    n, H, Lq, U, Hkv = c["cands"], c["H"], c["Lq"], c["users"], c["Hkv"]
    scale = 1.0 / math.sqrt(D)
    K, V = _histories(s["data"], s["table"])
    L = K.shape[2]
    # candidates grouped by user, each group padded to the largest
    order = torch.argsort(m, stable=True)
    count = torch.bincount(m, minlength=U)
    place = torch.arange(n, device="cuda") - (count.cumsum(0) - count)[m[order]]
    most = int(count.max())
    where = m[order] * most + place
    rows = Q.new_zeros((U * most, H, Lq, D)).index_copy(0, where, Q[order])
    rows = rows.view(U, most, Hkv, H // Hkv, Lq, D).permute(0, 2, 1, 3, 4, 5).reshape(U, Hkv, -1, D)

    def back(x):
        x = x.view(U, Hkv, most, H // Hkv, Lq, -1).permute(0, 2, 1, 3, 4, 5).reshape(U * most, Hkv, -1, x.shape[-1])
        return x.new_empty((n,) + x.shape[1:]).index_copy(0, order, x[where])

    there = torch.arange(L, device="cuda")[None, :] < s["lens"][:, None]
    V = torch.where(there[:, None, :, None], V, V.new_zeros(()))
    S = torch.matmul(rows, K.transpose(-1, -2)) * scale
    S = torch.where(there[:, None, None, :], S, S.new_full((), -math.inf))
    top = S.amax(-1, keepdim=True)
    floor = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(S - floor)
    hist_sum, hist_top, hist = back(p.sum(-1, keepdim=True)), back(floor), back(torch.matmul(p, V))   # [n, Hkv, group * Lq, ..]
    # the draft's own rows
    sees = _sees(s["parents"])
    Kn, Vn = s["K"].float().transpose(1, 2), s["V"].float().transpose(1, 2)                           # [n, Hkv, Lq, D]
    q = Q.view(n, Hkv, -1, D)
    S = torch.matmul(q, Kn.transpose(-1, -2)) * scale
    mask = sees[:, None, None].expand(n, Hkv, H // Hkv, Lq, Lq).reshape(S.shape)
    S = torch.where(mask, S, S.new_full((), -math.inf))
    empty = hist_sum == 0
    top = torch.maximum(S.amax(-1, keepdim=True), torch.where(empty, torch.full_like(hist_top, -math.inf), hist_top))
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p, keep = torch.exp(S - top), torch.where(empty, torch.zeros_like(top), torch.exp(hist_top - top))
    total = p.sum(-1, keepdim=True) + keep * hist_sum
    O = (torch.matmul(p, Vn) + keep * hist) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + torch.log(total)
    gone = ~(s["parents"] >= -1)[:, None, None].expand(n, Hkv, H // Hkv, Lq).reshape(lse.shape[:3])[..., None]
    O = torch.where(gone, torch.zeros_like(O), O).view(n, H, Lq, D).to(torch.bfloat16)
    lse = torch.where(gone, torch.full_like(lse, -math.inf), lse).view(n, H, Lq)
    return [O, lse] if c["lse"] else [O]


def _powers(decay, e):
    """decay[h] ** e for whole numbers e, [H, *e.shape], formed in 64 bits."""
    return (decay.double().view(-1, *[1] * e.dim()) ** e.double()).float()


def _scan(s, x, y, z, start, scale, reverse):
    """Outputs [rows, H, D] and the last state [U, H, D, D] of a scan with queries x, keys y, values z.

    Forward:  S_t = decay S_{t-1} + y_t z_t^T from S = start, o_t = scale x_t S_t.
    Reverse:  the same from the last token to the first, with scale on the products and not on the start, which stands for
              what the last token receives already decayed; the last state is decayed once more.
    Sequences are padded in front, cut into chunks: products within a chunk, then with the states before it."""
    c, lam = s["case"], s["decay"]
    U, H = c["users"], c["H"]
    lens = s["lens"].to(torch.int64)
    C = min(CHUNK, max(1, c["len"]))
    N = -(-max(1, c["len"]) // C)
    place = torch.arange(N * C, device="cuda")[None, :] - (N * C - lens[:, None])            # the token's number in its order
    there = place >= 0
    first = s["offsets"][:-1].to(torch.int64)[:, None]
    row = torch.where(there, first + (lens[:, None] - 1 - place if reverse else place), torch.zeros_like(place))
    cut = lambda t: torch.where(there[..., None, None], t[row].float(), t.new_zeros((), dtype=torch.float32)).permute(0, 2, 1, 3).reshape(U, H, N, C, D)  # noqa: E731
    y, z = cut(y) * (scale if reverse else 1.0), cut(z)
    i = torch.arange(C, device="cuda")
    M = torch.matmul((y * _powers(lam, C - 1 - i)[None, :, None, :, None]).transpose(-1, -2), z)   # [U, H, N, D, D]
    n = torch.arange(N + 1, device="cuda")
    gap = n[:, None] - 1 - n[None, :N]
    w = torch.where(gap >= 0, _powers(lam, gap.clamp(min=0) * C), torch.zeros((), device="cuda"))   # [H, N + 1, N]
    before = torch.matmul(w, M.reshape(U, H, N, -1)).view(U, H, N + 1, D, D)
    last = before[:, :, N]
    if start is not None:
        e = lens - (1 if reverse else 0)
        carry = torch.where(e >= 0, _powers(lam, e.clamp(min=0)), torch.ones((), device="cuda")).T     # [U, H]
        last = last + carry[..., None, None] * start
    if reverse:
        last = torch.where(lens[:, None, None, None] > 0, lam[:, None, None] * last, last)
    if x is None:
        return None, last
    x = cut(x)
    A = torch.matmul(x, y.transpose(-1, -2))
    e = i[:, None] - i[None, :]
    A = A * torch.where(e >= 0, _powers(lam, e.clamp(min=0)), torch.zeros((), device="cuda"))[None, :, None]
    out = torch.matmul(A, z) + torch.matmul(x * _powers(lam, i + 1)[None, :, None, :, None], before[:, :, :N])
    out = out.view(U, H, N * C, D) * (1.0 if reverse else scale)
    if start is not None:
        e = place.clamp(min=0) + (0 if reverse else 1)
        out = out + torch.matmul(x.view(U, H, N * C, D) * _powers(lam, e).transpose(0, 1)[..., None], start) * (1.0 if reverse else scale)
    flat = out.new_zeros((s["rows"], H, D))
    flat[row[there]] = out.permute(0, 2, 1, 3)[there]
    return flat, last


def _linear(s):
    c, scale, bf = s["case"], 1.0 / math.sqrt(D), torch.bfloat16
    Q, K, V = s["Q"], s["K"], s["V"]
    if not c["backward"]:
        O, last = _scan(s, Q if c["queries"] else None, K, V, s["S"], scale, False)
        return [last] if O is None else [O.to(bf), last]
    turned = lambda t: None if t is None else t.transpose(-1, -2)  # noqa: E731
    dQ, _ = _scan(s, s["dO"], V, K, turned(s["S"]), scale, False)
    dK, _ = _scan(s, V, s["dO"], Q, turned(s["dS"]), scale, True)
    dV, dS = _scan(s, K, Q, s["dO"], s["dS"], scale, True)
    return [dQ.to(bf), dK.to(bf), dV.to(bf), dS]


def _read(s):
    c, scale, m = s["case"], 1.0 / math.sqrt(D), s["map"].to(torch.int64)
    S = s["S"][m]
    if not c["backward"]:
        return [(torch.matmul(s["Q"].float(), S) * scale).to(torch.bfloat16)]
    dO = s["dO"].float()
    dQ = (torch.matmul(dO, S.transpose(-1, -2)) * scale).to(torch.bfloat16)
    dS = torch.matmul(s["Q"].float().transpose(-1, -2), dO) * scale
    return [dQ, torch.zeros_like(s["S"]).index_add_(0, m, dS)]


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
        if c["op"] == "axes":
            freqs = binding.ikbo_rope_frequencies(c["rot"], base=10000.0)
            s["rope"] = binding.Rope(c["rot"], freqs, interleaved=c["interleaved"], axes=s["axis"], n_axes=c["axes"])
    return s["plan"].plan


def _own(s):
    c, p = s["case"], _plan(s)
    if c["op"] == "axes":
        y = torch.empty_like(s["x"])
        call = p.rope_axes_backward if c["backward"] else p.rope_axes_forward
        call(s["rope"], s["x"], y, positions=s["positions"], start=s["start"], broadcast=bool(c["users"]))
        return y
    if c["op"] == "tree":
        O = torch.empty_like(s["Q"])
        lse = s["Q"].new_empty(s["Q"].shape[:3], dtype=torch.float32) if c["lse"] else None
        p.attn_qcache_tree_forward(s["Q"], s["data"], c["page"], s["table"], s["lens"], s["K"], s["V"], s["parents"], O, lse=lse,
                                   Lkv=max(1, s["rows"]))
        return [O] if lse is None else [O, lse]
    if c["op"] == "read":
        if not c["backward"]:
            O = torch.empty_like(s["Q"])
            p.linattn_read_forward(s["Q"], s["S"], O)
            return [O]
        dQ, dS = torch.empty_like(s["Q"]), torch.empty_like(s["S"])
        p.linattn_read_backward(s["Q"], s["S"], s["dO"], dQ, dS)
        return [dQ, dS]
    rows = lambda: torch.empty((s["rows"], c["H"], D), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    last = torch.empty((c["users"], c["H"], D, D), dtype=torch.float32, device="cuda")
    if c["backward"]:
        dQ, dK, dV = rows(), rows(), rows()
        p.linattn_backward(s["Q"], s["K"], s["V"], s["dO"], s["decay"], dQ, dK, dV, state_in=s["S"], d_state_out=s["dS"],
                           d_state_in=last, offsets=s["offsets"], max_len=c["len"])
        return [dQ, dK, dV, last]
    O = rows() if c["queries"] else None
    p.linattn_forward(s["Q"] if c["queries"] else None, s["K"], s["V"], s["decay"], O, state_in=s["S"], state_out=last,
                      offsets=s["offsets"], max_len=c["len"])
    return [last] if O is None else [O, last]


_PLAIN = {"axes": _axes, "tree": _tree, "scan": _linear, "read": _read}


def run(s):
    if own:
        return _own(s)
    return _PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------- work
def work(c):
    if c["op"] == "axes":
        values = c["n"] * c["H"] * c["L"] * c["d"]
        size = 4 if c["dtype"] == "fp32" else 2
        places = c["axes"] * ((c["users"] or c["n"]) + c["L"] * (1 if c["shared"] else c["n"]))
        return {"bytes": 2 * values * size + 4 * places + (4 * c["n"] if c["users"] else 0),
                "flops": 3 * c["n"] * c["H"] * c["L"] * c["rot"]}
    if c["op"] == "read":
        values, states = c["cands"] * c["H"] * c["Lq"] * D, c["users"] * c["H"] * D * D
        k = 3 if c["backward"] else 2
        return {"bytes": k * values * 2 + (k - 1) * states * 4 + 4 * c["cands"], "flops": (k - 1) * 2 * values * D}
    lens = _spread(c["users"], c["len"], c["spread"])
    rows = int(lens.sum())
    if c["op"] == "scan":
        values, states = rows * c["H"] * D, c["users"] * c["H"] * D * D
        if c["backward"]:  # by single tokens: two states kept up and three read, 2 D products an element each
            return {"bytes": 7 * values * 2 + 4 * states * (3 if c["start"] else 2), "flops": 5 * 2 * values * D}
        return {"bytes": (4 if c["queries"] else 2) * values * 2 + 4 * states * (2 if c["start"] else 1),
                "flops": (2 if c["queries"] else 1) * 2 * values * D}
    per = np.bincount(_users_of(c["cands"], c["users"], 1), minlength=c["users"])
    read = int(lens[per > 0].sum())
    values, drafted = c["cands"] * c["H"] * c["Lq"] * D, c["cands"] * c["Hkv"] * c["Lq"] * D
    return {"bytes": read * c["Hkv"] * 160 + 4 * values + 4 * drafted + (4 * values // D if c["lse"] else 0) + 4 * c["cands"] * (c["Lq"] + 1)
            + 4 * (rows // c["page"]), "flops": 4 * D * c["H"] * c["Lq"] * int((per * lens).sum() + c["cands"] * c["Lq"] // 2)}


# ------------------------------------------------- the definition, 64 bits
def _recur(q, k, v, lam, S, scale):
    """One user: q, k, v [H, L, D], S [H, D, D], block by block."""
    out, lam = [], lam.view(-1, 1, 1)
    for a in range(0, k.shape[1], 64):
        kb, vb = k[:, a:a + 64], v[:, a:a + 64]
        B = kb.shape[1]
        t = torch.arange(B, dtype=torch.float64, device="cuda").view(1, -1, 1)
        if q is not None:
            qb = q[:, a:a + 64]
            gap = t - t.transpose(1, 2)
            w = torch.where(gap >= 0, lam ** gap.clamp(min=0), 0.0)
            out.append(scale * (((qb @ kb.transpose(1, 2)) * w) @ vb + (lam ** (t + 1) * qb) @ S))
        S = lam ** B * S + (lam ** (B - 1 - t) * kb).transpose(1, 2) @ vb
    return (torch.cat(out, dim=1) if out else None), S


def _exact_scan(s):
    c, lens, scale = s["case"], s["lens"].tolist(), 1.0 / math.sqrt(D)
    H, lam = c["H"], s["decay"].double()
    names = ("Q", "K", "V") if c["queries"] else ("K", "V")
    res = {n: torch.zeros((s["rows"], H, D), dtype=torch.float64, device="cuda") for n in names}
    last = torch.zeros((c["users"], H, D, D), dtype=torch.float64, device="cuda")
    a = 0
    for u, n in enumerate(lens):
        S = s["S"][u].double() if s["S"] is not None else torch.zeros((H, D, D), dtype=torch.float64, device="cuda")
        x = {k: s[k][a:a + n].double().transpose(0, 1) for k in names}
        if c["backward"]:
            S.requires_grad_(True)
            x = {k: t.detach().requires_grad_(True) for k, t in x.items()}
        o, end = _recur(x.get("Q"), x["K"], x["V"], lam, S, scale)
        if c["backward"]:
            total = (end * s["dS"][u].double()).sum()
            if o is not None:
                total = total + (o * s["dO"][a:a + n].double().transpose(0, 1)).sum()
            total.backward()
            for k in names:
                if n:
                    res[k][a:a + n] = x[k].grad.transpose(0, 1)
            last[u] = S.grad
        else:
            if o is not None:
                res["Q"][a:a + n] = o.transpose(0, 1)
            last[u] = end
        a += n
    if c["backward"]:
        return [res["Q"], res["K"], res["V"], last]
    return [res["Q"], last] if c["queries"] else [last]


def _exact_tree(s):
    c = s["case"]
    n, H, Lq, Hkv, P = c["cands"], c["H"], c["Lq"], c["Hkv"], c["page"]
    O = torch.zeros((n, H, Lq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((n, H, Lq), -math.inf, dtype=torch.float64, device="cuda")
    lens, m = s["lens"].tolist(), s["map"].long()
    parents = s["parents"].cpu().numpy()
    line = np.zeros((n, Lq, Lq), dtype=bool)   # the rows on the way up, row by row
    for j in range(Lq):
        for i in np.nonzero(parents[:, j] >= -1)[0]:
            if parents[i, j] >= 0:
                line[i, j] = line[i, parents[i, j]]
            line[i, j, j] = True
    line = torch.from_numpy(line).cuda()
    G = H // Hkv
    for u in range(c["users"]):
        who = torch.nonzero(m == u).flatten()
        if not len(who):
            continue
        blocks = (lens[u] + P - 1) // P
        raw = s["data"][s["table"][u, :blocks].long()].transpose(0, 1).reshape(Hkv, -1, BLOCK)
        kv = []
        for a in (0, 1280):
            codes = raw[..., a:a + 1024].reshape(Hkv, -1, 64)
            code = torch.empty((Hkv, codes.shape[1], D), dtype=torch.float64, device="cuda")
            code[..., 0::2], code[..., 1::2] = (codes % 16).double(), (codes // 16).double()
            pair = raw[..., a + 1024:a + 1280].contiguous().view(torch.bfloat16).reshape(Hkv, -1, 4, 2).double()
            step, zero = (pair[..., i].repeat_interleave(GROUP, dim=-1) for i in (0, 1))
            kv.append((zero + (16.0 + code) * step).to(torch.bfloat16).double()[:, :lens[u]])
        there = line[who].any(-1)                                                             # [w, Lq]
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            q = s["Q"][who][:, heads].double()                                                 # [w, G, Lq, D]
            k, v = s["K"][who][:, :, h].double(), s["V"][who][:, :, h].double()                # [w, Lq, D]
            far = q @ kv[0][h].T / math.sqrt(D)
            near = torch.einsum("wgid,wjd->wgij", q, k) / math.sqrt(D)
            near = near.masked_fill(~line[who][:, None], -math.inf)
            logits = torch.cat([far, near], dim=-1)
            total = torch.logsumexp(logits, dim=-1)
            p = torch.exp(logits - total[..., None])
            o = p[..., :far.shape[-1]] @ kv[1][h] + torch.einsum("wgij,wjd->wgid", p[..., far.shape[-1]:], v)
            O[who, heads] = torch.where(there[:, None, :, None], o, 0.0)
            lse[who, heads] = torch.where(there[:, None], total, -math.inf)
    return [O, lse] if c["lse"] else [O]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "scan":
        return _exact_scan(s)
    if c["op"] == "tree":
        return _exact_tree(s)
    if c["op"] == "read":
        O, dO, S = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda"), s.get("dO"), s["S"].double() / math.sqrt(D)
        dS = torch.zeros_like(S)
        for u in range(c["users"]):
            who = torch.nonzero(s["map"].long() == u).flatten()
            q = s["Q"][who].double()
            if dO is None:
                O[who] = torch.einsum("ihld,hde->ihle", q, S[u])
            else:
                O[who] = torch.einsum("ihle,hde->ihld", dO[who].double(), S[u])
                dS[u] = torch.einsum("ihld,ihle->hde", q, dO[who].double()) / math.sqrt(D)
        return [O] if dO is None else [O, dS]
    x, half = s["x"].double(), c["rot"] // 2
    pos = (s["start"][s["map"].long()] if c["users"] else s["start"]).double()
    pos = pos[:, None, :] + s["positions"].double()
    out = x.clone()
    for j in range(half):
        f = math.exp(-2.0 * j / c["rot"] * math.log(10000.0))
        a = (pos[..., s["axis"][j]] * (-f if c["backward"] else f))[:, None, :]
        i, k = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
        out[..., i] = x[..., i] * torch.cos(a) - x[..., k] * torch.sin(a)
        out[..., k] = x[..., i] * torch.sin(a) + x[..., k] * torch.cos(a)
    return out
