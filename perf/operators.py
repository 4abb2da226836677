"""What is measured of the 8-bit key/value cache and its rotary positions: the cases, their inputs, the
operators in plain torch, and the library's calls of the same operators.

Three operators. Shapes are those of token-pruned video attention: a latent video of F x Hs x Ws tokens,
token n = (f * Hs + y) * Ws + x, H heads of d channels, an ascending list idx of the active tokens with its
count on the device, and `pad` rows behind the count that every operator leaves as they were.

rope   Rows j < count of q (and of k) turned to the position (f, x, y) of token idx[j]: a head's channels are
       the groups [t | x | y] of dims[a] channels, adjacent channels are a pair, pair j of group a turns by
       position_a * base^(-2j / dims[a]). The turn back (`back`) is its gradient.
sync   The fresh keys (turned the same way) and values of the active tokens go into a cache held in 8 bits
       (e4m3) with one power-of-two scale for each block of 128 tokens and head. The scale of a block is the
       smallest 2^e with amax <= 448 * 2^e; it only grows while some of the block's tokens are not fresh, and
       the values that stay are then held at the new scale.
attn   Active queries over all N keys and values of that cache, optionally only over the key blocks that the
       query's own block of 128 tokens keeps, with the log-sum-exp of each row's logits.
"""
import math

import torch

own = False

BLOCK = 128          # tokens of a scale block and of a mask block
BASE = 10000.0
E4M3 = torch.float8_e4m3fn


# ---- cases -------------------------------------------------------------------------------------------
def _rope(name, F, Hs, Ws, H, d, A, pad=0, both=True, back=False):
    return dict(name=name, op="rope", F=F, Hs=Hs, Ws=Ws, H=H, d=d, A=A, pad=pad, both=both, back=back)


def _sync(name, F, Hs, Ws, H, d, A, pad=0, run=False):
    return dict(name=name, op="sync", F=F, Hs=Hs, Ws=Ws, H=H, d=d, A=A, pad=pad, run=run)


def _attn(name, F, Hs, Ws, H, d, A, pad=0, keep=0, lse=False):
    return dict(name=name, op="attn", F=F, Hs=Hs, Ws=Ws, H=H, d=d, A=A, pad=pad, keep=keep, lse=lse)


def listed():
    return [
        # a few tokens of a thumbnail video: the launch is what counts
        _rope("rope tiny", 4, 8, 8, 2, 64, 100, pad=28),
        # the gradient of a rotation at the middle size, one tensor, every third token
        _rope("rope mid back", 13, 30, 52, 12, 128, 6761, both=False, back=True),
        # queries and keys of one step at the largest video, a third of the tokens active
        _rope("rope hsa", 33, 45, 80, 24, 128, 39600),
        # the same thumbnail, cache update
        _sync("sync tiny", 4, 8, 8, 2, 64, 100, pad=28),
        # a streaming chunk: whole new frames appended, so that most blocks are replaced entire
        _sync("sync frames", 21, 30, 52, 12, 128, 7800, run=True),
        # a pruned step at the largest video, active tokens scattered over every block
        _sync("sync hsa", 33, 45, 80, 24, 128, 39600),
        # the thumbnail's attention
        _attn("attn tiny", 4, 8, 8, 2, 64, 100, pad=28, lse=True),
        # one token over the whole cache of the largest video: the cache's bytes are what counts
        _attn("attn one", 33, 45, 80, 24, 128, 1),
        # a handful of changed tokens, odd sizes, small heads, two key sets to be merged later
        _attn("attn few", 7, 31, 53, 5, 64, 67, pad=3, lse=True),
        # key blocks kept for each query block
        _attn("attn blocks", 13, 30, 52, 12, 128, 8111, keep=24),
        # a pruned step of the middle video
        _attn("attn mid", 13, 30, 52, 12, 128, 6084),
        # half of the tokens of the wider video
        _attn("attn wan", 21, 30, 52, 12, 128, 16380),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "sync", "attn"])
    d = rng.choice([64, 128])
    if op == "attn":
        F, Hs, Ws = rng.randint(1, 21), rng.randint(3, 30), rng.randint(3, 52)
        H = rng.randint(1, 12)
        N = F * Hs * Ws
        A = min(N, _log(rng, 1, max(2, N // 2)))
        nb = -(-N // BLOCK)
        keep = rng.randint(1, nb) if rng.random() < 0.3 else 0
        return dict(op=op, F=F, Hs=Hs, Ws=Ws, H=H, d=d, A=A, pad=rng.choice([0, 0, 5]), keep=keep,
                    lse=rng.random() < 0.5)
    F, Hs, Ws = rng.randint(1, 33), rng.randint(3, 45), rng.randint(3, 80)
    H = rng.randint(1, 24)
    N = F * Hs * Ws
    A = min(N, 39600, _log(rng, 1, N))
    if op == "rope":
        return dict(op=op, F=F, Hs=Hs, Ws=Ws, H=H, d=d, A=A, pad=rng.choice([0, 0, 9]),
                    both=rng.random() < 0.5, back=rng.random() < 0.3)
    return dict(op=op, F=F, Hs=Hs, Ws=Ws, H=H, d=d, A=A, pad=rng.choice([0, 0, 9]), run=rng.random() < 0.4)


def work(case):
    F, Hs, Ws, H, d, A = (case[k] for k in ("F", "Hs", "Ws", "H", "d", "A"))
    N = F * Hs * Ws
    nb = -(-N // BLOCK)
    row = H * d
    if case["op"] == "rope":
        n = 2 if case["both"] else 1
        return {"bytes": A * 4 + n * A * row * 4, "flops": n * A * row * 3}
    if case["op"] == "sync":
        return {"bytes": A * 4 + 2 * A * row * 2 + 2 * A * row + 4 * nb * H * 4, "flops": A * row * 3 + 2 * A * row * 2}
    keys = min(N, case["keep"] * BLOCK) if case["keep"] else N
    return {"bytes": A * row * 4 + 2 * N * row + 2 * nb * H * 4 + (A * H * 4 if case["lse"] else 0)
            + (nb * nb if case["keep"] else 0), "flops": 4 * A * keys * row}


# ---- inputs ------------------------------------------------------------------------------------------
def _dims(d):
    g = 2 * (d // 6)
    return d - 2 * g, g, g


def _table(dims, sizes, dev):
    """(cos, sin) of every position and pair of the axes t, x, y, in 64 bits and rounded once: [entries, 2]."""
    parts = []
    for da, size in zip(dims, sizes):
        freq = BASE ** (-2.0 * torch.arange(da // 2, dtype=torch.float64, device=dev) / da)
        phi = torch.arange(size, dtype=torch.float64, device=dev)[:, None] * freq
        parts.append(torch.stack([phi.cos(), phi.sin()], -1).reshape(-1, 2))
    return torch.cat(parts).float().contiguous()


def _hold(x):
    """A [N, H, d] tensor as its e4m3 codes and the scales [nb, H] of its blocks."""
    N, H, d = x.shape
    nb = -(-N // BLOCK)
    amax = torch.zeros(nb * BLOCK, H, device=x.device)
    amax[:N] = x.abs().amax(-1)
    s = _scale_of(amax.view(nb, BLOCK, H).amax(1))
    return (x / s.repeat_interleave(BLOCK, 0)[:N, :, None]).to(E4M3), s


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, by the exponent and the fraction of amax; 0 for 0."""
    frac, ex = torch.frexp(amax)
    e = torch.where(frac <= 0.875, ex - 9, ex - 8).clamp(-100, 100)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    F, Hs, Ws, H, d, A, pad = (case[k] for k in ("F", "Hs", "Ws", "H", "d", "A", "pad"))
    N = F * Hs * Ws
    nb = -(-N // BLOCK)
    cap = A + pad

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if case.get("run"):
        first = int(torch.randint(0, N - A + 1, (1,), generator=g, device=dev))
        idx = torch.arange(first, first + A, device=dev)
    else:
        idx = torch.randperm(N, generator=g, device=dev)[:A].sort().values
    idx = torch.cat([idx, idx.new_zeros(pad)]).to(torch.int32)
    s = {"case": dict(case), "idx": idx, "count": torch.tensor([A], dtype=torch.int32, device=dev)}
    if case["op"] != "attn":
        s["dims"], s["grid"] = _dims(d), (F, Hs, Ws)
        s["table"] = _table(s["dims"], (F, Ws, Hs), dev)
    if case["op"] == "rope":
        s["q"] = rand(cap, H, d).bfloat16()
        s["q_out"] = rand(cap, H, d).bfloat16()
        if case["both"]:
            s["k"] = rand(cap, H, d).bfloat16()
            s["k_out"] = rand(cap, H, d).bfloat16()
        return s
    # the cache: heads of different strength, and blocks whose largest value differs
    strength = torch.exp(0.5 * rand(nb, H)).repeat_interleave(BLOCK, 0)[:N, :, None]
    s["k8"], s["ks"] = _hold(rand(N, H, d) * strength.clamp(max=1.5))
    s["v8"], s["vs"] = _hold(rand(N, H, d) * strength)
    if case["op"] == "sync":
        louder = torch.exp(0.3 * rand(cap, H, 1))
        s["k"] = (rand(cap, H, d) * louder).bfloat16()
        s["v"] = (rand(cap, H, d) * louder).bfloat16()
        return s
    s["q"] = (2.0 * rand(cap, H, d)).bfloat16()
    s["scale"] = 1.0 / math.sqrt(d)
    s["o"] = rand(cap, H, d).bfloat16()
    s["lse"] = rand(cap, H) if case["lse"] else None
    s["mask"] = None
    if case["keep"]:
        order = torch.rand(nb, nb, generator=g, device=dev).argsort(1)
        s["mask"] = (order < case["keep"]).to(torch.uint8)
    return s


# ---- the operators -------------------------------------------------------------------------------------
def run(s):
    if own:
        return _library(s)
    return {"rope": _plain_rope, "sync": _plain_sync, "attn": _plain_attn}[s["case"]["op"]](s)


def _library(s):
    from token_pruned_sparse_b200 import tps

    c = s["case"]
    if c["op"] == "rope":
        tps.rope_rows(s["q"], s["idx"], s["count"], s["table"], s["dims"], s["grid"], dst=s["q_out"],
                      src2=s.get("k"), dst2=s.get("k_out"), inverse=c["back"])
        return [s["q_out"], s["k_out"]] if c["both"] else [s["q_out"]]
    if c["op"] == "sync":
        tps.kv_sync_q8(s["k8"], s["v8"], s["ks"], s["vs"], s["k"], s["v"], s["idx"], s["count"],
                       rope=(s["table"], s["dims"], s["grid"]))
        return [s["k8"], s["v8"], s["ks"], s["vs"]]
    tps.pruned_attn_q8(s["q"], s["k8"], s["v8"], s["ks"], s["vs"], s["idx"], s["count"], s["scale"],
                       blockmask=s["mask"], o_act=s["o"], lse=s["lse"])
    return [s["o"], s["lse"]] if c["lse"] else [s["o"]]


def _turn(x, s, back=False):
    """x [rows, H, d] in 32 bits, its row j at the position of token idx[j]."""
    F, Hs, Ws = s["grid"]
    n = s["idx"].long()
    entries, at = [], 0
    for pos, da, size in zip((n // (Hs * Ws), n % Ws, (n // Ws) % Hs), s["dims"], (F, Ws, Hs)):
        entries.append(s["table"][at:at + size * (da // 2)].view(size, da // 2, 2)[pos])
        at += size * (da // 2)
    cs = torch.cat(entries, 1)[:, None]
    c, w = cs[..., 0], (-cs[..., 1] if back else cs[..., 1])
    a, b = x.float()[..., 0::2], x.float()[..., 1::2]
    return torch.stack([a * c - b * w, a * w + b * c], -1).flatten(-2)


def _plain_rope(s):
    c = s["case"]
    live = (torch.arange(s["idx"].numel(), device=s["idx"].device) < s["count"])[:, None, None]
    got = [torch.where(live, _turn(s["q"], s, c["back"]).bfloat16(), s["q_out"])]
    if c["both"]:
        got.append(torch.where(live, _turn(s["k"], s, c["back"]).bfloat16(), s["k_out"]))
    return got


def _plain_sync(s):
    A = s["case"]["A"]
    idx = s["idx"][:A].long()
    _plain_store(s["k8"], s["ks"], _turn(s["k"], s)[:A], idx)
    _plain_store(s["v8"], s["vs"], s["v"][:A].float(), idx)
    return [s["k8"], s["v8"], s["ks"], s["vs"]]


def _plain_store(codes, scale, x, idx):
    N, H, d = codes.shape
    nb = scale.shape[0]
    block = idx // BLOCK
    amax = torch.zeros_like(scale).scatter_reduce_(0, block[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    fresh = torch.bincount(block, minlength=nb)
    size = torch.bincount(torch.arange(N, device=idx.device) // BLOCK, minlength=nb)
    need = _scale_of(amax)
    new = torch.where((fresh == size)[:, None], need, torch.maximum(need, scale))
    new = torch.where((fresh > 0)[:, None], new, scale)
    turn = torch.where(new > 0, scale / new, torch.zeros_like(new)).repeat_interleave(BLOCK, 0)[:N, :, None]
    held = (codes.float() * turn).to(E4M3).view(torch.uint8)
    per = torch.where(new > 0, new, torch.ones_like(new))[block][:, :, None]
    held[idx] = (x / per).to(E4M3).view(torch.uint8)
    codes.copy_(held.view(E4M3))
    scale.copy_(new)


def _plain_attn(s):
    idx, q = s["idx"], s["q"]
    N, H, d = s["k8"].shape
    k = s["k8"].float() * s["ks"].repeat_interleave(BLOCK, 0)[:N, :, None]
    v = s["v8"].float() * s["vs"].repeat_interleave(BLOCK, 0)[:N, :, None]
    x = torch.matmul(q.float().transpose(0, 1), k.permute(1, 2, 0)).mul_(s["scale"])      # [H, rows, N]
    if s["mask"] is not None:
        kept = s["mask"][idx.long() // BLOCK].bool().repeat_interleave(BLOCK, 1)[:, :N]
        x.masked_fill_(~kept, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.transpose(0, 1)) / torch.where(total > 0, total, torch.ones_like(total))
    live = torch.arange(idx.numel(), device=idx.device) < s["count"]
    got = [torch.where(live[:, None, None], o.transpose(0, 1).bfloat16(), s["o"])]
    if s["lse"] is not None:
        got.append(torch.where(live[:, None], (top + total.log())[..., 0].transpose(0, 1), s["lse"]))
    return got


# ---- the same from the definition, in 64 bits ------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    A, d = case["A"], case["d"]
    idx = s["idx"][:A].long()
    if case["op"] == "attn":
        return _exact_attn(case, s, idx)
    F, Hs, Ws = s["grid"]
    pos = (idx // (Hs * Ws), idx % Ws, (idx // Ws) % Hs)
    angle = torch.cat([p.double()[:, None] * BASE ** (-torch.arange(0, da, 2, device=idx.device).double() / da)
                       for p, da in zip(pos, s["dims"])], 1)
    spin = torch.polar(torch.ones_like(angle), -angle if case.get("back") else angle)[:, None]

    def turned(x):
        z = torch.view_as_complex(x[:A].double().reshape(A, case["H"], d // 2, 2)) * spin
        return torch.view_as_real(z).reshape(A, case["H"], d)

    if case["op"] == "rope":
        outs = []
        for name in ("q", "k") if case["both"] else ("q",):
            o = s[name + "_out"].double()
            o[:A] = turned(s[name])
            outs.append(o)
        return outs
    k, ks = _exact_store(s["k8"], s["ks"], turned(s["k"]), idx)
    v, vs = _exact_store(s["v8"], s["vs"], s["v"][:A].double(), idx)
    return [k, v, ks, vs]


def _nearest_e4m3(x):
    """x in 64 bits on the grid of e4m3: 3 bits behind the leading one, steps of 2^-9 at the least, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_store(codes, scale, x, idx):
    N, H, d = codes.shape
    values, scales = codes.double(), scale.double()
    where = torch.full((scale.shape[0] * BLOCK,), -1, dtype=torch.long, device=idx.device)
    where[idx] = torch.arange(idx.numel(), device=idx.device)
    ladder = torch.exp2(torch.arange(-100, 101, device=idx.device).double())
    for b in torch.unique(idx // BLOCK).tolist():
        lo, hi = b * BLOCK, min(N, (b + 1) * BLOCK)
        rows = where[lo:hi]
        live = rows >= 0
        fresh = x[rows[live]]
        top = fresh.abs().amax((0, 2))
        need = torch.where(top > 0, ladder[torch.searchsorted(448.0 * ladder, top).clamp(max=200)], 0.0)
        new = need if bool(live.all()) else torch.maximum(need, scales[b])
        per = torch.where(new > 0, new, 1.0)[:, None]
        block = values[lo:hi] * scales[b][:, None]
        block[live] = fresh
        values[lo:hi] = _nearest_e4m3(block / per)
        scales[b] = new
    return values, scales


def _exact_attn(case, s, idx):
    A, H = case["A"], case["H"]
    N = s["k8"].shape[0]
    block = torch.arange(N, device=idx.device) // BLOCK
    outs = [s["o"].double()]
    lse = None if s["lse"] is None else s["lse"].double()
    for h in range(H):
        k = s["k8"][:, h].double() * s["ks"][block, h].double()[:, None]
        v = s["v8"][:, h].double() * s["vs"][block, h].double()[:, None]
        for at in range(0, A, 4096):
            rows = slice(at, min(A, at + 4096))
            x = s["q"][rows, h].double() @ k.T * s["scale"]
            if s["mask"] is not None:
                x = torch.where(s["mask"][idx[rows] // BLOCK][:, block] > 0, x, -math.inf)
            outs[0][rows, h] = torch.softmax(x, -1) @ v
            if lse is not None:
                lse[rows, h] = torch.logsumexp(x, -1)
    return outs if lse is None else outs + [lse]
