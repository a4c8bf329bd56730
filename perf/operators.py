"""The softmax-attention layer that alternates with the Gated DeltaNet layers of a hybrid model, at decode time:
what is measured of its operators, and their plain forms.

  append  : RMSNorm of each q and k head, rotary positions, k and v stored into the paged cache
  attn    : 1 to 16 new tokens per sequence over the paged cache
  branch  : the page tables of a search step: last step's children dropped, new ones forked from their parents,
            their next pages reserved, the partly filled pages and the GDN slots copied
  compact : the live pages moved to the front of the pool after sequences have left

Head shapes: 16 query and 2 key/value heads of 256 with a quarter of each head rotated (next to GDN layers of 16
and 32 heads of 128), and the common 32 query and 8 key/value heads of 128.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
EPS = 1e-6


# --------------------------------------------------------------------------------------------------- the cases
def listed():
    a = dict(op="append", Hq=16, Hkv=2, d=256, R=64, interleaved=False, page=64, kv="bf16", gated=True, yarn=False)
    t = dict(op="attn", Hq=16, Hkv=2, d=256, page=64, kv="bf16", gated=True, window=0, softcap=0.0)
    return [
        # one chat, one token: latency
        dict(a, name="append_b1", B=1, T=1, ragged=False, max_len=4096),
        # a ragged step of a wide batch with an 8-bit cache, positions far past the trained length
        dict(a, name="append_ragged_e4m3", B=200, T=16, ragged=True, max_len=1000000, Hq=32, Hkv=8, d=128, R=128,
             interleaved=True, page=16, kv="e4m3", gated=False, yarn=True),
        # 16 drafted tokens for each of 256 sequences
        dict(a, name="append_b256_t16", B=256, T=16, ragged=False, max_len=32768),
        # one chat, one token, a short context: latency
        dict(t, name="attn_b1_short", B=1, T=1, ragged=False, min_len=509, max_len=509),
        # one document of a quarter of a million tokens
        dict(t, name="attn_b1_long", B=1, T=1, ragged=False, min_len=262143, max_len=262143),
        # the ordinary step of a serving batch
        dict(t, name="attn_b64", B=64, T=1, ragged=False, min_len=200, max_len=12000),
        # 16 drafted tokens verified at once (128 query rows for each key/value head)
        dict(t, name="attn_verify_b32_t16", B=32, T=16, ragged=False, min_len=1000, max_len=8000),
        # mixed counts on an 8-bit cache, capped scores, a sliding window, small pages of an odd size
        dict(t, name="attn_ragged_e4m3", B=96, T=4, ragged=True, min_len=1, max_len=16000, Hq=32, Hkv=8, d=128,
             page=24, kv="e4m3", gated=False, window=4096, softcap=30.0),
        # the largest batch: 256 long conversations
        dict(t, name="attn_b256", B=256, T=1, ragged=False, min_len=500, max_len=16000),
        # a search of two beams in one sequence
        dict(op="branch", name="branch_n2", n=2, fan=2, page=16, layers=1, Hkv=2, d=128, max_len=400, T=1, Hv=4, dk=64),
        # 32 children of 8 parents, four layers of cache and the GDN state of the slot
        dict(op="branch", name="branch_n32", n=32, fan=4, page=64, layers=4, Hkv=2, d=256, max_len=16000, T=8, Hv=32, dk=128),
        # a pool half emptied by sequences that left
        dict(op="compact", name="compact_2k", pages=2000, slots=48, live=0.5, page=64, layers=2, Hkv=2, d=256),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "branch", "compact"])
    d = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8, 16])
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    T = rng.choice([1, 1, 1, 2, 3, 4, 7, 16])
    if op == "append":
        while Hkv * G > 64:
            G //= 2
        R = rng.choice([d, d // 2, d // 4, 2 * rng.randint(1, d // 2)])
        return dict(op=op, B=_logint(rng, 1, 256), T=T, ragged=rng.random() < 0.4, Hq=Hkv * G, Hkv=Hkv, d=d, R=R,
                    interleaved=rng.random() < 0.5, page=page, kv=kv, gated=rng.random() < 0.5,
                    yarn=rng.random() < 0.3, max_len=_logint(rng, 16, 1000000))
    if op == "attn":
        while Hkv * G > 64:
            G //= 2
        # at most about a gigabyte of cache, and 200 million scores in the plain form
        B = _logint(rng, 1, 256)
        most = min(262143, 2 ** 30 // (B * Hkv * d * 4), 200_000_000 // (B * T * Hkv * G))
        hi = _logint(rng, 16, max(17, most))
        page = max(page, 8) if hi > 4096 else page
        return dict(op=op, B=B, T=T, ragged=rng.random() < 0.4, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, kv=kv,
                    gated=rng.random() < 0.5, min_len=max(1, hi // rng.choice([1, 2, 16, 100])), max_len=hi,
                    window=rng.choice([0, 0, _logint(rng, 1, 8192)]), softcap=rng.choice([0.0, 0.0, 20.0, 50.0]))
    layers = rng.randint(1, 4)
    if op == "branch":
        n = _logint(rng, 1, 32)
        return dict(op=op, n=n, fan=rng.randint(-(-n // 8), 4), page=page, layers=layers, Hkv=min(Hkv, 2), d=d,
                    max_len=_logint(rng, 8, 16000 if page >= 32 else 2000), T=T, Hv=rng.choice([4, 16, 32]),
                    dk=rng.choice([64, 128]))
    pages = _logint(rng, 16, 2000)
    return dict(op=op, pages=pages, slots=rng.randint(1, 64), live=rng.choice([0.1, 0.5, 0.7, 0.95]),
                page=min(page, 64), layers=min(layers, 2), Hkv=min(Hkv, 2), d=d)


# -------------------------------------------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17), torch.Generator().manual_seed(int(seed) * 104729 + 5)


def _counts(c, cpu):
    """Tokens of each sequence in this call: T, or when ragged every count from 0 to T about as often, in any order."""
    if not c["ragged"]:
        return torch.full((c["B"],), c["T"], dtype=torch.int64)
    return (c["T"] - torch.arange(c["B"]) % (c["T"] + 1))[torch.randperm(c["B"], generator=cpu)]


def _inv_freq(c):
    """Rotation speed of each pair (radians a token) and the factor on cos and sin. yarn: positions stretched by 8
    over a trained length of 8192 (the slow pairs interpolated, the fast ones kept)."""
    R, theta = c["R"], 1e6
    i = torch.arange(R // 2, dtype=F64)
    f = theta ** (-2.0 * i / R)
    if not c["yarn"]:
        return f.to(F32).to(DEV), 1.0
    at = lambda turns: R * math.log(8192 / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), R - 1)
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return (f / 8 * ramp + f * (1 - ramp)).to(F32).to(DEV), 0.1 * math.log(8.0) + 1.0


def _quant(x, scale):
    return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)


def _batch(c, cpu, n, lens):
    """Slots, offsets and table rows that a serving program holds: sequences in random slots of twice as many."""
    B, rows = c["B"], 2 * c["B"]
    slots = torch.randperm(rows, generator=cpu)[:B]
    seq_lens = torch.zeros(rows, dtype=torch.int64)
    seq_lens[slots] = lens
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    return slots, seq_lens, cu


def _prepare_append(c, seed):
    gpu, cpu = _gen(seed)
    B, Hq, Hkv, d, ps = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    n = _counts(c, cpu)
    total = int(n.sum())
    lens = torch.randint(0, c["max_len"], (B,), generator=cpu)
    slots, seq_lens, cu = _batch(c, cpu, n, lens)
    # the pages that this step writes are the sequence's own; earlier ones are a shared prefix (page 0)
    width = -(-(c["max_len"] + c["T"]) // ps)
    first, last = lens // ps, (lens + n.clamp(min=1) - 1) // ps
    held = (last - first + 1)
    start = held.cumsum(0) - held + 1
    pages = 1 + B * ((c["T"] + ps - 2) // ps + 1)
    ids = torch.randperm(pages - 1, generator=cpu) + 1
    table = torch.zeros(2 * B, width, dtype=torch.int64)
    j = torch.arange(int(held.max()))
    for b in range(B):
        h = int(held[b])
        table[slots[b], first[b]:first[b] + h] = ids[start[b] - 1 + j[:h]]
    qd = 2 * d if c["gated"] else d
    proj = torch.randn(total, Hq * qd + 2 * Hkv * d, generator=gpu, device=DEV).to(BF16)
    inv, factor = _inv_freq(c)
    kv = BF16 if c["kv"] == "bf16" else torch.float8_e4m3fn
    s = dict(c=c, proj=proj, inv=inv, factor=factor, total=total,
             q=proj[:, :Hq * qd].view(total, Hq, qd)[..., :d],
             k=proj[:, Hq * qd:Hq * qd + Hkv * d].view(total, Hkv, d), v=proj[:, Hq * qd + Hkv * d:].view(total, Hkv, d),
             qw=(torch.randn(d, generator=gpu, device=DEV) * 0.1).to(BF16), kw=(torch.randn(d, generator=gpu, device=DEV) * 0.1).to(BF16),
             k_scale=1.0 if c["kv"] == "bf16" else 0.03125, v_scale=1.0 if c["kv"] == "bf16" else 0.02,
             kp=torch.zeros(pages, ps, Hkv, d, device=DEV).to(kv), vp=torch.zeros(pages, ps, Hkv, d, device=DEV).to(kv),
             table=table.to(I32).to(DEV), lens=seq_lens.to(I32).to(DEV), slots=slots.to(I32).to(DEV), cu=cu.to(I32).to(DEV),
             q_out=torch.empty(total, Hq, d, dtype=BF16, device=DEV), err=torch.zeros(1, dtype=I32, device=DEV))
    if own:
        import gated_delta_rule_102_b200 as gdn
        cfg = gdn.GdnAttnConfig.make(Hq, Hkv, d, ps, rotary_dim=c["R"], rope_interleaved=c["interleaved"], kv_dtype=kv, norm_eps=EPS,
                                     norm_offset=1.0, rope_scale=factor, k_scale=s["k_scale"], v_scale=s["v_scale"])
        s["plan"] = gdn.CallPlan(gdn.gdn_qk_rope_append, cfg, s["q"], s["k"], s["v"], s["qw"], s["kw"], inv, s["kp"], s["vp"], s["table"], s["lens"],
                                 s["slots"], s["q_out"], cu_seqlens=s["cu"], T_max=c["T"], err_flag=s["err"])
    return s


def _prepare_attn(c, seed):
    gpu, cpu = _gen(seed)
    B, Hq, Hkv, d, ps = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    n = _counts(c, cpu)
    total = int(n.sum())
    u = torch.rand(B, generator=cpu, dtype=F64)
    lens = (c["min_len"] * (c["max_len"] / c["min_len"]) ** u).round().long()  # tokens already held
    lens[int(torch.randint(0, B, (1,), generator=cpu))] = c["max_len"]
    slots, seq_lens, cu = _batch(c, cpu, n, lens)
    held = (lens + n + ps - 1) // ps
    pages, width = int(held.sum()) + 3, int(held.max())
    ids = torch.randperm(pages, generator=cpu)
    j = torch.arange(width)
    at = (held.cumsum(0) - held)[:, None] + j
    table = torch.full((2 * B, width), -1, dtype=torch.int64)
    table[slots] = torch.where(j < held[:, None], ids[at.clamp(max=pages - 1)], -1)
    k_scale, v_scale = (1.0, 1.0) if c["kv"] == "bf16" else (0.03125, 0.02)

    def pool(std, scale):
        x = torch.randn(pages, ps, Hkv, d, generator=gpu, device=DEV, dtype=BF16)
        if c["kv"] == "bf16":
            return x.mul_(std)
        return torch.cat([_quant(p * std, scale) for p in x.split(max(1, 2 ** 26 // (ps * Hkv * d)))])
    kp, vp = pool(1.5, k_scale), pool(1.0, v_scale)  # keys after their norm and its weight
    q = (torch.randn(total, Hq, d, generator=gpu, device=DEV) * 1.5).to(BF16)
    gate = torch.randn(total, Hq, 2 * d, generator=gpu, device=DEV).to(BF16)[..., d:] if c["gated"] else None
    s = dict(c=c, total=total, q=q, gate=gate, kp=kp, vp=vp, k_scale=k_scale, v_scale=v_scale, table=table.to(I32).to(DEV),
             lens=seq_lens.to(I32).to(DEV), slots=slots.to(I32).to(DEV), cu=cu.to(I32).to(DEV),
             out=torch.empty(total, Hq, d, dtype=BF16, device=DEV), lse=torch.empty(total, Hq, device=DEV),
             err=torch.zeros(1, dtype=I32, device=DEV))
    if own:
        import gated_delta_rule_102_b200 as gdn
        cfg = gdn.GdnAttnConfig.make(Hq, Hkv, d, ps, kv_dtype=kp.dtype, window=c["window"], softcap=c["softcap"], k_scale=k_scale, v_scale=v_scale)
        s["ws"] = gdn.attn_decode_workspace(cfg, B, c["T"], DEV)
        s["plan"] = gdn.CallPlan(gdn.gdn_attn_decode, cfg, q, kp, vp, s["table"], s["lens"], s["slots"], s["out"], s["ws"], gate=gate, lse=s["lse"],
                                 cu_seqlens=s["cu"], T_max=c["T"], err_flag=s["err"])
    return s


def _prepare_branch(c, seed):
    gpu, cpu = _gen(seed)
    n, ps = c["n"], c["page"]
    parents = -(-n // c["fan"])
    rows = parents + n + 3
    lens = torch.randint(1, c["max_len"] + 1, (parents,), generator=cpu)
    held = (lens + ps - 1) // ps
    width = -(-(c["max_len"] + c["T"]) // ps) + 1
    grow = n * (2 + -(-c["T"] // ps))
    pages = parents * -(-c["max_len"] // ps) + grow + 5
    ids = torch.randperm(pages, generator=cpu)
    slot = torch.randperm(rows, generator=cpu)
    src = slot[:parents].repeat_interleave(c["fan"])[:n]
    dst = slot[parents:parents + n]
    table = torch.full((rows, width), -1, dtype=torch.int64)
    j = torch.arange(width)
    at = (held.cumsum(0) - held)[:, None] + j
    table[slot[:parents]] = torch.where(j < held[:, None], ids[at.clamp(max=pages - 1)], -1)
    refs = torch.zeros(pages, dtype=torch.int64)
    refs[ids[:int(held.sum())]] = 1
    seq_lens = torch.zeros(rows, dtype=torch.int64)
    seq_lens[slot[:parents]] = lens
    caches = [torch.randn(pages, ps, c["Hkv"], c["d"], generator=gpu, device=DEV, dtype=BF16) for _ in range(2 * c["layers"])]
    pools = [torch.randn(rows, c["Hv"], c["dk"], c["dk"], generator=gpu, device=DEV),
             torch.randn(rows, 3, 2 * c["Hv"] * c["dk"], generator=gpu, device=DEV, dtype=BF16)]
    s = dict(c=c, table=table.to(I32).to(DEV), refs=refs.to(I32).to(DEV), lens=seq_lens.to(I32).to(DEV), src=src.to(I32).to(DEV), dst=dst.to(I32).to(DEV),
             caches=caches, pools=pools, csrc=torch.full((n,), -1, dtype=I32, device=DEV), cdst=torch.full((n,), -1, dtype=I32, device=DEV),
             err=torch.zeros(1, dtype=I32, device=DEV))
    if own:
        import gated_delta_rule_102_b200 as gdn
        e = s["err"]
        s["plans"] = [gdn.CallPlan(gdn.gdn_pages_free, s["dst"], s["table"], s["lens"], s["refs"], err_flag=e),
                      gdn.CallPlan(gdn.gdn_pages_fork, ps, s["src"], s["dst"], s["table"], s["lens"], s["refs"], s["csrc"], s["cdst"], err_flag=e),
                      gdn.CallPlan(gdn.gdn_pages_reserve, ps, s["dst"], c["T"], s["table"], s["lens"], s["refs"], err_flag=e),
                      gdn.CallPlan(gdn.gdn_copy_rows, caches, s["csrc"], s["cdst"], err_flag=e),
                      gdn.CallPlan(gdn.gdn_copy_rows, pools, s["src"], s["dst"], err_flag=e)]
    return s


def _prepare_compact(c, seed):
    gpu, cpu = _gen(seed)
    P, ps, S = c["pages"], c["page"], c["slots"]
    live = torch.rand(P, generator=cpu) < c["live"]
    live[int(torch.randint(0, P, (1,), generator=cpu))] = True
    ids = live.nonzero().flatten()[torch.randperm(int(live.sum()), generator=cpu)]
    width = -(-ids.numel() // S) + 2
    table = torch.full((S, width), -1, dtype=torch.int64)
    at = torch.arange(ids.numel())
    table[at % S, at // S] = ids
    refs = live.long()
    if S > 1:  # the first page of slot 0 is a prefix that the last slot holds too
        table[S - 1, width - 1] = table[0, 0]
        refs[table[0, 0]] += 1
    caches = [torch.randn(P, ps, c["Hkv"], c["d"], generator=gpu, device=DEV, dtype=BF16) for _ in range(2 * c["layers"])]
    both = torch.cat([table.flatten(), refs]).to(I32).to(DEV)  # one buffer: table | refs
    work = both.clone()
    s = dict(c=c, before=both, now=work, table=work[:S * width].view(S, width), refs=work[S * width:], caches=caches,
             csrc=torch.full((P,), -1, dtype=I32, device=DEV), cdst=torch.full((P,), -1, dtype=I32, device=DEV),
             count=torch.zeros(1, dtype=I32, device=DEV), remap=torch.empty(P, dtype=I32, device=DEV), err=torch.zeros(1, dtype=I32, device=DEV))
    if own:
        import gated_delta_rule_102_b200 as gdn
        s["plans"] = [gdn.CallPlan(gdn.gdn_pages_compact, s["table"], s["refs"], s["csrc"], s["cdst"], s["count"], s["remap"], err_flag=s["err"]),
                      gdn.CallPlan(gdn.gdn_copy_rows, caches, s["csrc"], s["cdst"], n_dev=s["count"], err_flag=s["err"])]
    return s


def prepare(case, seed):
    return {"append": _prepare_append, "attn": _prepare_attn, "branch": _prepare_branch, "compact": _prepare_compact}[case["op"]](case, seed)


# --------------------------------------------------------------------------------------------- the plain forms
def _tokens(s):
    """Sequence, place in its call and cache position of every packed token row."""
    row = torch.arange(s["total"], device=DEV)
    b = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    t = row - s["cu"][b].long()
    return b, t, s["lens"][s["slots"][b].long()].long() + t


def _rotate(x, cos, sin, R, interleaved):
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([r, x[..., R:]], -1)


def _run_append(s):
    c = s["c"]
    b, t, pos = _tokens(s)
    angle = pos.to(F64)[:, None] * s["inv"].to(F64)
    cos, sin = ((f(angle) * s["factor"]).to(F32)[:, None, :] for f in (torch.cos, torch.sin))

    def norm(x, w):
        x = x.float()
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (1.0 + w.float())
    q = _rotate(norm(s["q"], s["qw"]), cos, sin, c["R"], c["interleaved"])
    k = _rotate(norm(s["k"], s["kw"]), cos, sin, c["R"], c["interleaved"])
    page = s["table"][s["slots"][b].long(), pos // c["page"]].long()
    off = pos % c["page"]
    if c["kv"] == "bf16":
        s["kp"][page, off] = k.to(BF16)
        s["vp"][page, off] = s["v"]
    else:
        s["kp"].view(torch.uint8)[page, off] = _quant(k, s["k_scale"]).view(torch.uint8)
        s["vp"].view(torch.uint8)[page, off] = _quant(s["v"], s["v_scale"]).view(torch.uint8)
    s["q_out"].copy_(q)
    return {"q": s["q_out"], "k_pages": s["kp"], "v_pages": s["vp"]}


def _run_attn(s):
    c = s["c"]
    B, T, Hq, Hkv, d, ps = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    slots = s["slots"].long()
    table = s["table"][slots].long().clamp(min=0)                       # [B][pages]
    L = table.shape[1] * ps
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    past = s["lens"][slots].long()
    k = s["kp"].view(torch.uint8 if c["kv"] != "bf16" else BF16)[table].view(s["kp"].dtype).reshape(B, L, Hkv, d).float()
    k = k.permute(0, 2, 3, 1)                                           # [B][Hkv][d][L]
    row = (s["cu"][:-1].long()[:, None] + torch.arange(T, device=DEV)).clamp(max=s["total"] - 1)
    q = s["q"][row].float().view(B, T, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, d)
    x = torch.matmul(q, k) * (s["k_scale"] / math.sqrt(d))              # [B][Hkv][T*G][L]
    del k
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    at = torch.arange(L, device=DEV)
    pos = past[:, None] + torch.arange(T, device=DEV)                   # [B][T]
    seen = at <= pos[..., None]
    if c["window"]:
        seen &= at > pos[..., None] - c["window"]
    seen = seen[:, None, :, None, :].expand(B, 1, T, G, L).reshape(B, 1, T * G, L)
    x = x.masked_fill(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    del x
    total = p.sum(-1, keepdim=True)
    v = s["vp"].view(torch.uint8 if c["kv"] != "bf16" else BF16)[table].view(s["vp"].dtype).reshape(B, L, Hkv, d).float()
    v = v.masked_fill((at[None] >= (past + n)[:, None])[..., None, None], 0.0).permute(0, 2, 1, 3)
    o = torch.matmul(p, v) / total * s["v_scale"]                       # [B][Hkv][T*G][d]
    o = o.view(B, Hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d)
    lse = (top + torch.log(total)).view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)
    b, t, _ = _tokens(s)
    o, lse = o[b, t], lse[b, t]
    if s["gate"] is not None:
        o = o / (1.0 + torch.exp(-s["gate"].float()))
    s["out"].copy_(o)
    s["lse"].copy_(lse)
    return {"out": s["out"], "lse": s["lse"]}


def _free_ids(refs):
    """Page numbers, the free ones first, lowest first."""
    return torch.argsort(refs != 0, stable=True)


def _run_branch(s):
    c, table, refs, lens = s["c"], s["table"], s["refs"], s["lens"]
    ps, src, dst = c["page"], s["src"].long(), s["dst"].long()
    one = torch.ones((), dtype=I32, device=DEV)
    # last step's children go
    rows = table[dst]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), -(rows >= 0).to(I32).flatten())
    table[dst] = -one
    lens[dst] = 0 * one
    # fork: whole pages are shared, a partly filled one is copied
    length = lens[src].long()
    full, part = length // ps, length % ps > 0
    new = _free_ids(refs)[(part.long().cumsum(0) - 1).clamp(min=0)]
    j = torch.arange(table.shape[1], device=DEV)
    rows = torch.where(j < full[:, None], table[src].long(), torch.where((j == full[:, None]) & part[:, None], new[:, None], -1))
    table[dst] = rows.to(I32)
    refs.index_add_(0, rows.clamp(min=0).flatten(), (rows >= 0).to(I32).flatten())
    lens[dst] = length.to(I32)
    old = table[src, full.clamp(max=table.shape[1] - 1)].long()
    s["csrc"].copy_(torch.where(part, old, -1))
    s["cdst"].copy_(torch.where(part, new, -1))
    # the children's next T tokens get their pages
    have, want = (length + ps - 1) // ps, (length + c["T"] + ps - 1) // ps
    missing = (j >= have[:, None]) & (j < want[:, None])
    rank = (missing.flatten().long().cumsum(0) - 1).clamp(min=0).view(missing.shape)
    got = _free_ids(refs)[rank]
    table[dst] = torch.where(missing, got, table[dst].long()).to(I32)
    refs.index_add_(0, torch.where(missing, got, 0).flatten(), missing.to(I32).flatten())
    # the data: a child without a partly filled page copies a page of its parent onto itself
    keep = table[src, (full - 1).clamp(min=0)].long()
    a, z = torch.where(part, old, keep), torch.where(part, new, keep)
    for x in s["caches"]:
        x[z] = x[a]
    for x in s["pools"]:
        x[dst] = x[src]
    return _branch_out(s)


def _branch_out(s):
    return {"table": s["table"], "refs": s["refs"], "lens": s["lens"], "copy_src": s["csrc"], "copy_dst": s["cdst"], "caches": s["caches"], "pools": s["pools"]}


def _run_compact(s):
    s["now"].copy_(s["before"])  # the pool as the sequences left it, for every pass
    table, refs = s["table"], s["refs"]
    P = refs.shape[0]
    at = torch.arange(P, device=DEV)
    live = refs > 0
    k = live.sum()
    moves, hole = live & (at >= k), ~live & (at < k)
    holes, movers = torch.argsort(~hole, stable=True), torch.argsort(~moves, stable=True)
    remap = torch.where(moves, holes[(moves.long().cumsum(0) - 1).clamp(min=0)], torch.where(live, at, -1))
    count = moves.sum()
    s["count"].copy_(count)
    s["csrc"].copy_(torch.where(at < count, movers, -1))
    s["cdst"].copy_(torch.where(at < count, holes, -1))
    s["remap"].copy_(remap)
    moved = torch.zeros_like(refs).index_add_(0, remap.clamp(min=0), torch.where(live, refs, torch.zeros_like(refs)))
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()], -1))
    refs.copy_(moved)
    src = torch.empty_like(holes).scatter(0, holes, torch.where(at < count, movers, holes))
    for x in s["caches"]:
        x.copy_(x[src])
    return _compact_out(s)


def _compact_out(s):
    return {"table": s["table"], "refs": s["refs"], "remap": s["remap"], "count": s["count"], "copy_src": s["csrc"], "copy_dst": s["cdst"], "caches": s["caches"]}


def _run_own(s):
    op = s["c"]["op"]
    if op in ("append", "attn"):
        s["plan"].launch()
        return {"q": s["q_out"], "k_pages": s["kp"], "v_pages": s["vp"]} if op == "append" else {"out": s["out"], "lse": s["lse"]}
    if op == "compact":
        s["now"].copy_(s["before"])
    for p in s["plans"]:
        p.launch()
    return _branch_out(s) if op == "branch" else _compact_out(s)


def run(state):
    if own:
        return _run_own(state)
    return {"append": _run_append, "attn": _run_attn, "branch": _run_branch, "compact": _run_compact}[state["c"]["op"]](state)


# -------------------------------------------------------------------------------------- the work, and the values
def _expected_tokens(c):
    return sum(c["T"] - i % (c["T"] + 1) for i in range(c["B"])) if c["ragged"] else c["B"] * c["T"]


def work(case):
    c = case
    if c["op"] == "append":
        n, e = _expected_tokens(c), 2 if c["kv"] == "bf16" else 1
        vec = (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        return {"bytes": n * (2 * vec + 2 * c["Hq"] * c["d"] + 2 * e * c["Hkv"] * c["d"]), "flops": n * (c["Hq"] + c["Hkv"]) * (4 * c["d"] + 3 * c["R"])}
    if c["op"] == "attn":
        n, e = _expected_tokens(c), 2 if c["kv"] == "bf16" else 1
        a, b = c["min_len"], c["max_len"]
        mean = b if c["B"] == 1 or a == b else (b - a) / math.log(b / a)  # of lengths spread evenly in their logarithm
        if c["window"]:
            w = min(c["window"] + c["T"], b)
            mean = mean if w >= b else w if w <= a else ((w - a) + w * math.log(b / w)) / math.log(b / a)
        rows = n * c["Hq"] * c["d"]
        return {"bytes": c["B"] * (mean + n / c["B"]) * c["Hkv"] * c["d"] * 2 * e + rows * (6 if c["gated"] else 4) + n * c["Hq"] * 4,
                "flops": 4 * rows * mean}
    page = c["page"] * c["Hkv"] * c["d"] * 2 * 2 * c["layers"]
    if c["op"] == "branch":
        copied = c["n"] * (1 - 1 / c["page"])
        slot = c["Hv"] * c["dk"] * c["dk"] * 4 + 3 * 2 * c["Hv"] * c["dk"] * 2
        table = 3 * 4 * c["n"] * (c["max_len"] / 2 / c["page"] + 1)
        return {"bytes": 2 * copied * page + 2 * c["n"] * slot + table, "flops": 0}
    moved = c["pages"] * c["live"] * (1 - c["live"])
    return {"bytes": 2 * moved * page + 4 * c["pages"] * (5 + 2 * c["live"]), "flops": 0}


def _exact_append(s):
    c = s["c"]
    d, R, ps = c["d"], c["R"], c["page"]
    cu, lens, slots, table = (s[k].tolist() for k in ("cu", "lens", "slots", "table"))
    first = list(range(0, R, 2)) if c["interleaved"] else list(range(R // 2))
    second = [i + 1 for i in first] if c["interleaved"] else [i + R // 2 for i in first]
    f = s["inv"].double()
    kp, vp = torch.zeros(s["kp"].shape, dtype=F64, device=DEV), torch.zeros(s["vp"].shape, dtype=F64, device=DEV)
    qs = torch.empty(s["q_out"].shape, dtype=F64, device=DEV)

    def head(x, w, turn):
        x = x.double()
        y = x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt() * (1 + w.double())
        z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.full_like(turn, s["factor"]), turn)
        y[..., first], y[..., second] = z.real, z.imag
        return y
    for b, slot in enumerate(slots):
        r = slice(cu[b], cu[b + 1])
        if r.stop == r.start:
            continue
        where = [lens[slot] + t for t in range(r.stop - r.start)]
        turn = (torch.tensor(where, dtype=F64, device=DEV)[:, None, None] * f).expand(-1, 1, -1)
        qs[r] = head(s["q"][r], s["qw"], turn)
        pages, offs = [table[slot][p // ps] for p in where], [p % ps for p in where]
        kp[pages, offs] = head(s["k"][r], s["kw"], turn) / s["k_scale"]
        vp[pages, offs] = s["v"][r].double() / s["v_scale"]
    return {"q": qs, "k_pages": kp, "v_pages": vp}


def _exact_attn(s):
    c = s["c"]
    Hq, Hkv, d, ps = c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    cu, lens, slots = (s[k].tolist() for k in ("cu", "lens", "slots"))
    out, lse = torch.empty(s["out"].shape, dtype=F64, device=DEV), torch.empty(s["lse"].shape, dtype=F64, device=DEV)
    for b, slot in enumerate(slots):
        n, past = cu[b + 1] - cu[b], lens[slot]
        ids = s["table"][slot, :-(-(past + n) // ps)].long()
        raw = torch.uint8 if c["kv"] != "bf16" else BF16
        keys, values = (x.view(raw).index_select(0, ids).view(x.dtype).flatten(0, 1)[:past + n] for x in (s["kp"], s["vp"]))
        for t in range(n):
            lo, hi = max(0, past + t + 1 - c["window"]) if c["window"] else 0, past + t + 1
            q = s["q"][cu[b] + t].double().view(Hkv, G, d)
            sc = torch.einsum("hgd,lhd->hgl", q, keys[lo:hi].double()) * s["k_scale"] * d ** -0.5
            if c["softcap"]:
                sc = c["softcap"] * torch.tanh(sc / c["softcap"])
            o = torch.einsum("hgl,lhd->hgd", torch.softmax(sc, -1), values[lo:hi].double()).reshape(Hq, d) * s["v_scale"]
            out[cu[b] + t] = o * torch.sigmoid(s["gate"][cu[b] + t].double()) if s["gate"] is not None else o
            lse[cu[b] + t] = torch.logsumexp(sc, -1).reshape(Hq)
    return {"out": out, "lse": lse}


def _exact_branch(s):
    """The copied data (the tables are whole numbers): a child's pages and slot hold what its parent's do."""
    c, ps = s["c"], s["c"]["page"]
    table, refs, lens = s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist()
    free = (i for i, r in enumerate(refs) if r == 0)
    caches, pools = [x.double() for x in s["caches"]], [x.double() for x in s["pools"]]
    for a, z in zip(s["src"].tolist(), s["dst"].tolist()):
        if lens[a] % ps:
            page = next(free)
            for x in caches:
                x[page] = x[table[a][lens[a] // ps]]
        for x in pools:
            x[z] = x[a]
    return {"table": None, "refs": None, "lens": None, "copy_src": None, "copy_dst": None, "caches": caches, "pools": pools}


def _exact_compact(s):
    refs = s["before"][s["table"].numel():].tolist()
    k = sum(r > 0 for r in refs)
    caches = [x.double() for x in s["caches"]]
    holes = [i for i in range(k) if refs[i] == 0]
    for page, hole in zip((i for i in range(k, len(refs)) if refs[i] > 0), holes):
        for x in caches:
            x[hole] = x[page]
    return {"table": None, "refs": None, "remap": None, "count": None, "copy_src": None, "copy_dst": None, "caches": caches}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "branch": _exact_branch, "compact": _exact_compact}[case["op"]](s)
