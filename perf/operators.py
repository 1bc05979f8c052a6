"""The serving-side operators of the library, what they are measured on, and their plain forms:

* rotary positions on Q and K, forward and backward;
* K and V written into a paged cache (16-bit, or E4M3 with a scale for each token and head), K rotated on the way;
* a paged cache read back into dense K and V;
* attention of single tokens, or of a tree of drafted tokens, over a paged cache.

``own`` chooses between the plain forms (elementary torch operations in fp32, angles in fp64) and the library's calls.
Cache tensors are logical [pages, h_kv, page_size, d] views; the cache is stored token-major in each page.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -60          # rows with a smaller largest value are scaled as if it were this one
SCRATCH_BYTES = 128 << 20      # what a serving program keeps as workspace for the attention calls

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # Q and K of one new token for a few sequences: latency only.
        dict(name="rope_decode_b4", op="rope", b=4, s=1, h_q=32, h_kv=8, d=128, rot=128, dtype="bf16",
             interleaved=False, scaling="none", backward=False, far=8192),
        # The training shape, self-attention with as many K as Q heads.
        dict(name="rope_train_s8192", op="rope", b=2, s=8192, h_q=16, h_kv=16, d=128, rot=128, dtype="bf16",
             interleaved=False, scaling="none", backward=False, far=0),
        # Gradients of grouped heads, half of each head rotated in adjacent pairs, stretched for long contexts,
        # an odd length.
        dict(name="rope_bwd_gqa_partial", op="rope", b=1, s=4999, h_q=64, h_kv=8, d=128, rot=64, dtype="f16",
             interleaved=True, scaling="yarn", backward=True, far=100000),
        # One new token for each of 32 sequences goes into an E4M3 cache: latency.
        dict(name="write_decode_b32_e4m3", op="write", b=32, s=1, h_kv=8, d=128, page=64, lo=1000, hi=16000,
             dtype="bf16", cache="e4m3", rot=128, interleaved=False, scaling="none"),
        # Prompts of up to 8K tokens, ragged, quantised as they are written.
        dict(name="write_prompt_b4_e4m3", op="write", b=4, s=8192, h_kv=8, d=128, page=64, lo=5001, hi=8192,
             dtype="bf16", cache="e4m3", rot=128, interleaved=False, scaling="linear"),
        # The context of a chunk of prompt, read back for the dense attention call.
        dict(name="read_ctx_b2_e4m3", op="read", b=2, s=8192, h_kv=8, d=128, page=64, lo=6000, hi=8192,
             dtype="bf16", cache="e4m3"),
        # A 16-bit cache with small heads and small pages, ragged.
        dict(name="read_ragged_f16_d64", op="read", b=16, s=2048, h_kv=12, d=64, page=16, lo=1, hi=2048,
             dtype="f16", cache="f16"),
        # One token against a short 16-bit context: latency.
        dict(name="attend_1tok_b1_bf16", op="attend", b=1, s=1, h_q=32, h_kv=8, d=128, page=64, lo=1000, hi=1000,
             dtype="bf16", cache="bf16", mask="none"),
        # The ordinary serving step: 32 sequences of 1K..16K tokens, E4M3 cache, grouped heads.
        dict(name="attend_1tok_b32_e4m3", op="attend", b=32, s=1, h_q=64, h_kv=8, d=128, page=64, lo=1000, hi=16384,
             dtype="bf16", cache="e4m3", mask="none"),
        # One sequence with a long context.
        dict(name="attend_1tok_128k_bf16", op="attend", b=1, s=1, h_q=64, h_kv=8, d=128, page=128, lo=131000, hi=131000,
             dtype="bf16", cache="bf16", mask="none"),
        # 64 drafted tokens in a tree for 8 sequences.
        dict(name="attend_tree64_b8_e4m3", op="attend", b=8, s=64, h_q=64, h_kv=8, d=128, page=64, lo=4000, hi=8192,
             dtype="bf16", cache="e4m3", mask="tree"),
        # A small tree, heads that are not grouped, odd lengths.
        dict(name="attend_tree13_b4_f16_d64", op="attend", b=4, s=13, h_q=12, h_kv=12, d=64, page=16, lo=333, hi=1021,
             dtype="f16", cache="f16", mask="tree"),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend"])
    d = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["f16", "bf16"])
    if op == "rope":
        s, h_kv = _log_int(rng, 1, 8192), rng.choice([1, 2, 8, 12, 16])
        h_q = h_kv * rng.choice([1, 4, 8])
        b = max(1, min(_log_int(rng, 1, 16), (2 * 8192 * 32 * 128) // (s * (h_q + h_kv) * d)))
        return dict(op=op, b=b, s=s, h_q=h_q, h_kv=h_kv, d=d, rot=rng.choice([d, d, d // 2, d // 4, d - 6]), dtype=dtype,
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    backward=rng.random() < 0.5, far=rng.choice([0, 5000, 500000]))
    page = rng.choice([16, 32, 64, 128, 48])
    cache = rng.choice(["e4m3", "e4m3", dtype])
    h_kv = rng.choice([1, 4, 8, 12])
    if op == "write":
        s = _log_int(rng, 1, 8192)
        b = max(1, min(_log_int(rng, 1, 64), (4 * 8192 * 8 * 128) // (s * h_kv * d)))
        hi = s + _log_int(rng, 1, 4096)
        return dict(op=op, b=b, s=s, h_kv=h_kv, d=d, page=page, lo=max(1, hi // rng.choice([1, 2, 4])), hi=hi, dtype=dtype,
                    cache=cache, rot=rng.choice([0, d, d // 2, d - 6]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
    if op == "read":
        s = _log_int(rng, 1, 8192)
        b = max(1, min(_log_int(rng, 1, 64), (4 * 8192 * 8 * 128) // (s * h_kv * d)))
        return dict(op=op, b=b, s=s, h_kv=h_kv, d=d, page=page, lo=1, hi=s, dtype=dtype, cache=cache)
    s = rng.choice([1, 1, 1, _log_int(rng, 2, 64)])
    h_q = h_kv * rng.choice([1, 4, 8])
    hi = s + _log_int(rng, 1, 32768)
    room = (32 * 9000 * 8 * 128 if s == 1 else 8 * 6000 * 8 * 128 * 512 // (s * max(8, h_q // h_kv)))
    b = max(1, min(_log_int(rng, 1, 48), room // (hi * h_kv * d)))
    return dict(op=op, b=b, s=s, h_q=h_q, h_kv=h_kv, d=d, page=page, lo=max(s, hi // rng.choice([1, 2, 8])), hi=hi, dtype=dtype,
                cache=cache, mask="none" if s == 1 else rng.choice(["tree", "tree", "bottom_right"]))


def _lens(case):
    """Tokens of each sequence after the call: spread over [lo, hi], the last one hi."""
    b, lo, hi = case["b"], case["lo"], case["hi"]
    return [hi if i == b - 1 else lo + int((hi - lo) * ((i * 0.6180339887 + 0.31) % 1.0)) for i in range(b)]


def _news(case):
    """New tokens of each sequence: all ``s`` rows, or as many as the sequence has."""
    return [min(case["s"], n) for n in _lens(case)]


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        n = case["b"] * case["s"] * (case["h_q"] + case["h_kv"]) * d
        return {"bytes": 4 * n, "flops": 3 * n}
    cb, scale = (1, 4) if case["cache"] == "e4m3" else (2, 0)
    if case["op"] == "write":
        rows = 2 * sum(_news(case)) * case["h_kv"]
        return {"bytes": rows * (d * (2 + cb) + scale), "flops": rows * d * 4}
    if case["op"] == "read":
        rows = 2 * sum(_lens(case)) * case["h_kv"]
        return {"bytes": rows * (d * cb + scale) + 2 * case["b"] * case["s"] * case["h_kv"] * d * 2, "flops": rows * d}
    keys, rows = sum(_lens(case)), case["b"] * case["s"] * case["h_q"]
    pairs = sum(n * m for n, m in zip(_lens(case), _news(case))) * case["h_q"]
    return {"bytes": 2 * keys * case["h_kv"] * (d * cb + scale) + rows * (4 * d + 4), "flops": 4 * pairs * d}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _inv_freq(rot, scaling, base=10000.0, factor=8.0, context=8192):
    """Radians per position of each pair, and the factor on the rotated values: the plain geometric frequencies, all
    divided by the factor (linear), a larger base (ntk), or high frequencies kept and low ones divided (yarn)."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / max(1.0, rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        turns = context * f / (2 * math.pi)             # turns over the original context
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _table(inv_freq):
    """Turns per position as 64-bit binary fractions (what the library's rotary table holds)."""
    turns = [int(round(math.ldexp(f / (2 * math.pi), 64))) for f in inv_freq.tolist()]
    return torch.tensor([t - (1 << 64) if t >= (1 << 63) else t for t in turns], dtype=torch.int64, device="cuda")


def _quantise(x):
    """E4M3 codes and the fp32 scale of each row."""
    scale = x.float().abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
    return (x.float() * (1.0 / scale).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _randn(g, dtype, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _bshd(g, dtype, b, h, s, d):
    """A logical [b, h, s, d] view of token-major storage, as projections give it."""
    return _randn(g, dtype, b, s, h, d).permute(0, 2, 1, 3)


def _cache(g, case, lens):
    """A filled paged cache: pages in shuffled order, each sequence's last page partly used, a few spare pages."""
    b, h, d, ps = case["b"], case["h_kv"], case["d"], case["page"]
    need = [-(-n // ps) for n in lens]
    wide, pages = max(need) + 1, sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((b, wide), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    st = dict(page_table=table, seq_lens_kv=torch.tensor(lens, dtype=torch.int32, device="cuda"), k_scale=None, v_scale=None)
    for n in ("k", "v"):
        x = _randn(g, _DT[case["dtype"]], pages, ps, h, d)
        if n == "k":   # a few channels of each head are larger than the rest, as projections of activations have them
            x[..., : d // 16] *= 4
        if case["cache"] == "e4m3":
            x, scale = _quantise(x)
            st[n + "_scale"] = scale.permute(0, 2, 1).contiguous()
        st[n + "_cache"] = x.permute(0, 2, 1, 3)
    return st


def _tree(rng, n):
    """Visibility of n drafted tokens in a random tree (itself and its ancestors), and each one's depth."""
    see, depth = np.zeros((n, n), dtype=bool), np.zeros(n, dtype=np.int64)
    for j in range(n):
        parent = int(rng.integers(max(-1, j - 8), j)) if j else -1
        if parent >= 0:
            see[j], depth[j] = see[parent], depth[parent] + 1
        see[j, j] = True
    return see, depth


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, b, s, d = _DT[case["dtype"]], case["b"], case["s"], case["d"]
    st = dict(op=case["op"], case=case)
    if case.get("rot"):
        f, st["factor"] = _inv_freq(case["rot"], case["scaling"])
        st["inv_freq"] = torch.from_numpy(f).cuda()
        st["table"] = _table(f)
        st["interleaved"] = case["interleaved"]
    if case["op"] == "rope":
        st["backward"] = case["backward"]
        st["q"], st["k"] = _bshd(g, dt, b, case["h_q"], s, d), _bshd(g, dt, b, case["h_kv"], s, d)
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        start = torch.randint(0, case["far"] + 1, (b, 1), generator=g, device="cuda")
        st["positions"] = (start + torch.arange(s, device="cuda")).to(torch.int32)
        return st
    lens = _lens(case)
    st.update(_cache(g, case, lens))
    if case["op"] == "read":
        st["k"], st["v"] = (torch.empty(b, case["h_kv"], s, d, device="cuda", dtype=dt) for _ in range(2))
        return st
    st["seq_lens_q"] = torch.tensor(_news(case), dtype=torch.int32, device="cuda")
    if case["op"] == "write":
        st["k"], st["v"] = (_bshd(g, dt, b, case["h_kv"], s, d) for _ in range(2))
        return st
    st["q"] = _bshd(g, dt, b, case["h_q"], s, d)
    st["o"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(b, case["h_q"], s, device="cuda", dtype=torch.float32)
    st["workspace"] = torch.empty(SCRATCH_BYTES, device="cuda", dtype=torch.uint8)
    st["tree_mask"] = None
    if case["mask"] == "tree":
        rng = np.random.default_rng(seed)
        words = np.zeros((b, s, -(-s // 32)), dtype=np.uint32)
        for i in range(b):
            see, _ = _tree(rng, s)
            for j in range(s):
                words[i, :, j // 32] |= see[:, j].astype(np.uint32) << np.uint32(j % 32)
        st["tree_mask"] = torch.from_numpy(words.view(np.int32)).cuda()
    return st


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def run(st):
    return _library(st) if own else {"rope": _rope, "write": _write, "read": _read, "attend": _attend}[st["op"]](st)


def _library(st):
    import attention_flashattention_sdpa_gb300 as sdpa
    if st["op"] == "rope":
        call = sdpa.sdpa_rope_bwd if st["backward"] else sdpa.sdpa_rope_fwd
        call(st["q"], st["k"], st["q_out"], st["k_out"], st["table"], st["positions"], interleaved=st["interleaved"],
             attn_factor=st["factor"])
        return st["q_out"], st["k_out"]
    where = (st["k_cache"], st["v_cache"], st["page_table"], st["seq_lens_kv"])
    scales = dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
    if st["op"] == "write":
        rope = {}
        if "table" in st:
            rope = dict(rope_table=st["table"], interleaved=st["interleaved"], attn_factor=st["factor"])
        sdpa.sdpa_cache_write(st["k"], st["v"], *where, seq_lens_q=st["seq_lens_q"], **scales, **rope)
        return _cache_outputs(st)
    if st["op"] == "read":
        sdpa.sdpa_cache_read(*where, st["k"], st["v"], **scales)
        return st["k"], st["v"]
    sdpa.sdpa_decode(st["q"], *where, st["o"], st["lse"], workspace=st["workspace"], seq_lens_q=st["seq_lens_q"],
                     causal="bottom_right" if st["case"]["mask"] == "bottom_right" else False,
                     tree_mask=st["tree_mask"], **scales)
    return st["o"], st["lse"]


def _cache_outputs(st):
    out = [st["k_cache"], st["v_cache"]]
    return out + [st["k_scale"], st["v_scale"]] if st["k_scale"] is not None else out


def _rotate(x, positions, inv_freq, interleaved, factor):
    """x [b, h, s, d] (fp32) rotated by the angles of positions [b, s]; the elements behind the rotated ones as they are."""
    angle = positions.double().unsqueeze(-1) * inv_freq                     # [b, s, rot/2]
    cos, sin = (factor * torch.cos(angle)).float().unsqueeze(1), (factor * torch.sin(angle)).float().unsqueeze(1)
    rot = 2 * inv_freq.numel()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2: rot])
    y, z = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _rope(st):
    sign = -1.0 if st["backward"] else 1.0
    for n in ("q", "k"):
        st[n + "_out"].copy_(_rotate(st[n].float(), st["positions"], sign * st["inv_freq"], st["interleaved"], st["factor"]))
    return st["q_out"], st["k_out"]


def _raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _write(st):
    k, v = st["k"].float(), st["v"].float()
    ps, lens, news = st["k_cache"].shape[2], st["seq_lens_kv"].long(), st["seq_lens_q"].long()
    row = torch.arange(k.shape[2], device="cuda")
    pos = (lens - news).unsqueeze(1) + row                                   # [b, s]
    if "inv_freq" in st:
        k = _rotate(k, pos, st["inv_freq"], st["interleaved"], st["factor"])
    live = row < news.unsqueeze(1)
    bi, si = live.nonzero(as_tuple=True)
    page, slot = st["page_table"].long()[bi, pos[bi, si] // ps], pos[bi, si] % ps
    for n, x in (("k", k), ("v", v)):
        x = x.permute(0, 2, 1, 3)[bi, si]                                    # [tokens, h, d]
        if st["k_scale"] is not None:
            x, scale = _quantise(x)
            st[n + "_scale"][page, :, slot] = scale
        _raw(st[n + "_cache"])[page, :, slot] = _raw(x.to(st[n + "_cache"].dtype))
    return _cache_outputs(st)


def _gather(st, n, s):
    """Dense fp32 [b, h, s, d] of the first s positions, zeros behind each sequence's length."""
    cache, table = st[n + "_cache"], st["page_table"].long()
    ps = cache.shape[2]
    pos = torch.arange(s, device="cuda")
    live = pos < st["seq_lens_kv"].long().unsqueeze(1)                        # [b, s]
    page = torch.where(live, table[:, (pos // ps).clamp_max(table.shape[1] - 1)], 0)
    slot = (pos % ps).expand_as(page)
    x = _raw(cache)[page, :, slot]                                            # [b, s, h, d]
    x = x.view(torch.float8_e4m3fn).float() if cache.dtype == torch.float8_e4m3fn else x.float()
    if st[n + "_scale"] is not None:
        x = x * st[n + "_scale"][page, :, slot].unsqueeze(-1)
    return torch.where(live[..., None, None], x, 0.0).permute(0, 2, 1, 3)


def _read(st):
    for n in ("k", "v"):
        st[n].copy_(_gather(st, n, st[n].shape[2]))
    return st["k"], st["v"]


def _attend(st):
    q = st["q"].float()
    b, h_q, s, d = q.shape
    top = st["case"]["hi"]
    k, v = _gather(st, "k", top), _gather(st, "v", top)
    h = k.shape[1]
    lens, news = st["seq_lens_kv"].long(), st["seq_lens_q"].long()
    key, row = torch.arange(top, device="cuda"), torch.arange(s, device="cuda")
    draft = key - (lens - news).unsqueeze(1)                                  # [b, keys]: index among the new tokens
    see = (key < lens.unsqueeze(1)).unsqueeze(1) & (row < news.unsqueeze(1)).unsqueeze(2)   # [b, s, keys]
    if st["case"]["mask"] == "bottom_right":
        see &= draft.unsqueeze(1) <= row.unsqueeze(1)
    if st["tree_mask"] is not None:
        j = draft.clamp(0, s - 1)
        word = torch.gather(st["tree_mask"], 2, (j // 32).unsqueeze(1).expand(b, s, top))
        see &= (draft < 0).unsqueeze(1) | ((word >> (j % 32).unsqueeze(1)) & 1).bool()
    see = see[:, None, None]                                                  # [b, 1, 1, s, keys]
    score = torch.matmul(q.reshape(b, h, h_q // h * s, d), k.transpose(2, 3)).view(b, h, h_q // h, s, top) / math.sqrt(d)
    score = torch.where(see, score, -math.inf)
    big = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(big == -math.inf, 0.0, big))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, h, h_q // h * s, top), v).view(b, h, h_q // h, s, d) / torch.where(total > 0, total, 1.0)
    st["o"].copy_(o.reshape(b, h_q, s, d))
    st["lse"].copy_((big + torch.log(total)).reshape(b, h_q, s))
    return st["o"], st["lse"]


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------

def _turn64(x, pos, f, interleaved, factor):
    """Each pair as a complex number times factor * exp(i * pos * f); x [..., s, d], pos [s]."""
    n = f.numel()
    x = x.double().clone()
    unit = torch.polar(torch.full((pos.numel(), n), factor, dtype=torch.float64, device="cuda"), pos.double()[:, None] * f[None])
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * unit
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _nearest_e4m3(x):
    """The nearest E4M3 value, ties to the even one: a multiple of 2^(exponent - 3), of 2^-9 at least."""
    step = torch.ldexp(torch.ones_like(x), (torch.frexp(x).exponent - 4).clamp_min(-9))
    return torch.clamp(torch.round(x / step) * step, -E4M3_MAX, E4M3_MAX)


def _sequence64(st, i, n, count):
    """The first `count` cached rows of sequence i in 64 bits, [h, count, d]."""
    cache = st[n + "_cache"]
    ps = cache.shape[2]
    pages = st["page_table"][i, : -(-count // ps)].long()
    x = _raw(cache)[pages].contiguous()
    x = x.view(cache.dtype).double()
    if st[n + "_scale"] is not None:
        x = x * st[n + "_scale"][pages].double().unsqueeze(-1)
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :count]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        f = -st["inv_freq"] if case["backward"] else st["inv_freq"]
        return tuple(torch.stack([_turn64(st[n][i], st["positions"][i], f, case["interleaved"], st["factor"])
                                  for i in range(case["b"])]) for n in ("q", "k"))
    lens, news = _lens(case), _news(case)
    if case["op"] == "read":
        out = [torch.zeros(case["b"], case["h_kv"], case["s"], case["d"], dtype=torch.float64, device="cuda") for _ in range(2)]
        for i, n in enumerate(lens):
            for x, name in zip(out, ("k", "v")):
                x[i, :, :n] = _sequence64(st, i, name, n)
        return tuple(out)
    if case["op"] == "write":
        ps, values = case["page"], {n: st[n + "_cache"].double() for n in ("k", "v")}
        scales = {n: None if st[n + "_scale"] is None else st[n + "_scale"].double() for n in ("k", "v")}
        for i in range(case["b"]):
            pos = torch.arange(lens[i] - news[i], lens[i], device="cuda")
            page, slot = st["page_table"][i].long()[pos // ps], pos % ps
            for n in ("k", "v"):
                x = st[n][i, :, : news[i]].double()
                if n == "k" and "inv_freq" in st:
                    x = _turn64(x, pos, st["inv_freq"], case["interleaved"], st["factor"])
                if scales[n] is not None:
                    scale = x.abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
                    x = _nearest_e4m3(x / scale.unsqueeze(-1))
                    scales[n][page, :, slot] = scale.transpose(0, 1)
                values[n][page, :, slot] = x.transpose(0, 1)
        return [values["k"], values["v"]] + ([scales["k"], scales["v"]] if scales["k"] is not None else [])
    group = case["h_q"] // case["h_kv"]
    o = torch.zeros(case["b"], case["h_q"], case["s"], case["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((case["b"], case["h_q"], case["s"]), -math.inf, dtype=torch.float64, device="cuda")
    for i in range(case["b"]):
        n, m = lens[i], news[i]
        k, v = _sequence64(st, i, "k", n), _sequence64(st, i, "v", n)
        hide = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        if case["mask"] == "bottom_right":
            hide[:, n - m:] = torch.ones(m, m, dtype=torch.bool, device="cuda").triu(1)
        if case["mask"] == "tree":
            words = st["tree_mask"][i, :m].long() & 0xFFFFFFFF
            hide[:, n - m:] = torch.stack([(words[:, j // 32] >> (j % 32)) & 1 for j in range(m)], 1) == 0
        for h in range(case["h_q"]):
            x = st["q"][i, h, :m].double() @ k[h // group].T / math.sqrt(case["d"])
            x = x.masked_fill(hide, -math.inf)
            lse[i, h, :m] = torch.logsumexp(x, -1)
            o[i, h, :m] = torch.softmax(x, -1) @ v[h // group]
    return o, lse
