"""More serving-side operators of the library, what they are measured on, and their plain forms:

* rotary positions with several axes (time, height, width), forward, backward, and on the way into a paged cache;
* the pages of a cache: sequences forked, grown (with the copies of shared pages) and freed, the cache compacted;
* drafted tokens, a chain or a tree, verified against the target's probabilities, and the cache rows of the kept ones.

``own`` chooses between the plain forms (elementary torch operations in fp32, angles in fp64, masses of tokens as whole
numbers of 2^-42) and the library's calls.  Cache tensors are logical [pages, h_kv, page_size, d] views; the cache is stored
token-major in each page.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -60          # rows with a smaller largest value are scaled as if it were this one
UNIT = 2.0 ** 42               # a token's mass counts in whole 2^-42

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # Q and K of one new token for a few sequences that hold images: latency only.
        dict(name="axes_decode_b8", op="axes", b=8, s=1, h_q=32, h_kv=8, d=128, sections="16,24,24", order="blocks",
             dtype="bf16", interleaved=False, backward=False, far=8192),
        # The prompt of a clip: 16 frames of 32 x 32 patches, three axes, grouped heads.
        dict(name="axes_clip_s16384", op="axes", b=1, s=16384, h_q=32, h_kv=8, d=128, sections="16,24,24", order="blocks",
             dtype="bf16", interleaved=False, backward=False, far=2000),
        # Gradients in an image encoder: rows and columns, half of each head for each, adjacent pairs, an odd length.
        dict(name="axes_bwd_image_d64", op="axes", b=3, s=4899, h_q=16, h_kv=16, d=64, sections="16,16", order="blocks",
             dtype="f16", interleaved=True, backward=True, far=0),
        # Prompts with images go into an E4M3 cache, K rotated on the way, the axes dealt out pair by pair; ragged.
        dict(name="axes_write_b2_e4m3", op="write", b=2, s=8192, h_kv=8, d=128, page=64, lo=6001, hi=8192, sections="24,20,20",
             order="interleaved", dtype="bf16", cache="e4m3", interleaved=False, far=100),
        # One step of a beam search over a short context: rows taken over from others, a token's room, shared pages copied.
        dict(name="beams_b4", op="beams", b=4, beams=4, lo=1000, hi=1000, more=1, h_kv=8, d=128, page=64, dtype="bf16",
             cache="e4m3"),
        # The same for 8 prompts with 8 beams each, 1K to 16K tokens, 16-bit pages.
        dict(name="beams_b64_bf16", op="beams", b=64, beams=8, lo=1000, hi=16000, more=5, h_kv=8, d=128, page=64, dtype="bf16",
             cache="bf16"),
        # Two of four sequences end; what they leave is small.
        dict(name="retire_b4", op="retire", b=4, lo=100, hi=700, gone=0.5, h_kv=8, d=128, page=64, dtype="f16", cache="f16"),
        # Half of 96 sequences end, and the pages of the others move together so that the cache can shrink.
        dict(name="retire_b96_bf16", op="retire", b=96, lo=300, hi=3000, gone=0.5, h_kv=8, d=128, page=64, dtype="bf16",
             cache="bf16"),
        # Four drafted tokens of one sequence against a small vocabulary: latency.
        dict(name="verify_b1_v32000", op="verify", b=1, s=5, vocab=32000, dtype="f32", tree=False, draft=True),
        # Five drafted tokens for 64 sequences, a large vocabulary.
        dict(name="verify_b64_v131072", op="verify", b=64, s=6, vocab=131072, dtype="f32", tree=False, draft=True),
        # Trees of 48 tokens for 16 sequences: their rows written, the trees verified, the accepted rows kept.
        dict(name="tree48_b16_e4m3", op="draft", b=16, s=48, vocab=100003, dtype="bf16", tree=True, draft=False, lo=300, hi=2000,
             h_kv=8, d=128, page=64, cache="e4m3"),
        # Small trees, an odd vocabulary, small pages.
        dict(name="tree13_b4_f16_d64", op="draft", b=4, s=13, vocab=50257, dtype="f16", tree=True, draft=False, lo=333, hi=1021,
             h_kv=12, d=64, page=16, cache="f16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "axes", "write", "beams", "retire", "verify", "verify", "draft"])
    dtype, d = rng.choice(["f16", "bf16"]), rng.choice([64, 128, 128, 256])
    if op in ("axes", "write"):
        half, n = d // rng.choice([2, 2, 4]), rng.choice([2, 3, 3, 4])
        cuts = sorted(rng.sample(range(1, half), n - 1))
        case = dict(op=op, d=d, sections=",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [half])),
                    order=rng.choice(["blocks", "interleaved"]), dtype=dtype, interleaved=rng.random() < 0.5,
                    far=rng.choice([0, 5000, 500000]), h_kv=rng.choice([1, 2, 8, 12]), s=_log_int(rng, 1, 8192))
        if op == "axes":
            case["h_q"] = case["h_kv"] * rng.choice([1, 4, 8])
            top = (16384 * 40 * 128) // (case["s"] * (case["h_q"] + case["h_kv"]) * d)
            return dict(case, b=max(1, min(_log_int(rng, 1, 16), top)), backward=rng.random() < 0.5)
        hi = case["s"] + _log_int(rng, 1, 4096)
        return dict(case, b=max(1, min(_log_int(rng, 1, 32), (2 * 8192 * 8 * 128) // (case["s"] * case["h_kv"] * d))), hi=hi,
                    lo=max(1, hi // rng.choice([1, 2, 4])), page=rng.choice([16, 32, 64, 128, 48]),
                    cache=rng.choice(["e4m3", dtype]))
    page, cache, h_kv = rng.choice([16, 32, 64, 128, 48]), rng.choice(["e4m3", dtype]), rng.choice([1, 2, 4, 8, 12])
    if op in ("beams", "retire"):
        hi = _log_int(rng, 20, 16000)
        b = max(1, min(_log_int(rng, 1, 96), (96 * 1650 * 8 * 128) // (hi * h_kv * d)))
        case = dict(op=op, b=b, lo=max(1, hi // rng.choice([1, 2, 10])), hi=hi, h_kv=h_kv, d=d, page=page, dtype=dtype, cache=cache)
        if op == "retire":
            return dict(case, gone=rng.choice([0.2, 0.5, 0.8]))
        return dict(case, beams=rng.choice([1, 2, 4, 8]), more=_log_int(rng, 1, 200))
    s, vocab = _log_int(rng, 1, 64), _log_int(rng, 1000, 260000)
    if op == "draft":
        hi = s + _log_int(rng, 1, 2000)
        return dict(op=op, b=max(1, min(_log_int(rng, 1, 32), (16 * 48 * 100003) // (s * vocab))), s=s, vocab=vocab, dtype=dtype,
                    tree=True, draft=False, lo=max(s, hi // 2), hi=hi, h_kv=h_kv, d=d, page=page, cache=cache)
    tree = rng.random() < 0.4
    return dict(op=op, b=max(1, min(_log_int(rng, 1, 96), (64 * 6 * 131072) // (s * vocab))), s=s, vocab=vocab,
                dtype=rng.choice(["f32", "f32", dtype]), tree=tree, draft=not tree and rng.random() < 0.8)


def _lens(case):
    """Tokens of each sequence (of each prompt's beams): spread over [lo, hi], the last one hi."""
    b, lo, hi, k = case["b"], case["lo"], case["hi"], case.get("beams", 1)
    return [hi if i // k == (b - 1) // k else lo + int((hi - lo) * ((i // k * 0.6180339887 + 0.31) % 1.0)) for i in range(b)]


def _news(case):
    """New tokens of each sequence: all ``s`` rows, or as many as the sequence has."""
    return [min(case["s"], n) for n in _lens(case)]


def _page_bytes(case):
    es, scale = (1, 4) if case["cache"] == "e4m3" else (2, 0)
    return 2 * case["page"] * case["h_kv"] * (case["d"] * es + scale)


def work(case):
    """For the pages: what the tables, the counts and the expected copies come to.  For a verification: one row of the target's
    probabilities of each sequence, and the draft's where a drafted token is refused (three of four)."""
    op = case["op"]
    if op == "axes":
        n = case["b"] * case["s"] * (case["h_q"] + case["h_kv"]) * case["d"]
        return {"bytes": 4 * n, "flops": 3 * n}
    if op == "write":
        rows = 2 * sum(_news(case)) * case["h_kv"]
        cb, scale = (1, 4) if case["cache"] == "e4m3" else (2, 0)
        return {"bytes": rows * (case["d"] * (2 + cb) + scale), "flops": rows * case["d"] * 4}
    if op in ("beams", "retire"):
        pages = sum(-(-n // case["page"]) for n in _lens(case))
        if op == "retire":
            moves = int(case["gone"] * (1 - case["gone"]) * pages)
        else:
            moves = int(sum(n % case["page"] != 0 for n in _lens(case)) * (1 - 1 / case["beams"]) ** case["beams"])
        return {"bytes": 2 * moves * _page_bytes(case) + 24 * pages, "flops": 4 * pages}
    es = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    rows = case["b"] * (1.75 if case["draft"] else 1.0)
    w = {"bytes": int(rows * case["vocab"] * es), "flops": int(3 * rows * case["vocab"])}
    if op == "draft":
        w["bytes"] += sum(_news(case)) * _page_bytes(case) // case["page"] * 3
    return w


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _axis_of(case):
    """The axis of each pair: as many in a row as a section has, or dealt out in turns to the axes that still want one."""
    sections = [int(x) for x in case["sections"].split(",")]
    if case["order"] == "blocks":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    return [a for turn in range(max(sections)) for a, n in enumerate(sections) if turn < n]


def _table(inv_freq):
    """Turns per position as 64-bit binary fractions (what the library's rotary table holds)."""
    turns = [int(round(math.ldexp(f / (2 * math.pi), 64))) for f in inv_freq]
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


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _grid(g, case):
    """Positions [axes, b, s]: frames, rows and columns of a clip (rows and columns of an image), behind some text."""
    n, b, s = len(case["sections"].split(",")), case["b"], case["s"]
    i = torch.arange(s, device="cuda")
    side = max(1, min(32, math.isqrt(s)))
    axes = [i // (side * side), i // side % side, i % side, i] if n != 2 else [i // max(1, math.isqrt(s)), i % max(1, math.isqrt(s))]
    start = torch.randint(0, case["far"] + 1, (b, 1), generator=g, device="cuda")
    return torch.stack([start + a for a in axes[:n]]).to(torch.int32)


def _fill_cache(g, case, pages):
    st, ps, h, d = {"k_scale": None, "v_scale": None}, case["page"], case["h_kv"], case["d"]
    for n in ("k", "v"):
        x = _randn(g, _DT[case["dtype"]], pages, ps, h, d)
        if case["cache"] == "e4m3":
            x, scale = _quantise(x)
            st[n + "_scale"] = scale.permute(0, 2, 1).contiguous()
        st[n + "_cache"] = x.permute(0, 2, 1, 3)
    return st


def _cache(g, case, lens):
    """A filled paged cache: pages in shuffled order, each sequence's last page partly used, a few spare pages."""
    need = [-(-n // case["page"]) for n in lens]
    order = torch.randperm(sum(need) + 3, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return dict(_fill_cache(g, case, sum(need) + 3), page_table=table, seq_lens=_int32(lens))


def _beams(g, case, seed):
    """Prompts whose beams share all but their last pages, and the beams that the next step goes on with."""
    rng, lens, ps, k = np.random.default_rng(seed), _lens(case), case["page"], case["beams"]
    top = -(-(max(lens) + case["more"]) // ps)
    rows, at = np.full((case["b"], top), -1, dtype=np.int32), 0
    for i, n in enumerate(lens):
        need = -(-n // ps)
        shared = max(0, need - int(rng.integers(1, 4))) if i % k else 0
        rows[i, :shared] = rows[i - i % k, :shared]
        rows[i, shared:need] = np.arange(at, at + need - shared)
        at += need - shared
    room = sum(-(-n // ps) if i % k == 0 else min(3, -(-n // ps)) for i, n in enumerate(lens)) + case["b"] * (2 + case["more"] // ps) + 3
    order = rng.permutation(room).astype(np.int32)
    rows = np.where(rows >= 0, order[rows], -1).astype(np.int32)
    parents = [i - i % k + int(rng.integers(0, min(k, case["b"] - (i - i % k)))) for i in range(case["b"])]
    counts = np.bincount(rows[rows >= 0], minlength=room)
    return dict(_fill_cache(g, case, room), page_table=_int32(rows), seq_lens=_int32(lens), ref_counts=_int32(counts),
                parents=_int32(parents), new_lens=_int32([n + case["more"] for n in lens]))


def _retired(g, case, seed):
    rng, lens, ps = np.random.default_rng(seed), _lens(case), case["page"]
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + case["b"]
    order, at = rng.permutation(pages).astype(np.int32), 0
    rows = np.full((case["b"], max(need)), -1, dtype=np.int32)
    for i, n in enumerate(need):
        rows[i, :n] = order[at:at + n]
        at += n
    gone = rng.permutation(case["b"])[: int(round(case["gone"] * case["b"]))]
    kept = [0 if i in gone else n for i, n in enumerate(lens)]
    counts = np.bincount(rows[rows >= 0], minlength=pages)
    return dict(_fill_cache(g, case, pages), page_table=_int32(rows), seq_lens=_int32(lens), ref_counts=_int32(counts), kept_lens=_int32(kept))


def _drafted(g, case, seed):
    """The target's probabilities behind each token, drafted tokens (of a draft that agrees with it mostly) and random numbers."""
    b, s, n, dt = case["b"], case["s"], case["vocab"], _DT[case["dtype"]]
    logits = torch.randn(b, s, n, generator=g, device="cuda") * 2.5
    tokens = torch.zeros(b, s, dtype=torch.int64, device="cuda")
    st = dict(parents=None, draft_probs=None)
    if case["tree"]:
        rng = np.random.default_rng(seed)
        parents = np.full((b, s), -1, dtype=np.int64)
        rank = np.zeros((b, s), dtype=np.int64)
        for j in range(1, s):
            parents[:, j] = rng.integers(max(0, j - 6), j, b)
            rank[:, j] = (parents[:, :j] == parents[:, j:j + 1]).sum(1)
        likely = torch.topk(logits, min(8, n), -1).indices
        at, which = torch.from_numpy(parents).cuda().clamp_min(0), torch.from_numpy(rank).cuda().clamp_max(likely.shape[-1] - 1)
        tokens[:, 1:] = likely[torch.arange(b, device="cuda")[:, None], at, which][:, 1:]
        st["parents"] = torch.from_numpy(parents).cuda().to(torch.int32)
    else:
        # Row j of the draft's probabilities is what token j was drawn from: near the target's behind token j - 1.
        near = torch.softmax(torch.roll(logits, 1, 1) + 0.6 * torch.randn(b, s, n, generator=g, device="cuda"), -1).to(dt)
        drawn = torch.rand(b, s, 1, generator=g, device="cuda")
        tokens = (torch.cumsum(near.float(), -1) <= drawn).sum(-1).clamp_max(n - 1)
        if case["draft"]:
            st["draft_probs"] = near
    st["probs"] = torch.softmax(logits, -1).to(dt)
    st["tokens"] = tokens.to(torch.int32)
    st["uniform"] = torch.rand(b, s, generator=g, device="cuda")
    for name in ("path", "new_tokens"):
        st[name] = torch.empty(b, s, dtype=torch.int32, device="cuda")
    st["accepted"] = torch.empty(b, dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    st = dict(op=op, case=case)
    if op in ("axes", "write"):
        axis = _axis_of(case)
        st["inv_freq"] = [10000.0 ** (-i / len(axis)) for i in range(len(axis))]
        st["table"], st["axis"], st["positions"] = _table(st["inv_freq"]), bytes(axis), _grid(g, case)
        if op == "axes":
            st["q"], st["k"] = (_bshd(g, dt, case["b"], case[h], case["s"], case["d"]) for h in ("h_q", "h_kv"))
            st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
            return st
    if op in ("write", "draft"):
        st.update(_cache(g, case, _lens(case)))
        st["seq_lens_q"] = _int32(_news(case))
        st["k"], st["v"] = (_bshd(g, dt, case["b"], case["h_kv"], case["s"], case["d"]) for _ in range(2))
    if op in ("verify", "draft"):
        st.update(_drafted(g, case, seed))
    if op in ("beams", "retire"):
        st.update(_beams(g, case, seed) if op == "beams" else _retired(g, case, seed))
        pairs = case["b"] if op == "beams" else st["ref_counts"].numel() // 2 + 1
        st["src"], st["dst"] = (torch.empty(pairs, dtype=torch.int32, device="cuda") for _ in range(2))
        st["missing"] = torch.empty(1, dtype=torch.int32, device="cuda")
        for n in ("page_table", "seq_lens", "ref_counts"):
            st["new_" + n] = torch.empty_like(st[n])
    return st


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------

def run(st):
    if own:
        return _library(st)
    return {"axes": _axes, "write": _write, "beams": _beam_step, "retire": _retire, "verify": _verify, "draft": _draft_step}[st["op"]](st)


def _library(st):
    import attention_flashattention_sdpa_gb300 as sdpa
    op, case = st["op"], st["case"]
    if op == "axes":
        call = sdpa.sdpa_rope_bwd if case["backward"] else sdpa.sdpa_rope_fwd
        call(st["q"], st["k"], st["q_out"], st["k_out"], st["table"], st["positions"], interleaved=case["interleaved"], axes=st["axis"])
        return st["q_out"], st["k_out"]
    if op in ("beams", "retire"):
        new = (st["new_page_table"], st["new_ref_counts"])
        if op == "beams":
            sdpa.sdpa_cache_fork(st["page_table"], st["seq_lens"], st["parents"], st["ref_counts"], new[0], st["new_seq_lens"],
                                 new[1], page_size=case["page"])
            sdpa.sdpa_cache_grow(new[0], st["new_seq_lens"], st["new_lens"], new[1], st["src"], st["dst"], st["missing"],
                                 page_size=case["page"])
        else:
            sdpa.sdpa_cache_free(st["page_table"], st["seq_lens"], st["kept_lens"], st["ref_counts"], page_size=case["page"],
                                 page_table_out=new[0], ref_counts_out=new[1])
            sdpa.sdpa_cache_compact(new[0], st["kept_lens"], new[1], st["src"], st["dst"], page_size=case["page"])
        sdpa.sdpa_cache_copy(st["k_cache"], st["v_cache"], st["src"], st["dst"], k_scale=st["k_scale"], v_scale=st["v_scale"])
        return _page_outputs(st)
    where, scales = None, {}
    if op in ("write", "draft"):
        where = (st["k_cache"], st["v_cache"], st["page_table"], st["seq_lens"])
        scales = dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
        rope = {}
        if op == "write":
            rope = dict(rope_table=st["table"], positions=st["positions"], interleaved=case["interleaved"], axes=st["axis"])
        sdpa.sdpa_cache_write(st["k"], st["v"], *where, seq_lens_q=st["seq_lens_q"], **scales, **rope)
        if op == "write":
            return _cache_outputs(st)
    sdpa.sdpa_verify(st["tokens"], st["probs"], st["uniform"], st["accepted"], st["path"], st["new_tokens"], parents=st["parents"],
                     draft_probs=st["draft_probs"])
    if op == "draft":
        sdpa.sdpa_cache_keep(*where, st["path"], st["accepted"], seq_lens_q=st["seq_lens_q"], **scales)
        return [st["accepted"], st["path"], st["new_tokens"]] + _cache_outputs(st)
    return [st["accepted"], st["path"], st["new_tokens"]]


def _cache_outputs(st):
    out = [st["k_cache"], st["v_cache"]]
    return out + [st["k_scale"], st["v_scale"]] if st["k_scale"] is not None else out


def _page_outputs(st):
    out = [st["new_page_table"], st["new_ref_counts"], st["src"], st["dst"]]
    return out + ([st["new_seq_lens"], st["missing"]] if st["op"] == "beams" else []) + _cache_outputs(st)


def _rotate(x, st, backward=False):
    """x [b, h, s, d] (fp32) rotated: each pair by the position on its axis; the elements behind the pairs as they are."""
    freq = torch.tensor(st["inv_freq"], dtype=torch.float64, device="cuda")
    pos = st["positions"].double()[torch.tensor(list(st["axis"]), device="cuda")].permute(1, 2, 0)       # [b, s, pairs]
    angle = pos * (-freq if backward else freq)
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    rot, inter = 2 * len(st["axis"]), st["case"]["interleaved"]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
    y, z = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((y, z), -1).flatten(-2) if inter else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _axes(st):
    st["q_out"].copy_(_rotate(st["q"].float(), st, st["case"]["backward"]))
    st["k_out"].copy_(_rotate(st["k"].float(), st, st["case"]["backward"]))
    return st["q_out"], st["k_out"]


def _raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _write(st):
    k, v = st["k"].float(), st["v"].float()
    if "axis" in st:
        k = _rotate(k, st)
    ps, news = st["case"]["page"], st["seq_lens_q"].long()
    row = torch.arange(k.shape[2], device="cuda")
    bi, si = (row < news.unsqueeze(1)).nonzero(as_tuple=True)
    pos = (st["seq_lens"].long() - news)[bi] + si
    page, slot = st["page_table"].long()[bi, pos // ps], pos % ps
    for n, x in (("k", k), ("v", v)):
        x = x.permute(0, 2, 1, 3)[bi, si]                                    # [tokens, h, d]
        if st["k_scale"] is not None:
            x, scale = _quantise(x)
            st[n + "_scale"][page, :, slot] = scale
        _raw(st[n + "_cache"])[page, :, slot] = _raw(x.to(st[n + "_cache"].dtype))
    return _cache_outputs(st)


def _copy_pages(st, src, dst):
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if st[n] is not None:
            _raw(st[n])[dst] = _raw(st[n])[src]


def _count(pages, table, live, by):
    """`by` added to the count of every page that the live columns of a table name."""
    page = table[live].long()
    return pages.index_add_(0, page, torch.full_like(page, by, dtype=torch.int32))


def _columns(st, lens):
    """Columns of the page table that sequences of these lengths reach, and the columns."""
    col = torch.arange(st["page_table"].shape[1], device="cuda")
    return col < (-(-lens.long() // st["case"]["page"])).unsqueeze(1), col


def _beam_step(st):
    ps, parents, refs = st["case"]["page"], st["parents"].long(), st["ref_counts"].clone()
    # Each row takes over its parent's pages.
    reached, col = _columns(st, st["seq_lens"])
    lens = st["seq_lens"][parents]
    table = torch.where(reached[parents], st["page_table"][parents], -1)
    refs = _count(_count(refs, table, reached[parents], 1), st["page_table"], reached, -1)
    # Room for the new tokens: pages behind the last, and one of its own for a partly filled page that others hold too.
    more = st["new_lens"].long()
    tail = lens.long() // ps
    partly = (lens.long() % ps != 0) & (more > lens.long())
    at = torch.gather(table, 1, tail.clamp_max(table.shape[1] - 1).unsqueeze(1)).squeeze(1)
    before = ((at.unsqueeze(1) == at) & partly).tril(-1).sum(1)               # rows before this one that grow in the same page
    copied = partly & (refs[at.clamp_min(0).long()] - before > 1)
    wanted = (col >= -(-lens.long() // ps).unsqueeze(1)) & _columns(st, more)[0] | (copied.unsqueeze(1) & (col == tail.unsqueeze(1)))
    fresh = (refs == 0).nonzero().squeeze(1)[: int(wanted.sum())].to(torch.int32)
    table[wanted] = fresh
    refs[fresh.long()] = 1
    refs.index_add_(0, at[copied].long(), torch.full_like(at[copied], -1))
    new = torch.gather(table, 1, tail.clamp_max(table.shape[1] - 1).unsqueeze(1)).squeeze(1)
    st["src"].copy_(torch.where(copied, at, -1))
    st["dst"].copy_(torch.where(copied, new, -1))
    st["missing"].zero_()
    _copy_pages(st, at[copied].long(), new[copied].long())
    st["new_page_table"].copy_(table)
    st["new_seq_lens"].copy_(lens)
    st["new_ref_counts"].copy_(refs)
    return _page_outputs(st)


def _retire(st):
    reached, _ = _columns(st, st["seq_lens"])
    kept, _ = _columns(st, st["kept_lens"])
    refs = _count(st["ref_counts"].clone(), st["page_table"], reached & ~kept, -1)
    table = torch.where(reached & ~kept, -1, st["page_table"])
    # Pages in use at and behind the number of those in use move to the free ones before it, lowest to lowest.
    used = refs != 0
    n = int(used.sum())
    src, dst = n + used[n:].nonzero().squeeze(1), (~used[:n]).nonzero().squeeze(1)
    to = torch.arange(refs.numel(), dtype=torch.int32, device="cuda")
    to[src] = dst.to(torch.int32)
    st["new_page_table"].copy_(torch.where(kept, to[table.clamp_min(0).long()], table))
    st["new_ref_counts"].copy_(refs)
    st["new_ref_counts"][dst] = refs[src]
    st["new_ref_counts"][src] = 0
    for name, x in (("src", src), ("dst", dst)):
        st[name].fill_(-1)
        st[name][: x.numel()] = x.to(torch.int32)
    _copy_pages(st, src, dst)
    return _page_outputs(st)


def _mass(p):
    """Probabilities as whole numbers of 2^-42, of at most one each; NaN counts nothing."""
    return torch.round(torch.where(p > 0, p.float().clamp_max(1.0), 0.0).double() * UNIT).long()


def _verify(st):
    tokens, u, s, vocab = st["tokens"].long(), st["uniform"].double(), st["tokens"].shape[1], st["probs"].shape[2]
    b = tokens.shape[0]
    rows, node = torch.arange(b, device="cuda").unsqueeze(1), torch.arange(s, device="cuda")
    up = (node - 1).clamp_min(0).expand(b, s) if st["parents"] is None else st["parents"].long().clamp_min(0)
    target = st["probs"][rows, up, tokens]                                     # of each token, behind its parent
    drafted = node > 0
    if st["draft_probs"] is not None:
        good = u * st["draft_probs"][rows, node, tokens].double() < target.double()
    else:
        # Of the mass that earlier siblings have left (the same token twice leaves nothing for the second).
        mass = _mass(target)
        twin = (up.unsqueeze(2) == up.unsqueeze(1)) & drafted & drafted.unsqueeze(1)
        same = (twin & (tokens.unsqueeze(2) == tokens.unsqueeze(1))).tril(-1).any(2)
        mass = torch.where(same, 0, mass)
        left = (int(UNIT) - (twin.tril(-1) * mass.unsqueeze(1)).sum(2)).clamp_min(0)
        good = u * left.double() < mass.double()
        good &= ~(twin & good.unsqueeze(1)).tril(-1).any(2)                    # an earlier sibling was taken
    good |= ~drafted
    at = up                                                                    # accepted: every token on the way to the root is
    for _ in range(s.bit_length()):
        good, at = good & torch.gather(good, 1, at), torch.gather(at, 1, at)
    count = good.sum(1)
    path = torch.where(node < count.unsqueeze(1), torch.argsort(torch.where(good, 0, 1), dim=1, stable=True), -1)
    last = torch.gather(path, 1, (count - 1).unsqueeze(1)).squeeze(1)
    p = st["probs"][rows.squeeze(1), last]                                      # [b, vocab]
    mass = _mass(p)
    if st["draft_probs"] is not None:
        refused = last < s - 1
        q = st["draft_probs"][rows.squeeze(1), (last + 1).clamp_max(s - 1)]
        left = torch.where(refused.unsqueeze(1), _mass(p.float() - q.float()), mass)
    else:
        child = (up == last.unsqueeze(1)) & drafted
        taken = torch.zeros(b, vocab + 1, dtype=torch.bool, device="cuda").scatter_(1, torch.where(child, tokens, vocab), True)
        left = torch.where(taken[:, :vocab], 0, mass)
    mass = torch.where((left.sum(1) > 0).unsqueeze(1), left, mass)
    total = mass.sum(1)
    part = torch.floor(st["uniform"][:, 0].double() * 2.0 ** 31).long()
    at = (total >> 32) * part * 2 + (((total & 0xFFFFFFFF) * part) >> 31)
    drawn = (torch.cumsum(mass, 1) <= at.unsqueeze(1)).sum(1)
    drawn = torch.where(total > 0, drawn, -1)
    new = torch.gather(tokens, 1, torch.cat((path[:, 1:], path[:, :1]), 1).clamp_min(0))
    new = torch.where(node == (count - 1).unsqueeze(1), drawn.unsqueeze(1), torch.where(node < count.unsqueeze(1), new, -1))
    st["accepted"].copy_(count)
    st["path"].copy_(path)
    st["new_tokens"].copy_(new)
    return [st["accepted"], st["path"], st["new_tokens"]]


def _draft_step(st):
    _write(st)
    out = _verify(st)
    # Row path[j] of the newest rows moves to row j.
    ps, start = st["case"]["page"], (st["seq_lens"] - st["seq_lens_q"]).long()
    bi, j = (torch.arange(st["path"].shape[1], device="cuda") < st["accepted"].unsqueeze(1)).nonzero(as_tuple=True)
    here, there = start[bi] + st["path"].long()[bi, j], start[bi] + j
    table = st["page_table"].long()
    a, b = (table[bi, here // ps], here % ps), (table[bi, there // ps], there % ps)
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if st[n] is not None:
            _raw(st[n])[b[0], :, b[1]] = _raw(st[n])[a[0], :, a[1]]
    return out + _cache_outputs(st)


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------

def _turn64(x, st, i, backward=False):
    """Each pair of x [h, s, d] of sequence i as a complex number times exp(i * position * frequency), pair by pair."""
    x = x.double().clone()
    n, inter = len(st["axis"]), st["case"]["interleaved"]
    for pair in range(n):
        a, b = (2 * pair, 2 * pair + 1) if inter else (pair, pair + n)
        t = st["positions"][st["axis"][pair], i, : x.shape[1]].double() * st["inv_freq"][pair] * (-1.0 if backward else 1.0)
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(t), t)
        x[..., a], x[..., b] = z.real, z.imag
    return x


def _nearest_e4m3(x):
    """The nearest E4M3 value, ties to the even one: a multiple of 2^(exponent - 3), of 2^-9 at least."""
    step = torch.ldexp(torch.ones_like(x), (torch.frexp(x).exponent - 4).clamp_min(-9))
    return torch.clamp(torch.round(x / step) * step, -E4M3_MAX, E4M3_MAX)


def _stored64(st):
    return {n: None if st[n] is None else st[n].double() for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _listed64(values):
    return [x for x in (values["k_cache"], values["v_cache"], values["k_scale"], values["v_scale"]) if x is not None]


def _write64(st, values):
    case = st["case"]
    ps, lens, news = case["page"], _lens(case), _news(case)
    for i in range(case["b"]):
        pos = torch.arange(lens[i] - news[i], lens[i], device="cuda")
        page, slot = st["page_table"][i].long()[pos // ps], pos % ps
        for n in ("k", "v"):
            x = st[n][i, :, : news[i]].double()
            if n == "k" and "axis" in st:
                x = _turn64(x, st, i)
            if values[n + "_scale"] is not None:
                scale = x.abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
                x = _nearest_e4m3(x / scale.unsqueeze(-1))
                values[n + "_scale"][page, :, slot] = scale.transpose(0, 1)
            values[n + "_cache"][page, :, slot] = x.transpose(0, 1)


def _beams64(st):
    """Row by row, page by page, on the host."""
    case = st["case"]
    ps, lens, more = case["page"], st["seq_lens"].tolist(), st["new_lens"].tolist()
    old, counts, parents = st["page_table"].tolist(), st["ref_counts"].tolist(), st["parents"].tolist()
    width, rows = len(old[0]), []
    for i, j in enumerate(parents):
        rows.append([old[j][c] if c < -(-lens[j] // ps) else -1 for c in range(width)])
        for page in rows[i]:
            counts[page] += page >= 0
    for i, n in enumerate(lens):
        for page in old[i][: -(-n // ps)]:
            counts[page] -= 1
    lens = [lens[j] for j in parents]
    free = [page for page, c in enumerate(counts) if c == 0]
    src, dst = [-1] * len(lens), [-1] * len(lens)
    for i, n in enumerate(lens):
        if n % ps and more[i] > n and counts[rows[i][n // ps]] > 1:
            src[i], dst[i] = rows[i][n // ps], free.pop(0)
            counts[src[i]] -= 1
            counts[dst[i]], rows[i][n // ps] = 1, dst[i]
        for c in range(-(-n // ps), -(-more[i] // ps)):
            rows[i][c] = free.pop(0)
            counts[rows[i][c]] = 1
    return rows, counts, src, dst, lens


def _retire64(st):
    ps, lens, kept = st["case"]["page"], st["seq_lens"].tolist(), st["kept_lens"].tolist()
    rows, counts = st["page_table"].tolist(), st["ref_counts"].tolist()
    for row, n, m in zip(rows, lens, kept):
        for c in range(-(-m // ps), -(-n // ps)):
            counts[row[c]] -= 1
            row[c] = -1
    n = sum(c != 0 for c in counts)
    moves = dict(zip([p for p in range(n, len(counts)) if counts[p]], [p for p in range(n) if not counts[p]]))
    for a, b in moves.items():
        counts[b], counts[a] = counts[a], 0
    rows = [[moves.get(p, p) for p in row] for row in rows]
    room = st["src"].numel()
    src, dst = (list(x) + [-1] * (room - len(moves)) for x in (moves.keys(), moves.values()))
    return rows, counts, src, dst


def _verify64(st):
    """Token by token, on the host; masses as Python's whole numbers."""
    tokens, uniform, s = st["tokens"].tolist(), st["uniform"].double().tolist(), st["tokens"].shape[1]
    whole = lambda x: round(min(max(x, 0.0), 1.0) * UNIT)    # noqa: E731
    counts, paths, news = [], [], []
    for i, row in enumerate(tokens):
        parents = [j - 1 for j in range(s)] if st["parents"] is None else st["parents"][i].tolist()
        path, gone = [0], []
        while True:
            n, gone, step = path[-1], [], None
            for j in (j for j in range(n + 1, s) if parents[j] == n):
                p = float(st["probs"][i, n, row[j]])
                if st["draft_probs"] is not None:
                    good = uniform[i][j] * float(st["draft_probs"][i, j, row[j]]) < p
                else:
                    left = max(0, int(UNIT) - sum(whole(float(st["probs"][i, n, x])) for x in set(gone)))
                    good = uniform[i][j] * left < (0 if row[j] in gone else whole(p))
                if good:
                    step = j
                    break
                gone.append(row[j])
            if step is None:
                break
            path.append(step)
        p = st["probs"][i, path[-1]].float()
        mass = left = torch.round(p.clamp(0, 1).double() * UNIT).long()
        if st["draft_probs"] is not None and gone:
            left = torch.round((p - st["draft_probs"][i, path[-1] + 1].float()).clamp(0, 1).double() * UNIT).long()
        elif gone:
            left = mass.clone()
            left[gone] = 0
        sums = np.cumsum((left if int(left.sum()) else mass).cpu().numpy())
        at = int(sums[-1]) * int(math.floor(uniform[i][0] * 2 ** 31)) >> 31
        drawn = int(np.searchsorted(sums, at, side="right")) if sums[-1] else -1
        rest = [-1] * (s - len(path))
        counts.append(len(path))
        news.append([row[j] for j in path[1:]] + [drawn] + rest)
        paths.append(path + rest)
    return [_int32(counts), _int32(paths), _int32(news)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "axes":
        return tuple(torch.stack([_turn64(st[n][i], st, i, case["backward"]) for i in range(case["b"])]) for n in ("q", "k"))
    if case["op"] == "verify":
        return _verify64(st)
    values = _stored64(st)
    if case["op"] == "write":
        _write64(st, values)
        return _listed64(values)
    if case["op"] == "draft":
        _write64(st, values)
        out = _verify64(st)
        ps = case["page"]
        for i, (n, m) in enumerate(zip(_lens(case), _news(case))):
            row = st["page_table"][i].tolist()
            for j, r in enumerate(out[1][i, : int(out[0][i])].tolist()):
                here, there = n - m + r, n - m + j
                for x in _listed64(values):
                    x[row[there // ps], :, there % ps] = x[row[here // ps], :, here % ps]
        return out + _listed64(values)
    if case["op"] == "beams":
        rows, counts, src, dst, lens = _beams64(st)
        more = [_int32(lens), _int32([0])]
    else:
        (rows, counts, src, dst), more = _retire64(st), []
    for a, b in zip(src, dst):
        if a >= 0:
            for x in _listed64(values):
                x[b] = x[a]
    return [_int32(rows), _int32(counts), _int32(src), _int32(dst)] + more + _listed64(values)
