"""Shared helpers for the tests of the serving operators: caches filled page by page, and tolerances.

Tolerances count roundings.  One rounding to a type is off by at most half a step, finfo(t).eps / 2
relative to the value (bf16 2^-8, fp16 2^-11, e4m3 2^-4), or half of the smallest step below its
normal range (fp16 2^-25, e4m3 2^-10)."""
from __future__ import annotations

import dataclasses
from typing import Optional

import numpy as np
import torch

from oracle import serving_oracle as so
from sdpa_testlib import f64, lib

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10}


def values_of(t: torch.Tensor) -> np.ndarray:
    """The values an E4M3 or 16-bit tensor stands for, in fp64 (codes for E4M3)."""
    return t.detach().cpu().to(torch.float32).double().numpy()


def randn(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float32)


@dataclasses.dataclass
class PagedCache:
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor]
    v_scale: Optional[torch.Tensor]
    page_table: torch.Tensor
    lens: torch.Tensor

    def where(self):
        return self.k, self.v, self.page_table, self.lens

    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)

    def np(self):
        sc = lambda t: None if t is None else f64(t)
        return (values_of(self.k), values_of(self.v), sc(self.k_scale), sc(self.v_scale), self.page_table.cpu().numpy())


def make_cache(lens, h_kv, d, page, kind, seed=0, slot_major=True, spare=2, wide=None, device="cuda", fill=None,
               v_spread=1.0) -> PagedCache:
    """A cache whose sequences hold N(0, 1) rows in shuffled pages.  Slots that no sequence reaches hold
    ``fill`` in K and V (NaN codes by default) and NaN scales; unused columns of the page table hold -1.
    v_spread > 1 gives every row of V a magnitude of its own, up to that factor."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), wide or max(need + [1])), -1, dtype=torch.int32)
    used = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n].to(torch.int32)
        for j in range(n):
            used[order[at + j], : min(page, lens[i] - j * page)] = True
        at += n
    out = []
    for which in range(2):
        x = randn(g, pages, page, h_kv, d)
        if which == 1 and v_spread != 1.0:
            x = x * v_spread ** torch.rand(pages, page, h_kv, 1, generator=g)
        scale = None
        if kind == "e4m3":
            scale = (x.abs().amax(-1) / 448.0).clamp_min(2.0 ** -69)
            x = x / scale[..., None]
            scale = torch.where(used[..., None], scale, torch.full_like(scale, float("nan")))
            scale = scale.permute(0, 2, 1).contiguous().to(device)
        x = torch.where(used[..., None, None], x, torch.full_like(x, float("nan") if fill is None else fill)).to(DT[kind])
        if slot_major:
            x = x.to(device).permute(0, 2, 1, 3)
        else:
            x = x.permute(0, 2, 1, 3).contiguous().to(device)
        out.append((x, scale))
    return PagedCache(out[0][0], out[1][0], out[0][1], out[1][1], table.to(device),
                      torch.tensor(lens, dtype=torch.int32, device=device))


def random_tree(n, seed):
    """bool [n, n]: drafted token i sees itself and its ancestors in a random tree."""
    rng = np.random.default_rng(seed)
    see = np.zeros((n, n), dtype=bool)
    for j in range(n):
        parent = int(rng.integers(-1, j)) if j else -1
        if parent >= 0:
            see[j] = see[parent]
        see[j, j] = True
    return see


def pack_tree(see: np.ndarray) -> torch.Tensor:
    """int32 [b, s, ceil(s/32)] words of bool [b, s, s]."""
    b, s, _ = see.shape
    w = np.zeros((b, s, -(-s // 32)), dtype=np.uint32)
    for j in range(s):
        w[:, :, j // 32] |= see[:, :, j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(w.view(np.int32))


def kv_rounding(kind, rows, d, dtype):
    """Relative rounding of an E4M3 cache's values in the products of `rows` query rows a KV head (results in
    FP16: none, the weights carry what F16 has no room for)."""
    return 2.0 ** -11 if kind == "e4m3" and rows > 32 and d <= 128 and dtype == "bf16" else 0.0


def run_decode(cache: PagedCache, q, *, lens_q=None, causal=False, tree=None, scale=None, with_lse=True, stream=None):
    """sdpa_decode into guarded outputs; the workspace starts as NaNs."""
    from sdpa_testlib import check_guard, guarded_empty_like
    m = lib()
    o, ob = guarded_empty_like(q)
    lse = lb = None
    if with_lse:
        lse, lb = guarded_empty_like(torch.empty(q.shape[:3]), torch.float32)
    tm = None if tree is None else pack_tree(tree).cuda()
    lq = None if lens_q is None else torch.tensor(lens_q, dtype=torch.int32, device="cuda")
    n = m.sdpa_decode_workspace_size(q, *cache.where(), **cache.scales(), tree_mask=tm)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    m.sdpa_decode(q, *cache.where(), o, lse, workspace=ws, seq_lens_q=lq, **cache.scales(), attn_scale=scale,
                  causal=causal, tree_mask=tm, stream=stream)
    torch.cuda.synchronize()
    assert m.sdpa_device_error() == 0
    check_guard(ob, "O")
    if lb is not None:
        check_guard(lb, "LSE")
    return o, lse


def assert_attend_close(o, lse, ref, dtype, weights, what="", kv_rounding=0.0):
    """O within the roundings of its weights (to `weights`, 16-bit) and of its own store, LSE within
    that of its exponentials.

    A weight 2^x carries its rounding to 16 bits (half a step) and the errors of x: the fp32 sums of
    q.k (d products; with |q.k| <= 2^7 before the scale and up to d/16 partial sums in the tensor
    core's 2^-22 relative steps, times the scale <= 2^-3: under 2^-14) and of ex2 and log2 (2^-21).
    The sum l has the second kind only.  Together |dO| <= (half + 2^-13) * sum P|v| + half |O|.
    kv_rounding: relative rounding of V's elements on their way into the products (0: none; blocks of many
    rows widen E4M3 to F16 with its scale, 2^-11); it adds kv_rounding * sum P|v|."""
    O, L, spread = ref[:3]
    got = f64(o)
    assert np.isfinite(got).all(), f"{what} O: not finite"
    tol = (HALF_STEP[weights] + 2.0 ** -13 + kv_rounding) * spread + HALF_STEP[dtype] * np.abs(O) * 1.01 + TINY[dtype]
    bad = np.abs(got - O) > tol
    assert not bad.any(), f"{what} O: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - O) / tol):.2f} of the tolerance"
    if lse is not None:
        l = f64(lse)
        assert np.array_equal(np.isneginf(l), np.isneginf(L)), f"{what} LSE: empty rows differ"
        fin = np.isfinite(L)
        err = np.abs(l[fin] - L[fin])
        tol = 2.0 ** -13 + 2.0 ** -20 * np.abs(L[fin])
        assert np.isfinite(l[fin]).all() and (err <= tol).all(), f"{what} LSE: max err {err.max():.3e}"
