"""Attention over a key/value cache and its eviction against the float64 oracle.

Tolerance of an output (derived, per element).  With u the half step of the
storage type (bf16 2^-8, fp32 2^-24) and A = sum_j w_j |v_j|:
  * storing the output rounds it once: u |o|;
  * bf16: the weights are rounded to bf16 once before they meet the values:
    2^-8 A;
  * a score is a sum of D products in fp32: off by at most
    d = D 2^-24 scale sum_d |q_d k_d| (plus its scaling, d again); a weight
    exp(s - m) by 2 d relative, a normalised weight by 4 d: 4 d A;
  * exponentials and the final division: a few fp32 steps, 2^-20 A;
  * the sum over n keys in fp32: rounding errors of either sign, eight
    standard deviations of n of them: 8 sqrt(n) 2^-24 A.
"""
import math

import numpy as np
import pytest
import torch

import cache_bounds as cb
import step_adaptive_sparse_b200 as area
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

INT_MAX = 2 ** 31 - 1
NAN = float("nan")
TYPES = {"bf16": (torch.bfloat16, area.AREA_DTYPE_BF16, 2.0 ** -8),
         "f32": (torch.float32, area.AREA_DTYPE_F32, 2.0 ** -24)}
PAD = 64             # guard values before and after every output


class Guarded:
    """A device tensor inside a larger buffer filled with a marker."""

    def __init__(self, shape, dtype, fill=None):
        n = int(np.prod(shape))
        self.buf = torch.full((n + 2 * PAD,), 77.0 if dtype.is_floating_point else 77, dtype=dtype, device="cuda")
        self.t = self.buf[PAD:PAD + n].view(*shape)
        if fill is not None:
            self.t.fill_(fill)

    def check(self):
        assert (self.buf[:PAD] == 77).all() and (self.buf[-PAD:] == 77).all(), "guard values overwritten"


def make(seed, dtype, B, H, Hk, Nq, S, D, lens, P=0, poison=True):
    """Inputs on the device and their exact values as float64 arrays; the rows
    behind each sequence and the queries before its first token are NaN."""
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype][0]
    q = (torch.randn(B, H, Nq, D, generator=g) * 1.5).to(t)
    k, v = torch.randn(B, Hk, S, D, generator=g).to(t), torch.randn(B, Hk, S, D, generator=g).to(t)
    kp, vp = torch.randn(Hk, P, D, generator=g).to(t), torch.randn(Hk, P, D, generator=g).to(t)
    if poison:
        for b, n in enumerate(lens):
            n = min(max(n, 0), S)
            k[b, :, n:] = NAN
            v[b, :, n:] = NAN
    host = [x.double().numpy() for x in (q, k, v, kp, vp)]
    dev = [x.cuda() for x in (q, k, v, kp, vp)]
    return dev, host, torch.tensor(lens, dtype=torch.int32).cuda()


def workspace(nb):
    # filled with NaN: what a call does not write it may not read
    w = Guarded((max(nb // 4, 8),), torch.float32, NAN)
    return w


def bound(host, o, size, dtype, scale, n):
    q, k, _, kp, _ = host
    u = TYPES[dtype][2]
    kk = np.nan_to_num(np.abs(k))
    G = q.shape[1] // k.shape[1]
    top = np.maximum(kk.max(2, initial=0), np.abs(kp).max(1, initial=0)[None]).repeat(G, 1)   # [B, H, D]
    D = q.shape[-1]
    d = D * 2.0 ** -24 * scale * (np.abs(q) * top[:, :, None]).sum(-1, keepdims=True)
    w = 2.0 ** -8 if dtype == "bf16" else 0.0
    return u * np.abs(o) + (w + 4 * d + 2.0 ** -20 + 8 * math.sqrt(max(n, 1)) * 2.0 ** -24) * size + 1e-30


def close(got, want, tol):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - want) - tol
    assert bad.max() <= 0, f"off by {np.abs(got - want).max():.3e}, {bad.max():.3e} over, at {np.unravel_index(bad.argmax(), bad.shape)}"


def run_sink(dev, lens, dtype, window, sinks, scale, o, stream=None, ws=None):
    q, k, v, _, _ = dev
    B, H, Nq, D = q.shape
    Hk, S = k.shape[1:3]
    dt = TYPES[dtype][1]
    nb = area.area_sink_attn_ws_bytes(B, H, Hk, Nq, S, D, window, sinks, dt)
    w = ws or workspace(nb)
    area.area_sink_attn(q, k, v, lens, o, w.t, nb, B, H, Hk, Nq, S, D, window, sinks, scale, dt, stream)
    return w


def run_prefix(dev, lens, dtype, causal, scale, o, stream=None, ws=None):
    q, k, v, kp, vp = dev
    B, H, Nq, D = q.shape
    Hk, S, P = k.shape[1], k.shape[2], kp.shape[1]
    dt = TYPES[dtype][1]
    nb = area.area_prefix_attn_ws_bytes(B, H, Hk, Nq, P, S, D, dt)
    w = ws or workspace(nb)
    area.area_prefix_attn(q, kp if P else None, vp if P else None, k if S else None, v if S else None,
                          lens, o, w.t, nb, B, H, Hk, Nq, P, S, D, causal, scale, dt, stream)
    return w


def run_cache(dev, lens, dtype, scale, acc, o, acco, stream=None, ws=None):
    q, k, v, _, _ = dev
    B, H, Nq, D = q.shape
    Hk, S = k.shape[1:3]
    dt = TYPES[dtype][1]
    nb = area.area_cache_attn_ws_bytes(B, H, Hk, Nq, S, D, dt)
    w = ws or workspace(nb)
    area.area_cache_attn(q, k, v, lens, acc, o, acco, w.t, nb, B, H, Hk, Nq, S, D, scale, dt, stream)
    return w


# ---- sliding window with sinks ---------------------------------------------------------------

SINK = [
    # B, H, Hk, Nq, S, D, window, sinks, lens
    (1, 1, 1, 1, 1, 64, 1, 0, [1]),
    (1, 2, 1, 1, 5, 128, 1, 1, [5]),
    (5, 4, 2, 1, 130, 64, 64, 4, [0, 1, 64, 65, 130]),
    (4, 8, 2, 1, 1000, 128, 129, 4, [1000, 999, 127, 3]),
    (2, 8, 8, 1, 700, 128, INT_MAX, 0, [700, 513]),
    (3, 5, 5, 3, 333, 64, 50, 70, [333, 2, 71]),
    (2, 16, 1, 1, 2049, 128, 700, 0, [2049, 1]),
    (1, 16, 1, 2, 513, 64, 100, 7, [513]),
    (2, 6, 2, 8, 200, 128, 33, 500, [200, 5]),
    (1, 4, 1, 17, 300, 64, 16, 3, [300]),
    (2, 12, 4, 40, 160, 128, 65, 1, [160, 39]),
    (1, 2, 2, 64, 64, 128, 20, 2, [64]),
    (2, 2, 1, 65, 65, 64, 64, 0, [65, 64]),
    (1, 3, 3, 127, 400, 128, 128, 130, [400]),
    (1, 2, 1, 128, 128, 64, 128, 0, [128]),
    (2, 4, 2, 257, 257, 128, 100, 5, [257, 129]),
    (1, 2, 2, 300, 900, 64, 256, 1, [850]),
    (1, 2, 1, 513, 1024, 128, 384, 129, [1000]),
    (2, 2, 2, 640, 640, 128, INT_MAX, 0, [640, 333]),
    (1, 1, 1, 700, 700, 64, 1, 0, [700]),
    (1, 2, 1, 520, 520, 128, 5, 400, [520]),
    (1, 2, 2, 1100, 1100, 64, 900, 64, [1100]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S,D,window,sinks,lens", SINK)
def test_sink_attention(B, H, Hk, Nq, S, D, window, sinks, lens, dtype):
    dev, host, dl = make(1, dtype, B, H, Hk, Nq, S, D, lens)
    scale = D ** -0.5
    o = Guarded((B, H, Nq, D), TYPES[dtype][0], NAN)
    w = run_sink(dev, dl, dtype, window, sinks, scale, o.t)
    want, _, size = co.cache_attention(*host[:3], lens, scale, window=window, sinks=sinks)
    close(o.t, want, bound(host, want, size, dtype, scale, S))
    o.check(), w.check()
    again = torch.full_like(o.t, NAN)
    run_sink(dev, dl, dtype, window, sinks, scale, again)
    assert torch.equal(again, o.t)
    assert area.area_kernel_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lengths_outside_the_cache_are_cut_and_null_means_full(dtype):
    B, H, Hk, Nq, S, D = 3, 4, 2, 2, 90, 64
    dev, host, dl = make(2, dtype, B, H, Hk, Nq, S, D, [90, 90, 90])
    a, b, c = (torch.full_like(dev[0], NAN) for _ in range(3))
    run_sink(dev, dl, dtype, 40, 2, 0.125, a)
    run_sink(dev, None, dtype, 40, 2, 0.125, b)
    run_sink(dev, torch.tensor([91, 10 ** 9, INT_MAX], dtype=torch.int32).cuda(), dtype, 40, 2, 0.125, c)
    assert torch.equal(a, b) and torch.equal(a, c)
    run_sink(dev, torch.tensor([-1, 0, -INT_MAX - 1], dtype=torch.int32).cuda(), dtype, 40, 2, 0.125, c)
    assert (c == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 200])
def test_keys_outside_every_window_may_hold_anything(Nq, dtype):
    """Neither the tokens between the sinks and the first window nor scores of
    the lowest or highest finite value disturb a row."""
    B, H, Hk, S, D, window, sinks = 1, 4, 2, 600, 128, 70, 3
    dev, host, dl = make(3, dtype, B, H, Hk, Nq, S, D, [S])
    lo = S - Nq + 1 - window
    a, b = (torch.full_like(dev[0], NAN) for _ in range(2))
    run_sink(dev, dl, dtype, window, sinks, 0.1, a)
    for x in dev[1:3]:
        x[:, :, sinks:lo] = NAN
    run_sink(dev, dl, dtype, window, sinks, 0.1, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 140])
def test_large_scores(Nq, dtype):
    """Scores far apart, and growing along the keys, so that the running
    maximum moves by much in every tile."""
    B, H, Hk, S, D = 1, 2, 1, 700, 64
    dev, host, dl = make(4, dtype, B, H, Hk, Nq, S, D, [S])
    ramp = torch.linspace(-40, 40, S)[:, None].cuda()
    dev[1].copy_((dev[1].float() * 0.05 + ramp * torch.sign(dev[0][0, 0, 0].float())).to(dev[1].dtype))
    host[1] = dev[1].double().cpu().numpy()
    o = torch.full_like(dev[0], NAN)
    run_sink(dev, dl, dtype, 300, 5, 0.125, o)
    want, _, size = co.cache_attention(*host[:3], [S], 0.125, window=300, sinks=5)
    close(o, want, bound(host, want, size, dtype, 0.125, S))


def test_window_of_everything_equals_full_attention():
    """With one query row the new call and the library's full attention are the
    same operation (the last row sees every key)."""
    B, H, N, D = 1, 2, 384, 128
    dev, host, dl = make(5, "bf16", B, H, H, N, N, D, [N])
    o, full = torch.full_like(dev[0], NAN), torch.full_like(dev[0], NAN)
    run_sink(dev, dl, "bf16", INT_MAX, 0, D ** -0.5, o)
    area.area_full_attn(*dev[:3], full, B, H, N, D, D ** -0.5, area.AREA_DTYPE_BF16)
    assert (o[:, :, -1].float() - full[:, :, -1].float()).abs().max() < 2e-2


# ---- shared prefix ---------------------------------------------------------------------------

PREFIX = [
    # B, H, Hk, Nq, P, S, D, lens
    (1, 1, 1, 1, 1, 1, 64, [1]),
    (2, 2, 2, 1, 64, 1, 128, [1, 0]),
    (4, 8, 8, 1, 700, 130, 64, [130, 64, 1, 65]),
    (3, 8, 2, 1, 1000, 200, 128, [200, 3, 100]),
    (17, 16, 1, 1, 333, 40, 64, [i % 41 for i in range(5, 22)]),
    (2, 16, 2, 8, 129, 70, 128, [70, 5]),
    (3, 5, 5, 3, 127, 30, 64, [30, 2, 17]),
    (2, 6, 2, 21, 255, 64, 64, [64, 20]),
    (2, 4, 2, 100, 300, 150, 128, [150, 99]),
    (2, 2, 1, 300, 129, 300, 64, [300, 200]),
    (1, 3, 3, 257, 64, 400, 128, [400]),
    (5, 4, 2, 1, 500, 0, 128, [0, 0, 0, 0, 0]),
    (3, 4, 2, 2, 0, 100, 64, [100, 1, 50]),
    (1, 4, 2, 150, 200, 0, 64, [0]),
    (40, 4, 4, 1, 2100, 33, 128, [33 - i % 34 for i in range(40)]),
    # prefixes large enough to be read once for the batch
    (8, 8, 8, 1, 1100, 20, 128, [20, 0, 3, 20, 19, 20, 1, 20]),
    (2, 8, 4, 4, 9001, 30, 128, [30, 3]),
    (17, 16, 1, 1, 7901, 40, 64, [i % 41 for i in range(5, 22)]),
    (3, 6, 2, 21, 11003, 64, 128, [64, 20, 0]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("B,H,Hk,Nq,P,S,D,lens", PREFIX)
def test_prefix_attention(B, H, Hk, Nq, P, S, D, lens, causal, dtype):
    dev, host, dl = make(6, dtype, B, H, Hk, Nq, S, D, lens, P=P)
    scale = D ** -0.5
    o = Guarded((B, H, Nq, D), TYPES[dtype][0], NAN)
    w = run_prefix(dev, dl, dtype, causal, scale, o.t)
    want, _, size = co.cache_attention(*host[:3], lens, scale, causal=bool(causal), kp=host[3], vp=host[4])
    close(o.t, want, bound(host, want, size, dtype, scale, P + S))
    o.check(), w.check()
    again = torch.full_like(o.t, NAN)
    run_prefix(dev, dl, dtype, causal, scale, again)
    assert torch.equal(again, o.t)
    assert area.area_kernel_error() == 0


# ---- accumulated weights ---------------------------------------------------------------------

CACHE = [
    # B, H, Hk, Nq, S, D, lens
    (1, 1, 1, 1, 1, 64, [1]),
    (3, 8, 2, 1, 513, 64, [513, 1, 0]),
    (2, 8, 8, 1, 300, 128, [300, 257]),
    (2, 16, 1, 1, 2000, 128, [2000, 129]),
    (2, 6, 2, 5, 777, 64, [777, 3]),
    (1, 4, 2, 33, 400, 128, [400]),
    (2, 4, 4, 130, 260, 64, [260, 129]),
    (1, 20, 1, 1, 150, 128, [140]),
    (3, 8, 2, 8, 700, 128, [700, 300, 5]),
    (1, 3, 1, 200, 1500, 64, [1400]),
    (2, 4, 2, 256, 300, 128, [300, 129]),
    (2, 24, 3, 70, 2000, 128, [2000, 1111]),
    (1, 2, 2, 300, 300, 64, [300]),
    (2, 18, 1, 1, 4100, 64, [4100, 0]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S,D,lens", CACHE)
def test_cache_attention_and_weights(B, H, Hk, Nq, S, D, lens, dtype):
    dev, host, dl = make(7, dtype, B, H, Hk, Nq, S, D, lens)
    scale = D ** -0.5
    o = Guarded((B, H, Nq, D), TYPES[dtype][0], NAN)
    acco = Guarded((B, Hk, S), torch.float32, NAN)
    acc = torch.rand(B, Hk, S, generator=torch.Generator().manual_seed(8)).cuda()
    w = run_cache(dev, dl, dtype, scale, acc, o.t, acco.t)
    want, got, size = co.cache_attention(*host[:3], lens, scale)
    close(o.t, want, bound(host, want, size, dtype, scale, S))
    o.check(), w.check(), acco.check()
    # a weight is off by 4 d + 2^-20 relative (see above; d is at most this), the sums by one step per addition
    q, k = host[0], np.nan_to_num(host[1])
    d = D * 2.0 ** -24 * scale * np.abs(q).max() * np.abs(k).max() * D
    rows = H // Hk * Nq
    sums = acc.double().cpu().numpy() + got
    close(acco.t, sums, got * (4 * d + 2.0 ** -20) + (rows + 2) * 2.0 ** -24 * sums)
    # null counts as zeros, and the sums may be updated in place
    zero, inplace = torch.full_like(acc, NAN), acc.clone()
    run_cache(dev, dl, dtype, scale, None, o.t, zero)
    run_cache(dev, dl, dtype, scale, inplace, o.t, inplace)
    close(zero, got, got * (4 * d + 2.0 ** -20 + (rows + 2) * 2.0 ** -24))
    assert torch.equal(inplace, acco.t)
    assert area.area_kernel_error() == 0


# ---- eviction --------------------------------------------------------------------------------

EVICT = [
    # B, Hk, S, So, D, budget, sinks, recent, lens, weights
    (1, 1, 1, 1, 64, 1, 0, 0, [1], "plain"),
    (2, 2, 600, 250, 64, 250, 4, 64, [600, 251], "plain"),
    (3, 1, 1500, 1500, 128, 700, 0, 0, [1500, 700, 701], "plain"),
    (2, 3, 1025, 64, 128, 33, 1, 32, [1025, 0], "plain"),
    (1, 2, 3000, 2000, 64, 1999, 64, 1000, [2999], "ties"),
    (1, 2, 3000, 100, 64, 99, 0, 10, [3000], "all equal"),
    (1, 2, 2500, 600, 128, 600, 3, 7, [2500], "odd"),
    (1, 1, 40, 40, 64, 10, 10, 0, [40], "plain"),
    (1, 1, 40, 40, 64, 10, 0, 10, [40], "plain"),
    (1, 1, 5000, 6000, 64, 4000, 5, 1, [5000], "ties"),
    (2, 2, 20000, 9000, 64, 8999, 4, 500, [20000, 15001], "ties"),
    (1, 1, 70001, 3001, 64, 3000, 4, 500, [70001], "plain"),
]


def weights_of(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(shape, generator=g)
    if kind == "ties":
        return torch.floor(u * 50) / 8
    if kind == "all equal":
        return torch.full(shape, 0.25)
    if kind == "odd":
        u[..., ::7], u[..., 1::9], u[..., 2::11] = NAN, float("inf"), -float("inf")
        u[..., 3::5], u[..., 4::5] = 0.0, -0.0
        u[..., 6::13] = -u[..., 6::13]
        u[..., 10::17] = 1e-42
    return u


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,S,So,D,budget,sinks,recent,lens,kind", EVICT)
def test_eviction(B, Hk, S, So, D, budget, sinks, recent, lens, kind, dtype, in_place):
    if in_place:
        So = S = max(S, budget)
    t = TYPES[dtype][0]
    g = torch.Generator().manual_seed(11)
    k, v = (Guarded((B, Hk, S, D), t) for _ in range(2))
    acc = Guarded((B, Hk, S), torch.float32)
    k.t.copy_(torch.randn(B, Hk, S, D, generator=g)), v.t.copy_(torch.randn(B, Hk, S, D, generator=g))
    acc.t.copy_(weights_of(kind, (B, Hk, S), 12))
    k0, v0, a0 = (x.t.cpu().clone() for x in (k, v, acc))
    ko, vo = (k, v) if in_place else (Guarded((B, Hk, So, D), t, 5.0) for _ in range(2))
    acco = acc if in_place else Guarded((B, Hk, So), torch.float32, NAN)
    lenso, idx = Guarded((B,), torch.int32, -7), Guarded((B, Hk, So), torch.int32, -7)
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    area.area_cache_evict(k.t, v.t, acc.t, dl, ko.t, vo.t, acco.t, lenso.t, idx.t, B, Hk, S, So, D,
                          budget, sinks, recent, TYPES[dtype][1])
    torch.cuda.synchronize()
    for x in (k, v, acc, ko, vo, acco, lenso, idx):
        x.check()
    assert lenso.t.tolist() == [min(n, budget) for n in lens]
    gi, gk, gv, ga = (x.t.cpu() for x in (idx, ko, vo, acco))
    for b, n in enumerate(lens):
        for h in range(Hk):
            keep = co.kept_tokens(a0[b, h].tolist(), n, budget, sinks, recent)
            m = len(keep)
            assert gi[b, h, :m].tolist() == keep and (gi[b, h, m:] == -1).all()
            same = lambda x, y: torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))  # noqa: E731
            assert same(gk[b, h, :m], k0[b, h, keep]) and same(gv[b, h, :m], v0[b, h, keep])
            assert same(ga[b, h, :m], a0[b, h, keep]) and (ga[b, h, m:] == 0).all()
            if in_place:
                assert same(gk[b, h, m:], k0[b, h, m:]) and same(gv[b, h, m:], v0[b, h, m:])
            else:
                assert (gk[b, h, m:] == 5).all() and (gv[b, h, m:] == 5).all()


def test_eviction_without_lengths():
    B, Hk, S, D = 2, 2, 300, 64
    k = torch.randn(B, Hk, S, D, device="cuda")
    acc = torch.rand(B, Hk, S, device="cuda")
    out = []
    for lens in (None, torch.full((B,), S, dtype=torch.int32, device="cuda"),
                 torch.full((B,), INT_MAX, dtype=torch.int32, device="cuda")):
        ko, vo = torch.zeros(B, Hk, 100, D, device="cuda"), torch.zeros(B, Hk, 100, D, device="cuda")
        acco, idx = torch.zeros(B, Hk, 100, device="cuda"), torch.zeros(B, Hk, 100, dtype=torch.int32, device="cuda")
        lenso = torch.zeros(B, dtype=torch.int32, device="cuda")
        area.area_cache_evict(k, k.clone(), acc, lens, ko, vo, acco, lenso, idx, B, Hk, S, 100, D, 100, 4, 20,
                              area.AREA_DTYPE_F32)
        out.append((ko, acco, idx, lenso))
    for o in out[1:]:
        assert all(torch.equal(x, y) for x, y in zip(out[0], o))


@pytest.mark.parametrize("S,B,Hk", [(600, 40, 16), (300, 5, 60), (1500, 40, 16), (5000, 9, 16)])
def test_eviction_of_many_heads(S, B, Hk):
    """As many key heads as fill the GPU, so that fewer blocks share one."""
    D, budget, sinks, recent = 64, S // 3, 4, S // 9
    t, dt, _ = TYPES["bf16"]
    g = torch.Generator().manual_seed(51)
    k, v = (torch.randn(B, Hk, S, D, generator=g).to(t).cuda() for _ in range(2))
    acc = weights_of("ties", (B, Hk, S), 52).cuda()
    lens = [S - (i * 37) % S for i in range(B)]
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    ko, vo = (torch.zeros(B, Hk, budget, D, dtype=t, device="cuda") for _ in range(2))
    acco = torch.full((B, Hk, budget), NAN, device="cuda")
    lenso, idx = torch.zeros_like(dl), torch.zeros(B, Hk, budget, dtype=torch.int32, device="cuda")
    area.area_cache_evict(k, v, acc, dl, ko, vo, acco, lenso, idx, B, Hk, S, budget, D, budget, sinks, recent, dt)
    assert lenso.tolist() == [min(n, budget) for n in lens]
    gi, host = idx.cpu(), acc.cpu()
    for b, n in enumerate(lens):
        for h in range(0, Hk, 7):
            keep = co.kept_tokens(host[b, h].tolist(), n, budget, sinks, recent)
            assert gi[b, h, :len(keep)].tolist() == keep and (gi[b, h, len(keep):] == -1).all()
    had = idx >= 0
    src = torch.where(had, idx, 0).long()
    for x, y in ((k, ko), (v, vo)):
        rows = x.gather(2, src[..., None].expand(-1, -1, -1, D))
        assert torch.equal(torch.where(had[..., None], rows, 0), y)
    assert torch.equal(torch.where(had, acc.gather(2, src), 0.0), acco)


# ---- more sequences than run at once -----------------------------------------------------------

def uneven(B, S):
    """Lengths in no order, zeros, ones, equal ones and full ones among them."""
    return [(i * i * 131 + 7 * i) % (S + 1) if i % 9 else (0, 1, S, S)[i // 9 % 4] for i in range(B)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S,D", [(70, 16, 8, 1, 300, 64), (128, 8, 4, 1, 131, 128), (129, 8, 4, 2, 70, 64),
                                           (2, 240, 240, 1, 200, 64)])
def test_many_sequences_of_uneven_lengths(B, H, Hk, Nq, S, D, dtype):
    """The longest sequences' blocks start first: every call against the oracle."""
    lens = uneven(B, S)
    P = 33
    dev, host, dl = make(61, dtype, B, H, Hk, Nq, S, D, lens, P=P)
    scale = D ** -0.5
    o = Guarded((B, H, Nq, D), TYPES[dtype][0], NAN)
    run_sink(dev, dl, dtype, INT_MAX, 0, scale, o.t)
    want, got, size = co.cache_attention(*host[:3], lens, scale)
    close(o.t, want, bound(host, want, size, dtype, scale, S))
    acc = torch.rand(B, Hk, S, generator=torch.Generator().manual_seed(62)).cuda()
    acco = Guarded((B, Hk, S), torch.float32, NAN)
    w = run_cache(dev, dl, dtype, scale, acc, o.t, acco.t)
    close(o.t, want, bound(host, want, size, dtype, scale, S))
    # as in test_cache_attention_and_weights
    d = D * 2.0 ** -24 * scale * np.abs(host[0]).max() * np.nan_to_num(np.abs(host[1])).max() * D
    sums = acc.double().cpu().numpy() + got
    close(acco.t, sums, got * (4 * d + 2.0 ** -20) + (H // Hk * Nq + 2) * 2.0 ** -24 * sums)
    run_prefix(dev, dl, dtype, 1, scale, o.t)
    want, _, size = co.cache_attention(*host[:3], lens, scale, kp=host[3], vp=host[4])
    close(o.t, want, bound(host, want, size, dtype, scale, P + S))
    o.check(), acco.check(), w.check()
    assert area.area_kernel_error() == 0


# ---- as many rows as the kernels for many rows are for ---------------------------------------

MANY = [
    # B, H, Hk, Nq, S, D, window, sinks, P, lens
    (1, 64, 64, 130, 200, 64, 40, 5, 300, [200]),
    (2, 40, 20, 257, 300, 128, 100, 7, 1, [300, 129]),
    (1, 96, 32, 129, 129, 64, INT_MAX, 0, 65, [129]),
    (3, 96, 32, 70, 150, 128, 33, 70, 140, [150, 69, 3]),
    (1, 80, 80, 300, 420, 64, 256, 129, 128, [411]),
    (2, 64, 64, 128, 128, 128, 1, 0, 31, [128, 0]),
    # few queries on a long cache: the rows of a key head's heads share row tiles
    (2, 8, 2, 130, 3000, 64, INT_MAX, 0, 500, [3000, 135]),
    (1, 6, 1, 300, 2500, 128, 2499, 1, 64, [2100]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S,D,window,sinks,P,lens", MANY)
def test_many_heads_of_many_rows(B, H, Hk, Nq, S, D, window, sinks, P, lens, dtype):
    dev, host, dl = make(81, dtype, B, H, Hk, Nq, S, D, lens, P=P)
    scale = D ** -0.5
    o = Guarded((B, H, Nq, D), TYPES[dtype][0], NAN)
    w = run_sink(dev, dl, dtype, window, sinks, scale, o.t)
    want, _, size = co.cache_attention(*host[:3], lens, scale, window=window, sinks=sinks)
    close(o.t, want, bound(host, want, size, dtype, scale, S))
    w.check()
    for causal in (0, 1):
        w = run_prefix(dev, dl, dtype, causal, scale, o.t.fill_(NAN))
        want, _, size = co.cache_attention(*host[:3], lens, scale, causal=bool(causal), kp=host[3], vp=host[4])
        close(o.t, want, bound(host, want, size, dtype, scale, P + S))
        w.check()
    o.check()
    assert area.area_kernel_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S,D", [(20, 12, 1, 1, 130, 64), (3, 48, 4, 2, 300, 128), (2, 16, 1, 1, 9001, 64),
                                           (40, 24, 2, 1, 60, 128)])
def test_weights_of_twelve_to_24_rows(B, H, Hk, Nq, S, D, dtype):
    """Either kernel, as the sizes have it."""
    lens = uneven(B, S)
    dev, host, dl = make(82, dtype, B, H, Hk, Nq, S, D, lens)
    o, acco = Guarded((B, H, Nq, D), TYPES[dtype][0], NAN), Guarded((B, Hk, S), torch.float32, NAN)
    scale = D ** -0.5
    w = run_cache(dev, dl, dtype, scale, None, o.t, acco.t)
    want, got, size = co.cache_attention(*host[:3], lens, scale)
    close(o.t, want, bound(host, want, size, dtype, scale, S))
    # as in test_cache_attention_and_weights
    d = D * 2.0 ** -24 * scale * np.abs(host[0]).max() * np.nan_to_num(np.abs(host[1])).max() * D
    close(acco.t, got, got * (4 * d + 2.0 ** -20 + (H // Hk * Nq + 2) * 2.0 ** -24))
    o.check(), acco.check(), w.check()


# ---- together, on streams and in graphs -------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_cache_is_filled_read_and_evicted(dtype):
    """A prompt, then single tokens whose weights add up, an eviction in place
    when the cache is full, more tokens: every output and every choice against
    the oracle run beside it."""
    B, H, Hk, S, D, prompt, budget = 2, 8, 2, 160, 64, 140, 90
    t, dt, _ = TYPES[dtype]
    scale = D ** -0.5
    g = torch.Generator().manual_seed(21)
    lens = [prompt, prompt - 30]
    dev, host, dl = make(22, dtype, B, H, Hk, prompt, S, D, lens)
    o = torch.full_like(dev[0], NAN)
    run_sink(dev, dl, dtype, INT_MAX, 0, scale, o)
    want, _, size = co.cache_attention(*host[:3], lens, scale)
    close(o, want, bound(host, want, size, dtype, scale, S))
    k, v, hk, hv = dev[1], dev[2], host[1], host[2]
    acc, hacc = torch.zeros(B, Hk, S, device="cuda"), np.zeros((B, Hk, S))
    lenso, idx = torch.zeros_like(dl), torch.zeros(B, Hk, S, dtype=torch.int32, device="cuda")
    for step in range(40):
        q1 = (torch.randn(B, H, 1, D, generator=g) * 1.5).to(t)
        for x, hx in ((k, hk), (v, hv)):
            new = torch.randn(B, Hk, D, generator=g).to(t)
            for b in range(B):
                x[b, :, lens[b]] = new[b].cuda()
                hx[b, :, lens[b]] = new[b].double().numpy()
        lens = [n + 1 for n in lens]
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        o1 = torch.full((B, H, 1, D), NAN, dtype=t, device="cuda")
        run_cache((q1.cuda(), k, v, None, None), dl, dtype, scale, acc, o1, acc)
        h1 = [q1.double().numpy(), hk, hv, host[3], host[4]]
        want, got, size = co.cache_attention(*h1[:3], lens, scale)
        close(o1, want, bound(h1, want, size, dtype, scale, S))
        hacc += got
        assert np.abs(acc.cpu().numpy() - hacc).max() < 1e-4
        if max(lens) == S:
            have = acc.cpu().numpy()
            area.area_cache_evict(k, v, acc, dl, k, v, acc, lenso, idx, B, Hk, S, S, D, budget, 4, 30, dt)
            for b in range(B):
                for h in range(Hk):
                    keep = co.kept_tokens(have[b, h], lens[b], budget, 4, 30)
                    m = len(keep)
                    assert idx[b, h, :m].tolist() == keep
                    hk[b, h, :m], hv[b, h, :m] = hk[b, h, keep].copy(), hv[b, h, keep].copy()
                    hacc[b, h, :m], hacc[b, h, m:] = hacc[b, h, keep].copy(), 0
            lens = [min(n, budget) for n in lens]
            assert lenso.tolist() == lens


def test_replayed_graphs_and_other_streams_give_the_same():
    """A prompt's and a token's calls captured together: replays follow the
    inputs and the lengths that lie in the buffers, two graphs with workspaces
    of their own run at once."""
    B, H, Hk, S, D, P = 3, 8, 2, 900, 128, 400
    cases = []
    for seed in (31, 32):
        dev, host, dl = make(seed, "bf16", B, H, Hk, 1, S, D, [900, 450, 70], P=P, poison=False)
        cases.append((dev, dl))
    acc = [torch.rand(B, Hk, S, device="cuda") for _ in cases]
    outs = [[torch.full_like(c[0][0], NAN) for _ in range(3)] + [torch.full_like(a, NAN)]
            for c, a in zip(cases, acc)]
    wss = [[workspace(1 << 24) for _ in range(3)] for _ in cases]

    def step(c, a, o, w, s):
        run_sink(c[0], c[1], "bf16", 200, 4, 0.1, o[0], s, w[0])
        run_prefix(c[0], c[1], "bf16", 1, 0.1, o[1], s, w[1])
        run_cache(c[0], c[1], "bf16", 0.1, a, o[2], o[3], s, w[2])

    eager = []
    for lens in ([900, 450, 70], [64, 0, 129]):
        for c, a, o, w in zip(cases, acc, outs, wss):
            c[1].copy_(torch.tensor(lens, dtype=torch.int32))
            step(c, a, o, w, None)
        torch.cuda.synchronize()
        eager.append([[x.clone() for x in o] for o in outs])
    graphs, streams = [], [torch.cuda.Stream() for _ in cases]
    for c, a, o, w, s in zip(cases, acc, outs, wss, streams):
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            step(c, a, o, w, torch.cuda.current_stream())
        graphs.append(g)
    for lens, want in zip(([900, 450, 70], [64, 0, 129]), eager):
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            c[1].copy_(torch.tensor(lens, dtype=torch.int32))
            for x in o:
                x.fill_(NAN)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(o, e))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_replayed_graphs_of_prompts_and_of_an_eviction(dtype):
    """Calls of several launches, captured one after the other without a wait
    between them: replays follow the inputs, and two replays back to back leave
    what an eager run leaves."""
    B, H, Hk, S, D, Nq, P, budget = 2, 6, 2, 1500, 128, 70, 300, 600
    dt = TYPES[dtype][1]
    dev, _, dl = make(71, dtype, B, H, Hk, Nq, S, D, [1500, 1111], P=P, poison=False)
    acc = torch.rand(B, Hk, S, device="cuda")
    o = [torch.full_like(dev[0], NAN) for _ in range(3)]
    acco = torch.full_like(acc, NAN)
    ko, vo = (torch.zeros(B, Hk, budget, D, dtype=dev[1].dtype, device="cuda") for _ in range(2))
    small, idx = torch.zeros(B, Hk, budget, device="cuda"), torch.zeros(B, Hk, budget, dtype=torch.int32, device="cuda")
    lenso = torch.zeros_like(dl)
    ws = [workspace(1 << 26) for _ in range(3)]
    outs = [*o, acco, ko, vo, small, idx, lenso]

    def step(s):
        run_sink(dev, dl, dtype, INT_MAX, 0, 0.1, o[0], s, ws[0])
        run_prefix(dev, dl, dtype, 1, 0.1, o[1], s, ws[1])
        run_cache(dev, dl, dtype, 0.1, acc, o[2], acco, s, ws[2])
        area.area_cache_evict(dev[1], dev[2], acco, dl, ko, vo, small, lenso, idx, B, Hk, S, budget, D, budget, 4, 99,
                              dt, s)

    stream = torch.cuda.Stream()
    step(None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step(torch.cuda.current_stream())
    for lens in ([1500, 1111], [70, 601], [3, 0]):
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        dev[0].mul_(-0.9)
        step(None)
        torch.cuda.synchronize()
        want = [x.clone() for x in outs]
        for x in outs[:4]:
            x.fill_(NAN)
        idx.fill_(5)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            g.replay()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
    assert area.area_kernel_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S,D", [(3, 8, 2, 5, 90, 64), (2, 8, 2, 40, 700, 128), (2, 48, 48, 200, 300, 64)])
def test_queries_before_the_first_token_may_hold_anything(B, H, Hk, Nq, S, D, dtype):
    """Padding in front is NaN: rows of zeros, and nothing of it in the others or in the weights."""
    lens = [S, Nq // 2, 1][:B]
    dev, host, dl = make(91, dtype, B, H, Hk, Nq, S, D, lens, P=50)
    for b, n in enumerate(lens):
        dev[0][b, :, :max(0, Nq - n)] = NAN
    o, acco = Guarded((B, H, Nq, D), TYPES[dtype][0], NAN), Guarded((B, Hk, S), torch.float32, NAN)
    for run, kw in ((lambda: run_sink(dev, dl, dtype, 30, 2, 0.1, o.t), dict(window=30, sinks=2)),
                    (lambda: run_prefix(dev, dl, dtype, 1, 0.1, o.t), dict(kp=host[3], vp=host[4])),
                    (lambda: run_cache(dev, dl, dtype, 0.1, None, o.t, acco.t), {})):
        run()
        want, got, size = co.cache_attention(*host[:3], lens, 0.1, **kw)
        close(o.t, want, bound(host, want, size, dtype, 0.1, S + 50))
        for b, n in enumerate(lens):
            assert (o.t[b, :, :max(0, Nq - n)] == 0).all()
    # as in test_cache_attention_and_weights
    d = D * 2.0 ** -24 * 0.1 * np.abs(host[0]).max() * np.nan_to_num(np.abs(host[1])).max() * D
    close(acco.t, got, got * (4 * d + 2.0 ** -20 + (H // Hk * Nq + 2) * 2.0 ** -24))
    o.check(), acco.check()


def test_without_own_keys_lengths_are_not_read():
    B, H, P, D = 3, 4, 2000, 64
    dev, host, _ = make(72, "bf16", B, H, H, 1, 0, D, [0, 0, 0], P=P)
    o = torch.full_like(dev[0], NAN)
    run_prefix(dev, 16, "bf16", 0, 0.1, o)          # an address that holds nothing
    want, _, size = co.cache_attention(*host[:3], [0] * B, 0.1, causal=False, kp=host[3], vp=host[4])
    close(o, want, bound(host, want, size, "bf16", 0.1, P))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S,D", [(2, 4, 2, 5, 2, 64), (1, 4, 2, 33, 7, 128), (2, 2, 1, 300, 40, 64)])
def test_more_queries_than_the_cache_has_room(B, H, Hk, Nq, S, D, dtype):
    """Queries before the first token get rows of zeros, in every call."""
    lens = [S, S // 2][:B]
    dev, host, dl = make(73, dtype, B, H, Hk, Nq, S, D, lens, P=9)
    for run, kw in ((lambda o: run_sink(dev, dl, dtype, 3, 1, 0.1, o), dict(window=3, sinks=1)),
                    (lambda o: run_prefix(dev, dl, dtype, 1, 0.1, o), dict(kp=host[3], vp=host[4])),
                    (lambda o: run_cache(dev, dl, dtype, 0.1, None, o, torch.zeros(B, Hk, S, device="cuda")), {})):
        o = Guarded((B, H, Nq, D), TYPES[dtype][0], NAN)
        run(o.t)
        want, _, size = co.cache_attention(*host[:3], lens, 0.1, **kw)
        close(o.t, want, bound(host, want, size, dtype, 0.1, S + 9))
        o.check()


def test_long_cache_offsets_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 values per tensor: the last
    sequence's rows lie past both."""
    B, H, Hk, S, D = 3, 2, 2, 2_900_000, 128
    k = torch.zeros(B, Hk, S, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 2 ** 31
    n, tail = S - 5, 300
    g = torch.Generator().manual_seed(41)
    q = torch.randn(B, H, 1, D, generator=g).bfloat16()
    kt, vt = (torch.randn(B, Hk, tail, D, generator=g).bfloat16() for _ in range(2))
    k[:, :, n - tail:n], v[:, :, n - tail:n] = kt.cuda(), vt.cuda()
    lens = torch.full((B,), n, dtype=torch.int32).cuda()
    o = torch.full((B, H, 1, D), NAN, dtype=torch.bfloat16, device="cuda")
    run_sink((q.cuda(), k, v, None, None), lens, "bf16", tail, 0, 0.1, o)
    host = [x.double().numpy() for x in (q, kt, vt)] + [np.zeros((Hk, 0, D))] * 2
    want, _, size = co.cache_attention(*host[:3], [tail] * B, 0.1)
    close(o, want, bound(host, want, size, "bf16", 0.1, tail))


@pytest.mark.parametrize("B,H,Hk,Nq,S,D,P,lens", [
    # runs of sequences without a token: several units of a block in a row have no tile
    (64, 16, 16, 130, 260, 64, 0, [0] * 20 + [260] + [0] * 20 + [131, 1] + [0] * 21),
    (60, 24, 24, 129, 200, 128, 65, [0] * 30 + [200, 3] + [0] * 28),
    # splits of a long cache that holds few tokens
    (2, 2, 1, 70, 30000, 64, 0, [90, 0]),
])
def test_units_without_tiles_in_fp32(B, H, Hk, Nq, S, D, P, lens):
    dev, host, dl = make(101, "f32", B, H, Hk, Nq, S, D, lens, P=P)
    scale = D ** -0.5
    o = Guarded((B, H, Nq, D), torch.float32, NAN)
    some = [b for b in range(B) if lens[b] > 0]
    none = [b for b in range(B) if lens[b] == 0]
    top = max(lens)                            # (the oracle does without the cache's empty end)
    few = [host[0][some], host[1][some][:, :, :top], host[2][some][:, :, :top], host[3], host[4]]
    runs = [(lambda: run_sink(dev, dl, "f32", 100, 2, scale, o.t), dict(window=100, sinks=2))]
    if P:
        runs.append((lambda: run_prefix(dev, dl, "f32", 1, scale, o.t), dict(kp=host[3], vp=host[4])))
    for run, kw in runs:
        o.t.fill_(NAN)
        run()
        want, _, size = co.cache_attention(*few[:3], [lens[b] for b in some], scale, **kw)
        close(o.t[some], want, bound(few, want, size, "f32", scale, top + P))
        assert (o.t[none] == 0).all()
        o.check()
    assert area.area_kernel_error() == 0


# ---- fp32 is held to fp32: a bound that inputs of 16 significand bits leave (cache_bounds.py) ----

def fp32_case(case):
    B, H, Hk, Nq, P, S, D, window, sinks, lens = case
    x = cb.inputs(111, B, H, Hk, Nq, P, S, D)
    return x, [torch.from_numpy(y).cuda() for y in x], torch.tensor(lens, dtype=torch.int32).cuda()


@pytest.mark.parametrize("case", cb.SINK)
def test_fp32_window_attention_keeps_fp32(case):
    B, H, Hk, Nq, P, S, D, window, sinks, lens = case
    x, dev, dl = fp32_case(case)
    o = torch.full_like(dev[0], NAN)
    run_sink(dev, dl, "f32", window, sinks, cb.SCALE, o)
    want, tol, _, _ = cb.call(*x[:3], lens, cb.SCALE, lambda n: co.visible(n, Nq, S, window, sinks))
    close(o, want, tol)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("case", cb.PREFIX)
def test_fp32_prefix_attention_keeps_fp32(case, causal):
    B, H, Hk, Nq, P, S, D, window, sinks, lens = case
    x, dev, dl = fp32_case(case)
    o = torch.full_like(dev[0], NAN)
    run_prefix(dev, dl, "f32", causal, cb.SCALE, o)
    want, tol, _, _ = cb.call(*x[:3], lens, cb.SCALE, lambda n: co.visible(n, Nq, S, causal=bool(causal)),
                              kp=x[3], vp=x[4], causal=bool(causal))
    close(o, want, tol)


@pytest.mark.parametrize("case", cb.CACHE)
def test_fp32_weights_keep_fp32(case):
    B, H, Hk, Nq, P, S, D, window, sinks, lens = case
    x, dev, dl = fp32_case(case)
    o, acco = torch.full_like(dev[0], NAN), torch.full((B, Hk, S), NAN, device="cuda")
    run_cache(dev, dl, "f32", cb.SCALE, None, o, acco)
    want, tol, got, wtol = cb.call(*x[:3], lens, cb.SCALE, lambda n: co.visible(n, Nq, S))
    close(o, want, tol)
    close(acco, got, wtol)


# ---- infinities, and scores as large as they get ----------------------------------------------

@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), 3.3e38])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S", [(2, 4, 2, 1, 600), (2, 64, 64, 200, 600), (2, 8, 1, 3, 600)])
def test_infinities_where_nobody_looks(B, H, Hk, Nq, S, dtype, bad):
    """Behind the last token and between the sinks and the first window, in keys and in values."""
    D, window, sinks, lens = 64, 70, 3, [S, 400]
    dev, host, dl = make(121, dtype, B, H, Hk, Nq, S, D, lens)
    want, got = (torch.full_like(dev[0], NAN) for _ in range(2))
    run_sink(dev, dl, dtype, window, sinks, 0.125, want)
    for x in dev[1:3]:
        for b, n in enumerate(lens):
            x[b, :, n:] = bad
            x[b, :, sinks:n - Nq + 1 - window] = bad
    run_sink(dev, dl, dtype, window, sinks, 0.125, got)
    assert torch.equal(want, got) and torch.isfinite(got).all()


@pytest.mark.parametrize("bad", [float("inf"), NAN])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S", [(2, 4, 2, 1, 300), (2, 64, 32, 150, 300)])
def test_what_is_seen_and_not_finite_stays_with_its_key_head(B, H, Hk, Nq, S, dtype, which, bad):
    D, lens = 64, [S, S]
    dev, host, dl = make(122, dtype, B, H, Hk, Nq, S, D, lens)
    want, got = (torch.full_like(dev[0], NAN) for _ in range(2))
    zero, acco = (torch.full((B, Hk, S), NAN, device="cuda") for _ in range(2))
    run_cache(dev, dl, dtype, 0.125, None, want, zero)
    dev[1 if which == "k" else 2][1, Hk - 1, S - Nq, 5] = bad         # the first query's own token
    run_cache(dev, dl, dtype, 0.125, None, got, acco)
    G = H // Hk
    mine = torch.zeros(B, H, dtype=torch.bool)
    mine[1, H - G:] = True
    assert torch.equal(got[~mine], want[~mine])
    assert torch.equal(acco.view(-1, S)[:-1], zero.view(-1, S)[:-1])
    if which == "v":                            # it shows in its column for every row that gives it weight
        assert not torch.isfinite(got[mine][:, 0, 5]).any()
        assert torch.equal(acco, zero)


@pytest.mark.parametrize("size", [1e3, 1e6, 1e9, 2e38])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,Nq,S", [(1, 4, 2, 1, 500), (1, 64, 64, 300, 500), (2, 6, 2, 8, 5000)])
def test_scores_of_any_size(B, H, Hk, Nq, S, dtype, size):
    """One key of a score of +size, all others 0 or -size: the row is its value; without it, with
    scores of 0 and -size, the mean of the values that have 0."""
    D = 64
    t = TYPES[dtype][0]
    lens = [S] * B
    dev, host, dl = make(123, dtype, B, H, Hk, Nq, S, D, lens)
    q, k, v = dev[:3]
    q.zero_(), k.zero_()
    q[..., 7] = 1.0
    big = float(torch.tensor(size, dtype=torch.bfloat16))
    top = S - Nq // 2 - 1                       # seen by the later half of the rows
    k[:, :, 1::3, 7] = -big
    k[:, :, top] = 0
    k[:, :, top, 7] = big
    o = torch.full_like(q, NAN)
    run_sink(dev, dl, dtype, INT_MAX, 0, 1.0, o)
    pos = torch.arange(S - Nq, S, device="cuda")
    sees = pos >= top
    want = v[:, :, top].repeat_interleave(H // Hk, 1)[:, :, None].expand_as(o)
    # one weight is all there is, but it need not be 1: the kernels for many rows take 2^(s a - M) in one
    # step, M the rounded product of score and scale, which is 2^c with |c| <= 2^-24 M; bf16 rounds it to
    # 8 bits for the product with the value, and divides by what it was: 2^-8; fp32 divides by the same
    # value, with rounding errors of the product, the quotient and the result, under 2^-20
    off = (2.0 ** -8 if dtype == "bf16" else 0) + 2.0 ** -20 + TYPES[dtype][2]
    assert sees.any()
    close(o[:, :, sees], want[:, :, sees].double().cpu().numpy(), off * want[:, :, sees].double().abs().cpu().numpy())
    at = torch.arange(S, device="cuda")
    zero = ((at % 3 != 1)[None, :] & (at[None, :] <= pos[:, None]) & (at != top)[None, :]).double()
    mean = torch.einsum("ij,bhjd->bhid", zero / zero.sum(1, keepdim=True), v.double()).repeat_interleave(H // Hk, 1)
    # exact weights of one: the sum's rounding and the result's, and bf16 weights of one are exact
    size_ = torch.einsum("ij,bhjd->bhid", zero / zero.sum(1, keepdim=True), v.double().abs()).repeat_interleave(H // Hk, 1)
    tol = (2.0 ** -20 + 8 * math.sqrt(S) * 2.0 ** -24) * size_ + TYPES[dtype][2] * mean.abs() + 1e-30
    if (~sees).any():
        close(o[:, :, ~sees], mean[:, :, ~sees].cpu().numpy(), tol[:, :, ~sees].cpu().numpy())
    assert area.area_kernel_error() == 0


# ---- many rows and evictions past 2^31 values, evictions in replayed graphs ----------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_on_a_long_cache_past_32_bits(dtype):
    """The kernels for many rows and their weights on more than 2^31 values per tensor: the last
    head's rows lie past that.  All keys but the last 300 have a score 40 below theirs at least, so
    that their part of a row is under S e^-32."""
    B, H, Hk, Nq, S, D = 3, 2, 2, 200, 2_900_000, 128
    t = TYPES[dtype][0]
    n, tail, scale = S - 5, 300, 0.5
    g = torch.Generator().manual_seed(131)
    q = torch.randn(B, H, Nq, D, generator=g) * 0.2
    kt, vt = torch.randn(B, Hk, tail, D, generator=g) * 0.2, torch.randn(B, Hk, tail, D, generator=g)
    q[..., 0], kt[..., 0] = 10.0, 10.0                 # scores of 50, give or take 10 sd of 0.23
    q, kt, vt = (x.to(t) for x in (q, kt, vt))
    k = torch.zeros(B, Hk, S, D, dtype=t, device="cuda")
    assert k.numel() > 2 ** 31
    v = torch.zeros_like(k)
    k[:, :, n - tail:n], v[:, :, n - tail:n] = kt.cuda(), vt.cuda()
    lens = torch.full((B,), n, dtype=torch.int32).cuda()
    host = [x.double().numpy() for x in (q, kt, vt)] + [np.zeros((Hk, 0, D))] * 2
    dq, rest = q.cuda(), S * math.exp(-32)
    o = torch.full((B, H, Nq, D), NAN, dtype=t, device="cuda")
    run_sink((dq, k, v, None, None), lens, dtype, 128, 0, scale, o)
    want, _, size = co.cache_attention(*host[:3], [tail] * B, scale, window=128)
    # (q k is a sum of one large product and small ones: the docstring's bound takes all as large)
    close(o, want, bound(host, want, size, dtype, scale, tail))
    acco = torch.full((B, Hk, S), NAN, device="cuda")
    run_cache((dq, k, v, None, None), lens, dtype, scale, None, o.fill_(NAN), acco)
    want, got, size = co.cache_attention(*host[:3], [tail] * B, scale)
    close(o, want, bound(host, want, size, dtype, scale, tail) + rest * (size + np.abs(want)))
    have = acco[:, :, n - tail:n].double().cpu().numpy()
    d = D * 2.0 ** -24 * scale * 11.0 * 11.0 * D       # as in test_cache_attention_and_weights
    assert (np.abs(have - got) <= got * (4 * d + 2.0 ** -20 + (H // Hk * Nq + 2) * 2.0 ** -24) + rest * Nq).all()
    assert (acco[:, :, n:] == 0).all() and acco[:, :, :n - tail].max() <= Nq * math.exp(-32)
    assert area.area_kernel_error() == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_eviction_past_32_bits(in_place):
    B, Hk, S, D, budget, sinks, recent = 3, 2, 2_900_000, 128, 5000, 4, 1000
    g = torch.Generator(device="cuda").manual_seed(141)
    k = torch.empty(B, Hk, S, D, dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 2 ** 31
    # a token's row says which it is, in four values of 7 bits and its head
    at = torch.arange(S, device="cuda", dtype=torch.int32)
    mark = torch.stack([at >> 21, at >> 14 & 127, at >> 7 & 127, at & 127], -1).bfloat16()
    k.zero_()
    for b in range(B):
        for h in range(Hk):
            k[b, h, :, D - 5:D - 1] = mark
            k[b, h, :, D - 1] = 1 + b * Hk + h
    v = -k
    acc = torch.rand(B, Hk, S, generator=g, device="cuda")
    lens = torch.tensor([S, S - 7, S - 100], dtype=torch.int32, device="cuda")
    a0 = acc.clone()
    So = S if in_place else budget
    ko, vo, acco = (k, v, acc) if in_place else (torch.zeros(B, Hk, So, D, dtype=k.dtype, device="cuda"),
                                                  torch.zeros(B, Hk, So, D, dtype=k.dtype, device="cuda"),
                                                  torch.full((B, Hk, So), NAN, device="cuda"))
    idx = torch.full((B, Hk, So), 7, dtype=torch.int32, device="cuda")
    lenso = torch.zeros_like(lens)
    area.area_cache_evict(k, v, acc, lens, ko, vo, acco, lenso, idx, B, Hk, S, So, D, budget, sinks, recent,
                          area.AREA_DTYPE_BF16)
    assert lenso.tolist() == [budget] * B
    for b, n in enumerate([S, S - 7, S - 100]):
        for h in range(Hk):
            free = a0[b, h, sinks:n - recent]
            best = torch.sort(free, descending=True, stable=True).indices[:budget - sinks - recent]
            keep = torch.cat([at[:sinks].long(), best.sort().values + sinks, at[n - recent:n].long()])
            assert torch.equal(idx[b, h, :budget].long(), keep) and (idx[b, h, budget:] == -1).all()
            assert torch.equal(acco[b, h, :budget], a0[b, h, keep]) and (acco[b, h, budget:] == 0).all()
            for x, sign in ((ko, 1), (vo, -1)):
                rows = x[b, h, :budget].float() * sign
                assert torch.equal(rows[:, D - 5:D - 1], mark[keep].float())
                assert (rows[:, D - 1] == 1 + b * Hk + h).all() and (rows[:, :D - 5] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [700, 5000])
def test_replayed_graphs_of_an_eviction_in_place(S, dtype):
    """Captured with the copies that fill the cache: replays follow the lengths and the weights."""
    B, Hk, D, budget, sinks, recent = 3, 4, 64, S // 2, 4, S // 8
    t, dt, _ = TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(151)
    k0, v0 = (torch.randn(B, Hk, S, D, generator=g, device="cuda").to(t) for _ in range(2))
    acc0 = torch.rand(B, Hk, S, generator=g, device="cuda")
    k, v, acc = k0.clone(), v0.clone(), acc0.clone()
    lens = torch.tensor([S, S - 1, 3], dtype=torch.int32, device="cuda")
    lenso, idx = torch.zeros_like(lens), torch.zeros(B, Hk, S, dtype=torch.int32, device="cuda")

    def step(s):
        k.copy_(k0), v.copy_(v0), acc.copy_(acc0)
        area.area_cache_evict(k, v, acc, lens, k, v, acc, lenso, idx, B, Hk, S, S, D, budget, sinks, recent, dt, s)

    step(None)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        step(torch.cuda.current_stream())
    for new in ([S, S - 1, 3], [budget, budget + 1, 0], [S // 3, S, S]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        acc0.copy_(torch.rand(B, Hk, S, generator=g, device="cuda"))
        step(None)
        torch.cuda.synchronize()
        want = [x.clone() for x in (k, v, acc, lenso, idx)]
        for x in (k, v, acc, lenso, idx):
            x.fill_(5)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((k, v, acc, lenso, idx), want))
        for b in range(B):
            keep = co.kept_tokens(acc0[b, 1].tolist(), new[b], budget, sinks, recent)
            assert idx[b, 1, :len(keep)].tolist() == keep
            assert torch.equal(k[b, 1, :len(keep)], k0[b, 1, keep])
