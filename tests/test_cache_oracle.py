"""Pins of the cache oracle, and the refusals of the cache calls (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def area():
    import os
    import step_adaptive_sparse_b200 as area
    from step_adaptive_sparse_b200 import binding
    if not os.path.exists(binding.LIB_PATH):
        from step_adaptive_sparse_b200.build import build
        build()
    area.library()
    return area


# ---- the oracle ----------------------------------------------------------------------------

def test_visible_by_hand():
    # five tokens, the last three are queries, window 2, one sink
    got = co.visible(5, 3, 6, window=2, sinks=1)
    assert got.astype(int).tolist() == [[1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0]]
    # two tokens, three queries: the first is padding and sees nothing
    assert co.visible(2, 3, 3).astype(int).tolist() == [[0, 0, 0], [1, 0, 0], [1, 1, 0]]
    assert co.visible(2, 2, 3, causal=False).astype(int).tolist() == [[1, 1, 0], [1, 1, 0]]


def test_oracle_equals_library_attention_in_64_bits():
    rng = np.random.default_rng(3)
    B, H, Hk, Nq, S, P, D = 2, 4, 2, 5, 9, 3, 8
    q, k, v = rng.normal(size=(B, H, Nq, D)), rng.normal(size=(B, Hk, S, D)), rng.normal(size=(B, Hk, S, D))
    kp, vp = rng.normal(size=(Hk, P, D)), rng.normal(size=(Hk, P, D))
    o, got, _ = co.cache_attention(q, k, v, [9, 9], 0.3, kp=kp, vp=vp)
    kk = np.concatenate([np.broadcast_to(kp, (B, Hk, P, D)), k], 2).repeat(2, 1)
    vv = np.concatenate([np.broadcast_to(vp, (B, Hk, P, D)), v], 2).repeat(2, 1)
    mask = torch.ones(Nq, P + S, dtype=torch.bool).tril(P + S - Nq)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q), torch.from_numpy(kk), torch.from_numpy(vv), attn_mask=mask, scale=0.3)
    assert np.abs(o - want.numpy()).max() < 1e-12
    # weights: what each row spends on the prefix is missing from its own keys' sums
    o2, got2, _ = co.cache_attention(q, k, v, [9, 9], 0.3)
    assert np.allclose(got2.sum(-1), 2 * Nq) and (got.sum(-1) < 2 * Nq).all()


def test_oracle_ignores_what_is_not_seen():
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(size=(1, 1, 2, 4)), rng.normal(size=(1, 1, 7, 4)), rng.normal(size=(1, 1, 7, 4))
    o, _, _ = co.cache_attention(q, k, v, [5], 1.0, window=2, sinks=1)
    k[:, :, 5:], v[:, :, 5:], k[:, :, 1:2], v[:, :, 1:2] = np.nan, np.inf, np.nan, -np.inf
    o2, _, _ = co.cache_attention(q, k, v, [5], 1.0, window=2, sinks=1)
    assert np.array_equal(o, o2)


def test_kept_tokens_by_hand():
    acc = [0.1, 5, 3, 3, float("nan"), 3, 0.2, 0.3]
    assert co.kept_tokens(acc, 8, 4, 1, 1) == [0, 1, 2, 7]        # ties: the lowest index
    assert co.kept_tokens(acc, 8, 7, 1, 1) == [0, 1, 2, 3, 5, 6, 7]   # NaN goes first
    assert co.kept_tokens(acc, 8, 3, 0, 3) == [5, 6, 7]
    assert co.kept_tokens(acc, 3, 4, 1, 1) == [0, 1, 2]
    assert co.kept_tokens([float("nan"), float("-inf"), 0.0, -0.0], 4, 3, 0, 0) == [0, 2, 3]


# ---- workspace sizes and refusals (nothing is launched) -------------------------------------

A = 1 << 20          # addresses that are never read: validation fails first
FAR = 1 << 40


def sink(area, **kw):
    d = dict(q=A, k=A, v=A, lens=None, o=A, ws=A, nb=1 << 40, B=1, H=4, Hk=2, Nq=1, S=64, D=64, window=8,
             sinks=1, scale=1.0, dtype=1)
    d.update(kw)
    area.area_sink_attn(*d.values())


def prefix(area, **kw):
    d = dict(q=A, kp=A, vp=A, k=A, v=A, lens=None, o=A, ws=A, nb=1 << 40, B=2, H=4, Hk=2, Nq=1, P=64, S=64,
             D=64, causal=1, scale=1.0, dtype=1)
    d.update(kw)
    area.area_prefix_attn(*d.values())


def cache(area, **kw):
    d = dict(q=A, k=A, v=A, lens=None, acc=None, o=A, acco=A, ws=A, nb=1 << 40, B=1, H=4, Hk=2, Nq=1, S=64,
             D=64, scale=1.0, dtype=1)
    d.update(kw)
    area.area_cache_attn(*d.values())


def evict(area, **kw):
    d = dict(k=A, v=A + FAR, acc=A + 2 * FAR, lens=A + 3 * FAR, ko=A + 4 * FAR, vo=A + 5 * FAR,
             acco=A + 6 * FAR, lenso=A + 7 * FAR, idx=A + 8 * FAR, B=1, Hk=2, S=64, So=32, D=64, budget=32,
             sinks=1, recent=4, dtype=1)
    d.update(kw)
    area.area_cache_evict(*d.values())


EINVAL, EUNSUPPORTED, ENOSPACE = 1, 2, 3
ATTN = [({"q": None}, EINVAL), ({"o": None}, EINVAL), ({"k": None}, EINVAL), ({"v": None}, EINVAL),
        ({"q": A + 8}, EINVAL), ({"k": A + 2}, EINVAL), ({"o": A + 16}, EINVAL), ({"lens": A + 2}, EINVAL),
        ({"ws": A + 4}, EINVAL), ({"B": 0}, EINVAL), ({"H": 0}, EINVAL), ({"Hk": 0}, EINVAL),
        ({"Hk": 3}, EINVAL), ({"Hk": 8}, EINVAL), ({"Nq": 0}, EINVAL), ({"S": -1}, EINVAL),
        ({"D": 96}, EUNSUPPORTED), ({"D": 0}, EUNSUPPORTED), ({"dtype": 2}, EUNSUPPORTED),
        ({"dtype": -1}, EUNSUPPORTED), ({"scale": 0.0}, EINVAL), ({"scale": -1.0}, EINVAL),
        ({"scale": float("nan")}, EINVAL), ({"scale": float("inf")}, EINVAL),
        ({"S": INT_MAX}, EUNSUPPORTED), ({"B": INT_MAX, "H": INT_MAX, "Hk": 1, "Nq": INT_MAX}, EUNSUPPORTED),
        ({"B": 1 << 20, "H": 1 << 10, "Hk": 1 << 10, "Nq": 2}, EUNSUPPORTED)]


@pytest.mark.parametrize("change,status", ATTN + [
    ({"window": 0}, EINVAL), ({"window": -5}, EINVAL), ({"sinks": -1}, EINVAL), ({"S": 0}, EINVAL),
    ({"S": 100000, "window": 100000, "nb": 16}, ENOSPACE), ({"S": 100000, "window": 100000, "ws": None}, EINVAL)])
def test_sink_refusals(area, change, status):
    with pytest.raises(area.AreaError) as e:
        sink(area, **change)
    assert e.value.status == status


@pytest.mark.parametrize("change,status", ATTN + [
    ({"kp": None}, EINVAL), ({"vp": None}, EINVAL), ({"kp": A + 8}, EINVAL), ({"P": -1}, EINVAL),
    ({"causal": 2}, EINVAL), ({"causal": -1}, EINVAL), ({"P": 0, "S": 0}, EINVAL),
    ({"P": 1 << 30, "S": 1 << 30}, EUNSUPPORTED), ({"P": 100000, "nb": 16}, ENOSPACE),
    ({"P": 100000, "ws": None}, EINVAL)])
def test_prefix_refusals(area, change, status):
    with pytest.raises(area.AreaError) as e:
        prefix(area, **change)
    assert e.value.status == status


@pytest.mark.parametrize("change,status", ATTN + [
    ({"acco": None}, EINVAL), ({"acco": A + 1}, EINVAL), ({"acc": A + 2}, EINVAL), ({"S": 0}, EINVAL),
    ({"nb": 0}, ENOSPACE), ({"ws": None}, EINVAL)])
def test_cache_refusals(area, change, status):
    with pytest.raises(area.AreaError) as e:
        cache(area, **change)
    assert e.value.status == status


@pytest.mark.parametrize("change,status", [
    ({n: None}, EINVAL) for n in ("k", "v", "acc", "ko", "vo", "acco", "lenso", "idx")] + [
    ({"k": A + 8}, EINVAL), ({"vo": A + 5 * FAR + 4}, EINVAL), ({"idx": A + 8 * FAR + 2}, EINVAL),
    ({"lens": A + 3 * FAR + 1}, EINVAL), ({"B": 0}, EINVAL), ({"Hk": 0}, EINVAL), ({"S": 0}, EINVAL),
    ({"So": 31}, EINVAL), ({"So": 0}, EINVAL), ({"budget": 0}, EINVAL), ({"sinks": -1}, EINVAL),
    ({"recent": -1}, EINVAL), ({"sinks": 16, "recent": 17}, EINVAL),
    ({"sinks": INT_MAX, "recent": INT_MAX}, EINVAL), ({"dtype": 2}, EUNSUPPORTED),
    ({"D": 80}, EUNSUPPORTED), ({"S": INT_MAX}, EUNSUPPORTED),
    ({"B": 1 << 16, "Hk": 1 << 16}, EUNSUPPORTED),
    ({"ko": A}, EINVAL),                                     # in place, but not all three
    ({"ko": A, "vo": A + FAR, "acco": A + 2 * FAR}, EINVAL),  # in place with So != S
    ({"ko": A + 16}, EINVAL),                                # part of k
    ({"vo": A + 4 * FAR + 16}, EINVAL),                      # part of ko
    ({"lenso": A + 3 * FAR}, EINVAL), ({"idx": A + 2 * FAR}, EINVAL), ({"acco": A + 7 * FAR}, EINVAL)])
def test_evict_refusals(area, change, status):
    with pytest.raises(area.AreaError) as e:
        evict(area, **change)
    assert e.value.status == status


def test_workspace_sizes(area):
    lib = area.library()
    for fn, n in (("area_sink_attn_ws_bytes", 9), ("area_prefix_attn_ws_bytes", 8),
                  ("area_cache_attn_ws_bytes", 7)):
        assert getattr(lib, fn)(*([1] * n), None) == area.AREA_EINVAL
    with pytest.raises(area.AreaError):
        area.area_sink_attn_ws_bytes(1, 4, 3, 1, 64, 64, 8, 0, 1)
    with pytest.raises(area.AreaError):
        area.area_cache_attn_ws_bytes(1, 4, 2, 1, 64, 32, 1)
    # a long cache and one row need splits, many rows of a prompt none
    assert area.area_sink_attn_ws_bytes(1, 8, 8, 1, 65536, 128, INT_MAX, 0, 1) > 0
    assert area.area_sink_attn_ws_bytes(4, 24, 24, 8192, 8192, 128, 2048, 0, 1) == 0
    # the weights' call keeps one score per row and key where a key head has few rows
    assert area.area_cache_attn_ws_bytes(2, 8, 2, 2, 5000, 128, 1) >= 2 * 8 * 2 * 5000 * 4


def test_units_of_the_tensor_core_kernel_cover_what_rows_see(tmp_path):
    # how work units are cut is integer arithmetic (cache_unit.cuh): checked on
    # the host over random problems
    import os
    import shutil
    import subprocess
    from step_adaptive_sparse_b200 import build as b
    nvcc = b.nvcc()
    if shutil.which(nvcc) is None and not os.path.exists(nvcc):
        pytest.skip("nvcc is not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "cache_unit_check")
    subprocess.run([nvcc, "-O2", "-std=c++17", "-Wno-deprecated-gpu-targets", "-I",
                    os.path.join(root, "include"), "-I", b.CSRC,
                    os.path.join(root, "tests", "cache_unit_check.cu"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
    assert "problems checked" in r.stdout


def test_build_checks_the_tensor_core_kernel():
    from step_adaptive_sparse_b200 import build as b
    log = "\n".join(["ptxas info    : Compiling entry function '_ZN4area15cache_tc_kernelILi128EEEv' for 'sm_100a'",
                     "    0 bytes stack frame, %d bytes spill stores, 0 bytes spill loads",
                     "ptxas info    : Used %d registers, used 1 barriers"])
    assert b.check_attn_resources(log % (0, 168), "cache_tc_kernel") == []
    assert len(b.check_attn_resources(log % (0, 160), "cache_tc_kernel")) == 1
    assert len(b.check_attn_resources(log % (8, 168), "cache_tc_kernel")) == 1
    assert len(b.check_attn_resources(log % (0, 168))) == 1


def test_binding_of_the_cache_calls_refuses_what_it_cannot_pass(area, monkeypatch, tmp_path):
    from step_adaptive_sparse_b200 import binding

    class Address:                 # what a tensor and a stream offer
        def __init__(self, at):
            self.at, self.cuda_stream = at, 0

        def data_ptr(self):
            return self.at

    good = [Address(32)] * 6 + [0, 1, 4, 2, 1, 64, 64, 8, 0, 0.125, 1]
    with pytest.raises(area.AreaError) as e:           # a workspace too small or a bad scale get through to the call
        area.area_sink_attn(*good[:15], -1.0, 1, Address(0))
    assert e.value.status == area.AREA_EINVAL
    with pytest.raises(TypeError):
        area.area_sink_attn(*good[:7], "1", *good[8:])
    with pytest.raises(TypeError):
        area.area_sink_attn(*good[:7], 1.5, *good[8:])
    with pytest.raises(AttributeError):
        area.area_sink_attn("q", *good[1:])
    with pytest.raises(AttributeError):
        area.area_sink_attn(*good, "stream")
    with pytest.raises(OverflowError):
        area.area_sink_attn_ws_bytes(2 ** 31, 4, 2, 1, 64, 64, 8, 0, 1)
    with pytest.raises(OverflowError):
        area.area_sink_attn(*good[:6], -1, *good[7:])
    import numpy as np
    assert area.area_sink_attn_ws_bytes(np.int64(1), 8, 8, 1, 65536, 128, INT_MAX, 0, 1) == \
        area.area_sink_attn_ws_bytes(1, 8, 8, 1, S=65536, D=128, window=INT_MAX, sinks=0, dtype=1)
    monkeypatch.setattr(binding, "_CALL", None)
    monkeypatch.setattr(binding, "_CALL_PATH", str(tmp_path / "_areacall.so"))
    with pytest.raises(ImportError):
        area.area_cache_attn_ws_bytes(1, 4, 2, 1, 64, 64, 1)


@pytest.mark.parametrize("op", ["sink", "prefix", "cache"])
def test_overlapping_buffers_are_refused(area, op):
    """Nothing is launched: the call that overlaps nowhere is refused for its
    scale, as the last check but one."""
    at = {n: A + i * FAR for i, n in enumerate(["q", "kp", "vp", "k", "v", "lens", "acc", "o", "acco", "ws"])}
    sizes = {"q": 1 * 4 * 3 * 64 * 2, "k": 2 * 5000 * 64 * 2, "v": 2 * 5000 * 64 * 2, "kp": 2 * 40 * 64 * 2,
             "vp": 2 * 40 * 64 * 2, "lens": 4, "acc": 2 * 5000 * 4}
    names = {"sink": ["q", "k", "v", "lens", "o", "ws"], "prefix": ["q", "kp", "vp", "k", "v", "lens", "o", "ws"],
             "cache": ["q", "k", "v", "lens", "acc", "o", "acco", "ws"]}[op]
    size = {"sink": [1, 4, 2, 3, 5000, 64, 5000, 0], "prefix": [1, 4, 2, 3, 40, 5000, 64],
            "cache": [1, 4, 2, 3, 5000, 64]}[op]
    nb = getattr(area, f"area_{op}_attn_ws_bytes")(*size, 1)
    assert nb > 0
    call = getattr(area, f"area_{op}_attn")

    def status(**moved):
        args = [moved.get(n, at[n]) for n in names] + [nb, *size] + ([1] if op == "prefix" else [])
        with pytest.raises(area.AreaError) as e:
            call(*args, 1.0, 1, 0)
        return e.value.status

    for out in [n for n in ("o", "acco") if n in names]:
        for inp in [n for n in names if n in sizes]:
            assert status(**{out: at[inp]}) == EINVAL if (out, inp) != ("acco", "acc") else True
            assert status(**{out: at[inp] + (sizes[inp] - 1) // 32 * 32}) == EINVAL, (out, inp)   # its last bytes
        assert status(**{out: at["ws"] + 256}) == EINVAL
    assert status(ws=at["k"] + 4096) == EINVAL
    if op == "cache":
        assert status(acco=at["o"] + 32) == EINVAL and status(acco=at["acc"] + 4) == EINVAL
