"""The host side of the key/value cache's calls: what they accept and refuse, and the index
arithmetic of their kernels, through a library that launches nothing (cache_host.cu)."""
import ctypes
import os
import shutil
import subprocess

import pytest

INT_MAX = 2 ** 31 - 1
OK, EINVAL, EUNSUPPORTED, ENOSPACE = 0, 1, 2, 3
CALLS = ["area_sink_attn", "area_prefix_attn", "area_cache_attn", "area_cache_evict"]


@pytest.fixture(scope="session")
def host(tmp_path_factory):
    from step_adaptive_sparse_b200 import build as b
    nvcc = b.nvcc()
    if shutil.which(nvcc) is None and not os.path.exists(nvcc):
        pytest.skip("nvcc is not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = str(tmp_path_factory.mktemp("cache_host") / "cache_host.so")
    subprocess.run([nvcc, "-O1", "-std=c++17", "-Wno-deprecated-gpu-targets", "-shared", "-Xcompiler", "-fPIC",
                    "-Xlinker", "-Bsymbolic", "-I", os.path.join(root, "include"), "-I", b.CSRC,
                    os.path.join(root, "tests", "cache_host.cu"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    from step_adaptive_sparse_b200 import binding
    for name in CALLS + [c + "_ws_bytes" for c in CALLS[:3]]:
        getattr(lib, name).restype, getattr(lib, name).argtypes = binding._SIGS[name]
    return lib


# ---- how eviction shares the weights behind the kept tokens out ------------------------------

@pytest.mark.parametrize("n", [0, 1, 255, 4097, 166_000_000, INT_MAX - 4096])
@pytest.mark.parametrize("parts", [1, 2, 3, 148, 8_388_608, (INT_MAX - 4096) // 16])
def test_shares_follow_one_another_and_stay_within_32_bits(host, n, parts):
    """A block of 256 threads walks its share from thread to thread: no index on the way leaves 32
    bits, and the last share ends at n."""
    some = sorted(p for p in {0, 1, parts // 3, parts // 2, parts - 2, parts - 1} if 0 <= p < parts)
    assert host.host_share_of(n, 0, parts) == 0 and host.host_share_of(n, parts, parts) == n
    for p in some:
        a, b = host.host_share_of(n, p, parts), host.host_share_of(n, p + 1, parts)
        assert a == n * p // parts and b == n * (p + 1) // parts
        assert max(a + 255, b - 1 + 256) <= INT_MAX


# ---- lengths ---------------------------------------------------------------------------------

def test_lengths_are_read_only_where_there_is_room_for_tokens(host):
    """The kernels' own reading of a length, whatever the entry point has done before.  (A page
    that may not be read: a process that reads it ends, so a child process looks first.)"""
    import sys
    look = ("import ctypes, mmap\n"
            "libc = ctypes.CDLL(None)\n"
            "libc.mmap.restype = ctypes.c_void_p\n"
            "page = libc.mmap(None, 4096, 0, mmap.MAP_PRIVATE | mmap.MAP_ANONYMOUS, -1, 0)\n"
            f"h = ctypes.CDLL({host._name!r})\n"
            "h.host_cache_len.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]\n"
            "print(h.host_cache_len(page, 0, 1))\n")
    r = subprocess.run([sys.executable, "-c", look], capture_output=True, text=True)
    assert (r.returncode, r.stdout) == (0, "0\n")
    host.host_cache_len.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]
    lens = (ctypes.c_int * 5)(7, 0, -3, 100, -INT_MAX - 1)
    at = ctypes.addressof(lens)
    assert [host.host_cache_len(at, 9, b) for b in range(5)] == [7, 0, 0, 9, 0]
    assert host.host_cache_len(None, 9, 3) == 9


# ---- what the calls accept and refuse ---------------------------------------------------------

FAR = 1 << 40
BUFFERS = ["q", "kp", "vp", "k", "v", "lens", "acc", "o", "acco", "ws", "ko", "vo", "lenso", "idx"]
AT = {n: (i + 1) * FAR for i, n in enumerate(BUFFERS)}            # every buffer on its own
SIZES = {"B": 2, "H": 4, "Hk": 2, "Nq": 5, "P": 40, "S": 9000, "D": 64, "window": 6000, "sinks": 3}
ARGS = {
    "sink": "q k v lens o ws nb B H Hk Nq S D window sinks scale dtype stream",
    "prefix": "q kp vp k v lens o ws nb B H Hk Nq P S D causal scale dtype stream",
    "cache": "q k v lens acc o acco ws nb B H Hk Nq S D scale dtype stream",
    "evict": "k v acc lens ko vo acco lenso idx B Hk S So D budget sinks recent dtype stream",
}
EVICT = {"So": 3000, "budget": 2000, "sinks": 4, "recent": 100}


def given(op, dtype=1, **change):
    """A call's arguments: every buffer at an address of its own, unless `change` moves it."""
    a = {**AT, **SIZES, "dtype": dtype, "causal": 1, "scale": 0.125, "stream": 0, "nb": 1 << 36}
    if op == "evict":
        a.update(EVICT)
    a.update(change)
    return a


def ask(host, op, **kw):
    """The call's status.  Refused calls launch nothing, accepted ones something."""
    a = given(op, **kw)
    host.host_launches()
    status = getattr(host, "area_cache_evict" if op == "evict" else f"area_{op}_attn")(
        *[a[n] for n in ARGS[op].split()])
    assert (host.host_launches() > 0) == (status == OK)
    return status


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("op,change", [(op, {}) for op in ARGS] + [
    ("sink", {"lens": None}), ("sink", {"window": 1, "sinks": 0}), ("sink", {"window": INT_MAX, "sinks": INT_MAX}),
    ("sink", {"Nq": 9500}), ("sink", {"S": 1}), ("sink", {"Hk": 4}), ("sink", {"Hk": 1}), ("sink", {"D": 128}),
    ("sink", {"scale": 1e-30}), ("sink", {"scale": 1e38}), ("sink", {"stream": None}),
    ("sink", {"S": 100, "window": 50, "nb": 0, "ws": None}),
    ("prefix", {"causal": 0}), ("prefix", {"P": 0, "kp": None, "vp": None}),
    ("prefix", {"S": 0, "k": None, "v": None}), ("prefix", {"S": 0, "lens": AT["o"]}),
    ("cache", {"acc": None}), ("cache", {"acc": AT["acco"]}), ("cache", {"lens": None}), ("cache", {"Nq": 300}),
    ("evict", {"lens": None}), ("evict", {"budget": 1, "sinks": 0, "recent": 0}), ("evict", {"budget": 104}),
    ("evict", {"So": 2000}), ("evict", {"So": 12000, "budget": 9500}),
    ("evict", {"So": 9000, "ko": AT["k"], "vo": AT["v"], "acco": AT["acc"]})])
def test_accepted(host, op, change, dtype):
    """The calls that the refusals below change in one place each."""
    assert ask(host, op, dtype=dtype, **change) == OK


ATTN = ([{n: None} for n in ("q", "o", "k", "v", "ws")] +
        [{n: AT[n] + 8} for n in ("q", "k", "v")] + [{"o": AT["o"] + 16}, {"ws": AT["ws"] + 16}] +
        [{"lens": AT["lens"] + 2}] + [{n: 0} for n in ("B", "H", "Hk", "Nq")] +
        [{n: -1} for n in ("B", "H", "Hk", "Nq", "S")] +
        [{"Hk": 3}, {"Hk": 8}] + [{"scale": x} for x in (0.0, -0.125, float("nan"), float("inf"), -float("inf"), 2.4e38)])
REFUSED = (
    [(op, c, EINVAL) for op in ("sink", "prefix", "cache") for c in ATTN] +
    [(op, c, EUNSUPPORTED) for op in ("sink", "prefix", "cache") for c in
     ({"D": 0}, {"D": 96}, {"D": 256}, {"dtype": 2}, {"dtype": -1}, {"S": INT_MAX},
      {"B": INT_MAX, "H": INT_MAX, "Hk": 1, "Nq": INT_MAX}, {"B": 1 << 20, "H": 1 << 10, "Hk": 1 << 10, "Nq": 2})] +
    [(op, {"nb": 0}, ENOSPACE) for op in ("sink", "prefix", "cache")] +
    [("sink", c, EINVAL) for c in ({"window": 0}, {"window": -1}, {"sinks": -1}, {"S": 0})] +
    [("prefix", c, EINVAL) for c in ({"kp": None}, {"vp": None}, {"kp": AT["kp"] + 8}, {"vp": AT["vp"] + 4}, {"P": -1},
                                     {"P": 0, "S": 0}, {"causal": 2}, {"causal": -1})] +
    [("prefix", {"P": 1 << 30, "S": 1 << 30}, EUNSUPPORTED)] +
    [("cache", c, EINVAL) for c in ({"acco": None}, {"acco": AT["acco"] + 2}, {"acc": AT["acc"] + 1}, {"S": 0})] +
    [("evict", {n: None}, EINVAL) for n in ("k", "v", "acc", "ko", "vo", "acco", "lenso", "idx")] +
    [("evict", {n: AT[n] + 8}, EINVAL) for n in ("k", "v", "ko", "vo")] +
    [("evict", {n: AT[n] + 2}, EINVAL) for n in ("acc", "lens", "acco", "lenso", "idx")] +
    [("evict", {n: x}, EINVAL) for n in ("B", "Hk", "S", "So", "budget") for x in (0, -1)] +
    [("evict", c, EINVAL) for c in ({"budget": 0, "sinks": 0, "recent": 0}, {"sinks": -1}, {"recent": -1},
                                    {"sinks": 1901}, {"budget": 3001}, {"sinks": INT_MAX, "recent": INT_MAX})] +
    [("evict", c, EUNSUPPORTED) for c in ({"dtype": 2}, {"D": 80}, {"S": INT_MAX}, {"So": INT_MAX},
                                          {"B": 1 << 16, "Hk": 1 << 16})])


@pytest.mark.parametrize("op,change,status", REFUSED)
def test_refused_for_one_change(host, op, change, status):
    assert ask(host, op, **change) == status


@pytest.mark.parametrize("op", ["sink", "prefix", "cache"])
def test_a_workspace_of_the_size_asked_for_is_accepted_and_one_byte_less_refused(host, op):
    a = given(op)
    need = ctypes.c_size_t()
    names = [n for n in ARGS[op].split() if n in SIZES or n == "dtype"]
    assert getattr(host, f"area_{op}_attn_ws_bytes")(*[a[n] for n in names], ctypes.byref(need)) == OK
    assert need.value > 0 and getattr(host, f"area_{op}_attn_ws_bytes")(*[a[n] for n in names], None) == EINVAL
    assert ask(host, op, nb=need.value) == OK
    assert ask(host, op, nb=need.value - 1) == ENOSPACE


def bytes_of(host, op):
    a = given(op)
    e, kv = 2, a["B"] * a["Hk"] * a["D"] * 2
    n = {"q": a["B"] * a["H"] * a["Nq"] * a["D"] * e, "k": kv * a["S"], "v": kv * a["S"],
         "kp": a["Hk"] * a["P"] * a["D"] * e, "vp": a["Hk"] * a["P"] * a["D"] * e, "lens": a["B"] * 4,
         "acc": a["B"] * a["Hk"] * a["S"] * 4}
    n["o"], n["acco"] = n["q"], n["acc"]
    if op == "evict":
        out = a["B"] * a["Hk"] * a["So"]
        n.update(ko=out * a["D"] * e, vo=out * a["D"] * e, acco=out * 4, idx=out * 4, lenso=a["B"] * 4)
        return n
    need = ctypes.c_size_t()
    names = [x for x in ARGS[op].split() if x in SIZES or x == "dtype"]
    getattr(host, f"area_{op}_attn_ws_bytes")(*[a[x] for x in names], ctypes.byref(need))
    n["ws"] = need.value
    return n


@pytest.mark.parametrize("op", list(ARGS))
def test_overlaps_are_refused_and_neighbours_are_not(host, op):
    """Every output against every input and every other output: at its first and its last bytes,
    and just before and just behind it."""
    size = bytes_of(host, op)
    have = [n for n in ARGS[op].split() if n in AT]
    outs = {"o", "acco", "ws", "ko", "vo", "lenso", "idx"}
    step = {"o": 32, "ws": 32, "lens": 4, "lenso": 4, "acc": 4, "acco": 4, "idx": 4}      # alignments
    kw = {"nb": size["ws"]} if "ws" in size else {}
    for x in [n for n in have if n in outs]:
        for y in [n for n in have if n != x]:
            # the one of the two that may lie anywhere the other ends is moved
            mv, st = (x, y) if step.get(x, 16) <= step.get(y, 16) else (y, x)
            al = step.get(mv, 16)
            inside = (size[st] - 1) // al * al
            for at in (AT[st] + inside, AT[st] - size[mv] + al if size[mv] > al else AT[st]):
                assert ask(host, op, **{mv: at}, **kw) == EINVAL, (mv, "over", st, at - AT[st])
            if not (op == "cache" and {x, y} == {"acc", "acco"}):
                assert ask(host, op, **{mv: AT[st]}, **kw) == EINVAL, (mv, "on", st)
            for at in (AT[st] + -(-size[st] // al) * al, AT[st] - -(-size[mv] // al) * al):
                assert ask(host, op, **{mv: at}, **kw) == OK, (mv, "beside", st, at - AT[st])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,H,Hk,Nq,P,S,pools", [
    (64, 32, 8, 1, 30000, 100, 1), (1, 32, 8, 1, 30000, 100, 0), (64, 32, 8, 1, 64, 100, 0),
    (1 << 20, 8, 8, 1, 1 << 20, 1, 1),
    # the bytes that all sequences would read of the prefix pass 2^63 and 2^64
    (1 << 29, 1, 1, 1, 1 << 28, 1, 1), (1 << 30, 1, 1, 1, 1 << 30, 0, 1), (1 << 28, 4, 4, 1, 3 << 28, 1, 1)])
def test_long_prefixes_of_large_batches_are_read_once(host, B, H, Hk, Nq, P, S, pools, dtype):
    assert host.host_pools(B, H, Hk, Nq, P, S, 128, dtype) == pools


def test_row_and_key_indexes_end_where_the_header_says(host):
    """B * H * Nq and P + S up to 2^31 - 257: kernels round both up to their blocks in 32 bits."""
    need, top = ctypes.c_size_t(), 2 ** 31 - 257
    for dtype in (0, 1):
        for D in (64, 128):
            for by, want in ((0, OK), (1, EUNSUPPORTED), (256, EUNSUPPORTED)):
                at = ctypes.byref(need)
                assert host.area_sink_attn_ws_bytes(1, 1, 1, top + by, 10, D, 5, 0, dtype, at) == want
                assert host.area_prefix_attn_ws_bytes(1, 1, 1, top + by, 10, 10, D, dtype, at) == want
                assert host.area_prefix_attn_ws_bytes(1, 1, 1, 1, 7, top + by - 7, D, dtype, at) == want
                assert host.area_sink_attn_ws_bytes(1, 1, 1, 1, top + by, D, 5, 0, dtype, at) == want


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("op,B,H,Hk,Nq,P,S", [
    (0, 1, 32, 1, 1024, 0, 100_000_000), (0, 1, 64, 1, 2048, 0, 600_000_000), (1, 1, 64, 1, 1024, 300_000_000, 5000),
    (1, 64, 32, 1, 1, 200_000_000, 100), (1, 400, 60, 1, 1, 90_000_000, 0), (2, 1, 16, 1, 4096, 0, 50_000_000),
    (0, 8, 32, 8, 512, 0, 8 << 20), (0, 4, 24, 24, 4096, 0, 4096)])
def test_no_unit_of_many_rows_outlasts_the_bounded_waits(host, op, B, H, Hk, Nq, P, S, D, dtype):
    """A role of the persistent kernels may wait for as long as one unit takes: 2.1 us for 128 keys
    in bf16, 5.6 in fp32.  The waits end after 2 s, so that a unit's keys have a limit (2^23)."""
    host.host_unit_keys.restype = ctypes.c_int64
    most = host.host_unit_keys(op, B, H, Hk, Nq, P, S, D, dtype)
    assert 0 < most <= 1 << 23
    assert most / 128 * 5.6e-6 < 0.5
