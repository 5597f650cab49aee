"""The host side of the key/value cache's calls: what they accept and refuse, and the index
arithmetic of their kernels, through a library that launches nothing (cache_host.cu)."""
import ctypes
import os
import shutil
import subprocess

import pytest

INT_MAX = 2 ** 31 - 1


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
    return ctypes.CDLL(out)


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
