"""CPU checks of gdn_device_error and gdn_sync_status against a stand-in for the CUDA runtime's
copies between host and device symbols: how many copies a check makes, what it clears, and which of
several recorded codes it reports."""
import os
import subprocess
import sys
import textwrap

import pytest

import gated_deltanet_linear_mixer_gb300 as gdn
from gated_deltanet_linear_mixer_gb300 import _build
from conftest import ROOT

# Device words live in this file: one block of 16 ints for each symbol, in the order in which the
# symbols are first read, preset from WORDS ("symbol:index:code", ...).
FAKE = r"""
#include <cstddef>
#include <cstdio>
#include <cstdlib>
#include <cstring>
static const void* seen[16];
static int words[16][16], n_seen = 0, reads = 0, writes = 0;
static int* block_of(const void* symbol) {
    for (int i = 0; i < n_seen; ++i)
        if (seen[i] == symbol) return words[i];
    seen[n_seen] = symbol;
    for (const char* p = std::getenv("WORDS"); p && *p;) {
        int s, at, code, used = 0;
        if (std::sscanf(p, "%d:%d:%d%n", &s, &at, &code, &used) != 3) break;
        if (s == n_seen) words[s][at] = code;
        p += used;
        if (*p == ',') ++p;
    }
    return words[n_seen++];
}
extern "C" {
int cudaMemcpyFromSymbol(void* dst, const void* symbol, size_t n, size_t offset, int) {
    ++reads;
    std::memcpy(dst, reinterpret_cast<char*>(block_of(symbol)) + offset, n);
    return 0;
}
int cudaMemcpyToSymbol(const void* symbol, const void* src, size_t n, size_t offset, int) {
    ++writes;
    std::memcpy(reinterpret_cast<char*>(block_of(symbol)) + offset, src, n);
    return 0;
}
int cudaStreamSynchronize(void*) { return 0; }
int fake_counts(int* r, int* w, int* left) {
    *r = reads, *w = writes, *left = 0;
    for (int i = 0; i < 256; ++i) *left |= words[i / 16][i % 16];
    reads = writes = 0;
    return n_seen;
}
}
"""

CHILD = """
import ctypes, os
ctypes.CDLL(os.environ["FAKE"], mode=ctypes.RTLD_GLOBAL)
lib, fake = ctypes.CDLL(os.environ["LIB"]), ctypes.CDLL(os.environ["FAKE"])
lib.gdn_last_error.restype = ctypes.c_char_p
r, w, left = (ctypes.c_int() for _ in range(3))
for _ in range(2):
    st = lib.gdn_sync_status(None)
    n = fake.fake_counts(ctypes.byref(r), ctypes.byref(w), ctypes.byref(left))
    print(st, r.value, w.value, left.value, n, lib.gdn_last_error().decode() if st else "")
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    _build.build()
    folder = tmp_path_factory.mktemp("fake")
    source, library = folder / "fake.cpp", folder / "libfake.so"
    source.write_text(FAKE)
    subprocess.run([os.environ.get("CXX") or "g++", "-shared", "-fPIC", "-o", str(library), str(source)], check=True)
    return str(library)


def _checks(fake, words=""):
    """[(status, reads, writes, what is still set, symbols, message)] of two checks in a row."""
    env = dict(os.environ, LD_PRELOAD=fake, FAKE=fake, LIB=_build.LIB_PATH, WORDS=words)
    env["LD_LIBRARY_PATH"] = "/usr/local/cuda/lib64:" + env.get("LD_LIBRARY_PATH", "")
    out = subprocess.run([sys.executable, "-c", textwrap.dedent(CHILD)], env=env, cwd=ROOT, check=True,
                         capture_output=True, text=True).stdout
    rows = []
    for l in out.strip().splitlines():
        st, r, w, left, n, *msg = l.split(" ", 5)
        rows.append((int(st), int(r), int(w), int(left), int(n), msg[0] if msg else ""))
    return rows


def test_a_clean_check_reads_a_few_words_and_writes_none(fake):
    """The mixer's kernels have four words in as many files; the cache's cost no further copies."""
    for st, reads, writes, left, symbols, _ in _checks(fake):
        assert st == 0 and reads <= 4 and writes == 0 and left == 0


def test_a_recorded_code_is_reported_once_and_cleared(fake):
    symbols = _checks(fake)[0][4]
    for s in range(symbols):
        first, second = _checks(fake, f"{s}:0:23")
        assert first[0] == gdn.GDN_ERR_TIMEOUT and "23" in first[5] and first[2] >= 1 and first[3] == 0
        assert second[0] == 0 and second[2] == 0


@pytest.mark.parametrize("words,status,code", [
    ("0:1:40", 1, "code 40"), ("0:1:41", 1, "code 41"), ("0:1:45", gdn.GDN_ERR_TIMEOUT, "code 45"),
    ("0:0:11,0:1:40", gdn.GDN_ERR_TIMEOUT, "code 11"), ("0:1:40,1:0:23", gdn.GDN_ERR_TIMEOUT, "code 23"),
    ("0:1:41,2:0:30", gdn.GDN_ERR_TIMEOUT, "code 30"), ("0:1:40,3:0:13", gdn.GDN_ERR_TIMEOUT, "code 13"),
])
def test_a_wait_is_reported_before_data_out_of_range(fake, words, status, code):
    """Word 1 of the first symbol is the cache operators'."""
    first, second = _checks(fake, words)
    assert first[0] == status and code in first[5]
    assert second[0] == 0 and second[3] == 0
