"""Host pool calls whose memory cannot be had return a status: no C++ exception crosses the C boundary, and nothing has
changed. Each case runs in a process of its own with a limit on its address space."""

import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import ctypes, resource, sys
sys.path.insert(0, {root!r})
import paged_kv_cache_157_gb300 as kvc
lib = kvc.raw()

def limit(extra):  # address space from here on: what is mapped now and `extra` bytes
    pages = int(open("/proc/self/statm").read().split()[0])
    resource.setrlimit(resource.RLIMIT_AS, (pages * resource.getpagesize() + extra,) * 2)

def pool_of(blocks, bs):
    h = ctypes.c_void_p()
    assert lib.kvc_pool_create(blocks, bs, ctypes.byref(h)) == kvc.OK
    return h

def stats(h):
    s = kvc.PoolStats()
    assert lib.kvc_pool_get_stats(h, ctypes.byref(s)) == kvc.OK
    return s.free_blocks, s.table_entries, s.useful_tokens, s.live_seqs
"""

CASES = {
    # a batch of 2^28 sequences: 2 GB of pointers alone
    "evict_batch": """
        h = pool_of(8, 16)
        ids = (ctypes.c_int64 * 1)(0)
        n = ctypes.c_int64()
        assert lib.kvc_seq_add(h, ctypes.byref(n)) == kvc.OK
        slots = (ctypes.c_int64 * 40)()
        assert lib.kvc_seq_reserve(h, 0, 40, slots) == kvc.OK
        before = stats(h)
        limit(1 << 28)
        got = lib.kvc_seq_evict_batch(h, ids, 1 << 28, slots)
        assert got == kvc.ERR_NO_MEMORY, got
        assert lib.kvc_last_error_message() != b""
        assert stats(h) == before
        lens = (ctypes.c_int64 * 1)(16)
        assert lib.kvc_seq_evict_batch(h, ids, 1, lens) == kvc.OK
    """,
    "reserve_batch": """
        h = pool_of(8, 16)
        ids = (ctypes.c_int64 * 1)(0)
        n = ctypes.c_int64()
        assert lib.kvc_seq_add(h, ctypes.byref(n)) == kvc.OK
        slots = (ctypes.c_int64 * 40)()
        before = stats(h)
        limit(1 << 28)
        got = lib.kvc_seq_reserve_batch(h, ids, 1 << 28, 1, slots)
        assert got == kvc.ERR_NO_MEMORY, got
        assert stats(h) == before
        assert lib.kvc_seq_reserve_batch(h, ids, 1, 40, slots) == kvc.OK
    """,
    "pool_create": """
        limit(1 << 28)
        h = ctypes.c_void_p(1)
        got = lib.kvc_pool_create(1 << 28, 16, ctypes.byref(h))
        assert got == kvc.ERR_NO_MEMORY, got
        assert not h.value
        pool_of(8, 16)
    """,
    # one sequence with all 2^24 blocks; its table takes 128 MB, a copy of it as much again
    "fork": """
        h = pool_of(1 << 24, 1)
        n = ctypes.c_int64()
        assert lib.kvc_seq_add(h, ctypes.byref(n)) == kvc.OK
        slots = (ctypes.c_int64 * (1 << 24))()
        assert lib.kvc_seq_reserve(h, 0, 1 << 24, slots) == kvc.OK
        before = stats(h)
        limit(1 << 26)
        n.value = 77
        got = lib.kvc_seq_fork(h, 0, ctypes.byref(n))
        assert got == kvc.ERR_NO_MEMORY, got
        assert stats(h) == before and n.value == 77
        r = ctypes.c_int32()
        assert lib.kvc_block_refcount(h, 5, ctypes.byref(r)) == kvc.OK and r.value == 1
    """,
    # a prompt whose table cannot grow: no block is taken
    "reserve": """
        h = pool_of(1 << 24, 1)
        n = ctypes.c_int64()
        assert lib.kvc_seq_add(h, ctypes.byref(n)) == kvc.OK
        slots = (ctypes.c_int64 * (1 << 24))()
        before = stats(h)
        limit(1 << 26)
        got = lib.kvc_seq_reserve(h, 0, 1 << 24, slots)
        assert got == kvc.ERR_NO_MEMORY, got
        assert stats(h) == before
        assert lib.kvc_seq_reserve(h, 0, 100, slots) == kvc.OK
        assert list(slots[:100]) == list(range(100))
    """,
    # a fork that would copy its shared last block first
    "reserve_cow": """
        h = pool_of(1 << 24, 2)
        n = ctypes.c_int64()
        assert lib.kvc_seq_add(h, ctypes.byref(n)) == kvc.OK
        slots = (ctypes.c_int64 * (1 << 24))()
        assert lib.kvc_seq_reserve(h, 0, 3, slots) == kvc.OK
        assert lib.kvc_seq_fork(h, 0, ctypes.byref(n)) == kvc.OK
        pair = (ctypes.c_int64 * 2)()
        before = stats(h)
        limit(1 << 25)
        got = lib.kvc_seq_reserve_cow(h, 1, 1 << 24, slots, pair)
        assert got == kvc.ERR_NO_MEMORY, got
        assert stats(h) == before and list(pair) == [-1, -1]
        assert lib.kvc_seq_reserve_cow(h, 1, 1, slots, pair) == kvc.OK and list(pair) == [1, 2]
    """,
    # eviction to a new table that cannot be had, beside one that can
    "evict_tables": """
        h = pool_of(1 << 24, 1)
        n = ctypes.c_int64()
        slots = (ctypes.c_int64 * (1 << 23))()
        for i, rows in ((0, 1 << 23), (1, 10)):
            assert lib.kvc_seq_add(h, ctypes.byref(n)) == kvc.OK
            assert lib.kvc_seq_reserve(h, i, rows, slots) == kvc.OK
        before = stats(h)
        ids, lens = (ctypes.c_int64 * 2)(1, 0), (ctypes.c_int64 * 2)(5, (1 << 23) - 20)
        limit(1 << 24)
        got = lib.kvc_seq_evict_batch(h, ids, 2, lens)
        assert got == kvc.ERR_NO_MEMORY, got
        assert stats(h) == before
        t, l = (ctypes.c_int32 * 10)(), (ctypes.c_int32 * 1)()
        assert lib.kvc_build_block_tables(h, ids, 1, t, 10, l) == kvc.OK
        assert list(t) == list(range(1 << 23, (1 << 23) + 10)) and l[0] == 10
    """,
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_no_memory_is_a_status(kvc, name):
    code = SETUP.format(root=ROOT) + textwrap.dedent(CASES[name]) + "\nprint('done')\n"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "done", (r.returncode, r.stdout, r.stderr[-2000:])
