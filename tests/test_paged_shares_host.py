"""The work split of the paged attention kernels (paged_sched.cuh), compiled from
its source for the host and run thread by thread (block_emulator.h): the shares
of a call follow one another, begin where their cursor says, cut no item that
is to stay whole, and agree on who holds the pieces of those that are cut."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(TESTS), "full_gqa_decode_gb300", "csrc")


def host_source() -> str:
    def read(name):
        text = re.sub(r"^#(include|pragma).*$", "", open(os.path.join(CSRC, name)).read(), flags=re.M)
        return re.sub(r"asm volatile\([^;]*;[^;]*\);", "", text)

    def piece(pattern, text):
        found = re.findall(pattern, text, re.S)
        assert len(found) == 1, (pattern, len(found))
        return found[0]

    header, chunk = read("paged.h"), read("paged_chunk.cu")
    sched = read("paged_sched.cuh").replace("long long *tmp", "Shared<long long> *tmp").replace("int *at,", "Shared<int> *at,")
    sched, n = re.subn(r"(tmp\[(lane|warp - 1)\] : 0)\b", r"\1LL", sched)
    assert n == 2
    return "\n".join([
        '#include "block_emulator.h"', '#include "hybrid_decode.h"', "using std::max; using std::min;", "namespace hd {",
        piece(r"constexpr int kChunkRows = \d+;", header), piece(r"constexpr int kChunkKeys = \d+;", header),
        piece(r"struct PagedSeqs \{.*?\n\};", header), "struct PagedAttnArgs { PagedSeqs seqs; int32_t num_kv_heads, group_shift, window; };",
        "}", sched, "namespace hd {", piece(r"constexpr int kTileRows = [^;]*;", chunk), piece(r"constexpr int kItemCost = [^;]*;", chunk),
        piece(r"constexpr int kSnap = [^;]*;", chunk), piece(r"constexpr int kMinTiles = [^;]*;", chunk),
        piece(r"struct ChunkTile \{.*?\n\};", chunk), piece(r"__device__ __forceinline__ ChunkTile make_chunk_tile\(.*?\n\}", chunk),
        piece(r"__device__ __forceinline__ int num_chunk_tiles\(.*?\n\}", chunk),
        piece(r"__device__ __forceinline__ int longest_whole\(.*?\n\}", chunk),
        """
struct Share { long long x0, x1, T; int n, bad, b, tile, h, off; };
extern "C" int longest(const PagedAttnArgs *a) { return longest_whole(*a); }
// The items in order: units, one per (sequence, tile, kv head).
extern "C" int items(const PagedAttnArgs *a, int32_t *units) {
    int n = 0;
    for (int b = 0; b < a->seqs.batch; ++b) {
        int bit;
        const SeqSpan q = seq_span(a->seqs, b, &bit);
        for (int t = 0; t < num_chunk_tiles(*a, q.n); ++t)
            for (int h = 0; h < a->num_kv_heads; ++h) units[n++] = make_chunk_tile(*a, q, t).units + kItemCost;
    }
    return n;
}
extern "C" int share(const PagedAttnArgs *a, int who, int workers, int threads, Share *out, char *message, int room) {
    static Shared<long long> tmp[33];
    static Shared<int> at[5];
    emu::races.clear();
    std::vector<int> order(threads / 32);
    for (size_t i = 0; i < order.size(); ++i) order[i] = (int)(order.size() - 1 - i);
    std::vector<Share> all(threads);
    const bool ok = emu::run(threads, who, order, [&] {
        Share s{};
        const Start c = find_share(a->seqs, a->num_kv_heads, who, workers, kMinTiles, 0, longest_whole(*a), INT_MAX, tmp, at, &s.x0,
                                   &s.x1, &s.T, &s.n, &s.bad, [&](int n) { return num_chunk_tiles(*a, n); },
                                   [&](const SeqSpan &q, int i) { return make_chunk_tile(*a, q, i).units + kItemCost; });
        s.b = c.b, s.tile = c.tile, s.h = c.h, s.off = c.off;
        all[threadIdx.x] = s;
    });
    for (const Share &s : all)
        if (memcmp(&s, &all[0], sizeof s)) emu::races += "threads disagree; ";
    *out = all[0];
    snprintf(message, room, "%s", emu::races.c_str());
    return ok;
}
extern "C" int holder(long long x, long long T, int n) { return cta_of_unit(x, T, n); }
}
"""])


P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Args(ctypes.Structure):
    _fields_ = [("table", P), ("table_stride", I64), ("context", P), ("offsets", P), ("batch", I32), ("num_tokens", I32),
                ("max_tokens", I32), ("max_blocks", I32), ("max_context", I32), ("max_position", I32), ("page_shift", I32),
                ("num_pages", I32), ("err", P), ("num_kv_heads", I32), ("group_shift", I32), ("window", I32)]


class Share(ctypes.Structure):
    _fields_ = [("x0", I64), ("x1", I64), ("T", I64)] + [(n, I32) for n in ("n", "bad", "b", "tile", "h", "off")]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("shares")
    src, so = d / "shares.cpp", d / "shares.so"
    src.write_text(host_source())
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-shared", "-fPIC", "-I", TESTS, "-I",
                    os.path.join(os.path.dirname(CSRC), "..", "include"), str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.holder.argtypes = [I64, I64, I32]
    return lib


def shares(lib, spans, kv_heads=2, group_shift=2, window=0, pairs=76, max_tokens=None):
    """(share of every pair, items' units, longest whole item)."""
    offsets = np.concatenate([[0], np.cumsum([n for _, n in spans])]).astype(np.int32)
    context = np.array([c for c, _ in spans], np.int32)
    most = max(1, max(n for _, n in spans))
    a = Args(None, 0, context.ctypes.data, offsets.ctypes.data, len(spans), int(offsets[-1]), max_tokens or most, 1 << 20, 1 << 20,
             1 << 21, 6, 1, None, kv_heads, group_shift, window)
    units = np.zeros(sum((n << group_shift) // 256 + 1 for _, n in spans) * kv_heads, np.int32)
    units = units[: lib.items(ctypes.byref(a), units.ctypes.data_as(P))]
    got, message = [], ctypes.create_string_buffer(4096)
    for who in range(pairs):
        s = Share()
        threads = 352 if len(spans) <= 32 else 64   # 11 warps as in the kernel; more sequences: all threads share the work
        assert lib.share(ctypes.byref(a), who, pairs, threads, ctypes.byref(s), message, 4096), "a barrier that some threads never reach"
        assert message.value == b"", message.value.decode()
        got.append(s)
    return got, units, lib.longest(ctypes.byref(a))


def check(lib, got, units, whole):
    T = int(units.sum())
    ends = np.cumsum(units)
    assert all(s.T == T and s.n == got[0].n and not s.bad for s in got)
    busy = [s for s in got if s.x0 < s.x1]
    at = 0
    for s in busy:
        assert s.x0 == at, "shares follow one another"
        at = s.x1
    assert at == T
    starts = np.concatenate([[0], ends[:-1]])
    cuts = {s.x0 for s in busy}
    for i, (lo, hi) in enumerate(zip(starts, ends)):
        inside = [x for x in cuts if lo < x < hi]
        assert not (inside and units[i] <= whole), "an item that stays whole is cut"
        if inside:   # its pieces' holders, which merge it, by the borders before they were moved
            first, last = lib.holder(int(lo) + 2, T, got[0].n), lib.holder(int(hi) - 1, T, got[0].n)
            holders = [k for k, s in enumerate(got) if s.x0 < hi and s.x1 > lo + 2]
            assert holders == list(range(first, last + 1)), (i, holders, first, last)


def test_shares_of_random_calls(lib):
    rng = np.random.default_rng(1)
    for _ in range(25):
        n = int(rng.integers(1, 33))
        most = int(rng.choice([8, 60, 700]))
        spans = [(int(c), int(t)) for c, t in zip(rng.integers(0, rng.choice([50, 3000, 30000]), n), rng.integers(0, most, n))]
        if not any(t for _, t in spans):
            spans[0] = (5, 3)
        kw = dict(kv_heads=int(rng.integers(1, 5)), group_shift=int(rng.integers(0, 4)), window=int(rng.choice([0, 512])),
                  pairs=int(rng.choice([1, 7, 76])))
        check(lib, *shares(lib, spans, **kw))


def test_shares_of_many_sequences(lib):
    rng = np.random.default_rng(2)
    spans = [(int(c), int(t)) for c, t in zip(rng.integers(0, 4000, 90), rng.integers(0, 5, 90))]
    check(lib, *shares(lib, spans, pairs=9))


def test_one_sequence_of_few_tokens_is_shared_out(lib):
    """Four tokens behind 1700 keys at two kv heads: the merge of 16 rows is no reason to keep two pairs of 76 busy."""
    got, units, whole = shares(lib, [(1700, 4)])
    check(lib, got, units, whole)
    assert sum(s.x0 < s.x1 for s in got) > 2 * 2
    got, units, whole = shares(lib, [(0, 1500)])   # a prompt's tiles of 256 rows stay whole
    check(lib, got, units, whole)
    assert sum(s.x0 < s.x1 for s in got) <= len(units)
