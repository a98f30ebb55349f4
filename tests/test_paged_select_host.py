"""The kernels of select_pages, compiled from their source for the host and run
thread by thread (block_emulator.h): the chosen blocks against the definition in
64 bits, no barrier that only some threads reach, and no shared word that two
warps touch without a barrier between.  On a GPU such a race shows by chance at
most; here it shows in any order of the threads."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(TESTS), "full_gqa_decode_gb300", "csrc")
D = 256


def host_source() -> str:
    def read(name):
        text = open(os.path.join(CSRC, name)).read()
        text = re.sub(r"^#(include|pragma).*$", "", text, flags=re.M)
        return re.sub(r"asm volatile\([^;]*;[^;]*\);", "", text)

    def struct(name, text):
        return re.search(r"struct %s \{.*?\n\};" % name, text, re.S).group(0)

    header, select = read("paged.h"), read("paged_select.cu")
    select = select[: select.index("}  // namespace\n")] + "}  // namespace\n}  // namespace hd\n"
    sched = read("paged_sched.cuh").replace("long long *tmp", "Shared<long long> *tmp")
    sched, n = re.subn(r"(tmp\[(lane|warp - 1)\] : 0)\b", r"\1LL", sched)   # a Shared beside an int would become one
    assert n == 2
    # Shared arrays of the pick: tracked words, and the dynamic part.
    select, n = re.subn(r"extern __shared__ uint64_t fine\[\];", "uint64_t *fine = dynamic_shared;", select)
    assert n == 1
    select, n = re.subn(r"__shared__ (int|long long) ", r"static Shared<\1> ", select)
    assert n == 2
    select, n = re.subn(r"int \*hist, int \*state", "Shared<int> *hist, Shared<int> *state", select)
    assert n == 1
    return "\n".join([
        '#include "block_emulator.h"', '#include "hybrid_decode.h"', "static uint64_t dynamic_shared[16384 * 2];",
        "namespace hd {", "constexpr int kHeadDim = 256;", struct("PagedSeqs", header), struct("PagedSelectArgs", header),
        """inline void unpack_bf16x8(const uint4 &r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
}""", sched, select,
        """
extern "C" int run_select(const hd::PagedSelectArgs *a, int max_blocks, int reverse, char *message, int room) {
    emu::races.clear();
    bool ok = true;
    auto order = [&](int warps) {
        std::vector<int> w(warps);
        for (int i = 0; i < warps; ++i) w[i] = reverse ? warps - 1 - i : i;
        return w;
    };
    const int rh = a->seqs.num_tokens * a->num_kv_heads, per_warp = 4;
    const int chunks = (max_blocks + hd::kScoreWarps * per_warp - 1) / (hd::kScoreWarps * per_warp);
    for (int i = 0; i < rh * chunks && ok; ++i)
        ok = emu::run(hd::kScoreThreads, i, order(hd::kScoreWarps), [&] { hd::page_score_kernel(*a, chunks, per_warp); });
    for (int i = 0; i < rh && ok; ++i)
        ok = emu::run(hd::kPickThreads, i, order(hd::kPickThreads / 32), [&] { hd::page_pick_kernel(*a, max_blocks); });
    snprintf(message, room, "%s", emu::races.c_str());
    return ok;
}
extern "C" int args_size(void) { return (int)sizeof(hd::PagedSelectArgs); }
"""])


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("select")
    src, so = d / "select.cpp", d / "select.so"
    src.write_text(host_source())
    subprocess.run(["g++", "-std=c++17", "-O1", "-ffp-contract=off", "-w", "-shared", "-fPIC", "-I", TESTS, "-I",
                    os.path.join(os.path.dirname(CSRC), "..", "include"), str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    assert lib.args_size() == ctypes.sizeof(Args)
    return lib


P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Seqs(ctypes.Structure):
    _fields_ = [("table", P), ("table_stride", I64), ("context", P), ("offsets", P), ("batch", I32), ("num_tokens", I32),
                ("max_tokens", I32), ("max_blocks", I32), ("max_context", I32), ("max_position", I32), ("page_shift", I32),
                ("num_pages", I32), ("err", P)]


class Args(ctypes.Structure):
    _fields_ = [("seqs", Seqs), ("q", P), ("bounds", P), ("k_scale", P), ("scores", P), ("score_stride", I32),
                ("num_q_heads", I32), ("num_kv_heads", I32), ("group", I32), ("num_selected", I32), ("keep_first", I32),
                ("keep_last", I32), ("selected", P)]


def bf16(x):
    """Bits of x, which bf16 holds exactly."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    assert (u & 0xFFFF == 0).all()
    return (u >> 16).astype(np.uint16)


def select(lib, q, bounds, contexts, S, first, last, page_shift=4, reverse=False):
    """q [rows, Hq, 256], bounds [blocks, Hkv, 2, 256]; one token a sequence, whose block i is page i."""
    rows, Hq, Hkv = len(contexts), q.shape[1], bounds.shape[1]
    blocks = bounds.shape[0]
    keep = dict(table=np.tile(np.arange(blocks, dtype=np.int32), (rows, 1)), context=np.array(contexts, np.int32),
                err=np.zeros(1, np.int32), q=bf16(q), bounds=bf16(bounds), scores=np.full((rows, Hkv, blocks, 2), np.nan, np.float32),
                selected=np.full((rows, Hkv, S), 99, np.int32))
    at = {k: v.ctypes.data for k, v in keep.items()}
    a = Args(Seqs(at["table"], blocks, at["context"], None, rows, rows, 1, blocks, 1 << 20, 1 << 20, page_shift, blocks, at["err"]),
             at["q"], at["bounds"], None, at["scores"], blocks, Hq, Hkv, Hq // Hkv, S, first, last, at["selected"])
    message = ctypes.create_string_buffer(4096)
    assert lib.run_select(ctypes.byref(a), blocks, int(reverse), message, 4096), "a barrier that some threads never reach"
    assert message.value == b"", message.value.decode()
    assert keep["err"][0] == 0
    return keep["selected"]


def definition(q, bounds, contexts, S, first, last, page_shift=4):
    rows, Hkv = len(contexts), bounds.shape[1]
    group = q.shape[1] // Hkv
    got = np.full((rows, Hkv, S), -1, np.int32)
    for r, c in enumerate(contexts):
        n = (c >> page_shift) + 1
        for h in range(Hkv):
            x, b = q[r, h * group: (h + 1) * group].astype(np.float64), bounds[:n, h].astype(np.float64)
            score = np.maximum(x[:, None] * b[None, :, 0], x[:, None] * b[None, :, 1]).sum((0, 2))
            score[:first] = score[max(0, n - last):] = np.inf
            pick = np.sort(np.argsort(-score, kind="stable")[:S])
            got[r, h, : len(pick)] = pick
    return got


def rounded(x):
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("S,first,last", [(1, 0, 0), (7, 1, 1), (40, 2, 3), (200, 1, 1)])
def test_choice_without_races(lib, S, first, last, reverse):
    """Scores that binary32 tells apart (no second look), over one and two kv heads' rows and short and long lists."""
    rng = np.random.default_rng(1)
    q = rounded(rng.standard_normal((3, 4, D)))
    lo = rounded(rng.standard_normal((150, 2, D)))
    bounds = np.stack([lo, rounded(lo + 1)], 2)
    contexts = [150 * 16 - 1, 5 * 16, 1000]
    got = select(lib, q, bounds, contexts, S, first, last, reverse=reverse)
    assert np.array_equal(got, definition(q, bounds, contexts, S, first, last))


@pytest.mark.parametrize("reverse", [False, True])
def test_choice_between_near_equal_scores_without_races(lib, reverse):
    """Scores that differ far below a binary32 step, and equal ones: the second look and the lowest block."""
    rng = np.random.default_rng(2)
    q = np.ones((1, 2, D), np.float32)
    q[..., 0] = 2.0 ** -20
    bounds = np.broadcast_to(rounded(rng.standard_normal(D)), (90, 1, 2, D)).copy()
    for i, blk in enumerate(rng.permutation(90)):
        bounds[blk, :, :, 0] = 2.0 ** -8 * (1 + (i // 2) / 128)
    got = select(lib, q, bounds, [90 * 16 - 1], 21, 1, 1, reverse=reverse)
    assert np.array_equal(got, definition(q, bounds, [90 * 16 - 1], 21, 1, 1))
