// A CUDA thread block on one host thread, for tests of kernels that need no
// tensor core: every thread is a fiber, barriers and warp votes hand control
// on, and shared words of type Shared<T> record who touches them.  Two warps
// that touch one word without a block barrier between, one of them writing, are
// a race, whatever order the fibers happened to run in.  A barrier that some
// thread of the block never reaches shows as a block that cannot go on.
#pragma once

#include <ucontext.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <functional>
#include <string>
#include <vector>

#define __device__
#define __global__
#define __forceinline__ inline
#define __noinline__
#define __grid_constant__
#define __launch_bounds__(...)
#define threadIdx (Index{emu::at})
#define blockIdx (Index{emu::block})
#define blockDim (Index{(int)emu::lanes.size()})

struct Index {
    int x;
};
struct float2 {
    float x, y;
};
struct uint4 {
    uint32_t x, y, z, w;
};
struct __nv_bfloat16 {
    uint16_t bits;
};

namespace emu {

struct Fiber {
    ucontext_t ctx;
    std::vector<char> stack;
    bool done = false;
    const long *gate = nullptr;   // waits until *gate moves on from `seen`
    long seen = 0;
};
struct Warp {
    int arrived = 0;
    long rounds = 0;
    uint64_t word[2][32];
};

inline std::vector<Fiber> lanes;
inline std::vector<Warp> warps;
inline ucontext_t home;
inline int at = 0, block = 0, arrived = 0;
inline long epoch = 0;                 // block barriers passed
inline int any[2];                     // __syncthreads_or, by the epoch's parity
inline std::string races;
inline std::function<void()> body;

inline void wait(const long *gate, long seen) {
    Fiber &f = lanes[at];
    f.gate = gate;
    f.seen = seen;
    const int me = at;
    swapcontext(&f.ctx, &home);
    at = me;
}
inline void block_barrier() {
    const long seen = epoch;
    if (++arrived == (int)lanes.size()) {
        arrived = 0;
        any[++epoch & 1] = 0;
    } else {
        wait(&epoch, seen);
    }
}
// All lanes' words of a warp-wide operation.
inline const uint64_t *exchange(uint64_t mine) {
    Warp &w = warps[at >> 5];
    const long seen = w.rounds;
    uint64_t *words = w.word[seen & 1];
    words[at & 31] = mine;
    if (++w.arrived == 32) {
        w.arrived = 0;
        ++w.rounds;
    } else {
        wait(&w.rounds, seen);
    }
    return words;
}
inline void enter() {
    body();
    lanes[at].done = true;
}
// Runs a block of `threads`, the warps in the given order; false: it cannot go on.
inline bool run(int threads, int index, const std::vector<int> &warp_order, std::function<void()> f) {
    lanes.assign(threads, Fiber());
    warps.assign(threads / 32, Warp());
    block = index;
    arrived = 0;
    any[++epoch & 1] = 0;
    body = f;
    for (int i = 0; i < threads; ++i) {
        Fiber &x = lanes[i];
        x.stack.resize(64 * 1024);
        getcontext(&x.ctx);
        x.ctx.uc_stack.ss_sp = x.stack.data();
        x.ctx.uc_stack.ss_size = x.stack.size();
        x.ctx.uc_link = &home;
        makecontext(&x.ctx, enter, 0);
    }
    for (;;) {
        bool moved = false, all = true;
        for (int w : warp_order)
            for (int i = 32 * w; i < 32 * w + 32; ++i) {
                Fiber &x = lanes[i];
                if (x.done) continue;
                all = false;
                if (x.gate && *x.gate == x.seen) continue;
                x.gate = nullptr;
                at = i;
                moved = true;
                swapcontext(&home, &x.ctx);
            }
        if (all) return true;
        if (!moved) return false;
    }
}

struct Access {
    long epoch = -1;
    uint32_t warps = 0;
    void note() {
        if (epoch != emu::epoch) warps = 0;
        epoch = emu::epoch;
        warps |= 1u << (at >> 5);
    }
    bool by_others() const { return epoch == emu::epoch && (warps & ~(1u << (at >> 5))); }
};

}  // namespace emu

template <class T> struct Shared {
    T v{};
    mutable emu::Access reads, writes, atomics;
    void check(bool bad, const char *what) const {
        if (bad && emu::races.size() < 2000)
            emu::races += std::string(what) + " by warp " + std::to_string(emu::at >> 5) + " of a word that another warp touches; ";
    }
    operator T() const {
        check(writes.by_others() || atomics.by_others(), "read");
        reads.note();
        return v;
    }
    Shared &operator=(T x) {
        check(reads.by_others() || writes.by_others() || atomics.by_others(), "write");
        writes.note();
        v = x;
        return *this;
    }
    void atomic() {
        check(reads.by_others() || writes.by_others(), "atomic");
        atomics.note();
    }
};
inline void atomicAdd(Shared<int> *p, int x) { p->atomic(); p->v += x; }
inline void atomicMax(Shared<int> *p, int x) { p->atomic(); p->v = std::max(p->v, x); }
inline void atomicOr(int32_t *p, int x) { *p |= x; }

template <class T> inline T __ldg(const T *p) { return *p; }
template <class T> inline uint64_t word_of(T x) {
    uint64_t w = 0;
    memcpy(&w, &x, sizeof x);
    return w;
}
template <class T> inline T from_word(uint64_t w) {
    T x;
    memcpy(&x, &w, sizeof x);
    return x;
}
template <class T> inline T __shfl_sync(unsigned, T x, int src) { return from_word<T>(emu::exchange(word_of(x))[src & 31]); }
template <class T> inline T __shfl_xor_sync(unsigned, T x, int o) {
    const int lane = emu::at & 31;
    return from_word<T>(emu::exchange(word_of(x))[lane ^ o]);
}
template <class T> inline T __shfl_up_sync(unsigned, T x, int o) {
    const int lane = emu::at & 31;
    return from_word<T>(emu::exchange(word_of(x))[lane >= o ? lane - o : lane]);
}
inline unsigned __ballot_sync(unsigned, int p) {
    const uint64_t *w = emu::exchange(p != 0);
    unsigned m = 0;
    for (int i = 0; i < 32; ++i) m |= (unsigned)w[i] << i;
    return m;
}
inline int __any_sync(unsigned m, int p) { return __ballot_sync(m, p) != 0; }
inline void __syncthreads() { emu::block_barrier(); }
inline int __syncthreads_or(int p) {
    emu::any[emu::epoch & 1] |= p != 0;
    emu::block_barrier();
    return emu::any[~emu::epoch & 1];
}

inline int __clz(unsigned x) { return x ? __builtin_clz(x) : 32; }
inline int __ffs(unsigned x) { return __builtin_ffs((int)x); }
inline float __fadd_rn(float a, float b) { return a + b; }
inline float __fsub_rn(float a, float b) { return a - b; }
inline float __fmul_rn(float a, float b) { return a * b; }
inline uint32_t __float_as_uint(float f) { return from_word<uint32_t>(word_of(f)); }
inline float __uint_as_float(uint32_t u) { return from_word<float>(word_of(u)); }
inline int __float_as_int(float f) { return from_word<int>(word_of(f)); }
inline float __int_as_float(int i) { return from_word<float>(word_of(i)); }
inline long long __double_as_longlong(double d) { return from_word<long long>(word_of(d)); }
inline uint4 make_uint4(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return {x, y, z, w}; }
using std::max;
using std::min;
