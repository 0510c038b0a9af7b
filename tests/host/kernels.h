// Runs kernels on the host, in place of the HIP runtime's header: every lane of a
// workgroup is a context of its own, and what lanes exchange (ballots, shuffles,
// barriers) hands over from one to the next.  Checked on the way: every load to LDS
// against the allocation it reads, every other access by pages without access behind
// each allocation, and that a wave's lanes meet at the same exchange.
//
// Matrix instructions mix the bits of a lane's operands into its results instead of
// multiplying: what a kernel computes is not checked here, only whether it depends on
// when its loads land (at once, or as late as the kernel's own waits allow) and on which
// of a workgroup's waves runs ahead of the others.
#pragma once

#include <math.h>
#include <signal.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <sys/mman.h>
#include <unistd.h>

#include <algorithm>
#include <deque>
#include <functional>
#include <string>
#include <vector>

namespace host {

inline std::string what = "?";  // the case under way

[[noreturn]] inline void fail(const char* format, ...) {
    va_list args;
    va_start(args, format);
    printf("%s: ", what.c_str());
    vprintf(format, args);
    printf("\n");
    fflush(stdout);
    _exit(1);
}

// ---------------------------------------------------------------------------
// Memory
// ---------------------------------------------------------------------------
constexpr size_t kPage = 4096;

struct Buffer {
    char* at;
    size_t bytes, mapped;
    char* map;
};
inline std::vector<Buffer> buffers;

// `bytes` bytes that end (to 16 bytes) where the page behind them has no access.
inline void* alloc(size_t bytes) {
    const size_t mapped = (bytes + kPage - 1) / kPage * kPage + 2 * kPage;
    char* const map = static_cast<char*>(mmap(nullptr, mapped, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
    if (map == MAP_FAILED) fail("no memory");
    mprotect(map, kPage, PROT_NONE);
    mprotect(map + mapped - kPage, kPage, PROT_NONE);
    char* const at = map + mapped - kPage - (bytes + 15) / 16 * 16;
    buffers.push_back({at, bytes, mapped, map});
    return at;
}

inline void free_all() {
    for (const Buffer& b : buffers) munmap(b.map, b.mapped);
    buffers.clear();
}

inline void check(const char* from, size_t bytes, const char* base, uint32_t records, uint32_t offset) {
    for (const Buffer& b : buffers)
        if (from >= b.at && from + bytes <= b.at + b.bytes) return;
    for (const Buffer& b : buffers)
        if (base >= b.at && base <= b.at + b.bytes)
            fail("a load to LDS reads %ld bytes past the end of its operand (%zu bytes; base at %ld, %u records, offset %u)",
                 (long)(from + bytes - (b.at + b.bytes)), b.bytes, (long)(base - b.at), records, offset);
    fail("a load to LDS reads outside of every operand");
}

// ---------------------------------------------------------------------------
// Lanes
// ---------------------------------------------------------------------------
enum Exchange { kNone, kBallot, kReadLane, kXor, kDpp, kWave, kBarrier };

struct Landing {
    char* to;
    uint32_t bytes, value[4];
};

struct Lane {
    void* context;
    unsigned tid;
    bool done;
    Exchange exchange;
    int64_t value;
    int arg, mask;
    uint32_t m0;
    std::deque<Landing> flight;  // loads to LDS that have not landed
};

struct Index {
    unsigned x, y;
};

inline Lane* lane = nullptr;
inline std::vector<Lane> lanes;
inline std::vector<char> stacks;
inline void* scheduler = nullptr;
inline const std::function<void()>* kernel = nullptr;
inline Index block_index, grid;
inline bool late = false, backwards = false;  // loads land late; the last wave runs first
constexpr size_t kStack = 128 << 10;
constexpr unsigned kLanes = 64;

// Keeps the running context in *from and goes on with `to` (x86-64: the registers that
// a call preserves lie on the stack, which is all there is to a context).
__attribute__((naked, noinline)) inline void go(void** from, void* to) {
    asm("push %rbp\n\tpush %rbx\n\tpush %r12\n\tpush %r13\n\tpush %r14\n\tpush %r15\n\t"
        "mov %rsp, (%rdi)\n\tmov %rsi, %rsp\n\t"
        "pop %r15\n\tpop %r14\n\tpop %r13\n\tpop %r12\n\tpop %rbx\n\tpop %rbp\n\tret");
}

inline int64_t exchange(Exchange e, int64_t value, int arg = 0, int mask = 0) {
    lane->exchange = e;
    lane->value = value;
    lane->arg = arg;
    lane->mask = mask;
    go(&lane->context, scheduler);
    return lane->value;
}

inline void enter() {
    (*kernel)();
    if (!lane->flight.empty()) fail("the kernel ends with loads to LDS under way");
    lane->done = true;
    go(&lane->context, scheduler);
}

// What the lanes of a wave, all waiting, get from each other.
inline void answer(Lane* w) {
    int64_t out[kLanes];
    uint64_t ballot = 0;
    for (unsigned i = 0; i < kLanes; ++i)
        if (!w[i].done && w[i].value) ballot |= 1ull << i;
    for (unsigned i = 0; i < kLanes; ++i) {
        const int row = (int)i / 16, at = (int)i % 16, c = w[i].arg;
        switch (w[i].exchange) {
            case kBallot: out[i] = (int64_t)ballot; break;
            case kReadLane: out[i] = w[c].value; break;
            case kXor: out[i] = w[i ^ (unsigned)c].value; break;
            case kDpp: {
                int from = -1;
                if (c > 0x110 && c < 0x120 && at >= c - 0x110) from = (int)i - (c - 0x110);
                if (c == 0x142 && row > 0) from = row * 16 - 1;
                if (c == 0x143 && row > 1) from = 31;
                out[i] = from >= 0 && (w[i].mask >> row & 1) ? w[from].value : 0;
                break;
            }
            default: out[i] = 0;
        }
    }
    for (unsigned i = 0; i < kLanes; ++i) {
        w[i].value = out[i];
        w[i].exchange = kNone;
    }
}

// Runs a wave until it waits at a barrier (false) or has ended (true).
inline bool run_wave(Lane* w) {
    for (;;) {
        Exchange e = kNone;
        for (unsigned i = 0; i < kLanes; ++i) {
            if (w[i].done) continue;
            if (w[i].exchange == kNone) {
                lane = &w[i];
                go(&scheduler, w[i].context);
            }
            if (w[i].done) continue;
            if (e == kNone) e = w[i].exchange;
            if (w[i].exchange != e) fail("a wave's lanes wait at different exchanges");
        }
        if (e == kNone) return true;
        if (e == kBarrier) return false;
        answer(w);
    }
}

inline void run_workgroup(unsigned threads) {
    lanes.resize(threads);
    stacks.resize(threads * kStack);
    for (unsigned i = 0; i < threads; ++i) {
        Lane& l = lanes[i];
        l.tid = i;
        l.done = false;
        l.exchange = kNone;
        l.m0 = 0;
        l.flight.clear();
        // a stack from which go() returns to enter()
        uint64_t* const top = reinterpret_cast<uint64_t*>(reinterpret_cast<uintptr_t>(&stacks[(i + 1) * kStack]) & ~uintptr_t(15));
        top[-2] = reinterpret_cast<uint64_t>(&enter);
        l.context = top - 8;
    }
    const unsigned waves = threads / kLanes;
    std::vector<bool> ended(waves);
    for (;;) {
        bool any = false;
        for (unsigned k = 0; k < waves; ++k) {
            const unsigned v = backwards ? waves - 1 - k : k;
            if (ended[v]) continue;
            ended[v] = run_wave(&lanes[v * kLanes]);
            any |= !ended[v];
        }
        if (!any) return;
        for (Lane& l : lanes) l.exchange = kNone;  // the barrier is passed
    }
}

inline void launch(Index blocks, unsigned threads, const std::function<void()>& body) {
    grid = blocks;
    kernel = &body;
    for (unsigned y = 0; y < blocks.y; ++y)
        for (unsigned x = 0; x < blocks.x; ++x) {
            block_index = {x, y};
            run_workgroup(threads);
        }
}

// ---------------------------------------------------------------------------
// What the sources' inline assembly does
// ---------------------------------------------------------------------------
inline void land(Landing& l) { memcpy(l.to, l.value, l.bytes); }

inline void aim(uint32_t to) { lane->m0 = to; }

template <typename Descriptor>
void load(uint32_t bytes, Descriptor rs, int32_t offset) {
    const char* const base = reinterpret_cast<const char*>((uint64_t)(uint32_t)rs[0] | (uint64_t)(uint32_t)rs[1] << 32);
    const uint32_t records = (uint32_t)rs[2], each = bytes < 4 ? bytes : 4, i = lane->tid % kLanes;
    Landing l = {reinterpret_cast<char*>((uintptr_t)lane->m0) + i * (bytes < 4 ? 4 : bytes), bytes < 4 ? 4 : bytes, {}};
    if ((int32_t)records < 0) fail("a buffer of %d bytes", (int32_t)records);
    for (uint32_t k = 0; k < bytes; k += each) {
        const uint64_t at = (uint64_t)(uint32_t)offset + k;
        if (at + each > records) continue;  // zeros
        check(base + at, each, base, records, (uint32_t)offset);
        memcpy(&l.value[k / 4], base + at, each);
    }
    if (late)
        lane->flight.push_back(l);
    else
        land(l);
}

inline void vmcnt(size_t left) {
    while (lane->flight.size() > left) {
        land(lane->flight.front());
        lane->flight.pop_front();
    }
    exchange(kWave, 0);
}

// ---------------------------------------------------------------------------
// Builtins
// ---------------------------------------------------------------------------
template <typename V, typename R>
R mix(V a, V b, R c) {
    uint32_t x[4], y[4], z[4];
    memcpy(x, &a, 16);
    memcpy(y, &b, 16);
    memcpy(z, &c, 16);
    uint32_t h = 0x9E3779B9u;
    for (int k = 0; k < 4; ++k) h = (h ^ x[k]) * 0x85EBCA6Bu, h = (h ^ h >> 15 ^ y[k]) * 0xC2B2AE35u;
    for (int k = 0; k < 4; ++k) {
        z[k] = ((z[k] ^ h) + k) * 0x27D4EB2Fu;
        z[k] = 0x3F800000u | (z[k] ^ z[k] >> 11) >> 9;  // 1 to 2
    }
    memcpy(&c, z, 16);
    return c;
}

template <typename T>
T shfl_xor(T v, int o) {
    int64_t bits = 0;
    memcpy(&bits, &v, sizeof v);
    bits = exchange(kXor, bits, o);
    memcpy(&v, &bits, sizeof v);
    return v;
}

inline void segv(int, siginfo_t* info, void*) { fail("an access outside of every allocation, at %p", info->si_addr); }

inline void start() {
    static char stack[64 << 10];
    const stack_t alternate = {stack, 0, sizeof stack};
    sigaltstack(&alternate, nullptr);
    struct sigaction action = {};
    action.sa_sigaction = segv;
    action.sa_flags = SA_SIGINFO | SA_ONSTACK;
    sigaction(SIGSEGV, &action, nullptr);
    sigaction(SIGBUS, &action, nullptr);
}

}  // namespace host

#define __HIP_DEVICE_COMPILE__ 1
#define __device__
#define __host__
#define __global__
#define __forceinline__ inline
#define __shared__ static
#define __align__(n) __attribute__((aligned(n)))
#define __launch_bounds__(...)
#define amdgpu_waves_per_eu(...)
#define threadIdx (host::Index{host::lane->tid, 0})
#define blockIdx host::block_index
#define gridDim host::grid

enum hipError_t { hipSuccess = 0, hipErrorInvalidConfiguration = 9 };
typedef void* hipStream_t;
inline hipError_t hipGetLastError() { return hipSuccess; }
struct dim3 : host::Index {
    dim3(unsigned a, unsigned b = 1) : Index{a, b} {}
};
struct uint4 {
    uint32_t x, y, z, w;
};
#define hipLaunchKernelGGL(k, blocks, threads, lds, stream, ...) \
    host::launch(blocks, (threads).x, [=] { k(__VA_ARGS__); })

inline int32_t min(int32_t a, int32_t b) { return a < b ? a : b; }
inline int32_t max(int32_t a, int32_t b) { return a > b ? a : b; }
inline uint32_t min(uint32_t a, uint32_t b) { return a < b ? a : b; }
inline uint32_t max(uint32_t a, uint32_t b) { return a > b ? a : b; }
inline int64_t min(int64_t a, int64_t b) { return a < b ? a : b; }
inline int64_t max(int64_t a, int64_t b) { return a > b ? a : b; }
inline float __uint_as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
inline uint32_t __float_as_uint(float v) { return __builtin_bit_cast(uint32_t, v); }
inline int __popcll(uint64_t v) { return __builtin_popcountll(v); }

#define __syncthreads() ((void)host::exchange(host::kBarrier, 0))
#define __shfl_xor(v, o, width) host::shfl_xor(v, o)
#define __builtin_amdgcn_readfirstlane(v) (v)
#define __builtin_amdgcn_readlane(v, l) ((int32_t)host::exchange(host::kReadLane, (v), (l)))
#define __builtin_amdgcn_ballot_w64(v) ((uint64_t)host::exchange(host::kBallot, (v)))
#define __builtin_amdgcn_update_dpp(old, v, control, rows, banks, bound) \
    ((int32_t)host::exchange(host::kDpp, (v), (control), (rows)))
#define __builtin_amdgcn_mbcnt_lo(m, v) \
    ((uint32_t)__builtin_popcount((uint32_t)((m) & ((1ull << (host::lane->tid % 64)) - 1))) + (v))
#define __builtin_amdgcn_mbcnt_hi(m, v) \
    ((uint32_t)__builtin_popcount((uint32_t)((m) & ((1ull << (host::lane->tid % 64)) - 1 >> 32))) + (v))
#define __builtin_amdgcn_fence(...) ((void)0)
#define __builtin_amdgcn_s_barrier() __syncthreads()
#define __builtin_amdgcn_sched_barrier(m) ((void)0)
#define __builtin_amdgcn_sched_group_barrier(...) ((void)0)
#define __builtin_amdgcn_rcpf(v) (1.0f / (v))
#define __builtin_amdgcn_exp2f(v) exp2f(v)
#define __builtin_amdgcn_cvt_f32_fp8(w, at) (1.0f + ((uint32_t)(w) >> 8 * (at) & 0xFF) / 256.0f)
#define __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, at) \
    (f32x2_t{1.0f + ((w) >> 8 * (at) & 15) / 16.0f, 1.0f + ((w) >> (8 * (at) + 4) & 15) / 16.0f} * (scale))
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, x, y, z) host::mix(a, b, c)
#define __builtin_amdgcn_ds_read_tr16_b64_v4i16(p) (*(p))

// The compiler's rounding to bf16, where the host has no instruction for it.
extern "C" __attribute__((used)) __bf16 __truncsfbf2(float f) {
    uint32_t u = __builtin_bit_cast(uint32_t, f);
    u = (u + 0x7FFFu + (u >> 16 & 1u)) >> 16;
    return __builtin_bit_cast(__bf16, (uint16_t)u);
}
