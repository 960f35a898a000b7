// What the tensor-core kernels of the attention over a sliding window share.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "dn_tmap.h"
#include "dn_window.cuh"
#include "tc_ptx.cuh"
#include "dn_tc_sync.cuh"

namespace dn {

constexpr int kSinkCols = 32;  // keys of the narrow tile that holds the sinks alone, where they fit

__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {  // bits lo..hi of 32, where they are any
    lo = lo < 0 ? 0 : lo;
    hi = hi > 31 ? 31 : hi;
    return lo > hi ? 0u : (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
}

// Which of the keys k0 + 0..31 token t sees.
__device__ __forceinline__ uint32_t seen32(int t, int k0, const Sight &s) {
    const int hi = t - k0;
    const int lim = s.sinks - 1 - k0 < hi ? s.sinks - 1 - k0 : hi;
    return bit_range(hi - s.window + 1, hi) | bit_range(0, lim);
}

// log2 x; off by 2^-22 at most where x is between 1 and 2, else by two units of fp32's last place
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void store16(void *dst, const uint32_t *r) {  // 16 bytes at once
    asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void store32(void *dst, const uint32_t *r) {  // 32 bytes at once, to an address on 32 bytes
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// N columns of bf16 of 32 rows, a row a lane, to global memory: four neighbouring lanes swap their quarters
// first, so that each store fills 2 N bytes of a row (a row a lane, it takes twice as long).
// w: the columns two by two; `to`: the lane's own row; `stride`: elements from row to row, a multiple of 64; rows from
// `from` up to `rows` are written.
// Tensors begin on 16 bytes, and on 32 as a rule: then the quarters of 64 columns are stored whole.  By halves always
// (with pieces of 16 bytes exchanged, so that a store fills 64 bytes of a row): training step 224 to 228 us, packed
// prompts 298 to 301.
template <int N>
__device__ __forceinline__ void store_rows(__nv_bfloat16 *to, long long stride, int from, int rows, uint32_t (&w)[4][N / 8]) {
    static_assert(N == 32 || N == 64, "quarters of 16 or 32 bytes");
    const int lane = threadIdx.x & 31, q = lane & 3;
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (a & x) continue;
            const int b = a | x;
#pragma unroll
            for (int e = 0; e < N / 8; ++e) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, q & x ? w[a][e] : w[b][e], x);
                if (q & x) w[a][e] = got;
                else w[b][e] = got;
            }
        }
    __nv_bfloat16 *first = to - q * stride + N / 4 * q;
    const bool whole = N == 64 && (reinterpret_cast<uintptr_t>(first) & 31) == 0;  // the same for all rows
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if ((lane & ~3) + j < from || (lane & ~3) + j >= rows) continue;
        if (whole) {
            if constexpr (N == 64) store32(first + j * stride, w[j]);
        } else {
#pragma unroll
            for (int h = 0; h < N / 32; ++h) store16(first + j * stride + 8 * h, w[j] + 4 * h);
        }
    }
}

// Wait of a whole warp, bounded like wwait of dn_tc_sync.cuh but without a call: what is in
// registers stays there.
__device__ __forceinline__ bool hold(const tcs::Ctx &x, uint32_t bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = ptx::globaltimer();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
        const bool late = ptx::globaltimer() - t0 > tcs::kTimeoutNs;
        if (late) {
            *x.abort_flag = 1;
            atomicOr(x.status, kStatusTimeout);
        }
        if (__any_sync(0xffffffffu, late || *x.abort_flag)) return false;
    }
}

// Slot number i in the order in which items are taken: the last tiles of a sequence first (under a causal mask the
// long ones) or, `up`, the first ones.  Without offsets by tile, then by sequence, so that the short ones
// come last of all and fill the gaps; with offsets sequence by sequence.
__device__ __forceinline__ unsigned slot_in_order(const SeqView &s, unsigned i, unsigned slots, bool up) {
    if (s.cu) return up ? i : slots - 1 - i;
    const unsigned per = slots / s.N, c = i / s.N, n = i - c * s.N;
    return n * per + (up ? c : per - 1 - c);
}

// ---- items of a block ---------------------------------------------------------
// A block for every item is launched, as many as fit run, and a running block takes over items whose
// blocks have not begun: whoever is done first takes the next one.  One thread asks, some time before the
// block needs the item; `reply`: 16 bytes of shared memory.
struct Items {
    uint32_t bar, reply;
    unsigned item = blockIdx.x, asked = 0, got = 0;
    bool any = true;  // `item` is one
    __device__ __forceinline__ void ask() {
        if (!any || asked != got) return;
        ++asked;
        ptx::mbar_arrive_expect_tx(bar, 16);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the last reply was read
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(reply),
                     "r"(bar)
                     : "memory");
    }
    __device__ __forceinline__ bool next(const tcs::Ctx &x) {  // false: the block is giving up
        ask();
        if (!any) return true;
        if (!tcs::wait(x, bar, got & 1)) return false;
        ++got;
        uint32_t some;
        asm volatile(
            "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tld.shared.b128 r, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
            : "=r"(some), "=r"(item)
            : "r"(reply)
            : "memory");
        any = some != 0;
        return true;
    }
    __device__ __forceinline__ void drain() const {
        if (asked != got) tcs::wait_drain(bar, got & 1);
    }
};

// ---- MMAs of a whole warp ---------------------------------------------------
// One lane of a converged warp issues; the others run along, so that loops, waits and descriptors
// stay warp-uniform (a branch of one thread made every MMA take about 115 cycles to issue; it takes
// as long as the tensor cores need).

__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// Descriptors of swizzled rows by their halves: the upper one is the same for all (8 rows 1024 bytes apart,
// version 1, 128-byte swizzle), the lower one holds the address in units of 16 bytes, to which
// steps are added.  rows_of: operands read along their rows; cols_of: along their columns, panels of 64 of
// them 16 KB apart.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (ptx::kSwizzle128 << 29);
__device__ __forceinline__ uint32_t rows_of(uint32_t at) { return ((at & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t cols_of(uint32_t at) { return ((at & 0x3FFFFu) >> 4) | ((16384u >> 4) << 16); }

__device__ __forceinline__ void mma_ss_by(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t more) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(more), "r"(lead), "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts_by(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t more) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 y, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(more), "r"(lead), "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void commit_by(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
        : "memory");
}

}  // namespace dn
