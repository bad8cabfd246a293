// tkv_format.h -- device side of the cache's record format (tkv.h): where
// things lie, and how 8 codes become a matrix operand.
#pragma once

#include <hip/hip_runtime.h>

#include "tkv_internal.h"

namespace tkv {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

template <int D, int GROUP>
struct Format {
    static constexpr int W = D / 32;            // words of a lane in half a record's K (or V) codes
    static constexpr int S = W > 4 ? 2 : 1;     // ... in this many runs
    static constexpr int WV = W / S;            // ... of this many words
    static constexpr int NG = D / GROUP;        // groups of channels
    static constexpr int KG = GROUP / 32;       // K words of a group
    static constexpr int VG = GROUP / 16;       // V words of a group
    static constexpr int VC = 16 * D;           // byte offsets in a record
    static constexpr int KP = 32 * D;
    static constexpr int VP = 32 * D + 128 * NG;
    static constexpr int REC = 32 * D + 256 * NG;
};

// N consecutive words (2, 3 or 4), 4-byte aligned at least.
template <int N>
struct __attribute__((packed, aligned(4))) Words {
    uint32_t w[N];
};

template <int N>
__device__ __forceinline__ void load_words(const char *p, uint32_t *out) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        out[0] = v.x, out[1] = v.y, out[2] = v.z, out[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        out[0] = v.x, out[1] = v.y;
    } else {
        const Words<N> v = *reinterpret_cast<const Words<N> *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = v.w[i];
    }
}

template <int N>
__device__ __forceinline__ void store_words(char *p, const uint32_t *in) {
    if constexpr (N == 4) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(in[0], in[1], in[2], in[3]);
    } else if constexpr (N == 2) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(in[0], in[1]);
    } else {
        Words<N> v;
#pragma unroll
        for (int i = 0; i < N; ++i) v.w[i] = in[i];
        *reinterpret_cast<Words<N> *>(p) = v;
    }
}

// 8 codes minus BIAS as fp16, exactly.  0x6400 is 1024 in fp16, whose last
// place is 1: or-ing a code below it gives 1024 + code (or 1024 + 16 * code for
// the upper nibble of a byte), and the rest is taken off again: 1 shift, 4
// and-ors and 4 packed operations for 8 elements.
template <int BIAS>
__device__ __forceinline__ h8 codes_minus(uint32_t w) {
    const uint32_t x = w >> 8;
    // from a register, as an and-or takes one number that is not: the compiler
    // makes an and and an or of two that it knows
    uint32_t magic;
    asm("v_mov_b32 %0, 0x64006400" : "=v"(magic));
    const h2 low = {(_Float16)(1024.0f + BIAS), (_Float16)(1024.0f + BIAS)};
    const h2 s16 = {(_Float16)0.0625f, (_Float16)0.0625f};
    const h2 high = {(_Float16)(64.0f + BIAS), (_Float16)(64.0f + BIAS)};
    const h2 a0 = __builtin_bit_cast(h2, (w & 0x000F000Fu) | magic) - low;
    const h2 a1 = __builtin_bit_cast(h2, (w & 0x00F000F0u) | magic) * s16 - high;
    const h2 a2 = __builtin_bit_cast(h2, (x & 0x000F000Fu) | magic) - low;
    const h2 a3 = __builtin_bit_cast(h2, (x & 0x00F000F0u) | magic) * s16 - high;
    return (h8){a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
}

// 8 codes plus 64: bits 4..7 of 64 in fp16 count by 1, so 3 shifts and 4
// and-ors are all.  (As the subnormal numbers that their bits are codes would
// cost only 4 ands, but the matrix unit adds up products by the exponents of
// their factors, and 10 bits of its sums would go.)
constexpr float kPlus = 64.0f;
__device__ __forceinline__ h8 codes_plus(uint32_t w) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    uint32_t magic;
    asm("v_mov_b32 %0, 0x54005400" : "=v"(magic));
    constexpr uint32_t mask = 0x00F000F0u;
    return __builtin_bit_cast(h8, (u4){((w << 4) & mask) | magic, (w & mask) | magic, ((w >> 4) & mask) | magic,
                                       ((w >> 8) & mask) | magic});
}

// The nibble of code j in its word.
__device__ __forceinline__ constexpr int nibble_of(int j) { return (j >> 1) + 4 * (j & 1); }

__device__ __forceinline__ int divided(int n, Divisor d) {
    return (int)(((uint64_t)(uint32_t)n * d.mul) >> (31 + d.shift));
}
// n / d, and n becomes the rest
__device__ __forceinline__ int divide(int &n, int d, Divisor by) {
    const int q = divided(n, by);
    n -= q * d;
    return q;
}

// New tokens of sequence b: their first row and their number.  Without a
// branch, so that what it reads comes with what others read.
__device__ __forceinline__ void new_tokens(const Batch &b, int seq, int64_t &start, int &n) {
    const int32_t *from = b.starts ? b.starts + seq : b.lens;
    const int64_t s = from[0], e = from[b.starts ? 1 : 0];
    int64_t m = e - s;
    start = s;
    // rows outside the token tensors do not exist, whatever starts says
    if (s < 0 || m < 0 || e > b.n_tokens) m = 0, start = 0;
    if (!b.starts) m = b.uniform, start = (int64_t)seq * b.uniform;
    n = (int)(m < b.max_new ? m : b.max_new);
}

// The page of a position, or -1 where there is none.
__device__ __forceinline__ int page_at(const int32_t *row, int width, uint32_t n_pages, int index) {
    if (index < 0 || index >= width) return -1;
    const int p = row[index];
    return p >= 0 && (uint32_t)p < n_pages ? p : -1;
}

// The record of positions 32 * tile .. 32 * tile + 31 of `head`, in `page`.
// The address passes through a pointer to global memory, as a load through one
// to anything would wait, and be waited for, with accesses to LDS.
typedef __attribute__((address_space(1))) char global_char;
__device__ __forceinline__ char *record_at(const Cache &c, int page, int head, int tile) {
    const uint32_t in_page = (uint32_t)tile & ((1u << (c.page_shift - 5)) - 1);
    return (char *)(global_char *)(c.pool + (uint64_t)(uint32_t)page * c.page_bytes +
                                   (uint64_t)(uint32_t)head * c.head_bytes + in_page * c.record);
}

__device__ __forceinline__ float bf16_to_float(uint16_t u) { return __builtin_bit_cast(float, (uint32_t)u << 16); }

__device__ __forceinline__ uint16_t float_to_bf16(float f) {  // to nearest, ties to even; NaN stays NaN
    const uint32_t u = __builtin_bit_cast(uint32_t, f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1)) >> 16);
}

__device__ __forceinline__ float elem_to_float(uint16_t u, int type) {
    return type == kBf16 ? bf16_to_float(u) : (float)__builtin_bit_cast(_Float16, u);
}

__device__ __forceinline__ uint16_t float_to_elem(float f, int type) {
    return type == kBf16 ? float_to_bf16(f) : __builtin_bit_cast(uint16_t, (_Float16)f);
}

// 8 consecutive elements of a row as they lie, and as floats.
__device__ __forceinline__ uint4 load8_raw(const Tokens &t, int64_t offset) {
    const uint16_t *p = (const uint16_t *)t.data + offset;
    if (t.wide) return *reinterpret_cast<const uint4 *>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16>
__device__ __forceinline__ void raw_to_float(const uint4 &v, float *out) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (BF16) {
            out[i] = __builtin_bit_cast(float, i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        } else {
            out[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i / 2] >> (16 * (i & 1))));
        }
    }
}

__device__ __forceinline__ void load8(const Tokens &t, int64_t offset, float *out) {
    const uint4 v = load8_raw(t, offset);
    if (t.type == kBf16)
        raw_to_float<true>(v, out);
    else
        raw_to_float<false>(v, out);
}

// 4 consecutive elements of a row, rounded to its type, which is 16 bits wide.
__device__ __forceinline__ void store4(const Tokens &t, int64_t offset, f4 in) {
    uint16_t *p = (uint16_t *)t.data + offset;
    uint16_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = float_to_elem(in[i], t.type);
    if (t.wide) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(e[0] | ((uint32_t)e[1] << 16), e[2] | ((uint32_t)e[3] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = e[i];
    }
}

// 8 consecutive elements of a row, rounded to its type.
__device__ __forceinline__ void store8(const Tokens &t, int64_t offset, const float *in) {
    if (t.type == kF32) {
        float *p = (float *)t.data + offset;
        if (t.wide) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(in[0], in[1], in[2], in[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(in[4], in[5], in[6], in[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = in[i];
        }
        return;
    }
    uint16_t *p = (uint16_t *)t.data + offset;
    uint16_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = float_to_elem(in[i], t.type);
    if (t.wide) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = e[2 * i] | ((uint32_t)e[2 * i + 1] << 16);
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = e[i];
    }
}

// Wave-wide loads straight into LDS, N times 1 KiB (1 to 4): lane l's 16 bytes
// at base + 1024 i + 16 l, or zeros where they end past `bytes`, land at
// lds + 1024 i + 16 l (a load's offset counts for both).  From assembly, as the
// compiler would wait for them before every later access to LDS; wait_loads()
// waits.  (M0 holds the LDS address and is put back, since the compiler
// reserves it; the nops are for the hazards of M0 and of an SGPR just written.)
typedef int i4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ uint32_t lds_address(const void *p) { return (uint32_t)(uintptr_t)(lds_void *)p; }

template <int N>
__device__ __forceinline__ void load_to_lds(const char *base, uint32_t bytes, uint32_t lds, uint32_t lane16) {
    static_assert(N >= 1 && N <= 4, "an offset has 12 bits");
    const i4 d = {__builtin_amdgcn_readfirstlane((int)(uint32_t)(uint64_t)base),
                  __builtin_amdgcn_readfirstlane((int)((uint32_t)((uint64_t)base >> 32) & 0xFFFFu)),
                  __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
    const uint32_t m0 = __builtin_amdgcn_readfirstlane((int)lds);
    constexpr int kKiB = 1024;
    uint32_t saved;
#define TKV_LOADS(more)                                                     \
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\t"      \
                 "buffer_load_dwordx4 %2, %3, 0 offen lds\n\t" more         \
                 "s_nop 0\n\ts_mov_b32 m0, %0"                              \
                 : "=&s"(saved)                                             \
                 : "s"(m0), "v"(lane16), "s"(d), "n"(kKiB), "n"(2 * kKiB),  \
                   "n"(3 * kKiB)                                            \
                 : "memory")
    if constexpr (N == 1)
        TKV_LOADS("");
    else if constexpr (N == 2)
        TKV_LOADS("buffer_load_dwordx4 %2, %3, 0 offen offset:%4 lds\n\t");
    else if constexpr (N == 3)
        TKV_LOADS("buffer_load_dwordx4 %2, %3, 0 offen offset:%4 lds\n\t"
                  "buffer_load_dwordx4 %2, %3, 0 offen offset:%5 lds\n\t");
    else
        TKV_LOADS("buffer_load_dwordx4 %2, %3, 0 offen offset:%4 lds\n\t"
                  "buffer_load_dwordx4 %2, %3, 0 offen offset:%5 lds\n\t"
                  "buffer_load_dwordx4 %2, %3, 0 offen offset:%6 lds\n\t");
#undef TKV_LOADS
}

// The same for up to 12 KiB.
template <int N>
__device__ __forceinline__ void load_run_to_lds(const char *base, uint32_t bytes, uint32_t lds, uint32_t lane16) {
    load_to_lds<(N < 4 ? N : 4)>(base, bytes, lds, lane16);
    if constexpr (N > 4) load_run_to_lds<N - 4>(base + 4096, bytes ? bytes - 4096 : 0, lds + 4096, lane16);
}

// At most N of this wave's loads and stores are on their way: they end in the
// order of their issue.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "the counter's range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | 0x70 | 0xF00);
    asm volatile("" ::: "memory");
}
// Every LDS access of this wave has ended.
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
}

}  // namespace tkv
