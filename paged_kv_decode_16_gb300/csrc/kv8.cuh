// kv8.cuh -- the 8-bit cache: its element and scale formats, and the launchers
// of the kernels that write and read it.
//
// Elements are e4m3 (4 exponent bits, 3 of fraction, largest value 448, no
// infinity); every block of 16 tokens of a page has, for each KV head and each
// side (K, V), one scale 2^e, stored as E8M0 (the byte e + 127) in
// scales[page][head][block][side].  Powers of two because a block fills up one
// token at a time: when a later token needs a larger scale, the rows already
// there move to it with no second rounding, except where they fall below
// e4m3's smallest normal value.  (A scale of amax / 448 would round every
// earlier row again at each step up.)
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace pkv {

// Range of the scales' exponents.  100 binary orders: the attention keeps one
// running maximum for p * 2^e and the softmax's sum alike, and fp32 holds the
// terms of both ends beside each other that far apart (kv8_decode.cuh).
constexpr int kKv8MinExp = -60;
constexpr int kKv8MaxExp = 40;

// The smallest e with a <= 448 * 2^e, within the range; a >= 0, finite.
__host__ __device__ __forceinline__ int kv8_need_exp(float a) {
#ifdef __CUDA_ARCH__
    const uint32_t u = __float_as_uint(a);
#else
    union { float f; uint32_t u; } x = {a};
    const uint32_t u = x.u;
#endif
    // a = m 2^x, m in [1, 2): 448 = 1.75 * 2^8 (subnormal a: below the range)
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < kKv8MinExp ? kKv8MinExp : (e > kKv8MaxExp ? kKv8MaxExp : e);
}

__host__ __device__ __forceinline__ int kv8_clamp_exp(int e) {
    return e < kKv8MinExp ? kKv8MinExp : (e > kKv8MaxExp ? kKv8MaxExp : e);
}

// The weights P of a product are fp16, 2^(x - m + lift) for a reference m of the row that x
// may pass by `slack` before m moves up to it: they stay below 2^15.  x = s + ev holds
// the exponent of the V scale, so a block of a large one lifts m above the others'
// weights, whatever its own share in the softmax, down to zero in fp16 (a value of 2^28
// among ordinary ones: outputs off by as much as they are).  So m suits one exponent,
// ev_ref: m <= (the row's largest s) + ev_ref.  A block whose ev is larger moves ev_ref
// up; one whose ev is more than `span` below it moves m down first, to log2 of the row's
// sum of 2^s, + ev.  Either way a weight has all 11 bits down to 2^-14 of the row's sum,
// wherever the scales lie.  (One block of 16 tokens in 16 of a 2^20 times larger
// scale: 32 sequences of 512 to 4096 tokens 27.9 us instead of 26.7, with 5 query tokens
// 51.4 instead of 46.5.)  The fp32 sums cannot overflow by it: the row's l becomes
// 2^(lift - ev), at most 2^67, and o / l is a mean of values, at most 2^49.
constexpr float kKv8Slack = 8.f;
constexpr float kKv8Lift = 7.f;
constexpr int kKv8Span = 7;

// 2^e, e in [-126, 127].
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four e4m3 bytes -> two half2 words (every e4m3 value is an fp16 value).
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Two floats -> two e4m3 bytes (a in the low one), to nearest even, beyond 448
// to 448; NaN stays NaN.
__device__ __forceinline__ uint32_t f2_to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// --- decode (kv8_decode.cuh) ------------------------------------------------
// Batches up to this size: every CTA of the decode kernel works the ranges out
// for itself; larger ones: the plan kernel does, once (256 sequences of 100 to 500
// tokens: 34.5 us, 36.5 with the plan kernel; 400: 47.8 against 50.7).
constexpr int kKv8SelfPlan = 512;
// A unit's start (its queries, its result) counts as this many chunks when the
// ranges are cut (112 sequences of 5 to 4000 tokens, us with 1 / 2 / 4 / 7 / 10:
// 82.4 / 75.0 / 71.1 / 72.6 / 74.5).
constexpr int kKv8UnitCost = 4;
// Automatic worker count: at least this many positions each (us with 1 / 2 / 4 / 8; 32/8
// heads of 128, one query token; one sequence of 200: 8.4 / 9.1 / 10.0 / 12.5, of 1500:
// 10.8 / 10.1 / 10.9 / 12.8, of 4000: 13.0 / 11.5 / 11.6 / 13.5; 16 of 64 tokens, a
// unit no longer whole: 12.5 / 12.2 / 11.0 / -; 8 query tokens of 4 sequences of 900: 22.3
// / 21.7 / 24.1 / -; the tcgen05 kernel within 1 us of 1 to 8).
constexpr int kKv8MinPositions = 2;

constexpr int kKv8Warps = 4;  // workers (warps) of a CTA of the decode kernel

// k / cpp as the high word of k * magic, for cpp = 1 .. 16 (chunks of a page) and k
// below 2^27 (chunks of a sequence): magic * cpp exceeds 2^32 by less than 16.
// 0 stands for cpp = 1.
inline uint32_t kv8_page_magic(int cpp) {
    return cpp == 1 ? 0u : (uint32_t)(((1ull << 32) + cpp - 1) / cpp);
}
__device__ __forceinline__ int kv8_page_col(int k, uint32_t magic) {
    return magic ? (int)__umulhi((uint32_t)k, magic) : k;
}

// Workers and the split of `total` positions over them: sw each, one more for
// the first r.
__host__ __device__ __forceinline__ void kv8_ranges(int total, int workers_req, int workers_auto,
                                                    int* nw, int* sw, int* r) {
    int n;
    if (workers_req > 0) {
        n = workers_req < total ? workers_req : total;
    } else {
        n = total / kKv8MinPositions + (total % kKv8MinPositions ? 1 : 0);
        if (n > workers_auto) n = workers_auto;
    }
    *nw = n;
    *sw = n > 0 ? total / n : 0;
    *r = n > 0 ? total - *sw * n : 0;
}

// Rows of all units up to which the combine kernel gives a row of many segments a
// CTA instead of a warp (2 sequences of 8192 tokens, 16 query tokens, 1024 rows: a
// CTA a row 33.0 us in all, a warp 28.2).
constexpr int kKv8RowCtas = 512;

// Workers whose parts of one unit are merged by their CTA before they leave it:
// `most` (a CTA's, or 1 where a worker is a CTA) when units are few beside the
// workers (nw); else 1, none are.  us of a call, decode and combine together, none
// merged / all merged, 32/8 heads of 128: 32 sequences of 512 to 4096 tokens (7 workers a
// unit) 26.9 / 26.6, with 5 query tokens 46.5 / 48.8; 16 of them (14) 21.2 / 21.7, 8 (28)
// 14.5 / 14.9; 256 of 16 to 8192, 28/4 heads, 66.4 / 67.5.  Large states and many workers
// gain: 5 query tokens of 8 sequences of 1000 to 8192 (19 a unit) 33.7 / 31.5, of 4 (38)
// 33.1 / 26.5, 8 of 4 (19) 39.8 / 32.4; one sequence of 32768 (228) 24.2 / 22.9, with one
// KV head 28.2 / 20.1.
__host__ __device__ __forceinline__ int kv8_merge_warps(int units, int nw, int most) {
    return nw / 16 > units ? most : 1;
}

struct Kv8DecodeParams {
    const void* q;        // [B][n_queries][Hq][D]
    void* out;
    const int32_t* table;   // [B][table_stride]
    const int32_t* lens;    // [B], the caller's
    const uint16_t* scales;  // one word a block: the K scale's byte, then the V scale's
    WsHeader* hdr;          // ranges: written by this kernel (self_plan) or the plan kernel
    int32_t* prefix;        // [B + 1] first position of every sequence: likewise
    uint32_t* flags;        // [workers rounded up to whole CTAs] PKV_DEV_* bits of every worker
    float* partials;        // [slots][partial_slot_floats(gs, D)]
    RowShape rows;
    int gs;                 // rows of a full unit (the partial states' layout)
    int self_plan;
    int after_append;       // the kernel before it is the step's append (see kv8_decode.cuh)
    int unit_cost;          // positions a unit has beside its chunks
    int merge;              // workers whose parts of a unit may be merged by their CTA
    int workers_req, workers_auto;
    int batch, n_kv_heads, sub_groups, units_per_b, units, num_pages, table_stride;
    int chunks_per_page;
    uint32_t page_magic;    // kv8_page_magic(chunks_per_page)
    long long cap;          // tokens of a table row
    float scale_log2;       // scale * log2(e)
};

// Launch configuration of one instantiation (the kernel also takes the K and V
// tensor maps).
struct Kv8DecodeInfo {
    void (*fn)(Kv8DecodeParams, CUtensorMap, CUtensorMap) = nullptr;
    void (*umma)(Kv8DecodeParams, const uint8_t*, const uint8_t*) = nullptr;  // instead of fn
    int warps = 0;    // workers of a CTA
    int threads = 0;
    int smem_bytes = 0;
};

// rows: query rows of a unit, 1 .. 32.
Kv8DecodeInfo kv8_decode_info_bf16(int head_dim, int rows);
Kv8DecodeInfo kv8_decode_info_f16(int head_dim, int rows);

// Units of up to kKv8UmmaRows rows on the fifth-generation tensor cores
// (kv8_umma.cu); takes the pools' addresses.
constexpr int kKv8UmmaRows = 128;
Kv8DecodeInfo kv8_umma_info(bool bf16, int head_dim);

// The ranges of a batch of more than kKv8SelfPlan sequences.
cudaError_t launch_kv8_plan(const Kv8DecodeParams& p, cudaStream_t stream);

// Merges the units that several workers share, and sets the workspace's status
// to the OR of n_flags words (and of the plan kernel's, when it ran).
struct Kv8CombineArgs {
    const float* partials;
    const int32_t* prefix;
    WsHeader* hdr;
    const uint32_t* flags;
    int n_flags;
    int self_plan, unit_cost;
    int merge;  // as the decode kernel's
    void* out;
    int units, units_per_b, sub_groups, gs;
    RowShape rows;
};

cudaError_t launch_kv8_combine(bool bf16, int head_dim, const Kv8CombineArgs& a, int workers,
                               cudaStream_t stream);

// --- append (kv8_append.cu) -------------------------------------------------
struct Kv8AppendArgs {
    const void* q;       // [tokens][Hq][D] (null: no queries to rotate)
    void* q_out;
    const void* k_new;   // [tokens][Hkv][D]
    const void* v_new;
    uint8_t* k_pool;     // [NP][Hkv][P][D] e4m3
    uint8_t* v_pool;
    uint8_t* scales;     // [NP][Hkv][P / 16][2]
    const int32_t* table;      // [n_seqs][table_stride]
    const int32_t* positions;  // [tokens], < 0: not appended
    const int32_t* seq_ids;    // [tokens] table row of each token; null: token i's is row i
    int n_tokens, n_seqs, table_stride, n_q_heads, n_kv_heads, page_size, num_pages;
    int bf16;            // element type of q, k_new, v_new: bf16, else fp16
    int rope;            // rotate q and k_new
    const void* q_norm_w;  // null: no norm on that side
    const void* k_norm_w;
    float norm_eps;
    uint64_t turns[64];  // theta^(-2i/D) / 2 pi, its fraction times 2^64
};

// PKV_DEV_* bits of skipped runs: ORed into *status (nullable), or, without
// seq_ids and with flags, written to flags[i] for every token i.
cudaError_t launch_kv8_append(const Kv8AppendArgs& a, int head_dim, uint32_t* status,
                              uint32_t* flags, cudaStream_t stream);

}  // namespace pkv
