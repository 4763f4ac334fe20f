// kv8_append.cu -- appending keys and values to the 8-bit paged cache, with
// the optional norm and rotation of q and k in the same pass.
//
// A run is the longest stretch of consecutive tokens of one sequence, at
// consecutive positions, within one block of 16: the unit that sets a block's
// scale.  Its first token (its leader) is found from the token and the one
// before it alone, so a CTA needs no list of sequences: a CTA of group i has the runs
// whose leaders lie among tokens 16 i .. 16 i + 15, which are the tokens from
// its first leader up to the next group's.  The cos / sin of those tokens are
// formed once in shared memory for all heads; then a group of lanes takes a
// row of q, and a warp takes one (run, head, side): the whole block in
// registers, one pass over the data.  The CTAs of a group share these tasks.
//
// What bounds it: long prompts, HBM (q read and written in 16 bits, K and V read
// in 16 and written in 8) and the instructions around it -- 8 prompts of 509 to 4096
// tokens, 32/8 heads of 128, norm and rotation: 325 MB in 65.9 us, 73% of the
// measured copy rate, 53% of the issue slots; a step's single tokens, latency (256
// tokens, 28/4 heads: 3.3 us).
#include <math.h>

#include <algorithm>

#include "kv8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kDepth = 2;   // tasks of a warp whose rows are on the way
constexpr int kVecs = 8;    // 16-byte vectors a lane holds of a task's rows
constexpr int kSlots = 2 * 152;  // CTAs at the same time: two on each SM of a GB300
constexpr int kSpan = 16;   // tokens a CTA looks for leaders among
constexpr int kMaxSpan = kSpan + kChunk - 1;  // tokens it may own

// Pairs of floats: the packed multiply and fused multiply-add of this part (each
// half rounds as the scalar one does) halve the arithmetic's instructions.
using f2 = unsigned long long;

__device__ __forceinline__ f2 make_f2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split_f2(f2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 neg2(f2 a) { return a ^ 0x8000000080000000ull; }

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, f2 (&f)[4]) {
    float x[8];
    Cvt<T>::unpack8(v, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = make_f2(x[2 * e], x[2 * e + 1]);
}

template <typename T>
__device__ __forceinline__ uint4 pack(const f2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a, b;
        split_f2(f[e], a, b);
        w[e] = Cvt<T>::pack2(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Tables of N floats in shared memory, eight to a lane, are laid out as two halves
// of four floats a lane: a lane's two 16-byte reads then sit next to its
// neighbours'.  Place of float x:
template <int N>
__device__ __forceinline__ int place(int x) {
    return (x & 4) * (N / 8) + (x >> 3) * 4 + (x & 3);
}

// Floats 8 jl .. 8 jl + 7 of such a table.
template <int N>
__device__ __forceinline__ void load8(const float* p, int jl, f2 (&f)[4]) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p + 4 * jl);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(p + N / 2 + 4 * jl);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

// cos and sin of position * theta^(-2i/D), from the frequency in turns as a
// 64-bit binary fraction: the product wraps modulo one turn by itself, exactly
// (fp64 products would cost more on this part and lose low bits at far
// positions).  The top 32 bits as a signed fraction of half a turn give the
// angle to 2^-32 turns before its rounding to fp32.
__device__ __forceinline__ void turn_cos_sin(int pos, uint64_t turns, float* c, float* s) {
    const uint64_t ph = (uint64_t)(int64_t)pos * turns;
    const float x = (float)(int)(ph >> 32) * 4.6566128730773926e-10f;  // 2^-31: half turns
    sincospif(x, s, c);
}

// 1 / rms of the row whose elements D / 16 neighbouring lanes hold.
template <int D>
__device__ __forceinline__ float inv_rms(const f2 (&lo)[4], const f2 (&hi)[4], float eps) {
    f2 sum = mul2(lo[0], lo[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) sum = fma2(lo[e], lo[e], sum);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum = fma2(hi[e], hi[e], sum);
    float a, b;
    split_f2(sum, a, b);
    a += b;
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
    return 1.0f / sqrtf(a / (float)D + eps);
}

// Norm: a lane's elements lo and their partners hi times 1 / rms and the weights
// wlo, whi.
__device__ __forceinline__ void scale_row(f2 (&lo)[4], f2 (&hi)[4], float inv, const f2 (&wlo)[4],
                                          const f2 (&whi)[4]) {
    const f2 i2 = make_f2(inv, inv);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        lo[e] = mul2(mul2(lo[e], i2), wlo[e]);
        hi[e] = mul2(mul2(hi[e], i2), whi[e]);
    }
}

__device__ __forceinline__ void rotate_row(f2 (&lo)[4], f2 (&hi)[4], const f2 (&c)[4],
                                           const f2 (&s)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f2 a = lo[e], b = hi[e];
        lo[e] = fma2(a, c[e], mul2(b, neg2(s[e])));
        hi[e] = fma2(b, c[e], mul2(a, s[e]));
    }
}

// Eight elements times up (2^-e) as e4m3 bytes.
__device__ __forceinline__ uint2 quantise8(const f2 (&x)[4], float up) {
    const f2 u2 = make_f2(up, up);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a, b;
        split_f2(mul2(x[e], u2), a, b);
        w[e] = f2_to_e4m3x2(a, b);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

__device__ __forceinline__ float max_abs8(const f2 (&x)[4], float m) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a, b;
        split_f2(x[e], a, b);
        m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));  // a NaN is passed over
    }
    return m;
}

// A lane's vectors of a task come through shared memory by asynchronous copies
// (its own vectors only: no other lane waits for them), two tasks ahead: in
// registers the loads would wait for the arithmetic of the task before (82.5 us of
// the prompts above, against 68.0; three tasks ahead leave one CTA an SM: 98).
__device__ __forceinline__ void copy_vec(uint32_t dst, const uint4* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}

struct Run {
    int tok;   // its first token
    int n;     // tokens
    int lo;    // slot of the first token in its block
    long long blk;  // block of the pool at head 0: page * Hkv * (P / 16) + block of the page
};

// What a warp needs of the block that it appends to.
struct Target {
    uint8_t* rows;   // the block's rows
    uint8_t* scale;
    const uint4* src;        // the run's first row
    long long src_stride;    // 16-byte vectors from one token's row to the next's
    const float* ctab;       // of the run's first token (null: no rotation)
    const float* stab;
    const float* w;          // norm weights (null: none)
};

// The block's exponent after a run of largest element `top`; moves the rows below
// the run to it when it grows, and stores it.  Warp-collective.
template <int D>
__device__ __forceinline__ int settle_scale(const Target& t, int lo, float top, int lane) {
    int e = kv8_need_exp(top);
    if (lo > 0) {
        const int old = kv8_clamp_exp((int)*t.scale - 127);
        if (e > old) {
            // exact above e4m3's smallest normal value
            const float f = exp2i(old - e);
            uint32_t* w = reinterpret_cast<uint32_t*>(t.rows);
            for (int x = lane; x < lo * D / 4; x += 32) {
                uint32_t h0, h1;
                e4m3x4_to_h2(w[x], h0, h1);
                const float2 p = __half22float2(*reinterpret_cast<__half2*>(&h0));
                const float2 q = __half22float2(*reinterpret_cast<__half2*>(&h1));
                w[x] = f2_to_e4m3x2(p.x * f, p.y * f) | f2_to_e4m3x2(q.x * f, q.y * f) << 16;
            }
        } else {
            e = old;
        }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *t.scale = (uint8_t)(e + 127);
    return e;
}

// A lane's elements of row x of the run.
template <typename T, int D>
__device__ __forceinline__ void row_values(const Target& t, int x, int jl, float eps, f2 (&lo)[4],
                                           f2 (&hi)[4]) {
    constexpr int HALF = D / 2;
    if (t.w) {
        f2 wlo[4], whi[4];
        load8<HALF>(t.w, jl, wlo);
        load8<HALF>(t.w + HALF, jl, whi);
        scale_row(lo, hi, inv_rms<D>(lo, hi, eps), wlo, whi);
    }
    if (t.ctab) {
        f2 c[4], s[4];
        load8<HALF>(t.ctab + x * HALF, jl, c);
        load8<HALF>(t.stab + x * HALF, jl, s);
        rotate_row(lo, hi, c, s);
    }
}

// A run with an infinity among its values: it is stored as NaN and does not set
// the scale.  A row at a time, apart from the path below.
template <typename T, int D>
__device__ __noinline__ void append_block_with_inf(const Target& t, int n, int lo_slot, float eps,
                                                   int lane) {
    constexpr int HV = D / 16;
    const int jl = lane % HV, rl = lane / HV;
    float top = 0.f, up = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int x0 = 0; x0 < n; x0 += 32 / HV) {
            const int x = x0 + rl;
            const uint4* row = t.src + min(x, n - 1) * t.src_stride;
            f2 v[2][4];
            unpack<T>(row[jl], v[0]);
            unpack<T>(row[HV + jl], v[1]);
            row_values<T, D>(t, min(x, n - 1), jl, eps, v[0], v[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float p[2];
                    split_f2(v[k][e], p[0], p[1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const bool fin = fabsf(p[c]) <= 3.402823466e38f;
                        if (pass == 0 && fin) top = fmaxf(top, fabsf(p[c]));
                        if (!fin) p[c] = __uint_as_float(0x7fc00000u);
                    }
                    v[k][e] = make_f2(p[0], p[1]);
                }
            if (pass == 1 && x < n) {
                uint2* dst = reinterpret_cast<uint2*>(t.rows + (lo_slot + x) * D);
                dst[jl] = quantise8(v[0], up);
                dst[HV + jl] = quantise8(v[1], up);
            }
        }
        if (pass == 0) {
            top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
            up = exp2i(-settle_scale<D>(t, lo_slot, top, lane));
        }
    }
}

template <int D>
__device__ __forceinline__ Target block_target(const Kv8AppendArgs& a, const Run& r, int h, bool k,
                                               int tok0, const float* ctab, const float* stab,
                                               const float* wk) {
    const long long blk = r.blk + (long long)h * (a.page_size / kChunk);  // [page][head][block]
    Target t;
    t.rows = (k ? a.k_pool : a.v_pool) + blk * (kChunk * D);
    t.scale = a.scales + blk * 2 + (k ? 0 : 1);
    t.src_stride = (long long)a.n_kv_heads * (D / 8);
    t.src = static_cast<const uint4*>(k ? a.k_new : a.v_new) +
            ((long long)r.tok * a.n_kv_heads + h) * (D / 8);
    t.ctab = k && a.rope ? ctab + (r.tok - tok0) * (D / 2) : nullptr;
    t.stab = stab + (r.tok - tok0) * (D / 2);
    t.w = k && a.k_norm_w ? wk : nullptr;
    return t;
}

// One (run, head, side) by a warp; v: its rows, two vectors a lane and pass (the
// elements of a row's lower half, their partners).  They stay packed: what is
// computed from them (the norm, the rotation) is computed twice, for the largest
// element and for the bytes, which costs less than the registers for it would in
// warps at work (64 more a thread).
template <typename T, int D>
__device__ __forceinline__ void append_block(const Target& t, const uint4 (&v)[kVecs], int n,
                                             int slot, float eps, int lane) {
    constexpr int HV = D / 16;        // lanes a row
    constexpr int RPP = 32 / HV;      // rows a pass
    constexpr int PASSES = kChunk / RPP;
    static_assert(2 * PASSES <= kVecs, "a block's rows fit a task");
    const int jl = lane % HV, rl = lane / HV;
    float top = 0.f;
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
        if (ps * RPP >= n) break;  // warp-uniform
        f2 lo[4], hi[4];
        unpack<T>(v[2 * ps], lo);
        unpack<T>(v[2 * ps + 1], hi);
        row_values<T, D>(t, min(ps * RPP + rl, n - 1), jl, eps, lo, hi);
        if (ps * RPP + rl < n) top = max_abs8(hi, max_abs8(lo, top));
    }
    top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
    if (top > 3.402823466e38f) {
        append_block_with_inf<T, D>(t, n, slot, eps, lane);
        return;
    }
    const float up = exp2i(-settle_scale<D>(t, slot, top, lane));
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
        if (ps * RPP >= n) break;  // warp-uniform
        const int x = ps * RPP + rl;
        f2 lo[4], hi[4];
        unpack<T>(v[2 * ps], lo);
        unpack<T>(v[2 * ps + 1], hi);
        row_values<T, D>(t, min(x, n - 1), jl, eps, lo, hi);
        if (x < n) {
            uint2* row = reinterpret_cast<uint2*>(t.rows + (slot + x) * D);
            row[jl] = quantise8(lo, up);
            row[HV + jl] = quantise8(hi, up);
        }
    }
}

// cos / sin tables, weights, and the warps' rings.
template <int D>
constexpr int kSmemBytes = 2 * kMaxSpan * (D / 2) * 4 + 2 * D * 4 + kWarps * kDepth * kVecs * 512;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2)
kv8_append_kernel(const __grid_constant__ Kv8AppendArgs a, int alone, int rest,
                  int parts, uint32_t* status) {
    constexpr int HALF = D / 2, HV = D / 16;
    extern __shared__ __align__(16) uint8_t smem[];  // kSmemBytes<D>
    float* ctab = reinterpret_cast<float*>(smem);
    float* stab = ctab + kMaxSpan * HALF;
    float* wq = stab + kMaxSpan * HALF;
    float* wk = wq + D;
    const uint32_t ring = smem_u32(wk + D) + (threadIdx.x >> 5) * (kDepth * kVecs * 512) +
                          (threadIdx.x & 31) * 16;  // this lane's first vector
    __shared__ int s_pos[kMaxSpan];
    __shared__ Run s_runs[kMaxSpan];
    __shared__ int s_first, s_end, s_nruns;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the CTA's leaders: tokens base .. base + 15, the first `alone` groups of 16 a
    // CTA each, the others `parts`
    const int bx = blockIdx.x, past = bx - alone;
    const int base = (past < 0 ? bx : alone + past % rest) * kSpan;
    const int part = past < 0 ? 0 : past / rest, n_parts = past < 0 ? 1 : parts;

    pdl_wait();
    if (a.q_norm_w || a.k_norm_w) {
        for (int x = tid; x < D; x += kThreads) {
            const T* q = static_cast<const T*>(a.q_norm_w);
            const T* k = static_cast<const T*>(a.k_norm_w);
            const int at = x / HALF * HALF + place<HALF>(x % HALF);
            wq[at] = q ? (float)q[x] : 1.f;
            wk[at] = k ? (float)k[x] : 1.f;
        }
    }
    if (warp == 0) {
        // token base + lane and the one before it; the last one a CTA can own
        // is base + kSpan + 14, so lane 31 sees the next CTA's first leader
        const int i = base + lane;
        const bool in = i < a.n_tokens;
        const int pos = in ? a.positions[i] : -1;
        const int seq = in ? a.seq_ids[i] : -1;
        int ppos = __shfl_up_sync(kFull, pos, 1), pseq = __shfl_up_sync(kFull, seq, 1);
        if (lane == 0) {
            ppos = base > 0 ? a.positions[base - 1] : -1;
            pseq = base > 0 ? a.seq_ids[base - 1] : -1;
        }
        const bool cont = in && pos > 0 && ppos >= 0 && pseq == seq && pos - 1 == ppos &&
                          (pos & (kChunk - 1)) != 0;
        // tokens past the last one end the last run
        const unsigned lead = __ballot_sync(kFull, !cont);
        const int first = __ffs(lead & ((1u << kSpan) - 1u)) - 1;
        const unsigned after = lead >> kSpan << kSpan;
        const int end = min(after ? __ffs(after) - 1 : 32, a.n_tokens - base);
        const bool mine = first >= 0 && lane >= first && lane < end;
        // runs of the CTA: leaders among its tokens that are appended
        bool use = false;
        uint32_t skipped = 0;
        Run r = {0, 0, 0, 0};
        if (mine && !cont && pos >= 0) {
            const unsigned next = lead & ~((2u << lane) - 1u);
            r.tok = i;
            r.n = min(next ? __ffs(next) - 1 : 32, end) - lane;
            r.lo = pos & (kChunk - 1);
            const int col = pos / a.page_size;
            // the positions of one block must form one run: a run that goes on
            // in the block of the token before it is refused
            const bool again = ppos >= 0 && pseq == seq && ppos / kChunk == pos / kChunk;
            uint32_t bits = 0;
            int page = 0;
            if (seq < 0 || seq >= a.n_seqs) bits = PKV_DEV_BAD_SEQ;
            else if (col >= a.table_stride || again) bits = PKV_DEV_BAD_LEN;
            else {
                page = a.table[(long long)seq * a.table_stride + col];
                if (page < 0 || page >= a.num_pages) bits = PKV_DEV_BAD_PAGE;
            }
            use = bits == 0;
            skipped = bits;
            r.blk = (long long)page * a.n_kv_heads * (a.page_size / kChunk) +
                    (pos % a.page_size) / kChunk;
        }
        skipped = __reduce_or_sync(kFull, skipped);
        if (lane == 0 && skipped) set_status(status, skipped);
        const unsigned used = __ballot_sync(kFull, use);
        if (use) s_runs[__popc(used & ((1u << lane) - 1u))] = r;
        if (mine) s_pos[lane - first] = pos;
        if (lane == 0) {
            s_first = first;
            s_end = end;
            s_nruns = __popc(used);
        }
    }
    __syncthreads();
    if (s_first < 0 || s_end <= s_first) return;  // all its tokens belong to the CTA before
    const int tok0 = base + s_first;
    const int ntok = s_end - s_first;
    // a warp's tasks: K and V blocks, then stretches of one token's q rows (which
    // share the token's cos / sin, and the weights, in registers)
    constexpr int RPP = 32 / HV, PASSES = kChunk / RPP, U = kVecs / 2;
    const int per_run = a.n_kv_heads * 2;
    const int blocks = s_nruns * per_run;
    const int stretches = a.q ? (a.n_q_heads + U * RPP - 1) / (U * RPP) : 0;
    const int tasks = blocks + ntok * stretches;
    const int step = kWarps * n_parts, x0 = part * kWarps + warp;
    if (x0 - warp >= tasks) return;
    const int jl = lane % HV, rl = lane / HV;
    auto fetch = [&](int x, int buf) {
        const uint32_t dst = ring + buf * (kVecs * 512);
        if (x < blocks) {
            const int ri = x / per_run, y = x - ri * per_run;
            const Run& r = s_runs[ri];
            const uint4* src = static_cast<const uint4*>(y & 1 ? a.v_new : a.k_new) +
                               ((long long)r.tok * a.n_kv_heads + (y >> 1)) * (D / 8) + jl;
            const long long stride = (long long)a.n_kv_heads * (D / 8);
#pragma unroll
            for (int ps = 0; ps < PASSES; ++ps) {
                const int k = ps * RPP + rl;  // token of the run
                const uint4* row = src + (k < r.n ? k * stride : 0);
                copy_vec(dst + (2 * ps) * 512, row, k < r.n);
                copy_vec(dst + (2 * ps + 1) * 512, row + HV, k < r.n);
            }
        } else if (x < tasks) {
            const int tk = (x - blocks) / stretches;
            const int h0 = (x - blocks - tk * stretches) * (U * RPP) + rl;
            const uint4* src = static_cast<const uint4*>(a.q) +
                               (long long)(tok0 + tk) * a.n_q_heads * (D / 8) + jl;
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int h = h0 + k * RPP;
                const uint4* row = src + (h < a.n_q_heads ? h * (D / 8) : 0);
                copy_vec(dst + (2 * k) * 512, row, h < a.n_q_heads);
                copy_vec(dst + (2 * k + 1) * 512, row + HV, h < a.n_q_heads);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < kDepth; ++k) fetch(x0 + k * step, k);
    if (a.rope) {  // while the first rows come
        for (int x = tid; x < ntok * HALF; x += kThreads) {
            const int tk = x / HALF, i = x - tk * HALF;
            const int at = tk * HALF + place<HALF>(i);
            turn_cos_sin(s_pos[tk], a.turns[i], &ctab[at], &stab[at]);
        }
        __syncthreads();
    }
    int buf = 0;
    for (int x = x0; x < tasks; x += step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        uint4 v[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w)
                         : "r"(ring + (buf * kVecs + k) * 512));
        fetch(x + kDepth * step, buf);
        buf = buf + 1 == kDepth ? 0 : buf + 1;
        if (x < blocks) {
            const int ri = x / per_run, y = x - ri * per_run;
            const Run r = s_runs[ri];
            append_block<T, D>(block_target<D>(a, r, y >> 1, !(y & 1), tok0, ctab, stab, wk), v,
                               r.n, r.lo, a.norm_eps, lane);
            continue;
        }
        const int tk = (x - blocks) / stretches;
        const int h0 = (x - blocks - tk * stretches) * (U * RPP) + rl;
        uint4* qo = static_cast<uint4*>(a.q_out) +
                    (long long)(tok0 + tk) * a.n_q_heads * (D / 8) + jl;
        f2 c[4], sn[4], wlo[4], whi[4];
        if (a.q_norm_w) {
            load8<HALF>(wq, jl, wlo);
            load8<HALF>(wq + HALF, jl, whi);
        }
        if (a.rope) {
            load8<HALF>(ctab + tk * HALF, jl, c);
            load8<HALF>(stab + tk * HALF, jl, sn);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = h0 + k * RPP;
            if (h - rl >= a.n_q_heads) break;  // warp-uniform
            f2 lo[4], hi[4];
            unpack<T>(v[2 * k], lo);
            unpack<T>(v[2 * k + 1], hi);
            if (a.q_norm_w) scale_row(lo, hi, inv_rms<D>(lo, hi, a.norm_eps), wlo, whi);
            if (a.rope) rotate_row(lo, hi, c, sn);
            if (h < a.n_q_heads) {
                qo[h * (D / 8)] = pack<T>(lo);
                qo[h * (D / 8) + HV] = pack<T>(hi);
            }
        }
    }
    pdl_trigger();
}

// One token of every sequence (no seq_ids): every token is a run of its own, so
// nothing has to be found out before its rows are fetched, and D / 16 lanes take a
// row each -- of q, K or V -- instead of a warp a block.  A CTA per token.  What
// bounds it: latency (the position, the page, the block's scale, one after the
// other, with the rows on the way beside them).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2)
kv8_append_single_kernel(const __grid_constant__ Kv8AppendArgs a, uint32_t* status,
                         uint32_t* flags) {
    constexpr int HALF = D / 2, HV = D / 16, GROUPS = kThreads / HV, U = 2;
    __shared__ __align__(16) float ctab[HALF], stab[HALF];
    const int tid = threadIdx.x, lane = tid & 31;
    const int jl = lane % HV, grp = tid / HV;
    const int tok = blockIdx.x;
    pdl_wait();
    pdl_trigger();  // a step's decode works out its ranges beside this
    const int pos = a.positions[tok];
    const int nq = a.q ? a.n_q_heads : 0, rows = nq + 2 * a.n_kv_heads;
    // row r: q heads, then K heads, then V heads
    auto source = [&](int r) -> const uint4* {
        if (r < nq)
            return static_cast<const uint4*>(a.q) + ((long long)tok * nq + r) * (D / 8) + jl;
        const int h = r - nq;
        const bool k = h < a.n_kv_heads;
        return static_cast<const uint4*>(k ? a.k_new : a.v_new) +
               ((long long)tok * a.n_kv_heads + (k ? h : h - a.n_kv_heads)) * (D / 8) + jl;
    };
    uint4 vl[U], vh[U];
    auto fetch = [&](int r0) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int r = r0 + k * GROUPS;
            vl[k] = vh[k] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) {
                const uint4* src = source(r);
                vl[k] = src[0];
                vh[k] = src[HV];
            }
        }
    };
    fetch(grp);
    uint32_t bits = 0;
    long long blk0 = -1;  // the block at head 0; -1: nothing is appended
    if (pos >= 0) {
        const int col = pos / a.page_size;
        int page = -1;
        if (col < a.table_stride) page = a.table[(long long)tok * a.table_stride + col];
        else bits = PKV_DEV_BAD_LEN;
        if (page >= 0 && page < a.num_pages)
            blk0 = (long long)page * a.n_kv_heads * (a.page_size / kChunk) +
                   pos % a.page_size / kChunk;
        else if (!bits) bits = PKV_DEV_BAD_PAGE;
    }
    if (tid == 0) {
        if (flags) flags[blockIdx.x] = bits;
        else if (bits) set_status(status, bits);
    }
    if (a.rope) {
        for (int i = tid; i < HALF; i += kThreads)
            turn_cos_sin(pos, a.turns[i], &ctab[place<HALF>(i)], &stab[place<HALF>(i)]);
        __syncthreads();
    }
    const int slot = pos & (kChunk - 1);
    for (int r0 = grp; r0 - lane / HV < rows; r0 += U * GROUPS) {
        if (r0 != grp) fetch(r0);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int r = r0 + k * GROUPS;
            if (r - lane / HV >= rows) break;  // warp-uniform
            f2 lo[4], hi[4];
            unpack<T>(vl[k], lo);
            unpack<T>(vh[k], hi);
            const bool is_q = r < nq, is_k = !is_q && r < nq + a.n_kv_heads;
            const void* w = is_q ? a.q_norm_w : is_k ? a.k_norm_w : nullptr;
            if (a.q_norm_w || a.k_norm_w) {
                const float inv = inv_rms<D>(lo, hi, a.norm_eps);  // every lane takes part
                if (w) {
                    const T* wt = static_cast<const T*>(w);
                    f2 wlo[4], whi[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        wlo[e] = make_f2((float)wt[8 * jl + 2 * e], (float)wt[8 * jl + 2 * e + 1]);
                        whi[e] = make_f2((float)wt[HALF + 8 * jl + 2 * e],
                                         (float)wt[HALF + 8 * jl + 2 * e + 1]);
                    }
                    scale_row(lo, hi, inv, wlo, whi);
                }
            }
            if (a.rope && (is_q || is_k)) {
                f2 c[4], s[4];
                load8<HALF>(ctab, jl, c);
                load8<HALF>(stab, jl, s);
                rotate_row(lo, hi, c, s);
            }
            float top = max_abs8(hi, max_abs8(lo, 0.f));
#pragma unroll
            for (int o = HV / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            if (__any_sync(kFull, top > 3.402823466e38f && !is_q && r < rows)) {
                // an infinity: stored as NaN, and it does not set the scale
                top = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f2& x = e < 4 ? lo[e & 3] : hi[e & 3];
                    float p[2];
                    split_f2(x, p[0], p[1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (fabsf(p[c]) <= 3.402823466e38f) top = fmaxf(top, fabsf(p[c]));
                        else if (!is_q) p[c] = __uint_as_float(0x7fc00000u);
                    }
                    x = make_f2(p[0], p[1]);
                }
#pragma unroll
                for (int o = HV / 2; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            }
            if (is_q) {
                uint4* dst = static_cast<uint4*>(a.q_out) +
                             ((long long)tok * nq + r) * (D / 8) + jl;
                dst[0] = pack<T>(lo);
                dst[HV] = pack<T>(hi);
            }
            const bool put = !is_q && r < rows && blk0 >= 0;
            const int h = is_k ? r - nq : r - nq - a.n_kv_heads;
            const long long blk = blk0 + (long long)h * (a.page_size / kChunk);
            uint8_t* block = (is_k ? a.k_pool : a.v_pool) + (put ? blk * (kChunk * D) : 0);
            uint8_t* scale = a.scales + (put ? blk * 2 + (is_k ? 0 : 1) : 0);
            int e = kv8_need_exp(top);
            if (put && slot > 0) {
                const int old = kv8_clamp_exp((int)*scale - 127);
                if (e > old) {  // as settle_scale
                    const float f = exp2i(old - e);
                    uint32_t* p = reinterpret_cast<uint32_t*>(block);
                    for (int x = jl; x < slot * D / 4; x += HV) {
                        uint32_t h0, h1;
                        e4m3x4_to_h2(p[x], h0, h1);
                        const float2 y = __half22float2(*reinterpret_cast<__half2*>(&h0));
                        const float2 z = __half22float2(*reinterpret_cast<__half2*>(&h1));
                        p[x] = f2_to_e4m3x2(y.x * f, y.y * f) | f2_to_e4m3x2(z.x * f, z.y * f) << 16;
                    }
                } else {
                    e = old;
                }
            }
            __syncwarp();  // a row's lanes have read the old scale
            if (put) {
                if (jl == 0) *scale = (uint8_t)(e + 127);
                uint2* row = reinterpret_cast<uint2*>(block + slot * D);
                const float up = exp2i(-e);
                row[jl] = quantise8(lo, up);
                row[HV + jl] = quantise8(hi, up);
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, int head_dim, uint32_t* status,
                              uint32_t* flags, cudaStream_t stream) {
    if (a.n_tokens <= 0) return cudaSuccess;
    if (!a.seq_ids) {
#define PKV_KV8_SINGLE(T, D)                                                                  \
    return launch_pdl(kv8_append_single_kernel<T, D>, dim3((unsigned)a.n_tokens), dim3(kThreads), \
                      0, stream, a, status, flags)
        if (a.bf16) {
            if (head_dim == 128) PKV_KV8_SINGLE(__nv_bfloat16, 128);
            PKV_KV8_SINGLE(__nv_bfloat16, 64);
        }
        if (head_dim == 128) PKV_KV8_SINGLE(__half, 128);
        PKV_KV8_SINGLE(__half, 64);
#undef PKV_KV8_SINGLE
    }
    // Groups of 16 tokens: as many as fill the device once or several times have a CTA
    // each; the rest, or all when they are fewer, share what it holds, twice over:
    // several CTAs to a group, up to a task a warp where every token is a run of its
    // own, behind groups with a CTA each two tasks of a prompt's.  (8 prompts, 32/8 heads
    // of 128, norm and rotation, us with 1 / 2 / 4 / 8 CTAs to every group, and by this
    // rule: 567 tokens 29.4 / 16.5 / 10.5 / 9.2, 8.5; 1485: 29.2 / 17.9 / 14.9 / 15.5, 15.3;
    // 4095: 34.3 / 28.9 / 30.7 / 35.0, 29.0; 8192: 48.9 / 47.9 / 53.4 / 65.0, 44.1; 14433:
    // 68.7 / 73.3 / 88.0 / 109.2, 65.8: each forms the angles of its tokens again.  Of those
    // 14433, no norm and no rotation: 24.9 / 29.7 / 38.5 / 53.4, 24.8; D = 64, 16/2
    // heads: 24.1 / 30.3 / 41.4 / 56.7, 24.1.)
    const int groups = a.n_tokens / kSpan + (a.n_tokens % kSpan ? 1 : 0);
    const int alone = groups / kSlots * kSlots, rest = groups - alone;
    const int stretch = kVecs / 2 * (32 / (head_dim / 16));  // q rows of a task
    const long long per_tok = a.q ? (a.n_q_heads + stretch - 1) / stretch : 0;
    const long long most =
        alone ? (2LL * a.n_kv_heads + kSpan * per_tok) / (2 * kWarps)
              : (kSpan * (2LL * a.n_kv_heads + per_tok) + kWarps - 1) / kWarps;
    const int parts =
        rest ? (int)std::max(1LL, std::min(most, (long long)(2 * kSlots / rest))) : 1;
    const dim3 grid((unsigned)(alone + rest * parts));
    // more shared memory than a kernel has unasked (cheap, and per device: asked
    // for with every launch)
#define PKV_KV8_APPEND(T, D)                                                                     \
    do {                                                                                         \
        const cudaError_t e = cudaFuncSetAttribute(kv8_append_kernel<T, D>,                      \
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,  \
                                                   kSmemBytes<D>);                               \
        if (e != cudaSuccess) return e;                                                          \
        return launch_pdl(kv8_append_kernel<T, D>, grid, dim3(kThreads), kSmemBytes<D>, stream,  \
                          a, alone, rest, parts, status);                                        \
    } while (0)
    if (a.bf16) {
        if (head_dim == 128) PKV_KV8_APPEND(__nv_bfloat16, 128);
        PKV_KV8_APPEND(__nv_bfloat16, 64);
    }
    if (head_dim == 128) PKV_KV8_APPEND(__half, 128);
    PKV_KV8_APPEND(__half, 64);
#undef PKV_KV8_APPEND
}

}  // namespace pkv
