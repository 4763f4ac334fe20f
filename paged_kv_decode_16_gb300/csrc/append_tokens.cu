// append_tokens.cu -- rotary embedding of new tokens' q and k in every form, and
// the write of k and v into their slots.
//
// One pass over the rows: a task is two 16-byte vectors of one row that turn together
// (half layout: vector j and vector j + rotary_dim / 16, elements i and i + rotary_dim
// / 2; interleaved: two neighbouring vectors), so that no lane needs another's elements,
// and in both layouts the task's eight cosines and sines are those of pairs 8 j .. 8 j +
// 7.  The D / 16 tasks of a row lie on neighbouring lanes, which is where the optional
// norm sums its squares.  cos and sin are worked out once a token, into shared memory,
// behind the loads of the CTA's first tasks.
//
// What bounds it: memory, 2 bytes read and 2 written an element.
#include "selected.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // tokens of a CTA
constexpr int kBatch = 3;      // tasks of a thread whose loads are in flight together

template <typename T>
__device__ __forceinline__ void pack8(const float (&f)[8], uint4& v) {
    v.x = Cvt<T>::pack2(f[0], f[1]);
    v.y = Cvt<T>::pack2(f[2], f[3]);
    v.z = Cvt<T>::pack2(f[4], f[5]);
    v.w = Cvt<T>::pack2(f[6], f[7]);
}

// (x, y) turned by the angle of (c, s).
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
    const float a = x * c - y * s;
    y = y * c + x * s;
    x = a;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
append_tokens_kernel(const AppendTokensArgs a, int tokens_per_cta) {
    constexpr int kTasks = D / 16;  // of a row
    __shared__ __align__(16) float s_cos[kMaxTokens][64];
    __shared__ __align__(16) float s_sin[kMaxTokens][64];
    __shared__ long long s_slot[kMaxTokens];
    __shared__ int s_pos[kMaxTokens];

    const int t0 = blockIdx.x * tokens_per_cta;
    const int nt = min(tokens_per_cta, a.n_tokens - t0);
    const int rows = a.n_q_heads + 2 * a.n_kv_heads;
    const int per_token = rows * kTasks;
    const int n = nt * per_token;
    const bool rope = a.positions != nullptr;
    const bool normed = a.q_norm || a.k_norm;
    const int pairs = rope ? a.rope.rotary_dim >> 1 : 0;
    const int turning = rope ? a.rope.rotary_dim >> 4 : 0;  // tasks of a row that turn

    pdl_wait();
    pdl_trigger();
    if (threadIdx.x < nt) {
        long long s = a.slots[t0 + threadIdx.x];
        const int p = rope ? a.positions[t0 + threadIdx.x] : 0;
        uint32_t bits = 0;
        if (s >= a.n_slots) {
            bits = PKV_DEV_BAD_PAGE;
            s = -1;
        }
        if (p < 0) s = -1;
        s_slot[threadIdx.x] = s;
        s_pos[threadIdx.x] = p;
        if (bits) set_status(a.status, bits);
    }

    bool table = false;  // the CTA's cosines and sines are there
    for (int base = 0; base < n; base += kThreads * kBatch) {
        uint4 x[kBatch], y[kBatch];
        int tok[kBatch], row[kBatch], at[kBatch], v0[kBatch], v1[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int task = base + u * kThreads + threadIdx.x;
            const bool in = task < n;
            const int tk = in ? task / per_token : 0;
            const int rem = in ? task - tk * per_token : 0;
            const int r = rem / kTasks, j = rem % kTasks;
            tok[u] = in ? tk : -1;
            row[u] = r;
            at[u] = j;
            // the task's two vectors
            if (a.rope.interleaved || j >= turning) {
                v0[u] = 2 * j;
                v1[u] = 2 * j + 1;
            } else {
                v0[u] = j;
                v1[u] = j + turning;
            }
            if (!in) continue;
            const T* src;
            const long long t = t0 + tk;
            if (r < a.n_q_heads)
                src = static_cast<const T*>(a.q) + t * a.q_stride + r * D;
            else if (r < a.n_q_heads + a.n_kv_heads)
                src = static_cast<const T*>(a.k) + t * a.k_stride + (r - a.n_q_heads) * D;
            else
                src = static_cast<const T*>(a.v) + t * a.v_stride +
                      (r - a.n_q_heads - a.n_kv_heads) * D;
            x[u] = *reinterpret_cast<const uint4*>(src + v0[u] * 8);
            y[u] = *reinterpret_cast<const uint4*>(src + v1[u] * 8);
        }
        if (!table) {
            table = true;
            __syncthreads();
            for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
                const int tk = i / pairs, p = i - tk * pairs;
                // the turns' product wraps modulo one turn by itself; its top 32 bits as a
                // signed fraction of half a turn give the angle to 2^-32 turns
                const uint64_t ph = (uint64_t)(int64_t)s_pos[tk] * a.rope.turns[p];
                float s, c;
                sincospif((float)(int)(ph >> 32) * 4.6566128730773926e-10f, &s, &c);
                s_cos[tk][p] = c * a.rope.magnitude;
                s_sin[tk][p] = s * a.rope.magnitude;
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int tk = max(tok[u], 0), r = row[u], j = at[u];
            const bool is_q = r < a.n_q_heads, is_k = !is_q && r < a.n_q_heads + a.n_kv_heads;
            const bool turn = (is_q || is_k) && j < turning;
            const void* norm = is_q ? a.q_norm : (is_k ? a.k_norm : nullptr);
            float f[8], g[8];
            if (turn || normed) {
                Cvt<T>::unpack8(x[u], f);
                Cvt<T>::unpack8(y[u], g);
            }
            if (normed) {  // the same for the whole grid: every lane shuffles
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(f[e], f[e], fmaf(g[e], g[e], sum));
#pragma unroll
                for (int o = kTasks / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
                if (norm) {
                    const float inv = 1.0f / sqrtf(sum / (float)D + a.eps);
                    float w[8], z[8];
                    Cvt<T>::unpack8(reinterpret_cast<const uint4*>(norm)[v0[u]], w);
                    Cvt<T>::unpack8(reinterpret_cast<const uint4*>(norm)[v1[u]], z);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f[e] = f[e] * inv * w[e];
                        g[e] = g[e] * inv * z[e];
                    }
                }
            }
            if (turn) {
                float c[8], s[8];
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 c4 = *reinterpret_cast<const float4*>(&s_cos[tk][8 * j + e]);
                    const float4 s4 = *reinterpret_cast<const float4*>(&s_sin[tk][8 * j + e]);
                    c[e] = c4.x, c[e + 1] = c4.y, c[e + 2] = c4.z, c[e + 3] = c4.w;
                    s[e] = s4.x, s[e + 1] = s4.y, s[e + 2] = s4.z, s[e + 3] = s4.w;
                }
                if (a.rope.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        turn_pair(f[2 * e], f[2 * e + 1], c[e], s[e]);
                        turn_pair(g[2 * e], g[2 * e + 1], c[4 + e], s[4 + e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) turn_pair(f[e], g[e], c[e], s[e]);
                }
            }
            if (turn || norm) {
                pack8<T>(f, x[u]);
                pack8<T>(g, y[u]);
            }
            if (tok[u] < 0) continue;
            T* dst = nullptr;
            if (is_q) {
                if (s_pos[tk] >= 0)
                    dst = static_cast<T*>(a.q_out) + (long long)(t0 + tk) * a.q_out_stride + r * D;
            } else if (s_slot[tk] >= 0) {
                const long long slot = s_slot[tk], page = slot / a.page_size;
                const int h = r - a.n_q_heads - (is_k ? 0 : a.n_kv_heads);
                const long long to =
                    ((page * a.n_kv_heads + h) * a.page_size + (slot - page * a.page_size)) * D;
                dst = static_cast<T*>(is_k ? a.k_pool : a.v_pool) + to;
            }
            if (dst) {
                *reinterpret_cast<uint4*>(dst + v0[u] * 8) = x[u];
                *reinterpret_cast<uint4*>(dst + v1[u] * 8) = y[u];
            }
        }
    }
}

template <typename T>
cudaError_t launch(const AppendTokensArgs& a, int head_dim, cudaStream_t stream) {
    // a CTA a token while that fills the SMs, then up to kMaxTokens
    int per = (a.n_tokens + 607) / 608;
    per = per < 1 ? 1 : (per > kMaxTokens ? kMaxTokens : per);
    const dim3 grid((a.n_tokens + per - 1) / per);
    return launch_pdl(head_dim == 128 ? append_tokens_kernel<T, 128> : append_tokens_kernel<T, 64>,
                      grid, dim3(kThreads), 0, stream, a, per);
}

}  // namespace

cudaError_t launch_append_tokens(const AppendTokensArgs& a, bool bf16, int head_dim,
                                 cudaStream_t stream) {
    return bf16 ? launch<__nv_bfloat16>(a, head_dim, stream) : launch<__half>(a, head_dim, stream);
}

}  // namespace pkv
