// Attention of a chunk of new tokens per request over the paged cache: the
// prompt's (and plain decoding's) counterpart of the block attention.  Row i
// of request b is the token at position kv_len[b] + i; its K/V row goes to
// its page and it attends to every key at a position <= its own.
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch.h"
#include "plan.h"

namespace isd {

namespace {

struct ChunkArgs {
    int B, T, Hq, Hkv, grp, P, num_pages, max_pages;
    float scale_log2;
    const int32_t* page_table;
    const int32_t* kv_len;
    const int32_t* q_start;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_new;
    const __nv_bfloat16* v_new;
    __nv_bfloat16* k_pool;
    __nv_bfloat16* v_pool;
    __nv_bfloat16* out;
    int32_t* err_flag;
};

constexpr int kAppendTokens = 8;  // tokens (warps) per append CTA

// New tokens of request b if its page list can hold them, else 0 (negative
// or over-capacity length).  q_start is known to ascend within [0, T].
ISD_DEVINL int chunk_tokens(const ChunkArgs& a, int b, int kv, int n) {
    if (kv < 0) return 0;
    const long long t = (long long)kv + n;
    return (t + a.P - 1) / a.P > a.max_pages ? 0 : n;
}

// Whether q_start ascends within [0, T] (every thread of the CTA gets the answer).
ISD_DEVINL bool chunk_starts_ok(const ChunkArgs& a) {
    bool bad = false;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const int s = a.q_start[b], e = a.q_start[b + 1];
        bad |= s < 0 || e < s || e > a.T;
    }
    return !__syncthreads_or(bad);
}

// The request of token t (a warp asks together): the last b with
// q_start[b] <= t, or -1 for a row of no request.
ISD_DEVINL int chunk_request(const ChunkArgs& a, int t) {
    const int lane = threadIdx.x & 31;
    int count = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        count += __popc(__ballot_sync(0xffffffffu, b < a.B && a.q_start[b] <= t));
    }
    const int b = count - 1;
    return b >= 0 && t < a.q_start[b + 1] ? b : -1;
}

// One warp per token: its K and V rows go into their page, 16 bytes per lane
// and step; a request that cannot be served gets zero output rows.
template <int D>
__global__ void __launch_bounds__(32 * kAppendTokens) chunk_append_kernel(const __grid_constant__ ChunkArgs a) {
    const bool ok = chunk_starts_ok(a);
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_flag(a.err_flag, ISD_FLAG_CHUNK_RANGE);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kAppendTokens + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int b = chunk_request(a, t);
    if (b < 0) return;
    const int start = a.q_start[b], kv = a.kv_len[b];
    if (chunk_tokens(a, b, kv, a.q_start[b + 1] - start) == 0) {
        if (lane == 0) raise_flag(a.err_flag, ISD_FLAG_CAPACITY);
        uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)t * a.Hq * D);
        for (int i = lane; i < a.Hq * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int pos = kv + (t - start);
    const int page = a.page_table[(size_t)b * a.max_pages + pos / a.P];
    if (page < 0 || page >= a.num_pages) {
        if (lane == 0) raise_flag(a.err_flag, ISD_FLAG_PAGE_OOB);
        return;
    }
    const size_t dst = ((size_t)page * a.P + pos % a.P) * a.Hkv * D, src = (size_t)t * a.Hkv * D;
    for (int i = lane; i < a.Hkv * D / 8; i += 32) {
        reinterpret_cast<uint4*>(a.k_pool + dst)[i] = reinterpret_cast<const uint4*>(a.k_new + src)[i];
        reinterpret_cast<uint4*>(a.v_pool + dst)[i] = reinterpret_cast<const uint4*>(a.v_new + src)[i];
    }
}

// One warp per (token, query head); each lane owns D / 32 dimensions and the
// warp walks the visible keys with a running maximum and sum.
template <int D>
__global__ void __launch_bounds__(128) chunk_attention_kernel(const __grid_constant__ ChunkArgs a) {
    constexpr int E = D / 32;
    if (!chunk_starts_ok(a)) return;
    const int lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (id >= (long long)a.T * a.Hq) return;
    const int t = (int)(id / a.Hq), h = (int)(id % a.Hq), g = h / a.grp;
    const int b = chunk_request(a, t);
    if (b < 0) return;
    const int start = a.q_start[b], kv = a.kv_len[b];
    if (chunk_tokens(a, b, kv, a.q_start[b + 1] - start) == 0) return;
    float qv[E], o[E];
    for (int e = 0; e < E; ++e) {
        qv[e] = __bfloat162float(a.q[((size_t)t * a.Hq + h) * D + lane * E + e]);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int last = kv + (t - start);
    for (int key = 0; key <= last; ++key) {
        const int page = a.page_table[(size_t)b * a.max_pages + key / a.P];
        const bool bad = page < 0 || page >= a.num_pages;
        if (bad && lane == 0) raise_flag(a.err_flag, ISD_FLAG_PAGE_OOB);
        const size_t row = bad ? 0 : (((size_t)page * a.P + key % a.P) * a.Hkv + g) * D + lane * E;
        float s = 0.f, v[E];
        for (int e = 0; e < E; ++e) {
            s += bad ? 0.f : qv[e] * __bfloat162float(a.k_pool[row + e]);
            v[e] = bad ? 0.f : __bfloat162float(a.v_pool[row + e]);
        }
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.scale_log2;
        const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - mu), p = exp2f(s - mu);
        l = l * f + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * v[e];
        m = mn;
    }
    for (int e = 0; e < E; ++e)
        a.out[((size_t)t * a.Hq + h) * D + lane * E + e] = __float2bfloat16_rn(o[e] / l);
}

template <int D>
cudaError_t launch_chunk_d(const ChunkArgs& a, cudaStream_t st) {
    cudaError_t e = launch_kernel(false, chunk_append_kernel<D>, dim3((a.T + kAppendTokens - 1) / kAppendTokens),
                                  dim3(32 * kAppendTokens), 0, st, a);
    if (e != cudaSuccess) return e;
    const long long warps = (long long)a.T * a.Hq;
    return launch_kernel(false, chunk_attention_kernel<D>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st, a);
}

}  // namespace

cudaError_t launch_chunk_attention(const isd_dims* d, int T, const uint16_t* q, const uint16_t* k_new,
                                   const uint16_t* v_new, uint16_t* k_pool, uint16_t* v_pool,
                                   const int32_t* page_table, const int32_t* kv_len,
                                   const int32_t* q_start, uint16_t* out, void* ws, int32_t* err_flag,
                                   cudaStream_t st) {
    ChunkArgs a;
    a.B = d->B;
    a.T = T;
    a.Hq = d->Hq;
    a.Hkv = d->Hkv;
    a.grp = d->Hq / d->Hkv;
    a.P = d->page_size;
    a.num_pages = d->num_pages;
    a.max_pages = d->max_pages_per_req;
    a.scale_log2 = d->sm_scale * 1.4426950408889634f;
    a.page_table = page_table;
    a.kv_len = kv_len;
    a.q_start = q_start;
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.k_new = reinterpret_cast<const __nv_bfloat16*>(k_new);
    a.v_new = reinterpret_cast<const __nv_bfloat16*>(v_new);
    a.k_pool = reinterpret_cast<__nv_bfloat16*>(k_pool);
    a.v_pool = reinterpret_cast<__nv_bfloat16*>(v_pool);
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.err_flag = err_flag;
    (void)ws;
    return d->D == 64 ? launch_chunk_d<64>(a, st) : launch_chunk_d<128>(a, st);
}

}  // namespace isd
