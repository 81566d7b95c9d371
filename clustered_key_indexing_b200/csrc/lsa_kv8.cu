// lsa_kv8.cu -- the paged 8-bit K/V cache: writing tokens into its pages and
// copying pages [essay "《卡片柜》" (zhichai.net), ch. 8: the method stacks with
// FP8 / INT quantisation; the bucket cache decides which keys are read, this
// cache is what they are read from].
//
// A page holds `page` consecutive tokens of one sequence, per kv-head as
// [page, 128] codes, so the codes of one (page, head) are contiguous and a
// token's row is one 128-byte line.  Its scale is a power of two: dividing by
// it and multiplying with it are exact, a code is the only rounding, and an
// e4m3 code keeps its bits when the scale of an open page grows (unless the
// value falls into the format's subnormal range).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <algorithm>

#include "lsa_common.cuh"
#include "lsa_mma.cuh"

namespace lsa {

constexpr int kKv8MinExp = -100;  // exponent of an all-zero page's scale

// Exponent of the smallest power of two 2^e, e >= kKv8MinExp, with
// amax <= 2^e * QMAX, from amax's bf16 magnitude bits (8 exponent, 7 mantissa
// bits): QMAX = 448 = 1.75 * 2^8 (mantissa 96), 127 = 1.984375 * 2^6 (126).
// int8 ends at 2^121: 127 of it is within half a step of bf16's largest, while
// 64 times 2^122 would be 2^128.
template <int FMT>
__device__ __forceinline__ int kv8_exp(uint32_t m) {
    const int E = (int)(m >> 7) - 127, f = (int)(m & 127u);
    const int e = FMT == 0 ? E - 8 + (f > 96) : min(E - 6 + (f > 126), 121);
    return m == 0u || e < kKv8MinExp ? kKv8MinExp : e;
}

// Magnitude bits from which on int8's codes need a clamp: bf16's largest, which
// is 127.5 times 2^121.
constexpr uint32_t kKv8Ends = 0x7F7Fu;

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four values already divided by the scale to four codes (round to nearest
// even, saturating; NaN becomes the NaN code, or 0 in int8).
template <int FMT>
__device__ __forceinline__ uint32_t kv8_pack4(float a, float b, float c, float d) {
    if constexpr (FMT == 0) {
        uint32_t r;
        asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n"
            " cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}\n"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return r;
    } else {
        auto q = [](float x) -> uint32_t { return (uint32_t)max(-127, min(127, __float2int_rn(x))) & 255u; };
        return q(a) | (q(b) << 8) | (q(c) << 16) | (q(d) << 24);
    }
}

// The same for finite values within the format's range (below kKv8Ends).
template <int FMT>
__device__ __forceinline__ uint32_t kv8_pack4_finite(float a, float b, float c, float d) {
    if constexpr (FMT == 0) {
        return kv8_pack4<0>(a, b, c, d);
    } else {
        // adding 1.5 * 2^23 leaves the integer nearest (ties to even) in the low bits
        auto q = [](float x) -> uint32_t { return __float_as_uint(x + 12582912.f); };
        return __byte_perm(__byte_perm(q(a), q(b), 0x0040), __byte_perm(q(c), q(d), 0x0040), 0x5410);
    }
}

// Four e4m3 codes at the scale 2^120, where 256 and more would not be finite in
// fp32: magnitudes of 240 (0x77) at most, NaN (0x7F) stays.
__device__ __forceinline__ uint32_t kv8_cap4(uint32_t w) {
    const uint32_t m = w & 0x7F7F7F7Fu, over = __vcmpgtu4(m, 0x77777777u) & ~__vcmpeq4(m, 0x7F7F7F7Fu);
    return (w & ~over) | (((w & 0x80808080u) | 0x77777777u) & over);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The values of four codes (without their scale), exact.
template <int FMT>
__device__ __forceinline__ void kv8_unpack4(uint32_t w, float (&x)[4]) {
    if constexpr (FMT == 0) {
        const uint32_t lo = e4m3x2_to_f16x2(w & 0xFFFFu), hi = e4m3x2_to_f16x2(w >> 16);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
    }
}

constexpr int kKv8Warps = 8;  // warps of a CTA

// Sum of v over the CTA's threads before this one, and over all of them.
template <int WARPS = kKv8Warps>
__device__ __forceinline__ long long kv8_block_scan(long long v, long long& all) {
    __shared__ long long wsum[WARPS];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    long long inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += up;
    }
    if (lane == 31) wsum[wid] = inc;
    __syncthreads();
    long long before = inc - v;
    all = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        if (i < wid) before += wsum[i];
        all += wsum[i];
    }
    __syncthreads();
    return before;
}

struct Kv8WriteArgs {
    const uint16_t* K;       // new rows [n_tokens, hkv, 128], token rows k_stride / v_stride elements apart
    const uint16_t* V;
    int64_t k_stride, v_stride;
    uint8_t* Kp;             // codes [n_pages, hkv, page, 128]
    uint8_t* Vp;
    float* scale;            // [n_pages, hkv, 2]
    const int32_t* cu;       // [n_seq + 1], NULL: one token per sequence
    const int32_t* start;    // [n_seq], NULL: one sequence, all n_tokens from position 0 on
    const int32_t* table;    // [n_seq, max_pages]
    int64_t n_tokens, n_pages;
    int32_t n_seq, max_pages, hkv;
};

// New tokens of sequence b: rows [q0, q0 + n) of the call, at positions
// [s0, s0 + n).  A range that does not fit the call or the table (or 31 bits)
// is reported and counts as empty.
__device__ __forceinline__ void kv8_new_tokens(const Kv8WriteArgs& a, int b, int page, int& q0, int& n, int& s0) {
    q0 = a.cu ? a.cu[b] : b;
    const int64_t m = a.cu ? (int64_t)a.cu[b + 1] - q0 : a.start ? 1 : a.n_tokens;
    s0 = a.start ? a.start[b] : 0;
    n = (int)m;
    if (m == 0) return;
    const int64_t room = min((int64_t)a.max_pages * page, (int64_t)0x7FFFFFFF);
    if (q0 < 0 || m < 0 || q0 + m > a.n_tokens || s0 < 0 || s0 + m > room) {
        raise_device_error(kErrKv8Range);
        n = 0;
    }
}

// One CTA per (page the call touches, group of kv-heads): K and V of as many
// heads as fit 32 registers a thread (pages of 128 and 256 tokens: of one head
// either K or V, blockIdx.y tells which).  The new rows are held (16 rows a
// pass, 16 lanes of 16 bytes a row) between the pass that finds their largest
// magnitude and the one that writes their codes, so HBM sees each input once
// and each code once.  The heads of a page are neighbours in the grid: together
// they read whole token rows.  Every CTA finds its page by a scan over the
// sequences' page counts.  Bound by HBM: 128K tokens of 8 heads took 140 us with
// five CTAs an SM, 162 with the four that the compiler's registers left; 121 us
// (6.65 TB/s) with the maximum taken two values at a time.
__host__ __device__ constexpr int kv8_write_heads(int passes) { return passes >= 4 ? 1 : 4 / passes; }

template <int FMT, int PASSES>
__global__ void __launch_bounds__(256, PASSES <= 8 ? 5 : 2) kv8_write_kernel(Kv8WriteArgs a) {
    constexpr int page = 16 * PASSES, HEADS = kv8_write_heads(PASSES);
    constexpr int NKV = PASSES <= 4 ? 2 : 1, N = HEADS * NKV;  // tensors of this CTA: head j / NKV's K and V in turn
    __shared__ uint32_t s_max[N][8];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int groups = (a.hkv + HEADS - 1) / HEADS;
    const int item = (int)(blockIdx.x / groups);
    const int h0 = (int)(blockIdx.x % groups) * HEADS;
    auto head = [&](int j) { return h0 + j / NKV; };
    auto is_v = [&](int j) { return NKV == 2 ? (j & 1) : (int)blockIdx.y; };
    // the page: sequence s_at[0]'s page s_at[1], which the new tokens from
    // position s_at[4] on touch, s_at[3] of them, the first row s_at[2] of the call
    __shared__ int s_at[5];
    auto found = [&](int b, int pg, int q0, int n, int p0) { s_at[0] = b; s_at[1] = pg; s_at[2] = q0; s_at[3] = n; s_at[4] = p0; };
    int q0 = 0, n = 0, p0 = 0;
    auto pages = [&]() { return n > 0 ? (p0 + n - 1) / page - p0 / page + 1 : 0; };
    if (tid == 0) s_at[0] = -1;
    if (a.cu == nullptr) {  // one token per sequence (touched page b is sequence b's) or one sequence's first pages
        if (tid == 0) {
            const int b = a.start ? item : 0;
            kv8_new_tokens(a, b, page, q0, n, p0);
            if (n > 0) found(b, a.start ? p0 / page : item, q0, n, p0);
        }
    } else if (a.n_seq <= 32) {  // one warp, a sequence a lane
        if (wid == 0) {
            if (lane < a.n_seq) kv8_new_tokens(a, lane, page, q0, n, p0);
            const int m = pages();
            int inc = m;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += up;
            }
            const int k = item - (inc - m);
            __syncwarp();
            if (k >= 0 && k < m) found(lane, p0 / page + k, q0, n, p0);
        }
    } else {
        long long base = 0;
        for (int b0 = 0; b0 < a.n_seq && base <= item; b0 += 256) {  // uniform: every thread holds the same base
            const int b = b0 + tid;
            q0 = n = p0 = 0;
            if (b < a.n_seq) kv8_new_tokens(a, b, page, q0, n, p0);
            const int m = pages();
            long long all;
            const long long k = item - (base + kv8_block_scan(m, all));
            if (k >= 0 && k < m) found(b, p0 / page + (int)k, q0, n, p0);
            base += all;
        }
    }
    __syncthreads();
    const int seq = s_at[0], pg = s_at[1];
    if (seq < 0) return;
    const int first = pg * page - s_at[4];                   // the page's first row, counted from the first new token
    const int r0 = max(0, -first);                           // rows below r0 were written before
    const int r1 = (int)min((int64_t)page, (int64_t)s_at[3] - first);
    const int rr = tid >> 4, c = tid & 15;

    uint4 x[N][PASSES];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int64_t stride = is_v(j) ? a.v_stride : a.k_stride;
        const uint16_t* src = (is_v(j) ? a.V : a.K) + ((int64_t)s_at[2] + first) * stride + (int64_t)head(j) * kD;  // row 0 of the page
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int r = 16 * i + rr;
            x[j][i] = make_uint4(0u, 0u, 0u, 0u);
            if (r >= r0 && r < r1 && head(j) < a.hkv) x[j][i] = __ldg(reinterpret_cast<const uint4*>(src + r * stride + c * 8));
        }
    }
    const int64_t pid = a.table[(int64_t)seq * a.max_pages + pg];
    if (pid < 0 || pid >= a.n_pages) {
        if (tid == 0) raise_device_error(kErrKv8Page);
        return;
    }
    float* sp = a.scale + pid * a.hkv * 2;
    float old[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        old[j] = r0 > 0 && head(j) < a.hkv ? sp[head(j) * 2 + is_v(j)] : 0.f;
        uint32_t m2 = 0u;  // magnitudes order as integers; infinities and NaN are above all finite ones
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            m2 = max_u16x2(m2, max_u16x2(x[j][i].x & 0x7FFF7FFFu, x[j][i].y & 0x7FFF7FFFu));
            m2 = max_u16x2(m2, max_u16x2(x[j][i].z & 0x7FFF7FFFu, x[j][i].w & 0x7FFF7FFFu));
        }
        uint32_t mx = max(m2 & 0xFFFFu, m2 >> 16);
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0) s_max[j][wid] = mx;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (head(j) >= a.hkv) continue;
        uint8_t* dst = (is_v(j) ? a.Vp : a.Kp) + (pid * a.hkv + head(j)) * (int64_t)page * kD;
        uint32_t mx = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = max(mx, s_max[j][i]);
        const bool finite = mx < kKv8Ends;
        if (!finite) {  // infinities, NaN or nearly: the largest finite magnitude
            mx = 0u;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const uint32_t w[4] = {x[j][i].x, x[j][i].y, x[j][i].z, x[j][i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
                    mx = max(mx, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                }
            }
            mx = __reduce_max_sync(0xffffffffu, mx);
            __syncthreads();  // s_max[j] has been read
            if (lane == 0) s_max[j][wid] = mx;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) mx = max(mx, s_max[j][i]);
        }
        const int e = kv8_exp<FMT>(mx);
        const float need = pow2f(e);
        if (r0 > 0 && need > old[j]) {
            // the open page's scale grows: its kept rows move to the new one
            const float f = old[j] * pow2f(-e);
            for (int i = tid; i < r0 * (kD / 4); i += 256) {
                uint32_t* p = reinterpret_cast<uint32_t*>(dst) + i;
                float y[4];
                kv8_unpack4<FMT>(*p, y);
                *p = kv8_pack4<FMT>(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
            }
        }
        const float s = r0 > 0 ? fmaxf(need, old[j]) : need;
        const float inv = r0 > 0 && old[j] >= need ? 1.0f / old[j] : pow2f(-e);  // a power of two: exact
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int r = 16 * i + rr;
            if (r < r0 || r >= r1) continue;
            const uint32_t w[4] = {x[j][i].x, x[j][i].y, x[j][i].z, x[j][i].w};
            float y[8];
#pragma unroll
            for (int e2 = 0; e2 < 4; ++e2) {
                y[2 * e2] = __uint_as_float(w[e2] << 16) * inv;
                y[2 * e2 + 1] = __uint_as_float(w[e2] & 0xFFFF0000u) * inv;
            }
            uint2 w8 = finite ? make_uint2(kv8_pack4_finite<FMT>(y[0], y[1], y[2], y[3]), kv8_pack4_finite<FMT>(y[4], y[5], y[6], y[7]))
                              : make_uint2(kv8_pack4<FMT>(y[0], y[1], y[2], y[3]), kv8_pack4<FMT>(y[4], y[5], y[6], y[7]));
            if (FMT == 0 && s >= 0x1p120f) w8 = make_uint2(kv8_cap4(w8.x), kv8_cap4(w8.y));
            *reinterpret_cast<uint2*>(dst + r * kD + c * 8) = w8;
        }
        if (tid == 0) sp[head(j) * 2 + is_v(j)] = s;
    }
}

// Page copies.  The pairs travel in the launch's own arguments: no upload, and
// a captured launch keeps them; up to 4000 a launch (2000 at a time cost 4 to 8
// us more for 4096).  One CTA moves 16 KB: a part of one page's K or V, or of
// small pages as many as fit (4000 pairs of 2 KB: 8.1 us, 10.1 with a CTA for
// each); the CTA with a page's first part also moves its scales.  4096 pages of
// 64 tokens and 8 heads (0.54 GB read and written) take 168 us on the GPU, 6.4 TB/s;
// a CTA's share of 8 to 64 KB, or cached loads and stores, change it by 2%.
template <int N>
struct Kv8Pairs {
    int32_t src[N], dst[N];
};

constexpr int kCopyUnits = 1024;  // 16-byte units a CTA moves

// upp: units of a page; per: pages of a CTA; nchunk: CTAs of a page (one of the two is 1)
template <int N>
__global__ void __launch_bounds__(256) kv8_copy_kernel(const __grid_constant__ Kv8Pairs<N> p, uint4* K, uint4* V,
                                                       float* scale, int n, uint32_t upp, int per, int nchunk, int hkv) {
    const int i0 = blockIdx.x / nchunk * per, ch = blockIdx.x % nchunk;
    uint4* pool = blockIdx.y ? V : K;
    const int cnt = min(per, n - i0);
    uint4 x[4];
    uint4* to[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint32_t at = ch * (uint32_t)kCopyUnits + 256 * u + threadIdx.x, j = at / upp;
        to[u] = nullptr;
        if (j < (uint32_t)cnt) {
            x[u] = __ldcs(pool + p.src[i0 + j] * (int64_t)upp + (at - j * upp));
            to[u] = pool + p.dst[i0 + j] * (int64_t)upp + (at - j * upp);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (to[u]) __stcs(to[u], x[u]);
    if (ch == 0 && blockIdx.y == 0)
        for (int e = threadIdx.x; e < cnt * 2 * hkv; e += 256) {
            const int j = e / (2 * hkv), h = e % (2 * hkv);
            scale[p.dst[i0 + j] * (int64_t)(2 * hkv) + h] = scale[p.src[i0 + j] * (int64_t)(2 * hkv) + h];
        }
}

static lsa_status check_kv8(const lsa_kv8* c) {
    if (!c) return set_error(LSA_EINVAL, "kv8: cache is NULL");
    if (c->fmt != LSA_KV8_E4M3 && c->fmt != LSA_KV8_INT8) return set_error(LSA_EINVAL, "kv8: fmt must be 0 (e4m3) or 1 (int8)");
    if (c->hkv <= 0 || c->n_pages <= 0) return set_error(LSA_EINVAL, "kv8: hkv and n_pages must be positive");
    if (c->hkv > 65535) return set_error(LSA_EUNSUPPORTED, "kv8: hkv > 65535");
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256)
        return set_error(LSA_EUNSUPPORTED, "kv8: page must be 16, 32, 64, 128 or 256 tokens");
    if (c->n_pages > (int64_t)INT32_MAX / ((int64_t)c->hkv * c->page))
        return set_error(LSA_EUNSUPPORTED, "kv8: more than 2^31 rows of codes");
    if (!c->K || !c->V || !c->scale) return set_error(LSA_EINVAL, "kv8: K, V or scale is NULL");
    if ((((uintptr_t)c->K | (uintptr_t)c->V) & 127u) || ((uintptr_t)c->scale & 7u))
        return set_error(LSA_EINVAL, "kv8: K and V must be 128-byte aligned, scale 8-byte");
    return LSA_OK;
}

template <int FMT>
static void launch_kv8_write(const Kv8WriteArgs& a, int page, dim3 grid, cudaStream_t st) {
    switch (page) {
        case 16: kv8_write_kernel<FMT, 1><<<grid, 256, 0, st>>>(a); break;
        case 32: kv8_write_kernel<FMT, 2><<<grid, 256, 0, st>>>(a); break;
        case 64: kv8_write_kernel<FMT, 4><<<grid, 256, 0, st>>>(a); break;
        case 128: kv8_write_kernel<FMT, 8><<<grid, 256, 0, st>>>(a); break;
        default: kv8_write_kernel<FMT, 16><<<grid, 256, 0, st>>>(a); break;
    }
}

static lsa_status run_kv8_write(const lsa_kv8* kv, const Kv8WriteArgs& a, int64_t items, cudaStream_t st) {
    {
        KTime kt_("kv8_write_kernel", st);
        const int heads = kv8_write_heads(kv->page / 16);
        const dim3 grid((unsigned)(items * ceil_div(kv->hkv, heads)), kv->page <= 64 ? 1 : 2);
        if (kv->fmt == LSA_KV8_E4M3) launch_kv8_write<0>(a, kv->page, grid, st);
        else launch_kv8_write<1>(a, kv->page, grid, st);
    }
    return check_launch("kv8_write_kernel");
}

// A whole prompt into one sequence's pages (decode's load).
lsa_status launch_kv8_prompt(const lsa_kv8* kv, const uint16_t* K, const uint16_t* V, int64_t n, const int32_t* table,
                             int32_t max_pages, cudaStream_t st) {
    if (n <= 0) return LSA_OK;
    Kv8WriteArgs a{};
    a.K = K; a.V = V; a.k_stride = a.v_stride = (int64_t)kv->hkv * kD;
    a.Kp = kv->K; a.Vp = kv->V; a.scale = kv->scale;
    a.table = table; a.n_tokens = n; a.n_pages = kv->n_pages; a.n_seq = 1; a.max_pages = max_pages; a.hkv = kv->hkv;
    return run_kv8_write(kv, a, ceil_div<int64_t>(n, kv->page), st);
}

template <int N>
static void launch_kv8_copy(const lsa_kv8* c, const int32_t* src, const int32_t* dst, int n, cudaStream_t st) {
    Kv8Pairs<N> p;
    for (int i = 0; i < n; ++i) { p.src[i] = src[i]; p.dst[i] = dst[i]; }
    const uint32_t upp = (uint32_t)c->hkv * c->page * (kD / 16);
    const int per = std::max(1u, kCopyUnits / upp), nchunk = (int)ceil_div<int64_t>(upp, kCopyUnits);
    kv8_copy_kernel<N><<<dim3((unsigned)(ceil_div(n, per) * nchunk), 2), 256, 0, st>>>(
        p, reinterpret_cast<uint4*>(c->K), reinterpret_cast<uint4*>(c->V), c->scale, n, upp, per, nchunk, c->hkv);
}

}  // namespace lsa

extern "C" {

lsa_status lsa_kv8_write(const lsa_kv8* kv, const uint16_t* K, int64_t k_stride, const uint16_t* V, int64_t v_stride,
                         int64_t n_tokens, const int32_t* cu, const int32_t* start, const int32_t* table,
                         int32_t n_seq, int32_t max_pages, void* stream) {
    using namespace lsa;
    lsa_status s;
    if ((s = check_kv8(kv)) != LSA_OK) return s;
    if (n_tokens < 0 || n_seq < 0 || max_pages < 0) return set_error(LSA_EINVAL, "lsa_kv8_write: negative size");
    if (!cu && n_tokens != n_seq) return set_error(LSA_EINVAL, "lsa_kv8_write: without cu, n_tokens must equal n_seq");
    if (n_tokens == 0 || n_seq == 0) return LSA_OK;
    if (!K || !V || !start || !table) return set_error(LSA_EINVAL, "lsa_kv8_write: NULL pointer");
    if (k_stride < (int64_t)kv->hkv * kD || v_stride < (int64_t)kv->hkv * kD || (k_stride & 7) || (v_stride & 7))
        return set_error(LSA_EINVAL, "lsa_kv8_write: token strides must be multiples of 8 elements, at least hkv * 128");
    if (!aligned16(K) || !aligned16(V)) return set_error(LSA_EINVAL, "lsa_kv8_write: K and V must be 16-byte aligned");
    // pages a sequence touches: at most n / page + 2
    const int64_t items = cu ? n_tokens / kv->page + 2 * (int64_t)n_seq : n_seq;
    if (n_tokens > INT32_MAX || items * kv->hkv > INT32_MAX) return set_error(LSA_EUNSUPPORTED, "lsa_kv8_write: n_tokens beyond 2^31");
    Kv8WriteArgs a{};
    a.K = K; a.V = V; a.k_stride = k_stride; a.v_stride = v_stride;
    a.Kp = kv->K; a.Vp = kv->V; a.scale = kv->scale;
    a.cu = cu; a.start = start; a.table = table; a.n_tokens = n_tokens; a.n_pages = kv->n_pages;
    a.n_seq = n_seq; a.max_pages = max_pages; a.hkv = kv->hkv;
    return run_kv8_write(kv, a, items, (cudaStream_t)stream);
}

lsa_status lsa_kv8_copy_pages(const lsa_kv8* kv, const int32_t* src, const int32_t* dst, int64_t n, void* stream) {
    using namespace lsa;
    lsa_status s;
    if ((s = check_kv8(kv)) != LSA_OK) return s;
    if (n < 0) return set_error(LSA_EINVAL, "lsa_kv8_copy_pages: n < 0");
    if (n == 0) return LSA_OK;
    if (!src || !dst) return set_error(LSA_EINVAL, "lsa_kv8_copy_pages: NULL pointer");
    if (n > kv->n_pages) return set_error(LSA_EINVAL, "lsa_kv8_copy_pages: more copies than pages");
    for (int64_t i = 0; i < n; ++i)
        if (src[i] < 0 || src[i] >= kv->n_pages || dst[i] < 0 || dst[i] >= kv->n_pages)
            return set_error(LSA_EINVAL, "lsa_kv8_copy_pages: pair %lld (%d -> %d) is outside the pool's %lld pages",
                             (long long)i, src[i], dst[i], (long long)kv->n_pages);
    // the copies run in no order: no page may be written twice, or written and read
    uint8_t* mark = (uint8_t*)calloc((size_t)(kv->n_pages + 7) / 8, 1);
    if (!mark) return set_error(LSA_ENOSPACE, "lsa_kv8_copy_pages: out of host memory");
    int64_t bad = -1;
    for (int64_t i = 0; i < n && bad < 0; ++i) {
        if (mark[dst[i] >> 3] & (1u << (dst[i] & 7))) bad = i;
        mark[dst[i] >> 3] |= (uint8_t)(1u << (dst[i] & 7));
    }
    for (int64_t i = 0; i < n && bad < 0; ++i)
        if (mark[src[i] >> 3] & (1u << (src[i] & 7))) bad = i;
    free(mark);
    if (bad >= 0)
        return set_error(LSA_EINVAL, "lsa_kv8_copy_pages: pair %lld (%d -> %d): a page is written twice, or read and written",
                         (long long)bad, src[bad], dst[bad]);
    const cudaStream_t st = (cudaStream_t)stream;
    constexpr int kFew = 60, kMany = 4000;  // 480 bytes or 32 KB of arguments
    for (int64_t i = 0; i < n; i += kMany) {
        const int m = (int)(n - i < kMany ? n - i : kMany);
        {
            KTime kt_("kv8_copy_kernel", st);
            if (m <= kFew) launch_kv8_copy<kFew>(kv, src + i, dst + i, m, st);
            else launch_kv8_copy<kMany>(kv, src + i, dst + i, m, st);
        }
        if ((s = check_launch("kv8_copy_kernel")) != LSA_OK) return s;
    }
    return LSA_OK;
}

}  // extern "C"
