// lsa_kv8_attn.cu -- exact softmax attention over the paged 8-bit K/V cache
// [tutorial "隐空间稀疏注意力 (LSA)" (diosapp.com.cn), section 二: the attention
// formula is unchanged; essay "《卡片柜》" (zhichai.net), ch. 8: 8-bit storage].
//
// One warp step takes 16 keys of one kv-head against 8 columns (the query
// heads of the group; of several new tokens, 8 or 16 (token, head) pairs):
//   S^T = K Q^T   keys are the MMA's M dimension, columns its N;
//   O^T += V^T P^T.
// Codes go from global memory straight into registers, 16 bytes a lane, in
// an order that makes them MMA operands without a shuffle: the K dimension of
// S^T is a permutation of the 128 dims (lane (g, t) holds dims 16 t .. + 15
// and 64 + 16 t .. + 15 of key rows g and g + 8, Q follows the same order),
// and the M dimension of O^T is one too (lane (g, t) holds dims 16 g .. + 15
// of key rows 2t, 2t+1, 2t+8, 2t+9; byte pairs of two rows are interleaved
// with one byte permute).  Codes become fp16 exactly; Q is divided by its
// row's power of two and becomes fp16 (exact to 2^-17 of the row's largest
// element, absolute error 2^-25 of it below that); P is fp16 with 12 bits of
// headroom (an entry 2^-26 of the largest still has all its bits).  Scores,
// softmax sums and outputs are fp32.  The K scale multiplies the scores; the
// V scale, a power of two, multiplies P relative to the largest V scale seen
// so far.  The running maximum moves only when a score exceeds it by 2 (in
// base 2), so most steps skip the rescaling.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "lsa_common.cuh"
#include "lsa_mma.cuh"

namespace lsa {

constexpr int kKv8Warps = 8;
constexpr float kKv8Head = 12.f;   // log2 of P's headroom
constexpr float kKv8Lazy = 2.f;    // log2 growth that moves the running maximum

struct Kv8AttnArgs {
    const uint16_t* Q;     // [nq, hq, 128], token rows q_stride elements apart
    const uint8_t* K;      // [n_pages, hkv, page, 128]
    const uint8_t* V;
    const float* scale;    // [n_pages, hkv, 2]
    const int32_t* table;  // [n_seq, max_pages]
    const int32_t* lens;   // [n_seq]
    const int32_t* cu;     // dense: [n_seq + 1] or NULL (one query per sequence)
    const int32_t* seq;    // lists: [nq] or NULL (query i is sequence i's)
    const int32_t* idx;    // lists: [nq, hkv, n_idx]
    int64_t q_stride, nq, n_pages;
    int32_t n_seq, max_pages, hkv, G, lgp, n_idx;
    int32_t S, W;          // dense: sinks and window (W = 0: every key)
    uint16_t* O;           // [nq, hq, 128]
    float* lse;            // [nq, hq] or NULL
    float* part;           // split rows' partial states
    float scale_log2;
};

// ------------------------------------------------------- code conversion

// Four codes to two fp16 pairs (bytes 0, 1 and 2, 3), exact.  int8: the code
// biased by 128 is the low byte of the fp16 number 1024 + code + 128.
template <int FMT>
__device__ __forceinline__ void kv8_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (FMT == 0) {
        lo = e4m3x2_to_f16x2(w & 0xFFFFu);
        hi = e4m3x2_to_f16x2(w >> 16);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));  // 1152
        uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
    }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Transpose of an 8 x 8 matrix of 16-bit elements held one row per four lanes.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint4 ldg_codes(const uint8_t* p, bool ok) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (ok) v = __ldg(reinterpret_cast<const uint4*>(p));
    return v;
}

// ------------------------------------------------------------ warp state

template <int NT>
struct Kv8State {
    uint32_t qb[NT][8][2];  // Q as B operands
    float cf[NT][2];        // score factor of columns 2t, 2t + 1: Q's power of two * log2(e) / sqrt(d)
    float o[NT][8][4];
    float m[NT][2], l[NT][2];
    float vref;             // the V scale that O is relative to
};

// Q row of column n (gq within tile nt): 32 of its 128 dims per lane, to fp16
// B operands in the permuted order, with its power of two.
template <int NT>
__device__ __forceinline__ void kv8_load_q(Kv8State<NT>& s, const uint16_t* const (&row)[NT], float scale_log2) {
    const int lane = threadIdx.x & 31, tq = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row[nt]) x[i] = __ldg(reinterpret_cast<const uint4*>(row[nt] + (i >> 1) * 64 + 16 * tq + (i & 1) * 8));
        }
        uint32_t mx = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mx = max(mx, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
        }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // |q| < 2^(E - 126): divide by 2^e, e = E - 126 in [-120, 120]
        const int e = mx == 0u ? 0 : max(-120, min(120, (int)(mx >> 7) - 126));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23), f = __uint_as_float((uint32_t)(127 + e) << 23) * scale_log2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // dims (i >> 1) * 64 + 16 t + (i & 1) * 8 + 2 j, + 1: k-step (i >> 1) * 4 + (i & 1) * 2 + j / 2
                const float a = __uint_as_float(w[j] << 16) * inv, b = __uint_as_float(w[j] & 0xFFFF0000u) * inv;
                s.qb[nt][(i >> 1) * 4 + (i & 1) * 2 + (j >> 1)][j & 1] = pack_f16x2(a, b);
            }
        }
        s.cf[nt][0] = __shfl_sync(0xffffffffu, f, (2 * tq) * 4);
        s.cf[nt][1] = __shfl_sync(0xffffffffu, f, (2 * tq + 1) * 4);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s.o[nt][mt][i] = 0.f;
        s.m[nt][0] = s.m[nt][1] = -FLT_MAX;
        s.l[nt][0] = s.l[nt][1] = 0.f;
    }
    s.vref = 0x1p-100f;
}

// S^T of 16 keys: k[0..1] the lane's chunks of key row g, k[2..3] of row g + 8.
template <int FMT, int NT>
__device__ __forceinline__ void kv8_scores(const Kv8State<NT>& s, const uint4 (&k)[4], float (&sc)[NT][4]) {
    float c[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[nt][h][i] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t wa[4] = {k[h].x, k[h].y, k[h].z, k[h].w}, wb[4] = {k[2 + h].x, k[2 + h].y, k[2 + h].z, k[2 + h].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t a[4];
            kv8_f16<FMT>(wa[j], a[0], a[2]);
            kv8_f16<FMT>(wb[j], a[1], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816_f16(c[nt][h], a, s.qb[nt][4 * h + j][0], s.qb[nt][4 * h + j][1]);
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[nt][i] = c[nt][0][i] + c[nt][1][i];
}

// The interleaved fp16 A operands of V^T for words j of the lane's four rows:
// m-tiles 2j (dims 16 g + 4 j, + 1) and 2j + 1 (dims + 2, + 3).
template <int FMT>
__device__ __forceinline__ void kv8_v_operands(const uint32_t (&w)[4], uint32_t (&a0)[4], uint32_t (&a1)[4]) {
    kv8_f16<FMT>(__byte_perm(w[0], w[1], 0x5140), a0[0], a0[1]);
    kv8_f16<FMT>(__byte_perm(w[2], w[3], 0x5140), a0[2], a0[3]);
    kv8_f16<FMT>(__byte_perm(w[0], w[1], 0x7362), a1[0], a1[1]);
    kv8_f16<FMT>(__byte_perm(w[2], w[3], 0x7362), a1[2], a1[3]);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

template <int FMT, int NT>
__device__ __forceinline__ void kv8_pv(Kv8State<NT>& s, const uint4 (&v)[4], const uint32_t (&pb)[NT][2]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w[4] = {word_of(v[0], j), word_of(v[1], j), word_of(v[2], j), word_of(v[3], j)};
        uint32_t a0[4], a1[4];
        kv8_v_operands<FMT>(w, a0, a1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mma_16816_f16(s.o[nt][2 * j], a0, pb[nt][0], pb[nt][1]);
            mma_16816_f16(s.o[nt][2 * j + 1], a1, pb[nt][0], pb[nt][1]);
        }
    }
}

// Softmax of one step.  Scores in base 2, -inf where masked; vs0, vs1: the V
// scales of keys g and g + 8 (vmax: the step's largest, warp-uniform).
// Leaves P^T as B operands in pb.
template <int NT>
__device__ __forceinline__ void kv8_softmax(Kv8State<NT>& s, const float (&sc)[NT][4], float vs0, float vs1, float vmax,
                                            uint32_t (&pb)[NT][2]) {
    bool grew = vmax > s.vref;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        grew = grew || fmaxf(sc[nt][0], sc[nt][2]) > s.m[nt][0] + kKv8Lazy || fmaxf(sc[nt][1], sc[nt][3]) > s.m[nt][1] + kKv8Lazy;
    if (__any_sync(0xffffffffu, grew)) {
        const float nref = fmaxf(vmax, s.vref), rv = s.vref / nref;
        s.vref = nref;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float mx0 = fmaxf(sc[nt][0], sc[nt][2]), mx1 = fmaxf(sc[nt][1], sc[nt][3]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
            }
            const float n0 = fmaxf(s.m[nt][0], mx0), n1 = fmaxf(s.m[nt][1], mx1);
            const float a0 = exp2f(s.m[nt][0] - n0), a1 = exp2f(s.m[nt][1] - n1);
            s.m[nt][0] = n0;
            s.m[nt][1] = n1;
            s.l[nt][0] *= a0;
            s.l[nt][1] *= a1;
            const float f0 = a0 * rv, f1 = a1 * rv;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                s.o[nt][mt][0] *= f0; s.o[nt][mt][1] *= f1; s.o[nt][mt][2] *= f0; s.o[nt][mt][3] *= f1;
            }
        }
    }
    const float iv = 1.0f / s.vref, w0 = vs0 * iv, w1 = vs1 * iv;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float b0 = s.m[nt][0] - kKv8Head, b1 = s.m[nt][1] - kKv8Head;
        const float e0 = exp2f(sc[nt][0] - b0), e1 = exp2f(sc[nt][1] - b1);
        const float e2 = exp2f(sc[nt][2] - b0), e3 = exp2f(sc[nt][3] - b1);
        s.l[nt][0] += e0 + e2;
        s.l[nt][1] += e1 + e3;
        pb[nt][0] = movmatrix_t(pack_f16x2(e0 * w0, e1 * w0));
        pb[nt][1] = movmatrix_t(pack_f16x2(e2 * w1, e3 * w1));
    }
}

// Sum of l over the lanes that share a column.
template <int NT>
__device__ __forceinline__ void kv8_reduce_l(Kv8State<NT>& s) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            s.l[nt][0] += __shfl_xor_sync(0xffffffffu, s.l[nt][0], off);
            s.l[nt][1] += __shfl_xor_sync(0xffffffffu, s.l[nt][1], off);
        }
}

__device__ __forceinline__ uint16_t bf16_bits(float x) {
    const __nv_bfloat16 b = __float2bfloat16_rn(x);
    return *reinterpret_cast<const uint16_t*>(&b);
}

// --------------------------------------------------- index lists, one row

// Keys [16 tile, 16 tile + 16) of a list: lanes l and l + 16 hold entry l as
// its row of codes (-1: none) and its two scales (bf16 halves: powers of two).
struct Kv8List {
    const int32_t* list;   // NULL: the query's sequence number is out of range
    const int32_t* table;  // the sequence's row
    int32_t len, n_idx, max_pages, hkv, g, lgp;
    int64_t n_pages;
};

__device__ __forceinline__ Kv8List kv8_list(const Kv8AttnArgs& a, int64_t q, int g) {
    Kv8List r;
    int64_t b = a.seq ? (int64_t)__ldg(a.seq + q) : q;
    const bool ok = b >= 0 && b < a.n_seq;
    if (!ok) {
        raise_device_error(kErrKv8Range);
        b = 0;
    }
    r.list = ok ? a.idx + (q * a.hkv + g) * (int64_t)a.n_idx : nullptr;
    r.table = a.table + b * a.max_pages;
    r.len = __ldg(a.lens + b);
    r.n_idx = a.n_idx; r.max_pages = a.max_pages; r.hkv = a.hkv; r.g = g; r.lgp = a.lgp; r.n_pages = a.n_pages;
    return r;
}

__device__ __forceinline__ int kv8_entry(const Kv8List& r, int tile, int tend) {
    const int e = tile * 16 + (threadIdx.x & 15);
    return r.list != nullptr && tile < tend && e < r.n_idx ? __ldg(r.list + e) : -1;
}

__device__ __forceinline__ int kv8_row(const Kv8List& r, int p) {
    if (p < 0) return -1;
    const int pg = p >> r.lgp;
    if (p >= r.len || pg >= r.max_pages) {
        raise_device_error(kErrIndexRange);
        return -1;
    }
    const int pid = __ldg(r.table + pg);
    if (pid < 0 || pid >= r.n_pages) {
        raise_device_error(kErrKv8Page);
        return -1;
    }
    return (int)((((uint32_t)pid * r.hkv + r.g) << r.lgp) | (uint32_t)(p & ((1 << r.lgp) - 1)));
}

__device__ __forceinline__ uint32_t kv8_scales(const Kv8AttnArgs& a, int row) {
    if (row < 0) return 0u;
    const float2 s = __ldg(reinterpret_cast<const float2*>(a.scale) + (row >> a.lgp));
    return __byte_perm(__float_as_uint(s.x), __float_as_uint(s.y), 0x7632);  // K's upper half low, V's high
}

__device__ __forceinline__ void kv8_load_k_rows(const Kv8AttnArgs& a, int row, uint4 (&k)[4]) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const int r0 = __shfl_sync(0xffffffffu, row, gq), r1 = __shfl_sync(0xffffffffu, row, gq + 8);
    const uint8_t* p0 = a.K + (int64_t)r0 * kD + 16 * tq;
    const uint8_t* p1 = a.K + (int64_t)r1 * kD + 16 * tq;
    k[0] = ldg_codes(p0, r0 >= 0);
    k[1] = ldg_codes(p0 + 64, r0 >= 0);
    k[2] = ldg_codes(p1, r1 >= 0);
    k[3] = ldg_codes(p1 + 64, r1 >= 0);
}

__device__ __forceinline__ void kv8_load_v_rows(const Kv8AttnArgs& a, int row, uint4 (&v)[4]) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = __shfl_sync(0xffffffffu, row, 2 * tq + (i & 1) + 8 * (i >> 1));
        v[i] = ldg_codes(a.V + (int64_t)r * kD + 16 * gq, r >= 0);
    }
}

// Tiles [t, tend) of one list into the warp's state.
template <int FMT>
__device__ __forceinline__ void kv8_list_tiles(const Kv8AttnArgs& a, const Kv8List& r, int t, int tend, Kv8State<1>& s) {
    const int lane = threadIdx.x & 31, gq = lane >> 2;
    if (t >= tend) return;
    uint4 kc[4], vc[4];
    int row = kv8_row(r, kv8_entry(r, t, tend));
    int row1 = kv8_row(r, kv8_entry(r, t + 1, tend));
    int e2 = kv8_entry(r, t + 2, tend);
    uint32_t sc = kv8_scales(a, row);
    kv8_load_k_rows(a, row, kc);
    kv8_load_v_rows(a, row, vc);
    for (; t < tend; ++t) {
        uint4 kn[4], vn[4];
        const int e3 = kv8_entry(r, t + 3, tend);
        const int row2 = kv8_row(r, e2);
        const uint32_t sc1 = kv8_scales(a, row1);
        kv8_load_k_rows(a, row1, kn);
        const unsigned valid = __ballot_sync(0xffffffffu, row >= 0);
        float x[1][4];
        uint32_t pb[1][2] = {{0u, 0u}};
        if (valid) {
            kv8_scores<FMT, 1>(s, kc, x);
            const uint32_t c0 = __shfl_sync(0xffffffffu, sc, gq), c1 = __shfl_sync(0xffffffffu, sc, gq + 8);
            const bool v0 = (valid >> gq) & 1u, v1 = (valid >> (gq + 8)) & 1u;
            const float k0 = __uint_as_float(c0 << 16), k1 = __uint_as_float(c1 << 16);
            x[0][0] = v0 ? x[0][0] * (k0 * s.cf[0][0]) : -CUDART_INF_F;
            x[0][1] = v0 ? x[0][1] * (k0 * s.cf[0][1]) : -CUDART_INF_F;
            x[0][2] = v1 ? x[0][2] * (k1 * s.cf[0][0]) : -CUDART_INF_F;
            x[0][3] = v1 ? x[0][3] * (k1 * s.cf[0][1]) : -CUDART_INF_F;
            // the step's largest V scale: positive floats order as integers
            const float vmax = __uint_as_float(__reduce_max_sync(0xffffffffu, sc & 0xFFFF0000u));
            kv8_softmax<1>(s, x, __uint_as_float(c0 & 0xFFFF0000u), __uint_as_float(c1 & 0xFFFF0000u), vmax, pb);
        }
        kv8_load_v_rows(a, row1, vn);
        if (valid) kv8_pv<FMT, 1>(s, vc, pb);
#pragma unroll
        for (int i = 0; i < 4; ++i) { kc[i] = kn[i]; vc[i] = vn[i]; }
        row = row1; row1 = row2; e2 = e3; sc = sc1;
    }
}

// Many rows: one warp per (query, kv-head), kv-head major so that the warps
// resident at one time read one head's rows, which keeps them in L2.
template <int FMT>
__global__ void __launch_bounds__(32 * kKv8Warps, 2) kv8_list_kernel(Kv8AttnArgs a) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const int64_t wg = (int64_t)blockIdx.x * kKv8Warps + (threadIdx.x >> 5);
    if (wg >= a.nq * a.hkv) return;
    const int64_t q = wg % a.nq;
    const int g = (int)(wg / a.nq);
    const int hq = a.G * a.hkv;
    Kv8State<1> s;
    const uint16_t* const row[1] = {gq < a.G ? a.Q + q * a.q_stride + (int64_t)(g * a.G + gq) * kD : nullptr};
    kv8_load_q<1>(s, row, a.scale_log2);
    const Kv8List r = kv8_list(a, q, g);
    kv8_list_tiles<FMT>(a, r, 0, (a.n_idx + 15) / 16, s);
    kv8_reduce_l<1>(s);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (2 * tq + c >= a.G) continue;
        const float l = s.l[0][c], f = l > 0.f || l != l ? s.vref / l : 0.f;
        const int64_t orow = q * hq + g * a.G + 2 * tq + c;
        uint32_t w[8];
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) w[mt] = pack_bf16x2(s.o[0][mt][c] * f, s.o[0][mt][2 + c] * f);
        uint4* op = reinterpret_cast<uint4*>(a.O + orow * kD + 16 * gq);
        op[0] = make_uint4(w[0], w[1], w[2], w[3]);
        op[1] = make_uint4(w[4], w[5], w[6], w[7]);
        if (a.lse && gq == 0) a.lse[orow] = l > 0.f || l != l ? s.m[0][c] - kKv8Head + log2f(l) : -CUDART_INF_F;
    }
}

// ------------------------------------------------ rows split over the GPU

// The work is one stream of 16-key tiles: rows in the order (sequence,
// kv-head, column group), each with the tiles its mask leaves (at least one).
// CTA c takes tiles [c per, (c + 1) per): the same work for every CTA however
// ragged the lengths.  A row inside one CTA's range is finished there; a row
// that crosses CTAs leaves a partial state in every CTA it touches (slot 0 if
// it began before the CTA, slot 1 if it began inside), and kv8_join_kernel
// joins them.  Everyone derives the stream from lens and cu by the same scan.
struct Kv8Seq {
    int64_t base;     // first tile of the sequence in the stream
    int32_t tiles;    // tiles of each of its rows
    int32_t rows;     // hkv * column groups
    int32_t groups;
    int32_t n, len;   // new tokens, tokens in all
    int64_t q0;
    int32_t n_sink, t_lo;  // tiles [0, n_sink) and from t_lo on
};

template <int NT, bool LIST>
__device__ __forceinline__ void kv8_seq(const Kv8AttnArgs& a, int64_t b, Kv8Seq& q) {
    if constexpr (LIST) {  // "sequence" b is query b
        q.n = 1; q.q0 = b; q.len = 0; q.groups = 1; q.rows = a.hkv; q.n_sink = 0; q.t_lo = 0;
        q.tiles = max(1, (a.n_idx + 15) / 16);
    } else {
        q.q0 = a.cu ? (int64_t)__ldg(a.cu + b) : b;
        int64_t n = a.cu ? (int64_t)__ldg(a.cu + b + 1) - q.q0 : 1;
        int64_t len = __ldg(a.lens + b);
        if (n < 0 || (n > 0 && (q.q0 < 0 || q.q0 + n > a.nq))) {
            raise_device_error(kErrKv8Range);
            n = 0;
        }
        if (len < 0 || len > ((int64_t)a.max_pages << a.lgp)) {
            raise_device_error(kErrKv8Range);
            len = len < 0 ? 0 : (int64_t)a.max_pages << a.lgp;
        }
        q.n = (int)n;
        q.len = (int)len;
        q.groups = (int)((n * a.G + 8 * NT - 1) / (8 * NT));
        q.rows = a.hkv * q.groups;
        const int hi = (int)((len + 15) / 16);
        const int64_t lo = a.W > 0 ? len - n - a.W + 1 : 0;  // the first query's window begins there
        q.t_lo = lo > 0 ? (int)(lo / 16) : 0;
        q.n_sink = min((min(a.S, (int)len) + 15) / 16, q.t_lo);
        q.tiles = max(1, q.n_sink + hi - q.t_lo);
    }
}

template <int NT, bool LIST>
struct Kv8Scan {
    int64_t total, per;
    // Tiles of all sequences, and each CTA's share of them.  `least`: tiles a
    // CTA takes at least.
    __device__ __forceinline__ void init(const Kv8AttnArgs& a, int n_cta, int least) {
        if constexpr (LIST) {
            Kv8Seq q;
            kv8_seq<NT, true>(a, 0, q);
            total = a.nq * a.hkv * (int64_t)q.tiles;
        } else {
            __shared__ long long sum[kKv8Warps];
            long long mine = 0;
            for (int64_t b = threadIdx.x; b < a.n_seq; b += 32 * kKv8Warps) {
                Kv8Seq q;
                kv8_seq<NT, false>(a, b, q);
                mine += (int64_t)q.tiles * q.rows;
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
            if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = mine;
            __syncthreads();
            total = 0;
#pragma unroll
            for (int i = 0; i < kKv8Warps; ++i) total += sum[i];
            __syncthreads();
        }
        per = max((int64_t)least, (total + n_cta - 1) / n_cta);
    }
    // The sequence whose tiles hold position w of the stream (0 <= w < total).
    __device__ __forceinline__ int64_t find(const Kv8AttnArgs& a, int64_t w, Kv8Seq& out) {
        if constexpr (LIST) {
            kv8_seq<NT, true>(a, 0, out);
            const int64_t b = w / ((int64_t)out.tiles * out.rows);
            kv8_seq<NT, true>(a, b, out);
            out.base = b * out.tiles * out.rows;
            return b;
        } else {
            __shared__ long long wsum[kKv8Warps];
            __shared__ long long fb, fbase;
            const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
            long long base = 0;
            for (int64_t b0 = 0; b0 < a.n_seq; b0 += 32 * kKv8Warps) {
                const int64_t b = b0 + threadIdx.x;
                long long m = 0;
                if (b < a.n_seq) {
                    Kv8Seq q;
                    kv8_seq<NT, false>(a, b, q);
                    m = (int64_t)q.tiles * q.rows;
                }
                long long inc = m;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const long long up = __shfl_up_sync(0xffffffffu, inc, off);
                    if (lane >= off) inc += up;
                }
                if (lane == 31) wsum[wid] = inc;
                __syncthreads();
                long long before = base, all = base;
#pragma unroll
                for (int i = 0; i < kKv8Warps; ++i) {
                    if (i < wid) before += wsum[i];
                    all += wsum[i];
                }
                const long long first = before + inc - m;
                if (w >= first && w < first + m) { fb = b; fbase = first; }
                __syncthreads();
                base = all;
                if (w < base) break;  // uniform: every thread holds the same sums
            }
            const int64_t b = fb;
            kv8_seq<NT, false>(a, b, out);
            out.base = fbase;
            __syncthreads();
            return b;
        }
    }
};

// Keys of one dense tile: page row of the first (-1: none), its scales.
struct Kv8Dense {
    const int32_t* table;
    int32_t len, n_sink, t_lo, g;
};

__device__ __forceinline__ int kv8_tile_key(const Kv8Dense& d, int t) {
    return 16 * (t < d.n_sink ? t : t - d.n_sink + d.t_lo);
}

__device__ __forceinline__ int kv8_tile_page(const Kv8AttnArgs& a, const Kv8Dense& d, int t, int tend) {
    const int key = kv8_tile_key(d, t);
    return t < tend && key < d.len ? __ldg(d.table + (key >> a.lgp)) : -2;
}

__device__ __forceinline__ int kv8_tile_row(const Kv8AttnArgs& a, const Kv8Dense& d, int t, int pid) {
    if (pid == -2) return -1;
    if (pid < 0 || pid >= a.n_pages) {
        raise_device_error(kErrKv8Page);
        return -1;
    }
    return (int)((((uint32_t)pid * a.hkv + d.g) << a.lgp) | (uint32_t)(kv8_tile_key(d, t) & ((1 << a.lgp) - 1)));
}

// Keys of a tile that some column of the row attends: bit i = key i.
struct Kv8Mask {
    int tmin, tmax, lo, S;  // positions of the row's first and last query; first key of the first one's window
};

__device__ __forceinline__ unsigned kv8_tile_mask(const Kv8Mask& k, int key, int row) {
    if (row < 0 || key > k.tmax) return 0u;
    unsigned m = k.tmax - key >= 15 ? 0xFFFFu : (2u << (k.tmax - key)) - 1u;
    if (key < k.lo) {  // below the window only the sinks
        const unsigned below = k.lo - key >= 16 ? 0xFFFFu : (1u << (k.lo - key)) - 1u;
        const unsigned sink = k.S - key >= 16 ? 0xFFFFu : k.S > key ? (1u << (k.S - key)) - 1u : 0u;
        m &= ~below | sink;
    }
    return m;
}

__device__ __forceinline__ void kv8_load_k_tile(const Kv8AttnArgs& a, int row, unsigned m, uint4 (&k)[4]) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const uint8_t* p = a.K + ((int64_t)row + gq) * kD + 16 * tq;
    const bool v0 = (m >> gq) & 1u, v1 = (m >> (gq + 8)) & 1u;
    k[0] = ldg_codes(p, v0);
    k[1] = ldg_codes(p + 64, v0);
    k[2] = ldg_codes(p + 8 * kD, v1);
    k[3] = ldg_codes(p + 8 * kD + 64, v1);
}

__device__ __forceinline__ void kv8_load_v_tile(const Kv8AttnArgs& a, int row, unsigned m, uint4 (&v)[4]) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const uint8_t* p = a.V + ((int64_t)row + 2 * tq) * kD + 16 * gq;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int off = (i & 1) + 8 * (i >> 1);
        v[i] = ldg_codes(p + off * kD, (m >> (2 * tq + off)) & 1u);
    }
}

// O^T += V^T P^T for a tile whose mask differs between columns and which holds
// a NaN value: column by column, so that a NaN under one column's mask does
// not reach it through 0 * NaN.
template <int FMT, int NT>
__device__ __forceinline__ void kv8_pv_columns(Kv8State<NT>& s, const uint4 (&v)[4], const uint32_t (&pb)[NT][2],
                                            const int (&tc)[NT][2], int key, int W, int S) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
            const int t = __shfl_sync(0xffffffffu, (c & 1) ? tc[nt][1] : tc[nt][0], c >> 1);
            const uint32_t b0 = gq == c ? pb[nt][0] : 0u, b1 = gq == c ? pb[nt][1] : 0u;
            bool keep[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = key + 2 * tq + (i & 1) + 8 * (i >> 1);
                keep[i] = j <= t && (W == 0 || j > t - W || j < S);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = keep[i] ? word_of(v[i], j) : 0u;
                uint32_t a0[4], a1[4];
                kv8_v_operands<FMT>(w, a0, a1);
                float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
                mma_16816_f16(x, a0, b0, b1);
                mma_16816_f16(y, a1, b0, b1);
                if (tq == (c >> 1)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((i & 1) == (c & 1)) { s.o[nt][2 * j][i] += x[i]; s.o[nt][2 * j + 1][i] += y[i]; }
                }
            }
        }
}

// Tiles [t, tend) of one dense row into the warp's state; tc: the positions
// of the lane's columns (-1: no such column).
template <int FMT, int NT>
__device__ __forceinline__ void kv8_dense_tiles(const Kv8AttnArgs& a, const Kv8Dense& d, const Kv8Mask& mk,
                                                const int (&tc)[NT][2], int t, int tend, Kv8State<NT>& s) {
    const int lane = threadIdx.x & 31, gq = lane >> 2;
    if (t >= tend) return;
    uint4 kc[4], vc[4];
    int row = kv8_tile_row(a, d, t, kv8_tile_page(a, d, t, tend));
    int pid1 = kv8_tile_page(a, d, t + 1, tend);
    unsigned m = kv8_tile_mask(mk, kv8_tile_key(d, t), row);
    float2 sc = row >= 0 ? __ldg(reinterpret_cast<const float2*>(a.scale) + (row >> a.lgp)) : make_float2(0.f, 0.f);
    kv8_load_k_tile(a, row, m, kc);
    kv8_load_v_tile(a, row, m, vc);
    for (; t < tend; ++t) {
        uint4 kn[4], vn[4];
        const int pid2 = kv8_tile_page(a, d, t + 2, tend);
        const int row1 = kv8_tile_row(a, d, t + 1, pid1);
        const unsigned m1 = kv8_tile_mask(mk, kv8_tile_key(d, t + 1), row1);
        const float2 sc1 = row1 >= 0 ? __ldg(reinterpret_cast<const float2*>(a.scale) + (row1 >> a.lgp)) : make_float2(0.f, 0.f);
        kv8_load_k_tile(a, row1, m1, kn);
        float x[NT][4];
        uint32_t pb[NT][2];
        const int key = kv8_tile_key(d, t);
        // every column attends all 16 keys
        const bool whole = m == 0xFFFFu && key + 15 <= mk.tmin && (a.W == 0 || key >= mk.lo + (mk.tmax - mk.tmin) || key + 16 <= mk.S);
        if (m) {
            kv8_scores<FMT, NT>(s, kc, x);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float f0 = sc.x * s.cf[nt][0], f1 = sc.x * s.cf[nt][1];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[nt][i] *= (i & 1) ? f1 : f0;
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = key + gq + 8 * (i >> 1), tt = tc[nt][i & 1];
                        const bool ok = ((m >> (j - key)) & 1u) && j <= tt && (a.W == 0 || j > tt - a.W || j < a.S);
                        if (!ok) x[nt][i] = -CUDART_INF_F;
                    }
                }
            }
            kv8_softmax<NT>(s, x, sc.y, sc.y, sc.y, pb);
        }
        kv8_load_v_tile(a, row1, m1, vn);
        if (m) {
            bool slow = false;
            if constexpr (FMT == 0) {
                if (!whole && mk.tmin != mk.tmax) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) slow = slow || __vcmpeq4(word_of(vc[i], j) & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u;
                    slow = __any_sync(0xffffffffu, slow);
                }
            }
            if (slow) kv8_pv_columns<FMT, NT>(s, vc, pb, tc, key, a.W, a.S);
            else kv8_pv<FMT, NT>(s, vc, pb);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) { kc[i] = kn[i]; vc[i] = vn[i]; }
        row = row1; pid1 = pid2; m = m1; sc = sc1;
    }
}

constexpr int kKv8Pad = kD + 4;  // floats per column in shared memory: consecutive columns start 4 banks apart

// Floats of one partial state: 8 NT columns of 128 sums, then (m, l) each.
template <int NT>
__host__ __device__ constexpr int kv8_part_floats() { return 8 * NT * (kD + 2); }

// Output row of column c of a row: column group cg, kv-head g of a sequence.
template <int NT>
__device__ __forceinline__ int64_t kv8_out_row(const Kv8AttnArgs& a, const Kv8Seq& q, int cg, int g, int c) {
    const int64_t cc = (int64_t)cg * 8 * NT + c;
    if (cc >= (int64_t)q.n * a.G) return -1;
    return (q.q0 + cc / a.G) * (a.G * a.hkv) + g * a.G + cc % a.G;
}

__device__ __forceinline__ void kv8_store(const Kv8AttnArgs& a, int64_t orow, int d, float acc, float m, float l) {
    const bool any = l > 0.f || l != l;
    a.O[orow * kD + d] = bf16_bits(any ? acc / l : 0.f);
    if (d == 0 && a.lse) a.lse[orow] = any ? m - kKv8Head + log2f(l) : -CUDART_INF_F;
}

template <int FMT, int NT, bool LIST>
__global__ void __launch_bounds__(32 * kKv8Warps, NT == 1 ? 2 : 1) kv8_split_kernel(Kv8AttnArgs a, int least) {
    extern __shared__ __align__(16) float ksm[];
    float* so = ksm;                                              // [warps][8 NT][kKv8Pad]
    float* sml = ksm + kKv8Warps * 8 * NT * kKv8Pad;              // [warps][8 NT][2]
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, gq = lane >> 2, tq = lane & 3;
    Kv8Scan<NT, LIST> scan;
    scan.init(a, (int)gridDim.x, least);
    const int64_t w0 = (int64_t)blockIdx.x * scan.per, w1 = min(scan.total, w0 + scan.per);
    if (w0 >= w1) return;
    Kv8Seq q;
    int64_t b = scan.find(a, w0, q);
    for (int64_t w = w0; w < w1;) {
        while (w >= q.base + (int64_t)q.tiles * q.rows) {  // the next sequence that has rows
            const int64_t next = q.base + (int64_t)q.tiles * q.rows;
            kv8_seq<NT, LIST>(a, ++b, q);
            q.base = next;
        }
        const int64_t rel = w - q.base;
        const int r = (int)(rel / q.tiles), t0 = (int)(rel % q.tiles);
        const int g = r / q.groups, cg = r % q.groups;
        const int n = (int)min((int64_t)(q.tiles - t0), w1 - w);
        const int ta = t0 + (int)((int64_t)n * wid / kKv8Warps), tb = t0 + (int)((int64_t)n * (wid + 1) / kKv8Warps);

        if (ta < tb) {
            Kv8State<NT> s;
            const uint16_t* row[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int64_t cc = (int64_t)cg * 8 * NT + 8 * nt + gq;
                row[nt] = cc < (int64_t)q.n * a.G
                              ? a.Q + (q.q0 + cc / a.G) * a.q_stride + (int64_t)(g * a.G + cc % a.G) * kD : nullptr;
            }
            const uint16_t* const (&crow)[NT] = row;
            kv8_load_q<NT>(s, crow, a.scale_log2);
            if constexpr (LIST) {
                const Kv8List lr = kv8_list(a, q.q0, g);
                kv8_list_tiles<FMT>(a, lr, ta, tb, s);
            } else {
                const int first = q.len - q.n;  // position of the sequence's first query
                const int c0 = cg * 8 * NT, c1 = min((int)(q.n * a.G), c0 + 8 * NT) - 1;
                Kv8Mask mk;
                mk.tmin = first + c0 / a.G;
                mk.tmax = first + c1 / a.G;
                mk.lo = a.W > 0 ? mk.tmin - a.W + 1 : 0;
                mk.S = a.S;
                int tc[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int cc = c0 + 8 * nt + 2 * tq + c;
                        tc[nt][c] = cc <= c1 ? first + cc / a.G : -1;
                    }
                const Kv8Dense d{a.table + b * a.max_pages, q.len, q.n_sink, q.t_lo, g};
                kv8_dense_tiles<FMT, NT>(a, d, mk, tc, ta, tb, s);
            }
            kv8_reduce_l<NT>(s);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = wid * 8 * NT + 8 * nt + 2 * tq + c;
                    float4* p = reinterpret_cast<float4*>(so + col * kKv8Pad + 16 * gq);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        p[j] = make_float4(s.o[nt][2 * j][c] * s.vref, s.o[nt][2 * j][2 + c] * s.vref,
                                           s.o[nt][2 * j + 1][c] * s.vref, s.o[nt][2 * j + 1][2 + c] * s.vref);
                    if (gq == 0) { sml[2 * col] = s.m[nt][c]; sml[2 * col + 1] = s.l[nt][c]; }
                }
        } else {
            for (int col = lane; col < 8 * NT; col += 32) {
                sml[2 * (wid * 8 * NT + col)] = -FLT_MAX;
                sml[2 * (wid * 8 * NT + col) + 1] = -1.f;  // took no tile
            }
        }
        __syncthreads();
        const bool final_ = n == q.tiles;
        float* part = a.part + ((int64_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * kv8_part_floats<NT>();
        for (int e = tid; e < 8 * NT * kD; e += 32 * kKv8Warps) {
            const int c = e / kD, dim = e % kD;
            const int64_t orow = kv8_out_row<NT>(a, q, cg, g, c);
            if (orow < 0) continue;
            float M = -FLT_MAX, l = 0.f, acc = 0.f;
#pragma unroll
            for (int i = 0; i < kKv8Warps; ++i) M = fmaxf(M, sml[2 * (i * 8 * NT + c)]);
#pragma unroll
            for (int i = 0; i < kKv8Warps; ++i) {
                const int col = i * 8 * NT + c;
                const float li = sml[2 * col + 1];
                if (li == -1.f) continue;
                const float f = exp2f(sml[2 * col] - M);
                l += li * f;
                acc += so[col * kKv8Pad + dim] * f;
            }
            if (final_) {
                kv8_store(a, orow, dim, acc, M, l);
            } else {
                part[c * kD + dim] = acc;
                if (dim == 0) { part[8 * NT * kD + 2 * c] = M; part[8 * NT * kD + 2 * c + 1] = l; }
            }
        }
        __syncthreads();
        w += n;
    }
}

// Joins the partial states of the row that crosses the end of CTA c's range,
// if that row began inside it.  blockIdx.y: an eighth of the columns' sums.
template <int NT, bool LIST>
__global__ void __launch_bounds__(32 * kKv8Warps) kv8_join_kernel(Kv8AttnArgs a, int n_cta, int least) {
    Kv8Scan<NT, LIST> scan;
    scan.init(a, n_cta, least);
    const int64_t c = blockIdx.x, w0 = c * scan.per, w1 = w0 + scan.per;
    if (w1 >= scan.total) return;
    Kv8Seq q;
    scan.find(a, w1, q);
    const int64_t r = (w1 - q.base) / q.tiles;
    const int64_t begin = q.base + r * q.tiles, end = begin + q.tiles;
    if (begin == w1 || begin < w0) return;
    const int g = (int)(r / q.groups), cg = (int)(r % q.groups);
    const int more = (int)((end - 1) / scan.per - c);  // CTAs after c that hold tiles of the row
    const int e = blockIdx.y * 128 + (threadIdx.x & 127), half = threadIdx.x >> 7;
    const int col = e / kD, dim = e % kD;
    const int64_t orow = kv8_out_row<NT>(a, q, cg, g, col);
    if (orow < 0) return;
    const int64_t stride = 2 * kv8_part_floats<NT>();
    const float* first = a.part + (2 * c + 1) * kv8_part_floats<NT>();
    const float* rest = a.part + 2 * (c + 1) * kv8_part_floats<NT>();
    __shared__ float sh[3][128];
    auto at = [&](int i) { return i == 0 ? first : rest + (int64_t)(i - 1) * stride; };
    float M = -FLT_MAX, l = 0.f, acc = 0.f;
    for (int i = half; i <= more; i += 2) {
        const float* p = at(i);
        const float mi = p[8 * NT * kD + 2 * col], li = p[8 * NT * kD + 2 * col + 1], x = p[col * kD + dim];
        const float n = fmaxf(M, mi), fa = exp2f(M - n), fb = exp2f(mi - n);
        acc = acc * fa + x * fb;
        l = l * fa + li * fb;
        M = n;
    }
    if (half == 1) { sh[0][threadIdx.x & 127] = M; sh[1][threadIdx.x & 127] = l; sh[2][threadIdx.x & 127] = acc; }
    __syncthreads();
    if (half == 0) {
        const int i = threadIdx.x & 127;
        const float n = fmaxf(M, sh[0][i]), fa = exp2f(M - n), fb = exp2f(sh[0][i] - n);
        kv8_store(a, orow, dim, acc * fa + sh[2][i] * fb, n, l * fa + sh[1][i] * fb);
    }
}

// ------------------------------------------------------------- host side

constexpr int kKv8Least = 16;  // tiles a CTA takes at least: two a warp

template <int NT>
static int kv8_ctas() { return num_sms() * (NT == 1 ? 2 : 1); }

// Columns per warp step: 16 when a sequence has on average more than 8.
static int kv8_nt(int64_t nq, int64_t n_seq, int G) { return nq * G > 8 * n_seq ? 2 : 1; }

template <int NT>
static size_t kv8_ws_bytes() { return (size_t)kv8_ctas<NT>() * 2 * kv8_part_floats<NT>() * sizeof(float); }

template <int FMT, int NT, bool LIST>
static lsa_status launch_kv8_split(const Kv8AttnArgs& a, cudaStream_t st) {
    const int n = kv8_ctas<NT>();
    const size_t smem = (size_t)kKv8Warps * 8 * NT * (kKv8Pad + 2) * sizeof(float);
    cudaFuncSetAttribute(kv8_split_kernel<FMT, NT, LIST>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    lsa_status s;
    {
        KTime kt_("kv8_split_kernel", st);
        kv8_split_kernel<FMT, NT, LIST><<<n, 32 * kKv8Warps, smem, st>>>(a, kKv8Least);
    }
    if ((s = check_launch("kv8_split_kernel")) != LSA_OK) return s;
    {
        KTime kt_("kv8_join_kernel", st);
        kv8_join_kernel<NT, LIST><<<dim3(n - 1, 8 * NT), 32 * kKv8Warps, 0, st>>>(a, n, kKv8Least);
    }
    return check_launch("kv8_join_kernel");
}

static lsa_status check_kv8_attn(const char* what, const lsa_kv8* kv, const uint16_t* Q, int64_t q_stride, int64_t nq,
                                 int32_t hq, const int32_t* table, const int32_t* lens, int32_t n_seq,
                                 int32_t max_pages, const uint16_t* O, const void* ws) {
    lsa_status s;
    if ((s = check_kv8(kv)) != LSA_OK) return s;
    if ((s = check_heads(hq, kv->hkv)) != LSA_OK) return s;
    if (nq < 0 || n_seq < 0 || max_pages < 0) return set_error(LSA_EINVAL, "%s: negative size", what);
    if (nq == 0) return LSA_OK;
    if (n_seq == 0) return set_error(LSA_EINVAL, "%s: queries without a sequence", what);
    if (!Q || !lens || !O || (!table && max_pages > 0)) return set_error(LSA_EINVAL, "%s: NULL pointer", what);
    if (q_stride < (int64_t)hq * kD || (q_stride & 7))
        return set_error(LSA_EINVAL, "%s: q_stride must be a multiple of 8 elements, at least hq * 128", what);
    if (!aligned16(Q) || !aligned16(O) || !aligned16(ws))
        return set_error(LSA_EINVAL, "%s: Q, O and ws must be 16-byte aligned", what);
    if (nq > INT32_MAX || nq * kv->hkv > (int64_t)INT32_MAX * kKv8Warps || (int64_t)max_pages * kv->page > INT32_MAX - 16)
        return set_error(LSA_EUNSUPPORTED, "%s: sizes beyond 2^31", what);
    return LSA_OK;
}

static Kv8AttnArgs kv8_args(const lsa_kv8* kv, const uint16_t* Q, int64_t q_stride, int64_t nq, int32_t hq,
                            const int32_t* table, const int32_t* lens, int32_t n_seq, int32_t max_pages, uint16_t* O,
                            float* lse, void* ws) {
    Kv8AttnArgs a{};
    a.Q = Q; a.q_stride = q_stride; a.nq = nq; a.K = kv->K; a.V = kv->V; a.scale = kv->scale;
    a.table = table; a.lens = lens; a.n_seq = n_seq; a.max_pages = max_pages; a.hkv = kv->hkv; a.G = hq / kv->hkv;
    a.n_pages = kv->n_pages;
    while ((1 << a.lgp) < kv->page) ++a.lgp;
    a.O = O; a.lse = lse; a.part = (float*)ws;
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)kD);
    return a;
}

// Lists: rows that fill the GPU with one warp each take the one-warp kernel.
static bool kv8_many_rows(int64_t nq, int32_t hkv) { return nq * hkv >= (int64_t)num_sms() * 2 * kKv8Warps * 2; }

}  // namespace lsa

extern "C" {

size_t lsa_kv8_attn_workspace_bytes(int64_t nq, int32_t n_seq, int32_t hq, int32_t hkv) {
    using namespace lsa;
    if (nq <= 0 || n_seq <= 0 || check_heads(hq, hkv) != LSA_OK) return 0;
    return kv8_nt(nq, n_seq, hq / hkv) == 1 ? kv8_ws_bytes<1>() : kv8_ws_bytes<2>();
}

lsa_status lsa_kv8_attn(const lsa_kv8* kv, const uint16_t* Q, int64_t q_stride, int64_t nq, int32_t hq,
                        const int32_t* cu, const int32_t* table, const int32_t* lens, int32_t n_seq,
                        int32_t max_pages, int32_t sinks, int32_t window, uint16_t* O, float* lse, void* ws,
                        size_t ws_bytes, void* stream) {
    using namespace lsa;
    lsa_status s;
    if ((s = check_kv8_attn("lsa_kv8_attn", kv, Q, q_stride, nq, hq, table, lens, n_seq, max_pages, O, ws)) != LSA_OK)
        return s;
    if (sinks < 0 || window < 0) return set_error(LSA_EINVAL, "lsa_kv8_attn: need sinks >= 0 and window >= 0");
    if (!cu && nq != n_seq) return set_error(LSA_EINVAL, "lsa_kv8_attn: without cu, nq must equal n_seq");
    if (nq == 0) return LSA_OK;
    if (!ws || ws_bytes < lsa_kv8_attn_workspace_bytes(nq, n_seq, hq, kv->hkv))
        return set_error(LSA_ENOSPACE, "lsa_kv8_attn: workspace too small");
    Kv8AttnArgs a = kv8_args(kv, Q, q_stride, nq, hq, table, lens, n_seq, max_pages, O, lse, ws);
    a.cu = cu; a.S = window > 0 ? sinks : 0; a.W = window;
    const cudaStream_t st = (cudaStream_t)stream;
    const bool one = kv8_nt(nq, n_seq, a.G) == 1;
    if (kv->fmt == LSA_KV8_E4M3) return one ? launch_kv8_split<0, 1, false>(a, st) : launch_kv8_split<0, 2, false>(a, st);
    return one ? launch_kv8_split<1, 1, false>(a, st) : launch_kv8_split<1, 2, false>(a, st);
}

size_t lsa_kv8_sparse_attn_workspace_bytes(int64_t nq, int32_t hq, int32_t hkv) {
    using namespace lsa;
    if (nq <= 0 || check_heads(hq, hkv) != LSA_OK || kv8_many_rows(nq, hkv)) return 0;
    return kv8_ws_bytes<1>();
}

lsa_status lsa_kv8_sparse_attn(const lsa_kv8* kv, const uint16_t* Q, int64_t q_stride, int64_t nq, int32_t hq,
                               const int32_t* seq, const int32_t* table, const int32_t* lens, int32_t n_seq,
                               int32_t max_pages, const int32_t* idx, int32_t n_idx, uint16_t* O, float* lse, void* ws,
                               size_t ws_bytes, void* stream) {
    using namespace lsa;
    lsa_status s;
    if ((s = check_kv8_attn("lsa_kv8_sparse_attn", kv, Q, q_stride, nq, hq, table, lens, n_seq, max_pages, O, ws)) != LSA_OK)
        return s;
    if (n_idx < 0) return set_error(LSA_EINVAL, "lsa_kv8_sparse_attn: n_idx < 0");
    if (n_idx > INT32_MAX - 64) return set_error(LSA_EUNSUPPORTED, "lsa_kv8_sparse_attn: n_idx beyond 2^31");
    if (!seq && nq != n_seq) return set_error(LSA_EINVAL, "lsa_kv8_sparse_attn: without seq, nq must equal n_seq");
    if (nq == 0) return LSA_OK;
    if (!idx && n_idx > 0) return set_error(LSA_EINVAL, "lsa_kv8_sparse_attn: idx is NULL");
    if (ws_bytes < lsa_kv8_sparse_attn_workspace_bytes(nq, hq, kv->hkv) ||
        (!ws && lsa_kv8_sparse_attn_workspace_bytes(nq, hq, kv->hkv) > 0))
        return set_error(LSA_ENOSPACE, "lsa_kv8_sparse_attn: workspace too small");
    Kv8AttnArgs a = kv8_args(kv, Q, q_stride, nq, hq, table, lens, n_seq, max_pages, O, lse, ws);
    a.seq = seq; a.idx = idx; a.n_idx = n_idx;
    const cudaStream_t st = (cudaStream_t)stream;
    if (!kv8_many_rows(nq, kv->hkv))
        return kv->fmt == LSA_KV8_E4M3 ? launch_kv8_split<0, 1, true>(a, st) : launch_kv8_split<1, 1, true>(a, st);
    {
        KTime kt_("kv8_list_kernel", st);
        const unsigned grid = (unsigned)ceil_div<int64_t>(nq * kv->hkv, kKv8Warps);
        if (kv->fmt == LSA_KV8_E4M3) kv8_list_kernel<0><<<grid, 32 * kKv8Warps, 0, st>>>(a);
        else kv8_list_kernel<1><<<grid, 32 * kKv8Warps, 0, st>>>(a);
    }
    return check_launch("kv8_list_kernel");
}

}  // extern "C"
