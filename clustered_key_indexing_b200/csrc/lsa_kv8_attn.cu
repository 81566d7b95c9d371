// lsa_kv8_attn.cu -- exact softmax attention over the paged 8-bit K/V cache
// [tutorial "隐空间稀疏注意力 (LSA)" (diosapp.com.cn), section 二: the attention
// formula is unchanged; essay "《卡片柜》" (zhichai.net), ch. 8: 8-bit storage].
//
// One warp step takes 16 keys of one kv-head against 8 columns (the query
// heads of the group; of several new tokens, 8 or 16 (token, head) pairs):
//   S^T = K Q^T   keys are the MMA's M dimension, columns its N;
//   O^T += V^T P^T.
// Rows of codes travel through a per-warp ring in shared memory (cp.async, two
// steps ahead; through registers instead, with one step ahead, a million
// tokens took 667 us against 420: too few bytes in flight) and are read in an
// order that makes them MMA operands without a shuffle: the K dimension of S^T
// is a permutation of the 128 dims (lane (g, t) holds dims 32 t .. + 31 of two
// key rows, 16 bytes a load; Q follows the same order), its M dimension one of
// the 16 keys, which is the order in which the transposing 8-bit ldmatrix
// leaves V's keys (byte permutes of row-wise loads in its place cost an eighth
// of the step's integer instructions).  Codes become fp16 exactly; Q is divided by its
// row's power of two and becomes fp16 (exact to 2^-17 of the row's largest
// element, absolute error 2^-25 of it below that; with an e4m3 mma.sync for S
// 1000 index rows took 1127 us in place of 960).  P, a probability times its
// key's V scale, is fp16 in units of its column: the largest such product the
// column has attended stands between 2^12 and 2^15, so that a product 2^-26 of
// it still has all its bits, and pages of large values take none from the
// columns that do not attend them.  Scores, softmax sums and outputs are fp32;
// the K scale multiplies the scores.  A column's running maximum and unit move
// only when a score exceeds the maximum by 2 (in base 2) or P would pass 2^15,
// so most steps skip the rescaling.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "lsa_common.cuh"
#include "lsa_mma.cuh"

namespace lsa {

constexpr int kKv8ListWarps = 8;
constexpr float kKv8MostE = 4.f;      // a probability above this moves the running maximum
constexpr float kKv8MostP = 32768.f;  // a P above this the column's unit (fp16 ends at 65504)
constexpr float kKv8TopP = 4096.f;    // P of the product that the unit is taken from
constexpr float kKv8MaxIv = 0x1p112f; // largest 1 / unit: of the smallest V scale, 2^-100, attended whole
static_assert(kKv8MinExp == -100, "the smallest V scale");

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
    int32_t n_seq, max_pages, hkv, G, lgG, lgp, n_idx;
    int32_t S, W;          // dense: sinks and window (W = 0: every key)
    uint16_t* O;           // [nq, hq, 128]
    float* lse;            // [nq, hq] or NULL
    float* part;           // split rows' partial states
    int32_t own;           // a CTA for each row: 1 sequences have one row a kv-head, 2 rows by the scan
    float scale_log2;
};

// ------------------------------------------------------- code conversion

// Four codes to two fp16 pairs (bytes 0, 1 and 2, 3), exact.  int8: the code
// biased by 128 is the low byte of the fp16 number 1024 + code + 128.
template <int FMT>
__device__ __forceinline__ void kv8_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (FMT == 0) {
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
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

// 2^x, subnormal results flushed (they are below 2^-126 of the largest).
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

// ------------------------------------------------------------ warp state

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

template <int NT>
struct Kv8State {
    uint32_t qb[NT][8][2];  // Q as B operands
    float cf[NT][2];        // Q's power of two of columns 2t, 2t + 1
    float o[NT][8][4];
    float m[NT][2], l[NT][2];
    float iv[NT][2];        // 1 / unit: P = probability * V scale * iv, O is in units
};

// Q row of each column (gq within tile nt; NULL: none), dims 32 t .. + 31 on
// this lane, divided by the row's power of two.
template <int NT>
__device__ __forceinline__ void kv8_load_q(Kv8State<NT>& s, const uint16_t* const (&row)[NT]) {
    const int lane = threadIdx.x & 31, tq = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row[nt]) x[i] = __ldg(reinterpret_cast<const uint4*>(row[nt] + 32 * tq + 8 * i));
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
        // |q| < 2^(E - 126): below 1 after the division by 2^e
        const int e = mx == 0u ? 0 : max(-126, min(126, (int)(mx >> 7) - 126));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23), f = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i)  // dims 32 t + 4 i .. + 3
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w = word_of(x[i >> 1], 2 * (i & 1) + h);
                s.qb[nt][i][h] = pack_f16x2(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xFFFF0000u) * inv);
            }
        s.cf[nt][0] = __shfl_sync(0xffffffffu, f, (2 * tq) * 4);
        s.cf[nt][1] = __shfl_sync(0xffffffffu, f, (2 * tq + 1) * 4);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s.o[nt][mt][i] = 0.f;
        s.m[nt][0] = s.m[nt][1] = -FLT_MAX;
        s.l[nt][0] = s.l[nt][1] = 0.f;
        s.iv[nt][0] = s.iv[nt][1] = kKv8MaxIv;
    }
}

// The lane's 32 codes (dims 32 t .. + 31) of key rows g and g + 8.
struct Kv8K {
    uint4 a[2], b[2];
};

// S^T of 16 keys.
template <int FMT, int NT>
__device__ __forceinline__ void kv8_scores(const Kv8State<NT>& s, const Kv8K& k, float (&sc)[NT][4]) {
    float c[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[nt][h][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t a[4];
        kv8_f16<FMT>(word_of(k.a[i >> 2], i & 3), a[0], a[2]);
        kv8_f16<FMT>(word_of(k.b[i >> 2], i & 3), a[1], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816_f16(c[nt][i & 1], a, s.qb[nt][i][0], s.qb[nt][i][1]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[nt][i] = c[nt][0][i] + c[nt][1][i];
}

// V^T of a step as the transposing 8-bit ldmatrix delivers it: the codes of keys
// 4 t .. 4 t + 3 in dims 16 mt + g (w[2 mt]) and 16 mt + g + 8 (w[2 mt + 1]).
struct Kv8V {
    uint32_t w[16];
};

// O^T += V^T P^T: keys 4 t, 4 t + 1 are the MMA's k = 2 t, 2 t + 1 and keys
// 4 t + 2, + 3 its k = 2 t + 8, + 9, which is the order of S^T's rows (kv8_key).
template <int FMT, int NT>
__device__ __forceinline__ void kv8_pv(Kv8State<NT>& s, const Kv8V& v, const uint32_t (&pb)[NT][2]) {
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
        uint32_t a[4];
        kv8_f16<FMT>(v.w[2 * mt], a[0], a[2]);
        kv8_f16<FMT>(v.w[2 * mt + 1], a[1], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816_f16(s.o[nt][mt], a, pb[nt][0], pb[nt][1]);
    }
}

// Key of a step that row g of S^T stands for; row g + 8 is the key two after.
__device__ __forceinline__ int kv8_key(int gq) { return 4 * (gq >> 1) + (gq & 1); }

// 2^-d, 0 from d = 126 on.
__device__ __forceinline__ float pow2_down(int d) { return d < 126 ? __uint_as_float((uint32_t)(127 - d) << 23) : 0.f; }

// Softmax of one step.  Scores in base 2, -inf where masked; vs0, vs1: the V
// scales of rows g and g + 8.  Leaves P^T as B operands in pb.  Scores are taken
// relative to the maximum before anything else is added: next to it the
// differences are exact, however far the floats of large scores are apart.
// ONE_PAGE: all keys of the step have the same V scale.
template <int NT, bool ONE_PAGE>
__device__ __forceinline__ void kv8_softmax(Kv8State<NT>& s, const float (&sc)[NT][4], float vs0, float vs1,
                                            uint32_t (&pb)[NT][2]) {
    float e[NT][4], p[NT][4];
    auto probabilities = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[nt][i] = ex2(sc[nt][i] - s.m[nt][i & 1]);
                // in this order: where e is 0 so is P, although V scale / unit may overflow
                p[nt][i] = e[nt][i] * (i < 2 ? vs0 : vs1) * s.iv[nt][i & 1];
            }
    };
    probabilities();
    float most_e = 0.f, most_p = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            most_e = fmaxf(most_e, e[nt][i]);
            most_p = fmaxf(most_p, p[nt][i]);
        }
    if (__any_sync(0xffffffffu, most_e > kKv8MostE || most_p > kKv8MostP)) {
        float top[NT][2], m[NT][2];  // of each column: the largest score, later product; the new maximum
        auto over_keys = [&]() {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
#pragma unroll
                for (int i = 0; i < 2 * NT; ++i) top[i >> 1][i & 1] = fmaxf(top[i >> 1][i & 1], __shfl_xor_sync(0xffffffffu, top[i >> 1][i & 1], off));
        };
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) top[i >> 1][i & 1] = fmaxf(sc[i >> 1][i & 1], sc[i >> 1][2 + (i & 1)]);
        over_keys();
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            const int nt = i >> 1, c = i & 1;
            // a whole number, so that what was summed before is worth 2^-d, d whole
            m[nt][c] = fmaxf(s.m[nt][c], ceilf(top[nt][c]));
            top[nt][c] = ONE_PAGE ? ex2(top[nt][c] - m[nt][c]) * vs0
                                  : fmaxf(ex2(sc[nt][c] - m[nt][c]) * vs0, ex2(sc[nt][2 + c] - m[nt][c]) * vs1);
        }
        if (!ONE_PAGE) over_keys();
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            const int nt = i >> 1, c = i & 1;
            const int d = (int)fminf(m[nt][c] - s.m[nt][c], 126.f);  // 126 or more: nothing is left
            // 1 / unit: what it was, moved with the maximum, or what makes the step's
            // largest product 2^12, without rounding: where one key outweighs the
            // others, its P is exact
            const float was = s.iv[nt][c], keep = d < 126 ? was * __uint_as_float((uint32_t)(127 + d) << 23) : CUDART_INF_F;
            const float now = fminf(fminf(keep, __fdividef(kKv8TopP, top[nt][c])), kKv8MaxIv);
            const float f = now == keep ? 1.f : d < 126 ? __fdividef(now, was) * pow2_down(d) : 0.f;  // now <= was 2^d
            s.m[nt][c] = m[nt][c];
            s.iv[nt][c] = now;
            s.l[nt][c] *= pow2_down(d);
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                s.o[nt][mt][c] *= f;
                s.o[nt][mt][2 + c] *= f;
            }
        }
        probabilities();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        s.l[nt][0] += e[nt][0] + e[nt][2];
        s.l[nt][1] += e[nt][1] + e[nt][3];
        pb[nt][0] = movmatrix_t(pack_f16x2(p[nt][0], p[nt][1]));
        pb[nt][1] = movmatrix_t(pack_f16x2(p[nt][2], p[nt][3]));
    }
}

// f / l, 0 for a state without a key (a NaN stays).
__device__ __forceinline__ float kv8_over(float f, float l) { return l > 0.f || l != l ? f / l : 0.f; }

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

// ------------------------------------------------- the keys of one row

// A row's keys come in chunks of 32 entries, one a lane: the positions of an
// index list, or (dense) those that the row's mask leaves, in order.
template <bool LIST>
struct Kv8Keys {
    const int32_t* list;   // lists: entries (NULL: none)
    const int32_t* table;  // the sequence's pages
    int32_t len, n_idx, g;
    // dense: chunks [0, n_sink) and from c_lo on; positions of the row's first
    // and last query, first key of the first one's window
    int32_t n_sink, c_lo, tmin, tmax, lo;

    __device__ __forceinline__ int key0(int c) const { return 32 * (c < n_sink ? c : c - n_sink + c_lo); }

    // Entry of this lane in chunk c, -1 for none.
    __device__ __forceinline__ int entry(const Kv8AttnArgs& a, int c, int cend) const {
        const int lane = threadIdx.x & 31;
        if (c >= cend) return -1;
        if constexpr (LIST) {
            const int e = 32 * c + lane;
            return list != nullptr && e < n_idx ? __ldg(list + e) : -1;
        } else {
            const int j = key0(c) + lane;
            return j <= tmax && (j >= lo || j < a.S) ? j : -1;
        }
    }

    // Page of an entry (-1: none, or out of range).  Only the load: what it
    // brings is looked at a chunk later.
    __device__ __forceinline__ int page(const Kv8AttnArgs& a, int p) const {
        const bool ok = LIST ? p >= 0 && p < len : p >= 0;
        return ok ? __ldg(table + (p >> a.lgp)) : -1;
    }

    // Row of codes of an entry from its page, -1 for none.
    __device__ __forceinline__ int row(const Kv8AttnArgs& a, int p, int pid) const {
        if ((uint32_t)pid >= (uint32_t)a.n_pages) {
            if (p >= 0) raise_device_error(LIST && p >= len ? kErrIndexRange : kErrKv8Page);
            return -1;
        }
        return (int)((((uint32_t)pid * a.hkv + g) << a.lgp) | (uint32_t)(p & ((1 << a.lgp) - 1)));
    }
};

__device__ __forceinline__ Kv8Keys<true> kv8_list(const Kv8AttnArgs& a, int64_t q, int g) {
    Kv8Keys<true> r{};
    int64_t b = a.seq ? (int64_t)__ldg(a.seq + q) : q;
    const bool ok = b >= 0 && b < a.n_seq;
    if (!ok) {
        raise_device_error(kErrKv8Range);
        b = 0;
    }
    r.list = ok ? a.idx + (q * a.hkv + g) * (int64_t)a.n_idx : nullptr;
    r.table = a.table + b * a.max_pages;
    r.len = min(__ldg(a.lens + b), a.max_pages << a.lgp);
    r.n_idx = a.n_idx;
    r.g = g;
    return r;
}

// The scales of a row; K's brings the scores to base 2 when it is noted (not
// Q's factor: with a small Q that would be subnormal).
__device__ __forceinline__ float2 kv8_scales(const Kv8AttnArgs& a, int row) {
    return __ldg(reinterpret_cast<const float2*>(a.scale) + (row >> a.lgp));
}

// Which of the 32 entries are keys, and a row for every lane.  A lane without
// a key takes the row of a key of its 16-entry step (row 0 if the step has
// none and is skipped), so that copies need no predicate and what they bring
// is multiplied by a probability of 0 only where that row is attended anyway.
__device__ __forceinline__ unsigned kv8_fill_rows(int& row) {
    const unsigned valid = __ballot_sync(0xffffffffu, row >= 0);
    if (valid != 0xffffffffu) {
        const int step = threadIdx.x & 16;
        const unsigned mine = (valid >> step) & 0xFFFFu;
        const int other = __shfl_sync(0xffffffffu, row, step + (mine ? __ffs(mine) - 1 : 0));
        if (row < 0) row = max(other, 0);
    }
    return valid;
}

// ------------------------------------------------- a warp's ring of steps

// Steps of 16 keys travel through a per-warp ring in shared memory: 16 rows of
// K and 16 of V, 128 bytes each, the 16-byte chunk c of row r at c ^ (r & 7),
// which makes both the copies and the operand reads free of bank conflicts.
constexpr int kKv8Stages = 3;
constexpr int kKv8Step = 16 * kD;                       // bytes of K (or V) in a step
constexpr int kKv8Note = 32 * 8 + 32 * 4;               // a chunk's scales (float2) and rows, beside the ring
constexpr int kKv8Ring = kKv8Stages * 2 * kKv8Step;     // bytes of a warp's ring ...
constexpr int kKv8Warp = kKv8Ring + 2 * kKv8Note + 256; // ... and of all it has (a multiple of 1024)
static_assert(kKv8Warp % 1024 == 0, "rings start on a swizzle's period");

// Where this lane's copies come from and go to.
struct Kv8Copy {
    const uint8_t* K;  // its 16-byte chunk of row 0
    const uint8_t* V;
    uint32_t ring, even, odd;  // places of its chunk in rows r0 and r0 + 4 of a step (r0 = lane / 8)
    uint32_t note;             // two chunks' scales and rows
};

__device__ __forceinline__ Kv8Copy kv8_copy(const Kv8AttnArgs& a, uint32_t ring) {
    const int lane = threadIdx.x & 31, r0 = lane >> 3, c = lane & 7;
    Kv8Copy p;
    p.K = a.K + 16 * c;
    p.V = a.V + 16 * c;
    p.ring = ring;
    p.note = ring + kKv8Ring;
    p.even = ring + r0 * kD + ((c ^ r0) << 4);
    p.odd = ring + (r0 + 4) * kD + ((c ^ (r0 + 4)) << 4);
    return p;
}

__device__ __forceinline__ uint4 lds_16(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}

// A chunk's rows go through shared memory to the lanes that copy them: row 16
// st + 4 i + r as word 16 st + 4 r + i, so that a lane reads its four at once.
__device__ __forceinline__ void kv8_note_rows(uint32_t note, int row) {
    const int e = threadIdx.x & 31;
    asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(note + 256 + 4 * ((e & 16) + 4 * (e & 3) + ((e >> 2) & 3))), "r"(row) : "memory");
}

__device__ __forceinline__ void kv8_note_scales(const Kv8AttnArgs& a, uint32_t note, float2 sc) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};\n" ::"r"(note + 8 * (threadIdx.x & 31)), "f"(sc.x * a.scale_log2), "f"(sc.y)
                 : "memory");
}

__device__ __forceinline__ float2 kv8_scale_of(uint32_t note, int e) {
    float2 s;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];\n" : "=f"(s.x), "=f"(s.y) : "r"(note + 8 * e));
    return s;
}

// Copies of step `st` (0, 1) of the noted rows into the ring slot at byte `slot`.
__device__ __forceinline__ void kv8_issue(const Kv8Copy& p, uint32_t note, int slot, int st, unsigned valid) {
    if (valid) {
        const uint4 r = lds_16(note + 256 + 64 * st + 16 * ((threadIdx.x & 31) >> 3));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = (int32_t)word_of(r, i);
            const uint32_t at = (i & 1 ? p.odd : p.even) + slot + 8 * kD * (i >> 1);
            cp_async_16(at, p.K + row * kD, 16);
            cp_async_16(at + kKv8Step, p.V + row * kD, 16);
        }
    }
    cp_async_commit();
}

__device__ __forceinline__ void kv8_read_k(uint32_t slot, Kv8K& k) {
    const int lane = threadIdx.x & 31, tq = lane & 3, key = kv8_key(lane >> 2);
    const uint32_t p = slot + key * kD + (((2 * tq) ^ (key & 7)) << 4), q = (p ^ 32u) + 2 * kD;
    k.a[0] = lds_16(p);
    k.a[1] = lds_16(p ^ 16u);
    k.b[0] = lds_16(q);
    k.b[1] = lds_16(q ^ 16u);
}

__device__ __forceinline__ void kv8_read_v(uint32_t slot, Kv8V& v) {
    const int lane = threadIdx.x & 31;
    // lanes 0 .. 15 address the rows of dims 32 i .. + 15, the others of + 16 .. + 31
    const uint32_t p = slot + kKv8Step + (lane & 15) * kD + (((lane >> 4) ^ (lane & 7)) << 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(v.w[4 * i]), "=r"(v.w[4 * i + 1]), "=r"(v.w[4 * i + 2]), "=r"(v.w[4 * i + 3])
                     : "r"(p ^ (32u * i)));
}

// O^T += V^T P^T for a step whose mask differs between columns and which holds
// a NaN value: column by column, so that a NaN under one column's mask does
// not reach it through 0 * NaN.
template <int FMT, int NT>
__device__ __forceinline__ void kv8_pv_columns(Kv8State<NT>& s, const Kv8V& v, const uint32_t (&pb)[NT][2],
                                               const int (&tc)[NT][2], int key, int W, int S) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
            const int t = __shfl_sync(0xffffffffu, (c & 1) ? tc[nt][1] : tc[nt][0], c >> 1);
            const uint32_t b0 = gq == c ? pb[nt][0] : 0u, b1 = gq == c ? pb[nt][1] : 0u;
            uint32_t keep = 0u;  // bytes of keys 4 t .. 4 t + 3 that the column attends
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = key + 4 * tq + i;
                if (j <= t && (W == 0 || j > t - W || j < S)) keep |= 0xFFu << (8 * i);
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                uint32_t a[4];
                kv8_f16<FMT>(v.w[2 * mt] & keep, a[0], a[2]);
                kv8_f16<FMT>(v.w[2 * mt + 1] & keep, a[1], a[3]);
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                mma_16816_f16(x, a, b0, b1);
                if (tq == (c >> 1)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((i & 1) == (c & 1)) s.o[nt][mt][i] += x[i];
                }
            }
        }
}

// One step.  note: the 32 rows' scales; valid: the step's 16 keys; tc (dense):
// positions of the lane's columns, -1 for no column; key: the step's first.
template <int FMT, int NT, bool LIST>
__device__ __forceinline__ void kv8_step(const Kv8AttnArgs& a, const Kv8Keys<LIST>& r, Kv8State<NT>& s, uint32_t slot,
                                         uint32_t note, int st, unsigned valid, const int (&tc)[NT][2], int key) {
    const int kr = kv8_key((threadIdx.x & 31) >> 2);  // this lane's keys of the step: kr and kr + 2
    Kv8K k;
    kv8_read_k(slot, k);
    float x[NT][4];
    kv8_scores<FMT, NT>(s, k, x);
    // the 16 keys of a dense step lie in one page
    const float2 s0 = kv8_scale_of(note, 16 * st + (LIST ? kr : 0)), s1 = LIST ? kv8_scale_of(note, 16 * st + kr + 2) : s0;
    const float k0 = s0.x, v0 = s0.y, k1 = s1.x, v1 = s1.y;
    // dense: every column attends all 16 keys
    const bool whole = valid == 0xFFFFu &&
                       (LIST || (key + 15 <= r.tmin && (a.W == 0 || key >= r.lo + (r.tmax - r.tmin) || key + 16 <= a.S)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        x[nt][0] *= k0 * s.cf[nt][0];
        x[nt][1] *= k0 * s.cf[nt][1];
        x[nt][2] *= k1 * s.cf[nt][0];
        x[nt][3] *= k1 * s.cf[nt][1];
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = kr + 2 * (i >> 1);
                bool ok = (valid >> j) & 1u;
                if constexpr (!LIST) {
                    const int t = tc[nt][i & 1];
                    ok = ok && key + j <= t && (a.W == 0 || key + j > t - a.W || key + j < a.S);
                }
                if (!ok) x[nt][i] = -CUDART_INF_F;
            }
        }
    }
    uint32_t pb[NT][2];
    kv8_softmax<NT, !LIST>(s, x, v0, v1, pb);
    Kv8V v;
    kv8_read_v(slot, v);
    if constexpr (FMT == 0 && !LIST) {
        if (!whole && r.tmin != r.tmax) {
            bool nan = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) nan = nan || __vcmpeq4(v.w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u;
            if (__any_sync(0xffffffffu, nan)) {
                kv8_pv_columns<FMT, NT>(s, v, pb, tc, key, a.W, a.S);
                return;
            }
        }
    }
    kv8_pv<FMT, NT>(s, v, pb);
}

// Chunks c, c + STEP, ... below cend of a row into the warp's state.  Copies
// run two steps ahead of their use, page numbers and scales a chunk further,
// list entries two.  start() sends the first chunk on its way, so that Q can be
// read meanwhile.
template <bool LIST, int STEP>
struct Kv8Walk {
    Kv8Copy cp;
    int c, cend;
    int p1, pid1, p2;
    unsigned valid;

    __device__ __forceinline__ void start(const Kv8AttnArgs& a, const Kv8Keys<LIST>& r, int c_, int cend_, uint32_t ring) {
        c = c_;
        cend = cend_;
        cp = kv8_copy(a, ring);
        const int p0 = r.entry(a, c, cend);
        p1 = r.entry(a, c + STEP, cend);
        p2 = r.entry(a, c + 2 * STEP, cend);
        const int pid0 = r.page(a, p0);
        pid1 = r.page(a, p1);
        int row = r.row(a, p0, pid0);
        valid = kv8_fill_rows(row);
        kv8_note_rows(cp.note, row);
        __syncwarp();
        kv8_issue(cp, cp.note, 0, 0, valid & 0xFFFFu);
        kv8_issue(cp, cp.note, 2 * kKv8Step, 1, valid >> 16);
        kv8_note_scales(a, cp.note, kv8_scales(a, row));
    }

    template <int FMT, int NT>
    __device__ __forceinline__ void run(const Kv8AttnArgs& a, const Kv8Keys<LIST>& r, const int (&tc)[NT][2], Kv8State<NT>& s) {
        constexpr int kSlot = 2 * kKv8Step, kLast = (kKv8Stages - 1) * kSlot;
        int slot = 0;
        uint32_t note = cp.note, note1 = cp.note + kKv8Note;
        for (; c < cend; c += STEP) {
            int row1 = r.row(a, p1, pid1);
            const unsigned valid1 = kv8_fill_rows(row1);
            const int key = LIST ? 0 : r.key0(c);
            kv8_note_rows(note1, row1);
            const float2 sc1 = kv8_scales(a, row1);
            cp_async_wait<1>();
            __syncwarp();
            kv8_issue(cp, note1, slot == 0 ? kLast : slot - kSlot, 0, valid1 & 0xFFFFu);
            const int pid2 = r.page(a, p2), p3 = r.entry(a, c + 3 * STEP, cend);
            if (valid & 0xFFFFu) kv8_step<FMT, NT, LIST>(a, r, s, cp.ring + slot, note, 0, valid & 0xFFFFu, tc, key);
            cp_async_wait<1>();
            __syncwarp();
            kv8_issue(cp, note1, slot, 1, valid1 >> 16);
            slot = slot == kLast ? 0 : slot + kSlot;
            if (valid >> 16) kv8_step<FMT, NT, LIST>(a, r, s, cp.ring + slot, note, 1, valid >> 16, tc, key + 16);
            slot = slot == kLast ? 0 : slot + kSlot;
            kv8_note_scales(a, note1, sc1);
            const uint32_t other = note;
            note = note1;
            note1 = other;
            p1 = p2; pid1 = pid2; p2 = p3; valid = valid1;
        }
        cp_async_wait<0>();
        __syncwarp();
    }
};

// Many rows: one warp per (query, kv-head), kv-head major so that the warps
// resident at one time read one head's rows, which keeps them in L2.  A step
// is about 240 instructions, 115 of them integer and conversion (64 turn codes
// into fp16, two cycles each): 59% of that pipe's cycles, 62% of the issue slots
// and 62% of the L1 data pipe are used, the tensor pipe a third; the copies alone
// take 324 us.  1000 rows x 8 kv-heads of 3076 entries: 561 us captured, 11.4
// TB/s from L2 (bf16 rows of the same keys are twice the bytes; int8 codes, five
// instructions for four values instead of two, 729).  A third of the entries are
// windows that neighbouring queries share; each reads its own.  Two steps
// interleaved with 12 warps an SM took 686 us instead of 603, 20 warps of 96
// registers 684.
template <int FMT>
__global__ void __launch_bounds__(32 * kKv8ListWarps, 2) kv8_list_kernel(Kv8AttnArgs a) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const int64_t wg = (int64_t)blockIdx.x * kKv8ListWarps + (threadIdx.x >> 5);
    if (wg >= a.nq * a.hkv) return;
    const int64_t q = wg % a.nq;
    const int g = (int)(wg / a.nq);
    const int hq = a.G * a.hkv;
    Kv8State<1> s;
    const uint16_t* const row[1] = {gq < a.G ? a.Q + q * a.q_stride + (int64_t)(g * a.G + gq) * kD : nullptr};
    const Kv8Keys<true> r = kv8_list(a, q, g);
    extern __shared__ __align__(1024) uint8_t lsm[];
    const int tc[1][2] = {{0, 0}};
    Kv8Walk<true, 1> walk;
    walk.start(a, r, 0, (a.n_idx + 31) / 32, smem_u32(lsm) + (threadIdx.x >> 5) * kKv8Warp);
    kv8_load_q<1>(s, row);
    walk.template run<FMT, 1>(a, r, tc, s);
    kv8_reduce_l<1>(s);
    // through shared memory (the ring's), [8][128] bf16, to whole lines
    uint16_t* os = reinterpret_cast<uint16_t*>(lsm + (threadIdx.x >> 5) * kKv8Warp);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float l = s.l[0][c], f = kv8_over(1.f / s.iv[0][c], l);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            os[(2 * tq + c) * kD + 16 * mt + gq] = bf16_bits(s.o[0][mt][c] * f);
            os[(2 * tq + c) * kD + 16 * mt + gq + 8] = bf16_bits(s.o[0][mt][2 + c] * f);
        }
        if (a.lse && gq == 0 && 2 * tq + c < a.G)
            a.lse[q * hq + g * a.G + 2 * tq + c] = l > 0.f || l != l ? s.m[0][c] + log2f(l) : -CUDART_INF_F;
    }
    __syncwarp();
    uint4* orow = reinterpret_cast<uint4*>(a.O + (q * hq + g * a.G) * kD);
    for (int c = lane; c < a.G * kD / 8; c += 32) orow[c] = reinterpret_cast<const uint4*>(os)[c];
}

// ------------------------------------------------ rows split over the GPU

// The work is one stream of 32-key chunks: rows in the order (sequence,
// kv-head, column group), each with the chunks its mask leaves (at least one).
// CTA c takes chunks [c per, (c + 1) per): the same work for every CTA however
// ragged the lengths.  A row inside one CTA's range is finished there; a row
// that crosses CTAs leaves a partial state in every CTA it touches (slot 0 if
// it began before the CTA, slot 1 if it began inside), and kv8_join_kernel
// joins them.  Everyone derives the stream from lens and cu by the same scan.
// Where the call's shapes alone say that every row is short, each row gets a
// CTA of its own instead (own > 0), or where rows are few a cluster of 2, 4 or 8,
// whose CTAs take equal shares and join their sums through one another's shared
// memory: no second kernel, no workspace.  8 rows of 282 chunks (9000 tokens):
// 12.1 us, 17.8 in the stream (captured).  A row's bound comes from the table's
// width: 777 tokens take 6.8 us in a table of their size, 11.1 in one for 128K.
//
// Bound by HBM (captured, calls on the same cache): a million tokens of 8
// kv-heads (2.15 GB) in 340 to 350 us, 32 sequences of 2K to 32K tokens (1.21 GB)
// in 193 us, 6.2 TB/s; the warps of a CTA take neighbouring chunks, so that it
// reads whole pages at a time.
struct Kv8Seq {
    int64_t base;     // first chunk of the sequence in the stream
    int32_t chunks;   // chunks of each of its rows
    int32_t rows;     // hkv * column groups
    int32_t groups;
    int32_t n, len;   // new tokens, tokens in all
    int64_t q0;
    int32_t n_sink, c_lo;  // chunks [0, n_sink) and from c_lo on
};

template <int NT, bool LIST>
__device__ __forceinline__ void kv8_seq(const Kv8AttnArgs& a, int64_t b, Kv8Seq& q) {
    if constexpr (LIST) {  // "sequence" b is query b
        q.n = 1; q.q0 = b; q.len = 0; q.groups = 1; q.rows = a.hkv; q.n_sink = 0; q.c_lo = 0;
        q.chunks = max(1, (a.n_idx + 31) / 32);
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
        const int hi = (int)((len + 31) / 32);
        const int64_t lo = a.W > 0 ? len - n - a.W + 1 : 0;  // the first query's window begins there
        q.c_lo = lo > 0 ? (int)(lo / 32) : 0;
        q.n_sink = min((min(a.S, (int)len) + 31) / 32, q.c_lo);
        q.chunks = max(1, q.n_sink + hi - q.c_lo);
    }
}

// What a row costs a CTA of the stream beside its chunks, in chunks: its last
// warp is waited for, its sums are joined, the next one's copies begin.  It
// counts in the shares where they are long enough (kKv8Padded chunks a CTA), or
// CTAs with many short rows would come last (64 sequences of 480 to 8000 tokens,
// one call after another: 98 us, 124 without; 8 and 32 in place of 16 104 and 99).
constexpr int kKv8RowCost = 16, kKv8Padded = 64;

// A sequence's share of a stream: its chunks and its rows' cost, or (ROWS) its rows.
template <int NT, bool LIST, int WARPS = kKv8Warps, bool ROWS = false>
struct Kv8Scan {
    int64_t total, per;
    int pad;                        // what a row counts beside its chunks
    long long begin, count, round;  // this thread's sequence in the CTA's first round: its place, its share; the round's

    __device__ __forceinline__ long long share_of(const Kv8AttnArgs& a, int64_t b) const {
        if (b >= a.n_seq) return 0;
        Kv8Seq q;
        kv8_seq<NT, LIST>(a, b, q);
        return ROWS ? q.rows : (int64_t)(q.chunks + pad) * q.rows;
    }
    __device__ __forceinline__ void sum(const Kv8AttnArgs& a) {
        count = share_of(a, threadIdx.x);
        begin = kv8_block_scan<WARPS>(count, round);
        total = round;
        for (int64_t b0 = 32 * WARPS; b0 < a.n_seq; b0 += 32 * WARPS) {
            long long all;
            kv8_block_scan<WARPS>(share_of(a, b0 + threadIdx.x), all);
            total += all;
        }
    }
    // The stream's length and each CTA's share of it (`least`: a CTA takes at
    // least so much).
    __device__ __forceinline__ void init(const Kv8AttnArgs& a, int n_cta, int least) {
        pad = 0;
        if constexpr (LIST) {
            total = a.nq * a.hkv * (int64_t)max(1, (a.n_idx + 31) / 32);
        } else {
            sum(a);
            if (!ROWS && total >= (int64_t)kKv8Padded * n_cta) {
                pad = kKv8RowCost;
                sum(a);
            }
        }
        // `least` a CTA, but no more than the rows have on average: short rows
        // are not queued behind one another while CTAs are idle
        const int64_t rows = (LIST ? a.nq : (int64_t)a.n_seq) * a.hkv;
        const int64_t few = total < rows * least ? max((int64_t)1, (total + rows - 1) / rows) : least;
        per = max(few, (total + n_cta - 1) / n_cta);
    }
    // The sequence that holds position w of the stream (0 <= w < total).
    __device__ __forceinline__ int64_t find(const Kv8AttnArgs& a, int64_t w, Kv8Seq& out) {
        int64_t b, base;
        if constexpr (LIST) {
            b = w / (total / a.nq);
            base = b * (total / a.nq);
        } else {
            __shared__ long long found[2];
            long long first = begin, m = count, end = round;
            b = threadIdx.x;
            while (w >= end) {  // uniform
                long long all;
                b += 32 * WARPS;
                m = share_of(a, b);
                first = end + kv8_block_scan<WARPS>(m, all);
                end += all;
            }
            if (w >= first && w < first + m) { found[0] = b; found[1] = first; }
            __syncthreads();
            b = found[0];
            base = found[1];
        }
        kv8_seq<NT, LIST>(a, b, out);
        out.base = base;
        return b;
    }
};

constexpr int kKv8Pad = kD + 4;  // floats per column in shared memory: consecutive columns start 4 banks apart

// Floats of one partial state: 8 NT columns of 128 sums, then (m, l) each.
template <int NT>
__host__ __device__ constexpr int kv8_part_floats() { return 8 * NT * (kD + 2); }

// Output row of column c of a row: column group cg, kv-head g of a sequence.
template <int NT>
__device__ __forceinline__ int64_t kv8_out_row(const Kv8AttnArgs& a, const Kv8Seq& q, int cg, int g, int c) {
    const int64_t cc = (int64_t)cg * 8 * NT + c;
    if (cc >= (int64_t)q.n * a.G) return -1;
    return (q.q0 + (cc >> a.lgG)) * (a.G * a.hkv) + g * a.G + (cc & (a.G - 1));
}

constexpr int kKv8Cluster = 8;  // CTAs of a cluster at most

// Partial states are kept as (m, l) and the output that their keys alone would
// give, which is within V's range.  Sums of l times that are not, before they are
// divided by l: joins scale them by 2^-k, with 2^k at least the row's l (a key's
// probability is 4 at most).
struct Kv8Join {
    float down, up;  // 2^-k, 2^k
    float M, l;
    float4 acc;

    __device__ __forceinline__ explicit Kv8Join(int chunks) {
        const int k = 39 - __clz(chunks);  // 2^k > 4 * 32 * chunks
        down = __uint_as_float((uint32_t)(127 - k) << 23);
        up = __uint_as_float((uint32_t)(127 + k) << 23);
        M = -FLT_MAX;
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // One state more: x times weight, both relative to M.
    __device__ __forceinline__ void add(const float4& x, float weight) {
        l += weight;
        weight *= down;
        acc = make_float4(acc.x + x.x * weight, acc.y + x.y * weight, acc.z + x.z * weight, acc.w + x.w * weight);
    }
    // A state with a maximum of its own.
    __device__ __forceinline__ void add(const float4& x, float2 ml) {
        const float m = fmaxf(M, ml.x), f = ex2(M - m);
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
        l *= f;
        M = m;
        add(x, ml.y * ex2(ml.x - m));
    }
    // Another join of the same row.
    __device__ __forceinline__ void merge(const float4& x, float2 ml) {
        const float m = fmaxf(M, ml.x), f = ex2(M - m), g = ex2(ml.x - m);
        acc = make_float4(acc.x * f + x.x * g, acc.y * f + x.y * g, acc.z * f + x.z * g, acc.w * f + x.w * g);
        l = l * f + ml.y * g;
        M = m;
    }
    __device__ __forceinline__ float4 out() const {
        const float f = kv8_over(up, l);
        return make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    }
};

// Four elements of one output row (dims d .. d + 3).
__device__ __forceinline__ void kv8_store(const Kv8AttnArgs& a, int64_t orow, int d, const Kv8Join& j) {
    const float4 x = j.out();
    *reinterpret_cast<uint2*>(a.O + orow * kD + d) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    if (d == 0 && a.lse) a.lse[orow] = j.l > 0.f || j.l != j.l ? j.M + log2f(j.l) : -CUDART_INF_F;
}

// Number of this CTA in its cluster, CTAs of the cluster, the cluster's barrier
// (which orders shared memory), and a load from CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

__device__ __forceinline__ uint32_t peer_smem(uint32_t p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(p), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 peer_f4(uint32_t p) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p) : "memory");
    return v;
}

__device__ __forceinline__ float2 peer_f2(uint32_t p) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(p) : "memory");
    return v;
}

// WARPS = 16 (twice the steps at a time, one CTA an SM): only a CTA or cluster a row.
template <int FMT, int NT, bool LIST, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, NT == 1 && WARPS == 8 ? 2 : 1) kv8_split_kernel(Kv8AttnArgs a, int least) {
    extern __shared__ __align__(1024) uint8_t ksm[];
    constexpr bool CLUSTER = WARPS != kKv8Warps || NT == 2;  // may run as clusters
    __shared__ __align__(8) float sml[WARPS * 8 * NT * 2];                     // (m, l) of every warp's columns
    __shared__ __align__(8) float cml[CLUSTER ? 8 * NT * 2 : 2];               // and of the CTA's, for its cluster
    // what a CTA of the stream knows of its row stands here while the keys are
    // walked, for which every register is needed (a CTA that has one row only
    // would wait for it: 777 tokens 6.8 us, 6.4 without)
    __shared__ struct { Kv8Seq q; int64_t b, w, w1; int32_t g, cg, pad; bool whole, begins; } s_row;
    const uint32_t ring = smem_u32(ksm) + (threadIdx.x >> 5) * kKv8Warp;
    // a warp's sums go where its ring was: [8 NT][kKv8Pad] floats
    auto so = [&](int w) { return reinterpret_cast<float*>(ksm + w * kKv8Warp); };
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, gq = lane >> 2, tq = lane & 3;
    // a CTA's sums of column c, for its cluster: behind the sums in warp c % 8's ring
    auto sc = [&](int c) { return ksm + (c & 7) * kKv8Warp + 8 * NT * kKv8Pad * 4 + (c >> 3) * kD * 4; };
    static_assert(8 * NT * kKv8Pad * 4 + NT * kD * 4 <= kKv8Warp, "sums fit");
    constexpr bool kStream = WARPS == kKv8Warps;   // may take pieces of the stream
    const bool own = !kStream || a.own;            // a CTA or a cluster for each row
    const int csize = CLUSTER && own ? (int)cluster_size() : 1;
    Kv8Seq q;
    int64_t b, w0 = 0, w1 = 0;
    int r = 0, t0 = 0, n = 0;  // row of the sequence, its first chunk here, how many
    int pad = 0;
    if (own) {
        const int item = (int)(blockIdx.x / csize);
        if (LIST || a.own == 1) {
            b = item / a.hkv;
            r = item % a.hkv;
            kv8_seq<NT, LIST>(a, b, q);
            if (q.rows == 0) return;
        } else {
            Kv8Scan<NT, LIST, WARPS, true> scan;
            scan.init(a, (int)gridDim.x, 1);
            if (item >= scan.total) return;
            b = scan.find(a, item, q);
            r = (int)(item - q.base);
        }
        const int per = (q.chunks + csize - 1) / csize;
        t0 = CLUSTER && csize > 1 ? (int)cluster_rank() * per : 0;
        n = max(0, min(per, q.chunks - t0));
    } else {
        asm volatile("griddepcontrol.launch_dependents;\n");
        Kv8Scan<NT, LIST> scan;
        scan.init(a, (int)gridDim.x, least);
        w0 = (int64_t)blockIdx.x * scan.per;
        w1 = min(scan.total, w0 + scan.per);
        if (w0 >= w1) return;
        b = scan.find(a, w0, q);
        pad = scan.pad;
    }
    for (int64_t w = w0;;) {
        bool whole = true, begins = true;  // the piece is the whole row, begins it
        if (!own) {
            while (w >= q.base + (int64_t)(q.chunks + pad) * q.rows) {  // the next sequence that has rows
                const int64_t next = q.base + (int64_t)(q.chunks + pad) * q.rows;
                kv8_seq<NT, LIST>(a, ++b, q);
                q.base = next;
            }
            const int units = q.chunks + pad;
            const int64_t rel = w - q.base;
            r = rel >> 31 ? (int)(rel / units) : (int)((uint32_t)rel / (uint32_t)units);
            const int u0 = (int)(rel - (int64_t)r * units), nu = (int)min((int64_t)(units - u0), w1 - w);
            begins = u0 == 0;
            whole = nu == units;
            t0 = max(0, u0 - pad);
            n = max(0, u0 + nu - pad) - t0;
            w += nu;
        }
        int g = r / q.groups, cg = r % q.groups;
        const int ta = t0 + wid, tb = t0 + n;  // neighbouring chunks at the same time: whole pages of DRAM
        if (kStream && tid == 0) s_row = {q, b, w, w1, g, cg, pad, whole, begins};

        if (ta < tb) {
            Kv8State<NT> s;
            Kv8Keys<LIST> keys{};
            int tc[NT][2] = {};
            if constexpr (LIST) {
                keys = kv8_list(a, q.q0, g);
            } else {
                const int first = q.len - q.n;  // position of the sequence's first query
                const int c0 = cg * 8 * NT, c1 = min((int)(q.n * a.G), c0 + 8 * NT) - 1;
                keys.table = a.table + b * a.max_pages;
                keys.len = q.len;
                keys.g = g;
                keys.n_sink = q.n_sink;
                keys.c_lo = q.c_lo;
                keys.tmin = first + (c0 >> a.lgG);
                keys.tmax = first + (c1 >> a.lgG);
                keys.lo = a.W > 0 ? keys.tmin - a.W + 1 : 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int cc = c0 + 8 * nt + 2 * tq + c;
                        tc[nt][c] = cc <= c1 ? first + (cc >> a.lgG) : -1;
                    }
            }
            Kv8Walk<LIST, WARPS> walk;
            walk.start(a, keys, ta, tb, ring);
            const uint16_t* row[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int64_t cc = (int64_t)cg * 8 * NT + 8 * nt + gq;
                row[nt] = cc < (int64_t)q.n * a.G
                              ? a.Q + (q.q0 + (cc >> a.lgG)) * a.q_stride + (g * a.G + (cc & (a.G - 1))) * kD : nullptr;
            }
            const uint16_t* const (&crow)[NT] = row;
            kv8_load_q<NT>(s, crow);
            walk.template run<FMT, NT>(a, keys, tc, s);
            kv8_reduce_l<NT>(s);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = wid * 8 * NT + 8 * nt + 2 * tq + c;
                    float* p = so(wid) + (8 * nt + 2 * tq + c) * kKv8Pad + gq;
                    const float f = kv8_over(1.f / s.iv[nt][c], s.l[nt][c]);
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                        p[16 * mt] = s.o[nt][mt][c] * f;
                        p[16 * mt + 8] = s.o[nt][mt][2 + c] * f;
                    }
                    if (gq == 0) { sml[2 * col] = s.m[nt][c]; sml[2 * col + 1] = s.l[nt][c]; }
                }
        } else {
            for (int col = lane; col < 8 * NT; col += 32) {
                sml[2 * (wid * 8 * NT + col)] = -FLT_MAX;
                sml[2 * (wid * 8 * NT + col) + 1] = -1.f;  // took no chunk
            }
        }
        __syncthreads();
        if (kStream) {
            q = s_row.q; b = s_row.b; w = s_row.w; w1 = s_row.w1;
            g = s_row.g; cg = s_row.cg; pad = s_row.pad; whole = s_row.whole; begins = s_row.begins;
        }
        float* part = a.part + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * kv8_part_floats<NT>();
        for (int e = tid; e < 8 * NT * kD / 4; e += 32 * WARPS) {  // four sums of a column
            const int c = e / (kD / 4), dim = e % (kD / 4) * 4;
            const int64_t orow = kv8_out_row<NT>(a, q, cg, g, c);
            if (orow < 0) continue;
            Kv8Join join(q.chunks);
            float weight[WARPS];
#pragma unroll
            for (int i = 0; i < WARPS; ++i) join.M = fmaxf(join.M, sml[2 * (i * 8 * NT + c)]);
#pragma unroll
            for (int i = 0; i < WARPS; ++i) {
                const float2 ml = *reinterpret_cast<const float2*>(sml + 2 * (i * 8 * NT + c));
                weight[i] = ml.y == -1.f ? 0.f : ml.y * ex2(ml.x - join.M);
            }
#pragma unroll
            for (int i = 0; i < WARPS; ++i) {
                if (weight[i] != 0.f) join.add(*reinterpret_cast<const float4*>(so(i) + c * kKv8Pad + dim), weight[i]);
            }
            if (CLUSTER && csize > 1) {
                *reinterpret_cast<float4*>(sc(c) + dim * 4) = join.out();
                if (dim == 0) *reinterpret_cast<float2*>(cml + 2 * c) = make_float2(join.M, join.l);
            } else if (whole) {
                kv8_store(a, orow, dim, join);
            } else {
                *reinterpret_cast<float4*>(part + c * kD + dim) = join.out();
                if (dim == 0) *reinterpret_cast<float2*>(part + 8 * NT * kD + 2 * c) = make_float2(join.M, join.l);
            }
        }
        if (CLUSTER && csize > 1) {
            cluster_barrier();
            for (int e = (int)cluster_rank() * 32 * WARPS + tid; e < 8 * NT * kD / 4; e += csize * 32 * WARPS) {
                const int c = e / (kD / 4), dim = e % (kD / 4) * 4;
                const int64_t orow = kv8_out_row<NT>(a, q, cg, g, c);
                if (orow < 0) continue;
                const uint32_t pm = smem_u32(cml + 2 * c), ps = smem_u32(sc(c) + dim * 4);
                Kv8Join join(q.chunks);
                float2 ml[kKv8Cluster];
                float4 x[kKv8Cluster];
#pragma unroll
                for (int i = 0; i < kKv8Cluster; ++i) {
                    ml[i] = make_float2(-FLT_MAX, 0.f);
                    x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < csize) {
                        ml[i] = peer_f2(peer_smem(pm, i));
                        x[i] = peer_f4(peer_smem(ps, i));
                    }
                    join.M = fmaxf(join.M, ml[i].x);
                }
#pragma unroll
                for (int i = 0; i < kKv8Cluster; ++i) join.add(x[i], ml[i].y * ex2(ml[i].x - join.M));
                kv8_store(a, orow, dim, join);
            }
            cluster_barrier();  // nobody leaves while others read its sums
            return;
        }
        if (own || w >= w1) return;
        __syncthreads();
    }
}

// One column of n partial states, a lane four of its elements: states i0, i0 +
// di, ... of which the first is CTA c's slot 1 and the others the slots 0 of the
// CTAs after it.
template <int NT>
__device__ __forceinline__ void kv8_join_column(const Kv8AttnArgs& a, int64_t c, int col, int i0, int di, int n, Kv8Join& join) {
    constexpr int kPart = kv8_part_floats<NT>();
    const int lane = threadIdx.x & 31;
#pragma unroll 4
    for (int i = i0; i < n; i += di) {
        const float* p = a.part + (2 * (c + i) + (i == 0)) * kPart;
        const float2 ml = *reinterpret_cast<const float2*>(p + 8 * NT * kD + 2 * col);
        join.add(*reinterpret_cast<const float4*>(p + col * kD + 4 * lane), ml);
    }
}

// Joins the row that crosses the end of CTA c's range, if that row began
// inside it.  gridDim.y == 1 (rows in few pieces): a warp takes whole columns;
// else blockIdx.y is the column and every warp takes each eighth state.
template <int NT, bool LIST>
__global__ void __launch_bounds__(32 * kKv8Warps) kv8_join_kernel(Kv8AttnArgs a, int n_cta, int least) {
    Kv8Scan<NT, LIST> scan;
    scan.init(a, n_cta, least);
    const int64_t c = blockIdx.x, w0 = c * scan.per, w1 = w0 + scan.per;
    Kv8Seq q{};
    if (w1 < scan.total) scan.find(a, w1, q);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // before any exit: this grid's end is the call's end
    if (w1 >= scan.total) return;
    const int units = q.chunks + scan.pad;
    const int64_t rel = w1 - q.base;
    const int r = rel >> 31 ? (int)(rel / units) : (int)((uint32_t)rel / (uint32_t)units);
    const int64_t begin = q.base + (int64_t)r * units, end = begin + units;
    if (begin == w1 || begin < w0) return;
    const int n = (int)((end - 1) / scan.per - c) + 1;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, cg = r % q.groups, g = r / q.groups;
    if (gridDim.y == 1) {
        for (int col = wid; col < 8 * NT; col += kKv8Warps) {
            const int64_t orow = kv8_out_row<NT>(a, q, cg, g, col);
            if (orow < 0) return;
            Kv8Join join(q.chunks);
            kv8_join_column<NT>(a, c, col, 0, 1, n, join);
            kv8_store(a, orow, 4 * lane, join);
        }
        return;
    }
    const int64_t orow = kv8_out_row<NT>(a, q, cg, g, blockIdx.y);
    if (orow < 0) return;
    __shared__ float4 s_acc[kKv8Warps][32];
    __shared__ float2 s_ml[kKv8Warps];
    Kv8Join join(q.chunks);
    kv8_join_column<NT>(a, c, blockIdx.y, wid, kKv8Warps, n, join);
    s_acc[wid][lane] = join.acc;
    if (lane == 0) s_ml[wid] = make_float2(join.M, join.l);
    __syncthreads();
    if (wid > 0) return;
#pragma unroll
    for (int i = 1; i < kKv8Warps; ++i) join.merge(s_acc[i][lane], s_ml[i]);
    kv8_store(a, orow, 4 * lane, join);
}

// ------------------------------------------------------------- host side

// Chunks a CTA of the stream takes at least (one a warp).
constexpr int kKv8Least = 8;

template <int NT>
static int kv8_ctas() { return num_sms() * (NT == 1 ? 2 : 1); }

// Columns per warp step: 16 when a sequence has on average more than 8, which
// halves what is read; where little is, 8 columns and twice the rows are quicker
// by up to 1.7 us (us, 16 / 8 columns, captured; 8 kv-heads of 4 heads unless said
// otherwise: 4 new tokens on 128K 76 / 106, 32 x 5 on 32K 755 / 969, 4 x 64 on 4K
// 133 / 159; 2 kv-heads of 8 heads, a window of 1024: 16 x 5 16.6 / 17.2, 64 x 5
// 45 / 41, 1 x 5 10.0 / 8.5).
static int kv8_nt(int64_t nq, int64_t n_seq, int G) { return nq * G > 8 * n_seq ? 2 : 1; }

// A kernel's dynamic shared memory limit, raised once a device.
static void kv8_allow_smem(const void* kern, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess)
        done.fetch_or(bit, std::memory_order_release);
}

// Clusters of 2^lg CTAs (one an SM) that run at the same time: fewer than the SMs
// make, because a cluster stays inside a group of SMs.  Asked once a device.
static int kv8_clusters(int lg) {
    static std::atomic<int> known[64][4];
    static std::atomic<uint64_t> allowed{0};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return num_sms() * 3 / 4 >> lg;
    if (dev >= 0 && dev < 64 && (n = known[dev][lg].load(std::memory_order_relaxed)) > 0) return n;
    const auto kern = kv8_split_kernel<0, 1, false, 16>;
    constexpr size_t smem = 16 * kKv8Warp;
    kv8_allow_smem((const void*)kern, smem, allowed);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(num_sms() >> lg << lg);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {1u << lg, 1u, 1u};
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();
        n = num_sms() * 3 / 4 >> lg;
    }
    if (dev >= 0 && dev < 64) known[dev][lg].store(n, std::memory_order_relaxed);
    return n;
}

// Chunks a CTA may have of a row that is not in the stream, where `ctas` of them
// run: a CTA takes 4.5 us and 2 us for a chunk of each of its 16 warps; the
// stream 13 us, and then the same on all SMs (its shares are equal, so the cap
// is for rows of unequal lengths).  More CTAs than SMs, two of 8 warps an SM: 128
// where they nearly fill the GPU once (own / stream, us: 256 rows of 125 chunks
// 48 / 54, of unequal lengths up to that 43 / 48), else 64 (384 rows of 125
// 82 / 73, 60 / 49; of 63 46 / 45, 36 / 47; 1024 rows of 94 131 / 141, 87 / 83).
static int64_t kv8_cta_chunks(int64_t ctas) {
    const int64_t n = num_sms();
    if (ctas > n) return 4 * ctas >= 5 * n && ctas <= 2 * n ? 128 : 64;
    return std::min<int64_t>(160, 720 * n / (10 * n - 9 * ctas));
}

// How a call's rows meet the GPU: one warp a row (lists only), one CTA or
// cluster a row (rows > 0 of them at most), or the stream (rows = 0).  It goes
// by what the host knows: the numbers of rows and an upper bound of a row's
// chunks.
struct Kv8Plan {
    int nt;
    bool warps;
    int64_t rows;
    int cluster;  // CTAs of a row
    size_t ws;
};

static Kv8Plan kv8_plan(bool lists, int64_t nq, int64_t n_seq, int G, int32_t hkv, bool one_each, int64_t max_chunks) {
    Kv8Plan p{};
    p.nt = lists ? 1 : kv8_nt(nq, n_seq, G);
    p.cluster = 1;
    const int ctas = p.nt == 1 ? kv8_ctas<1>() : kv8_ctas<2>(), C = 8 * p.nt;
    // lists: a warp a row from 1184 rows on (half the warps that fit), of short
    // lists from 592 on.  Measured (warp / CTA a row, us): 97 chunks, 1024 rows
    // 105 / 104, 2368 rows 169 / 218, 8000 rows 563 / 712; 25 chunks, 512 rows
    // 30 / 23, 1024 rows 33 / 42; 7 chunks, 512 rows 12 / 13
    p.warps = lists && (nq * hkv >= 4 * ctas || (nq * hkv >= 2 * ctas && max_chunks <= 32));
    if (p.warps) return p;
    // rows at most (a sequence's last group of columns may be a part), and with
    // equally many new tokens a sequence
    const bool each = lists || one_each;
    const int64_t rows = each ? nq * hkv : hkv * ((nq * G + n_seq * (C - G)) / C);
    const int64_t likely = each ? rows : std::min(rows, hkv * n_seq * ceil_div<int64_t>(ceil_div<int64_t>(nq, n_seq) * G, C));
    for (int lg = 3; lg > 0 && p.cluster == 1; --lg)
        if (max_chunks > 16 && max_chunks > 4 << lg && likely <= kv8_clusters(lg)) p.cluster = 1 << lg;
    if (max_chunks <= p.cluster * kv8_cta_chunks(likely * p.cluster) && rows * p.cluster <= INT32_MAX) p.rows = rows;
    else p.ws = (size_t)ctas * 2 * (p.nt == 1 ? kv8_part_floats<1>() : kv8_part_floats<2>()) * sizeof(float);
    return p;
}

// Chunks a dense row has at most.
static int64_t kv8_max_chunks(int64_t nq, int32_t page, int32_t max_pages, int32_t sinks, int32_t window) {
    const int64_t all = ceil_div<int64_t>((int64_t)max_pages * page, 32);
    if (window <= 0) return all;
    const int64_t some = ceil_div<int64_t>(sinks, 32) + ceil_div<int64_t>(nq + window, 32) + 1;
    return some < all ? some : all;
}

template <int FMT, int NT, bool LIST, int WARPS>
static lsa_status launch_kv8_ctas(const Kv8AttnArgs& a, int n, int cluster, cudaStream_t st) {
    constexpr size_t smem = (size_t)WARPS * kKv8Warp;
    static std::atomic<uint64_t> allowed{0};
    kv8_allow_smem((const void*)kv8_split_kernel<FMT, NT, LIST, WARPS>, smem, allowed);
    {
        KTime kt_("kv8_split_kernel", st);
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(n * cluster);
        cfg.blockDim = dim3(32 * WARPS);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim = {(unsigned)cluster, 1u, 1u};
        cfg.attrs = &at;
        cfg.numAttrs = cluster > 1;
        cudaLaunchKernelEx(&cfg, kv8_split_kernel<FMT, NT, LIST, WARPS>, a, kKv8Least);
    }
    return check_launch("kv8_split_kernel");
}

template <int FMT, int NT, bool LIST>
static lsa_status launch_kv8_split(Kv8AttnArgs a, const Kv8Plan& p, int64_t n_seq, bool one_each, cudaStream_t st) {
    if (p.rows > 0) {
        a.own = LIST || one_each ? 1 : 2;
        if constexpr (NT == 1)
            if (p.rows <= num_sms()) return launch_kv8_ctas<FMT, 1, LIST, 16>(a, (int)p.rows, p.cluster, st);
        return launch_kv8_ctas<FMT, NT, LIST, kKv8Warps>(a, (int)p.rows, p.cluster, st);
    }
    const int n = kv8_ctas<NT>();
    lsa_status s;
    if ((s = launch_kv8_ctas<FMT, NT, LIST, kKv8Warps>(a, n, 1, st)) != LSA_OK) return s;
    // the join's own scan runs while the split kernel drains
    cudaLaunchConfig_t cfg{};
    // a row's pieces: about n over the rows; rows of up to 16 by whole columns
    const bool few = n_seq * a.hkv * 16 >= n;
    cfg.gridDim = dim3(n - 1, few ? 1 : LIST || one_each ? a.G : 8 * NT);
    cfg.blockDim = dim3(32 * kKv8Warps);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    {
        KTime kt_("kv8_join_kernel", st);
        cudaLaunchKernelEx(&cfg, kv8_join_kernel<NT, LIST>, a, n, kKv8Least);
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
    while ((1 << a.lgG) < a.G) ++a.lgG;
    a.O = O; a.lse = lse; a.part = (float*)ws;
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)kD);
    return a;
}

}  // namespace lsa

extern "C" {

size_t lsa_kv8_attn_workspace_bytes(const lsa_kv8* kv, int64_t nq, int32_t hq, int32_t one_each, int32_t n_seq,
                                    int32_t max_pages, int32_t sinks, int32_t window) {
    using namespace lsa;
    if (check_kv8(kv) != LSA_OK || check_heads(hq, kv->hkv) != LSA_OK || nq <= 0 || n_seq <= 0 || max_pages < 0) return 0;
    return kv8_plan(false, nq, n_seq, hq / kv->hkv, kv->hkv, one_each != 0,
                    kv8_max_chunks(nq, kv->page, max_pages, sinks, window)).ws;
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
    Kv8AttnArgs a = kv8_args(kv, Q, q_stride, nq, hq, table, lens, n_seq, max_pages, O, lse, ws);
    // a window as long as the longest sequence hides nothing
    a.cu = cu; a.W = window < (int64_t)max_pages * kv->page ? window : 0; a.S = a.W > 0 ? sinks : 0;
    const Kv8Plan p = kv8_plan(false, nq, n_seq, a.G, kv->hkv, cu == nullptr,
                               kv8_max_chunks(nq, kv->page, max_pages, sinks, window));
    if (p.ws > 0 && (!ws || ws_bytes < p.ws)) return set_error(LSA_ENOSPACE, "lsa_kv8_attn: workspace too small");
    const cudaStream_t st = (cudaStream_t)stream;
    const bool each = cu == nullptr;
    if (kv->fmt == LSA_KV8_E4M3)
        return p.nt == 1 ? launch_kv8_split<0, 1, false>(a, p, n_seq, each, st)
                         : launch_kv8_split<0, 2, false>(a, p, n_seq, each, st);
    return p.nt == 1 ? launch_kv8_split<1, 1, false>(a, p, n_seq, each, st)
                     : launch_kv8_split<1, 2, false>(a, p, n_seq, each, st);
}

size_t lsa_kv8_sparse_attn_workspace_bytes(const lsa_kv8* kv, int64_t nq, int32_t hq, int32_t n_idx) {
    using namespace lsa;
    if (check_kv8(kv) != LSA_OK || check_heads(hq, kv->hkv) != LSA_OK || nq <= 0 || n_idx < 0) return 0;
    return kv8_plan(true, nq, nq, hq / kv->hkv, kv->hkv, true, ceil_div<int64_t>(n_idx, 32)).ws;
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
    if (n_idx > INT32_MAX - 128) return set_error(LSA_EUNSUPPORTED, "lsa_kv8_sparse_attn: n_idx beyond 2^31");
    if (nq == 0) return LSA_OK;  // before seq is looked at: an empty array may have no address
    if (!seq && nq != n_seq) return set_error(LSA_EINVAL, "lsa_kv8_sparse_attn: without seq, nq must equal n_seq");
    if (!idx && n_idx > 0) return set_error(LSA_EINVAL, "lsa_kv8_sparse_attn: idx is NULL");
    Kv8AttnArgs a = kv8_args(kv, Q, q_stride, nq, hq, table, lens, n_seq, max_pages, O, lse, ws);
    a.seq = seq; a.idx = idx; a.n_idx = n_idx;
    const Kv8Plan p = kv8_plan(true, nq, nq, a.G, kv->hkv, true, ceil_div<int64_t>(n_idx, 32));
    if (p.ws > 0 && (!ws || ws_bytes < p.ws)) return set_error(LSA_ENOSPACE, "lsa_kv8_sparse_attn: workspace too small");
    const cudaStream_t st = (cudaStream_t)stream;
    if (!p.warps)
        return kv->fmt == LSA_KV8_E4M3 ? launch_kv8_split<0, 1, true>(a, p, nq, true, st)
                                       : launch_kv8_split<1, 1, true>(a, p, nq, true, st);
    {
        KTime kt_("kv8_list_kernel", st);
        const unsigned grid = (unsigned)ceil_div<int64_t>(nq * kv->hkv, kKv8ListWarps);
        auto kern = kv->fmt == LSA_KV8_E4M3 ? kv8_list_kernel<0> : kv8_list_kernel<1>;
        const int smem = kKv8ListWarps * kKv8Warp;
        static std::atomic<uint64_t> allowed[2];
        kv8_allow_smem((const void*)kern, smem, allowed[kv->fmt]);
        kern<<<grid, 32 * kKv8ListWarps, smem, st>>>(a);
    }
    return check_launch("kv8_list_kernel");
}

}  // extern "C"
