// attn_cache_append.cuh -- rotate a step's queries and keys by their positions
// and write its keys and values into the pages of the cache.
//
// Each pair (x, y) of a rotated row at position p turns by the angle p f:
//     (x cos pf - y sin pf,  y cos pf + x sin pf).
// The angle is taken in FP64 as a number of turns, p f / 2 pi, of which only
// the fraction goes on (in FP32), so far positions keep their phase.
//
// E4M3 pages: every (page, head) has the scale 2^e, the smallest power of two
// with bound <= 448 * 2^e.  The bound of a rotated pair is |x| + |y|, which no
// rotation of it exceeds: the scale depends on the BF16 inputs alone.  A power
// of two costs a floating-point format no precision, and coding a page again
// under a larger one only shifts exponents.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "attn_common.cuh"

namespace sdpa10 {
namespace cache {

struct AppendParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    __nv_bfloat16* q_out;
    uint8_t* k_pages;
    uint8_t* v_pages;
    float* k_scale;
    float* v_scale;
    const int* table;
    const int* seqlens;
    const int* cu;  // null: n_uniform rows each
    const float* inv_freq;
    long long q_stride, k_stride, v_stride;
    long long page_stride, token_stride, head_stride;
    int batch, max_pages, total, max_seqlen, n_uniform;
    int h_q, h_kv, num_pages, page_size;
    int rotary_dim, interleaved;
    int page_blocks;      // CTAs of the page role (E4M3), before those of the row role
    int pages_per_seq;    // pages that max_seqlen rows can enter
    int row_heads;        // heads in the row role: h_q (E4M3) or h_q + 2 h_kv (BF16)
    int heads_per_unit;   // of which one group of 8 lanes takes this many
};

// Eight lanes hold a row of 128 elements: two vectors of eight each, so that
// the partner of every rotated element is in the same lane.
struct RowLane {
    int va, vb;  // the lane's two vectors (16 bytes of BF16 each)
    int f0;      // first of its eight frequencies; -1: its elements pass
};

__device__ __forceinline__ RowLane row_lane(int u, int rotary_dim, int interleaved) {
    RowLane r;
    const int turned = rotary_dim >> 4;  // lanes that rotate
    r.f0 = u < turned ? 8 * u : -1;
    if (interleaved || u >= turned) {
        r.va = 2 * u;
        r.vb = 2 * u + 1;
    } else {
        r.va = u;
        r.vb = u + turned;
    }
    return r;
}

__device__ __forceinline__ void row_angles(const AppendParams& p, const RowLane& rl, int pos,
                                           float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
        if (rl.f0 >= 0) {
            constexpr double kInv2Pi = 0.15915494309189533577;
            const double turns =
                static_cast<double>(pos) * static_cast<double>(p.inv_freq[rl.f0 + e]) * kInv2Pi;
            sincospif(2.f * static_cast<float>(turns - rint(turns)), &s[e], &c[e]);
        }
    }
}

__device__ __forceinline__ void unpack8(const uint4 w, float (&x)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                      ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float inv) {
    return make_uint2(ptx::pack_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                      ptx::pack_e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// Rotate a lane's two vectors in place.
__device__ __forceinline__ void rotate(const RowLane& rl, int interleaved, const float (&c)[8],
                                       const float (&s)[8], float (&a)[8], float (&b)[8]) {
    if (rl.f0 < 0) return;
    if (!interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = a[e], y = b[e];
            a[e] = x * c[e] - y * s[e];
            b[e] = y * c[e] + x * s[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = a[2 * e], y = a[2 * e + 1];
            a[2 * e] = x * c[e] - y * s[e];
            a[2 * e + 1] = y * c[e] + x * s[e];
            const float z = b[2 * e], w = b[2 * e + 1];
            b[2 * e] = z * c[4 + e] - w * s[4 + e];
            b[2 * e + 1] = w * c[4 + e] + z * s[4 + e];
        }
    }
}

// Largest |x| of a lane's elements, or |x| + |y| of its pairs where it rotates.
__device__ __forceinline__ float row_bound(const RowLane& rl, int interleaved, const float (&a)[8],
                                           const float (&b)[8], bool pairs) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float x = fabsf(a[e]), y = fabsf(b[e]);
        if (pairs && rl.f0 >= 0) {
            if (!interleaved) {
                x += y;
            } else if ((e & 1) == 0) {
                x += fabsf(a[e + 1]);
                y += fabsf(b[e + 1]);
            } else {
                x = y = 0.f;
            }
        }
        m = fmaxf(m, fmaxf(x, y));
    }
    return m;
}

// The smallest power of two s with bound <= 448 s (0 for 0), from the bits:
// bound = m 2^E with 1 <= m < 2 and 448 = 1.75 * 2^8.  Kept to the normal
// range (a subnormal bound gives 2^-126, an infinite one 2^119).
__device__ __forceinline__ float pow2_scale(float bound) {
    if (!(bound > 0.f)) return 0.f;
    const uint32_t bits = __float_as_uint(bound);
    int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, -126), 119);
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// 1 / scale (exact for the powers of two that this file writes); a page of
// zeros has scale 0.
__device__ __forceinline__ float scale_inverse(float s) { return s > 0.f ? 1.f / s : 0.f; }

// Four E4M3 codes as numbers.
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float (&x)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[0] = f0.x;
    x[1] = f0.y;
    x[2] = f1.x;
    x[3] = f1.y;
}

// A sequence's rows and positions.
struct SeqRows {
    int row0, n, len;
};
__device__ __forceinline__ SeqRows seq_rows(const AppendParams& p, int b) {
    SeqRows s;
    if (p.cu != nullptr) {
        const int r0 = p.cu[b], r1 = p.cu[b + 1];
        s.row0 = min(max(r0, 0), p.total);
        s.n = min(max(r1, s.row0), p.total) - s.row0;
    } else {
        s.row0 = b * p.n_uniform;
        s.n = p.n_uniform;
    }
    s.len = p.seqlens[b];
    return s;
}

// ------------------------------------------------------------------ pages
// One CTA per (sequence, page that its new rows enter, head): the bounds of
// the page's new rows, the scales, the older tokens if a scale grew, then the
// rows themselves.  The rows are read twice, the second time from L2.
__device__ __forceinline__ void append_page(const AppendParams& p, int block) {
    const int h = block % p.h_kv;
    const int bj = block / p.h_kv;
    const int b = bj / p.pages_per_seq;
    const SeqRows s = seq_rows(p, b);
    const int n = min(s.n, p.max_seqlen);
    const long long cap = static_cast<long long>(p.max_pages) * p.page_size;
    // Positions of this call's rows in the cache: [lo, hi).
    const long long first = static_cast<long long>(s.len) - s.n;
    long long lo = first < 0 ? 0 : first;
    long long hi = first + n < cap ? first + n : cap;
    if (hi <= lo) return;
    const long long page = lo / p.page_size + bj % p.pages_per_seq;
    const long long page0 = page * p.page_size;
    if (page0 >= hi) return;
    lo = lo > page0 ? lo : page0;
    hi = hi < page0 + p.page_size ? hi : page0 + p.page_size;
    const int pid = p.table[static_cast<long long>(b) * p.max_pages + page];
    if (pid < 0 || pid >= p.num_pages) return;

    const int slots = blockDim.x >> 3, slot = threadIdx.x >> 3;
    const RowLane rl = row_lane(threadIdx.x & 7, p.rotary_dim, p.interleaved);
    const int rows = static_cast<int>(hi - lo), begin = static_cast<int>(lo - page0);
    const int row0 = s.row0 + static_cast<int>(lo - first);
    const __nv_bfloat16* k = p.k + static_cast<long long>(row0) * p.k_stride + h * kHeadDim;
    const __nv_bfloat16* v = p.v + static_cast<long long>(row0) * p.v_stride + h * kHeadDim;

    float kb = 0.f, vb = 0.f;
    for (int r = slot; r < rows; r += slots) {
        float a[8], c[8];
        const uint4* kr = reinterpret_cast<const uint4*>(k + r * p.k_stride);
        const uint4* vr = reinterpret_cast<const uint4*>(v + r * p.v_stride);
        const uint4 k0 = kr[rl.va], k1 = kr[rl.vb], v0 = vr[rl.va], v1 = vr[rl.vb];
        unpack8(k0, a);
        unpack8(k1, c);
        kb = fmaxf(kb, row_bound(rl, p.interleaved, a, c, true));
        unpack8(v0, a);
        unpack8(v1, c);
        vb = fmaxf(vb, row_bound(rl, p.interleaved, a, c, false));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        kb = fmaxf(kb, __shfl_xor_sync(0xffffffffu, kb, o));
        vb = fmaxf(vb, __shfl_xor_sync(0xffffffffu, vb, o));
    }
    __shared__ float red[2][8];
    if ((threadIdx.x & 31) == 0) {
        red[0][threadIdx.x >> 5] = kb;
        red[1][threadIdx.x >> 5] = vb;
    }
    const long long si = static_cast<long long>(pid) * p.h_kv + h;
    const float k_old = begin > 0 ? p.k_scale[si] : 0.f;
    const float v_old = begin > 0 ? p.v_scale[si] : 0.f;
    __syncthreads();
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
        kb = fmaxf(kb, red[0][w]);
        vb = fmaxf(vb, red[1][w]);
    }
    const float k_new = fmaxf(k_old, pow2_scale(kb)), v_new = fmaxf(v_old, pow2_scale(vb));
    if (threadIdx.x == 0) {
        p.k_scale[si] = k_new;
        p.v_scale[si] = v_new;
    }
    const long long base = pid * p.page_stride + h * p.head_stride;
    // Older tokens under a scale that grew: 16 codes at a time.
    auto recode = [&](uint8_t* pages, float factor) {
        for (int i = threadIdx.x; i < begin * 8; i += blockDim.x) {
            uint4* at = reinterpret_cast<uint4*>(pages + base + (i >> 3) * p.token_stride) + (i & 7);
            uint4 w = *at;
            uint32_t* c = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x[4];
                e4m3x4_to_float(c[j], x);
                c[j] = ptx::pack_e4m3x4(x[0] * factor, x[1] * factor, x[2] * factor, x[3] * factor);
            }
            *at = w;
        }
    };
    if (k_old > 0.f && k_new > k_old) recode(p.k_pages, k_old * scale_inverse(k_new));
    if (v_old > 0.f && v_new > v_old) recode(p.v_pages, v_old * scale_inverse(v_new));

    const float k_inv = scale_inverse(k_new), v_inv = scale_inverse(v_new);
    for (int r = slot; r < rows; r += slots) {
        float a[8], c[8], co[8], sn[8];
        const uint4* kr = reinterpret_cast<const uint4*>(k + r * p.k_stride);
        const uint4* vr = reinterpret_cast<const uint4*>(v + r * p.v_stride);
        const uint4 k0 = kr[rl.va], k1 = kr[rl.vb], v0 = vr[rl.va], v1 = vr[rl.vb];
        row_angles(p, rl, static_cast<int>(lo) + r, co, sn);
        const long long at = base + (begin + r) * p.token_stride;
        unpack8(k0, a);
        unpack8(k1, c);
        rotate(rl, p.interleaved, co, sn, a, c);
        reinterpret_cast<uint2*>(p.k_pages + at)[rl.va] = pack8_e4m3(a, k_inv);
        reinterpret_cast<uint2*>(p.k_pages + at)[rl.vb] = pack8_e4m3(c, k_inv);
        unpack8(v0, a);
        unpack8(v1, c);
        reinterpret_cast<uint2*>(p.v_pages + at)[rl.va] = pack8_e4m3(a, v_inv);
        reinterpret_cast<uint2*>(p.v_pages + at)[rl.vb] = pack8_e4m3(c, v_inv);
    }
}

// ------------------------------------------------------------------ rows
// Eight lanes take one token and heads_per_unit of its heads: queries, and for
// BF16 pages keys and values.  The angles are computed once for all of them.
__device__ __forceinline__ void append_rows(const AppendParams& p, int block) {
    const int groups = (p.row_heads + p.heads_per_unit - 1) / p.heads_per_unit;
    const long long unit = static_cast<long long>(block) * (blockDim.x >> 3) + (threadIdx.x >> 3);
    const long long tok = unit / groups;
    if (tok >= p.total) return;
    const int t = static_cast<int>(tok), g = static_cast<int>(unit % groups);
    int b;
    if (p.cu != nullptr) {
        int lo = 0, hi = p.batch;  // the last sequence that starts at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.cu[mid] <= t) lo = mid; else hi = mid;
        }
        b = lo;
    } else {
        b = t / p.n_uniform;
    }
    const SeqRows s = seq_rows(p, b);
    const int i = t - s.row0;
    if (i < 0 || i >= min(s.n, p.max_seqlen)) return;  // padding
    const int pos = s.len - s.n + i;
    const RowLane rl = row_lane(threadIdx.x & 7, p.rotary_dim, p.interleaved);
    float co[8], sn[8];
    row_angles(p, rl, pos, co, sn);

    const int h1 = min(p.row_heads, (g + 1) * p.heads_per_unit);
    // Where this token's keys and values go (BF16 pages).
    long long at = -1;
    if (h1 > p.h_q && pos >= 0 && pos / p.page_size < p.max_pages) {
        const int pid = p.table[static_cast<long long>(b) * p.max_pages + pos / p.page_size];
        if (pid >= 0 && pid < p.num_pages)
            at = pid * p.page_stride + (pos % p.page_size) * p.token_stride;
    }
#pragma unroll 4
    for (int r = g * p.heads_per_unit; r < h1; ++r) {
        const __nv_bfloat16* src;
        __nv_bfloat16* dst;
        bool turn = true;
        if (r < p.h_q) {
            src = p.q + t * p.q_stride + r * kHeadDim;
            dst = p.q_out + (static_cast<long long>(t) * p.h_q + r) * kHeadDim;
        } else {
            if (at < 0) break;  // the remaining heads are keys and values
            int h = r - p.h_q;
            turn = h < p.h_kv;
            if (!turn) h -= p.h_kv;
            src = turn ? p.k + t * p.k_stride + h * kHeadDim : p.v + t * p.v_stride + h * kHeadDim;
            dst = reinterpret_cast<__nv_bfloat16*>(turn ? p.k_pages : p.v_pages) + at +
                  h * p.head_stride;
        }
        uint4 w0 = reinterpret_cast<const uint4*>(src)[rl.va];
        uint4 w1 = reinterpret_cast<const uint4*>(src)[rl.vb];
        if (turn && rl.f0 >= 0) {
            float a[8], c[8];
            unpack8(w0, a);
            unpack8(w1, c);
            rotate(rl, p.interleaved, co, sn, a, c);
            w0 = pack8(a);
            w1 = pack8(c);
        }
        reinterpret_cast<uint4*>(dst)[rl.va] = w0;
        reinterpret_cast<uint4*>(dst)[rl.vb] = w1;
    }
}

__global__ void __launch_bounds__(256) attn_cache_append_kernel(const __grid_constant__ AppendParams p) {
    if (static_cast<int>(blockIdx.x) < p.page_blocks)
        append_page(p, blockIdx.x);
    else
        append_rows(p, blockIdx.x - p.page_blocks);
}

}  // namespace cache
}  // namespace sdpa10
