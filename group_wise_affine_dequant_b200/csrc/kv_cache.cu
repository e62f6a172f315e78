// The paged 8-bit key/value cache: writing a step's keys and values into it
// (nv_kv_quantize) and reading them back (nv_kv_dequantize).
//
// One fp32 scale per (page, head): scale = amax / 127 (int8) or amax / 448
// (E4M3) of what the block holds; a code is the representable value nearest to
// x / scale (ties to even), exactly: the quotient's rounding never decides.
// Tokens appended to a part-filled block keep its scale unless they need a
// larger one; then the codes already there are read, scaled by old / new and
// rounded again through a 256-entry table (a code has only 256 values).
//
// Write: one CTA per (block of tokens, head, K or V) holds the block's new
// values in registers (64 per thread), so they are read once: maximum, scale,
// codes. Read back: one CTA per block of tokens and head. Both are bound by
// memory: 2 bytes in and 1 out per bf16 value, and the reverse.
#include <cstdint>

#include "kv.cuh"
#include "tma.cuh"

namespace nvq {
namespace {

constexpr int kChunks = 8;  // 8-value chunks per thread
constexpr int kMaxThreads = 512;  // block 128 x D 256: 64 values per thread

struct Values8 {
    float v[8];
};

template <int DT>
__device__ __forceinline__ Values8 load8(const void* p, int64_t i) {
    Values8 r;
    if constexpr (DT == NV_F32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
        const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i) + 1);
        r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
        r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.v[2 * j] = __uint_as_float(u[j] << 16);
            r.v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
    }
    return r;
}

// The integer nearest to x / s (ties to even), |x / s| <= 127.5: a first guess
// by the reciprocal is off by at most one, and the remainder x - c s is exact
// in fp32 (both are multiples of s's unit, below 2 s), so comparing it with
// s / 2 settles the guess. Returned as magic + c, whose low byte is the code.
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
__device__ __forceinline__ uint32_t int8_code(float x, float s, float inv) {
    float t = fmaf(x, inv, kMagic);
    const float c = t - kMagic;
    const float e = fmaf(-c, s, x), half = 0.5f * s;
    if (fabsf(e) >= half) {
        const bool odd = __float_as_uint(t) & 1u;
        if (fabsf(e) > half || odd) t += copysignf(1.f, e);
    }
    t = fminf(fmaxf(t, kMagic - kInt8Max), kMagic + kInt8Max);
    return __float_as_uint(t) & 0xFFu;
}

// x / s as a float that rounds to E4M3 as the exact quotient does: only a
// quotient that landed on a 5-bit value (a tie's place) by rounding is moved
// off it, by one unit towards the exact value.
__device__ __forceinline__ float e4m3_quotient(float x, float s) {
    const float q = __fdiv_rn(x, s);
    if ((__float_as_uint(q) & 0x3FFFFu) == 0u) {
        const float r = fmaf(-q, s, x);
        if (r != 0.f && q != 0.f)
            return __uint_as_float(__float_as_uint(q) + ((r > 0.f) == (q > 0.f) ? 1u : 0xFFFFFFFFu));
    }
    return q;
}

template <int MODE>
__device__ __forceinline__ uint2 encode8(const Values8& x, float s, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (MODE == NV_KV_INT8) {
            uint32_t b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = int8_code(x.v[4 * h + j], s, inv);
            w[h] = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
        } else {
            float q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = e4m3_quotient(x.v[4 * h + j], s);
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | (hi << 16);
        }
    }
    return make_uint2(w[0], w[1]);
}

// A code of the old scale as a code of the larger new one: the nearest to the
// exact c * old / new. In fp64 the product is exact and the quotient never
// rounds onto a tie that it is not on (both scales have 24 bits).
template <int MODE>
__device__ __forceinline__ uint8_t recode(uint32_t byte, float old_scale, float new_scale) {
    const double q = static_cast<double>(code_value<MODE>(byte)) * old_scale / new_scale;
    if constexpr (MODE == NV_KV_INT8) {
        return static_cast<uint8_t>(static_cast<int8_t>(__double2int_rn(q)));
    } else {
        // to fp32 by rounding to odd, which E4M3's rounding cannot tell from the exact value
        float f = __double2float_rz(q);
        if (static_cast<double>(f) != q) f = __uint_as_float(__float_as_uint(f) | 1u);
        return static_cast<uint8_t>(__nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3));
    }
}

// Largest of one unsigned value per thread, over the CTA; every thread gets it.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* warp_max) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = blockDim.x >> 5;
    uint32_t r = 0;
    for (int i = 0; i < warps; ++i) r = max(r, warp_max[i]);
    return r;
}

struct QuantArgs {
    const void* x[2];  // k, v
    int64_t stride[2];
    KvCache c;
    KvSteps st;
};

template <int DT, int MODE>
__global__ void __launch_bounds__(kMaxThreads) kv_quantize_kernel(const __grid_constant__ QuantArgs a) {
    __shared__ uint32_t warp_max[kMaxThreads / 32];
    __shared__ uint8_t table[256];
    const KvCache& c = a.c;
    pdl_launch_dependents();
    pdl_wait();
    const int which = blockIdx.y & 1, h = blockIdx.y >> 1;
    const int s = kv_find_seq(a.st, blockIdx.x, 1, c.block, 2);
    const SeqSpan span = seq_span(a.st, s, c.block);
    const int first = span.first < 0 ? 0 : span.first;
    const int64_t j = static_cast<int64_t>(blockIdx.x) - kv_first_item(a.st, s, 1, c.block, 2);
    const int64_t b = first / c.block + j;
    if (j < 0 || span.n == 0 || b * c.block >= span.len) return;
    const int page = page_of(a.st, c, s, static_cast<int>(b));
    if (page < 0) return;
    // this block's new tokens: slots slot0 .. slot1, rows from row0 on
    const int base = static_cast<int>(b * c.block);
    const int slot0 = first > base ? first - base : 0;
    const int slot1 = span.len - base < c.block ? span.len - base : c.block;
    const int64_t row0 = span.row0 + (base + slot0 - span.first);
    const int vecs = c.D / 8;
    const int chunks = (slot1 - slot0) * vecs;
    const void* x = a.x[which];
    const int64_t stride = a.stride[which];
    uint8_t* codes = (which ? c.v_codes : c.k_codes) +
                     (static_cast<int64_t>(page) * c.H + h) * (static_cast<int64_t>(c.block) * c.D);
    float* scale_at = (which ? c.v_scales : c.k_scales) + static_cast<int64_t>(page) * c.H + h;
    const float old = slot0 > 0 ? *scale_at : 0.f;

    Values8 val[kChunks];
    uint32_t most = 0;  // largest finite magnitude, as bits; bit 31: something is not finite
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at >= chunks) break;
        const int tok = at / vecs, d = (at - tok * vecs) * 8;
        val[i] = load8<DT>(x, (row0 + tok) * stride + static_cast<int64_t>(h) * c.D + d);
    }
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        if (threadIdx.x + i * blockDim.x >= chunks) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t u = __float_as_uint(val[i].v[j]) & 0x7FFFFFFFu;
            if (u < 0x7F800000u)
                most = max(most, u);
            else
                odd = 1;
        }
    }
    most = block_max(most, warp_max);
    const bool any_odd = __syncthreads_or(odd);
    constexpr float kLargest = MODE == NV_KV_INT8 ? kInt8Max : kE4m3Max;
    const float scale = fmaxf(old, __fdiv_rn(__uint_as_float(most), kLargest));
    if (threadIdx.x == 0) *scale_at = scale;

    if (slot0 > 0 && scale > old) {  // the same for the whole CTA
        for (int i = threadIdx.x; i < 256; i += blockDim.x) table[i] = recode<MODE>(i, old, scale);
        __syncthreads();
        uint32_t* words = reinterpret_cast<uint32_t*>(codes);
        for (int i = threadIdx.x; i < slot0 * c.D / 4; i += blockDim.x) {
            const uint32_t w = words[i];
            words[i] = table[w & 255u] | (table[w >> 8 & 255u] << 8) | (table[w >> 16 & 255u] << 16) |
                       (static_cast<uint32_t>(table[w >> 24]) << 24);
        }
    }

    // a tiny scale's reciprocal or remainders would leave the normal range: move both by 2^64, exactly
    const float lift = scale < 8.6736174e-19f ? 18446744073709551616.f : 1.f;  // 2^-60, 2^64
    const float s2 = scale * lift, inv = scale > 0.f ? 1.f / s2 : 0.f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at >= chunks) break;
        uint2 w = make_uint2(0u, 0u);
        if (scale > 0.f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float f = val[i].v[j];
                if (any_odd) {  // NaN is kept as 0, an infinity as the largest code
                    f = f == f ? f : 0.f;
                    f = fminf(fmaxf(f, -kLargest * scale), kLargest * scale);
                }
                val[i].v[j] = f * lift;
            }
            w = encode8<MODE>(val[i], s2, inv);
        }
        const int tok = at / vecs, d = (at - tok * vecs) * 8;
        *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(slot0 + tok) * c.D + d) = w;
    }
}

struct DequantArgs {
    void* out[2];  // k, v [rows, H, D]
    KvCache c;
    KvSteps st;
};

template <int DT, int MODE>
__global__ void __launch_bounds__(256) kv_dequantize_kernel(const __grid_constant__ DequantArgs a) {
    const KvCache& c = a.c;
    pdl_launch_dependents();
    pdl_wait();
    const int which = blockIdx.y & 1, h = blockIdx.y >> 1;
    const int s = kv_find_seq(a.st, blockIdx.x, 1, c.block, 2);
    const SeqSpan span = seq_span(a.st, s, c.block);
    // rows in front of the sequence's first token (a bad descriptor) read as zeros, with its first block
    const int first = span.first < 0 ? 0 : span.first;
    const int64_t j = static_cast<int64_t>(blockIdx.x) - kv_first_item(a.st, s, 1, c.block, 2);
    const int64_t b = first / c.block + j;
    if (j < 0) return;
    const int vecs = c.D / 16;
    auto store = [&](int64_t row, int d, const float* f) {
        const int64_t at = (row * c.H + h) * c.D + d;
        if constexpr (DT == NV_F32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out[which]) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        } else {
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[which]) + at);
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
            o[0] = make_uint4(w[0], w[1], w[2], w[3]);
            o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    };
    float f[16];
    if (j == 0 && span.first < 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 0.f;
        const int64_t missing = span.n < -span.first ? span.n : -span.first;
        for (int64_t i = threadIdx.x; i < missing * vecs; i += blockDim.x)
            store(span.row0 + i / vecs, static_cast<int>(i % vecs) * 16, f);
    }
    if (span.n == 0 || b * c.block >= span.len) return;
    const int page = page_of(a.st, c, s, static_cast<int>(b));
    const int base = static_cast<int>(b * c.block);
    const int slot0 = first > base ? first - base : 0;
    const int slot1 = span.len - base < c.block ? span.len - base : c.block;
    const int64_t row0 = span.row0 + (base + slot0 - span.first);
    const int chunks = (slot1 - slot0) * vecs;
    const int64_t block_at = page < 0 ? 0 : static_cast<int64_t>(page) * c.H + h;
    const uint8_t* codes = (which ? c.v_codes : c.k_codes) + block_at * (static_cast<int64_t>(c.block) * c.D);
    const float scale = page < 0 ? 0.f : __ldg((which ? c.v_scales : c.k_scales) + block_at);
    for (int i = threadIdx.x; i < chunks; i += blockDim.x) {
        const int tok = i / vecs, d = (i - tok * vecs) * 16;
        if (page < 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = 0.f;
        } else {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(codes + static_cast<int64_t>(slot0 + tok) * c.D + d));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = code_value<MODE>(u[e / 4] >> (8 * (e & 3)) & 255u) * scale;
        }
        store(row0 + tok, d, f);
    }
}

template <typename... Args>
cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t stream, Args... args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_kv_quantize(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int dt,
                               const KvCache& c, const KvSteps& st, cudaStream_t stream) {
    QuantArgs a{{k, v}, {k_stride, v_stride}, c, st};
    const int threads = (c.block * c.D / 64 + 31) / 32 * 32;
    const dim3 grid(static_cast<unsigned>(kv_items(st.rows, st.S, 1, c.block, 2)), 2 * c.H, 1);
    if (dt == NV_F32)
        return c.mode == NV_KV_INT8 ? launch_pdl(kv_quantize_kernel<NV_F32, NV_KV_INT8>, grid, threads, stream, a)
                                    : launch_pdl(kv_quantize_kernel<NV_F32, NV_KV_E4M3>, grid, threads, stream, a);
    return c.mode == NV_KV_INT8 ? launch_pdl(kv_quantize_kernel<NV_BF16, NV_KV_INT8>, grid, threads, stream, a)
                                : launch_pdl(kv_quantize_kernel<NV_BF16, NV_KV_E4M3>, grid, threads, stream, a);
}

cudaError_t launch_kv_dequantize(void* k, void* v, int dt, const KvCache& c, const KvSteps& st,
                                 cudaStream_t stream) {
    DequantArgs a{{k, v}, c, st};
    int threads = (c.block * c.D / 16 + 31) / 32 * 32;
    threads = threads < 256 ? threads : 256;
    const dim3 grid(static_cast<unsigned>(kv_items(st.rows, st.S, 1, c.block, 2)), 2 * c.H, 1);
    if (dt == NV_F32)
        return c.mode == NV_KV_INT8 ? launch_pdl(kv_dequantize_kernel<NV_F32, NV_KV_INT8>, grid, threads, stream, a)
                                    : launch_pdl(kv_dequantize_kernel<NV_F32, NV_KV_E4M3>, grid, threads, stream, a);
    return c.mode == NV_KV_INT8 ? launch_pdl(kv_dequantize_kernel<NV_BF16, NV_KV_INT8>, grid, threads, stream, a)
                                : launch_pdl(kv_dequantize_kernel<NV_BF16, NV_KV_E4M3>, grid, threads, stream, a);
}

}  // namespace nvq
